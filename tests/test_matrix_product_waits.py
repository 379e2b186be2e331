"""CPU test of the built language-model library: results of matrix products are waited for along every path.

The hardware does not hold back an instruction that reads the result of a matrix product which is still under way; the compiler
puts wait states in between.  Where blocks of code join it has been seen to count along one of the paths only.  Here they are
counted along all of them, in the machine code of every kernel with such products."""
import collections
import os
import re
import shutil
import subprocess

import pytest

import selective_state_space_51_amd as S

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", "/opt/rocm/lib/llvm/bin/llvm-objdump") if os.path.exists(p)), None)
# wait states between a product and another instruction's use of its result
NEED = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}
STORES = ("ds_write", "buffer_store", "global_store", "flat_store", "scratch_store")
FAR = 24  # beyond every product's


def registers(operand):
    m = re.match(r"^-?\|?([av])(?:(\d+)|\[(\d+):(\d+)\])", operand)
    if not m:
        return []
    lo, hi = (m.group(2), m.group(2)) if m.group(2) else (m.group(3), m.group(4))
    return [m.group(1) + str(i) for i in range(int(lo), int(hi) + 1)]


def kernels(text):
    """{name: [(offset, op, operands, target of a branch)]} of a disassembly."""
    out, ins, start = {}, None, 0
    for line in text.split("\n"):
        m = re.match(r"^([0-9a-f]+) <(\w+)>:", line)
        if m:
            start, ins = int(m.group(1), 16), []
            out[m.group(2)] = ins
            continue
        m = re.match(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)", line)
        if ins is None or not m:
            continue
        to = re.search(r"<\w+(?:\+0x([0-9a-f]+))?>", m.group(4)) if "branch" in m.group(1) else None
        ops = [o.strip().split()[0] for o in m.group(2).split(",") if o.strip()]
        ins.append((int(m.group(3), 16) - start, m.group(1), ops, None if to is None else int(to.group(1) or "0", 16)))
    return out


def fewest_waits(ins):
    """{product: (wait states, offset) of the use of a result that follows it most closely on any path}"""
    at = {x[0]: i for i, x in enumerate(ins)}
    starts = {0}
    for i, (_, op, _, to) in enumerate(ins):
        if to is not None:
            starts.add(at[to])
        if ("branch" in op or op == "s_endpgm") and i + 1 < len(ins):
            starts.add(i + 1)
    order = sorted(starts)
    ends = dict(zip(order, order[1:] + [len(ins)]))
    fewest = {}

    def walk(s, state, seen):
        state = dict(state)  # register -> (wait states since its product, product)
        for i in range(s, ends[s]):
            offset, op, ops, _ = ins[i]
            vector = op.startswith(("v_", "ds_", "buffer_", "global_", "flat_", "scratch_"))
            product = op.startswith("v_mfma")
            used = ops[1:3] if product else ops  # (a sum goes into the next product of its kind without a wait)
            if vector:
                for r in (r for o in used for r in registers(o) if r in state):
                    n, p = state[r]
                    if seen is not None and n < seen.get(p, (FAR,))[0]:
                        seen[p] = (n, offset)
                if not product and not op.startswith(STORES + ("v_cmp",)):
                    for r in registers(ops[0]) if ops else ():
                        state.pop(r, None)
            step = int(ops[0], 0) + 1 if op == "s_nop" else 1
            state = {r: (n + step, p) for r, (n, p) in state.items() if n + step < FAR}
            if product:
                state.update((r, (0, op)) for r in registers(ops[0]))
        return state

    into = {order[0]: {}}
    todo = collections.deque(order[:1])
    while todo:
        s = todo.popleft()
        state = walk(s, into[s], None)
        _, op, _, to = ins[ends[s] - 1]
        after = [] if op in ("s_endpgm", "s_branch") or ends[s] == len(ins) else [ends[s]]
        for n in after + ([] if to is None else [at[to]]):
            old = into.get(n)
            new = dict(old or {})
            for r, v in state.items():
                if r not in new or v[0] < new[r][0]:
                    new[r] = v
            if old is None or new != old:
                into[n] = new
                todo.append(n)
    for s, state in into.items():
        walk(s, state, fewest)
    return fewest


def test_the_count_itself():
    text = """
0000000000001000 <k>:
	v_mfma_f32_16x16x4_f32 v[0:3], v4, v5, 0                   // 000000001000: 0
	s_cbranch_scc0 2                                           // 000000001008: 0 <k+0x14>
	s_nop 9                                                    // 00000000100C: 0
	s_nop 0                                                    // 000000001010: 0
	v_add_f32_e32 v9, v2, v9                                   // 000000001014: 0
	v_add_f32_e32 v1, v9, v9                                   // 000000001018: 0
	s_endpgm                                                   // 00000000101C: 0
"""
    assert fewest_waits(kernels(text)["k"]) == {"v_mfma_f32_16x16x4_f32": (1, 0x14)}
    assert fewest_waits(kernels(text.replace("k+0x14", "k+0xc"))["k"]) == {"v_mfma_f32_16x16x4_f32": (12, 0x14)}


@pytest.mark.skipif(OBJDUMP is None, reason="no disassembler")
def test_results_of_matrix_products_are_waited_for(tmp_path):
    shutil.copy(S.LM_LIB_PATH, tmp_path / "lm.so")
    subprocess.run([OBJDUMP, "--offloading", "lm.so"], cwd=tmp_path, check=True, capture_output=True)
    looked = 0
    for f in sorted(os.listdir(tmp_path)):
        if "gfx950" not in f:
            continue
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", f], cwd=tmp_path, check=True, capture_output=True, text=True).stdout
        for name, ins in kernels(text).items():
            if not any(x[1].startswith("v_mfma") for x in ins):
                continue
            looked += 1
            for product, (n, offset) in fewest_waits(ins).items():
                assert n >= NEED[product], (name, product, n, hex(offset))
    assert looked >= 32

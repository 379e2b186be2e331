"""GPU tests of the operators of generation together (prompts read by convolution and linear attention, cache entries forked,
tokens drawn, single tokens), on streams named by raw handles, captured into graphs, and past 32-bit offsets.  Bars as in the
operators' own tests."""
import math
import sys

import numpy as np
import pytest

from tests import test_gpu_lm_linattn as LA
from tests import test_gpu_lm_sample as SA

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


class Mixer:
    """Tokens -> v through a convolution, and linear attention with q, k and decays looked up: fp32, seeded."""

    def __init__(self, vocab=97, heads=4, groups=2, dk=32, dv=16, nslots=9):
        import torch
        g = torch.Generator(device="cuda").manual_seed(11)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.q, self.k, self.x, self.w = rn(vocab, groups, dk), rn(vocab, groups, dk), rn(vocab, heads * dv), rn(heads * dv, 4)
        self.g = -torch.rand(vocab, heads, generator=g, device="cuda")
        self.out = rn(heads * dv, vocab) / 8
        self.heads, self.dv = heads, dv
        self.conv, self.state = torch.full((nslots, 3, heads * dv), 7.0, device="cuda"), torch.full((nslots, heads, dk, dv), 7.0, device="cuda")

    def prompt(self, tokens, cu, slots, carry=None):
        import selective_state_space_51_amd as S
        v = S.causal_conv1d_packed_fwd(self.x[tokens], self.w, cu, self.conv, slots=slots, carry=carry).unflatten(1, (self.heads, self.dv))
        return v, S.linear_attn_packed_fwd(self.q[tokens], self.k[tokens], v, self.g[tokens], cu, self.state, slots=slots, carry=carry)

    def step(self, tokens, slots):
        import selective_state_space_51_amd as S
        v = S.causal_conv1d_step(self.x[tokens], self.w, self.conv, slots=slots).unflatten(1, (self.heads, self.dv))
        return v, S.linear_attn_step(self.q[tokens], self.k[tokens], v, self.g[tokens], self.state, slots=slots)


def test_forked_continuations():
    """Two prompts, each forked into continuations that draw their own tokens; one is moved and its entry freed on the way."""
    import torch

    import selective_state_space_51_amd as S
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    m = Mixer()
    prompts = [list(range(1, 41)), [5, 96, 2]]
    v, out = m.prompt(torch.tensor(sum(prompts, []), device="cuda"), i32(0, 40, 43), i32(6, 0))
    rows = [(39, 6), (39, 1), (39, 2), (42, 0), (42, 8)]  # (last token's row, entry) of each continuation
    S.cache_entries_copy([m.conv, m.state], i32(6, 6, 0), i32(1, 2, 8))
    seqs = [list(prompts[0]) for _ in range(3)] + [list(prompts[1]) for _ in range(2)]
    vs = [[v[:40]] for _ in range(3)] + [[v[40:43]] for _ in range(2)]
    outs = [[out[:40]] for _ in range(3)] + [[out[40:43]] for _ in range(2)]
    o, slots = out[[r for r, _ in rows]], i32(*(s for _, s in rows))
    for n in range(6):
        logits = o.flatten(1) @ m.out
        u = torch.rand(5, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
        tok, lp, kept = SA.check(logits, u, 0.9, 20, 0.95, 0.01)
        if n == 3:  # the last continuation moves to entry 3, the entry is freed
            S.cache_entries_copy([m.conv, m.state], i32(8, -1), i32(3, 8))
            slots = i32(6, 1, 2, 0, 3)
        vn, o = m.step(tok, slots)
        for r in range(5):
            seqs[r].append(int(tok[r])), vs[r].append(vn[r:r + 1]), outs[r].append(o[r:r + 1])
    torch.cuda.synchronize()
    assert not m.conv[8].any() and not m.state[8].any()
    assert bool((m.state[[4, 5, 7]] == 7).all()) and bool((m.conv[[4, 5, 7]] == 7).all())
    for r, s in enumerate(slots.tolist()):
        t = torch.tensor(seqs[r], device="cuda")
        i = dict(lens=[len(t)], q=m.q[t], k=m.k[t], v=torch.cat(vs[r]), g=m.g[t], state=torch.zeros_like(m.state[:1]))
        whole = S.causal_conv1d_packed_fwd(m.x[t], m.w, i32(0, len(t))).view_as(i["v"])
        assert float((whole - i["v"]).abs().max()) <= 2.0 ** -20 * float(whole.abs().max())  # five terms, rounded to 24 bits
        LA.compare(i, torch.cat(outs[r]), m.state[s:s + 1], LA.reference(i))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_prompts_go_on_from_the_cache_they_write(dtype):
    """Prompts in segments whose first reads the entry that the last, of few tokens, writes."""
    import selective_state_space_51_amd as S
    lens = [1537, 1601, 1540, 3]
    _say("go on", lens, dtype)
    i = LA.make(lens, 8, 1, 64, 64, dtype, seed=9)
    assert S.linear_attn_packed_workspace_bytes(sum(lens), 4, max(lens), 8, 64, 64, 1 if dtype == "bf16" else 0) > 0
    carry, slots = [1, 0, 1, 1], [2, 3, 0, 1]
    out, st = LA.run(i, slots, carry)
    LA.compare(i, out, st, LA.reference(i, slots, carry))


def test_many_steps_of_a_slow_decay():
    """8,192 tokens, one after another, under decays whose power is next to 1.  A sum is rounded twice per token (24 bits), each
    as likely up as down: a walk of 2 n roundings of at most half a step, 2^-24 of the largest state each, whose spread is below
    sqrt(2 n) 2^-24; 8 of those.  (A power rounded to 24 bits is off in one direction, which adds up to as much as n 2^-25.)"""
    import torch

    import selective_state_space_51_amd as S
    n, H = 8192, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    decay = -torch.rand(H, generator=g, device="cuda") * 1e-5
    k, v = torch.rand(n, 1, 1, 16, generator=g, device="cuda"), torch.rand(n, 1, H, 16, generator=g, device="cuda")
    st = torch.ones(1, H, 16, 16, device="cuda") * 100
    want, e = st.double(), decay.double().exp()[None, :, None, None]
    for t in range(n):
        S.linear_attn_step(k[t], k[t], v[t], decay, st)
        want = e * want + k[t].double()[..., None] * v[t].double()[:, :, None]
    err = (st.double() - want).abs() / want.abs()
    assert float(err.max()) <= 8 * math.sqrt(2 * n) * 2.0 ** -24


@pytest.mark.parametrize("which", ["default", "side"])
def test_work_is_ordered_on_the_stream_of_a_raw_handle(which):
    import torch

    import selective_state_space_51_amd as S
    _say("raw handle", which)
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    named = torch.cuda.default_stream() if which == "default" else torch.cuda.Stream()
    handle = named.cuda_stream
    L, H, d = 900, 2, 16
    new, cu = rn(L, H * d), torch.tensor([0, 25, L], dtype=torch.int32, device="cuda")
    gd, u = -torch.rand(L, H, device="cuda"), torch.rand(L, device="cuda")
    src, dst = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([1, 0, 5], [0, 1, 7]))
    heads = lambda x: x.unflatten(1, (H, d))

    def move(x, **k):
        S.cache_entries_copy(x, src, dst, **k)
        return x
    ops = {
        "prompt": lambda x, **k: S.linear_attn_packed_fwd(heads(x), heads(x), heads(x), gd, cu, **k),
        "sample": lambda x, **k: S.token_sample(x, u, 0.7, 20, 0.9, 0.01, **k)[1],
        "move": move,
    }
    for name, op in ops.items():
        want = op(new.clone())
        x = torch.full_like(new, 7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(named):
            torch.cuda._sleep(20_000_000)  # some ms of device clocks
            x.copy_(new)
        with torch.cuda.stream(torch.cuda.Stream()):
            got = op(x, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got, want), name
    st = [torch.zeros(L, H, d, d, device="cuda") for _ in range(2)]
    want = S.linear_attn_step(heads(new), heads(new), heads(new), gd, st[0])
    x = torch.full_like(new, 7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(named):
        torch.cuda._sleep(20_000_000)
        x.copy_(new)
    with torch.cuda.stream(torch.cuda.Stream()):
        got = S.linear_attn_step(heads(x), heads(x), heads(x), gd, st[1], stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(*st)


def test_operands_on_another_device_are_refused():
    import torch

    import selective_state_space_51_amd as S
    f = dict(device="cuda")

    class Far(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError(f"{func} on a tensor without memory")

    def far(t):
        return torch.Tensor._make_wrapper_subclass(Far, t.shape, dtype=t.dtype, device="cuda:1")

    n = 3
    q, v, g, st = torch.zeros(n, 1, 8, **f), torch.zeros(n, 2, 8, **f), torch.zeros(n, 2, **f), torch.zeros(n, 2, 8, 8, **f)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, **f)
    x, vec = torch.zeros(n, 50, **f), torch.zeros(n, **f)
    calls = [
        (S.linear_attn_packed_fwd, dict(q=q, k=q.clone(), v=v, log_decay=g, cu_seqlens=i32(0, n), state=st, slots=i32(0),
                                        carry=torch.zeros(1, dtype=torch.uint8, **f), out=v.clone())),
        (S.linear_attn_step, dict(q=q, k=q.clone(), v=v, log_decay=g, state=st, slots=i32(0, 1, 2), out=v.clone())),
        (S.token_sample, dict(logits=x, uniform=vec, temperature=vec.clone(), top_k=i32(1, 2, 3), top_p=vec.clone(), min_p=vec.clone())),
    ]
    for fn, kw in calls:
        first = next(iter(kw))
        for name in [k for k, t in kw.items() if isinstance(t, torch.Tensor) and k != first]:
            with pytest.raises(ValueError, match=f"{name} is on cuda:1, the first argument is on cuda:0"):
                fn(**{**kw, name: far(kw[name])})
        fn(**kw)
    for kw in (dict(src=far(i32(0)), dst=i32(1)), dict(src=i32(0), dst=far(i32(1)))):
        with pytest.raises(ValueError, match="is on cuda:1, the first argument is on cuda:0"):
            S.cache_entries_copy(st, **kw)
    with pytest.raises(ValueError, match="a cache is on cuda:1"):
        S.cache_entries_copy([st, far(vec)], i32(0), i32(1))
    torch.cuda.synchronize()


def test_graphs_of_a_token_and_of_prompts():
    """A token's work and two prompts of several segments that share a workspace, each in a graph of its own, replayed in turn with
    eager work between: every replay gives what the eager calls give from the same state."""
    import torch

    import selective_state_space_51_amd as S
    m = Mixer(heads=8, groups=1, dk=64, dv=64)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    tokens, u, slots = torch.randint(0, 97, (4,), generator=gen, device="cuda"), torch.rand(4, generator=gen, device="cuda"), i32(0, 3, 1, 8)
    src, dst = i32(0, 3), i32(5, 6)

    def token():
        _, o = m.step(tokens, slots)
        t = S.token_sample((o.flatten(1) @ m.out), u, 0.8, 30, 0.9)
        S.cache_entries_copy([m.conv, m.state], src, dst)
        return (o, *t)

    p = [LA.make([1500, 20], 8, 1, 64, 64, "bf16", seed=1), LA.make([9, 2000], 8, 1, 64, 64, "f32", seed=2)]
    need = max(S.linear_attn_packed_workspace_bytes(sum(i["lens"]), 2, max(i["lens"]), 8, 64, 64, c) for i, c in zip(p, (1, 0)))
    assert need > 0
    ws, carry = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.tensor([1, 1], dtype=torch.uint8, device="cuda")

    def prompt(i):
        return S.linear_attn_packed_fwd(i["q"], i["k"], i["v"], i["g"], i["cu"], i["state"], carry=carry, max_seqlen=max(i["lens"]), workspace=ws)

    jobs = [(token, [m.conv, m.state]), (lambda: (prompt(p[0]),), [p[0]["state"]]), (lambda: (prompt(p[1]),), [p[1]["state"]])]
    m.conv.normal_(generator=gen), m.state.normal_(generator=gen)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for job, _ in jobs:
            job()
    torch.cuda.synchronize()
    for job, _ in jobs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = job()
        graphs.append((graph, got))
    for n in range(4):
        tokens.random_(0, 97, generator=gen), u.uniform_(generator=gen), p[0]["v"].normal_(generator=gen)
        for (job, states), (graph, got) in zip(jobs, graphs):
            before = [s.clone() for s in states]
            want = [w.clone() for w in job()]
            after = [s.clone() for s in states]
            for s, b in zip(states, before):
                s.copy_(b)
            if n % 2:
                torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip([*got, *states], [*want, *after]):
                assert torch.equal(a, b), n


def test_linear_attention_past_32_bit_offsets():
    """Decays of e^-1 and less, so that 160 tokens tell what a token's output is (what lies before counts e^-160)."""
    import torch

    import selective_state_space_51_amd as S
    lens, H, dk, dv = [300_000, 7, 240_000, 33, 20_000], 64, 64, 64
    T = sum(lens)
    assert T * H * dv > 2 ** 31 and (T - lens[-1] - lens[-2]) * H * dv > 2 ** 31
    _say("large linear attention", T)
    g = torch.Generator(device="cuda").manual_seed(7)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    v = torch.empty(T, H, dv, **bf)
    for i in range(0, T, 1 << 16):
        v[i:i + (1 << 16)].normal_(0, 1, generator=g)
    q, k = torch.empty(T, 1, dk, **bf).normal_(0, 1, generator=g), torch.empty(T, 1, dk, **bf).normal_(0, 1, generator=g)
    d = -1 - torch.rand(T, H, generator=g, device="cuda")
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    st = torch.full((5, H, dk, dv), 7.0, device="cuda")
    out = S.linear_attn_packed_fwd(q, k, v, d, cu, st, max_seqlen=max(lens))
    torch.cuda.synchronize()
    at = 0
    for s, n in enumerate(lens):
        for last in {n, max(1, n // 2), min(n, 100)}:
            b, e = at + max(0, last - 160), at + last
            i = dict(lens=[e - b], q=q[b:e], k=k[b:e], v=v[b:e], g=d[b:e], state=torch.zeros(1, H, dk, dv, device="cuda"))
            want = LA.reference(i)
            skip = slice(0 if last <= 160 else 150, None)
            own = st[s:s + 1] if last == n else torch.from_numpy(want[1])
            LA.compare(i, out[b:e][skip], own, (want[0][skip], want[1], want[2][skip], want[3]))
        at += n


def test_a_cache_of_states_past_32_bit_offsets():
    import torch

    import selective_state_space_51_amd as S
    H, dk, dv, nslots = 64, 128, 64, 4200
    assert nslots * H * dk * dv > 2 ** 31
    _say("large cache of states")
    st = torch.zeros(nslots, H, dk, dv, device="cuda")
    i = LA.make([1, 1, 1, 50, 300], H, 1, dk, dv, "bf16", seed=4)
    slots = [nslots - 1, 0, 4096, 4097, 4198]
    st[slots] = i["state"]
    small = dict(i, lens=[1, 1, 1], q=i["q"][:3], k=i["k"][:3], v=i["v"][:3], g=i["g"][:3], state=i["state"][:3])
    out = S.linear_attn_step(small["q"], small["k"], small["v"], small["g"], st, slots=torch.tensor(slots[:3], dtype=torch.int32, device="cuda"))
    LA.compare(small, out, st[slots[:3]], LA.reference(small, None, [1] * 3))
    rest = dict(i, lens=[50, 300], q=i["q"][3:], k=i["k"][3:], v=i["v"][3:], g=i["g"][3:], state=i["state"][3:])
    cu = torch.tensor([0, 50, 350], dtype=torch.int32, device="cuda")
    out = S.linear_attn_packed_fwd(rest["q"], rest["k"], rest["v"], rest["g"], cu, st, slots=torch.tensor(slots[3:], dtype=torch.int32, device="cuda"),
                                   carry=torch.ones(2, dtype=torch.bool, device="cuda"), max_seqlen=300)
    LA.compare(rest, out, st[slots[3:]], LA.reference(rest, None, [1, 1]))
    assert not st[1:4096].any() and not st[4098:4198].any()


@pytest.mark.parametrize("rows,vocab,dtype", [(43_000, 50280, "bf16"), (1100, 1 << 21, "f32")])
def test_logits_past_32_bit_offsets(rows, vocab, dtype):
    import torch

    import selective_state_space_51_amd as S
    assert rows * vocab > 2 ** 31
    _say("large logits", rows, vocab, dtype)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.empty(rows, vocab, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    for i in range(0, rows, 500):
        x[i:i + 500].normal_(0, 2.5, generator=g)
    u = torch.rand(rows, generator=g, device="cuda")
    got = S.token_sample(x, u, 0.9, 0, 0.9, 0.001)
    torch.cuda.synchronize()
    for r in (0, 1, rows // 2, rows - 2, rows - 1):
        alone = SA.check(x[r:r + 1], u[r:r + 1], 0.9, 0, 0.9, 0.001)
        for a, b in zip(got, alone):
            assert torch.equal(a[r:r + 1], b), r


def test_states_past_the_caches_are_the_rows_in_parts():
    import torch

    import selective_state_space_51_amd as S
    rows, H, dk, dv = 131, 32, 128, 128
    assert rows * H * dk * dv * 4 >= 256 << 20 > (rows + 1) // 2 * H * dk * dv * 4
    _say("many states", rows)
    i = LA.make([1] * rows, H, 2, dk, dv, "bf16", nslots=rows + 3, seed=6)
    slots = torch.randperm(rows + 3, device="cuda")[:rows].int()
    slots[5] = -1
    a, b = i["state"].clone(), i["state"].clone()
    whole = S.linear_attn_step(i["q"], i["k"], i["v"], i["g"], a, slots=slots)
    half = (rows + 1) // 2
    parts = [S.linear_attn_step(i["q"][p], i["k"][p], i["v"][p], i["g"][p], b, slots=slots[p]) for p in (slice(0, half), slice(half, rows))]
    torch.cuda.synchronize()
    assert torch.equal(whole, torch.cat(parts)) and torch.equal(a, b) and not torch.equal(a, i["state"])
    few = dict(i, lens=[1] * 4, **{n: i[n][:4] for n in "qkvg"}, state=i["state"][slots[:4].long()])
    LA.compare(few, whole[:4], a[slots[:4].long()], LA.reference(few, None, [1] * 4))


def test_drawn_continuations_of_the_example():
    """At temperature 0 they are the greedy ones; without limits a drawn token's log probability is the one that a pass over the
    whole sequence gives (fp32 through two layers; 1e-3 as in the example's own tests)."""
    import torch

    from tests.test_gpu_lm_example import _example, _prompts
    m = _example().MambaLM(vocab=301, width=128, layers=2, slots=6, dtype=torch.float32, seed=3)
    prompts = _prompts((3, 40))
    greedy, _, _ = m.generate(prompts, 5)
    same, logp = m.continuations(prompts, 5, 3, temperature=0.0)
    assert torch.equal(same, greedy.repeat_interleave(3, 0)) and not logp.any()
    drawn, logp = m.continuations(prompts, 5, 3, generator=torch.Generator(device="cuda").manual_seed(1))
    whole = [prompts[i // 3] + t for i, t in enumerate(drawn.tolist())]
    score, at = m.score(whole), 0
    for i, w in enumerate(whole):
        assert float((score[at + len(w) - 6:at + len(w) - 1] - logp[i]).abs().max()) <= 1e-3
        at += len(w)
    with pytest.raises(ValueError, match="without tokens"):
        m.continuations([[1], []], 2, 2)


@pytest.mark.parametrize("nseq", [5, 63, 64, 65])
def test_prompts_dealt_out_by_length_are_the_prompts_alone(nseq):
    """More whole sequences than compute units have room for at once, of mixed and equal lengths and empty ones: each gives the
    bits that it gives alone."""
    import torch

    import selective_state_space_51_amd as S
    H = 60
    lens = [int(n) for n in np.random.default_rng(nseq).choice([0, 1, 40, 64, 64, 130, 200], nseq)]
    _say("dealt", nseq, lens[:8])
    assert nseq * H > 256 and S.linear_attn_packed_workspace_bytes(sum(lens), nseq, max(lens), H, 16, 32) == 0
    i = LA.make(lens, H, 1, 16, 32, "bf16", nslots=nseq, seed=nseq)
    slots = list(np.random.default_rng(1).permutation(nseq))
    out, st = LA.run(i, slots, [s % 2 for s in range(nseq)])
    for s in sorted(set(range(0, nseq, 9)) | {1, 2, nseq - 1}):
        b = sum(lens[:s])
        own = {n: i[n][b:b + lens[s]] for n in "qkvg"}
        one = dict(i, lens=[lens[s]], cu=torch.tensor([0, lens[s]], dtype=torch.int32, device="cuda"), state=i["state"][slots[s]:slots[s] + 1], **own)
        alone, st1 = LA.run(one, None, [s % 2])
        assert torch.equal(alone, out[b:b + lens[s]]) and torch.equal(st1[0], st[slots[s]]), s


@pytest.mark.parametrize("cu", [[700, 2300], [1500, 1500, 2300], [0, 1200, 100, 2300, 50], [2300, 0, 2300, 0], [900, 100, 60, 20]])
def test_segments_of_offsets_that_start_late_or_fall(cu):
    """Offsets that begin past 0, or fall, in a call of several segments: sequences before the first fall are right, and nothing is
    written outside the output and the cache."""
    import torch

    import selective_state_space_51_amd as S
    T, H, n = 2300, 2, len(cu) - 1
    _say("late or falling", cu)
    assert S.linear_attn_packed_workspace_bytes(T, n, T, H, 32, 32) > 0
    i = LA.make([T], H, 1, 32, 32, "bf16", nslots=n, seed=8)
    guard, cache = torch.full((T + 800, H, 32), 7.0, device="cuda", dtype=torch.bfloat16), torch.full((n + 8, H, 32, 32), 7.0, device="cuda")
    out, st = guard[400:T + 400], cache[4:n + 4]
    need = S.linear_attn_packed_workspace_bytes(T, n, T, H, 32, 32)
    ws = torch.full((need + 65536,), 7, dtype=torch.uint8, device="cuda")
    S.linear_attn_packed_fwd(i["q"], i["k"], i["v"], i["g"], torch.tensor(cu, dtype=torch.int32, device="cuda"), st, out=out,
                             max_seqlen=T, workspace=ws[32768:need + 32768])
    torch.cuda.synchronize()
    assert bool((guard[:400] == 7).all()) and bool((guard[T + 400:] == 7).all())
    assert bool((cache[:4] == 7).all()) and bool((cache[n + 4:] == 7).all())
    assert bool((ws[:32768] == 7).all()) and bool((ws[need + 32768:] == 7).all())
    if sorted(cu) == cu:
        for s in range(n):
            b, e = cu[s], cu[s + 1]
            one = dict(i, lens=[e - b], **{x: i[x][b:e] for x in "qkvg"}, state=torch.zeros_like(st[:1]))
            LA.compare(one, out[b:e], st[s:s + 1], LA.reference(one))


@pytest.mark.parametrize("carry", [None, [1, 0, 1]])
def test_prompts_without_tokens(carry):
    import torch

    import selective_state_space_51_amd as S
    i = LA.make([0, 0, 0], 2, 1, 32, 32, "bf16", nslots=3)
    out, st = LA.run(i, None, carry)
    assert out.shape == (0, 2, 32)
    for s in range(3):
        assert torch.equal(st[s], i["state"][s]) if carry and carry[s] else not st[s].any()

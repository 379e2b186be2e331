"""GPU tests of the convolution and the scan on packed prompts and single tokens
(causal_conv1d_packed_fwd, selscan_packed_fwd, causal_conv1d_step, selscan_step), against the fp64
oracle run on each sequence by itself.

Bars: parity.TOL on outputs, as for the framework's other forwards (the arithmetic is the same: a
recurrence in fp32 whose coefficients come from v_exp_f32, rounded once to the io type); states are
fp32 and held to the fp32 bar.  Cached convolution rows are copies: equal bit for bit."""
import sys

import numpy as np
import pytest

import oracle
from tests import parity as PT

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def _torch():
    import torch
    return torch


def make(lens, dim, dtype, seed=0, nslots=None, softplus=True, wide=0, bc_pad=0, width=4):
    """Seeded device inputs; wide: extra columns between the rows of x and z, bc_pad: of B and C."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    io = PT.torch_dtype(dtype)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    n, T = len(lens), sum(lens)
    nslots = nslots or max(n, 1)
    d = torch.exp(torch.rand(T, dim, generator=g, device="cuda") * np.log(100.0) + np.log(1e-3))
    bias = 0.1 * rn(dim) if softplus else None
    if softplus:
        d = d + torch.log(-torch.expm1(-d)) - bias
    return dict(
        lens=lens, cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda"),
        x=rn(T, dim + wide).to(io)[:, :dim], z=rn(T, dim + wide).to(io)[:, wide:], u=rn(T, dim).to(io), delta=d.to(io),
        bias=bias, bc=(bc := rn(T, bc_pad + 32).to(io)), B=bc[:, bc_pad:bc_pad + 16], C=bc[:, bc_pad + 16:],
        A=-torch.exp(0.7 * rn(dim, 16)), D=rn(dim), w=rn(dim, width) / width ** 0.5, cb=rn(dim),
        conv_state=rn(nslots, width - 1, dim).to(io), h_state=rn(nslots, dim, 16))


def f64(t):
    return None if t is None else PT.from_dev(t)


def check(name, got, want, tol):
    got = f64(got) if not isinstance(got, np.ndarray) else got
    err = PT.rel_err(got, want) if want.size else 0.0
    assert err <= tol, (name, err)
    return err


def run_conv_case(i, slots, carry, dtype, silu=True, use_bias=True):
    """The packed convolution against the oracle, sequence by sequence; returns nothing."""
    import selective_state_space_51_amd as S
    torch = _torch()
    n = len(i["lens"])
    old = i["conv_state"].clone()
    st = i["conv_state"].clone()
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    ca = None if carry is None else torch.tensor(carry, dtype=torch.bool, device="cuda")
    out = S.causal_conv1d_packed_fwd(i["x"], i["w"], i["cu"], st, bias=i["cb"] if use_bias else None, slots=sl, carry=ca,
                                     silu=silu)
    torch.cuda.synchronize()
    K = i["w"].shape[1]
    want_state = old.clone()
    cu = i["cu"].tolist()
    x64, out64 = f64(i["x"]), f64(out)
    for s in range(n):
        slot = s if slots is None else slots[s]
        ok = 0 <= slot < old.shape[0]
        kept = old[slot] if ok and carry and carry[s] else torch.zeros_like(old[0])
        xs = x64[cu[s]:cu[s + 1]]
        if len(xs):
            r = oracle.causal_conv1d(xs[None], f64(i["w"]), bias=f64(i["cb"]) if use_bias else None,
                                     state=f64(kept)[None] if K > 1 else None, silu=silu)
            check(("conv", s), out64[cu[s]:cu[s + 1]][None], r, PT.TOL[dtype])
        if ok and K > 1:
            want_state[slot] = torch.cat([kept, i["x"][cu[s]:cu[s + 1]]])[len(xs):]
    assert torch.equal(st, want_state)


def run_scan_case(i, slots, carry, dtype, softplus=True, zoh=False, use_D=True, use_z=True, max_seqlen=None):
    import selective_state_space_51_amd as S
    torch = _torch()
    old = i["h_state"].clone()
    h = i["h_state"].clone()
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    ca = None if carry is None else torch.tensor(carry, dtype=torch.bool, device="cuda")
    y = S.selscan_packed_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["cu"], h, D=i["D"] if use_D else None,
                             z=i["z"] if use_z else None, delta_bias=i["bias"], delta_softplus=softplus, zoh=zoh,
                             slots=sl, carry=ca, max_seqlen=max_seqlen)
    torch.cuda.synchronize()
    cu = i["cu"].tolist()
    u, d, B, C, z, y64, A = (f64(i[k]) if k != "y" else f64(y) for k in ("u", "delta", "B", "C", "z", "y", "A"))
    touched = set()
    worst = 0.0
    for s in range(len(i["lens"])):
        slot = s if slots is None else slots[s]
        ok = 0 <= slot < old.shape[0]
        h0 = f64(old[slot]) if ok and carry and carry[s] else np.zeros(old.shape[1:])
        k = slice(cu[s], cu[s + 1])
        if cu[s + 1] > cu[s]:
            r, hl = oracle.selscan(u[k][None], d[k][None], A, B[k][None], C[k][None], D=f64(i["D"]) if use_D else None,
                                   z=z[k][None] if use_z else None, delta_bias=f64(i["bias"]), delta_softplus=softplus,
                                   zoh=zoh, h0=h0[None], return_h_last=True)
            worst = max(worst, check(("y", s), y64[k][None], r, PT.TOL[dtype]))
            hl = hl[0]
        else:
            hl = h0
        if ok:
            touched.add(slot)
            check(("h", s), h[slot], hl, PT.TOL["f32"])
    for slot in set(range(old.shape[0])) - touched:
        assert torch.equal(h[slot], old[slot])
    return worst


LENS = {
    "one": [1], "two": [2], "empties": [0, 1, 0, 2, 3, 0], "short": [4, 5, 17, 3, 1, 16, 15, 33, 8],
    "cut": [100, 257, 31, 64, 700], "long": [2050],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dim", [1, 24, 65, 200])
def test_packed(dtype, lens, dim):
    ls = LENS[lens]
    _say("packed", dtype, lens, dim)
    n = len(ls)
    rng = np.random.default_rng(dim + n)
    i = make(ls, dim, dtype, seed=dim, nslots=n + 3, wide=8 if dim % 8 == 0 else 0, bc_pad=4 if dim % 8 == 0 else 0)
    slots = rng.permutation(n + 3)[:n].tolist()
    carry = (rng.random(n) < 0.5).tolist()
    run_conv_case(i, slots, carry, dtype)
    run_scan_case(i, slots, carry, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [1, 2, 3, 4])
def test_conv_widths_and_options(dtype, width):
    _say("conv width", dtype, width)
    i = make([3, 0, 40, 1, 2], 20, dtype, seed=width, width=width)
    run_conv_case(i, None, None, dtype, silu=False, use_bias=False)
    run_conv_case(i, [4, 3, 2, 1, 0], [True] * 5, dtype)
    # a slot outside the cache: starts from zeros, keeps nothing
    run_conv_case(i, [-1, 3, 99, 1, 0], [True] * 5, dtype)


@pytest.mark.parametrize("softplus,zoh,use_D,use_z", [(False, False, False, False), (True, True, True, True),
                                                      (False, True, False, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_options(dtype, softplus, zoh, use_D, use_z):
    _say("scan options", dtype, softplus, zoh, use_D, use_z)
    # lengths that run whole and lengths cut into segments
    for lens in ([5, 33, 0, 9], [300, 70, 1]):
        i = make(lens, 40, dtype, softplus=softplus)
        run_scan_case(i, [-1] + list(range(1, len(lens))), [True] * len(lens), dtype, softplus, zoh, use_D, use_z)


@pytest.mark.parametrize("bc_pad", [1, 3, 4])
def test_scan_unaligned_rows(bc_pad):
    # B and C rows that do not start on 4-byte boundaries; z rows at odd offsets
    _say("unaligned", bc_pad)
    i = make([77, 300], 33, "bf16", wide=1, bc_pad=bc_pad)
    run_scan_case(i, None, [True, False], "bf16")
    run_conv_case(i, None, [True, False], "bf16")


def test_split_does_not_change_the_result():
    # max_seqlen only chooses the split: a bound too low runs the sequences whole
    import selective_state_space_51_amd as S
    torch = _torch()
    i = make([1500, 64, 999], 72, "f32")
    assert S.selscan_packed_workspace_bytes(2563, 3, 1500, 72) > 0
    assert S.selscan_packed_workspace_bytes(2563, 3, 1, 72) == 0
    out = []
    for ms in (1500, 1):
        h = i["h_state"].clone()
        y = S.selscan_packed_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["cu"], h, D=i["D"], z=i["z"],
                                 delta_bias=i["bias"], delta_softplus=True, carry=torch.ones(3, dtype=torch.uint8, device="cuda"),
                                 max_seqlen=ms)
        out.append((f64(y), f64(h)))
    check("y", out[0][0], out[1][0], PT.TOL["f32"])
    check("h", out[0][1], out[1][1], PT.TOL["f32"])


def test_many_sequences():
    # more sequences than one search step covers, most of them short
    _say("many sequences")
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 7, size=5000).tolist()
    i = make(lens, 16, "f32", seed=9)
    import selective_state_space_51_amd as S
    torch = _torch()
    st, h = i["conv_state"].clone(), i["h_state"].clone()
    out = S.causal_conv1d_packed_fwd(i["x"], i["w"], i["cu"], st, bias=i["cb"])
    y = S.selscan_packed_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["cu"], h, D=i["D"], z=i["z"],
                             delta_bias=i["bias"], delta_softplus=True, max_seqlen=6)
    torch.cuda.synchronize()
    cu = i["cu"].tolist()
    x, u, d, B, C, z = (f64(i[k]) for k in ("x", "u", "delta", "B", "C", "z"))
    out, y = f64(out), f64(y)
    for s in range(0, 5000, 61):
        k = slice(cu[s], cu[s + 1])
        if lens[s]:
            check(("conv", s), out[k][None], oracle.causal_conv1d(x[k][None], f64(i["w"]), bias=f64(i["cb"])), 1e-5)
            check(("y", s), y[k][None], oracle.selscan(u[k][None], d[k][None], f64(i["A"]), B[k][None], C[k][None],
                                                       D=f64(i["D"]), z=z[k][None], delta_bias=f64(i["bias"]),
                                                       delta_softplus=True), 1e-5)
        else:
            assert float(h[s].abs().max()) == 0 and float(st[s].abs().max()) == 0


def test_a_nan_stays_in_its_sequence():
    import selective_state_space_51_amd as S
    torch = _torch()
    lens = [70, 40, 200]
    i = make(lens, 64, "bf16")
    cu = i["cu"].tolist()
    for k in ("x", "u", "delta", "bc"):
        i[k][cu[1]:cu[2]] = float("nan")
    st, h = i["conv_state"].clone(), i["h_state"].clone()
    out = S.causal_conv1d_packed_fwd(i["x"], i["w"], i["cu"], st, bias=i["cb"])
    y = S.selscan_packed_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["cu"], h, D=i["D"], z=i["z"],
                             delta_bias=i["bias"], delta_softplus=True)
    for t in (out, y):
        assert bool(torch.isfinite(t[:cu[1]].float()).all() and torch.isfinite(t[cu[2]:].float()).all())
        assert bool(torch.isnan(t[cu[1]:cu[2]].float()).all())
    assert bool(torch.isfinite(h[[0, 2]]).all()) and bool(torch.isnan(h[1]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 200), (3, 24), (5, 65), (64, 520), (300, 1024)])
def test_step(dtype, rows, dim):
    import selective_state_space_51_amd as S
    torch = _torch()
    _say("step", dtype, rows, dim)
    i = make([1] * rows, dim, dtype, nslots=rows + 2, wide=8 if dim % 8 == 0 else 0, bc_pad=1 if dim == 65 else 4)
    slots = np.random.default_rng(rows).permutation(rows + 2)[:rows]
    if rows > 2:
        slots[1], slots[2] = -1, rows + 2  # rows without a cache entry
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    ones = torch.ones(rows, dtype=torch.uint8, device="cuda")
    for zoh in (False, True):
        st, h = i["conv_state"].clone(), i["h_state"].clone()
        u = S.causal_conv1d_step(i["x"], i["w"], st, bias=i["cb"], slots=sl)
        y = S.selscan_step(i["u"], i["delta"], i["A"], i["B"], i["C"], h, D=i["D"], z=i["z"], delta_bias=i["bias"],
                           delta_softplus=True, zoh=zoh, slots=sl)
        # the same tokens as one-token prompts
        st2, h2 = i["conv_state"].clone(), i["h_state"].clone()
        u2 = S.causal_conv1d_packed_fwd(i["x"], i["w"], i["cu"], st2, bias=i["cb"], slots=sl, carry=ones)
        assert torch.equal(u, u2) and torch.equal(st, st2)
        keep = f64(i["h_state"])
        h0 = np.stack([keep[s] if 0 <= s < rows + 2 else np.zeros_like(keep[0]) for s in slots])
        r, hl = oracle.selscan(f64(i["u"])[:, None], f64(i["delta"])[:, None], f64(i["A"]), f64(i["B"])[:, None],
                               f64(i["C"])[:, None], D=f64(i["D"]), z=f64(i["z"])[:, None], delta_bias=f64(i["bias"]),
                               delta_softplus=True, zoh=zoh, h0=h0, return_h_last=True)
        check("y", f64(y)[:, None], r, PT.TOL[dtype])
        h64 = f64(h)
        for row, s in enumerate(slots):
            if 0 <= s < rows + 2:
                check(("h", row), h64[s], hl[row], PT.TOL["f32"])
        for s in set(range(rows + 2)) - set(slots.tolist()):
            assert torch.equal(h[s], i["h_state"][s])


def test_prompt_then_steps_equals_one_prompt():
    # a prompt, then its last tokens one by one on the cache, against the prompt read at once
    import selective_state_space_51_amd as S
    torch = _torch()
    dim, L, tail = 48, 90, 6
    i = make([L], dim, "f32")
    full_st, full_h = torch.zeros_like(i["conv_state"]), torch.zeros_like(i["h_state"])
    args = lambda k: (i["u"][k], i["delta"][k], i["A"], i["B"][k], i["C"][k])
    kw = dict(D=i["D"], delta_bias=i["bias"], delta_softplus=True)
    u = S.causal_conv1d_packed_fwd(i["x"], i["w"], i["cu"], full_st, bias=i["cb"])
    y = S.selscan_packed_fwd(*args(slice(None)), i["cu"], full_h, z=i["z"], **kw)
    st, h = torch.zeros_like(full_st), torch.zeros_like(full_h)
    cu = torch.tensor([0, L - tail], dtype=torch.int32, device="cuda")
    head = slice(0, L - tail)
    us = [S.causal_conv1d_packed_fwd(i["x"][head], i["w"], cu, st, bias=i["cb"])]
    ys = [S.selscan_packed_fwd(*args(head), cu, h, z=i["z"][head], **kw)]
    for t in range(L - tail, L):
        k = slice(t, t + 1)
        us.append(S.causal_conv1d_step(i["x"][k], i["w"], st, bias=i["cb"]))
        ys.append(S.selscan_step(*args(k), h, z=i["z"][k], **kw))
    assert torch.equal(torch.cat(us), u) and torch.equal(st, full_st)
    check("y", torch.cat(ys), f64(y), PT.TOL["f32"])
    check("h", h, f64(full_h), PT.TOL["f32"])


def test_side_stream_and_empty_calls():
    import selective_state_space_51_amd as S
    torch = _torch()
    i = make([600, 33], 64, "bf16")
    args = (i["u"], i["delta"], i["A"], i["B"], i["C"], i["cu"])
    kw = dict(D=i["D"], z=i["z"], delta_bias=i["bias"], delta_softplus=True)
    y = S.selscan_packed_fwd(*args, i["h_state"].clone(), **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = S.selscan_packed_fwd(*args, i["h_state"].clone(), stream=side, **kw)
    side.synchronize()
    assert torch.equal(y, y2)
    none = i["u"][:0]
    cu0 = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert S.causal_conv1d_packed_fwd(none, i["w"], cu0, bias=i["cb"]).shape == (0, 64)
    assert S.selscan_packed_fwd(none, none, i["A"], i["B"][:0], i["C"][:0], cu0).shape == (0, 64)
    assert S.selscan_step(none, none, i["A"], i["B"][:0], i["C"][:0], i["h_state"]).shape == (0, 64)


def test_graph_replays_equal_eager():
    import selective_state_space_51_amd as S
    torch = _torch()
    i = make([600, 33, 2], 64, "bf16")
    one = make([1] * 3, 64, "bf16", seed=4)

    def work(st, h):
        out = [S.causal_conv1d_packed_fwd(i["x"], i["w"], i["cu"], st, bias=i["cb"]),
               S.selscan_packed_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["cu"], h, D=i["D"], z=i["z"],
                                    delta_bias=i["bias"], delta_softplus=True)]
        out.append(S.causal_conv1d_step(one["x"], i["w"], st, bias=i["cb"]))
        out.append(S.selscan_step(one["u"], one["delta"], i["A"], one["B"], one["C"], h, D=i["D"], z=one["z"]))
        return out + [st, h]

    eager = [t.clone() for t in work(i["conv_state"].clone(), i["h_state"].clone())]
    st, h = i["conv_state"].clone(), i["h_state"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(st, h)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = work(st, h)
    for _ in range(3):
        for t in cap[:4]:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cap, eager))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,dim", [((1, 2, 5, 15, 16, 17, 31), 24), ((515, 3), 70)])
def test_an_infinity_in_a_sequence_s_last_token(lens, dim, dtype):
    """State n of each channel takes delta x B[n] = +-inf from the last token and is that, neither NaN nor in another state;
    B holds no other infinity, and nothing follows."""
    torch = _torch()
    import selective_state_space_51_amd as S
    _say("last token", lens, dim, dtype)
    i = make(list(lens), dim, dtype, seed=23)
    last = (torch.tensor(np.cumsum(lens), device="cuda") - 1).long()
    i["x"][last] = torch.where(i["x"][last] < 0, -1.0, 1.0).to(i["x"].dtype)
    want_sign = i["x"][last].float()
    i["bc"][last, 3] = float("inf")
    h = torch.zeros_like(i["h_state"])
    S.selscan_packed_fwd(i["x"].contiguous(), i["delta"], i["A"], i["B"], i["C"], i["cu"], h, D=i["D"], z=i["z"],
                         delta_bias=i["bias"], delta_softplus=True, max_seqlen=max(lens))
    torch.cuda.synchronize()
    assert torch.equal(h[:, :, 3], want_sign * float("inf"))
    h[:, :, 3] = 0
    assert torch.isfinite(h).all()

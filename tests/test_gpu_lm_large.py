"""GPU tests of the language-model operators on arrays past 2^31 elements (and 2^32 bytes), so that every index is
formed in 64 bits: sampled rows and channels against the same sums in 64 bits.  Bars as in the operators' own tests."""
import sys

import numpy as np
import pytest

import oracle
from tests import parity as PT

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def fill(t, seed, scale=1.0):
    """Seeded normal values, block by block (no second array of the size)."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        flat[i:i + (1 << 28)].normal_(0, scale, generator=g)
    return t


def test_packed_prompts_past_32_bit_offsets():
    import selective_state_space_51_amd as S
    torch = _torch()
    lens, dim = [300_001, 7, 255_000, 1, 61_000], 3800
    T = sum(lens)
    assert T * dim > 2 ** 31
    _say("large packed", T, dim)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x = fill(torch.empty(T, dim, **bf), 1)
    z = fill(torch.empty(T, dim, **bf), 2)
    delta = fill(torch.empty(T, dim, **bf), 3, 0.7)
    bc = fill(torch.empty(T, 32, **bf), 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    A, D, bias = -torch.exp(0.5 * rn(dim, 16)), rn(dim), rn(dim) - 4.0
    w, cb = rn(dim, 4) / 2, rn(dim)
    conv, h = rn(5, 3, dim).bfloat16(), rn(5, dim, 16)
    conv0, h0 = conv.clone(), h.clone()
    carry = torch.tensor([0, 1, 1, 1, 0], dtype=torch.uint8, device="cuda")
    out = S.causal_conv1d_packed_fwd(x, w, cu, conv, bias=cb, carry=carry)
    y = S.selscan_packed_fwd(x, delta, A, bc[:, :16], bc[:, 16:], cu, h, D=D, z=z, delta_bias=bias, delta_softplus=True,
                             carry=carry, max_seqlen=max(lens))
    torch.cuda.synchronize()
    ch = torch.tensor([0, 1, 1900, dim - 2, dim - 1], device="cuda")
    pick = lambda t: PT.from_dev(t[:, ch].contiguous())
    x5, z5, d5, o5, y5 = map(pick, (x, z, delta, out, y))
    B, C = PT.from_dev(bc[:, :16].contiguous()), PT.from_dev(bc[:, 16:].contiguous())
    f = lambda t: PT.from_dev(t)
    cuh = cu.tolist()
    for s in range(5):
        k = slice(cuh[s], cuh[s + 1])
        keep = bool(carry[s])
        cs = f(conv0[s][:, ch]) if keep else np.zeros((3, 5))
        r = oracle.causal_conv1d(x5[k][None], f(w[ch]), bias=f(cb[ch]), state=cs[None])
        assert PT.rel_err(o5[k][None], r) <= PT.TOL["bf16"]
        hs = f(h0[s][ch]) if keep else np.zeros((5, 16))
        r, hl = oracle.selscan(x5[k][None], d5[k][None], f(A[ch]), B[k][None], C[k][None], D=f(D[ch]), z=z5[k][None],
                               delta_bias=f(bias[ch]), delta_softplus=True, h0=hs[None], return_h_last=True)
        assert PT.rel_err(y5[k][None], r) <= PT.TOL["bf16"]
        assert PT.rel_err(f(h[s][ch]), hl[0]) <= PT.TOL["f32"]
    assert torch.equal(conv[2], x[cuh[3] - 3:cuh[3]]) and torch.equal(conv[4], x[-3:])


def test_steps_on_a_large_cache():
    import selective_state_space_51_amd as S
    torch = _torch()
    dim, slots = 4096, 33_000  # 2.16e9 state values
    _say("large cache", slots, dim)
    h = torch.zeros(slots, dim, 16, device="cuda")
    conv = torch.zeros(slots, 3, dim, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    sl = torch.tensor([slots - 1, 0, 32_800], dtype=torch.int32, device="cuda")
    h[sl.long()] = rn(3, dim, 16)
    conv[sl.long()] = rn(3, 3, dim).bfloat16()
    small_h, small_c = h[sl.long()].clone(), conv[sl.long()].clone()
    x, delta, bc = rn(3, dim).bfloat16(), rn(3, dim).bfloat16(), rn(3, 32).bfloat16()
    A, D, w = -torch.exp(rn(dim, 16)), rn(dim), rn(dim, 4)
    args = (x, delta, A, bc[:, :16], bc[:, 16:])
    y = S.selscan_step(*args, h, D=D, delta_softplus=True, slots=sl)
    u = S.causal_conv1d_step(x, w, conv, slots=sl)
    assert torch.equal(y, S.selscan_step(*args, small_h, D=D, delta_softplus=True))
    assert torch.equal(u, S.causal_conv1d_step(x, w, small_c))
    assert torch.equal(h[sl.long()], small_h) and torch.equal(conv[sl.long()], small_c)
    assert int(torch.count_nonzero(h)) == int(torch.count_nonzero(small_h))


def test_norm_past_32_bit_offsets():
    import selective_state_space_51_amd as S
    torch = _torch()
    rows, width = 140_000, 16_000
    assert rows * width > 2 ** 31
    _say("large norm", rows, width)
    x = fill(torch.empty(rows, width, dtype=torch.bfloat16, device="cuda"), 1)
    r = fill(torch.empty(rows, width, dtype=torch.float32, device="cuda"), 2, 2.0)
    w = 1 + 0.1 * torch.randn(width, device="cuda")
    y, s, rs = S.add_rms_norm_fwd(x, w, residual=r, rstd=True)
    g = S.add_rms_norm_bwd(x, s, w, rs, dresidual_out=r)
    for k in (slice(0, 3), slice(70_000, 70_002), slice(rows - 3, rows)):
        s64 = x[k].double() + r[k].double()
        r64 = 1 / torch.sqrt((s64 * s64).mean(1, keepdim=True) + 1e-5)
        assert torch.equal(s[k], x[k].float() + r[k])
        want = s64 * r64 * w.double()
        assert float(((y[k].double() - want).abs() - 2.0 ** -8 * 1.01 * want.abs()).max()) <= 1e-6
        gw, xh = x[k].double() * w.double(), s64 * r64
        ds = r64 * (gw - xh * (gw * xh).mean(1, keepdim=True)) + r[k].double()
        assert float((g["dresidual"][k].double() - ds).abs().max()) <= 1e-5
    part = torch.zeros(width, dtype=torch.float64, device="cuda")
    mags = torch.zeros_like(part)
    for i in range(0, rows, 5000):
        t = x[i:i + 5000].double() * s[i:i + 5000].double() * rs[i:i + 5000].double()[:, None]
        part += t.sum(0)
        mags += t.abs().sum(0)
    # slots of 274 rows in a row, then 64 additions: 340 u of the magnitudes
    assert float(((g["dweight"].double() - part).abs() - 340 * 2.0 ** -24 * mags).max()) <= 0


def test_logprobs_past_32_bit_offsets():
    import selective_state_space_51_amd as S
    torch = _torch()
    rows, vocab = 43_000, 50_280
    assert rows * vocab > 2 ** 31
    _say("large logprobs", rows, vocab)
    x = fill(torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda"), 1, 2.0)
    t = torch.randint(0, vocab, (rows,), device="cuda")
    lp, ent, st, val, idx = S.token_logprobs_fwd(x, t, top=4)
    g = S.token_logprobs_bwd(x, t, st, ent, dlogprob=torch.ones(rows, device="cuda"))
    for k in (slice(0, 2), slice(42_700, 42_702), slice(rows - 2, rows)):
        want = torch.log_softmax(x[k].double(), 1)
        assert float((lp[k].double() - want.gather(1, t[k][:, None])[:, 0]).abs().max()) <= 2e-5
        assert float((ent[k].double() - torch.special.entr(want.exp()).sum(1)).abs().max()) <= 2e-4
        _, order = torch.sort(x[k].float(), dim=1, descending=True, stable=True)
        assert torch.equal(idx[k], order[:, :4])
        d = -want.exp()
        d[torch.arange(2), t[k]] += 1
        assert float(((g[k].double() - d).abs() - 2.0 ** -8 * 1.01 * d.abs()).max()) <= 1e-7


def test_matvec_past_32_bit_offsets():
    import selective_state_space_51_amd as S
    torch = _torch()
    n, k, grp = 540_000, 16_384, 128
    assert n * k // 2 > 2 ** 32
    _say("large matvec", n, k)
    q = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    for i in range(0, n, 60_000):
        q[i:i + 60_000].random_(0, 256, generator=gen)
    s = (0.01 * torch.rand(n, k // grp, generator=gen, device="cuda") + 0.01).bfloat16()
    x = torch.randn(3, k, generator=gen, device="cuda").bfloat16()
    y = S.w4_matvec(x, q, s, group=grp)
    for i in (slice(0, 40), slice(524_280, 524_300), slice(n - 40, n)):
        w = torch.empty(q[i].shape[0], k, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (q[i] & 15).double(), (q[i] >> 4).double()
        want = x.double() @ ((w - 8) * s[i].double().repeat_interleave(grp, 1)).t()
        assert float(((y[:, i].double() - want).abs() - 2.0 ** -8 * 1.01 * want.abs()).max()) <= 1e-4

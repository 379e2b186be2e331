"""GPU tests of the language-model operators at sizes where they read past the caches: the same rows in parts, each too
small for that, give the same bits.  Only dweight, which adds over all rows, adds in another order."""
import sys

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _torch():
    import torch
    return torch


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def _rn(seed):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zoh", [False, True])
@pytest.mark.parametrize("rows,dim", [(101, 1537), (513, 260), (1030, 129)])
def test_step(rows, dim, zoh, dtype):
    torch = _torch()
    import selective_state_space_51_amd as S
    assert rows * dim * 64 >= 8 << 20 > (rows + 1) // 2 * dim * 64
    _say("step", rows, dim, zoh, dtype)
    rn = _rn(rows)
    io = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, delta, z = rn(rows, dim).to(io), torch.rand(rows, dim, device="cuda").to(io), rn(rows, dim).to(io)
    bc = rn(rows, 32).to(io)
    A, D, db = -torch.rand(dim, 16, device="cuda"), rn(dim), rn(dim)
    h = rn(rows + 9, dim, 16)
    slots = torch.randperm(rows + 9, device="cuda")[:rows].int()
    slots[[3, rows - 1]] = -1
    slots[7] = rows + 9
    hs = [h.clone(), h.clone()]
    args = lambda p: (x[p], delta[p], A, bc[p, :16], bc[p, 16:])
    kw = lambda p: dict(D=D, z=z[p], delta_bias=db, delta_softplus=True, zoh=zoh, slots=slots[p])
    y = S.selscan_step(*args(slice(None)), hs[0], **kw(slice(None)))
    half = (rows + 1) // 2
    parts = [S.selscan_step(*args(p), hs[1], **kw(p)) for p in (slice(0, half), slice(half, rows))]
    torch.cuda.synchronize()
    assert torch.isfinite(y.float()).all() and not torch.equal(hs[0], h)
    assert torch.equal(y, torch.cat(parts)) and torch.equal(hs[0], hs[1])


@pytest.mark.parametrize("rows,vocab,dtype", [(1171, 50280, "bf16"), (7350, 8001, "bf16"), (920, 32001, "f32"), (3750, 8192, "f32")])
def test_logprobs(rows, vocab, dtype):
    torch = _torch()
    import selective_state_space_51_amd as S
    size = 2 if dtype == "bf16" else 4
    assert rows * vocab * size >= 112 << 20 > (rows + 1) // 2 * vocab * size
    _say("logprobs", rows, vocab, dtype)
    rn = _rn(vocab)
    x = (3 * rn(rows, vocab)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x[5] = -float("inf")
    x[6, 1:] = -float("inf")
    x[rows // 2, 17] = float("nan")
    t = torch.randint(-2, vocab, (rows,), device="cuda")
    half = (rows + 1) // 2
    whole = S.token_logprobs_fwd(x, t, top=3, scale=1.3)
    parts = [S.token_logprobs_fwd(x[p], t[p], top=3, scale=1.3) for p in (slice(0, half), slice(half, rows))]
    torch.cuda.synchronize()
    for a, b, c in zip(whole, *parts):
        b = torch.cat((b, c))
        assert torch.equal(torch.nan_to_num(a, 7.0), torch.nan_to_num(b, 7.0))
        assert torch.equal(torch.isnan(a), torch.isnan(b)) if a.is_floating_point() else True


@pytest.mark.parametrize("rows,vocab,dtype", [(1701, 50280, "bf16"), (1311, 32003, "f32")])
def test_logprobs_gradient(rows, vocab, dtype):
    torch = _torch()
    import selective_state_space_51_amd as S
    size = 2 if dtype == "bf16" else 4
    assert rows * vocab * size >= 160 << 20 > (rows + 1) // 2 * vocab * size
    _say("logprobs gradient", rows, vocab, dtype)
    rn = _rn(vocab)
    x = (3 * rn(rows, vocab)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x[5] = -float("inf")
    t = torch.randint(-2, vocab, (rows,), device="cuda")
    _, ent, st = S.token_logprobs_fwd(x, t)
    gl, gh = rn(rows), rn(rows)
    half = (rows + 1) // 2
    whole = S.token_logprobs_bwd(x, t, st, ent, dlogprob=gl, dentropy=gh)
    parts = [S.token_logprobs_bwd(x[p], t[p], st[p], ent[p], dlogprob=gl[p], dentropy=gh[p])
             for p in (slice(0, half), slice(half, rows))]
    torch.cuda.synchronize()
    assert torch.isfinite(whole.float()).all()
    assert torch.equal(whole, torch.cat(parts))


@pytest.mark.parametrize("rows,width", [(7201, 2048), (1810, 8120), (14501, 1016)])
def test_norm_gradients_of_a_16_bit_stream(rows, width):
    torch = _torch()
    import selective_state_space_51_amd as S
    assert rows * width * 8 >= 112 << 20 > (rows + 1) // 2 * width * 8
    _say("norm gradients", rows, width)
    rn = _rn(rows)
    x, r, dy, dres = (rn(rows, width).bfloat16() for _ in range(4))
    w = 1 + 0.2 * rn(width)

    def both(p):
        y, s, saved = S.add_rms_norm_fwd(x[p], w, residual=r[p], rstd=True)
        return y, s, S.add_rms_norm_bwd(dy[p], s, w, saved, dresidual_out=dres[p])
    half = (rows + 1) // 2
    y, s, g = both(slice(None))
    (ya, sa, ga), (yb, sb, gb) = both(slice(0, half)), both(slice(half, rows))
    torch.cuda.synchronize()
    assert torch.equal(y, torch.cat((ya, yb))) and torch.equal(s, torch.cat((sa, sb)))
    assert torch.equal(g["dx"], torch.cat((ga["dx"], gb["dx"]))) and torch.equal(g["dresidual"], torch.cat((ga["dresidual"], gb["dresidual"])))
    # each sum's order: at most rows / 512 + 1 rows in a chain, then 64 chains' worth of partial sums; both sides, in u of
    # the sum of magnitudes
    s64 = x.double() + r.double()
    mag = (dy.double() * s64 / (s64.square().mean(1, keepdim=True) + 1e-5).sqrt()).abs().sum(0)
    bar = 2 * (rows / 512 + 1 + 64) * U * mag
    assert ((g["dweight"].double() - ga["dweight"].double() - gb["dweight"].double()).abs() <= bar).all()

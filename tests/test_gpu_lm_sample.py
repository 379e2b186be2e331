"""GPU tests of token_sample against its definition in 64 bits: tokens and counts are equal, log probabilities off by the rounding
to fp32 (2^-24 of the value) and by what whole multiples of 2^-45 lose of up to 2^17 weights (2^-28)."""
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def draw(x, u, T=1.0, k=0, p=1.0, m=0.0):
    """(token, logprob, kept) of one row by the definition; x, u as 64-bit numbers, settings as fp32 has them."""
    T, p, m = (float(np.float32(v)) for v in (T, p, m))
    if np.isnan(x).any() or (x == np.inf).any():
        return -1, math.nan, 0
    if not (x > -np.inf).any():
        return -1, -math.inf, 0
    if not T > 0:
        return int(np.argmax(x)), 0.0, 1
    live = np.flatnonzero(x > -np.inf)
    order = live[np.argsort(-x[live], kind="stable")]
    w = np.exp((x[order] - x[order[0]]) / T)
    n = len(order)
    if 0 < k < n:
        n = k
    if p < 1:
        before = np.concatenate([[0.0], np.cumsum(w[:n])[:-1]])
        n = max(1, int((before < max(p, 0.0) * w[:n].sum()).sum()))
    n = max(1, int((w[:n] >= min(max(m, 0.0), 1.0)).sum()))
    ids = np.sort(order[:n])
    w = np.exp((x[ids] - x[order[0]]) / T)
    cum = np.cumsum(w)
    u = 0.0 if not u > 0 else u
    at = min(int((cum <= u * cum[-1]).sum()), int(np.flatnonzero(w > 0)[-1]))
    return int(ids[at]), (x[ids[at]] - x[order[0]]) / T - math.log(cum[-1]), n


def check(x, u, T=1.0, k=0, p=1.0, m=0.0):
    import torch

    import selective_state_space_51_amd as S
    out = S.token_sample(x, u, temperature=T, top_k=k, top_p=p, min_p=m)
    torch.cuda.synchronize()
    tok, lp, kept = (o.cpu().numpy() for o in out)
    x64, u64 = x.double().cpu().numpy(), u.double().cpu().numpy()
    at = lambda v, r: v[r].item() if isinstance(v, torch.Tensor) else v
    for r in range(x64.shape[0]):
        want = draw(x64[r], u64[r], at(T, r), at(k, r), at(p, r), at(m, r))
        assert (tok[r], kept[r]) == (want[0], want[2]), (r, tok[r], kept[r], want)
        if math.isfinite(want[1]):
            assert abs(lp[r] - want[1]) <= 2.0 ** -24 * abs(want[1]) + 2.0 ** -28, (r, lp[r], want)
        else:
            assert np.array_equal(lp[r], np.float32(want[1]), equal_nan=True)
    return out


def logits(rows, vocab, dtype, seed=0, spread=2.5, wide=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    io = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (spread * torch.randn(rows, vocab + wide, generator=g, device="cuda")).to(io)[:, wide:]
    return x, torch.rand(rows, generator=g, device="cuda")


VOCABS = [1, 2, 7, 63, 64, 65, 255, 1000, 1024, 1025, 4099, 8192, 8193, 32001, 50280, 66000, 131072]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_settings(vocab, dtype):
    for n, (T, k, p, m) in enumerate(((1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.05), (0.8, 50, 0.95, 0.02),
                                      (1.0, 1, 1.0, 0.0), (0.0, 5, 0.5, 0.5), (1.0, vocab, 0.5, 0.0), (1.0, vocab // 2 + 1, 0.999, 0.0),
                                      (4.0, 700, 0.99, 0.0))):
        _say("settings", vocab, dtype, T, k, p, m)
        x, u = logits(4, vocab, dtype, seed=n + vocab, wide=n % 3)
        check(x, u, T, k, p, m)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_settings_of_each_row(dtype):
    import torch
    rows = 64
    x, u = logits(rows, 5003, dtype, seed=1)
    g = torch.Generator().manual_seed(2)
    pick = lambda *s: torch.tensor(s)[torch.randint(len(s), (rows,), generator=g)].cuda()
    T, k = pick(0.0, 0.5, 1.0, 1.0, 2.0, -1.0, math.nan), pick(0, 0, 1, 5, 300, 9999, -3).to(torch.int32)
    p, m = pick(1.0, 0.9, 0.3, 0.0, -0.5, 1.5), pick(0.0, 0.0, 0.1, 1.0, 2.0, -1.0)
    check(x, u, T, k, p, m)
    check(x, u, T, 7, 0.9, m)
    nan = torch.full((rows,), math.nan, device="cuda")
    a, b = check(x, u, 1.0, 0, 1.0, 0.0), __import__("selective_state_space_51_amd").token_sample(x, u, top_p=nan, min_p=nan)
    assert all(torch.equal(i, j) for i, j in zip(a, b))  # a NaN is no limit


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties_go_to_the_lowest_index(dtype):
    import torch
    io = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(4)
    u = torch.rand(40, generator=g, device="cuda")
    for vocab in (10, 1500, 20001):
        few = torch.randint(0, 4, (40, vocab), generator=g, device="cuda").to(io)  # four values: rows of ties
        for T, k, p, m in ((1.0, 3, 1.0, 0.0), (1.0, vocab // 3, 1.0, 0.0), (1.0, 0, 0.37, 0.0), (2.0, vocab // 2, 0.6, 0.0), (0.0, 0, 1.0, 0.0),
                           (1.0, 0, 1.0, 1.0)):
            _say("ties", vocab, dtype, T, k, p, m)
            check(few, u, T, k, p, m)
        check(torch.zeros(40, vocab, device="cuda", dtype=io), u, 1.0, 0, 0.9, 0.0)
        zeros = torch.where(few > 1, 0.0, -0.0).to(io)  # both zeros are one value
        check(zeros, u, 1.0, 5, 1.0, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_rows_and_far_values(dtype):
    import torch
    io = torch.bfloat16 if dtype == "bf16" else torch.float32
    low, big = torch.finfo(io).min, torch.finfo(io).max
    for vocab in (300, 9001):
        x, u = logits(16, vocab, dtype, seed=vocab)
        x[0] = -math.inf
        x[1, 5] = math.nan
        x[2, vocab - 1] = math.inf
        x[3, :] = -math.inf
        x[3, vocab - 2] = -5.0
        x[4] = low
        x[5, 1:] = low
        x[6, ::2] = -math.inf
        x[7, : vocab - 3] = -math.inf
        x[8] = big
        x[9, 3] = big
        x[10] *= 1e-30
        x[11] *= 1e30
        x[12, 1::2] = -1e10
        x[13] = math.nan
        x[14, 0] = -math.inf
        x[14, 1] = math.nan
        for T, k, p, m in ((1.0, 0, 1.0, 0.0), (0.5, 20, 1.0, 0.0), (1.0, 0, 0.8, 0.0), (1.0, 40, 0.9, 0.1), (0.0, 0, 1.0, 0.0),
                           (1e-6, 0, 0.9, 0.0), (1e6, 0, 0.9, 0.0), (1e-38, 3, 1.0, 0.0), (3e38, 0, 0.5, 0.0)):
            _say("masks", vocab, dtype, T, k, p, m)
            check(x, u, T, k, p, m)


def test_numbers_at_and_past_the_ends():
    import torch
    x, _ = logits(8, 3001, "f32", seed=6)
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan, math.inf, 1e-30], device="cuda")
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (1.0, 10, 0.9, 0.0)):
        check(x, u, T, k, p, m)


def test_frequencies():
    """Evenly spaced numbers draw each token as often as its probability says: counts differ by less than 2 of 20,000, one at each
    end of its stretch."""
    import torch

    import selective_state_space_51_amd as S
    n, vocab = 20000, 40
    x = logits(1, vocab, "f32", seed=9)[0]
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    tok, _, kept = S.token_sample(x.expand(n, vocab).contiguous(), u, temperature=0.9)
    p = torch.softmax(x[0].double() / float(np.float32(0.9)), 0)
    count = torch.bincount(tok, minlength=vocab).double()
    assert bool((kept == vocab).all()) and float((count - n * p).abs().max()) < 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_batches_are_the_rows_alone(dtype):
    import torch

    import selective_state_space_51_amd as S
    x, u = logits(700, 20011, dtype, seed=11)
    for kw in (dict(top_p=0.9), dict(top_k=30, temperature=0.7), dict()):
        tok, lp, kept = S.token_sample(x, u, **kw)
        for a, b in ((0, 3), (300, 301), (690, 700)):
            t2, l2, k2 = S.token_sample(x[a:b], u[a:b], **kw)
            assert torch.equal(tok[a:b], t2) and torch.equal(lp[a:b], l2) and torch.equal(kept[a:b], k2)
    check(x[:24], u[:24], 1.0, 0, 0.9, 0.0)


def test_largest_vocabulary():
    _say("vocab 2^21")
    x, u = logits(2, 1 << 21, "bf16", seed=12)
    check(x, u, 1.0, 0, 0.9, 0.0)
    check(x, u, 1.0, 1000, 1.0, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1 << 19, (1 << 19) + 1, (1 << 20) + 3, 1 << 21])
def test_ties_of_large_vocabularies(vocab, dtype):
    """Borders of top-k and top-p among so many tokens of one value that they are told apart in more than one round."""
    import torch
    io = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(vocab)
    u = torch.rand(3, generator=g, device="cuda")
    # one value, two values next to each other, and four
    x = torch.zeros(3, vocab, device="cuda", dtype=io)
    x[1] = 1 - torch.finfo(io).eps * torch.randint(0, 2, (vocab,), generator=g, device="cuda") / 2
    x[2] = torch.randint(0, 4, (vocab,), generator=g, device="cuda")
    for T, k, p, m in ((1.0, vocab // 3, 1.0, 0.0), (1.0, vocab - 1, 1.0, 0.0), (1.0, 0, 0.37, 0.0), (1.0, 0, 0.9, 0.0),
                       (1.0, vocab // 3, 0.9, 0.0), (2.0, 70_000, 0.37, 0.01)):
        _say("large ties", vocab, dtype, T, k, p, m)
        check(x, u, T, k, p, m)


def test_settings_that_are_no_numbers():
    import torch

    import selective_state_space_51_amd as S
    x, u = logits(2, 50, "f32")
    for name in ("temperature", "top_k", "top_p", "min_p"):
        for bad in (None, "1", [1.0, 1.0]):
            with pytest.raises(TypeError, match=f"{name} must be a number or a tensor"):
                S.token_sample(x, u, **{name: bad})
    want = S.token_sample(x, u, temperature=0.5, top_k=3, top_p=0.5, min_p=0.25)
    got = S.token_sample(x, u, temperature=np.float32(0.5), top_k=np.int64(3), top_p=np.float64(0.5), min_p=np.float32(0.25))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties_of_large_vocabularies_in_large_batches(dtype):
    """More rows than compute units, whose workgroups are smaller: the rows alone, bit for bit."""
    import torch

    import selective_state_space_51_amd as S
    vocab = (1 << 19) + 3
    _say("large ties, 258 rows", dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.zeros(258, vocab, device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    x[1::2] = torch.randint(0, 3, (129, vocab), generator=g, device="cuda").to(x.dtype)
    u = torch.rand(258, generator=g, device="cuda")
    for kw in (dict(top_p=0.6), dict(top_k=vocab // 2), dict(top_k=300_000, top_p=0.9)):
        whole = S.token_sample(x, u, **kw)
        for r in (0, 1, 256, 257):
            assert all(torch.equal(a[r:r + 1], b) for a, b in zip(whole, S.token_sample(x[r:r + 1], u[r:r + 1], **kw))), (kw, r)
    check(x[:2], u[:2], 1.0, vocab // 2, 0.9, 0.0)

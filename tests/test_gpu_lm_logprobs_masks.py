"""GPU tests of token_logprobs_fwd and token_logprobs_bwd on logits of any magnitude: masks of -1e9 to the type's lowest
value over whole slices of a row or whole rows, and rows whose largest logit is that large, against the formulas in 64 bits.

Bars, u = 2^-24, from the exponents as they are formed.  c = scale log2 e carries 3 u (scale and log2 e as fp32, their
product).  A term's exponent is c x - fl(c m) in one rounding where |c m| < 2^24, else (x - m) c in two, so it is off by at
most 5 u |a| with a = c (x - m), and the term by ln 2 times that and v_exp_f32's 1 ulp.  Weighted with the terms themselves,
|a| averages to at most log2(vocab) <= 15 here (the entropy is log2 s plus that average, and at most log2(vocab)), so s is off by
(0.7 5 15 + 2) u, its additions (64 in a chain, then lanes, waves and slices) by 80 u more: 135 u in log s, and the same in ln 2 t
/ s per unit of |a|.  logprob adds the roundings of x - m, of its product with the scale and of the sum: 8 u of itself.  The
gradient is scale p (k0 + k1 log p), p off by 135 u and 5 u |log p|, and log p + entropy by 300 u and 8 u |log p|."""
import sys

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
INF = float("inf")
FLT_MAX = 3.4028234663852886e38


def _torch():
    import torch
    return torch


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [5000, 20000])
def test_a_masked_logit_of_the_lowest_value_has_its_log_probability(vocab, dtype):
    """scale (x - m) = -FLT_MAX less a little is a number of fp32, log2 e times it is not."""
    import selective_state_space_51_amd as S
    torch = _torch()
    _say("lowest", vocab, dtype)
    io = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(4, vocab, generator=g, device="cuda").to(io)
    x[:, 3:] = torch.finfo(io).min
    t = torch.tensor([2, 3, vocab - 1, -1], device="cuda")
    for scale in (1.0, 0.75):
        lp, _, _, val, _ = S.token_logprobs_fwd(x, t, top=5, scale=scale)
        want = torch.log_softmax(x.double() * scale, 1)
        assert bool(torch.isfinite(lp).all()) and bool(torch.isfinite(val).all())
        for got, w in ((lp[:3], want.gather(1, t[:3, None])[:, 0]), (val[:, 3:], want[:, 3:5])):
            assert float(((got.double() - w).abs() - 135 * U - 8 * U * w.abs()).max()) <= 0

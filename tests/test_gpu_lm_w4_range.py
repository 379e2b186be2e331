"""GPU tests of w4_matvec on infinite, NaN and very large x and scales: what the formula gives in 64 bits, infinities by
their sign and NaN where it is NaN; finite outputs to the bar of the operator's other tests, whose derivation does not
depend on the size of x."""
import sys

import pytest

from tests import test_gpu_lm_w4 as W

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros,bias", [(True, True), (False, False)])
@pytest.mark.parametrize("group,rows,n,k", [(32, 12, 70, 288), (64, 12, 200, 1024), (128, 20, 33, 384),
                                            (64, 12, 33_000, 192), (32, 20, 33_000, 160)])  # the last two: many rows of the matrix
def test_any_x(group, rows, n, k, zeros, bias, dtype):
    import torch

    import selective_state_space_51_amd as S
    _say("w4 range", group, rows, n, k, zeros, dtype)
    i = W.make(rows, n, k, group, dtype, zeros=zeros, bias=bias, pad=3, seed=9)
    x = i["x"]
    x[1, 5] = INF
    x[2, k - 1] = -INF
    x[3, 0], x[3, k - 2] = INF, INF
    x[4, 1], x[4, 2] = INF, -INF
    x[5, k // 2] = NAN
    x[6] *= 1e37          # every term passes fp32's range at 16 times its size, few sums of the formula do
    x[7, 9] = 3e38
    x[8, 9], x[8, 10] = 3e38, -3e38
    x[9] *= 1e30
    x[10] *= 3e38 / 8
    if bias:
        i["b"][3] = INF
    # rows of the matrix with a scale that is no number
    i["s"][7, 0], i["s"][8, 0] = INF, NAN
    # what a weight of zero does to an infinite x
    i["q"][9] = 0x88
    if zeros:
        i["z"][9] = 8
    got = S.w4_matvec(x, i["q"], i["s"], zeros=i["z"], group=group, bias=i["b"]).double()
    torch.cuda.synchronize()
    pick = torch.tensor(sorted(set(list(range(16)) + [n // 2, n - 17, n - 16, n - 1])), device="cuda")
    j = dict(x=x, q=i["q"][pick], s=i["s"][pick], z=i["z"][pick] if zeros else None, b=i["b"][pick] if bias else None, group=group)
    # the sums term by term: a library product may split them
    q = torch.stack((j["q"] & 15, j["q"] >> 4), 2).reshape(len(pick), k).double()
    z = j["z"].double().repeat_interleave(group, 1) if zeros else torch.full_like(q, 8.0)
    w = (q - z) * j["s"].double().repeat_interleave(group, 1)
    want = torch.stack([(x[r].double() * w).sum(1) for r in range(rows)])
    if bias:
        want = want + j["b"].double()
    _, bar = W.reference(j)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    got = got[:, pick]
    most = float(torch.finfo(x.dtype).max)
    near = (want.abs() > most * 0.99) & (want.abs() < most * 1.01)
    over = want.abs() >= most * 1.01
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[over], want[over].sign() * INF)
    ok = ~(near | over | torch.isnan(want))
    bar = bar + half * (want.abs() + bar)
    assert bool(torch.isfinite(got[ok]).all())
    # (a bar that is no number: a scale of the row's is none, or x, and those are compared above)
    assert bool(((got - want).abs() <= bar)[ok & torch.isfinite(bar)].all())
    assert int((ok & torch.isfinite(bar)).sum()) > 0.3 * ok.numel() and int(over.sum()) > 20

"""GPU tests of the packed scan and the token step at the ends of what A and delta can be, against the fp64 oracle sequence
by sequence; bars as in the operator's other tests."""
import sys

import numpy as np
import pytest

from tests import test_gpu_lm_scan as T

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("zoh", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,whole", [((1, 2, 3, 5, 18, 31), True), ((100, 7, 333, 16, 35), False), ((700, 2), False),
                                        ((1300, 2), False)])
def test_states_that_forget_at_once(lens, whole, dtype, zoh):
    """A of -inf: the state is what the last token put there.  The lengths end inside groups of four tokens and blocks."""
    import selective_state_space_51_amd as S
    _say("A of -inf", lens, dtype, zoh)
    n, dim = len(lens), 70
    assert (S.selscan_packed_workspace_bytes(sum(lens), n, max(lens), dim) == 0) == whole
    i = T.make(list(lens), dim, dtype, seed=n)
    i["A"][:, 3] = -float("inf")
    i["A"][5] = -float("inf")
    i["A"][6, ::2] = -3e38
    with np.errstate(all="ignore"):
        T.run_scan_case(i, list(range(n))[::-1], [s % 2 == 0 for s in range(n)], dtype, zoh=zoh, max_seqlen=max(lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [(200, 190), (700, 333), (1500, 333)])  # the second launch's walk, and a join of its own
def test_zero_states_outlast_growth(lens, dtype):
    """delta below zero (no softplus): exp(A sum delta) of 16 tokens is exp(32 n) for state n, and nothing comes in before
    token 60, so that every state is 0 until then and whatever delta does matters not."""
    import selective_state_space_51_amd as S
    torch = T._torch()
    _say("zero states", lens, dtype)
    dim = 40
    assert S.selscan_packed_workspace_bytes(sum(lens), 2, max(lens), dim) > 0
    i = T.make(list(lens), dim, dtype, seed=3, softplus=False)
    i["A"] = -torch.arange(1, 17, device="cuda", dtype=torch.float32).repeat(dim, 1)
    for b in i["cu"].tolist()[:-1]:
        i["delta"][b:b + 60] = -2.0
        i["u"][b:b + 60] = 0.0
    T.run_scan_case(i, None, None, dtype, softplus=False, max_seqlen=max(lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [(200, 190), (700, 333), (1500, 333)])
def test_small_states_that_grow_past_the_exponents(lens, dtype):
    """States of about 2^-110 that one segment's 16 tokens raise by exp(6.25 n), up to exp(100) = 2^144, and the next 16 let
    fall again.  Up to 100 nats of exponent in fp32, each with three roundings (A log2 e, its product with delta, the constant),
    and 32 exponentials of an ulp: 100 3 2^-24 + 32 2^-23 = 2.2e-5 of a state; 3e-5 is the bar."""
    import oracle
    import selective_state_space_51_amd as S
    torch = T._torch()
    _say("small states", lens, dtype)
    dim = 40
    i = T.make(list(lens), dim, dtype, seed=3, softplus=False)
    i["A"] = -torch.arange(1, 17, device="cuda", dtype=torch.float32).repeat(dim, 1)
    i["u"].zero_()
    i["delta"].fill_(2.0 ** -10)
    for b in i["cu"].tolist()[:-1]:
        i["u"][b] = 2.0 ** -100
        i["delta"][b + 16:b + 32] = -0.390625
        i["delta"][b + 32:b + 48] = 0.390625
    h = i["h_state"].clone()
    y = S.selscan_packed_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["cu"], h, max_seqlen=max(lens))
    torch.cuda.synchronize()
    u, d, B, C, A = (T.f64(i[k].contiguous()) for k in ("u", "delta", "B", "C", "A"))
    cu = i["cu"].tolist()
    for s in range(2):
        k = slice(cu[s], cu[s + 1])
        r, hl = oracle.selscan(u[k][None], d[k][None], A, B[k][None], C[k][None], return_h_last=True)
        T.check(("y", s), T.f64(y)[k][None], r, 3e-5 + (2.0 ** -8 if dtype == "bf16" else 0))
        T.check(("h", s), h[s], hl[0], 3e-5)

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
@pytest.mark.parametrize("lens,whole", [((1, 2, 3, 5, 18, 31), True), ((100, 7, 333, 16, 35), False), ((700, 2), False)])
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

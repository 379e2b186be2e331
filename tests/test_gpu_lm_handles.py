"""GPU tests of calls that name their stream by its raw handle: handle 0, the default stream, from within another current
stream, and a side stream's.  The work is ordered on the stream that the handle names: an input written there by a
copy behind a wait of some milliseconds is read as the copy leaves it."""
import sys

import pytest

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("which", ["default", "side"])
def test_work_is_ordered_on_the_stream_of_a_raw_handle(which):
    import torch

    import selective_state_space_51_amd as S
    _say("raw handle", which)
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    named = torch.cuda.default_stream() if which == "default" else torch.cuda.Stream()
    handle = named.cuda_stream
    assert (handle == 0) == (which == "default")
    dim, L = 64, 40
    new, cu = rn(L, dim), torch.tensor([0, 25, L], dtype=torch.int32, device="cuda")
    delta, A, bc, w = torch.rand(L, dim, device="cuda"), -torch.rand(dim, 16, device="cuda"), rn(L, 32), rn(dim, 4)
    B, C, h, wt = bc[:, :16], bc[:, 16:], torch.zeros(2, dim, 16, device="cuda"), rn(dim)
    Bw, Cw, dw = B.contiguous()[None], C.contiguous()[None], delta[None]
    q = torch.randint(0, 256, (30, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales, t = rn(30, 1).bfloat16(), torch.randint(0, dim, (L,), generator=g, device="cuda")
    ops = {
        "conv": lambda x, **k: S.causal_conv1d_packed_fwd(x, w, cu, **k),
        "scan": lambda x, **k: S.selscan_packed_fwd(x, delta, A, B, C, cu, h, **k),
        "norm": lambda x, **k: S.add_rms_norm_fwd(x, wt, residual=delta, **k)[0],
        "logprobs": lambda x, **k: S.token_logprobs_fwd(x, t, **k)[0],
        "4-bit": lambda x, **k: S.w4_matvec(x, q, scales, group=64, **k),
        "whole batch": lambda x, **k: S.selscan_fwd(x[None], dw, A, Bw, Cw, **k),
    }
    for name, op in ops.items():
        want = op(new)
        x = torch.full_like(new, 7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(named):
            torch.cuda._sleep(20_000_000)  # some ms of device clocks
            x.copy_(new)
        with torch.cuda.stream(torch.cuda.Stream()):
            got = op(x, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got, want), name

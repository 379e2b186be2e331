"""CPU tests of which stream a call's `stream` argument names, with torch's stream functions replaced by recorders: a raw
handle 0 is the default stream of the operands' device, another handle a stream of that device, and a torch stream of
another device is refused.  The calls themselves end at the operands, which are not device tensors."""
import contextlib

import pytest

import selective_state_space_51_amd as S


class Recorder:
    def __init__(self, monkeypatch, torch):
        self.made, self.entered = [], []
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: self.make("default", device))
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: self.make(handle, device))
        monkeypatch.setattr(torch.cuda, "stream", self.enter)

    def make(self, *what):
        self.made.append(what)
        return what

    def enter(self, stream):
        self.entered.append(stream)
        return contextlib.nullcontext()


def calls(torch):
    x, w = torch.zeros(2, 64), torch.zeros(64)
    q, s = torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3, 1, dtype=torch.bfloat16)
    seq = torch.zeros(1, 4, 8)
    A, bc = torch.zeros(8, 16), torch.zeros(1, 4, 16)
    return [lambda st: S.w4_matvec(x, q, s, group=64, stream=st),
            lambda st: S.add_rms_norm_fwd(x, w, stream=st),
            lambda st: S.token_logprobs_fwd(x, torch.zeros(2, dtype=torch.int64), stream=st),
            lambda st: S.selscan_fwd(seq, seq, A, bc, bc, stream=st),
            lambda st: S.selscan_scan_fwd(S.SELSCAN_OP_FWD, seq, seq, A, bc, bc, stream=st)]


@pytest.mark.parametrize("i", range(5))
def test_raw_handles(monkeypatch, i):
    torch = pytest.importorskip("torch")
    for handle, made in ((0, ("default", None)), (0x1230, (0x1230, None))):
        r = Recorder(monkeypatch, torch)
        with pytest.raises(Exception):
            calls(torch)[i](handle)
        assert r.made == [made] and r.entered == [made]


def test_the_operands_device_decides(monkeypatch):
    torch = pytest.importorskip("torch")

    class OnDevice(torch.Tensor):
        device = torch.device("cuda", 3)

    class OfDevice:
        def __init__(self, i):
            self.device = torch.device("cuda", i)

    t = OnDevice()
    assert t.device.index == 3
    r = Recorder(monkeypatch, torch)
    S._launch_stream(0, (1, t))
    S._launch_stream(7, (t,))
    assert r.made == [("default", t.device), (7, t.device)]
    monkeypatch.setattr(torch.cuda, "Stream", OfDevice)
    same = OfDevice(3)
    assert S._launch_stream(same, (t,)) is same
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        S._launch_stream(OfDevice(0), (t,))

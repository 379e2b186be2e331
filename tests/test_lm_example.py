"""CPU test of examples/serve_mamba_lm.py: a prompt without tokens is refused before anything is read (its "last token" would
be the one before it in the pack, another prompt's), and the slots of a generation may be a list."""
import importlib.util
import os

import pytest


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_mamba_lm.py")
    spec = importlib.util.spec_from_file_location("serve_mamba_lm_cpu", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_prompts_and_slots(monkeypatch):
    import torch
    m = _example().MambaLM(vocab=40, width=64, layers=1, slots=3, dtype=torch.float32, device="cpu")
    read = []

    def prefill(prompts, slots, carry=None):
        read.append(slots)
        raise RuntimeError("no device here")

    monkeypatch.setattr(m, "prefill", prefill)
    for prompts in ([[1, 2], []], [[], [3]]):
        with pytest.raises(ValueError, match="without tokens"):
            m.generate(prompts, 2)
    assert not read
    for slots in ([2, 0], None):
        with pytest.raises(RuntimeError, match="no device"):
            m.generate([[1, 2], [3]], 2, slots)
    assert read[0].tolist() == [2, 0] and read[1].tolist() == [0, 1] and read[0].dtype == torch.int32


def test_more_sequences_than_entries(monkeypatch):
    import torch
    m = _example().MambaLM(vocab=40, width=64, layers=1, slots=5, dtype=torch.float32, device="cpu")
    read = []

    def prefill(prompts, slots, carry=None):
        read.append(slots)
        raise RuntimeError("no device here")

    monkeypatch.setattr(m, "prefill", prefill)
    for call in (lambda: m.continuations([[1], [2]], 2, 3), lambda: m.generate([[1]] * 6, 2)):
        with pytest.raises(ValueError, match="6 sequences do not fit into the 5 entries"):
            call()
    assert not read
    with pytest.raises(RuntimeError, match="no device"):
        m.continuations([[1]], 2, 5)
    with pytest.raises(RuntimeError, match="no device"):
        m.generate([[1]] * 5, 2)
    assert [s.tolist() for s in read] == [[0], [0, 1, 2, 3, 4]]

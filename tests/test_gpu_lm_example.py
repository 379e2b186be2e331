"""GPU test of examples/serve_mamba_lm.py: the operators together.  In fp32, generating token by token from the
cache gives what one pass over the whole sequences gives, and a step of training raises the likelihood."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_mamba_lm.py")
    spec = importlib.util.spec_from_file_location("serve_mamba_lm", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _prompts(lens, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 300, (n,), generator=g).tolist() for n in lens]


def test_generation_equals_one_pass():
    import torch
    E = _example()
    m = E.MambaLM(vocab=301, width=128, layers=3, slots=6, dtype=torch.float32, seed=3)
    prompts = _prompts((3, 1, 70, 18))
    slots = torch.tensor([5, 0, 2, 3], dtype=torch.int32, device="cuda")
    tokens, logp, _ = m.generate(prompts, 7, slots)
    assert tokens.shape == (4, 7)
    whole = [p + t for p, t in zip(prompts, tokens.tolist())]
    score = m.score(whole)
    # fp32 through three layers: the two ways round at 1e-7 per operation; 1e-3 leaves room for their sums over 128-wide
    # products in another order, and is far below the log probabilities' spread
    at = 0
    for i, (p, w) in enumerate(zip(prompts, whole)):
        got = score[at + len(p) - 1:at + len(w) - 1]
        assert float((got - logp[i]).abs().max()) <= 1e-3, i
        assert float(score[at + len(w) - 1]) == 0
        at += len(w)


def test_a_prompt_read_in_two_parts():
    import torch
    E = _example()
    m = E.MambaLM(vocab=301, width=128, layers=2, slots=2, dtype=torch.float32, seed=4)
    a, b = _prompts((50, 41), seed=1)
    x, r, last = m.prefill([a, b], [0, 1])
    one = m.logits(x[last], r[last])
    m.conv.fill_(7)
    m.state.fill_(7)
    m.prefill([a[:33], b[:1]], [0, 1])
    x, r, last = m.prefill([a[33:], b[1:]], [0, 1], carry=[True, True])
    two = m.logits(x[last], r[last])
    assert float((one - two).abs().max()) <= 1e-3 * float(one.abs().max())


def test_training_raises_the_likelihood():
    import torch
    E = _example()
    m = E.MambaLM(vocab=301, width=128, layers=2, slots=4, dtype=torch.bfloat16, seed=5)
    seqs = _prompts((40, 25, 60), seed=2)
    values = [m.train_norm(seqs, lr=0.2, entropy_weight=0.0) for _ in range(6)]
    assert values[-1] > values[0]

"""A small Mamba language model (random weights) that reads packed prompts, generates token by token from the cached
states, forks what it has read into several continuations that are drawn at random, scores what it generated, and takes a
training step of its last norm: the operators of include/selscan_lm.h as a program would run them.

    python examples/serve_mamba_lm.py [--layers 4] [--width 512] [--tokens 16]

A layer: residual add + norm -> 4-bit input projection (convolution input | gate) -> convolution -> two small
projections (delta, B, C) -> scan -> 4-bit output projection.  After the last layer: norm, 4-bit projection onto the
vocabulary, log probabilities.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_51_amd as S  # noqa: E402

N_STATE, WIDTH, GROUP = 16, 4, 64


def quantize(w, group=GROUP):
    """w [n, k] as 4-bit numbers with a scale and a zero point per group of k: what w4_matvec takes."""
    n, k = w.shape
    g = w.float().reshape(n, k // group, group)
    lo, hi = g.amin(2), g.amax(2)
    scale = ((hi - lo) / 15).clamp(min=1e-8).to(torch.bfloat16)
    zero = torch.round(-lo / scale.float()).clamp(0, 15)
    q = (torch.round(g / scale.float()[:, :, None]) + zero[:, :, None]).clamp(0, 15).to(torch.uint8).reshape(n, k)
    return dict(qweight=(q[:, 0::2] | q[:, 1::2] << 4).contiguous(), scales=scale, zeros=zero.to(torch.uint8), group=group)


class MambaLM:
    def __init__(self, vocab=1000, width=512, layers=4, slots=8, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device=device)
        self.dim, self.rank, self.dtype = 2 * width, -(-width // 16), dtype
        self.embed = rn(vocab, width).to(dtype)
        dim = self.dim
        # a step size between 1e-3 and 1e-1 where the projection gives 0
        dt = torch.exp(torch.rand(layers, dim, generator=g, device=device) * math.log(100.0) + math.log(1e-3))
        self.layers = [dict(
            norm=torch.ones(width, device=device),
            inp=quantize(rn(2 * dim, width) / width ** 0.5),
            conv_w=rn(dim, WIDTH) / 2, conv_b=torch.zeros(dim, device=device),
            x_proj=(rn(self.rank + 2 * N_STATE, dim) / dim ** 0.5).to(dtype),
            dt_proj=(rn(dim, self.rank) / self.rank ** 0.5).to(dtype),
            dt_bias=dt[i] + torch.log(-torch.expm1(-dt[i])),
            A=-torch.arange(1, N_STATE + 1, device=device, dtype=torch.float32).repeat(dim, 1).contiguous(),
            D=torch.ones(dim, device=device),
            out=quantize(rn(width, dim) / dim ** 0.5)) for i in range(layers)]
        self.norm = torch.ones(width, device=device)
        self.head = quantize(rn(vocab, width) / width ** 0.5)
        # the cache: per layer the last inputs of the convolution and the state of the scan, of `slots` sequences
        self.conv = torch.zeros(layers, slots, WIDTH - 1, dim, dtype=dtype, device=device)
        self.state = torch.zeros(layers, slots, dim, N_STATE, device=device)

    def _mix(self, i, u, mixer):
        """Between the convolution and the scan: delta (before its bias), B and C from the convolution's output."""
        p = self.layers[i]
        low = u @ p["x_proj"].t()
        delta = low[:, :self.rank] @ p["dt_proj"].t()
        B, C = low[:, self.rank:self.rank + N_STATE], low[:, self.rank + N_STATE:]
        return mixer(u, delta, p["A"], B, C)

    def _run(self, tokens, conv, scan):
        """The residual stream's last output and sum for `tokens`; conv(i, x, p) and scan(i, p, z) are the two mixers."""
        x, residual = self.embed[tokens], None
        for i, p in enumerate(self.layers):
            y, residual = S.add_rms_norm_fwd(x, p["norm"], residual=residual, residual_dtype=torch.float32)
            xz = S.w4_matvec(y, **p["inp"])
            u = conv(i, xz[:, :self.dim], p)
            x = S.w4_matvec(self._mix(i, u, scan(i, p, xz[:, self.dim:])), **p["out"])
        return x, residual

    def prefill(self, prompts, slots, carry=None):
        """Reads prompts (lists of tokens) into the cache entries `slots`; a sequence whose carry is set continues from
        its entry.  Returns the residual stream of every token and where each prompt ends."""
        lens = [len(p) for p in prompts]
        dev = self.embed.device
        cu = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
        slots = torch.as_tensor(slots, dtype=torch.int32, device=dev)
        carry = None if carry is None else torch.as_tensor(carry, dtype=torch.bool, device=dev)
        tokens = torch.tensor([t for p in prompts for t in p], device=dev)
        kw = dict(slots=slots, carry=carry)

        def conv(i, x, p):
            return S.causal_conv1d_packed_fwd(x, p["conv_w"], cu, self.conv[i], bias=p["conv_b"], **kw)

        def scan(i, p, z):
            return lambda u, delta, A, B, C: S.selscan_packed_fwd(
                u, delta, A, B, C, cu, self.state[i], D=p["D"], z=z, delta_bias=p["dt_bias"], delta_softplus=True,
                max_seqlen=max(lens), **kw)

        x, residual = self._run(tokens, conv, scan)
        return x, residual, cu[1:].long() - 1

    def step(self, tokens, slots):
        """One token for each of the sequences in `slots`; returns the residual stream."""
        def conv(i, x, p):
            return S.causal_conv1d_step(x, p["conv_w"], self.conv[i], bias=p["conv_b"], slots=slots)

        def scan(i, p, z):
            return lambda u, delta, A, B, C: S.selscan_step(u, delta, A, B, C, self.state[i], D=p["D"], z=z,
                                                            delta_bias=p["dt_bias"], delta_softplus=True, slots=slots)

        return self._run(tokens, conv, scan)

    def logits(self, x, residual):
        return S.w4_matvec(S.add_rms_norm_fwd(x, self.norm, residual=residual)[0], **self.head)

    def _entries(self, n):
        """n, if the cache has as many entries: a sequence without one would start every token from zeros."""
        if n > self.state.shape[1]:
            raise ValueError(f"{n} sequences do not fit into the {self.state.shape[1]} entries of the cache")
        return n

    def generate(self, prompts, n, slots=None):
        """n greedy tokens after each prompt: ([sequences][n] tokens, their log probabilities, the entropies)."""
        if not all(prompts):
            raise ValueError("a prompt without tokens has no last one to go on from")
        if slots is None:
            slots = range(self._entries(len(prompts)))
        slots = torch.as_tensor(slots, dtype=torch.int32, device=self.embed.device)
        x, residual, last = self.prefill(prompts, slots)
        out = []
        x, residual = x[last], residual[last]
        ignore = torch.full((len(prompts),), -1, dtype=torch.int64, device=x.device)
        for i in range(n):
            _, ent, _, val, idx = S.token_logprobs_fwd(self.logits(x, residual), ignore, top=1)
            out.append((idx[:, 0], val[:, 0], ent))
            if i + 1 < n:
                x, residual = self.step(idx[:, 0], slots)
        return tuple(torch.stack(o, 1) for o in zip(*out))

    def continuations(self, prompts, n, count, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, generator=None):
        """`count` continuations of n tokens drawn for each prompt, which is read once: ([sequences * count][n] tokens, their
        log probabilities among those that could be drawn).  Takes as many entries of the cache as there are continuations."""
        if not all(prompts):
            raise ValueError("a prompt without tokens has no last one to go on from")
        dev = self.embed.device
        slots = torch.arange(self._entries(len(prompts) * count), dtype=torch.int32, device=dev)
        first = slots[::count].contiguous()
        x, residual, last = self.prefill(prompts, first)
        src, caches = first.repeat_interleave(count), [*self.conv, *self.state]
        S.cache_entries_copy(caches, src, slots)
        x, residual = x[last].repeat_interleave(count, 0), residual[last].repeat_interleave(count, 0)
        out = []
        for i in range(n):
            u = torch.rand(len(slots), device=dev, generator=generator)
            token, logp, _ = S.token_sample(self.logits(x, residual), u, temperature, top_k, top_p, min_p)
            out.append((token, logp))
            if i + 1 < n:
                x, residual = self.step(token, slots)
        return tuple(torch.stack(o, 1) for o in zip(*out))

    def score(self, sequences):
        """Log probability of every token of `sequences` given those before it (0 for the first of each)."""
        x, residual, last = self.prefill(sequences, list(range(len(sequences))))
        targets = torch.full((x.shape[0],), -1, dtype=torch.int64, device=x.device)
        flat = torch.tensor([t for s in sequences for t in s], device=x.device)
        targets[:-1] = flat[1:]
        targets[last] = -1  # the next token belongs to the next sequence
        return S.token_logprobs_fwd(self.logits(x, residual), targets)[0]

    def train_norm(self, sequences, lr=0.5, entropy_weight=0.01):
        """One gradient step of the last norm's weight towards likelier `sequences` and a higher entropy; returns the
        mean log probability before it."""
        x, residual, last = self.prefill(sequences, list(range(len(sequences))))
        targets = torch.full((x.shape[0],), -100, dtype=torch.int64, device=x.device)
        flat = torch.tensor([t for s in sequences for t in s], device=x.device)
        targets[:-1] = flat[1:]
        targets[last] = -100
        count = int((targets >= 0).sum())
        y, s, saved = S.add_rms_norm_fwd(x, self.norm, residual=residual, rstd=True)
        logits = S.w4_matvec(y, **self.head)
        logp, ent, stats = S.token_logprobs_fwd(logits, targets)
        up = torch.full_like(logp, -1.0 / count)  # the loss is the mean of -logp - entropy_weight * entropy
        dlogits = S.token_logprobs_bwd(logits, targets, stats, ent, up, up * entropy_weight)
        h = self.head
        q = torch.stack([h["qweight"] & 15, h["qweight"] >> 4], -1).reshape(h["scales"].shape[0], -1, h["group"]).float()
        w = ((q - h["zeros"].float()[:, :, None]) * h["scales"].float()[:, :, None]).reshape(q.shape[0], -1)
        grads = S.add_rms_norm_bwd((dlogits.float() @ w).to(y.dtype), s, self.norm, saved)
        self.norm -= lr * grads["dweight"]
        return float(logp.sum()) / count


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    m = MambaLM(layers=a.layers, width=a.width)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1000, (n,), generator=g).tolist() for n in (5, 1, 33, 120)]
    tokens, logp, ent = m.generate(prompts, a.tokens)
    for p, t, l, e in zip(prompts, tokens.tolist(), logp, ent):
        print(f"prompt of {len(p):3d} -> {t[:8]}...  mean log probability {float(l.mean()):.3f}, entropy {float(e.mean()):.3f}")
    drawn, _ = m.continuations(prompts[:2], a.tokens, 4, temperature=0.9, top_k=50, top_p=0.95)
    for i, t in enumerate(drawn.tolist()):
        print(f"prompt of {len(prompts[i // 4]):3d}, drawn -> {t[:8]}...")
    whole = [p + t for p, t in zip(prompts, tokens.tolist())]
    score = m.score(whole)
    at = len(whole[0]) - 1  # the first sequence's generated tokens, scored in one pass over it
    again = score[len(prompts[0]) - 1:at]
    print(f"first sequence rescored: log probabilities differ by at most {float((again - logp[0]).abs().max()):.4f}")
    losses = [m.train_norm(whole) for _ in range(5)]
    print("mean log probability over five training steps of the last norm:", " ".join(f"{v:.4f}" for v in losses))


if __name__ == "__main__":
    main()

"""The operators next to the scan when Mamba layers serve and train a language model, on torch tensors.

Every function has the name of the C-ABI entry point it calls (see include/selscan_lm.h) and is
also a name of the package.  The checks of the tensors and the allocation of outputs (on the launch's stream)
are native code (csrc/lm_binding.cpp), since a token step lasts no longer than they do.  Row-strided
inputs (column slices of a wider array, as the halves
of an input projection's output) are taken as they are; everything else must be contiguous.  If
libselscan_lm.so or the binding is missing the import fails loudly: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch  # its HIP runtime first, as for libselscan.so

_PKG = os.path.dirname(os.path.abspath(__file__))
LM_LIB_PATH = os.path.join(_PKG, "libselscan_lm.so")
LM_HEADER = os.path.join(os.path.dirname(_PKG), "include", "selscan_lm.h")


def _load():
    """The C ABI itself (size queries, and callers that have pointers)."""
    for path in (LM_LIB_PATH, os.path.join(_PKG, "_lm_binding.so")):
        if not os.path.exists(path):
            raise ImportError(f"{path} not found; build it with `python selective_state_space_51_amd/build.py` "
                              "(hipcc, gfx950)")
    lib = ctypes.CDLL(LM_LIB_PATH)
    vp, i64, ci, cu, sz, cf = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t,
                               ctypes.c_float)

    def sig(name, args, ret=ci):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ret

    sig("causal_conv1d_packed_fwd", [vp, i64] + [vp] * 6 + [cu, vp] + [i64] * 5 + [ci, vp])
    sig("causal_conv1d_step", [vp, i64] + [vp] * 4 + [cu, vp] + [i64] * 4 + [ci, vp])
    sig("selscan_packed_fwd", [vp] * 5 + [i64, vp, vp, i64, vp, cu] + [vp] * 5 + [i64] * 6 + [ci, vp, sz, vp])
    sig("selscan_packed_workspace_bytes", [i64] * 5, sz)
    sig("selscan_step", [vp] * 5 + [i64, vp, vp, i64, vp, cu] + [vp] * 3 + [i64] * 4 + [ci, vp])
    sig("add_rms_norm_fwd", [vp, i64, vp, vp, cf, ci] + [vp] * 4 + [i64, i64, ci, ci, vp])
    sig("add_rms_norm_bwd", [vp] * 3 + [i64] + [vp] * 6 + [i64, i64, ci, ci, vp, sz, vp])
    sig("add_rms_norm_bwd_workspace_bytes", [i64, i64], sz)
    sig("token_logprobs_fwd", [vp, i64, vp, cf, ci] + [vp] * 5 + [i64, i64, ci, vp, sz, vp])
    sig("token_logprobs_workspace_bytes", [i64, i64, ci], sz)
    sig("token_logprobs_bwd", [vp, i64] + [vp] * 5 + [cf, vp, i64, i64, ci, vp])
    sig("w4_matvec", [vp, i64] + [vp] * 5 + [i64] * 4 + [ci, vp])
    sig("selscan_lm_abi_version", [])
    sig("selscan_lm_last_hip_error", [], ctypes.c_char_p)
    return lib


lm_lib = _load()
from . import _launch_stream, _lm_binding as _C  # noqa: E402


def lm_abi_version() -> int:
    return int(lm_lib.selscan_lm_abi_version())


def _run(stream, fn, *args):
    """fn(*args) with `stream` (a torch stream or a raw handle; None: the current one) as the current one: kernels run
    there, and what a call allocates belongs to it."""
    if stream is None:
        return fn(*args)
    with torch.cuda.stream(_launch_stream(stream, args)):
        return fn(*args)


def causal_conv1d_packed_fwd(x, weight, cu_seqlens, conv_state=None, bias=None, slots=None, carry=None, silu=True,
                             out=None, stream=None):
    """Depthwise causal convolution of packed prompts: x [tokens, dim], weight [dim, width], cu_seqlens
    int32 [nseq + 1].  conv_state [nslots, width - 1, dim] (io dtype) is read for the sequences whose carry
    (uint8 or bool [nseq]) is set and updated in place for all, at entry slots[s] (int32; None: s)."""
    return _run(stream, _C.causal_conv1d_packed_fwd, x, weight, cu_seqlens, conv_state, bias, slots, carry, silu, out)


def causal_conv1d_step(x, weight, conv_state, bias=None, slots=None, silu=True, out=None, stream=None):
    """One token of the depthwise causal convolution for each of x's rows [rows, dim]; conv_state
    [nslots, width - 1, dim] is shifted in place at entry slots[r] (int32; None: r)."""
    return _run(stream, _C.causal_conv1d_step, x, weight, conv_state, bias, slots, silu, out)


def selscan_packed_workspace_bytes(tokens: int, nseq: int, max_seqlen: int, dim: int, dstate: int = 16) -> int:
    return int(lm_lib.selscan_packed_workspace_bytes(tokens, nseq, max_seqlen, dim, dstate))


def selscan_packed_fwd(x, delta, A, B, C, cu_seqlens, h_state=None, D=None, z=None, delta_bias=None,
                       delta_softplus=False, zoh=False, slots=None, carry=None, max_seqlen=None, y=None,
                       workspace=None, stream=None):
    """selscan_fwd on packed prompts: x, delta, z [tokens, dim]; B, C [tokens, 16]; A [dim, 16]; cu_seqlens int32
    [nseq + 1].  h_state fp32 [nslots, dim, 16] is read for the sequences whose carry is set and updated in
    place for all.  max_seqlen: the longest length or a bound on it (speed only; None: all tokens could be one sequence's,
    which costs a set of short ones a second launch that finds little to do)."""
    return _run(stream, _C.selscan_packed_fwd, x, delta, A, B, C, cu_seqlens, h_state, D, z, delta_bias, delta_softplus,
                zoh, slots, carry, max_seqlen, y, workspace)


def selscan_step(x, delta, A, B, C, h_state, D=None, z=None, delta_bias=None, delta_softplus=False, zoh=False,
                 slots=None, y=None, stream=None):
    """One token of the scan for each row: x, delta, z [rows, dim]; B, C [rows, 16]; h_state fp32 [nslots, dim, 16] is
    updated in place at entry slots[r] (int32; None: r)."""
    return _run(stream, _C.selscan_step, x, delta, A, B, C, h_state, D, z, delta_bias, delta_softplus, zoh, slots, y)


def add_rms_norm_fwd(x, weight, residual=None, eps=1e-5, out="io", residual_dtype=None, rstd=False, stream=None):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the rows of x [rows, width].

    residual: [rows, width], fp32 or x's dtype (None: s = x, kept as residual_dtype, by default x's).
    out: "io" (y in x's dtype), "int8" or "fp8" (e4m3; y stands for scale[:, None] * y).
    Returns (y, s[, scale][, saved]): s in the residual's dtype, scale fp32 [rows] for the 8-bit outputs.
    rstd=True adds what add_rms_norm_bwd needs beside s: rstd fp32 [rows]; where s was rounded to 16 bits, the
    tuple (rstd, x, residual), since the sum that was normed is theirs and not the rounded one."""
    return _run(stream, _C.add_rms_norm_fwd, x, weight, residual, eps, out, residual_dtype, rstd)


def add_rms_norm_bwd_workspace_bytes(rows: int, width: int) -> int:
    return int(lm_lib.add_rms_norm_bwd_workspace_bytes(rows, width))


def add_rms_norm_bwd(dy, s, weight, rstd, x_dtype=None, dresidual_out=None, workspace=None, stream=None):
    """Gradients of add_rms_norm_fwd's "io" output: dy [rows, width]; s and rstd (its rstd=True result, as it is)
    from the forward; dresidual_out the gradient that reaches s by the residual path (None: none).  Returns a dict:
    dx (x_dtype, which is dy's), dresidual (the same numbers in s's dtype; dx itself where the dtypes agree) and dweight (fp32 [width])."""
    if x_dtype not in (None, dy.dtype):
        raise TypeError("dy must have x's dtype")
    # a sum that was rounded to 16 bits is formed anew from x and the residual
    rs, x, base = rstd if isinstance(rstd, tuple) else (rstd, None, s)
    dx, dres, dw = _run(stream, _C.add_rms_norm_bwd, dy, base, weight, rs, x, dresidual_out, workspace)
    return {"dx": dx, "dresidual": dres, "dweight": dw}


def token_logprobs_workspace_bytes(rows: int, vocab: int, top: int = 0) -> int:
    return int(lm_lib.token_logprobs_workspace_bytes(rows, vocab, top))


def token_logprobs_fwd(logits, targets, top=0, scale=1.0, workspace=None, stream=None):
    """Log probability of targets (int64 [rows]; outside [0, vocab): 0) under softmax(scale * logits), logits
    [rows, vocab], and the entropy.  Returns (logprob, entropy, stats), fp32 [rows], [rows] and [rows, 2]
    (the largest logit; log sum exp of scale * (logits - it)), and with top > 0 also (top_logprob fp32,
    top_index int64), [rows, top], largest first, equal logits by index."""
    return _run(stream, _C.token_logprobs_fwd, logits, targets, top, scale, workspace)


def token_logprobs_bwd(logits, targets, stats, entropy, dlogprob=None, dentropy=None, scale=1.0, stream=None):
    """Gradient of sum(dlogprob * logprob + dentropy * entropy) for the logits (contiguous, their dtype); stats and
    entropy from token_logprobs_fwd with the same scale; dlogprob, dentropy fp32 [rows], one at least."""
    return _run(stream, _C.token_logprobs_bwd, logits, targets, stats, entropy, dlogprob, dentropy, scale)


def w4_matvec(x, qweight, scales, zeros=None, group=128, bias=None, out=None, stream=None):
    """x [rows, k] times the transpose of a 4-bit matrix: qweight uint8 [n, k // 2] (q[2i] in the low, q[2i+1] in the
    high bits of byte i), weight (q - zero) * scale with scales bf16 and zeros uint8 (None: 8), [n, k // group]
    each; bias fp32 [n].  Returns [rows, n] in x's dtype."""
    return _run(stream, _C.w4_matvec, x, qweight, scales, zeros, group, bias, out)

"""Python binding of libselscan_lm (argument marshalling only): the operators next to the scan when
Mamba layers serve and train a language model.

Every function has the name of the C-ABI entry point it calls (see include/selscan_lm.h) and is
also a name of the package.  Row-strided inputs (column slices of a wider array, as the halves
of an input projection's output) are taken as they are; everything else must be contiguous.  If
libselscan_lm.so is missing the import fails loudly: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

from . import (SELSCAN_FLAG_SILU, SelscanError, _dtype_code, _flags, _on_launch_stream, _ptr, _shape_check, _stream,
               _torch)

_PKG = os.path.dirname(os.path.abspath(__file__))
LM_LIB_PATH = os.environ.get("SELSCAN_LM_LIB") or os.path.join(_PKG, "libselscan_lm.so")
LM_HEADER = os.path.join(os.path.dirname(_PKG), "include", "selscan_lm.h")

_OUT_KINDS = {"io": 0, "int8": 1, "fp8": 2}


def _load(path=None):
    import torch  # noqa: F401  (its HIP runtime first, as for libselscan.so)
    path = path or LM_LIB_PATH
    if not os.path.exists(path):
        raise ImportError(
            f"libselscan_lm.so not found at {path}; build it with "
            "`python selective_state_space_51_amd/build.py` (hipcc, gfx950)")
    lib = ctypes.CDLL(path)
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


def lm_abi_version() -> int:
    return int(lm_lib.selscan_lm_abi_version())


def _check(rc, what):
    if rc != 0:
        raise SelscanError(rc, what, hip_error=lm_lib.selscan_lm_last_hip_error)


def _typed(t, name, dtype):
    """Pointer of a contiguous device tensor of one dtype (None passes)."""
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    return _ptr(t, name)


def _rows(t, name, io):
    """Pointer and row stride of a two-dimensional device tensor whose rows are contiguous."""
    torch = _torch()
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != io:
        raise TypeError(f"{name} must have the io dtype {io}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    rows, width = t.shape
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    stride = t.stride(0) if rows > 1 else width
    if rows > 1 and stride < width:
        raise ValueError(f"the rows of {name} overlap")
    return (t.data_ptr() if t.numel() else None), max(stride, width)


def _same_stride(a, b, name_a, name_b, io):
    pa, sa = _rows(a, name_a, io)
    pb, sb = _rows(b, name_b, io)
    if sa != sb:
        raise ValueError(f"{name_a} and {name_b} must have the same row stride")
    return pa, pb, sa


def _workspace(need, given, device):
    torch = _torch()
    if need == 0:
        return None, 0, None
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=device)
    return given.data_ptr(), given.numel() * given.element_size(), given


def _scan_shapes(x, delta, A, B, C, D, z, delta_bias):
    rows, dim = x.shape
    N = A.shape[-1]
    for n_, t_, s_ in (("delta", delta, (rows, dim)), ("A", A, (dim, N)), ("B", B, (rows, N)), ("C", C, (rows, N)),
                       ("D", D, (dim,)), ("z", z, (rows, dim)), ("delta_bias", delta_bias, (dim,))):
        _shape_check(n_, t_, s_)
    return rows, dim, N


def _packed_indices(cu_seqlens, slots, carry, cache, name):
    torch = _torch()
    nseq = cu_seqlens.numel() - 1
    if cu_seqlens.dim() != 1 or nseq < 0:
        raise ValueError("cu_seqlens must be a vector of nseq + 1 offsets")
    _shape_check("slots", slots, (nseq,))
    _shape_check("carry", carry, (nseq,))
    if carry is not None and carry.dtype == torch.bool:
        carry = carry.view(torch.uint8)
    nslots = cache.shape[0] if cache is not None else 0
    return nseq, nslots, _typed(cu_seqlens, "cu_seqlens", torch.int32), _typed(slots, "slots", torch.int32), \
        _typed(carry, "carry", torch.uint8)


@_on_launch_stream
def causal_conv1d_packed_fwd(x, weight, cu_seqlens, conv_state=None, bias=None, slots=None, carry=None, silu=True,
                             out=None, stream=None):
    """Depthwise causal convolution of packed prompts: x [tokens, dim], weight [dim, width], cu_seqlens
    int32 [nseq + 1].  conv_state [nslots, width - 1, dim] (io dtype) is read for the sequences whose carry
    (uint8 or bool [nseq]) is set and updated in place for all, at entry slots[s] (int32; None: s)."""
    torch = _torch()
    tokens, dim = x.shape
    width = weight.shape[-1]
    io = x.dtype
    _shape_check("weight", weight, (dim, width))
    _shape_check("bias", bias, (dim,))
    if conv_state is not None:
        _shape_check("conv_state", conv_state, (conv_state.shape[0], width - 1, dim))
    nseq, nslots, cu_p, slots_p, carry_p = _packed_indices(cu_seqlens, slots, carry, conv_state, "conv_state")
    if out is None:
        out = torch.empty(tokens, dim, dtype=io, device=x.device)
    _shape_check("out", out, (tokens, dim))
    xp, xs = _rows(x, "x", io)
    rc = lm_lib.causal_conv1d_packed_fwd(xp, xs, _ptr(weight, "weight", f32=True), _ptr(bias, "bias", f32=True), cu_p,
                                         slots_p, carry_p, _ptr(conv_state, "conv_state", io),
                                         SELSCAN_FLAG_SILU if silu else 0, _ptr(out, "out", io), tokens, nseq, nslots,
                                         dim, width, _dtype_code(x), _stream(stream))
    _check(rc, "causal_conv1d_packed_fwd")
    return out


@_on_launch_stream
def causal_conv1d_step(x, weight, conv_state, bias=None, slots=None, silu=True, out=None, stream=None):
    """One token of the depthwise causal convolution for each of x's rows [rows, dim]; conv_state
    [nslots, width - 1, dim] is shifted in place at entry slots[r] (int32; None: r)."""
    torch = _torch()
    rows, dim = x.shape
    width = weight.shape[-1]
    io = x.dtype
    _shape_check("weight", weight, (dim, width))
    _shape_check("bias", bias, (dim,))
    _shape_check("conv_state", conv_state, (conv_state.shape[0], width - 1, dim))
    _shape_check("slots", slots, (rows,))
    if out is None:
        out = torch.empty(rows, dim, dtype=io, device=x.device)
    _shape_check("out", out, (rows, dim))
    xp, xs = _rows(x, "x", io)
    rc = lm_lib.causal_conv1d_step(xp, xs, _ptr(weight, "weight", f32=True), _ptr(bias, "bias", f32=True),
                                   _typed(slots, "slots", torch.int32), _ptr(conv_state, "conv_state", io),
                                   SELSCAN_FLAG_SILU if silu else 0, _ptr(out, "out", io), rows, conv_state.shape[0],
                                   dim, width, _dtype_code(x), _stream(stream))
    _check(rc, "causal_conv1d_step")
    return out


def selscan_packed_workspace_bytes(tokens: int, nseq: int, max_seqlen: int, dim: int, dstate: int = 16) -> int:
    return int(lm_lib.selscan_packed_workspace_bytes(tokens, nseq, max_seqlen, dim, dstate))


@_on_launch_stream
def selscan_packed_fwd(x, delta, A, B, C, cu_seqlens, h_state=None, D=None, z=None, delta_bias=None,
                       delta_softplus=False, zoh=False, slots=None, carry=None, max_seqlen=None, y=None,
                       workspace=None, stream=None):
    """selscan_fwd on packed prompts: x, delta, z [tokens, dim]; B, C [tokens, 16]; A [dim, 16]; cu_seqlens int32
    [nseq + 1].  h_state fp32 [nslots, dim, 16] is read for the sequences whose carry is set and updated in
    place for all.  max_seqlen: the longest length or a bound on it (speed only)."""
    torch = _torch()
    tokens, dim, N = _scan_shapes(x, delta, A, B, C, D, z, delta_bias)
    io = x.dtype
    if h_state is not None:
        _shape_check("h_state", h_state, (h_state.shape[0], dim, N))
    nseq, nslots, cu_p, slots_p, carry_p = _packed_indices(cu_seqlens, slots, carry, h_state, "h_state")
    if max_seqlen is None:
        max_seqlen = tokens
    if y is None:
        y = torch.empty(tokens, dim, dtype=io, device=x.device)
    _shape_check("y", y, (tokens, dim))
    ws, wsb, _keep = _workspace(selscan_packed_workspace_bytes(tokens, nseq, max_seqlen, dim, N), workspace, x.device)
    bp, cp, bcs = _same_stride(B, C, "B", "C", io)
    zp, zs = _rows(z, "z", io)
    rc = lm_lib.selscan_packed_fwd(_ptr(x, "x", io), _ptr(delta, "delta", io), _ptr(A, "A", f32=True), bp, cp, bcs,
                                   _ptr(D, "D", f32=True), zp, zs, _ptr(delta_bias, "delta_bias", f32=True),
                                   _flags(delta_softplus, zoh), cu_p, slots_p, carry_p,
                                   _ptr(h_state, "h_state", f32=True), _ptr(y, "y", io), tokens, nseq, nslots,
                                   max_seqlen, dim, N, _dtype_code(x), ws, wsb, _stream(stream))
    _check(rc, "selscan_packed_fwd")
    return y


@_on_launch_stream
def selscan_step(x, delta, A, B, C, h_state, D=None, z=None, delta_bias=None, delta_softplus=False, zoh=False,
                 slots=None, y=None, stream=None):
    """One token of the scan for each row: x, delta, z [rows, dim]; B, C [rows, 16]; h_state fp32 [nslots, dim, 16] is
    updated in place at entry slots[r] (int32; None: r)."""
    torch = _torch()
    rows, dim, N = _scan_shapes(x, delta, A, B, C, D, z, delta_bias)
    io = x.dtype
    _shape_check("h_state", h_state, (h_state.shape[0], dim, N))
    _shape_check("slots", slots, (rows,))
    if y is None:
        y = torch.empty(rows, dim, dtype=io, device=x.device)
    _shape_check("y", y, (rows, dim))
    bp, cp, bcs = _same_stride(B, C, "B", "C", io)
    zp, zs = _rows(z, "z", io)
    rc = lm_lib.selscan_step(_ptr(x, "x", io), _ptr(delta, "delta", io), _ptr(A, "A", f32=True), bp, cp, bcs,
                             _ptr(D, "D", f32=True), zp, zs, _ptr(delta_bias, "delta_bias", f32=True),
                             _flags(delta_softplus, zoh), _typed(slots, "slots", torch.int32),
                             _ptr(h_state, "h_state", f32=True), _ptr(y, "y", io), rows, h_state.shape[0], dim, N,
                             _dtype_code(x), _stream(stream))
    _check(rc, "selscan_step")
    return y


@_on_launch_stream
def add_rms_norm_fwd(x, weight, residual=None, eps=1e-5, out="io", residual_dtype=None, rstd=False, stream=None):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the rows of x [rows, width].

    residual: [rows, width], fp32 or x's dtype (None: s = x, kept as residual_dtype, by default x's).
    out: "io" (y in x's dtype), "int8" or "fp8" (e4m3; y stands for scale[:, None] * y).
    Returns (y, s[, scale][, saved]): s in the residual's dtype, scale fp32 [rows] for the 8-bit outputs.
    rstd=True adds what add_rms_norm_bwd needs beside s: rstd fp32 [rows]; where s was rounded to 16 bits, the
    tuple (rstd, x, residual), since the sum that was normed is theirs and not the rounded one."""
    torch = _torch()
    rows, width = x.shape
    io = x.dtype
    if out not in _OUT_KINDS:
        raise ValueError(f"out must be one of {sorted(_OUT_KINDS)}")
    rdt = residual.dtype if residual is not None else residual_dtype or io
    if rdt not in (torch.float32, io):
        raise TypeError("the residual must be float32 or have the io dtype")
    _shape_check("weight", weight, (width,))
    _shape_check("residual", residual, (rows, width))
    y = torch.empty(rows, width, dtype={"io": io, "int8": torch.int8, "fp8": torch.float8_e4m3fn}[out], device=x.device)
    s = torch.empty(rows, width, dtype=rdt, device=x.device)
    scale = torch.empty(rows, dtype=torch.float32, device=x.device) if out != "io" else None
    rs = torch.empty(rows, dtype=torch.float32, device=x.device) if rstd else None
    xp, xs = _rows(x, "x", io)
    rc = lm_lib.add_rms_norm_fwd(xp, xs, _ptr(residual, "residual", rdt), _ptr(weight, "weight", f32=True), eps,
                                 _OUT_KINDS[out], _ptr(y, "y"), _ptr(s, "s"), _ptr(scale, "scale"), _ptr(rs, "rstd"),
                                 rows, width, _dtype_code(x), _dtype_code(s), _stream(stream))
    _check(rc, "add_rms_norm_fwd")
    saved = (rs, x, residual) if residual is not None and rdt != torch.float32 else rs
    return (y, s) + ((scale,) if scale is not None else ()) + ((saved,) if rstd else ())


def add_rms_norm_bwd_workspace_bytes(rows: int, width: int) -> int:
    return int(lm_lib.add_rms_norm_bwd_workspace_bytes(rows, width))


@_on_launch_stream
def add_rms_norm_bwd(dy, s, weight, rstd, x_dtype=None, dresidual_out=None, workspace=None, stream=None):
    """Gradients of add_rms_norm_fwd's "io" output: dy [rows, width]; s and rstd (its rstd=True result, as it is)
    from the forward; dresidual_out the gradient that reaches s by the residual path (None: none).  Returns a dict: dx (x_dtype, which is dy's),
    dresidual (the same numbers in s's dtype; dx itself where the dtypes agree) and dweight (fp32 [width])."""
    torch = _torch()
    rows, width = dy.shape
    io = dy.dtype
    if x_dtype not in (None, io):
        raise TypeError("dy must have x's dtype")
    base, x = s, None
    if isinstance(rstd, tuple):
        rstd, x, base = rstd
        _shape_check("x", x, (rows, width))
        _shape_check("residual", base, (rows, width))
    xp, xs = _rows(x, "x", io)
    for n_, t_, s_ in (("s", s, (rows, width)), ("weight", weight, (width,)), ("rstd", rstd, (rows,)),
                       ("dresidual_out", dresidual_out, (rows, width))):
        _shape_check(n_, t_, s_)
    g = {"dx": torch.empty(rows, width, dtype=io, device=dy.device),
         "dresidual": torch.empty_like(s) if s.dtype != io else None,
         "dweight": torch.empty(width, dtype=torch.float32, device=dy.device)}
    ws, wsb, _keep = _workspace(add_rms_norm_bwd_workspace_bytes(rows, width), workspace, dy.device)
    rc = lm_lib.add_rms_norm_bwd(_ptr(dy, "dy"), _ptr(base, "s", s.dtype), xp, xs, _ptr(weight, "weight", f32=True),
                                 _ptr(rstd, "rstd", f32=True), _ptr(dresidual_out, "dresidual_out", s.dtype),
                                 _ptr(g["dx"], "dx"), _ptr(g["dresidual"], "dresidual"), _ptr(g["dweight"], "dweight"),
                                 rows, width, _dtype_code(dy), _dtype_code(s), ws, wsb, _stream(stream))
    _check(rc, "add_rms_norm_bwd")
    if g["dresidual"] is None:
        g["dresidual"] = g["dx"]
    return g


def token_logprobs_workspace_bytes(rows: int, vocab: int, top: int = 0) -> int:
    return int(lm_lib.token_logprobs_workspace_bytes(rows, vocab, top))


@_on_launch_stream
def token_logprobs_fwd(logits, targets, top=0, scale=1.0, workspace=None, stream=None):
    """Log probability of targets (int64 [rows]; outside [0, vocab): 0) under softmax(scale * logits), logits
    [rows, vocab], and the entropy.  Returns (logprob, entropy, stats), fp32 [rows], [rows] and [rows, 2]
    (the largest logit; log sum exp of scale * (logits - it)), and with top > 0 also (top_logprob fp32,
    top_index int64), [rows, top], largest first, equal logits by index."""
    torch = _torch()
    rows, vocab = logits.shape
    io = logits.dtype
    _shape_check("targets", targets, (rows,))
    f32 = dict(dtype=torch.float32, device=logits.device)
    out = [torch.empty(rows, **f32), torch.empty(rows, **f32), torch.empty(rows, 2, **f32)]
    if top:
        out += [torch.empty(rows, top, **f32), torch.empty(rows, top, dtype=torch.int64, device=logits.device)]
    val, idx = out[3:] if top else (None, None)
    ws, wsb, _keep = _workspace(token_logprobs_workspace_bytes(rows, vocab, top), workspace, logits.device)
    xp, xs = _rows(logits, "logits", io)
    rc = lm_lib.token_logprobs_fwd(xp, xs, _typed(targets, "targets", torch.int64), scale, top, _ptr(out[0], "logprob"),
                                   _ptr(out[1], "entropy"), _ptr(out[2], "stats"), _ptr(val, "top_logprob"),
                                   _ptr(idx, "top_index"), rows, vocab, _dtype_code(logits), ws, wsb, _stream(stream))
    _check(rc, "token_logprobs_fwd")
    return tuple(out)


@_on_launch_stream
def token_logprobs_bwd(logits, targets, stats, entropy, dlogprob=None, dentropy=None, scale=1.0, stream=None):
    """Gradient of sum(dlogprob * logprob + dentropy * entropy) for the logits (contiguous, their dtype); stats and
    entropy from token_logprobs_fwd with the same scale; dlogprob, dentropy fp32 [rows], one at least."""
    torch = _torch()
    rows, vocab = logits.shape
    io = logits.dtype
    for n_, t_ in (("targets", targets), ("entropy", entropy), ("dlogprob", dlogprob), ("dentropy", dentropy)):
        _shape_check(n_, t_, (rows,))
    _shape_check("stats", stats, (rows, 2))
    dx = torch.empty(rows, vocab, dtype=io, device=logits.device)
    xp, xs = _rows(logits, "logits", io)
    rc = lm_lib.token_logprobs_bwd(xp, xs, _typed(targets, "targets", torch.int64), _ptr(stats, "stats", f32=True),
                                   _ptr(entropy, "entropy", f32=True), _ptr(dlogprob, "dlogprob", f32=True),
                                   _ptr(dentropy, "dentropy", f32=True), scale, _ptr(dx, "dlogits"), rows, vocab,
                                   _dtype_code(logits), _stream(stream))
    _check(rc, "token_logprobs_bwd")
    return dx


@_on_launch_stream
def w4_matvec(x, qweight, scales, zeros=None, group=128, bias=None, out=None, stream=None):
    """x [rows, k] times the transpose of a 4-bit matrix: qweight uint8 [n, k // 2] (q[2i] in the low, q[2i+1] in the
    high bits of byte i), weight (q - zero) * scale with scales bf16 and zeros uint8 (None: 8), [n, k // group]
    each; bias fp32 [n].  Returns [rows, n] in x's dtype."""
    torch = _torch()
    rows, k = x.shape
    n = qweight.shape[0]
    io = x.dtype
    if group <= 0 or k % group:
        raise ValueError(f"group {group} does not divide k = {k}")
    for n_, t_, s_ in (("qweight", qweight, (n, k // 2)), ("scales", scales, (n, k // group)),
                       ("zeros", zeros, (n, k // group)), ("bias", bias, (n,))):
        _shape_check(n_, t_, s_)
    if out is None:
        out = torch.empty(rows, n, dtype=io, device=x.device)
    _shape_check("out", out, (rows, n))
    xp, xs = _rows(x, "x", io)
    rc = lm_lib.w4_matvec(xp, xs, _typed(qweight, "qweight", torch.uint8), _typed(scales, "scales", torch.bfloat16),
                          _typed(zeros, "zeros", torch.uint8), _ptr(bias, "bias", f32=True), _ptr(out, "out", io), rows, n,
                          k, group, _dtype_code(x), _stream(stream))
    _check(rc, "w4_matvec")
    return out

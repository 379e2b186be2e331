"""CPU tests of libselscan_lm's C ABI: it exports what include/selscan_lm.h declares and refuses bad arguments
on the host before any HIP call (every call here returns from validation; pointers are never followed)."""
import re
import subprocess

import pytest

import selective_state_space_51_amd as S

L = S.lm_lib
P = 0x10000
MB = 1 << 20
OK, NULL, SHAPE, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = range(7)


def test_exports_every_declared_symbol():
    text = open(S.LM_HEADER).read()
    declared = set(re.findall(r"^(?:int|size_t|const char \*)\s*\**\s*(\w+)\s*\(", text, re.M))
    out = subprocess.run(["nm", "-D", "--defined-only", S.LM_LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert declared and declared <= exported
    assert S.lm_abi_version() == 1
    assert all(hasattr(L, n) for n in declared)


def conv(x=P, xs=64, w=P + MB, b=None, cu=P + 2 * MB, slots=None, carry=None, st=P + 3 * MB, flags=4, out=P + 4 * MB,
         tokens=10, nseq=3, nslots=3, dim=64, width=4, dt=1):
    return L.causal_conv1d_packed_fwd(x, xs, w, b, cu, slots, carry, st, flags, out, tokens, nseq, nslots, dim, width, dt, None)


def test_conv_packed_refusals():
    for kw in ("x", "w", "cu", "out"):
        assert conv(**{kw: None}) == NULL, kw
    for kw in ("tokens", "nseq", "nslots", "dim"):
        assert conv(**{kw: -1}) == SHAPE, kw
    assert conv(xs=63) == SHAPE
    assert conv(nslots=2) == SHAPE  # no slots: sequence s is on entry s
    assert conv(nseq=0) == SHAPE  # tokens without a sequence
    assert conv(nseq=0, tokens=0, x=None) == OK and conv(dim=0, x=None) == OK
    assert conv(width=5) == UNSUPPORTED and conv(width=0) == UNSUPPORTED
    assert conv(dt=2) == UNSUPPORTED and conv(flags=1) == UNSUPPORTED
    assert conv(tokens=1 << 31) == UNSUPPORTED
    assert conv(x=P + 1) == ALIGN and conv(w=P + MB + 2) == ALIGN and conv(cu=P + 2 * MB + 1) == ALIGN
    assert conv(st=P + 3 * MB + 1) == ALIGN and conv(b=P + 5 * MB + 2) == ALIGN and conv(slots=P + 5 * MB + 2) == ALIGN
    assert conv(out=P + 16) == ALIAS and conv(st=P + 128) == ALIAS and conv(st=P + 4 * MB) == ALIAS
    assert conv(out=P + 2 * 64, xs=128) == ALIAS  # between the columns of strided rows


def step(x=P, xs=64, w=P + MB, slots=None, st=P + 3 * MB, flags=4, out=P + 4 * MB, rows=3, nslots=3, dim=64, width=4, dt=1):
    return L.causal_conv1d_step(x, xs, w, None, slots, st, flags, out, rows, nslots, dim, width, dt, None)


def test_conv_step_refusals():
    for kw in ("x", "w", "st", "out"):
        assert step(**{kw: None}) == NULL, kw
    assert step(rows=-1) == SHAPE and step(nslots=2) == SHAPE and step(xs=8) == SHAPE
    assert step(rows=0, x=None) == OK
    assert step(width=6) == UNSUPPORTED
    assert step(out=P) == ALIAS


def scan(x=P, d=P + MB, A=P + 2 * MB, B=P + 3 * MB, C=P + 4 * MB, bcs=32, D=None, z=None, zs=64, bias=None, flags=0,
         cu=P + 5 * MB, slots=None, carry=None, h=P + 6 * MB, y=P + 7 * MB, tokens=1000, nseq=2, nslots=2, longest=1000,
         dim=64, N=16, dt=1, ws=P + 16 * MB, wsb=1 << 24):
    return L.selscan_packed_fwd(x, d, A, B, C, bcs, D, z, zs, bias, flags, cu, slots, carry, h, y, tokens, nseq, nslots,
                                longest, dim, N, dt, ws, wsb, None)


def test_scan_packed_refusals():
    for kw in ("x", "d", "A", "B", "C", "cu", "y"):
        assert scan(**{kw: None}) == NULL, kw
    for kw in ("tokens", "nseq", "nslots", "dim", "longest", "N"):
        assert scan(**{kw: -1}) == SHAPE, kw
    assert scan(bcs=15) == SHAPE and scan(z=P + 8 * MB, zs=63) == SHAPE and scan(nslots=1) == SHAPE
    assert scan(nseq=0) == SHAPE and scan(nseq=0, tokens=0) == OK and scan(dim=0) == OK
    assert scan(N=8) == UNSUPPORTED and scan(dt=3) == UNSUPPORTED and scan(flags=4) == UNSUPPORTED
    far = (1 << 26) + 1  # 16 rows of a longer stride do not lie within 32 bits
    assert scan(dim=far) == UNSUPPORTED and scan(bcs=far) == UNSUPPORTED and scan(z=P + 8 * MB, zs=far) == UNSUPPORTED
    assert scan(A=P + 2 * MB + 2) == ALIGN and scan(h=P + 6 * MB + 4) == ALIGN and scan(B=P + 3 * MB + 1) == ALIGN
    need = S.selscan_packed_workspace_bytes(1000, 2, 1000, 64)
    assert need > 0
    assert scan(wsb=need - 1) == WORKSPACE and scan(ws=None) == WORKSPACE and scan(ws=P + 16 * MB + 4) == ALIGN
    assert scan(y=P + 2) == ALIAS and scan(h=P + MB) == ALIAS and scan(ws=P + 7 * MB) == ALIAS
    assert S.selscan_packed_workspace_bytes(0, 2, 10, 64) == 0
    assert S.selscan_packed_workspace_bytes(64, 2, 32, 64) == 0


def sstep(x=P, d=P + MB, A=P + 2 * MB, B=P + 3 * MB, C=P + 4 * MB, bcs=32, z=None, zs=64, slots=None, h=P + 6 * MB,
          y=P + 7 * MB, rows=3, nslots=3, dim=64, N=16, dt=1, flags=0):
    return L.selscan_step(x, d, A, B, C, bcs, None, z, zs, None, flags, slots, h, y, rows, nslots, dim, N, dt, None)


def test_scan_step_refusals():
    for kw in ("x", "d", "A", "B", "C", "h", "y"):
        assert sstep(**{kw: None}) == NULL, kw
    assert sstep(rows=-1) == SHAPE and sstep(nslots=2) == SHAPE and sstep(bcs=8) == SHAPE
    assert sstep(N=4) == UNSUPPORTED and sstep(flags=8) == UNSUPPORTED
    assert sstep(h=P + 6 * MB + 8) == ALIGN
    assert sstep(y=P) == ALIAS and sstep(h=P + 64) == ALIAS
    assert sstep(rows=0) == OK


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        S.causal_conv1d_step(x, torch.zeros(8, 4), torch.zeros(4, 3, 8))
    with pytest.raises(ValueError, match="shape"):
        S.selscan_step(x, torch.zeros(4, 9), torch.zeros(8, 16), torch.zeros(4, 16), torch.zeros(4, 16), torch.zeros(4, 8, 16))
    with pytest.raises(ValueError, match="shape"):
        S.causal_conv1d_packed_fwd(x, torch.zeros(8, 4), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, 8))


def norm(x=P, xs=64, res=P + MB, w=P + 2 * MB, eps=1e-5, kind=0, y=P + 3 * MB, ro=P + 4 * MB, scale=None, rstd=None,
         rows=8, width=64, dt=1, rdt=0):
    return L.add_rms_norm_fwd(x, xs, res, w, eps, kind, y, ro, scale, rstd, rows, width, dt, rdt, None)


def test_norm_refusals():
    for kw in ("x", "w", "y"):
        assert norm(**{kw: None}) == NULL, kw
    assert norm(kind=1) == NULL  # an 8-bit output needs its scales
    assert norm(rows=-1) == SHAPE and norm(width=-1) == SHAPE and norm(xs=63) == SHAPE
    assert norm(rows=0, x=None) == OK and norm(width=0) == OK
    assert norm(kind=3) == UNSUPPORTED and norm(dt=2) == UNSUPPORTED and norm(dt=0, rdt=1) == UNSUPPORTED
    assert norm(width=32769, xs=32769) == UNSUPPORTED
    for eps in (-1e-5, float("nan"), float("inf")):
        assert norm(eps=eps) == UNSUPPORTED
    assert norm(x=P + 1) == ALIGN and norm(res=P + MB + 2) == ALIGN and norm(w=P + 2 * MB + 1) == ALIGN
    assert norm(y=P) == ALIAS and norm(ro=P + MB + 64) == ALIAS and norm(rstd=P + 3 * MB) == ALIAS
    assert norm(ro=P + 16) == ALIAS


def norm_bwd(dy=P, s=P + MB, x=None, xs=64, w=P + 2 * MB, rstd=P + 3 * MB, dres=None, dx=P + 4 * MB, dr=P + 5 * MB, dw=P + 6 * MB, rows=8,
             width=64, dt=1, rdt=0, ws=P + 7 * MB, wsb=MB):
    return L.add_rms_norm_bwd(dy, s, x, xs, w, rstd, dres, dx, dr, dw, rows, width, dt, rdt, ws, wsb, None)


def test_norm_bwd_refusals():
    for kw in ("dy", "s", "w", "rstd"):
        assert norm_bwd(**{kw: None}) == NULL, kw
    assert norm_bwd(rows=-1) == SHAPE and norm_bwd(dt=9) == UNSUPPORTED and norm_bwd(x=P + 9 * MB, xs=63) == SHAPE
    assert norm_bwd(x=P + 9 * MB + 1) == ALIGN and norm_bwd(x=P + 4 * MB) == ALIAS
    assert norm_bwd(rows=0, dw=None) == OK
    need = S.add_rms_norm_bwd_workspace_bytes(8, 64)
    assert need == 8 * 64 * 4 and S.add_rms_norm_bwd_workspace_bytes(0, 64) == 0
    assert norm_bwd(wsb=need - 1) == WORKSPACE and norm_bwd(ws=None) == WORKSPACE
    assert norm_bwd(ws=P + 7 * MB + 4) == ALIGN and norm_bwd(s=P + MB + 2) == ALIGN
    assert norm_bwd(dx=P) == ALIAS and norm_bwd(dr=P + 4 * MB) == ALIAS and norm_bwd(ws=P + 6 * MB) == ALIAS


def lp_fwd(x=P, xs=100, t=P + MB, scale=1.0, top=0, lp=P + 2 * MB, ent=P + 3 * MB, st=P + 4 * MB, tv=None, ti=None, rows=4,
           vocab=100, dt=1, ws=P + 5 * MB, wsb=MB):
    return L.token_logprobs_fwd(x, xs, t, scale, top, lp, ent, st, tv, ti, rows, vocab, dt, ws, wsb, None)


def test_logprobs_refusals():
    for kw in ("x", "t", "lp", "ent", "st"):
        assert lp_fwd(**{kw: None}) == NULL, kw
    assert lp_fwd(top=3) == NULL
    assert lp_fwd(rows=-1) == SHAPE and lp_fwd(vocab=-1) == SHAPE and lp_fwd(xs=99) == SHAPE
    assert lp_fwd(vocab=0) == SHAPE and lp_fwd(rows=0) == OK
    assert lp_fwd(top=30, vocab=20, tv=P + 6 * MB, ti=P + 7 * MB) == SHAPE
    assert lp_fwd(top=33) == UNSUPPORTED and lp_fwd(top=-1) == UNSUPPORTED and lp_fwd(dt=4) == UNSUPPORTED
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert lp_fwd(scale=s) == UNSUPPORTED
    assert lp_fwd(t=P + MB + 4) == ALIGN and lp_fwd(x=P + 1) == ALIGN
    assert S.token_logprobs_workspace_bytes(4, 100, 0) == 0  # one workgroup takes a whole row
    big = dict(vocab=90_000, xs=90_000, x=P + 100 * MB)
    need = S.token_logprobs_workspace_bytes(4, 90_000, 0)
    assert need > 0 and lp_fwd(**big, wsb=need - 1) == WORKSPACE and lp_fwd(**big, ws=None) == WORKSPACE
    assert lp_fwd(**big, ws=P + 5 * MB + 8) == ALIGN and lp_fwd(**big, ws=P + 4 * MB) == ALIAS
    assert lp_fwd(lp=P + 8) == ALIAS and lp_fwd(ent=P + 2 * MB) == ALIAS


def lp_bwd(x=P, xs=100, t=P + MB, st=P + 2 * MB, ent=P + 3 * MB, dl=P + 4 * MB, dh=None, scale=1.0, dx=P + 5 * MB, rows=4,
           vocab=100, dt=1):
    return L.token_logprobs_bwd(x, xs, t, st, ent, dl, dh, scale, dx, rows, vocab, dt, None)


def test_logprobs_bwd_refusals():
    for kw in ("x", "t", "st", "ent", "dl", "dx"):
        assert lp_bwd(**{kw: None}) == NULL, kw
    assert lp_bwd(rows=0) == OK and lp_bwd(vocab=0) == OK
    assert lp_bwd(xs=10) == SHAPE and lp_bwd(scale=0.0) == UNSUPPORTED
    assert lp_bwd(dx=P + 1) == ALIGN and lp_bwd(dx=P) == ALIAS


def w4(x=P, xs=256, q=P + MB, s=P + 2 * MB, z=None, b=None, y=P + 4 * MB, rows=2, n=64, k=256, group=64, dt=1):
    return L.w4_matvec(x, xs, q, s, z, b, y, rows, n, k, group, dt, None)


def test_w4_refusals():
    for kw in ("x", "q", "s", "y"):
        assert w4(**{kw: None}) == NULL, kw
    assert w4(rows=-1) == SHAPE and w4(k=0) == SHAPE and w4(k=96) == SHAPE and w4(xs=255) == SHAPE
    assert w4(rows=0) == OK and w4(n=0) == OK
    assert w4(group=16) == UNSUPPORTED and w4(dt=5) == UNSUPPORTED
    assert w4(q=P + MB + 8) == ALIGN and w4(s=P + 2 * MB + 1) == ALIGN and w4(b=P + 3 * MB + 2) == ALIGN
    assert w4(y=P) == ALIAS and w4(y=P + MB) == ALIAS and w4(z=P + 4 * MB + 16) == ALIAS

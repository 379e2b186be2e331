"""CPU tests of the C ABI of linear attention, sampling and cache moves: bad arguments are refused on the host before any HIP
call (every call here returns from validation; the addresses are never followed), and so are bad tensors by the binding."""
import ctypes

import pytest

import selective_state_space_51_amd as S

L = S.lm_lib
P = 0x10000
MB = 1 << 20
OK, NULL, SHAPE, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = range(7)
A = lambda i: (i + 1) << 50  # arrays far from one another


def packed(q=A(0), qs=128, k=A(1), ks=128, v=A(2), vs=256, g=A(3), gs=4, scale=1.0, cu=A(4), slots=None, carry=None, state=A(5),
           out=A(6), tokens=10, nseq=3, nslots=3, longest=10, heads=4, groups=2, dk=64, dv=64, dt=1, ws=A(7), wsb=1 << 40):
    return L.linear_attn_packed_fwd(q, qs, k, ks, v, vs, g, gs, scale, cu, slots, carry, state, out, tokens, nseq, nslots, longest,
                                    heads, groups, dk, dv, dt, ws, wsb, None)


def test_linear_attn_packed_refusals():
    for kw in ("q", "k", "v", "g", "cu", "out"):
        assert packed(**{kw: None}) == NULL, kw
    for kw in ("tokens", "nseq", "nslots", "longest", "heads", "groups", "dk", "dv"):
        assert packed(**{kw: -1}) == SHAPE, kw
    assert packed(qs=127) == SHAPE and packed(ks=127) == SHAPE and packed(vs=255) == SHAPE and packed(gs=3) == SHAPE
    assert packed(groups=3) == SHAPE and packed(groups=0) == SHAPE and packed(dk=0) == SHAPE
    assert packed(nslots=2) == SHAPE and packed(nseq=0) == SHAPE
    assert packed(nseq=0, tokens=0) == OK and packed(heads=0) == OK and packed(dv=0) == OK
    assert packed(dk=257, qs=600, ks=600) == UNSUPPORTED and packed(dv=1025, vs=5000) == UNSUPPORTED and packed(dt=2) == UNSUPPORTED
    for scale in (float("nan"), float("inf")):
        assert packed(scale=scale) == UNSUPPORTED
    far = (1 << 26) + 1
    assert packed(qs=far) == UNSUPPORTED and packed(ks=far) == UNSUPPORTED and packed(vs=far) == UNSUPPORTED and packed(gs=far) == UNSUPPORTED
    assert packed(tokens=(1 << 31) - 1) == UNSUPPORTED
    assert packed(q=A(0) + 1) == ALIGN and packed(g=A(3) + 2) == ALIGN and packed(state=A(5) + 4) == ALIGN and packed(cu=A(4) + 2) == ALIGN
    assert packed(out=A(0)) == ALIAS and packed(state=A(2)) == ALIAS and packed(out=A(5) + 64) == ALIAS and packed(out=A(3)) == ALIAS


def test_linear_attn_workspace():
    need = S.linear_attn_packed_workspace_bytes(20000, 1, 20000, 4, 64, 64)
    assert need > 0 and S.linear_attn_packed_workspace_bytes(64, 1, 64, 4, 64, 64) == 0
    big = dict(tokens=20000, nseq=1, nslots=1, longest=20000)
    assert packed(**big, wsb=need - 1) == WORKSPACE and packed(**big, ws=None) == WORKSPACE and packed(**big, ws=A(7) + 8) == ALIGN
    assert packed(**big, ws=A(6)) == ALIAS
    # what is kept of segments is kept of those that another follows: sequences do not count
    assert need == S.linear_attn_packed_workspace_bytes(20000, 5000, 20000, 4, 64, 64)
    for bad in ((0, 1, 10, 4, 64, 64), (10, 0, 10, 4, 64, 64), (10, 1, 0, 4, 64, 64), (10, 1, 10, 0, 64, 64), (10, 1, 10, 4, 0, 64),
                (10, 1, 10, 4, 64, 0), (10, 1, 10, 4, 300, 64), (-5, -5, -5, -5, -5, -5), (20000, 1, 20000, 4, 64, 64, 7)):
        assert S.linear_attn_packed_workspace_bytes(*bad) == 0


def step(q=A(0), qs=128, k=A(1), ks=128, v=A(2), vs=256, g=A(3), gs=4, scale=1.0, slots=None, state=A(5), out=A(6), rows=3, nslots=3,
         heads=4, groups=2, dk=64, dv=64, dt=1):
    return L.linear_attn_step(q, qs, k, ks, v, vs, g, gs, scale, slots, state, out, rows, nslots, heads, groups, dk, dv, dt, None)


def test_linear_attn_step_refusals():
    for kw in ("q", "k", "v", "g", "state", "out"):
        assert step(**{kw: None}) == NULL, kw
    assert step(rows=-1) == SHAPE and step(nslots=2) == SHAPE and step(groups=3) == SHAPE and step(vs=255) == SHAPE
    assert step(rows=0) == OK and step(heads=0) == OK
    assert step(dk=300, qs=600, ks=600) == UNSUPPORTED and step(dt=7) == UNSUPPORTED
    assert step(state=A(5) + 8) == ALIGN and step(out=A(1)) == ALIAS and step(state=A(3)) == ALIAS
    assert step(rows=1 << 30, slots=A(8), nslots=10) == UNSUPPORTED  # past what a launch holds


def sample(x=A(0), xs=100, u=A(1), t=None, t_=1.0, k=None, k_=0, p=None, p_=1.0, m=None, m_=0.0, tok=A(2), lp=A(3), kept=A(4),
           rows=4, vocab=100, dt=1):
    return L.token_sample(x, xs, u, t, t_, k, k_, p, p_, m, m_, tok, lp, kept, rows, vocab, dt, None)


def test_sample_refusals():
    for kw in ("x", "u", "tok", "lp", "kept"):
        assert sample(**{kw: None}) == NULL, kw
    assert sample(rows=-1) == SHAPE and sample(vocab=-1) == SHAPE and sample(xs=99) == SHAPE and sample(vocab=0) == SHAPE
    assert sample(rows=0) == OK
    assert sample(vocab=(1 << 21) + 1, xs=1 << 22) == UNSUPPORTED and sample(dt=3) == UNSUPPORTED
    nan, inf = float("nan"), float("inf")
    for t in (-1.0, nan, inf):
        assert sample(t_=t) == UNSUPPORTED
    assert sample(k_=-1) == UNSUPPORTED
    for q in (-0.1, 1.1, nan):
        assert sample(p_=q) == UNSUPPORTED and sample(m_=q) == UNSUPPORTED
    for kw, at in (("t", A(5)), ("k", A(5)), ("p", A(5)), ("m", A(5)), ("u", A(1)), ("lp", A(3)), ("kept", A(4))):
        assert sample(**{kw: at + 2}) == ALIGN, kw
    assert sample(tok=A(2) + 4) == ALIGN and sample(x=A(0) + 1) == ALIGN
    assert sample(lp=A(2)) == ALIAS and sample(kept=A(0)) == ALIAS and sample(t=A(3)) == ALIAS
    assert sample(rows=1 << 24) == UNSUPPORTED


def copy(caches=(A(0), A(1)), sizes=(1000, 64), src=A(2), dst=A(3), n=5, nslots=10, count=None):
    c = None if caches is None else (ctypes.c_void_p * len(caches))(*caches)
    b = None if sizes is None else (ctypes.c_int64 * len(sizes))(*sizes)
    return L.cache_entries_copy(c, b, len(caches or sizes) if count is None else count, src, dst, n, nslots, None)


def test_cache_copy_refusals():
    assert copy(caches=None) == NULL and copy(sizes=None) == NULL and copy(src=None) == NULL and copy(dst=None) == NULL
    assert copy(caches=(A(0), None)) == NULL
    assert copy(n=-1) == SHAPE and copy(nslots=-1) == SHAPE and copy(count=-1) == SHAPE and copy(sizes=(1000, -1)) == SHAPE
    assert copy(n=0) == OK and copy(nslots=0) == OK and copy(count=0) == OK and copy(caches=(None, None), sizes=(0, 0)) == OK
    assert copy(n=16385) == UNSUPPORTED and copy(sizes=((1 << 32) + 1, 64)) == UNSUPPORTED
    assert copy(src=A(2) + 2) == ALIGN and copy(dst=A(3) + 1) == ALIGN
    assert copy(caches=(A(0), A(0) + 9999)) == ALIAS and copy(src=A(0) + 100) == ALIAS and copy(dst=A(1)) == ALIAS
    assert copy(sizes=(1 << 32, 64), n=16000) == UNSUPPORTED  # past what a launch holds


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    q, v, g, st = torch.zeros(4, 2, 8), torch.zeros(4, 4, 6), torch.zeros(4, 4), torch.zeros(4, 4, 8, 6)
    with pytest.raises(ValueError, match="device tensor"):
        S.linear_attn_step(q, q.clone(), v, g, st)
    with pytest.raises(ValueError, match="state has shape"):
        S.linear_attn_step(q, q.clone(), v, g, torch.zeros(4, 4, 6, 8))
    with pytest.raises(ValueError, match="log_decay has shape"):
        S.linear_attn_step(q, q.clone(), v, torch.zeros(4, 3), st)
    with pytest.raises(ValueError, match="do not divide"):
        S.linear_attn_step(torch.zeros(4, 3, 8), torch.zeros(4, 3, 8), v, g, st)
    with pytest.raises(ValueError, match="k has shape"):
        S.linear_attn_packed_fwd(q, torch.zeros(4, 2, 9), v, g, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="uniform has shape"):
        S.token_sample(torch.zeros(3, 9), torch.zeros(4))
    with pytest.raises(ValueError, match="dst has shape"):
        S.cache_entries_copy(torch.zeros(3, 9), torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        S.cache_entries_copy([torch.zeros(3, 9)], torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    assert S.cache_entries_copy([], torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)) is None

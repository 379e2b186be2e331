"""GPU tests of add_rms_norm_fwd and add_rms_norm_bwd against the same formulas in 64 bits.

Bars, from the arithmetic.  u = 2^-24.  A row's sum of squares, added in 32 bits in chains of at most 32
fused steps, then 6 + 16 across lanes and waves, would be off by at most 54 u, half of it in rstd (it is added in 64 bits); y adds three
roundings, so |y - exact| <= 32 u |y| (2e-6) in fp32, plus half an ulp (2^-8 |y|, bf16 having 8 significant bits) where it is rounded to bf16.
8-bit outputs add half a step of their grid.  ds = rstd (g - xhat mean(g xhat)): the mean carries 54 u of
mean|g xhat|, every other factor a few u.  dweight adds rows_per + 64 terms in order: that many u of the sum of
magnitudes."""
import sys

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _torch():
    import torch
    return torch


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def make(rows, width, dtype, res, seed=0, pad=0):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * rows + width)
    io = torch.bfloat16 if dtype == "bf16" else torch.float32
    rdt = torch.float32 if res == "f32" else io
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return dict(x=rn(rows, width + pad).to(io)[:, :width], r=(2 * rn(rows, width)).to(rdt), w=1 + 0.3 * rn(width),
                dy=rn(rows, width).to(io), dres=rn(rows, width).to(rdt))


def half_ulp(t):
    """Rounding to t's type, relative."""
    return 2.0 ** -8 if t.dtype == _torch().bfloat16 else 0.0


def within(name, got, want, bar):
    torch = _torch()
    d = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), name
    over = d - bar
    assert float(over.max()) <= 0, (name, float(d.max()), float(over.max()))


def forward64(i, eps):
    torch = _torch()
    s = i["x"].double() + (i["r"].double() if i["r"] is not None else 0)
    rstd = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s, rstd, s * rstd * i["w"].double()


WIDTHS = [1, 7, 8, 100, 512, 520, 1001, 1024, 2048, 2049, 4096, 5000, 8192, 10001, 16384, 20000, 32768]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,res", [("bf16", "f32"), ("bf16", "io"), ("f32", "f32")])
def test_forward(width, dtype, res):
    import selective_state_space_51_amd as S
    torch = _torch()
    eps = 1e-5
    for rows, pad in ((1, 0), (5, 8), (66, 3)):
        _say("norm fwd", width, dtype, res, rows, pad)
        i = make(rows, width, dtype, res, pad=pad)
        s, rstd, y = forward64(i, eps)
        got, so, rs = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], eps=eps, rstd=True)
        rs = rs[0] if isinstance(rs, tuple) else rs
        assert torch.equal(so, (i["x"].float() + i["r"].float()).to(i["r"].dtype))
        # the fp32 sum of x and residual is rounded before it is normed: 1 u of |s|, which u |y| covers; 2^-40: tiny y
        within("y", got, y, (34 * U + half_ulp(got) * (1 + 64 * U)) * y.abs() + 2.0 ** -40)
        within("rstd", rs[:, None], rstd, 32 * U * rstd)
        for kind, top in (("int8", 127.0), ("fp8", 448.0)):
            q, so2, sc = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], eps=eps, out=kind)
            assert torch.equal(so, so2)
            step = y.abs().amax(1, keepdim=True) / top
            within(kind + " scale", sc[:, None], step, 36 * U * step)
            back = q.double() * sc.double()[:, None]
            if kind == "int8":
                bar = step * (0.5 + 127 * 80 * U)
            else:  # 3 bits after the leading one: half a step is 2^-4 of the value, 2^-10 of the smallest normal's grid
                bar = torch.maximum(y.abs() * 2.0 ** -4, step * 2.0 ** -10) * (1 + 1e-4)
            within(kind, back, y, bar)
            assert float(q.float().abs().max()) <= top


def test_no_residual_and_first_layer_types():
    import selective_state_space_51_amd as S
    torch = _torch()
    i = make(9, 768, "bf16", "f32")
    i["r"] = None
    _, _, y = forward64(i, 1e-6)
    got, s = S.add_rms_norm_fwd(i["x"], i["w"], eps=1e-6, residual_dtype=torch.float32)
    assert s.dtype == torch.float32 and torch.equal(s, i["x"].float())
    within("y", got, y, (34 * U + 2.0 ** -8 * 1.001) * y.abs() + 2.0 ** -40)
    got2, s2 = S.add_rms_norm_fwd(i["x"], i["w"], eps=1e-6)
    assert torch.equal(got, got2) and torch.equal(s2, i["x"])


def test_rows_that_hold_nothing_or_too_much():
    import selective_state_space_51_amd as S
    torch = _torch()
    inf, nan = float("inf"), float("nan")
    i = make(8, 640, "f32", "f32")
    i["r"].zero_()
    i["x"][1] = 0
    i["x"][2, 5] = nan
    i["x"][3, 639] = inf
    i["x"][4] *= 1e-30   # squares underflow: eps alone is left
    i["x"][5] *= 1e30    # squares overflow: rstd is 0
    i["x"][6] = 1e-40
    y, s, rs = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], rstd=True)
    assert torch.equal(s.nan_to_num(nan=7.0), i["x"].nan_to_num(nan=7.0))
    for r in (0, 7):
        assert torch.isfinite(y[r]).all() and float(y[r].abs().max()) > 0.1
    assert float(y[1].abs().max()) == 0
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 639])
    for r in (4, 5, 6):
        assert torch.isfinite(y[r]).all()
    for kind in ("int8", "fp8"):
        q, _, sc = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], out=kind)
        assert float(sc[1]) == 0 and float(q[1].float().abs().max()) == 0
        assert float(sc[6]) == 0 and float(q[6].float().abs().max()) == 0
        for r in (2, 3, 5):
            assert bool(torch.isnan(sc[r])) and float(q[r].float().abs().max()) == 0
        for r in (0, 4, 7):
            assert float(sc[r]) > 0 and float(q[r].float().abs().max()) == (127 if kind == "int8" else 448)


def backward64(i, s, rstd, dres=True):
    xh = s * rstd
    g = i["dy"].double() * i["w"].double()
    m = (g * xh).mean(1, keepdim=True)
    ds = rstd * (g - xh * m)
    if dres:
        ds = ds + i["dres"].double()
    dw = (i["dy"].double() * xh).sum(0)
    mags = (i["dy"].double() * xh).abs().sum(0)
    bar = rstd * (4 * g.abs() + (g * xh).abs().mean(1, keepdim=True) * xh.abs() * 64) * U + 2 * U * ds.abs()
    return ds, dw, mags, bar


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,res", [("bf16", "f32"), ("bf16", "io"), ("f32", "f32")])
def test_backward(width, dtype, res):
    import selective_state_space_51_amd as S
    torch = _torch()
    for rows in (1, 37, 4200 if width <= 1024 else 1100):
        _say("norm bwd", width, dtype, res, rows)
        i = make(rows, width, dtype, res, seed=3, pad=8 if rows == 37 else 0)
        _, s, rs = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], rstd=True)
        assert isinstance(rs, tuple) == (i["r"].dtype == torch.bfloat16)  # a rounded sum is formed anew
        s64 = i["x"].double() + i["r"].double()
        r64 = (rs[0] if isinstance(rs, tuple) else rs).double()[:, None]
        ds, dw, mags, bar = backward64(i, s64, r64)
        g = S.add_rms_norm_bwd(i["dy"], s, i["w"], rs, dresidual_out=i["dres"])
        for k, t in (("dx", i["x"]), ("dresidual", i["r"])):
            assert g[k].dtype == t.dtype
            within(k, g[k], ds, bar + half_ulp(g[k]) * (ds.abs() + bar) + 2.0 ** -40)
        within("dweight", g["dweight"], dw, (5 + 72) * U * mags + 2.0 ** -40)
    g2 = S.add_rms_norm_bwd(i["dy"], s, i["w"], rs, dresidual_out=i["dres"])
    assert all(torch.equal(g[k], g2[k]) for k in g)
    ds, *_, bar = backward64(i, s64, r64, dres=False)
    g = S.add_rms_norm_bwd(i["dy"], s, i["w"], rs)
    within("dx alone", g["dx"], ds, bar + half_ulp(g["dx"]) * (ds.abs() + bar) + 2.0 ** -40)


def test_backward_against_differences():
    # directional derivative of sum(dy y) + sum(dres s) by central differences of the 64-bit forward.  The step
    # 1e-5 leaves 1e-10 of relative truncation and 1e-11 of rounding; the fp32 gradients carry 64 u of magnitudes
    import selective_state_space_51_amd as S
    torch = _torch()
    i = make(6, 300, "f32", "f32", seed=11)
    _, s, rs = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], rstd=True)
    g = S.add_rms_norm_bwd(i["dy"], s, i["w"], rs, dresidual_out=i["dres"])

    def loss(dx, dw):
        j = dict(i, x=i["x"].double() + dx, w=i["w"].double() + dw)
        s64, _, y = forward64(j, 1e-5)
        return float((y * i["dy"].double()).sum() + (s64 * i["dres"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(4):
        vx = torch.randn(6, 300, generator=gen, device="cuda", dtype=torch.float64)
        vw = torch.randn(300, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        num = (loss(h * vx, 0) - loss(-h * vx, 0)) / (2 * h)
        mag = float((g["dx"].double() * vx).abs().sum())
        assert abs(num - float((g["dx"].double() * vx).sum())) <= 70 * U * mag + 1e-6
        num = (loss(0, h * vw) - loss(0, -h * vw)) / (2 * h)
        mag = float((g["dweight"].double() * vw).abs().sum())
        assert abs(num - float((g["dweight"].double() * vw).sum())) <= 80 * U * 10 * mag + 1e-6


def test_empty_in_place_stream_graph():
    import selective_state_space_51_amd as S
    torch = _torch()
    i = make(33, 512, "bf16", "f32")
    e = i["x"][:0]
    y, s = S.add_rms_norm_fwd(e, i["w"], residual=i["r"][:0])
    assert y.shape == (0, 512)
    g = S.add_rms_norm_bwd(e, s, i["w"], torch.empty(0, device="cuda"))
    assert float(g["dweight"].abs().max()) == 0 and g["dx"].shape == (0, 512)
    # the C entry writes the sum over the residual where asked to
    want, so = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"])
    r = i["r"].clone()
    y = torch.empty_like(want)
    rc = S.lm_lib.add_rms_norm_fwd(i["x"].data_ptr(), 512, r.data_ptr(), i["w"].data_ptr(), 1e-5, 0, y.data_ptr(), r.data_ptr(),
                                   None, None, 33, 512, S.SELSCAN_BF16, S.SELSCAN_F32, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(r, so) and torch.equal(y, want)

    def work():
        y, s, rs = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], rstd=True)
        q, _, sc = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], out="int8")
        g = S.add_rms_norm_bwd(i["dy"], s, i["w"], rs, dresidual_out=i["dres"])
        return [y, s, rs, q, sc, g["dx"], g["dresidual"], g["dweight"]]

    eager = [t.clone() for t in work()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, _ = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], stream=side)
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    assert torch.equal(y2, eager[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = work()
    for _ in range(3):
        for t in cap:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cap, eager))


@pytest.mark.parametrize("width", [5, 520, 1536, 5000, 20000, 32768])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rstd_is_rounded_four_times(width, dtype):
    """The squares are added in 64 bits, so rstd carries the roundings of mean, + eps, square root and reciprocal
    alone: (1/2 + 1/2 + 1 + 1) u, u^2 terms aside, at every width.  And the grid of an 8-bit output is its row's largest
    magnitude over 127 or 448: that element is the grid's last."""
    torch = _torch()
    import selective_state_space_51_amd as S
    _say("rstd", width, dtype)
    i = make(130, width, dtype, "f32", seed=11)
    s = (i["x"].float() + i["r"]).double()
    want = 1 / torch.sqrt((s * s).mean(1) + 1e-5)
    for out, top in (("int8", 127), ("fp8", 448)):
        y, _, scale, rstd = S.add_rms_norm_fwd(i["x"], i["w"], residual=i["r"], out=out, rstd=True)
        torch.cuda.synchronize()
        assert float(((rstd.double() - want) / want).abs().max()) <= 3.01 * U
        assert (y.float().abs().amax(1) == top).all()

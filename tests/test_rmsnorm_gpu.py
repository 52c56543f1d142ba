"""GPU tests of the residual RMS norm and its gradient against the float64 oracle.

Bounds. A row's mean of squares is a sum of at most 64 terms per thread and 10 levels of a
tree, each rounded once, so rstd is within 64 * 2^-24 relative; y and the 8-bit scales carry
that and at most four roundings more, y its own rounding to the output type. The magnitudes in
dx's bound are the oracle's (rmsnorm_bwd); dweight is a sum of N terms in fp32."""

import numpy as np
import pytest
import torch

from linear_cross_entropy_logits_gb300 import build as B
from linear_cross_entropy_logits_gb300 import flce
from oracle import ops_oracle as oo
from ops_util import DT, F32, FLOOR, ULP, close, np64, odd_rows, strided

pytestmark = pytest.mark.gpu
RSTD = 80 * F32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    flce.load()


def _rows(N, H, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, H, generator=g) * (0.1 + 3 * torch.rand(N, 1, generator=g))
    x[:, ::37] *= 12
    return x.to(DT[dt]), (torch.randn(N, H, generator=g) * 0.7).to(DT[dt]), (1 + 0.3 * torch.randn(H, generator=g)).to(DT[dt])


def _sum32(x, r):
    """h as the kernel has it: one fp32 addition."""
    h = x.float().numpy()
    return h + r.float().numpy() if r is not None else h


SHAPES = [(1, 1, "f32"), (1, 4096, "bf16"), (3, 128, "bf16"), (5, 130, "f16"), (4, 127, "f32"), (33, 256, "bf16"),
          (9, 2048, "f16"), (7, 1337, "f32"), (6, 5376, "bf16"), (2, 8192, "f32"), (3, 16384, "bf16"), (5, 4099, "bf16"),
          (2, 20000, "f16"), (2, 9001, "bf16"), (70, 64, "f32"), (1000, 520, "bf16"), (3, 8191, "f16"), (2, 8193, "f32"),
          (4, 5121, "f32"), (33, 1166, "bf16"), (5, 5122, "f32"), (3, 8190, "f16"), (2, 8194, "bf16"), (70, 66, "f16")]


@pytest.mark.parametrize("N,H,dt", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(N, H, dt, residual):
    x, r, w = _rows(N, H, dt, N + H)
    r = r if residual else None
    o = flce.rmsnorm_fwd(x.cuda(), w.cuda(), None if r is None else r.cuda(), eps=1e-5, weight_offset=0.25, want_h=True,
                         want_y8=True, want_h8=True)
    h32 = _sum32(x, r)
    h = h32.astype(np.float64)
    y, rstd = oo.rmsnorm_fwd(h, np64(w), 1e-5, 0.25)
    close(o["rstd"], rstd, RSTD * rstd)
    close(o["y"], y, (ULP[dt] + RSTD) * np.abs(y) + FLOOR[dt])
    assert torch.equal(o["h"].cpu(), torch.from_numpy(h32).to(DT[dt]))
    # the checkpoint of h: every bit
    q, s = oo.pack(h)
    assert np.array_equal(np64(o["h8"]), q) and np.array_equal(np64(o["h8_scale"]), s)
    # the 8-bit output: e4m3 of h * weight (fp32), its scale times rstd
    u = (h32 * (w.float().numpy() + np.float32(0.25))).astype(np.float64)
    q, s = oo.pack(u)
    assert np.array_equal(np64(o["y8"]), q)
    want = s * rstd[:, None]
    close(o["y8_scale"], want, (RSTD + F32) * want)


@pytest.mark.parametrize("dt,H,extra,offset", [("bf16", 136, 8, 8), ("bf16", 136, 1, 3), ("f32", 64, 4, 4), ("f16", 260, 3, 0),
                                               ("bf16", 136, 2, 2), ("f32", 66, 2, 6)])
def test_forward_strides_and_in_place(dt, H, extra, offset):
    N = 37
    x, r, w = _rows(N, H, dt, 5)
    xd, rd = strided(x.cuda(), extra, offset), strided(r.cuda(), extra, offset)
    outs = {"h": rd, "y": odd_rows(N, H, DT[dt], extra, offset),
            "y8": odd_rows(N, H, torch.float8_e4m3fn, extra, offset), "h8": odd_rows(N, H, torch.float8_e4m3fn, extra, offset)}
    a = flce.rmsnorm_fwd(xd, w.cuda(), rd, outputs=outs, want_y8=True, want_h8=True)     # h over the residual
    b = flce.rmsnorm_fwd(x.cuda(), w.cuda(), r.cuda(), want_y8=True, want_h8=True)
    assert a["h"].data_ptr() == rd.data_ptr()
    for k in ("h", "y", "h8", "h8_scale", "y8"):
        close(a[k], np64(b[k]), 0.0 if k != "y" else (2 * ULP[dt] + RSTD) * np.abs(np64(b[k])) + FLOOR[dt], k)


def test_outputs_as_wanted():
    x, r, w = _rows(4, 256, "bf16", 1)
    o = flce.rmsnorm_fwd(x.cuda(), w.cuda(), want_y=False)
    assert set(o) == {"rstd"}
    o = flce.rmsnorm_fwd(x.cuda(), w.cuda(), r.cuda(), want_y=False, want_h8=True)
    assert set(o) == {"rstd", "h", "h8", "h8_scale"}


def test_rows_of_zeros_infinities_and_nan():
    """A row of zeros gives y = 0 and rstd = eps^-1/2; a NaN or an infinity stays in its row and
    its 8-bit copies are NaN codes, whatever stands beside it."""
    H = 300
    x = torch.randn(5, H).bfloat16()
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 200] = float("nan")
    x[4, 0] = -torch.finfo(torch.bfloat16).max
    w = torch.ones(H).bfloat16()
    o = flce.rmsnorm_fwd(x.cuda(), w.cuda(), eps=1e-4, want_y8=True, want_h8=True)
    f = lambda k: o[k].float().cpu()  # noqa: E731
    assert torch.all(f("y")[1] == 0) and abs(float(o["rstd"][1]) - 100) < 1e-3 and torch.all(f("y8")[1] == 0)
    assert torch.all(f("h8_scale")[1] == 1)
    assert torch.isfinite(f("y")[0]).all() and torch.isfinite(f("h8")[0]).all()
    assert torch.isnan(f("h8")[2, 7]) and torch.isfinite(f("h8")[2, :7]).all() and torch.isfinite(f("h8_scale")).all()
    assert torch.isnan(f("y")[2, 7]) and torch.isnan(f("y")[3]).all()
    assert torch.isnan(f("h8")[3, 200]) and torch.isfinite(f("h8")[3, :200]).all()
    assert float(o["rstd"][4]) == 0.0          # the squares overflow: 1 / sqrt(inf)
    q, s = oo.pack(np64(x))
    assert np.array_equal(np64(o["h8"]), q, equal_nan=True) and np.array_equal(np64(o["h8_scale"]), s)


def test_no_rows():
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    o = flce.rmsnorm_fwd(e, w, e, want_y8=True, want_h8=True)
    assert o["y"].shape == (0, 64)
    dw = torch.ones(64, device="cuda")
    flce.rmsnorm_bwd(e, w, o["rstd"], e, dweight=dw)
    assert torch.all(dw == 1)
    assert torch.all(flce.rmsnorm_bwd(e, w, o["rstd"], e)["dweight"] == 0)


BWD = [(1, 1, "f32"), (1, 4096, "bf16"), (3, 130, "f16"), (65, 256, "bf16"), (200, 1337, "f32"), (17, 5376, "bf16"),
       (5, 16384, "f16"), (9, 9001, "bf16"), (4, 20000, "bf16"), (3000, 72, "bf16"), (2, 8192, "f32"), (12000, 136, "f16"),
       (700, 8192, "f32"), (310, 6112, "f32"), (700, 5121, "bf16"), (3, 8191, "f16"), (1000, 1167, "bf16"),
       (1000, 1166, "bf16"), (300, 5122, "bf16"), (40, 2050, "f32"), (9, 8194, "f16")]


@pytest.mark.parametrize("N,H,dt", BWD)
@pytest.mark.parametrize("q8,with_dh,same", [(False, True, False), (True, False, True), (True, True, False)])
def test_gradient(N, H, dt, q8, with_dh, same):
    x, d, w = _rows(N, H, dt, N + 3 * H)
    dh = torch.randn(N, H, generator=torch.Generator().manual_seed(1)).to(DT[dt]) if with_dh else None
    off = 0.5
    h = np64(x)
    _, rstd = oo.rmsnorm_fwd(h, np64(w), 1e-5, off)
    rd = torch.from_numpy(rstd).float().cuda()
    wdt = dt if same else "f32"
    init = torch.randn(H, generator=torch.Generator().manual_seed(2)).to(DT[wdt])
    dw = init.clone().cuda()
    kw = dict(dh=None if dh is None else dh.cuda(), weight_offset=off, dweight=dw)
    if q8:
        p = flce.ckpt8_pack(x.cuda())
        o = flce.rmsnorm_bwd(d.cuda(), w.cuda(), rd, h8=p["q"], h8_scale=p["scale"], **kw)
        h = np64(p["q"]) * oo.spread(np64(p["scale"]), H)
    else:
        o = flce.rmsnorm_bwd(d.cuda(), w.cuda(), rd, x.cuda(), **kw)
    dx, dwt, mag, wmag = oo.rmsnorm_bwd(np64(d), h, np64(rd), np64(w), off, None if dh is None else np64(dh))
    close(o["dx"], dx, ULP[dt] * np.abs(dx) + F32 * mag + FLOOR[dt], "dx")
    total = dwt + np64(init)
    close(dw, total, ULP[wdt] * np.abs(total) + F32 * ((N + 8) * wmag + 2 * np.abs(np64(init))) + FLOOR[wdt], "dweight")
    # overwriting, and one output at a time, give the same
    ow = torch.full((H,), float("nan"), dtype=DT[wdt], device="cuda")
    src = dict(h8=p["q"], h8_scale=p["scale"]) if q8 else dict(h=x.cuda())
    a = flce.rmsnorm_bwd(d.cuda(), w.cuda(), rd, **src, dweight=ow, want_dx=False, weight_offset=off,
                         flags=flce.FLAG_DW_OVERWRITE)
    assert "dx" not in a
    close(ow, dwt, ULP[wdt] * np.abs(dwt) + F32 * (N + 8) * wmag + FLOOR[wdt], "dweight alone")
    b = flce.rmsnorm_bwd(d.cuda(), w.cuda(), rd, **src, want_dweight=False, weight_offset=off, dh=kw["dh"])
    assert torch.equal(b["dx"], o["dx"]) and "dweight" not in b


@pytest.mark.parametrize("dt,H,extra,offset", [("bf16", 136, 8, 8), ("bf16", 136, 1, 3), ("f32", 67, 4, 4),
                                               ("bf16", 136, 2, 2), ("f32", 66, 2, 6)])
def test_gradient_strides_and_in_place(dt, H, extra, offset):
    N = 300
    x, d, w = _rows(N, H, dt, 8)
    rd = torch.rand(N).cuda() + 0.5
    s = lambda t: strided(t.cuda(), extra, offset)  # noqa: E731
    want = flce.rmsnorm_bwd(d.cuda(), w.cuda(), rd, x.cuda(), dh=x.cuda())
    dd = s(d)
    got = flce.rmsnorm_bwd(dd, w.cuda(), rd, s(x), dh=s(x), outputs={"dx": dd})          # dx over dy
    assert got["dx"].data_ptr() == dd.data_ptr()
    ref, _, mag, wmag = oo.rmsnorm_bwd(np64(d), np64(x), np64(rd), np64(w), 0.0, np64(x))
    close(dd, np64(want["dx"]), 2 * (ULP[dt] * np.abs(ref) + F32 * mag))
    close(got["dweight"], np64(want["dweight"]), 2 * F32 * (N + 8) * wmag)


@pytest.mark.parametrize("N,H,dt,extra,offset", [(3, 20000, "bf16", 0, 0), (5, 9001, "f16", 0, 0), (2, 16392, "f32", 0, 0),
                                                 (4, 8194, "bf16", 0, 0), (3, 9216, "bf16", 1, 3), (70, 8193, "f32", 0, 0)])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("over", ["dy", "dh"])
def test_gradient_of_long_rows_in_place(N, H, dt, extra, offset, q8, over):
    """Rows that two kernels read, with dx in the place of dy or of dh: dweight is that of the
    dy that was given."""
    x, d, w = _rows(N, H, dt, N + H)
    rd = torch.rand(N, generator=torch.Generator().manual_seed(6)).cuda() + 0.5
    dh = torch.randn(N, H, generator=torch.Generator().manual_seed(7)).to(DT[dt])
    dd, hh = strided(d.cuda(), extra, offset), strided(dh.cuda(), extra, offset)
    h = np64(x)
    kw = dict(h=strided(x.cuda(), extra, offset))
    if q8:
        p = flce.ckpt8_pack(x.cuda())
        h = np64(p["q"]) * oo.spread(np64(p["scale"]), H)
        kw = dict(h8=p["q"], h8_scale=p["scale"])
    into = dd if over == "dy" else hh
    o = flce.rmsnorm_bwd(dd, w.cuda(), rd, **kw, dh=hh, outputs={"dx": into})
    assert o["dx"].data_ptr() == into.data_ptr()
    dx, dw, mag, wmag = oo.rmsnorm_bwd(np64(d), h, np64(rd), np64(w), 0.0, np64(dh))
    close(into, dx, ULP[dt] * np.abs(dx) + F32 * mag + FLOOR[dt], "dx")
    close(o["dweight"], dw, F32 * ((N + 8) * wmag + np.abs(dw)), "dweight")


def test_gradient_is_the_derivative_of_the_forward():
    """dx and dweight of L = sum(c * y) in fp32 against central differences of the float64
    forward (step 1e-5: truncation below 1e-8 of the second derivative's scale)."""
    N, H, eps = 3, 40, 1e-3
    x, c, w = _rows(N, H, "f32", 12)
    o = flce.rmsnorm_fwd(x.cuda(), w.cuda(), eps=eps)
    got = flce.rmsnorm_bwd(c.cuda(), w.cuda(), o["rstd"], x.cuda())
    L = lambda h, ww: (np64(c) * oo.rmsnorm_fwd(h, ww, eps, 0.0)[0]).sum()  # noqa: E731
    h, ww, st = np64(x), np64(w), 1e-5
    for i, j in [(0, 0), (1, 37), (2, 39), (2, 5)]:
        p, m = h.copy(), h.copy()
        p[i, j] += st
        m[i, j] -= st
        assert abs((L(p, ww) - L(m, ww)) / (2 * st) - float(got["dx"][i, j])) <= 1e-4
        p, m = ww.copy(), ww.copy()
        p[j] += st
        m[j] -= st
        assert abs((L(h, p) - L(h, m)) / (2 * st) - float(got["dweight"][j])) <= 1e-4


def test_same_bits_and_side_stream():
    x, d, w = (t.cuda() for t in _rows(5000, 1000, "bf16", 4))
    o = flce.rmsnorm_fwd(x, w, d, want_y8=True, want_h8=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p = flce.rmsnorm_fwd(x, w, d, want_y8=True, want_h8=True, stream=s)
    a = flce.rmsnorm_bwd(d, w, o["rstd"], o["h"])
    b = flce.rmsnorm_bwd(d, w, p["rstd"], p["h"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for k in o:
        assert torch.equal(o[k].float(), p[k].float()), k
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])

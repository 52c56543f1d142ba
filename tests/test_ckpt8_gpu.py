"""GPU tests of 8-bit checkpoint rows and of the weight gradient that reads them.

Packing is compared bit for bit with the float64 oracle. Bounds of the product over M rows:
fp32 FMA kernels add M products, each sum rounded to 2^-24 relative; the tensor cores may
truncate (2^-23) each addition of 16 products: M * 2^-23 * sum|dy x| covers both. An expanded
value that is not exact in dy's 16-bit type adds a half ulp of it per product. Over all elements
the relative error (2-norm) of an fp32 result is held to 1e-5, as for the other fp32 results of
this package."""

import numpy as np
import pytest
import torch

from linear_cross_entropy_logits_gb300 import build as B
from linear_cross_entropy_logits_gb300 import flce
from oracle import ops_oracle as oo
from ops_util import DT, FLOOR, ULP, close, np64, odd_rows, strided
from parity_util import rel_fro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    flce.load()


def _rows(N, H, dt, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, H, generator=g) * torch.exp(spread * torch.randn(N, 1, generator=g))
    x[:, ::29] *= 20
    return x.to(DT[dt])


@pytest.mark.parametrize("N,H,dt,extra,offset", [
    (1, 1, "f32", 0, 0), (1, 128, "bf16", 0, 0), (3, 129, "f16", 0, 0), (50, 4096, "bf16", 0, 0), (7, 1336, "f16", 0, 0),
    (9, 1000, "f32", 0, 0), (5, 20001, "bf16", 0, 0), (33, 200, "bf16", 3, 1), (33, 200, "f32", 4, 4), (1000, 77, "bf16", 0, 0),
    (16, 136, "f16", 8, 8), (65, 1166, "bf16", 0, 0), (9, 130, "f32", 2, 2), (33, 200, "f16", 2, 4), (3, 2, "f32", 0, 0)])
def test_pack(N, H, dt, extra, offset):
    x = _rows(N, H, dt, N + H)
    o = {"q": odd_rows(N, H, torch.float8_e4m3fn, extra, offset)} if extra else None
    o = flce.ckpt8_pack(strided(x.cuda(), extra, offset), outputs=o)
    q, s = oo.pack(np64(x))
    assert np.array_equal(np64(o["q"]), q) and np.array_equal(np64(o["scale"]), s)


def test_pack_extremes():
    """Blocks of zeros, of the type's largest and smallest values, and with non-finite values."""
    fi = torch.finfo(torch.float32)
    x = torch.randn(8, 256)
    x[0] = 0
    x[1] = fi.max
    x[2] = -fi.tiny / 8
    x[3, 5] = float("inf")
    x[4, 130:] = float("nan")
    x[5] *= 1e-30
    x[6, :128] = 448.0
    x[6, 128:] = 449.0
    x[7, :] = float("-inf")
    o = flce.ckpt8_pack(x.cuda())
    q, s = oo.pack(np64(x))
    assert np.array_equal(np64(o["q"]), q, equal_nan=True) and np.array_equal(np64(o["scale"]), s)
    assert np64(o["scale"])[6].tolist() == [1.0, 2.0] and np64(o["scale"])[7].tolist() == [1.0, 1.0]


def test_pack_nothing():
    o = flce.ckpt8_pack(torch.empty(0, 40, device="cuda"))
    assert o["q"].shape == (0, 40) and o["scale"].shape == (0, 1)


def _dw_bound(dy, x, M, dt, wdt, total, base, inexact):
    mag = np.abs(dy).T @ np.abs(x)
    b = M * 2.0 ** -23 * mag + 2 * ULP[wdt] * np.abs(total) + 2.0 ** -23 * np.abs(base) + FLOOR[wdt]
    return b + (ULP[dt] * mag if inexact else 0.0)


DW = [(1, 1, 1, "f32", "f32"), (1, 8, 16, "bf16", "f32"), (1, 300, 520, "bf16", "bf16"), (63, 64, 128, "f16", "f32"),
      (64, 256, 256, "bf16", "f32"), (65, 264, 272, "bf16", "f32"), (200, 257, 133, "bf16", "f32"),
      (130, 520, 1336, "f16", "f16"), (1000, 136, 400, "f32", "f32"), (777, 72, 2000, "bf16", "bf16"),
      (2049, 512, 640, "bf16", "f32"), (5000, 256, 384, "bf16", "f32"), (4100, 264, 300, "f16", "f32"),
      (300, 1030, 90, "f32", "f32"), (129, 2000, 31, "f16", "f32"),
      (40, 300, 261, "bf16", "bf16"), (40, 300, 260, "f16", "f16"), (33, 270, 262, "bf16", "bf16"), (2, 257, 519, "f16", "f32")]


@pytest.mark.parametrize("M,N,K,dt,wdt", DW)
@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("simt", [False, True])
def test_dw(M, N, K, dt, wdt, accumulate, simt):
    g = torch.Generator().manual_seed(M + N + K)
    dy = (torch.randn(M, N, generator=g) * 0.3).to(DT[dt])
    p = flce.ckpt8_pack(_rows(M, K, dt, M + K, 1.0).cuda())
    x = np64(p["q"]) * oo.spread(np64(p["scale"]), K)
    init = torch.randn(N, K, generator=g).to(DT[wdt]) if accumulate else torch.full((N, K), float("nan"), dtype=DT[wdt])
    dW = init.clone().cuda()
    o = flce.ckpt8_dw(dy.cuda(), p["q"], p["scale"], dW=dW, flags=(0 if accumulate else flce.FLAG_DW_OVERWRITE)
                      | (flce.FLAG_FORCE_SIMT if simt else 0))
    assert o["status_code"] == flce.FLCE_OK
    base = np64(init) if accumulate else np.zeros((N, K))
    want = np64(dy).T @ x
    total = want + base
    close(dW, total, _dw_bound(np64(dy), x, M, dt, wdt, total, base, dt == "f16" and not simt))
    if wdt == "f32" and dt != "f16":
        assert rel_fro(np64(dW), total) <= 1e-5


def test_dw_long_sum_keeps_fp32():
    """16384 rows of one sign: the sum's error grows with the rows summed without a rounding
    to nearest, which the kernel bounds."""
    g = torch.Generator().manual_seed(1)
    M, N, K = 16384, 256, 256
    dy = (1 + 0.1 * torch.rand(M, N, generator=g)).bfloat16().cuda()
    p = flce.ckpt8_pack((1 + torch.rand(M, K, generator=g)).bfloat16().cuda())
    want = dy.double().t() @ (p["q"].double() * p["scale"].double().repeat_interleave(128, dim=1))
    got = flce.ckpt8_dw(dy, p["q"], p["scale"])["dW"]
    assert rel_fro(np64(got), np64(want)) <= 1e-5


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1000, 512, 512), (2048, 1024, 1024), (8192, 2560, 2560)])
def test_dw_error_stays_below_1e_6(dt, M, N, K):
    """Activations of either sign, tiles whole and in parts: of the order of a plain fp32 product's
    error, whose relative 2-norm is 1.5e-7 to 1.6e-6 at these sizes."""
    g = torch.Generator().manual_seed(M)
    dy = (0.01 * torch.randn(M, N, generator=g)).to(DT[dt]).cuda()
    p = flce.ckpt8_pack((torch.randn(M, K, generator=g) * (0.5 + torch.rand(M, 1, generator=g))).to(DT[dt]).cuda())
    want = dy.double().t() @ (p["q"].double() * p["scale"].double().repeat_interleave(128, dim=1))
    got = flce.ckpt8_dw(dy, p["q"], p["scale"])["dW"].double()
    assert float((got - want).norm() / want.norm()) <= 1e-6


@pytest.mark.parametrize("extra,offset", [(8, 8), (3, 1), (16, 0)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_dw_strides(dt, extra, offset):
    M, N, K = 300, 136, 272
    g = torch.Generator().manual_seed(2)
    dy = torch.randn(M, N, generator=g).to(DT[dt]).cuda()
    p = flce.ckpt8_pack(_rows(M, K, dt, 3, 1.0).cuda())
    want = flce.ckpt8_dw(dy, p["q"], p["scale"])["dW"]
    dW = strided(torch.zeros(N, K, device="cuda"), extra, offset)
    flce.ckpt8_dw(strided(dy, extra, offset), strided(p["q"], extra, offset), p["scale"], dW=dW)
    x = np64(p["q"]) * oo.spread(np64(p["scale"]), K)
    ref = np64(dy).T @ x
    close(dW, ref, _dw_bound(np64(dy), x, M, dt, "f32", ref, 0 * ref, False))
    close(want, ref, _dw_bound(np64(dy), x, M, dt, "f32", ref, 0 * ref, False))


@pytest.mark.parametrize("M", [20, 3000])
@pytest.mark.parametrize("K,extra,offset", [(134, 2, 0), (133, 3, 4), (135, 1, 1), (390, 0, 0)])
@pytest.mark.parametrize("wdt", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [True, False])
def test_dw_last_columns(M, K, extra, offset, wdt, accumulate):
    """Rows whose pitch allows wide accesses and whose last columns do not, and the reverse; the
    elements between the rows stay as they were."""
    N = 270
    g = torch.Generator().manual_seed(M + K)
    dy = (torch.randn(M, N, generator=g) * 0.3).to(DT["bf16"])
    p = flce.ckpt8_pack(_rows(M, K, "bf16", K, 1.0).cuda())
    x = np64(p["q"]) * oo.spread(np64(p["scale"]), K)
    flat = torch.randn(N * (K + extra) + offset, generator=g).to(DT[wdt]).cuda()
    keep = flat.clone()
    dW = flat[offset:].view(N, K + extra)[:, :K]
    init = np64(dW) if accumulate else 0 * np64(dW)
    flce.ckpt8_dw(dy.cuda(), p["q"], p["scale"], dW=dW, flags=0 if accumulate else flce.FLAG_DW_OVERWRITE)
    ref = init + np64(dy).T @ x
    close(dW, ref, _dw_bound(np64(dy), x, M, "bf16", wdt, ref, init, accumulate))
    between = flat[offset:].view(N, K + extra)[:, K:]
    assert torch.equal(between, keep[offset:].view(N, K + extra)[:, K:]) and torch.equal(flat[:offset], keep[:offset])


def test_dw_scales_that_are_no_powers_of_two():
    """The norm's 8-bit output as the projection's input."""
    M, N, K = 500, 128, 384
    x = _rows(M, K, "bf16", 6, 0.5).cuda()
    w = (1 + 0.2 * torch.randn(K, generator=torch.Generator().manual_seed(3))).bfloat16().cuda()
    o = flce.rmsnorm_fwd(x, w, want_y8=True)
    dy = torch.randn(M, N, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    got = flce.ckpt8_dw(dy, o["y8"], o["y8_scale"])["dW"]
    xs = np64(o["y8"]) * oo.spread(np64(o["y8_scale"]), K)
    want = np64(dy).T @ xs
    close(got, want, _dw_bound(np64(dy), xs, M, "bf16", "f32", want, 0 * want, True))


def _odd_scales(M, nblk, seed):
    """Scales as the norm's 8-bit output has them: powers of two times any fp32 factor."""
    g = torch.Generator().manual_seed(seed)
    return torch.exp2(torch.randint(-6, 7, (M, nblk), generator=g).float()) * (0.5 + torch.rand(M, nblk, generator=g))


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (63, 72, 130), (500, 128, 384), (1000, 257, 133), (3000, 520, 300),
                                   (130, 2000, 1336), (9000, 64, 128)])
@pytest.mark.parametrize("accumulate", [True, False])
def test_dw_fp32_gradient_with_any_scales(M, N, K, accumulate):
    """fp32 dy, whose 24 bits count, times checkpoint values that have as many."""
    p = flce.ckpt8_pack(_rows(M, K, "f32", M + K, 0.5).cuda())
    s = _odd_scales(M, (K + 127) // 128, M).cuda()
    g = torch.Generator().manual_seed(4)
    dy = torch.randn(M, N, generator=g)
    init = torch.randn(N, K, generator=g) if accumulate else torch.full((N, K), float("nan"))
    dW = init.clone().cuda()
    o = flce.ckpt8_dw(dy.cuda(), p["q"], s, dW=dW, flags=0 if accumulate else flce.FLAG_DW_OVERWRITE)
    assert o["status_code"] == flce.FLCE_OK
    x = np64(p["q"]) * oo.spread(np64(s), K)
    base = np64(init) if accumulate else np.zeros((N, K))
    want = np64(dy).T @ x + base
    close(dW, want, _dw_bound(np64(dy), x, M, "f32", "f32", want, base, True))
    assert rel_fro(np64(dW), want) <= 1e-5


def _fp16_rows(kind, M, K, g):
    x = torch.randn(M, K, generator=g)
    if kind == "large":                       # past fp16's largest value
        return x * 3e6
    if kind == "small":                       # below its smallest
        return x * 1e-10
    if kind == "rows":                        # rows 2^-20 ... 1 of the largest
        return x * torch.exp2(16 - torch.randint(0, 21, (M, 1), generator=g).float())
    e = torch.randint(0, 61, (M, (K + 127) // 128), generator=g).float().repeat_interleave(128, dim=1)[:, :K]
    return x * torch.exp2(30 - e)             # "far": blocks 2^-60 ... 1 of the largest


@pytest.mark.parametrize("kind", ["large", "small", "rows", "far"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 16), (65, 264, 272), (1531, 136, 390), (4100, 520, 133)])
@pytest.mark.parametrize("wdt,accumulate", [("f32", True), ("f32", False), ("f16", False)])
def test_dw_fp16_gradient_of_checkpoints_of_any_size(kind, M, N, K, wdt, accumulate):
    """The checkpoint need not fit fp16. With e the exponent of the largest scale, its values are
    exact down to 2^(e - 31) and off by 2^(e - 32) below; the largest value is over 224 * 2^e."""
    g = torch.Generator().manual_seed(M + N)
    p = flce.ckpt8_pack(_fp16_rows(kind, M, K, g).cuda())
    x = np64(p["q"]) * oo.spread(np64(p["scale"]), K)
    # (fp16 results stay in range)
    unit = 1.0 if wdt == "f32" else 2.0 ** -np.ceil(np.log2(np.abs(x).max() * M))
    x = x * unit
    s = p["scale"] * unit
    dy = (torch.randn(M, N, generator=g) * 0.3).half()
    base = torch.randn(N, K, generator=g).float() * np.abs(x).max() if accumulate else torch.zeros(N, K)
    dW = base.to(DT[wdt]).cuda()
    flce.ckpt8_dw(dy.cuda(), p["q"], s, dW=dW, flags=0 if accumulate else flce.FLAG_DW_OVERWRITE)
    base = np64(base)
    want = np64(dy).T @ x + base
    bound = _dw_bound(np64(dy), x, M, "f16", wdt, want, base, False)
    bound += 2.0 ** -39 * np.abs(x).max() * np.abs(np64(dy)).sum(axis=0)[:, None]
    close(dW, want, bound)
    if wdt == "f32" and kind != "far":
        assert rel_fro(np64(dW), want) <= 1e-5


def test_dw_fp16_gradient_of_the_norms_checkpoint():
    """h = x + r of fp16 values can pass fp16's range; its checkpoint holds it."""
    M, N, K = 300, 64, 256
    g = torch.Generator().manual_seed(12)
    x = (50000 + 10000 * torch.rand(M, K, generator=g)).half().cuda()
    o = flce.rmsnorm_fwd(x, torch.ones(K, dtype=torch.float16, device="cuda"), x, want_h=False, want_h8=True)
    h = np64(o["h8"]) * oo.spread(np64(o["h8_scale"]), K)
    assert h.max() > 65504
    dy = (torch.randn(M, N, generator=g) * 0.01).half()
    got = flce.ckpt8_dw(dy.cuda(), o["h8"], o["h8_scale"])["dW"]
    assert rel_fro(np64(got), np64(dy).T @ h) <= 1e-5


@pytest.mark.parametrize("K,extra,offset", [(272, 0, 0), (256, 16, 0), (390, 3, 1), (130, 0, 0)])
@pytest.mark.parametrize("one", [False, True])
def test_dw_fp16_gradient_beside_blocks_of_zeros(K, extra, offset, one):
    """A block of zeros has scale 1 whatever the others have, and a block whose scale is 1 may
    hold a single value, its last."""
    M, N = 700, 72
    g = torch.Generator().manual_seed(K)
    x = torch.randn(M, K, generator=g) * 1e-9
    x[::3] = 0
    x[1::3, :128] = 0
    x[2::3, K // 128 * 128 - 128:] = 0
    if one:
        x[0, 127] = 400.0
        x[3, K - 1] = -300.0
    p = flce.ckpt8_pack(x.cuda())
    assert (p["scale"] == 1).any()
    q = strided(p["q"], extra, offset)
    dy = (torch.randn(M, N, generator=g) * 0.3).half()
    xs = np64(p["q"]) * oo.spread(np64(p["scale"]), K)
    want = np64(dy).T @ xs
    got = flce.ckpt8_dw(dy.cuda(), q, p["scale"])["dW"]
    bound = _dw_bound(np64(dy), xs, M, "f16", "f32", want, 0 * want, False)
    close(got, want, bound + 2.0 ** -39 * np.abs(xs).max() * np.abs(np64(dy)).sum(axis=0)[:, None])
    assert rel_fro(np64(got), want) <= 1e-5


@pytest.mark.parametrize("M,N,K,extra", [(1, 8, 260, 0), (47, 170, 171, 0), (700, 72, 272, 1), (4100, 40, 520, 0)])
@pytest.mark.parametrize("most", [1, 5])
def test_dw_fp16_gradient_beside_zeros_of_any_scale(M, N, K, extra, most):
    """Blocks of zeros whose scales pass the others' by 2^10 to 2^60, most of the blocks or some; and
    nothing but such blocks."""
    g = torch.Generator().manual_seed(M)
    nblk = (K + 127) // 128
    p = flce.ckpt8_pack(torch.randn(M, K, generator=g).cuda())
    zero = torch.randint(0, 6, (M, nblk), generator=g) < most
    zero[0, 0] = False
    p["q"].view(torch.int8)[zero.repeat_interleave(128, dim=1)[:, :K].cuda()] = 0
    up = torch.exp2(torch.randint(10, 61, (M, nblk), generator=g).float())
    s = p["scale"] * torch.where(zero, up, 1.0).cuda()
    dy = (torch.randn(M, N, generator=g) * 0.3).half()
    xs = np64(p["q"]) * oo.spread(np64(s), K)
    want = np64(dy).T @ xs
    got = flce.ckpt8_dw(dy.cuda(), strided(p["q"], extra, 0), s)["dW"]
    close(got, want, _dw_bound(np64(dy), xs, M, "f16", "f32", want, 0 * want, False)
          + 2.0 ** -39 * np.abs(xs).max() * np.abs(np64(dy)).sum(axis=0)[:, None])
    p["q"].view(torch.int8).zero_()
    got = flce.ckpt8_dw(dy.cuda(), strided(p["q"], extra, 0), 2.0 ** 60 * s)["dW"]
    assert torch.all(got == 0)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_dw_scales_that_are_not_finite(dt, bad):
    """They spoil their block's columns and no others."""
    M, N, K = 200, 72, 300
    g = torch.Generator().manual_seed(13)
    x = 1 + torch.rand(M, K, generator=g)
    p = flce.ckpt8_pack(x.cuda())
    s = p["scale"].clone()
    s[77, 1] = bad
    dy = (1 + torch.rand(M, N, generator=g)).to(DT[dt])
    dW = np64(flce.ckpt8_dw(dy.cuda(), p["q"], s)["dW"])
    assert not np.isfinite(dW[:, 128:256]).any()
    xs = np64(p["q"]) * oo.spread(np64(p["scale"]), K)
    want = np64(dy).T @ xs
    keep = np.r_[0:128, 256:300]
    assert rel_fro(dW[:, keep], want[:, keep]) <= 1e-5


def test_dw_non_finite_rows_stay_in_their_columns():
    M, N, K = 70, 64, 256
    x = torch.randn(M, K)
    x[3, 17] = float("inf")
    x[60, 200] = float("nan")
    dy = torch.randn(M, N)
    dy[5, 9] = float("nan")
    p = flce.ckpt8_pack(x.bfloat16().cuda())
    dW = flce.ckpt8_dw(dy.bfloat16().cuda(), p["q"], p["scale"])["dW"].cpu()
    bad = torch.zeros(N, K, dtype=torch.bool)
    bad[:, 17] = bad[:, 200] = True
    bad[9] = True
    assert torch.equal(torch.isnan(dW), bad)


def test_dw_no_rows():
    dy, q, s = torch.empty(0, 8, device="cuda"), torch.empty(0, 16, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(0, 1, device="cuda")
    dW = torch.ones(8, 16, device="cuda")
    flce.ckpt8_dw(dy, q, s, dW=dW)
    assert torch.all(dW == 1)
    assert torch.all(flce.ckpt8_dw(dy, q, s)["dW"] == 0)


def test_dw_is_the_derivative_of_the_projection():
    """Central differences of L(W) = sum(c * x W^T), linear in W, over a step of 1."""
    M, N, K = 90, 6, 40
    g = torch.Generator().manual_seed(7)
    p = flce.ckpt8_pack(torch.randn(M, K, generator=g).cuda())
    x = np64(p["q"]) * oo.spread(np64(p["scale"]), K)
    c, W = np.asarray(torch.randn(M, N, generator=g).double()), np.asarray(torch.randn(N, K, generator=g).double())
    dW = np64(flce.ckpt8_dw(torch.from_numpy(c).float().cuda(), p["q"], p["scale"])["dW"])
    for n, k in [(0, 0), (5, 39), (2, 20)]:
        Wp, Wm = W.copy(), W.copy()
        Wp[n, k] += 1
        Wm[n, k] -= 1
        diff = ((c * (x @ Wp.T)).sum() - (c * (x @ Wm.T)).sum()) / 2
        assert abs(diff - dW[n, k]) <= 1e-4


def test_dw_same_bits_and_side_stream():
    g = torch.Generator().manual_seed(8)
    p = flce.ckpt8_pack(torch.randn(3000, 520, generator=g).bfloat16().cuda())
    dy = torch.randn(3000, 264, generator=g).bfloat16().cuda()
    a = flce.ckpt8_dw(dy, p["q"], p["scale"])["dW"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = flce.ckpt8_dw(dy, p["q"], p["scale"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert b["status_code"] == flce.FLCE_OK and torch.equal(a, b["dW"])


def test_dw_wait_limit():
    """A pipeline stage that is never filled: the bounded waits run out, the call reports it, and
    the next call is normal."""
    g = torch.Generator().manual_seed(9)
    p = flce.ckpt8_pack(torch.randn(1000, 512, generator=g).bfloat16().cuda())
    dy = torch.randn(1000, 300, generator=g).bfloat16().cuda()
    a = flce.ckpt8_dw(dy, p["q"], p["scale"])["dW"]
    o = flce.ckpt8_dw(dy, p["q"], p["scale"], flags=flce.FLAG_DEBUG_STALL, wait_timeout_ms=50)
    assert o["status_code"] == flce.FLCE_ERR_TIMEOUT
    b = flce.ckpt8_dw(dy, p["q"], p["scale"])
    assert b["status_code"] == flce.FLCE_OK and torch.equal(a, b["dW"])


@pytest.mark.parametrize("dt,wdt", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("M", [60, 5000])
@pytest.mark.parametrize("accumulate", [True, False])
def test_dw_wait_limit_leaves_nan(dt, wdt, M, accumulate):
    """A caller who does not look at the status sees it in dW: the tile that a pair gave up on is
    NaN (60 rows: whole, 5000: the sum of parts), the others are right."""
    N, K = 300, 520
    g = torch.Generator().manual_seed(M)
    p = flce.ckpt8_pack(torch.randn(M, K, generator=g).cuda())
    dy = torch.randn(M, N, generator=g).to(DT[dt]).cuda()
    init = torch.randn(N, K, generator=g).to(DT[wdt]).cuda()
    flags = 0 if accumulate else flce.FLAG_DW_OVERWRITE
    a, b = init.clone(), init.clone()
    flce.ckpt8_dw(dy, p["q"], p["scale"], dW=a, flags=flags)
    o = flce.ckpt8_dw(dy, p["q"], p["scale"], dW=b, flags=flags | flce.FLAG_DEBUG_STALL, wait_timeout_ms=50)
    assert o["status_code"] == flce.FLCE_ERR_TIMEOUT
    assert torch.isnan(b[:256, :256]).all()
    a[:256, :256] = b[:256, :256] = 0
    assert torch.equal(a, b)


def test_calls_in_a_graph():
    """The operators enqueue kernels and memsets only: captured once, replayed on new inputs."""
    g = torch.Generator().manual_seed(10)
    x = torch.randn(700, 520, generator=g).bfloat16().cuda()
    dy = torch.randn(700, 264, generator=g).bfloat16().cuda()
    t = torch.randint(0, 90, (700,), generator=g).cuda()
    w = torch.ones(520).bfloat16().cuda()
    dE, dW = torch.zeros(90, 520, device="cuda"), torch.zeros(264, 520, device="cuda")

    def call():
        o = flce.rmsnorm_fwd(x, w, want_h8=True)
        b = flce.rmsnorm_bwd(o["y"], w, o["rstd"], h8=o["h8"], h8_scale=o["h8_scale"])
        flce.embed_bwd(t, b["dx"], dE=dE, flags=flce.FLAG_DW_OVERWRITE, check=False)
        p = flce.ckpt8_pack(o["y"])
        flce.ckpt8_dw(dy, p["q"], p["scale"], dW=dW, flags=flce.FLAG_DW_OVERWRITE, check=False)
        return flce.embed_fwd(t, dE, check=False)["out"], b["dweight"]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, dweight = call()
    x.copy_(torch.randn(700, 520, generator=g).bfloat16())
    graph.replay()
    got = [v.clone() for v in (out, dweight, dE, dW)]
    want = call()
    for a, b in zip(got, (*want, dE, dW)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(300, 72, 272), (3000, 75, 133)])
def test_dw_scales_change_between_replays(dt, M, N, K):
    """What the scales ask for is decided on the device: a captured call replayed on others."""
    g = torch.Generator().manual_seed(14)
    p = flce.ckpt8_pack(torch.randn(M, K, generator=g).cuda())
    dy = torch.randn(M, N, generator=g).to(DT[dt]).cuda()
    s = p["scale"].clone()
    dW = torch.empty(N, K, device="cuda")
    call = lambda w: flce.ckpt8_dw(dy, p["q"], s, dW=w, flags=flce.FLAG_DW_OVERWRITE, check=False)  # noqa: E731
    call(dW)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(dW)
    for f in (1.0, 2.0 ** 40, 1.1, 2.0 ** -60, 0.3, 1.0):
        s.copy_(p["scale"] * f)
        graph.replay()
        got = dW.clone()
        call(dW)
        assert torch.equal(got, dW)
        if dt == "f32" or f in (1.0, 2.0 ** 40, 2.0 ** -60):
            assert rel_fro(np64(got), np64(dy).T @ (np64(p["q"]) * oo.spread(np64(s), K))) <= 1e-5


def test_dw_status_word_in_the_workspace():
    """Without a status word of the caller's, flce_get_status reads the workspace's."""
    p = flce.ckpt8_pack(torch.randn(200, 128, device="cuda"))
    o = flce.ckpt8_dw(torch.randn(200, 64, device="cuda"), p["q"], p["scale"], check=False)
    lib, s = flce.load(), torch.cuda.current_stream().cuda_stream
    assert lib.flce_get_status(None, o["workspace"].data_ptr(), s) == flce.FLCE_OK
    o = flce.ckpt8_dw(torch.randn(200, 64, device="cuda"), p["q"], p["scale"], check=False, wait_timeout_ms=50,
                      flags=flce.FLAG_DEBUG_STALL)
    assert lib.flce_get_status(None, o["workspace"].data_ptr(), s) == flce.FLCE_ERR_TIMEOUT


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows go through packing, the norm and its gradient."""
    N, H = 530_000, 4096
    x = torch.zeros(N, H, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(7, H, generator=torch.Generator().manual_seed(11)).bfloat16().cuda()
    x[-7:] = tail
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    p, q = flce.ckpt8_pack(x), flce.ckpt8_pack(tail)
    assert torch.equal(p["q"][-7:].float(), q["q"].float()) and torch.equal(p["scale"][-7:], q["scale"])
    o, s = flce.rmsnorm_fwd(x, w, eps=1e-5), flce.rmsnorm_fwd(tail, w, eps=1e-5)
    assert torch.equal(o["y"][-7:], s["y"]) and torch.equal(o["rstd"][-7:], s["rstd"])
    b = flce.rmsnorm_bwd(x, w, o["rstd"], h8=p["q"], h8_scale=p["scale"])
    c = flce.rmsnorm_bwd(tail, w, s["rstd"], h8=q["q"], h8_scale=q["scale"])
    assert torch.equal(b["dx"][-7:], c["dx"])
    assert torch.all(b["dx"][:-7] == 0)
    dy = torch.zeros(N, 64, dtype=torch.bfloat16, device="cuda")
    dy[-7:] = 1
    a = flce.ckpt8_dw(dy, p["q"], p["scale"])["dW"]
    assert torch.equal(a, flce.ckpt8_dw(dy[-7:], q["q"], q["scale"])["dW"])

"""GPU tests of the token embedding and its gradient against the float64 oracle.

Bounds. Forward: one product in fp32 and one rounding to the output type. Gradient of a token
with n rows: n fp32 additions, a product by the scale and the rounding to dE's type (accumulating:
one more fp32 addition), so |error| <= (n + 3) 2^-24 sum|scale dout| + 2 half-ulps of dE's type."""

import numpy as np
import pytest
import torch

from linear_cross_entropy_logits_gb300 import build as B
from linear_cross_entropy_logits_gb300 import flce
from oracle import ops_oracle as oo
from ops_util import DT, F32, FLOOR, ULP, close, np64, strided

pytestmark = pytest.mark.gpu
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    flce.load()


def _tokens(kind, N, V, g):
    if kind == "uniform":
        t = torch.randint(0, V, (N,), generator=g)
    elif kind == "one":                       # every position the same token: one run over all pieces
        t = torch.full((N,), V - 1, dtype=torch.int64)
    elif kind == "skewed":
        t = (torch.exp(torch.rand(N, generator=g, dtype=torch.float64) * np.log(V + 1.0)).long() - 1).clamp(0, V - 1)
    elif kind == "ignored":
        t = torch.full((N,), IGN, dtype=torch.int64)
    else:                                     # blocks of 32 equal tokens: runs that end with a piece
        t = (torch.arange(N) // 32) % V
    if kind in ("uniform", "skewed") and N > 3:
        t[torch.rand(N, generator=g) < 0.2] = IGN
    return t


FWD = [(1, 64, 10, "bf16", 1.0, 0, 0), (5, 1, 7, "f32", 0.5, 0, 0), (33, 1003, 500, "f16", 2.0, 0, 0),
       (300, 2048, 1000, "bf16", 45.25, 0, 0), (17, 136, 40, "bf16", 1.0, 3, 1), (64, 520, 99, "f32", 1.0, 8, 4),
       (2, 20000, 5, "f16", 1.0, 0, 0), (40, 8, 3, "bf16", 3.0, 8, 8),
       (333, 40, 50, "bf16", 0.5, 0, 0), (1001, 130, 77, "f16", 1.0, 2, 2), (155, 65, 9, "f32", 1.0, 1, 1)]


@pytest.mark.parametrize("N,H,V,dt,scale,extra,offset", FWD)
def test_forward(N, H, V, dt, scale, extra, offset):
    g = torch.Generator().manual_seed(N * 7 + H)
    E = torch.randn(V, H, generator=g).to(DT[dt])
    t = _tokens("uniform", N, V, g)
    Ed = strided(E.cuda(), extra, offset)
    out = strided(torch.full((N, H), 7.0, dtype=DT[dt], device="cuda"), extra, offset)
    o = flce.embed_fwd(t.cuda(), Ed, scale=scale, ignore_index=IGN, out=out)
    assert o["status_code"] == flce.FLCE_OK
    want = oo.embed_fwd(t.numpy(), np64(E), scale, IGN)
    close(out, want, (ULP[dt] + F32) * np.abs(want) + FLOOR[dt])
    if scale == 1.0:
        assert np.array_equal(np64(out), want)


def test_forward_leaves_the_pitch_alone():
    buf = torch.full((6, 40), 5.0, device="cuda")
    flce.embed_fwd(torch.tensor([0, 1, IGN, 1, 0, 1], device="cuda"), torch.randn(2, 33, device="cuda"), out=buf[:, :33])
    assert torch.all(buf[:, 33:] == 5.0)


def test_no_tokens():
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    E = torch.randn(4, 16, device="cuda")
    assert flce.embed_fwd(t, E)["out"].shape == (0, 16)
    dE = torch.ones(4, 16, device="cuda")
    flce.embed_bwd(t, torch.empty(0, 16, device="cuda"), dE=dE)
    assert torch.all(dE == 1)
    flce.embed_bwd(t, torch.empty(0, 16, device="cuda"), dE=dE, flags=flce.FLAG_DW_OVERWRITE)
    assert torch.all(dE == 0)


BWD = [(1, 64, 10, "uniform", "bf16", "f32"), (7, 1, 5, "uniform", "f32", "f32"),
       (31, 136, 100, "one", "bf16", "f32"), (32, 136, 100, "one", "bf16", "bf16"),
       (33, 136, 100, "one", "f16", "f16"), (1000, 264, 50, "blocks", "bf16", "f32"),
       (1000, 65, 600, "uniform", "f16", "f32"), (5000, 40, 3, "uniform", "f32", "f32"),
       (9001, 72, 32000, "skewed", "bf16", "bf16"), (3000, 8, 128256, "skewed", "bf16", "f32"),
       (40000, 16, 262144, "skewed", "f16", "f32"), (200, 33, 511, "ignored", "bf16", "f32"),
       (300, 40, 512, "uniform", "bf16", "f32"), (64, 5000, 20, "uniform", "bf16", "f32"),
       (2000, 16, 1, "uniform", "f32", "f32"), (70000, 8, 300000, "skewed", "bf16", "f32"),
       (4097, 24, 1 << 20, "skewed", "f32", "f32"), (600, 24, 40, "skewed", "f32", "f32"), (66000, 8, 90, "uniform", "f16", "f32")]


@pytest.mark.parametrize("N,H,V,kind,dt,dE_dt", BWD)
@pytest.mark.parametrize("accumulate", [True, False])
def test_gradient(N, H, V, kind, dt, dE_dt, accumulate):
    g = torch.Generator().manual_seed(N + H + V)
    t = _tokens(kind, N, V, g)
    d = torch.randn(N, H, generator=g).to(DT[dt])
    d[t == IGN] = float("nan")                # a row that takes no part reaches nothing
    init = torch.randn(V, H, generator=g).to(DT[dE_dt]) if accumulate else torch.full((V, H), float("nan"), dtype=DT[dE_dt])
    dE = init.clone().cuda()
    o = flce.embed_bwd(t.cuda(), d.cuda(), dE=dE, scale=1.5, ignore_index=IGN,
                       flags=0 if accumulate else flce.FLAG_DW_OVERWRITE)
    assert o["status_code"] == flce.FLCE_OK
    want, mag, n = oo.embed_bwd(t.numpy(), np64(d), V, 1.5, IGN)
    base = np64(init) if accumulate else 0.0
    total = want + base
    bound = (n[:, None] + 3) * F32 * (mag + np.abs(base)) + 2 * ULP[dE_dt] * np.abs(total) + FLOOR[dE_dt]
    close(dE, total, bound)
    if accumulate:                            # rows without a token keep their bits
        assert torch.equal(dE.cpu()[n == 0], init[n == 0])
    else:
        assert torch.all(dE.cpu()[n == 0] == 0)


@pytest.mark.parametrize("dt,dE_dt,H,extra,offset", [("bf16", "f32", 72, 5, 1), ("f16", "f16", 72, 8, 8),
                                                     ("f32", "f32", 30, 2, 2), ("bf16", "bf16", 7, 1, 3)])
def test_gradient_strides(dt, dE_dt, H, extra, offset):
    g = torch.Generator().manual_seed(3)
    N, V = 700, 90
    t = _tokens("skewed", N, V, g)
    d = torch.randn(N, H, generator=g).to(DT[dt])
    dE = strided(torch.zeros(V, H, dtype=DT[dE_dt], device="cuda"), extra, offset)
    flce.embed_bwd(t.cuda(), strided(d.cuda(), extra, offset), dE=dE, ignore_index=IGN)
    want, mag, n = oo.embed_bwd(t.numpy(), np64(d), V, 1.0, IGN)
    close(dE, want, (n[:, None] + 3) * F32 * mag + 2 * ULP[dE_dt] * np.abs(want) + FLOOR[dE_dt])


@pytest.mark.parametrize("dt,dE_dt,H,extra,offset", [("bf16", "f32", 72, 5, 1), ("f16", "f16", 72, 8, 8), ("f16", "f16", 1003, 2, 3),
                                                     ("bf16", "bf16", 7, 1, 3), ("f32", "f32", 20000, 4, 0),
                                                     ("bf16", "bf16", 40000, 3, 1)])
@pytest.mark.parametrize("N", [3, 700])
def test_gradient_overwrites_a_table_with_a_pitch(dt, dE_dt, H, extra, offset, N):
    """Every row of dE is written, and the elements between the rows stay as they were."""
    g = torch.Generator().manual_seed(H + N)
    V = 61
    t = _tokens("skewed", N, V, g)
    d = torch.randn(N, H, generator=g).to(DT[dt])
    flat = torch.randn(V * (H + extra) + offset, generator=g).to(DT[dE_dt]).cuda()
    keep = flat.clone()
    view = lambda f: f[offset:].view(V, H + extra)  # noqa: E731
    dE = view(flat)[:, :H]
    dE.fill_(float("nan"))
    flce.embed_bwd(t.cuda(), d.cuda(), dE=dE, ignore_index=IGN, flags=flce.FLAG_DW_OVERWRITE)
    want, mag, n = oo.embed_bwd(t.numpy(), np64(d), V, 1.0, IGN)
    close(dE, want, (n[:, None] + 3) * F32 * mag + 2 * ULP[dE_dt] * np.abs(want) + FLOOR[dE_dt])
    assert torch.equal(view(flat)[:, H:], view(keep)[:, H:]) and torch.equal(flat[:offset], keep[:offset])


@pytest.mark.parametrize("N", [5, 1000, 70000])
def test_ignore_index_inside_the_vocabulary(N):
    """The usual padding id: its rows are zero, its gradient is nothing, and it is in range."""
    g = torch.Generator().manual_seed(N)
    V, H, pad = 50, 24, 7
    t = torch.randint(0, V, (N,), generator=g)
    t[::2] = pad
    E, d = torch.randn(V, H, generator=g), torch.randn(N, H, generator=g)
    d[t == pad] = float("nan")
    o = flce.embed_fwd(t.cuda(), E.cuda(), ignore_index=pad)
    assert o["status_code"] == flce.FLCE_OK
    assert np.array_equal(np64(o["out"]), oo.embed_fwd(t.numpy(), np64(E), 1.0, pad))
    b = flce.embed_bwd(t.cuda(), d.cuda(), V=V, ignore_index=pad)
    assert b["status_code"] == flce.FLCE_OK
    want, mag, n = oo.embed_bwd(t.numpy(), np64(d), V, 1.0, pad)
    assert n[pad] == 0
    close(b["dE"], want, (n[:, None] + 3) * F32 * mag)


def test_gradient_is_the_derivative_of_the_forward():
    """Central differences of L(E) = sum(c * embed(tokens, E)) in fp32: L is linear in E, so a
    difference over a step of 1 is exact up to the rounding of the two sums."""
    g = torch.Generator().manual_seed(5)
    N, H, V = 200, 24, 13
    t = _tokens("uniform", N, V, g).cuda()
    E = torch.randn(V, H, generator=g).cuda()
    c = torch.randn(N, H, generator=g).cuda()
    dE = flce.embed_bwd(t, c, V=V, scale=0.7, ignore_index=IGN)["dE"]
    for v, h in [(0, 0), (5, 23), (12, 7), (3, 11)]:
        L = []
        for s in (1.0, -1.0):
            Es = E.clone()
            Es[v, h] += s
            L.append((flce.embed_fwd(t, Es, scale=0.7, ignore_index=IGN)["out"].double() * c.double()).sum())
        diff = float(L[0] - L[1]) / 2
        n = int((t == v).sum())
        # n products of a value below 6 rounded to fp32 in each sum
        assert abs(diff - float(dE[v, h])) <= 4 * n * F32 * 6 * float(c.abs().max())


def test_same_bits_and_side_stream():
    g = torch.Generator().manual_seed(9)
    t = _tokens("skewed", 9000, 5000, g).cuda()
    d = torch.randn(9000, 200, generator=g).bfloat16().cuda()
    a = flce.embed_bwd(t, d, V=5000, ignore_index=IGN)["dE"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = flce.embed_bwd(t, d, V=5000, ignore_index=IGN, stream=s, check=False)["dE"]
    c = flce.embed_fwd(t, a, ignore_index=IGN, stream=s)["out"]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b)
    live = t != IGN
    assert torch.equal(c[live], a[t[live]]) and torch.all(c[~live] == 0)


def test_tokens_out_of_range_are_reported_and_left_out():
    t = torch.tensor([1, 5, -3, 2, IGN], device="cuda")
    E = torch.randn(5, 16, device="cuda")
    o = flce.embed_fwd(t, E)
    assert o["status_code"] == flce.FLCE_ERR_TARGET_RANGE
    assert torch.equal(o["out"][0], E[1]) and torch.equal(o["out"][3], E[2])
    assert torch.all(o["out"][[1, 2, 4]] == 0)
    b = flce.embed_bwd(t, torch.ones(5, 16, device="cuda"), V=5)
    assert b["status_code"] == flce.FLCE_ERR_TARGET_RANGE
    assert b["dE"].sum(dim=1).tolist() == [0, 16, 16, 0, 0]
    assert flce.embed_bwd(t[:1], torch.ones(1, 16, device="cuda"), V=5)["status_code"] == flce.FLCE_OK


def test_offsets_past_32_bits():
    """A table of more than 2^32 bytes: the last rows are read and written."""
    V, H = 1_200_000, 2048
    E = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    E[V - 1] = 3.0
    E[V - 2, -1] = 2.0
    t = torch.tensor([V - 1, V - 2, 0], device="cuda")
    out = flce.embed_fwd(t, E)["out"]
    assert torch.all(out[0] == 3) and float(out[1, -1]) == 2 and torch.all(out[2] == 0)
    flce.embed_bwd(t, torch.ones(3, H, dtype=torch.bfloat16, device="cuda"), dE=E)
    assert torch.all(E[V - 1] == 4) and float(E[V - 2, -1]) == 3 and torch.all(E[0] == 1) and torch.all(E[1] == 0)

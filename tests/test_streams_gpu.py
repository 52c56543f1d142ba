"""Calls on a given stream: every tensor that a call makes comes from that stream's memory, so no
kernel that another stream still has queued can be using it, and the results are those of the
current stream's call."""

import pytest
import torch

from linear_cross_entropy_logits_gb300 import build as B
from linear_cross_entropy_logits_gb300 import flce

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    flce.load()


def _owner(t):
    """The stream whose memory t lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def _calls():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    x, res, w, W = r(300, 200), r(300, 200), r(200), r(900, 200)
    t = torch.randint(0, 900, (300,), generator=g).cuda()
    p = flce.ckpt8_pack(x)
    rstd = torch.ones(300, device="cuda")
    X, V = r(256, 128), r(1024, 128)
    y = torch.randint(0, 1024, (256,), generator=g).cuda()
    Xt, Vt = r(256, 192), r(1024, 192)
    return {
        "embed_fwd": lambda **k: flce.embed_fwd(t, W, check=False, **k),
        "embed_bwd": lambda **k: flce.embed_bwd(t, x, V=900, **k),
        "rmsnorm_fwd": lambda **k: flce.rmsnorm_fwd(x, w, res, want_y8=True, want_h8=True, **k),
        "rmsnorm_bwd": lambda **k: flce.rmsnorm_bwd(x, w, rstd, res, **k),
        "ckpt8_pack": lambda **k: flce.ckpt8_pack(x, **k),
        "ckpt8_dw": lambda **k: flce.ckpt8_dw(res, p["q"], p["scale"], **k),
        "fwd_bwd": lambda **k: flce.fwd_bwd(X, V, y, **k),
        "fused_linear_jsd": lambda **k: flce.fused_linear_jsd(X, V, Xt, Vt, y, **k),
    }


@pytest.mark.parametrize("name", ["embed_fwd", "embed_bwd", "rmsnorm_fwd", "rmsnorm_bwd", "ckpt8_pack", "ckpt8_dw", "fwd_bwd",
                                  "fused_linear_jsd"])
def test_what_a_call_makes_belongs_to_its_stream(name):
    call = _calls()[name]
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert got.keys() == want.keys()
    for k, t in got.items():
        if torch.is_tensor(t):
            assert _owner(t) == s.cuda_stream, k
            if k not in ("workspace", "q", "y8", "h8"):
                assert torch.equal(t, want[k]), k
            elif k != "workspace":
                assert torch.equal(t.float(), want[k].float()), k


def test_given_outputs_stay_the_callers():
    x = torch.randn(64, 128, device="cuda")
    out = {"y": torch.empty_like(x), "rstd": torch.empty(64, device="cuda")}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = flce.rmsnorm_fwd(x, x[0].contiguous(), outputs=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert o["y"] is out["y"] and o["rstd"] is out["rstd"]
    want = flce.rmsnorm_fwd(x, x[0].contiguous())
    assert torch.equal(o["y"], want["y"]) and torch.equal(o["rstd"], want["rstd"])

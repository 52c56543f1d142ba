"""Host-side checks of the embedding, RMS norm and 8-bit checkpoint operators: their structs
match the header, their refusals come before any CUDA call, the binding's argument checks, and
the oracles they are tested against (the oracle's gradients against differences)."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from linear_cross_entropy_logits_gb300 import build as B
from linear_cross_entropy_logits_gb300 import flce, torch_ops
from oracle import ops_oracle as oo
from ops_util import DT, F32, FLOOR, ULP, close

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNS, WS = flce.FLCE_ERR_INVALID_ARG, flce.FLCE_ERR_UNSUPPORTED, flce.FLCE_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return flce.load()


STRUCTS = [(flce.FlceEmbedArgs, "flce_embed_args"), (flce.FlceRmsnormArgs, "flce_rmsnorm_args"),
           (flce.FlceRmsnormBwdArgs, "flce_rmsnorm_bwd_args"), (flce.FlceCkpt8Args, "flce_ckpt8_args"),
           (flce.FlceCkpt8DwArgs, "flce_ckpt8_dw_args")]


def test_struct_layouts_match_c(lib, tmp_path):
    src = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{ROOT}/include/flce.h"', "int main(void){"]
    for cls, cname in STRUCTS:
        src.append(f'printf("%zu\\n", sizeof({cname}));')
        src += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(src + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-o", str(exe), str(c)], check=True)
    vals = iter(int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    for cls, _ in STRUCTS:
        assert next(vals) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert getattr(cls, f).offset == next(vals), f


def _set(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _embed(**kw):
    return _set(flce.FlceEmbedArgs(4, 16, 10, 1, 0, 0x1000, -100, 1.0, 0, 0x2000, 16, 0x3000, 16, 0x4000, 16, 0x5000, 16,
                                   0x10000, 1 << 20, None), kw)


@pytest.mark.parametrize("kw", [dict(N=-1), dict(H=0), dict(V=0), dict(V=1 << 31), dict(dtype=3), dict(scale=NAN),
                                dict(scale=INF), dict(tokens=None), dict(tokens=0x1004), dict(E=None), dict(out=None),
                                dict(ldE=15), dict(ldout=15), dict(E=0x2001), dict(out=0x3001), dict(flags=1),
                                dict(status=0x6001)])
def test_embed_fwd_refusals(lib, kw):
    assert lib.flce_embed_fwd(_embed(**kw), None) == BAD


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(dtype=9), BAD), (dict(dE_dtype=2), UNS), (dict(dout=None), BAD), (dict(dE=None), BAD),
    (dict(lddout=8), BAD), (dict(lddE=8), BAD), (dict(dE=0x5002), BAD), (dict(workspace=None), BAD),
    (dict(workspace=0x10010), BAD), (dict(workspace_bytes=64), WS), (dict(flags=1), BAD), (dict(tokens=None), BAD)])
def test_embed_bwd_refusals(lib, kw, code):
    assert lib.flce_embed_bwd(_embed(**kw), None) == code


def _norm(**kw):
    return _set(flce.FlceRmsnormArgs(4, 16, 1, 1e-5, 0.0, 0, 0x1000, 16, None, 0, 0x2000, None, 0, 0x3000, 16, 0x4000,
                                     None, 0, None, None, 0, None), kw)


@pytest.mark.parametrize("kw", [dict(N=-1), dict(H=0), dict(dtype=5), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN),
                                dict(eps=INF), dict(weight_offset=NAN), dict(flags=4), dict(x=None), dict(x=0x1001),
                                dict(ldx=15), dict(weight=None), dict(residual=0x5000), dict(h=0x5000), dict(ldy=3),
                                dict(y=0x3001), dict(rstd=0x4002), dict(y8=0x5000, ldy8=16), dict(y8=0x5000, y8_scale=0x6000),
                                dict(h8=0x5000, ldh8=16), dict(h8=0x5000, h8_scale=0x6000, ldh8=15)])
def test_rmsnorm_fwd_refusals(lib, kw):
    assert lib.flce_rmsnorm_fwd(_norm(**kw), None) == BAD


def _norm_bwd(**kw):
    return _set(flce.FlceRmsnormBwdArgs(4, 16, 1, 0, 0.0, 0, 0x1000, 16, 0x2000, 16, None, 0, None, 0x3000, 0x4000, None, 0,
                                        0x5000, 16, 0x6000, 0x10000, 1 << 30), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(dtype=5), BAD), (dict(dweight_dtype=2), UNS), (dict(dy=None), BAD), (dict(lddy=1), BAD),
    (dict(h=None), BAD), (dict(h8=0x7000, ldh8=16, h8_scale=0x8000), BAD), (dict(h=None, h8=0x7000, ldh8=16), BAD),
    (dict(rstd=None), BAD), (dict(weight=None), BAD), (dict(dh=0x7001, lddh=16), BAD), (dict(lddx=2), BAD),
    (dict(workspace=None), BAD), (dict(workspace=0x10004), BAD), (dict(workspace_bytes=100), WS), (dict(flags=1), BAD),
    (dict(weight_offset=INF), BAD)])
def test_rmsnorm_bwd_refusals(lib, kw, code):
    assert lib.flce_rmsnorm_bwd(_norm_bwd(**kw), None) == code


@pytest.mark.parametrize("kw", [dict(N=-1), dict(H=0), dict(dtype=4), dict(flags=1), dict(x=None), dict(q=None),
                                dict(scale=None), dict(ldx=8), dict(ldq=8), dict(x=0x1001), dict(scale=0x3002)])
def test_pack_refusals(lib, kw):
    assert lib.flce_ckpt8_pack(_set(flce.FlceCkpt8Args(4, 16, 1, 0, 0x1000, 16, 0x2000, 16, 0x3000), kw), None) == BAD


def _dw(**kw):
    return _set(flce.FlceCkpt8DwArgs(4, 8, 16, 1, 0, 0, 0, 0x1000, 8, 0x2000, 16, 0x3000, 0x4000, 16, 0x10000, 1 << 30, None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(dtype=8), BAD), (dict(dW_dtype=2), UNS),
    (dict(dtype=0, dW_dtype=1), UNS), (dict(dy=None), BAD), (dict(q=None), BAD), (dict(scale=None), BAD),
    (dict(dW=None), BAD), (dict(lddy=7), BAD), (dict(ldq=15), BAD), (dict(lddW=15), BAD), (dict(dW=0x4002), BAD),
    (dict(workspace=None), BAD), (dict(workspace=0x10020), BAD), (dict(workspace_bytes=8), WS), (dict(flags=2), BAD)])
def test_dw_refusals(lib, kw, code):
    assert lib.flce_ckpt8_dw(_dw(**kw), None) == code


def test_null_argument_structs(lib):
    for name in ("embed_fwd", "embed_bwd", "rmsnorm_fwd", "rmsnorm_bwd", "ckpt8_pack", "ckpt8_dw"):
        assert getattr(lib, "flce_" + name)(None, None) == BAD


def test_no_rows_need_no_pointers(lib):
    """N = 0 with nothing to overwrite returns at once (an empty tensor's pointer is null)."""
    assert lib.flce_embed_fwd(_embed(N=0, tokens=None, E=None, out=None), None) == flce.FLCE_OK
    assert lib.flce_embed_bwd(_embed(N=0, tokens=None, dout=None, workspace=None, workspace_bytes=0), None) == flce.FLCE_OK
    assert lib.flce_rmsnorm_fwd(_norm(N=0, x=None, y=None, rstd=None), None) == flce.FLCE_OK
    assert lib.flce_rmsnorm_bwd(_norm_bwd(N=0, dy=None, h=None, rstd=None, dx=None), None) == flce.FLCE_OK
    assert lib.flce_ckpt8_pack(flce.FlceCkpt8Args(0, 16, 1, 0, None, 16, None, 16, None), None) == flce.FLCE_OK
    assert lib.flce_ckpt8_dw(_dw(M=0, dy=None, q=None, scale=None), None) == flce.FLCE_OK


def test_workspace_sizes(lib):
    assert lib.flce_embed_workspace_size(-1, 4, 4) == 0 and lib.flce_embed_workspace_size(4, 0, 4) == 0
    assert lib.flce_embed_workspace_size(0, 4, 4) > 0
    assert lib.flce_rmsnorm_workspace_size(4, 0) == 0 and lib.flce_rmsnorm_workspace_size(0, 8) > 0
    size = lib.flce_ckpt8_dw_workspace_size
    assert size(_dw(K=0)) == 0 and size(_dw(dtype=7)) == 0 and size(None) == 0 and size(_dw(M=0)) > 0
    big = dict(M=4096, N=1024, K=2048, lddy=1024, ldq=2048, lddW=2048)
    plain = size(_dw(**big))
    assert size(_dw(**big, flags=1)) < plain                              # no tensor cores, no parts
    assert size(_dw(**dict(big, lddy=1025))) - plain >= 4096 * 1024 * 2   # dy copied to a TMA pitch
    assert size(_dw(**dict(big, ldq=2049))) - plain >= 4096 * 2048        # q copied
    assert size(_dw(**big, dtype=0)) - plain >= 3 * 4096 * 1024 * 2       # fp32 dy: three bf16 terms


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("N,K", [(256, 256), (1024, 4352), (1024, 4096), (2048, 2048), (4096, 4608), (520, 2008)])
def test_dw_workspace_stays_within_the_header(lib, dtype, N, K):
    """Parts of at most 75 tiles (152 SMs), 16 of 256 KB each, beside the copies of fp32 dy."""
    for M in (1, 1000, 8192, 32768, 65536, 1 << 20, 1 << 24, 1 << 29):
        size = lib.flce_ckpt8_dw_workspace_size(_dw(M=M, N=N, K=K, lddy=N, ldq=(K + 15) & ~15, lddW=K, dtype=dtype))
        copy = 6 * ((M + 63) // 64 * 64) * N if dtype == 0 else 0
        assert 0 < size - copy <= 300 * 2 ** 20 + 2048


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    x, w = torch.randn(4, 8), torch.randn(8)
    for f in (lambda: flce.rmsnorm_fwd(x, w), lambda: flce.ckpt8_pack(x),
              lambda: flce.embed_fwd(torch.zeros(3, dtype=torch.int64), x),
              lambda: flce.embed_bwd(torch.zeros(4, dtype=torch.int64), x, V=3),
              lambda: flce.ckpt8_dw(x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_matrix_check():
    """The binding's check of a matrix operand, which needs no GPU."""
    cpu = torch.device("cpu")
    x = torch.randn(6, 8)
    assert flce._matrix("x", x, 6, 8, torch.float32, cpu) == (x.data_ptr(), 8)
    assert flce._matrix("x", x[:, 2:5], 6, 3, torch.float32, cpu) == (x.data_ptr() + 8, 8)
    for bad in (x.t(), x[:, ::2], x.half(), x[:1].expand(6, 8), x[:5]):
        with pytest.raises(ValueError):
            flce._matrix("x", bad, 6, bad.shape[1], torch.float32, cpu)
    with pytest.raises(ValueError):
        flce._dense("v", x[:, 0], (6,), torch.float32, cpu)
    with pytest.raises(ValueError):
        flce._dense("s", x[:, :4], (6, 4), torch.float32, cpu)


class _Stream:
    device = torch.device("cpu")


@pytest.fixture
def streams(monkeypatch):
    """The binding on the CPU with stand-ins for streams and kernels: a log of (event, current
    stream, tensor) for allocations, launches and records."""
    log, cur = [], [_Stream()]

    class use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            cur.append(self.s)

        def __exit__(self, *a):
            cur.pop()

    def logged(make):
        def f(*a, **kw):
            t = make(*a, **kw)
            log.append(("new", cur[-1], t))
            return t
        return f

    for name in ("empty", "zeros", "empty_strided", "empty_like"):
        monkeypatch.setattr(torch, name, logged(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: cur[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("record", s, t)))
    monkeypatch.setattr(flce, "_cuda_2d", lambda name, t: (t.device, t.shape, flce.DTYPES[t.dtype]))
    monkeypatch.setattr(flce, "_launch", lambda fn, where, args, dev: log.append(("launch", cur[-1], None)))
    return log, cur


def _call(name, x, status, stream):
    t, kw = torch.zeros(6, dtype=torch.int64), dict(check=False, status=status, stream=stream)
    if name == "embed_fwd":
        return flce.embed_fwd(t, x, **kw)
    if name == "embed_bwd":
        return flce.embed_bwd(t, x, V=3, **kw)
    if name == "rmsnorm_fwd":
        return flce.rmsnorm_fwd(x, x[0].clone(), x.clone(), want_y8=True, want_h8=True, stream=stream)
    if name == "rmsnorm_bwd":
        return flce.rmsnorm_bwd(x, x[0].clone(), torch.ones(6), x.clone(), stream=stream)
    if name == "ckpt8_pack":
        return flce.ckpt8_pack(x, stream=stream)
    return flce.ckpt8_dw(x, x.to(torch.float8_e4m3fn), torch.ones(6, 1), **kw)


@pytest.mark.parametrize("name", ["embed_fwd", "embed_bwd", "rmsnorm_fwd", "rmsnorm_bwd", "ckpt8_pack", "ckpt8_dw"])
def test_a_given_stream_owns_what_the_call_makes(lib, streams, name):
    """Outputs and workspaces come from the given stream's memory: another's block may still be in
    use by kernels that the given stream does not wait for. And memory is not handed out again
    before the caller's stream is done with the outputs, and the given one with the inputs."""
    log, cur = streams
    x, s, status = torch.randn(6, 8), _Stream(), torch.zeros(1, dtype=torch.int32)
    log.clear()
    o = _call(name, x, status, s)
    mine = [t for t in o.values() if torch.is_tensor(t) and t is not status]
    new = [(st, t) for ev, st, t in log if ev == "new"]
    for t in mine:
        assert any(t is u and st is s for st, u in new)
    assert [st for ev, st, _ in log if ev == "launch"] == [s]
    rec = [(st, t) for ev, st, t in log if ev == "record"]
    for t in mine:
        assert any(t is u and st is cur[-1] for st, u in rec)
    assert any(x is u and st is s for st, u in rec)
    # the stream that is current anyway: nothing to record
    log.clear()
    _call(name, x, status, cur[-1])
    assert not [e for e in log if e[0] == "record"]


def test_results_hold_nothing_that_the_call_did_not_write(lib, streams):
    """Outputs of an earlier call given again, with fewer of them wanted."""
    x, w = torch.randn(6, 8), torch.ones(8)
    a = flce.rmsnorm_fwd(x, w, x.clone(), want_y8=True, want_h8=True)
    assert set(a) == {"rstd", "y", "h", "y8", "y8_scale", "h8", "h8_scale"}
    b = flce.rmsnorm_fwd(x, w, outputs=a)
    assert set(b) == {"rstd", "y"} and b["y"] is a["y"] and b["rstd"] is a["rstd"]
    assert set(flce.rmsnorm_fwd(x, w, want_y=False, want_h8=True, outputs=a)) == {"rstd", "h8", "h8_scale"}
    c = flce.rmsnorm_bwd(x, w, a["rstd"], x)
    assert set(c) == {"dx", "dweight", "workspace"}
    assert set(flce.rmsnorm_bwd(x, w, a["rstd"], x, want_dweight=False, outputs=c)) == {"dx"}
    d = flce.rmsnorm_bwd(x, w, a["rstd"], x, want_dx=False, outputs=c)
    assert set(d) == {"dweight", "workspace"} and d["dweight"] is not c["dweight"]
    p = flce.ckpt8_pack(x)
    assert set(flce.ckpt8_pack(x, outputs=dict(p, y=x))) == {"q", "scale"}


def test_a_stream_of_another_device_is_refused(streams):
    s = _Stream()
    s.device = torch.device("meta")
    with pytest.raises(ValueError, match="stream"):
        flce.ckpt8_pack(torch.randn(2, 8), stream=s)


def test_kernels_that_start_early_do_not_read_by_the_read_only_path():
    """A kernel that may start before the one it follows has finished (after_previous) reads memory
    that is written during its life: neither it nor its helpers may use loads for constant data."""
    seen = 0
    for name in os.listdir(B.CSRC):
        with open(os.path.join(B.CSRC, name)) as f:
            src = f.read()
        if "after_previous();" not in src:
            continue
        assert "__ldg(" not in src and "ld.global.nc" not in src, name
        for kernel in src.split("__global__")[1:]:
            head, body = kernel.split("{", 1)
            if "after_previous();" in body.split("\n}\n")[0]:
                seen += 1
                assert "__restrict__" not in head, head
    assert seen >= 5


@pytest.fixture
def plain_ckpt8(monkeypatch):
    """linear_ckpt8 on the CPU: packing and the weight gradient in plain torch; counts the packings."""
    calls = []

    def pack(x):
        calls.append(x.shape)
        return {"q": x.detach().to(torch.float8_e4m3fn), "scale": torch.ones(len(x), (x.shape[1] + 127) // 128)}

    def dw(dy, q, scale, *, dW, flags, check):
        dW.copy_(dy.float().t() @ q.float())

    monkeypatch.setattr(flce, "ckpt8_pack", pack)
    monkeypatch.setattr(flce, "ckpt8_dw", dw)
    return calls


def test_linear_ckpt8_packs_only_for_a_gradient_of_its_weight(plain_ckpt8):
    g = torch.Generator().manual_seed(1)
    x, W = torch.randn(3, 5, 40, generator=g).requires_grad_(), torch.randn(7, 40, generator=g).requires_grad_()
    want = x.detach() @ W.detach().t()
    with torch.no_grad():
        assert torch.equal(torch_ops.linear_ckpt8(x, W), want)
    with torch.inference_mode():
        torch_ops.linear_ckpt8(x, W)
    frozen = torch_ops.linear_ckpt8(x, W.detach())
    assert frozen.requires_grad and not plain_ckpt8
    frozen.sum().backward()
    # sums of 7 and of 15 fp32 terms
    Wd = W.detach().double()
    assert ((x.grad.double() - Wd.sum(0)).abs() <= 7 * 2.0 ** -24 * Wd.abs().sum(0)).all()
    y = torch_ops.linear_ckpt8(x.detach(), W)
    assert torch.equal(y.detach(), want) and plain_ckpt8 == [(15, 40)]
    y.sum().backward()
    q = x.detach().reshape(15, 40).to(torch.float8_e4m3fn).double()
    assert ((W.grad.double() - q.sum(0)).abs() <= 15 * 2.0 ** -24 * q.abs().sum(0)).all()


@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16])
def test_linear_ckpt8_under_autocast(plain_ckpt8, x_dtype):
    """fp32 weights, a 16-bit product: gradients come back in the types of x and W."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(6, 40, generator=g).to(x_dtype).requires_grad_()
    W = torch.randn(7, 40, generator=g).requires_grad_()
    with torch.autocast("cpu", torch.bfloat16):
        y = torch_ops.linear_ckpt8(x, W)
    assert y.dtype is torch.bfloat16
    c = torch.randn(6, 7, generator=g).bfloat16()
    y.backward(c)
    assert x.grad.dtype is x_dtype and W.grad.dtype is torch.float32
    Wb = W.detach().bfloat16().double()
    # sums of 7 products of bf16 values, rounded to bf16
    close = lambda a, b, tol: ((a.double() - b).abs() <= tol).all()  # noqa: E731
    assert close(x.grad, c.double() @ Wb, 2.0 ** -8 * (c.double().abs() @ Wb.abs()))
    q = x.detach().to(torch.float8_e4m3fn).double()
    assert close(W.grad, c.double().t() @ q, 2.0 ** -20 * (c.double().abs().t() @ q.abs()))


def _storages(outs):
    return [t.untyped_storage()._cdata for t in outs]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("checkpoint8", [True, False])
def test_norm_op_outputs_are_tensors_of_their_own(monkeypatch, dtype, residual, checkpoint8):
    """The autograd form on the CPU, with the norm's kernels replaced by plain tensors: outputs of
    a custom op share no memory with one another, the empty ones included."""
    def norm(x, weight, res, *, eps, weight_offset, want_h8):
        N, H = x.shape
        o = {"y": x.clone(), "rstd": torch.ones(N)}
        if res is not None:
            o["h"] = x + res
        if want_h8:
            o["h8"], o["h8_scale"] = x.to(torch.float8_e4m3fn), torch.ones(N, (H + 127) // 128)
        return o

    monkeypatch.setattr(flce, "rmsnorm_fwd", norm)
    x, w = torch.randn(6, 40).to(dtype).requires_grad_(), torch.ones(40, dtype=dtype, requires_grad=True)
    r = torch.randn(6, 40).to(dtype) if residual else None
    out = torch_ops.add_rms_norm(x, w, r, checkpoint8=checkpoint8)
    y, h = out if residual else (out, None)
    assert y.requires_grad and y.dtype is dtype and (h is None or h.requires_grad)
    outs = torch_ops.add_rms_norm_op(x, w, r, 1e-6, 0.0, checkpoint8)
    assert len(set(_storages(outs))) == 5
    fake = [dtype, dtype, torch.float32, torch.float8_e4m3fn, torch.float32]
    assert [t.dtype for t in outs] == fake and [t.numel() == 0 for t in outs[1:]] == [not residual, False] + 2 * [not checkpoint8]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("need_x", [True, False])
@pytest.mark.parametrize("need_w", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_head_op_outputs_are_tensors_of_their_own(monkeypatch, dtype, need_x, need_w, with_bias):
    """The same of the head's op, in evaluation and with either gradient."""
    def head(X, W, targets, bias, *, want_dX, **kw):
        f = lambda n: torch.zeros(n)  # noqa: E731
        o = {"loss": f(1), "z_loss": f(1), "acc": f(1), "lse": f(len(X)), "pred": torch.zeros(len(X), dtype=torch.int64)}
        if want_dX:
            o["dX"] = torch.zeros_like(X)
        return o

    monkeypatch.setattr(flce, "fwd_bwd", head)
    X, W = torch.randn(5, 8, dtype=dtype, requires_grad=need_x), torch.randn(7, 8, dtype=dtype, requires_grad=need_w)
    b = torch.zeros(7, dtype=dtype, requires_grad=need_w) if with_bias else None
    t = torch.zeros(5, dtype=torch.int64)
    assert torch_ops.fused_linear_cross_entropy(X, W, t, b).requires_grad == (need_x or need_w)
    outs = torch_ops.fused_linear_cross_entropy_op(X, W, t, b, None, -100, "mean", 0.0, need_x, need_w, True)
    assert len(set(_storages(outs))) == 8


# ---- the oracles

def test_e4m3_rounding_against_torch():
    """Every quotient near every e4m3 value rounds as torch's conversion does."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mids = (codes[1:] + codes[:-1]) / 2
    x = torch.cat([codes, mids, mids * (1 + 2.0 ** -20), mids * (1 - 2.0 ** -20), torch.rand(5000).double() * 448])
    x = torch.cat([x, -x]).float()
    assert np.array_equal(oo.round_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_block_scales_are_the_smallest_that_fit():
    x = np.random.default_rng(0).standard_normal((50, 300)) * np.exp(np.random.default_rng(1).standard_normal((50, 1)) * 8)
    x[0, :128] = 0
    x[1, :128] = 448.0
    x[2, :128] = np.nextafter(448.0, 1e9)
    e = oo.block_exponent(x)
    assert e[0, 0] == 0 and e[1, 0] == 0 and e[2, 0] == 1
    for b in range(3):
        m = np.abs(x[:, b * 128:(b + 1) * 128]).max(axis=1)
        live = m > 0
        assert np.all(m[live] <= 448 * np.exp2(e[live, b])) and np.all(m[live] > 448 * np.exp2(e[live, b] - 1))


def test_rmsnorm_oracle_gradient_against_differences():
    rng = np.random.default_rng(2)
    h, w, c = rng.standard_normal((4, 9)), rng.standard_normal(9), rng.standard_normal((4, 9))
    _, rstd = oo.rmsnorm_fwd(h, w, 1e-3, 0.5)
    dx, dw, _, _ = oo.rmsnorm_bwd(c, h, rstd, w, 0.5)
    L = lambda hh, ww: (c * oo.rmsnorm_fwd(hh, ww, 1e-3, 0.5)[0]).sum()  # noqa: E731
    st = 1e-6
    for i in range(4):
        for j in range(9):
            d = np.zeros_like(h)
            d[i, j] = st
            assert abs((L(h + d, w) - L(h - d, w)) / (2 * st) - dx[i, j]) < 1e-7
    for j in range(9):
        d = np.zeros_like(w)
        d[j] = st
        assert abs((L(h, w + d) - L(h, w - d)) / (2 * st) - dw[j]) < 1e-7


def test_embed_oracle_gradient_against_differences():
    rng = np.random.default_rng(3)
    t = np.array([0, 2, 2, -100, 1, 2])
    E, c = rng.standard_normal((4, 5)), rng.standard_normal((6, 5))
    dE, _, n = oo.embed_bwd(t, c, 4, 1.3, -100)
    assert n.tolist() == [1, 1, 3, 0]
    L = lambda e: (c * oo.embed_fwd(t, e, 1.3, -100)).sum()  # noqa: E731
    for v in range(4):
        for j in range(5):
            d = np.zeros_like(E)
            d[v, j] = 1.0
            assert abs((L(E + d) - L(E - d)) / 2 - dE[v, j]) < 1e-12


# ---- planted mistakes: the GPU tests' comparisons pass a right result in the type's rounding and
# reject each of these

def _rounded(a, dt):
    return torch.from_numpy(np.asarray(a)).to(DT[dt])


def _check(good, bad, check):
    check(good)
    for what, b in bad.items():
        try:
            check(b)
        except AssertionError:
            continue
        pytest.fail(f"not rejected: {what}")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_planted_mistakes_in_the_norm(dt):
    rng = np.random.default_rng(5)
    N, H, off, eps = 40, 300, 0.25, 1e-5
    # (values of the type, as the tests' inputs are)
    r = lambda *s: _rounded(rng.standard_normal(s), dt).double().numpy()  # noqa: E731
    h, dy, dh, w = r(N, H), r(N, H), r(N, H), r(H)
    y, rstd = oo.rmsnorm_fwd(h, w, eps, off)
    RSTD = 80 * F32
    _check(_rounded(y, dt), {
        "no offset": _rounded(oo.rmsnorm_fwd(h, w, eps, 0.0)[0], dt),
        "one column short": _rounded(h * (w + off) / np.sqrt(np.mean(h[:, :-1] ** 2, axis=1) + eps)[:, None], dt),
        "mean over the padded row": _rounded(h * (w + off) / np.sqrt((h * h).sum(axis=1) / 304 + eps)[:, None], dt),
    }, lambda got: close(got, y, (ULP[dt] + RSTD) * np.abs(y) + FLOOR[dt]))
    dx, dw, mag, wmag = oo.rmsnorm_bwd(dy, h, rstd, w, off, dh)
    xh = h * rstd[:, None]
    g = dy * (w + off)
    _check(_rounded(dx, dt), {
        "no mean": _rounded(rstd[:, None] * g + dh, dt),
        "no offset": _rounded(oo.rmsnorm_bwd(dy, h, rstd, w, 0.0, dh)[0], dt),
        "no residual gradient": _rounded(dx - dh, dt),
        "rstd once": _rounded(g * rstd[:, None] - h * np.mean(g * xh, axis=1, keepdims=True) + dh, dt),
    }, lambda got: close(got, dx, ULP[dt] * np.abs(dx) + F32 * mag + FLOOR[dt]))
    _check(torch.from_numpy(dw).float(), {
        "of the dx written in dy's place": torch.from_numpy((dx * xh).sum(axis=0)).float(),
        "a row left out": torch.from_numpy((dy[:-1] * xh[:-1]).sum(axis=0)).float(),
        "of h": torch.from_numpy((dy * h).sum(axis=0)).float(),
    }, lambda got: close(got, dw, F32 * ((N + 8) * wmag + np.abs(dw))))


def test_planted_mistakes_in_the_packing():
    x = np.random.default_rng(6).standard_normal((30, 300))
    q, s = oo.pack(x)

    def check(qs):
        assert np.array_equal(qs[0], q) and np.array_equal(qs[1], s)

    half = np.clip(x / oo.spread(s / 2, 300), -448, 448)
    _check((q.copy(), s.copy()), {
        "a scale too small": (oo.round_e4m3(half), s / 2),
        "a scale too large": (oo.round_e4m3(x / oo.spread(2 * s, 300)), 2 * s),
        "truncated": (np.sign(q) * np.minimum(np.abs(q), oo.round_e4m3(np.abs(x) / oo.spread(s, 300) * (1 - 2.0 ** -5))), s),
    }, check)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_planted_mistakes_in_the_embedding_gradient(dt):
    rng = np.random.default_rng(7)
    N, H, V, scale = 200, 24, 20, 1.5
    t = rng.integers(0, V, N)
    t[::9] = -100
    d = _rounded(rng.standard_normal((N, H)), dt).double().numpy()
    want, mag, n = oo.embed_bwd(t, d, V, scale, -100)
    one = np.flatnonzero(t == t[1])[1]            # a token's second row
    less, zero = t.copy(), t.copy()
    less[one] = -100
    zero[t == -100] = 0
    of = lambda tt, sc=scale: _rounded(oo.embed_bwd(tt, d, V, sc, -100)[0], dt)  # noqa: E731
    bound = (n[:, None] + 3) * F32 * mag + 2 * ULP[dt] * np.abs(want) + FLOOR[dt]
    _check(of(t), {"a token's second row left out": of(less), "ignored rows counted": of(zero), "no scale": of(t, 1.0),
                   "another token's row": of(np.where(np.arange(N) == one, (t + 1) % V, t))},
           lambda got: close(got, want, bound))


@pytest.mark.parametrize("wdt", ["f32", "bf16"])
def test_planted_mistakes_in_the_weight_gradient(wdt):
    rng = np.random.default_rng(8)
    M, N, K = 130, 40, 300
    dy = _rounded(rng.standard_normal((M, N)), "bf16").double().numpy()
    q, s = oo.pack(rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1))))
    x = q * oo.spread(s, K)
    want = dy.T @ x
    mag = np.abs(dy).T @ np.abs(x)
    bound = M * 2.0 ** -23 * mag + 2 * ULP[wdt] * np.abs(want) + FLOOR[wdt]
    next_block = q * oo.spread(np.roll(s, 1, axis=1), K)
    late = q * oo.spread(np.roll(s, 1, axis=0), K)
    _check(_rounded(want, wdt), {"a row left out": _rounded(dy[:-1].T @ x[:-1], wdt), "the neighbouring block's scale": _rounded(dy.T @ next_block, wdt),
                                 "the neighbouring row's scale": _rounded(dy.T @ late, wdt), "no scale": _rounded(dy.T @ q, wdt),
                                 "a step of rows twice": _rounded(want + dy[64:128].T @ x[64:128], wdt)},
           lambda got: close(got, want, bound))

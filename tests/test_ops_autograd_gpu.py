"""The differentiable forms of the operators around the head, and the example step that runs all
of them, against plain PyTorch models in float64.

Bounds (2-norm of the difference over 2-norm). fp32 without checkpoints: 1e-5, as the package's
other fp32 results. An e4m3 value is within 2^-4 of its own, 2^-4 / sqrt(3) = 0.036 as an rms at
most, and a gradient is linear in the checkpoint that it reads: 0.036 for it alone, 0.05 where the
roundings of a bf16 model (a few times 2^-9 rms) come on top."""

import importlib.util
import os

import pytest
import torch

from linear_cross_entropy_logits_gb300 import build as B
from linear_cross_entropy_logits_gb300 import flce, torch_ops
from ops_util import np64
from parity_util import rel_fro

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    flce.load()


def _leaf(t):
    return t.detach().clone().requires_grad_()


def _norm(h, w, eps, off=0.0):
    return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * (w + off)


def _near(got, want, tol):
    for a, b in zip(got, want):
        assert a.shape == b.shape
        assert rel_fro(np64(a), np64(b)) <= tol


def test_embedding():
    g = torch.Generator().manual_seed(0)
    E = torch.randn(50, 24, generator=g).cuda()
    t = torch.randint(0, 50, (6, 9), generator=g).cuda()
    t[2, 3] = -100
    a, r = _leaf(E), _leaf(E.double())
    out = torch_ops.embedding(t, a, scale=3.0)
    ref = torch.where((t >= 0)[..., None], r[t.clamp(min=0)] * 3.0, 0.0)
    c = torch.randn(out.shape, generator=g).cuda()
    (out * c).sum().backward()
    (ref * c.double()).sum().backward()
    _near((out, a.grad), (ref, r.grad), 1e-6)
    assert a.grad.dtype == E.dtype


def test_embedding_of_tokens_out_of_range():
    E = _leaf(torch.randn(5, 16, device="cuda"))
    t = torch.tensor([[1, 5], [-3, -100]], device="cuda")
    out = torch_ops.embedding(t, E)
    assert torch.equal(out[0, 0], E[1]) and torch.all(out[0, 1] == 0) and torch.all(out[1] == 0)
    out.sum().backward()
    assert E.grad.sum(dim=1).tolist() == [0, 16, 0, 0, 0]
    for bad in (t, t[:1], t[1:]):
        with pytest.raises(flce.FlceError) as e:
            torch_ops.embedding(bad, E, check=True)
        assert e.value.code == flce.FLCE_ERR_TARGET_RANGE
    assert torch.equal(torch_ops.embedding(t[1:, 1:], E, check=True), torch.zeros(1, 1, 16, device="cuda"))


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("checkpoint8,tol", [(False, 1e-5), (True, 0.036)])
def test_add_rms_norm(residual, checkpoint8, tol):
    g = torch.Generator().manual_seed(1)
    x, r = torch.randn(4, 11, 200, generator=g).cuda(), torch.randn(4, 11, 200, generator=g).cuda()
    w = (1 + 0.1 * torch.randn(200, generator=g)).cuda()
    mine, ref = [_leaf(v) for v in (x, w, r)], [_leaf(v.double()) for v in (x, w, r)]
    out = torch_ops.add_rms_norm(mine[0], mine[1], mine[2] if residual else None, eps=1e-4, weight_offset=0.5,
                                 checkpoint8=checkpoint8)
    h = ref[0] + ref[2] if residual else ref[0]
    want = _norm(h, ref[1], 1e-4, 0.5)
    c, d = torch.randn(x.shape, generator=g).cuda(), torch.randn(x.shape, generator=g).cuda()
    if residual:
        _near(out, (want, h), 1e-6)
        ((out[0] * c).sum() + (out[1] * d).sum()).backward()
        ((want * c.double()).sum() + (h * d.double()).sum()).backward()
    else:
        _near([out], [want], 1e-6)
        (out * c).sum().backward()
        (want * c.double()).sum().backward()
    n = 3 if residual else 2
    _near([v.grad for v in mine[:n]], [v.grad for v in ref[:n]], tol)


def test_add_rms_norm_with_one_output_used():
    x, r = torch.randn(5, 64, device="cuda"), torch.randn(5, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for i in (0, 1):
        a, b = [_leaf(v) for v in (x, r)], [_leaf(v.double()) for v in (x, r)]
        torch_ops.add_rms_norm(a[0], w, a[1])[i].square().sum().backward()
        h = b[0] + b[1]
        (h if i else _norm(h, w.double(), 1e-6)).square().sum().backward()
        # the norm of y is constant up to eps: its gradient is of the order of eps, h's is not
        for p, q in zip(a, b):
            assert (p.grad.double() - q.grad).abs().max() <= 1e-5 * (1 + q.grad.abs().max())


def test_add_rms_norm_keeps_a_broadcast_gradient_right():
    """An upstream gradient that is an expanded scalar (stride 0)."""
    x, w = _leaf(torch.randn(7, 40, device="cuda")), torch.randn(40, device="cuda")
    y = torch_ops.add_rms_norm(x, w, eps=1e-2)
    y.sum().backward()
    r = _leaf(x.double())
    _norm(r, w.double(), 1e-2).sum().backward()
    assert rel_fro(np64(x.grad), np64(r.grad)) <= 1e-5


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_linear_ckpt8(dt):
    g = torch.Generator().manual_seed(2)
    x, W = torch.randn(3, 70, 144, generator=g).to(dt).cuda(), (0.1 * torch.randn(88, 144, generator=g)).to(dt).cuda()
    mine, ref = [_leaf(v) for v in (x, W)], [_leaf(v.double()) for v in (x, W)]
    y, want = torch_ops.linear_ckpt8(*mine), ref[0] @ ref[1].t()
    c = torch.randn(y.shape, generator=g).to(dt).cuda()
    (y * c).sum().backward()
    (want * c.double()).sum().backward()
    plain = 1e-5 if dt == torch.float32 else 1e-2
    _near([y, mine[0].grad], [want, ref[0].grad], plain)
    _near([mine[1].grad], [ref[1].grad], 0.036 + plain)


@pytest.mark.parametrize("scale", [1.0, 1e-6, 2e4])
def test_linear_ckpt8_fp16(scale):
    """fp16 activations from its subnormals to its largest. y and dx are a library's fp16 products
    (1e-2, where the result is in fp16's range); dW's only other rounding is its own to fp16."""
    g = torch.Generator().manual_seed(5)
    x = (scale * torch.randn(210, 144, generator=g).clamp(-3.2, 3.2)).half().cuda()
    W = (0.1 * torch.randn(88, 144, generator=g)).half().cuda()
    mine, ref = [_leaf(v) for v in (x, W)], [_leaf(v.double()) for v in (x, W)]
    y, want = torch_ops.linear_ckpt8(*mine), ref[0] @ ref[1].t()
    c = torch.randn(y.shape, generator=g).half().cuda() * (1.0 if scale == 1.0 else 0.01 if scale > 1 else 1000.0)
    y.backward(c)
    want.backward(c.double())
    if scale >= 1:
        fits = want.abs() < 65000
        assert fits.float().mean() > 0.95
        _near([torch.where(fits, y, 0), mine[0].grad], [torch.where(fits, want, 0), ref[0].grad], 1e-2)
    _near([mine[1].grad], [ref[1].grad], 0.036 + 1e-2)


@pytest.mark.parametrize("name", ["embedding", "linear_ckpt8", "add_rms_norm"])
def test_each_form_compiled_equals_eager(name):
    g = torch.Generator().manual_seed(6)
    t = torch.randint(0, 30, (64,), generator=g).cuda()
    x, W, w = torch.randn(64, 128, generator=g), torch.randn(30, 128, generator=g), torch.randn(128, generator=g)

    def f(x, W, w):
        if name == "embedding":
            return (torch_ops.embedding(t, W, scale=2.0) * x * w).sum()
        if name == "linear_ckpt8":
            return (torch_ops.linear_ckpt8(x * w, W) * 0.5).sum()
        return (torch_ops.add_rms_norm(x + W.sum(0), w) * 2).sum()     # no residual, no checkpoint

    out = []
    for fn in (f, torch.compile(f, backend="aot_eager", fullgraph=True)):
        a = [_leaf(v.cuda()) for v in (x, W, w)]
        loss = fn(*a)
        loss.backward()
        out.append([loss] + [v.grad for v in a])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_compiled_equals_eager():
    x, r = torch.randn(64, 128, device="cuda"), torch.randn(64, 128, device="cuda")
    w = torch.randn(128, device="cuda")

    def f(x, r, w):
        y, h = torch_ops.add_rms_norm(x, w, r, checkpoint8=True)
        return (y * 2).sum() + h.sum()

    out = []
    for fn in (f, torch.compile(f, backend="aot_eager", fullgraph=True)):
        a = [_leaf(v) for v in (x, r, w)]
        loss = fn(*a)
        loss.backward()
        out.append([loss] + [v.grad for v in a])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def _example():
    spec = importlib.util.spec_from_file_location("tied_step", os.path.join(ROOT, "examples", "tied_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_step_against_a_plain_model():
    ex = _example()
    V, H, F, N = 700, 256, 384, 900
    p = ex.init(V, H, F, seed=3)
    g = torch.Generator().manual_seed(4)
    tokens = torch.randint(0, V, (N,), generator=g).cuda()
    targets = torch.randint(0, V, (N,), generator=g).cuda()
    tokens[:5] = -100
    targets[100:160] = -100
    loss, grads, kept = ex.step(p, tokens, targets)
    r = {k: _leaf(v.double()) for k, v in p.items()}
    h0 = torch.where((tokens >= 0)[:, None], r["E"][tokens.clamp(min=0)] * H ** 0.5, 0.0)
    z = torch.relu(_norm(h0, r["n1"], ex.EPS) @ r["W1"].t()) @ r["W2"].t()
    x = _norm(z + h0, r["n2"], ex.EPS)
    want = torch.nn.functional.cross_entropy(x @ r["E"].t(), targets, ignore_index=-100)
    want.backward()
    assert abs(float(loss[0]) - want.item()) <= 5e-3 * want.item()
    for k in p:
        assert grads[k].dtype == torch.float32
        assert rel_fro(np64(grads[k]), np64(r[k].grad)) <= 0.05, k
    assert kept < 0.55 * N * (3 * H + F) * 2

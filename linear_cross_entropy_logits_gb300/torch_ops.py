"""PyTorch integration: a torch.library custom op over the C ABI and an autograd Function.

The op runs the fused forward+backward in one call, so the gradients are produced in the
forward (as the pages' op does: "Liger-Kernel PR #1554: skip ignore_index rows", Summary:
the forward runs the logits, grad_input and grad_weight GEMMs) and the backward only
applies the upstream gradient:

  * mean / sum: the gradients are linear in the scalar upstream gradient g, so the forward
    computes them for g = 1 and the backward scales them by g;
  * none with a frozen head (W, bias without grad): dX row i is linear in g_i, so the
    backward scales the rows;
  * none with a trained head: dW mixes rows with their own g_i, so the backward calls the
    fused op again with the per-token upstream gradient.

The custom op has a fake (meta) implementation, so torch.compile traces it as one opaque op
(no graph break) and compiled results equal eager ones. Marshalling only: every step of the
computation runs in libflce.so.

Around the head, each with its gradient: embedding (lookup with scaling), add_rms_norm (the
residual's addition and the RMS norm, optionally keeping an 8-bit checkpoint of its input for
the backward) and linear_ckpt8 (a projection that keeps its input in 8 bits for the weight
gradient; the two products with W itself are plain library GEMMs).
"""

from __future__ import annotations

from typing import Optional

import torch

from . import flce

_REDUCTIONS = ("mean", "sum", "none")


@torch.library.custom_op("flce_gb300::fused_linear_cross_entropy", mutates_args=())
def fused_linear_cross_entropy_op(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                                  bias: Optional[torch.Tensor], grad_out: Optional[torch.Tensor],
                                  ignore_index: int, reduction: str, z_loss_scale: float,
                                  want_dX: bool, want_dW: bool, dW_fp32: bool
                                  ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor,
                                             torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(loss, z_loss, acc, lse, pred, dX, dW, dbias); dX/dW/dbias are empty when not wanted."""
    V, H = W.shape
    dW_dtype = torch.float32 if dW_fp32 else W.dtype
    # fresh gradient buffers, written (not accumulated) by the op: no zero fill
    dW = torch.empty(V, H, dtype=dW_dtype, device=X.device) if want_dW else None
    db = torch.empty(V, dtype=dW_dtype, device=X.device) if (want_dW and bias is not None) else None
    out = flce.fwd_bwd(X.contiguous(), W.contiguous(), targets.contiguous(),
                       None if bias is None else bias.contiguous(), ignore_index=ignore_index,
                       reduction=reduction, z_loss_scale=z_loss_scale, grad_out=grad_out,
                       want_dX=want_dX, want_dW=want_dW, dW=dW, dbias=db, check=False,
                       flags=flce.FLAG_DW_OVERWRITE)
    empty = lambda dtype: torch.empty(0, dtype=dtype, device=X.device)  # noqa: E731  (outputs share no memory)
    return (out["loss"], out["z_loss"], out["acc"], out["lse"], out["pred"],
            out["dX"] if want_dX else empty(X.dtype), dW if want_dW else empty(torch.float32),
            db if db is not None else empty(torch.float32))


@fused_linear_cross_entropy_op.register_fake
def _(X, W, targets, bias, grad_out, ignore_index, reduction, z_loss_scale, want_dX, want_dW,
      dW_fp32):
    BT, H = X.shape
    V = W.shape[0]
    nl = BT if reduction == "none" else 1
    f32 = dict(dtype=torch.float32, device=X.device)
    dW_dtype = torch.float32 if dW_fp32 else W.dtype
    return (X.new_empty(nl, **{"dtype": torch.float32}), X.new_empty(nl, **{"dtype": torch.float32}),
            X.new_empty(nl, **{"dtype": torch.float32}), torch.empty(BT, **f32),
            torch.empty(BT, dtype=torch.int64, device=X.device),
            X.new_empty(BT, H) if want_dX else X.new_empty(0),
            torch.empty(V, H, dtype=dW_dtype, device=X.device) if want_dW else torch.empty(0, **f32),
            torch.empty(V, dtype=dW_dtype, device=X.device) if (want_dW and bias is not None)
            else torch.empty(0, **f32))


class FusedLinearCrossEntropy(torch.autograd.Function):
    """loss = CE(X W^T + b, targets) (+ z-loss) with ignore_index rows skipped; see module
    docstring for how the backward uses the gradients computed in the forward."""

    @staticmethod
    def forward(ctx, X, W, targets, bias, ignore_index, reduction, z_loss_scale, dW_fp32):
        if reduction not in _REDUCTIONS:
            raise ValueError(f"reduction must be one of {_REDUCTIONS}")
        need_x = ctx.needs_input_grad[0]
        need_w = ctx.needs_input_grad[1] or (bias is not None and ctx.needs_input_grad[3])
        loss, z, acc, lse, pred, dX, dW, db = fused_linear_cross_entropy_op(
            X, W, targets, bias, None, ignore_index, reduction, z_loss_scale,
            need_x, need_w, dW_fp32)
        ctx.reduction = reduction
        ctx.args = (ignore_index, z_loss_scale, dW_fp32)
        ctx.need = (need_x, need_w)
        if reduction == "none" and need_w:
            ctx.save_for_backward(X, W, targets, bias)   # recomputed with g_i in backward
        else:
            ctx.save_for_backward(dX, dW, db)
        ctx.has_bias = bias is not None
        ctx.mark_non_differentiable(z, acc, lse, pred)
        return loss, z, acc, lse, pred

    @staticmethod
    def backward(ctx, g_loss, *unused):
        need_x, need_w = ctx.need
        if ctx.reduction == "none" and need_w:
            X, W, targets, bias = ctx.saved_tensors
            ignore_index, z, dW_fp32 = ctx.args
            _, _, _, _, _, dX, dW, db = fused_linear_cross_entropy_op(
                X, W, targets, bias, g_loss.float().contiguous(), ignore_index, "none", z,
                need_x, True, dW_fp32)
        else:
            dX, dW, db = ctx.saved_tensors
            if ctx.reduction == "none":
                dX = dX * g_loss.to(dX.dtype)[:, None] if need_x else dX
            elif torch.compiler.is_compiling():
                # traced backward (torch.compile): plain tensor ops
                g = g_loss.reshape(())
                dX = dX * g.to(dX.dtype) if need_x else dX
                dW = dW * g.to(dW.dtype) if need_w else dW
                db = db * g.to(db.dtype) if (need_w and ctx.has_bias) else db
            else:
                g = g_loss.reshape(1).float().contiguous()
                prev = getattr(ctx, "applied_scale", None)
                if prev is None:
                    # eager, first backward: scale the op's own gradient buffers in place on
                    # the device and hand them out; nothing is done (no pass over dW) when
                    # the upstream gradient is exactly 1
                    ctx.applied_scale = g.clone()
                    if need_x:
                        flce.scale_by(dX, g)
                    if need_w:
                        flce.scale_by(dW, g)
                        if ctx.has_bias:
                            flce.scale_by(db, g)
                else:
                    # a later backward through a retained graph: the buffers were handed
                    # out scaled by the first upstream gradient, and whoever holds them
                    # (torch.autograd.grad's result, a hook) must keep what they got, so
                    # the new gradients are fresh tensors scaled by the ratio (if the handed
                    # out buffers were modified in place since, autograd's own check on the
                    # saved tensors raises before this backward runs)
                    if float(prev) == 0.0:
                        raise RuntimeError(
                            "fused_linear_cross_entropy: a second backward through a retained "
                            "graph cannot follow a first backward whose upstream gradient was 0")
                    r = (g / prev).contiguous()
                    dX = dX.clone() if need_x else dX
                    dW = dW.clone() if need_w else dW
                    db = db.clone() if (need_w and ctx.has_bias) else db
                    if need_x:
                        flce.scale_by(dX, r)
                    if need_w:
                        flce.scale_by(dW, r)
                        if ctx.has_bias:
                            flce.scale_by(db, r)
        return (dX if need_x else None, dW if need_w else None, None,
                db if (need_w and ctx.has_bias) else None, None, None, None, None)


def fused_linear_cross_entropy(X, W, targets, bias=None, *, ignore_index=-100, reduction="mean",
                               z_loss_scale=0.0, accum_dtype=None, return_extras=False):
    """Differentiable fused linear cross entropy. X [BT,H], W [V,H] (bf16/fp16/fp32, same
    dtype), targets int64 [BT]. ``accum_dtype=torch.float32`` accumulates dW/dbias in fp32
    (the pages' accum_dtype path); by default they come out in W's dtype. Returns the loss,
    or (loss, z_loss, accuracy, lse, pred) when ``return_extras``."""
    dW_fp32 = accum_dtype == torch.float32 or W.dtype == torch.float32
    outs = FusedLinearCrossEntropy.apply(X, W, targets, bias, ignore_index, reduction,
                                         float(z_loss_scale), dW_fp32)
    loss = outs[0] if reduction == "none" else outs[0].reshape(())
    if return_extras:
        return (loss,) + tuple(outs[1:])
    return loss


# ---------------------------------------------------------------------------------------
# Around the head: embedding, residual RMS norm, a projection with an 8-bit checkpoint
# ---------------------------------------------------------------------------------------

@torch.library.custom_op("flce_gb300::embedding", mutates_args=())
def embedding_op(tokens: torch.Tensor, E: torch.Tensor, scale: float, ignore_index: int,
                 check: bool = False) -> torch.Tensor:
    o = flce.embed_fwd(tokens.contiguous(), E, scale=scale, ignore_index=ignore_index, check=check)
    if check and o["status_code"] != flce.FLCE_OK:
        raise flce.FlceError(o["status_code"], "embedding")
    return o["out"]


@embedding_op.register_fake
def _(tokens, E, scale, ignore_index, check=False):
    return E.new_empty(tokens.shape[0], E.shape[1])


@torch.library.custom_op("flce_gb300::embedding_bwd", mutates_args=())
def embedding_bwd_op(tokens: torch.Tensor, dout: torch.Tensor, V: int, scale: float, ignore_index: int) -> torch.Tensor:
    dE = torch.empty(V, dout.shape[1], dtype=dout.dtype, device=dout.device)
    flce.embed_bwd(tokens.contiguous(), dout.contiguous(), dE=dE, scale=scale, ignore_index=ignore_index,
                   flags=flce.FLAG_DW_OVERWRITE, check=False)
    return dE


@embedding_bwd_op.register_fake
def _(tokens, dout, V, scale, ignore_index):
    return dout.new_empty(V, dout.shape[1])


def _embedding_setup(ctx, inputs, output):
    tokens, E, scale, ignore_index, check = inputs
    ctx.save_for_backward(tokens)
    ctx.args = (E.shape[0], scale, ignore_index)


def _embedding_backward(ctx, g):
    tokens, = ctx.saved_tensors
    V, scale, ignore_index = ctx.args
    return None, embedding_bwd_op(tokens, g, V, scale, ignore_index), None, None, None


embedding_op.register_autograd(_embedding_backward, setup_context=_embedding_setup)


def embedding(tokens, E, *, scale=1.0, ignore_index=-100, check=False):
    """scale * E[tokens], a zero row where tokens == ignore_index; differentiable in E (a dense
    gradient in E's dtype, each row summed in fp32 in a fixed order). tokens: int64 of any
    shape; E [V, H]. A token outside [0, V) gives a zero row and no gradient; ``check`` raises
    FlceError for it instead, which waits for the stream."""
    return embedding_op(tokens.reshape(-1), E, float(scale), ignore_index, check).reshape(*tokens.shape, E.shape[1])


def _rows(x):
    """x as [rows, width] with unit column stride, without a copy where it has one."""
    return x if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= x.shape[1] else x.reshape(-1, x.shape[-1]).contiguous()


@torch.library.custom_op("flce_gb300::add_rms_norm", mutates_args=())
def add_rms_norm_op(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor], eps: float,
                    weight_offset: float, checkpoint8: bool
                    ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, h, rstd, h8, h8_scale); h is empty without a residual, h8 and h8_scale without checkpoint8."""
    o = flce.rmsnorm_fwd(_rows(x), weight, None if residual is None else _rows(residual), eps=eps,
                         weight_offset=weight_offset, want_h8=checkpoint8)
    empty = lambda dtype: torch.empty(0, dtype=dtype, device=x.device)  # noqa: E731  (outputs share no memory)
    return (o["y"], o["h"] if residual is not None else empty(x.dtype), o["rstd"],
            o["h8"] if checkpoint8 else empty(torch.float8_e4m3fn), o["h8_scale"] if checkpoint8 else empty(torch.float32))


@add_rms_norm_op.register_fake
def _(x, weight, residual, eps, weight_offset, checkpoint8):
    N, H = x.shape
    f32 = dict(dtype=torch.float32, device=x.device)
    f8 = dict(dtype=torch.float8_e4m3fn, device=x.device)
    return (x.new_empty(N, H), x.new_empty(N, H) if residual is not None else x.new_empty(0), torch.empty(N, **f32),
            torch.empty_strided((N, H), ((H + 15) // 16 * 16, 1), **f8) if checkpoint8 else torch.empty(0, **f8),
            torch.empty(N, (H + 127) // 128, **f32) if checkpoint8 else torch.empty(0, **f32))


@torch.library.custom_op("flce_gb300::add_rms_norm_bwd", mutates_args=())
def add_rms_norm_bwd_op(dy: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, h: Optional[torch.Tensor],
                        h8: Optional[torch.Tensor], h8_scale: Optional[torch.Tensor], dh: Optional[torch.Tensor],
                        weight_offset: float) -> tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight)"""
    dw = torch.empty_like(weight)
    o = flce.rmsnorm_bwd(_rows(dy), weight, rstd, None if h is None else _rows(h), h8=h8, h8_scale=h8_scale,
                         dh=None if dh is None else _rows(dh), weight_offset=weight_offset, dweight=dw,
                         flags=flce.FLAG_DW_OVERWRITE)
    return o["dx"], dw


@add_rms_norm_bwd_op.register_fake
def _(dy, weight, rstd, h, h8, h8_scale, dh, weight_offset):
    return dy.new_empty(dy.shape), torch.empty_like(weight)


def _add_rms_norm_setup(ctx, inputs, output):
    x, weight, residual, eps, weight_offset, checkpoint8 = inputs
    y, h, rstd, h8, h8_scale = output
    ctx.mark_non_differentiable(rstd, h8, h8_scale)
    ctx.set_materialize_grads(False)
    if checkpoint8:
        ctx.save_for_backward(weight, rstd, h8, h8_scale)
    else:
        ctx.save_for_backward(weight, rstd, x if residual is None else h)
    ctx.args = (residual is not None, weight_offset, checkpoint8, x.shape, x.dtype)


def _add_rms_norm_backward(ctx, dy, dh, *unused):
    has_residual, weight_offset, checkpoint8, shape, dtype = ctx.args
    if dy is None and dh is None:
        return (None,) * 6
    weight, rstd = ctx.saved_tensors[:2]
    if dy is None:
        dy = torch.zeros(shape, dtype=dtype, device=weight.device)
    if not has_residual:
        dh = None
    kept = ctx.saved_tensors[2:]
    h, h8, h8_scale = (None, *kept) if checkpoint8 else (kept[0], None, None)
    dx, dw = add_rms_norm_bwd_op(dy, weight, rstd, h, h8, h8_scale, dh, weight_offset)
    return dx, dw, dx if has_residual else None, None, None, None


add_rms_norm_op.register_autograd(_add_rms_norm_backward, setup_context=_add_rms_norm_setup)


def add_rms_norm(x, weight, residual=None, *, eps=1e-6, weight_offset=0.0, checkpoint8=False):
    """y = h / rms(h) * (weight + weight_offset) with h = x + residual; returns (y, h) with a
    residual, y without. Differentiable in x, residual and weight. With ``checkpoint8`` the
    backward uses an 8-bit checkpoint of h (e4m3, a scale per 128 columns) instead of keeping
    h itself. x and residual [..., H], weight [H], one dtype."""
    shape = x.shape
    y, h, _, _, _ = add_rms_norm_op(x.reshape(-1, shape[-1]), weight,
                                    None if residual is None else residual.reshape(-1, shape[-1]), float(eps),
                                    float(weight_offset), bool(checkpoint8))
    return y.reshape(shape) if residual is None else (y.reshape(shape), h.reshape(shape))


@torch.library.custom_op("flce_gb300::ckpt8_pack", mutates_args=())
def ckpt8_pack_op(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    o = flce.ckpt8_pack(_rows(x))
    return o["q"], o["scale"]


@ckpt8_pack_op.register_fake
def _(x):
    N, H = x.shape
    return (torch.empty_strided((N, H), ((H + 15) // 16 * 16, 1), dtype=torch.float8_e4m3fn, device=x.device),
            torch.empty(N, (H + 127) // 128, dtype=torch.float32, device=x.device))


@torch.library.custom_op("flce_gb300::ckpt8_dw", mutates_args=())
def ckpt8_dw_op(dy: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, dW_fp32: bool) -> torch.Tensor:
    dW = torch.empty(dy.shape[1], q.shape[1], dtype=torch.float32 if dW_fp32 else dy.dtype, device=dy.device)
    flce.ckpt8_dw(_rows(dy), q, scale, dW=dW, flags=flce.FLAG_DW_OVERWRITE, check=False)
    return dW


@ckpt8_dw_op.register_fake
def _(dy, q, scale, dW_fp32):
    return torch.empty(dy.shape[1], q.shape[1], dtype=torch.float32 if dW_fp32 else dy.dtype, device=dy.device)


class LinearCkpt8(torch.autograd.Function):
    """y = x W^T that keeps x in 8 bits for the weight gradient."""

    @staticmethod
    def forward(ctx, x, W):
        ctx.save_for_backward(W, *ckpt8_pack_op(x))
        return torch.mm(x, W.t())

    @staticmethod
    def backward(ctx, dy):
        W, q, scale = ctx.saved_tensors
        # (under autocast y and dy have its type; autograd takes dx and dW to x's and W's)
        dx = torch.mm(dy, W.to(dy.dtype)) if ctx.needs_input_grad[0] else None
        return dx, ckpt8_dw_op(dy, q, scale, W.dtype == torch.float32)


def linear_ckpt8(x, W):
    """x W^T for x [..., K] and W [N, K] of one dtype; the backward's dW = dy^T x reads an 8-bit
    checkpoint of x (its rounding, half of 2^-3 of a value, is the only approximation; dx is
    exact). x itself is not kept. Without a gradient of W to come (frozen, or in evaluation) it is
    a plain product."""
    rows = x.reshape(-1, x.shape[-1])
    y = LinearCkpt8.apply(rows, W) if torch.is_grad_enabled() and W.requires_grad else torch.mm(rows, W.t())
    return y.reshape(*x.shape[:-1], W.shape[0])

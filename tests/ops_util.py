"""Shared by the tests of the embedding, RMS norm and 8-bit checkpoint operators."""

import numpy as np
import torch

from linear_cross_entropy_logits_gb300 import inputs as I

DT = I.TORCH_DTYPES
# half the spacing of a type's values, relative; and an absolute floor for fp16's subnormals
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
FLOOR = {"f32": 2.0 ** -140, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}
F32 = 2.0 ** -24


def np64(t):
    return t.detach().double().cpu().numpy()


def odd_rows(N, H, dtype, extra, offset):
    """An uninitialised [N, H] view with row pitch H + extra that starts `offset` elements in."""
    buf = torch.empty(N * (H + extra) + offset + 1, dtype=dtype, device="cuda")
    return buf[offset:offset + N * (H + extra)].view(N, H + extra)[:, :H]


def strided(t, extra, offset):
    """A copy of t in such a view (extra = offset = 0: a dense copy)."""
    v = odd_rows(*t.shape, t.dtype, extra, offset)
    v.copy_(t)
    return v


def close(got, want, bound, what=""):
    got = np64(got) if torch.is_tensor(got) else got
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(err - bound)} over its bound"

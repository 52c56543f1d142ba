"""Measured cases of the operators around the fused head: the tied embedding and its gradient,
the residual-adding RMS norm and its gradient, and 8-bit activation checkpoints with the
weight gradient that reads them.

``run`` computes a case either in plain torch operations in 32 bits (``own`` false) or through
the package's entry points (``own`` true). ``exact`` gives the same outputs from the
definitions in 64 bits.

8-bit tensors are e4m3 with one fp32 scale per row and 128 columns. A checkpoint's scale is the
smallest power of two that brings the block's largest magnitude to at most 448; the norm's
8-bit output has that power of two for h * weight, times the row's 1/rms.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 128
IGNORE = -100
EPS = 1e-5


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------

def listed():
    return [
        # the token lookup of a short prompt, 1B-shaped model: launch latency
        {"name": "embed_fwd prompt", "op": "embed_fwd", "dtype": "bf16", "N": 48, "H": 2048, "V": 128256,
         "scaled": False, "ignored": 0.0},
        # the lookup of a training step of the large-vocabulary workload, scaled by sqrt(H)
        {"name": "embed_fwd step", "op": "embed_fwd", "dtype": "bf16", "N": 16384, "H": 5376, "V": 262144,
         "scaled": True, "ignored": 0.1},
        # the tied head's shared fp32 gradient buffer takes the lookup's part: 8B-shaped step
        {"name": "embed_bwd tied", "op": "embed_bwd", "dtype": "bf16", "N": 8192, "H": 4096, "V": 128256,
         "scaled": False, "ignored": 0.1, "dE": "f32", "accumulate": True},
        # a fresh same-dtype gradient of an untied table, odd row count and width
        {"name": "embed_bwd fresh", "op": "embed_bwd", "dtype": "f16", "N": 2999, "H": 1003, "V": 32000,
         "scaled": True, "ignored": 0.0, "dE": "f16", "accumulate": False},
        # the norm in a few rows' decoding step, 16-bit output alone: latency
        {"name": "norm_fwd few rows", "op": "norm_fwd", "dtype": "bf16", "N": 16, "H": 4096,
         "residual": True, "y8": False, "h8": False},
        # a layer's norm in an 8B-shaped training step: 16-bit and 8-bit output and its own
        # 8-bit checkpoint beside the residual stream
        {"name": "norm_fwd step", "op": "norm_fwd", "dtype": "bf16", "N": 8192, "H": 4096,
         "residual": True, "y8": True, "h8": True},
        # its gradient from the 8-bit checkpoint
        {"name": "norm_bwd 8-bit", "op": "norm_bwd", "dtype": "bf16", "N": 8192, "H": 4096,
         "h8": True, "dh": True, "dw": "f32"},
        # the gradient from a kept fp32 input, odd width, no residual gradient
        {"name": "norm_bwd odd", "op": "norm_bwd", "dtype": "f32", "N": 1500, "H": 1337,
         "h8": False, "dh": False, "dw": "f32"},
        # a layer input kept in 8 bits: 16384 rows of a 4096-wide model
        {"name": "pack step", "op": "pack", "dtype": "bf16", "N": 16384, "H": 4096},
        # the same for a short ragged fp16 batch
        {"name": "pack ragged", "op": "pack", "dtype": "f16", "N": 777, "H": 1336},
        # a 4096 x 4096 projection's weight gradient from the 8-bit checkpoint of its input
        {"name": "dw step", "op": "dw", "dtype": "bf16", "M": 8192, "N": 4096, "K": 4096,
         "dW": "f32", "accumulate": True},
        # a ragged batch of a small projection, same-dtype gradient
        {"name": "dw ragged", "op": "dw", "dtype": "f16", "M": 1531, "N": 520, "K": 2008,
         "dW": "f16", "accumulate": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width spread over [lo, hi]: two in three are multiples of 8, the others any number."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.67:
        n = max(8, n // 8 * 8)
    return n + 8 if n == 3072 else n


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "pack", "dw"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "dw":
        M, N, K = _log(rng, 1, 16384), _width(rng, 64, 8192), _width(rng, 64, 8192)
        top = 8192 * 4096 * 4096
        if M * N * K > top:
            M = max(1, top // (N * K))
        return {"op": op, "dtype": dtype, "M": M, "N": N, "K": K, "dW": rng.choice(["f32", dtype]),
                "accumulate": flip()}
    N, H = _log(rng, 1, 32768), _width(rng, 64, 8192)
    N = max(1, min(N, 8192 * 4096 // H))
    if op in ("embed_fwd", "embed_bwd"):
        V = _log(rng, 1000, 262144)
        V = max(1000, min(V, 128256 * 4096 // H))
        c = {"op": op, "dtype": dtype, "N": N, "H": H, "V": V, "scaled": flip(), "ignored": rng.choice([0.0, 0.1, 0.5])}
        if op == "embed_bwd":
            c.update(dE=rng.choice(["f32", dtype]), accumulate=flip())
        return c
    c = {"op": op, "dtype": dtype, "N": N, "H": H}
    if op == "norm_fwd":
        c.update(residual=flip(), y8=flip(), h8=flip())
    elif op == "norm_bwd":
        c.update(h8=flip(), dh=flip(), dw=rng.choice(["f32", dtype]))
    return c


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------

def _tokens(g, N, V, ignored):
    """Token ids whose frequency falls as 1 / (id + 1), as in running text."""
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    t = torch.exp(u * math.log(V + 1.0)).long() - 1
    t = t.clamp_(0, V - 1)
    if ignored:
        t[torch.rand(N, generator=g, device="cuda") < ignored] = IGNORE
    return t


def _activations(g, N, H, dtype):
    """Rows of differing size with a few wide columns, as a residual stream has."""
    x = torch.randn(N, H, generator=g, device="cuda")
    x *= 0.5 + torch.rand(N, 1, generator=g, device="cuda")
    x[:, :: 61] *= 8.0
    return x.to(dtype)


def _blocks(x):
    """[N, H] as [N, blocks, BLOCK] with zeros past H."""
    N, H = x.shape
    nb = (H + BLOCK - 1) // BLOCK
    p = torch.nn.functional.pad(x, (0, nb * BLOCK - H))
    return p.reshape(N, nb, BLOCK)


def _pow2_scale(amax):
    """The smallest power of two s (at least 2^-117) with amax <= 448 s; 1 for an empty block."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875).int()).clamp(min=-117))
    return torch.where(amax > 0, s, torch.ones_like(s))


def _pitched(N, H, dtype):
    """[N, H] with a row pitch of 16 bytes, as the package keeps 8-bit rows."""
    p = (H + 15) // 16 * 16
    return torch.empty(N, p, dtype=dtype, device="cuda")[:, :H]


def _quantise(x):
    """(q, scale) of fp32 [N, H] in plain torch."""
    N, H = x.shape
    b = _blocks(x)
    s = _pow2_scale(b.abs().amax(dim=2))
    q = _pitched(N, H, torch.float8_e4m3fn)
    q.copy_((b / s[:, :, None]).reshape(N, -1)[:, :H].to(torch.float8_e4m3fn))
    return q, s


def _dequantise(q, s):
    N, H = q.shape
    return (_blocks(q.float()) * s[:, :, None]).reshape(N, -1)[:, :H]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c, "dtype": DTYPES[c["dtype"]]}
    dt = st["dtype"]
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if c["op"] in ("embed_fwd", "embed_bwd"):
        N, H, V = c["N"], c["H"], c["V"]
        st["scale"] = math.sqrt(H) if c["scaled"] else 1.0
        st["tokens"] = _tokens(g, N, V, c["ignored"])
        if c["op"] == "embed_fwd":
            st["E"] = torch.empty(V, H, dtype=dt, device="cuda").normal_(0, 0.02, generator=g)
            st["out"] = torch.empty(N, H, dtype=dt, device="cuda")
        else:
            st["dout"] = (randn(N, H) * 0.01).to(dt)
            st["dE"] = torch.empty(V, H, dtype=DTYPES[c["dE"]], device="cuda").normal_(0, 0.01, generator=g)
    elif c["op"] == "norm_fwd":
        N, H = c["N"], c["H"]
        st["x"] = _activations(g, N, H, dt)
        st["residual"] = _activations(g, N, H, dt) if c["residual"] else None
        st["weight"] = (1.0 + 0.2 * randn(H)).to(dt)
    elif c["op"] == "norm_bwd":
        N, H = c["N"], c["H"]
        h = _activations(g, N, H, dt).float()
        st["rstd"] = torch.rsqrt(h.square().mean(dim=1) + EPS)
        if c["h8"]:
            st["h8"], st["h8_scale"] = _quantise(h)
        else:
            st["h"] = h.to(dt)
        st["dy"] = (randn(N, H) * 0.01).to(dt)
        st["dh"] = (randn(N, H) * 0.01).to(dt) if c["dh"] else None
        st["weight"] = (1.0 + 0.2 * randn(H)).to(dt)
        st["dweight"] = torch.zeros(H, dtype=DTYPES[c["dw"]], device="cuda")
    elif c["op"] == "pack":
        st["x"] = _activations(g, c["N"], c["H"], dt)
    else:
        M, N, K = c["M"], c["N"], c["K"]
        st["q"], st["scale"] = _quantise(_activations(g, M, K, dt).float())
        st["dy"] = (randn(M, N) * 0.01).to(dt)
        st["dW"] = (randn(N, K) * 0.01).to(DTYPES[c["dW"]])
    return st


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from linear_cross_entropy_logits_gb300 import flce
    c = s["case"]
    op = c["op"]
    if op == "embed_fwd":
        return flce.embed_fwd(s["tokens"], s["E"], scale=s["scale"], ignore_index=IGNORE, out=s["out"],
                              check=False)["out"]
    if op == "embed_bwd":
        return flce.embed_bwd(s["tokens"], s["dout"], dE=s["dE"], scale=s["scale"], ignore_index=IGNORE,
                              flags=0 if c["accumulate"] else flce.FLAG_DW_OVERWRITE, check=False)["dE"]
    if op == "norm_fwd":
        o = flce.rmsnorm_fwd(s["x"], s["weight"], s["residual"], eps=EPS, want_y8=c["y8"], want_h8=c["h8"])
        names = ["y", "rstd"] + (["h"] if c["residual"] else [])
        names += (["y8", "y8_scale"] if c["y8"] else []) + (["h8", "h8_scale"] if c["h8"] else [])
        return {k: o[k] for k in names}
    if op == "norm_bwd":
        o = flce.rmsnorm_bwd(s["dy"], s["weight"], s["rstd"], s.get("h"), h8=s.get("h8"),
                             h8_scale=s.get("h8_scale"), dh=s["dh"], dweight=s["dweight"],
                             flags=flce.FLAG_DW_OVERWRITE)
        return {"dx": o["dx"], "dweight": o["dweight"]}
    if op == "pack":
        o = flce.ckpt8_pack(s["x"])
        return {"q": o["q"], "scale": o["scale"]}
    return flce.ckpt8_dw(s["dy"], s["q"], s["scale"], dW=s["dW"],
                         flags=0 if c["accumulate"] else flce.FLAG_DW_OVERWRITE, check=False)["dW"]


def _run_plain(s):
    c, dt = s["case"], s["dtype"]
    op = c["op"]
    if op == "embed_fwd":
        keep = s["tokens"] != IGNORE
        rows = s["E"][torch.where(keep, s["tokens"], 0)].float() * s["scale"]
        return torch.where(keep[:, None], rows, 0.0).to(dt)
    if op == "embed_bwd":
        keep = s["tokens"] != IGNORE
        g = torch.where(keep[:, None], s["dout"].float() * s["scale"], 0.0)
        at = torch.where(keep, s["tokens"], 0)
        dE = s["dE"]
        if c["accumulate"] and dE.dtype == torch.float32:
            return dE.index_add_(0, at, g)
        sums = dE.float() if c["accumulate"] else torch.zeros(dE.shape, dtype=torch.float32, device="cuda")
        return dE.copy_(sums.index_add_(0, at, g))
    if op == "norm_fwd":
        h = s["x"].float()
        if c["residual"]:
            h = h + s["residual"].float()
        w = s["weight"].float()
        r = torch.rsqrt(h.square().mean(dim=1) + EPS)
        o = {"y": (h * r[:, None] * w).to(dt), "rstd": r}
        if c["residual"]:
            o["h"] = h.to(dt)
        if c["y8"]:
            o["y8"], sc = _quantise(h * w)
            o["y8_scale"] = sc * r[:, None]
        if c["h8"]:
            o["h8"], o["h8_scale"] = _quantise(h)
        return o
    if op == "norm_bwd":
        h = _dequantise(s["h8"], s["h8_scale"]) if c["h8"] else s["h"].float()
        r = s["rstd"][:, None]
        xhat = h * r
        dy = s["dy"].float()
        g = dy * s["weight"].float()
        dx = r * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
        if c["dh"]:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": s["dweight"].copy_((dy * xhat).sum(dim=0))}
    if op == "pack":
        q, sc = _quantise(s["x"].float())
        return {"q": q, "scale": sc}
    d = s["dy"].float().t() @ _dequantise(s["q"], s["scale"])
    return s["dW"].copy_(s["dW"].float() + d if c["accumulate"] else d)


# --------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------

def _exact_pow2(x):
    """Per block of 128 columns of float64 [N, H]: 2^ceil(log2(amax / 448)), checked at the edges."""
    N, H = x.shape
    cols = [x[:, j:j + BLOCK].abs().amax(dim=1) for j in range(0, H, BLOCK)]
    amax = torch.stack(cols, dim=1)
    e = torch.ceil(torch.log2(amax / 448.0))
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
    return torch.where(amax > 0, torch.exp2(e.clamp(min=-117.0)), torch.ones_like(amax))


def _wide(s, H):
    """Block scales [N, blocks] spread over the H columns."""
    return s[:, torch.arange(H, device=s.device) // BLOCK]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point() and k not in ("E", "dE", "out")}
    if op == "embed_fwd":
        t = s["tokens"]
        out = torch.zeros(c["N"], c["H"], dtype=torch.float64, device="cuda")
        live = (t >= 0).nonzero().reshape(-1)
        out[live] = s["E"][t[live]].double() * s["scale"]
        return out
    if op == "embed_bwd":
        # the sum of each token's rows as differences of running sums over the rows in token order
        t = s["tokens"]
        live = (t >= 0).nonzero().reshape(-1)
        order = live[torch.argsort(t[live], stable=True)]
        ids, n = torch.unique_consecutive(t[order], return_counts=True)
        out = s["dE"].double() if c["accumulate"] else torch.zeros(c["V"], c["H"], dtype=torch.float64, device="cuda")
        if ids.numel():
            run_sum = torch.cumsum(d["dout"][order] * s["scale"], dim=0)
            end = torch.cumsum(n, dim=0)
            seg = run_sum[end - 1]
            seg[1:] -= run_sum[end[:-1] - 1]
            out[ids] += seg
        return out
    if op == "norm_fwd":
        h = d["x"] + d["residual"] if c["residual"] else d["x"]
        r = 1.0 / torch.sqrt((h * h).sum(dim=1) / c["H"] + EPS)
        o = {"y": h * d["weight"] * r[:, None], "rstd": r}
        if c["residual"]:
            o["h"] = h
        # an 8-bit value's exact value is the quotient that is rounded to it
        if c["y8"]:
            u = h * d["weight"]
            sc = _exact_pow2(u)
            o["y8"], o["y8_scale"] = u / _wide(sc, c["H"]), sc * r[:, None]
        if c["h8"]:
            sc = _exact_pow2(h)
            o["h8"], o["h8_scale"] = h / _wide(sc, c["H"]), sc
        return o
    if op == "norm_bwd":
        h = d["h8"] * _wide(d["h8_scale"], c["H"]) if c["h8"] else d["h"]
        r, H = d["rstd"], c["H"]
        dot = (d["dy"] * d["weight"] * h).sum(dim=1)
        dx = d["dy"] * d["weight"] * r[:, None] - h * (r ** 3 * dot / H)[:, None]
        if c["dh"]:
            dx += d["dh"]
        return {"dx": dx, "dweight": torch.einsum("nh,nh,n->h", d["dy"], h, r)}
    if op == "pack":
        sc = _exact_pow2(d["x"])
        return {"q": d["x"] / _wide(sc, c["H"]), "scale": sc}
    out = torch.einsum("mn,mk->nk", d["dy"], d["q"] * _wide(d["scale"], c["K"]))
    return out + d["dW"] if c["accumulate"] else out


# --------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------

def _distinct(N, V, ignored):
    """Expected number of different tokens among N drawn as _tokens draws them."""
    v = np.arange(1, V + 1, dtype=np.float64)
    p = (1.0 - ignored) * np.log1p(1.0 / v) / math.log(V + 1.0)
    return float(-np.expm1(N * np.log1p(-p)).sum())


def _sz(name):
    return 4 if name == "f32" else 2


def work(case):
    c = case
    e = _sz(c["dtype"])
    if c["op"] in ("embed_fwd", "embed_bwd"):
        N, H, V = c["N"], c["H"], c["V"]
        live, rows = N * (1.0 - c["ignored"]), _distinct(N, V, c["ignored"])
        if c["op"] == "embed_fwd":
            return {"bytes": 8 * N + rows * H * e + N * H * e, "flops": live * H}
        g = _sz(c["dE"])
        return {"bytes": 8 * N + live * H * e + (2 * rows if c["accumulate"] else V) * H * g, "flops": 2 * live * H}
    if c["op"] == "dw":
        M, N, K = c["M"], c["N"], c["K"]
        nb = (K + BLOCK - 1) // BLOCK
        return {"bytes": M * N * e + M * K + 4 * M * nb + N * K * _sz(c["dW"]) * (2 if c["accumulate"] else 1),
                "flops": 2.0 * M * N * K}
    N, H = c["N"], c["H"]
    eight = N * H + 4 * N * ((H + BLOCK - 1) // BLOCK)
    if c["op"] == "norm_fwd":
        wide = 2 + (2 if c["residual"] else 0)
        return {"bytes": wide * N * H * e + H * e + 4 * N + eight * (int(c["y8"]) + int(c["h8"])), "flops": 5.0 * N * H}
    if c["op"] == "norm_bwd":
        n = 2 + int(c["dh"])
        return {"bytes": n * N * H * e + (eight if c["h8"] else N * H * e) + 4 * N + H * (e + _sz(c["dw"])),
                "flops": 10.0 * N * H}
    return {"bytes": N * H * e + eight, "flops": 2.0 * N * H}

"""A training step of a small tied-weight language model on the fused operators.

    h0   = scale * E[tokens]                                   embed_fwd
    x, h = rms_norm(h0) ;  z = relu(x W1^T) W2^T               rmsnorm_fwd, ckpt8_pack
    x, h = rms_norm(z + h0)                                    rmsnorm_fwd with the residual
    loss = cross entropy(x E^T, targets)                       fwd_bwd (no logits kept)

and its gradients, which need neither the norms' inputs nor the projections' inputs in 16 bits:
the norms go back from 8-bit checkpoints (rmsnorm_bwd), the weight gradients are made from 8-bit
checkpoints (ckpt8_dw), and the head's and the lookup's gradients of E meet in one fp32 buffer
(fwd_bwd writes it, embed_bwd adds to it). The four products with W1 and W2 themselves are
plain library GEMMs.

    python examples/tied_step.py --steps 20
"""

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_cross_entropy_logits_gb300 import flce  # noqa: E402

EPS = 1e-5


def init(V, H, F, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return {"E": (0.02 * r(V, H)).to(dtype), "n1": torch.ones(H, dtype=dtype, device="cuda"),
            "n2": torch.ones(H, dtype=dtype, device="cuda"), "W1": (r(F, H) / math.sqrt(H)).to(dtype),
            "W2": (r(H, F) / math.sqrt(F)).to(dtype)}


def step(p, tokens, targets, ignore_index=-100):
    """(loss, fp32 gradients by name, bytes kept between forward and backward)."""
    E, scale = p["E"], math.sqrt(p["E"].shape[1])
    h0 = flce.embed_fwd(tokens, E, scale=scale, ignore_index=ignore_index, check=False)["out"]
    a = flce.rmsnorm_fwd(h0, p["n1"], eps=EPS, want_h8=True)
    x8 = flce.ckpt8_pack(a["y"])
    u = torch.relu(torch.mm(a.pop("y"), p["W1"].t()))
    u8 = flce.ckpt8_pack(u)
    z = torch.mm(u, p["W2"].t())
    del u
    b = flce.rmsnorm_fwd(z, p["n2"], h0, eps=EPS, want_h=False, want_h8=True)
    del z, h0
    kept = sum(t.numel() * t.element_size() for d in (a, b, x8, u8) for k, t in d.items() if k != "y")

    g = {"E": torch.empty(E.shape, dtype=torch.float32, device=E.device)}
    head = flce.fwd_bwd(b.pop("y"), E, targets, ignore_index=ignore_index, dW=g["E"], flags=flce.FLAG_DW_OVERWRITE,
                        check=False)
    o = flce.rmsnorm_bwd(head["dX"], p["n2"], b["rstd"], h8=b["h8"], h8_scale=b["h8_scale"])
    g["n2"], dh = o["dweight"], o["dx"]
    g["W2"] = flce.ckpt8_dw(dh, u8["q"], u8["scale"], check=False)["dW"]
    # relu passes a gradient where its output is positive, and there its 8-bit code is too (unless the
    # output is below 2^-17 of its block's largest)
    du = torch.mm(dh, p["W2"]).mul_(u8["q"].view(torch.int8) > 0)
    g["W1"] = flce.ckpt8_dw(du, x8["q"], x8["scale"], check=False)["dW"]
    o = flce.rmsnorm_bwd(torch.mm(du, p["W1"]), p["n1"], a["rstd"], h8=a["h8"], h8_scale=a["h8_scale"], dh=dh)
    g["n1"] = o["dweight"]
    flce.embed_bwd(tokens, o["dx"], dE=g["E"], scale=scale, ignore_index=ignore_index, check=False)
    return head["loss"], g, kept


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rows", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=8192)
    ap.add_argument("--vocab", type=int, default=128256)
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args()
    p = init(a.vocab, a.hidden, a.inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, a.vocab, (a.rows,), generator=g, device="cuda")
    targets = torch.roll(tokens, -1)  # the next token
    targets[-1] = -100
    for i in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        loss, grads, kept = step(p, tokens, targets)
        for k, d in grads.items():
            p[k].sub_((a.lr * d).to(p[k].dtype))
        torch.cuda.synchronize()
        print(f"step {i}: loss {float(loss[0]):.4f}  {1e3 * (time.perf_counter() - t):.2f} ms  "
              f"kept for the backward {kept / 1e6:.1f} MB (16-bit: {a.rows * (3 * a.hidden + a.inner) * 2 / 1e6:.1f} MB)")


if __name__ == "__main__":
    main()

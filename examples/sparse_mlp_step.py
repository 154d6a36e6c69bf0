"""A sparse-MLP layer under the LM-head loss, trained for a few steps.

One decoder block's second half as a user of a mixture-of-experts model has
it: router logits from a linear layer, `route_experts` to top_k of E experts,
`experts_mlp` over them, the residual sum, then `linear_cross_entropy`
against the vocabulary. Synthetic tokens from a seed; plain SGD in fp32
master weights. After each step the router's selection bias is nudged
towards experts with few tokens (balance without an auxiliary loss).

    python examples/sparse_mlp_step.py [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_lm_head_gemm_gb300 as lce  # noqa: E402


def run(steps=8, L=1024, H=256, I=128, E=16, top_k=4, V=4096, lr=0.5,
        device="cuda"):
    """Returns the losses of `steps` steps on one fixed batch."""
    g = torch.Generator(device=device).manual_seed(0)

    def normal(*shape, std):
        return torch.randn(*shape, device=device, generator=g) * std

    x = normal(L, H, std=1.0).bfloat16()
    labels = torch.randint(0, V, (L,), device=device, generator=g)
    master = dict(Wr=normal(E, H, std=H ** -0.5),
                  Wg=normal(E, I, H, std=H ** -0.5),
                  Wu=normal(E, I, H, std=H ** -0.5),
                  Wd=normal(E, H, I, std=I ** -0.5),
                  head=normal(V, H, std=0.05))
    bias = torch.zeros(E, device=device)
    losses = []
    for _ in range(steps):
        w = {k: v.bfloat16().requires_grad_(True) for k, v in master.items()}
        logits = x @ w["Wr"].t()
        weights, experts = lce.route_experts(logits, top_k, scoring="sigmoid",
                                             bias=bias)
        h = x + lce.experts_mlp(x, w["Wg"], w["Wu"], w["Wd"], weights, experts)
        loss = lce.linear_cross_entropy(h, w["head"], labels, fused=True)
        loss.backward()
        with torch.no_grad():
            for k, v in master.items():
                v -= lr * w[k].grad.float()
            load = torch.bincount(experts.flatten(), minlength=E).float()
            bias -= 1e-3 * torch.sign(load - load.mean())
        losses.append(loss.item())
    status = lce.get_error()
    if status != 0:
        raise RuntimeError(f"device error status {status}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    for i, loss in enumerate(run(ap.parse_args().steps)):
        print(f"step {i}: loss {loss:.4f}")

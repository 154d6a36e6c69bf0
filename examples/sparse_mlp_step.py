"""A sparse-MLP layer under the LM-head loss, trained for a few steps.

One decoder block's second half as a user of a mixture-of-experts model has
it: router logits from a linear layer, `route_experts` to top_k of E experts,
`experts_mlp` over them, the residual sum, then `linear_cross_entropy`
against the vocabulary. Synthetic tokens from a seed; plain SGD in fp32
master weights. After each step the router's selection bias is nudged
towards experts with few tokens (balance without an auxiliary loss; the load
from `expert_counts`).

Options: `--norm rms|layer` puts a norm in front of the router and experts
and one in front of the head (`rms_norm`, `layer_norm`), `--balance C` adds
the auxiliary `balance_loss` with coefficient C in place of the bias,
`--max-norm N` clips the gradients' global norm (`clip_grad_norm`).

    python examples/sparse_mlp_step.py [--steps 8] [--norm rms]
        [--balance 0.01] [--max-norm 1.0]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_lm_head_gemm_gb300 as lce  # noqa: E402


def run(steps=8, L=1024, H=256, I=128, E=16, top_k=4, V=4096, lr=0.5,
        device="cuda", norm=None, balance=0.0, max_norm=None):
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
    for name in ("n1", "n2") if norm else ():
        master[name] = torch.ones(H, device=device)
        if norm == "layer":
            master[name + "b"] = torch.zeros(H, device=device)
    bias = torch.zeros(E, device=device)
    losses = []

    def normed(t, w, name):
        if norm == "layer":
            return lce.layer_norm(t, w[name], w[name + "b"])
        return lce.rms_norm(t, w[name]) if norm else t

    for _ in range(steps):
        w = {k: v.bfloat16().requires_grad_(True) for k, v in master.items()}
        xn = normed(x, w, "n1")
        logits = xn @ w["Wr"].t()
        weights, experts = lce.route_experts(logits, top_k, scoring="sigmoid",
                                             bias=bias)
        h = x + lce.experts_mlp(xn, w["Wg"], w["Wu"], w["Wd"], weights,
                                experts)
        loss = lce.linear_cross_entropy(normed(h, w, "n2"), w["head"], labels,
                                        fused=True)
        total, load = loss, None
        if balance:
            aux, load = lce.balance_loss(logits, experts, scoring="sigmoid",
                                         coef=balance)
            total = loss + aux
        total.backward()
        with torch.no_grad():
            if max_norm is not None:
                lce.clip_grad_norm([t.grad for t in w.values()], max_norm)
            for k, v in master.items():
                v -= lr * w[k].grad.float()
            if load is None:
                load = lce.expert_counts(experts, E).float()
                bias -= 1e-3 * torch.sign(load - load.mean())
        losses.append(loss.item())
    status = lce.get_error()
    if status != 0:
        raise RuntimeError(f"device error status {status}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--norm", choices=("rms", "layer"))
    ap.add_argument("--balance", type=float, default=0.0)
    ap.add_argument("--max-norm", type=float)
    a = ap.parse_args()
    for i, loss in enumerate(run(a.steps, norm=a.norm, balance=a.balance,
                                 max_norm=a.max_norm)):
        print(f"step {i}: loss {loss:.4f}")

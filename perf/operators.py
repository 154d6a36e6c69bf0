"""The sparse-MLP operators as a user's program calls them, and what they
compute in elementary torch operations: routing of tokens to experts (with
its gradient) and the experts' gated MLP (forward alone for serving, forward
and backward for training).

A case is a dict of plain values; `prepare` makes its inputs on the GPU from
a seed, `run` makes one pass. With `own` set, `run` calls this package;
otherwise it computes the same in torch, in 32 bits (the selection of
experts in 64, where near-equal values decide), rounded once at the end.
`exact` is the definition in 64 bits, written apart from both.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _route(name, L, E, K, scoring, dtype, train, *, bias=False, n_group=1,
           topk_group=1, group_top=1, renorm=True, scale=1.0, masked=0.0):
    c = dict(op="route", L=L, E=E, K=K, scoring=scoring, dtype=dtype,
             train=train, bias=bias, n_group=n_group, topk_group=topk_group,
             group_top=group_top, renorm=renorm, scale=scale, masked=masked)
    return dict(c, name=name) if name else c


def _experts(name, L, H, I, E, K, train, *, skew=0.3, drop=0.0, wdtype="bf16"):
    c = dict(op="experts", L=L, H=H, I=I, E=E, K=K, train=train, skew=skew,
             drop=drop, wdtype=wdtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a decode loop: a launch and its latency
        _route("route_one_token", 1, 128, 8, "softmax", "f32", False),
        # a decode batch under bias-balanced, group-limited routing
        _route("route_decode_grouped", 64, 256, 8, "sigmoid", "f32", False,
               bias=True, n_group=8, topk_group=4, group_top=2, scale=2.5),
        # odd sizes, weights left as probabilities, some experts masked out
        _route("route_odd_train", 4099, 60, 4, "softmax", "bf16", True,
               renorm=False, masked=0.1),
        # a training step of a 128-expert layer
        _route("route_train", 32768, 128, 8, "softmax", "bf16", True),
        # a long training step, sigmoid scores, bias and groups
        _route("route_train_grouped", 65536, 256, 8, "sigmoid", "f32", True,
               bias=True, n_group=8, topk_group=4, group_top=2, scale=2.5),
        # one token of a decode loop: the chosen experts' weights are read
        _experts("experts_one_token", 1, 2048, 768, 128, 8, False),
        # a decode batch: most experts are touched, few rows each
        _experts("experts_decode_32", 32, 2048, 768, 128, 8, False),
        # a prompt
        _experts("experts_prompt", 4096, 2048, 768, 128, 8, False),
        # few wide experts over a longer prompt
        _experts("experts_wide_prompt", 8192, 4096, 8192, 8, 2, False,
                 wdtype="f32"),
        # odd sizes with dropped slots, forward and backward
        _experts("experts_odd_train", 1537, 1000, 424, 10, 2, True,
                 drop=0.03),
        # a training step over many small experts
        _experts("experts_train", 8192, 1024, 512, 64, 6, True),
        # a long training step
        _experts("experts_train_long", 32768, 2048, 768, 128, 8, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        n_group = rng.choice([1, 1, 2, 4, 8])
        per = _log_int(rng, 4, 384 // n_group)
        E = n_group * per
        scoring = rng.choice(["softmax", "sigmoid"])
        topk_group = rng.randint(1, n_group)
        K = rng.randint(1, min(8, topk_group * per))
        return _route(None, _log_int(rng, 1, 40000), E, K, scoring,
                      rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                      bias=rng.random() < 0.5, n_group=n_group,
                      topk_group=topk_group, group_top=rng.choice([1, 2]),
                      # one weight alone, renormalised, has no gradient
                      renorm=K > 1 and rng.random() < 0.7,
                      scale=rng.choice([1.0, 2.5]),
                      masked=rng.choice([0.0, 0.0, 0.1]))
    train = rng.random() < 0.5
    while True:
        H = 8 * _log_int(rng, 8, 512)
        I = 8 * _log_int(rng, 8, 512)
        E = _log_int(rng, 2, 160)
        K = rng.randint(1, min(8, E))
        L = _log_int(rng, 1, 16384)
        if E * H * I <= 128 * 2048 * 768 and L * K * H * I <= 1.5e11:
            break
    return _experts(None, L, H, I, E, K, train, skew=rng.choice([0.0, 0.3]),
                    drop=rng.choice([0.0, 0.0, 0.05]),
                    wdtype="bf16" if train else rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + k)
    return g


def _normal(shape, std, seed, k, dtype=torch.float32):
    """N(0, std^2), drawn in `dtype`."""
    return torch.randn(shape, device="cuda", dtype=dtype,
                       generator=_gen(seed, k)).mul_(std)


def prepare(case, seed):
    L, E, K = case["L"], case["E"], case["K"]
    if case["op"] == "route":
        # router logits: experts differ in popularity, tokens in confidence
        z = _normal((L, E), 1.5, seed, 0) + _normal((E,), 0.3, seed, 1)
        if case["masked"]:
            off = torch.rand((L, E), device="cuda", generator=_gen(seed, 2))
            z = z.masked_fill(off < case["masked"], -math.inf)
            z[0] = -math.inf  # and a row whose mask leaves nothing
        dt = DTYPES[case["dtype"]]
        return dict(case=case, logits=z.to(dt),
                    bias=_normal((E,), 0.05, seed, 3) if case["bias"] else None,
                    dweights=_normal((L, K), 1.0, seed, 4, dt)
                    if case["train"] else None)
    H, I = case["H"], case["I"]
    z = _normal((L, E), 1.0, seed, 0) + _normal((E,), case["skew"], seed, 1)
    top, experts = torch.topk(torch.softmax(z, -1), K, dim=-1)
    weights = top / top.sum(-1, keepdim=True)
    experts = experts.to(torch.int32)
    if case["drop"]:
        off = torch.rand((L, K), device="cuda", generator=_gen(seed, 2))
        experts = experts.masked_fill(off < case["drop"], -1)
    bf = torch.bfloat16
    return dict(case=case, experts=experts,
                weights=weights.to(DTYPES[case["wdtype"]]),
                x=_normal((L, H), 1.0, seed, 5, bf),
                Wg=_normal((E, I, H), H ** -0.5, seed, 6, bf),
                Wu=_normal((E, I, H), H ** -0.5, seed, 7, bf),
                Wd=_normal((E, H, I), I ** -0.5, seed, 8, bf),
                dy=_normal((L, H), 1.0, seed, 9, bf) if case["train"] else None)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _scores(z, scoring):
    """Scores of logits z in z's type; a row without a finite logit is 0."""
    if scoring == "sigmoid":
        return torch.sigmoid(z)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, torch.zeros_like(m), m))
    t = p.sum(-1, keepdim=True)
    return p / torch.where(t == 0, torch.ones_like(t), t)


def _select(logits, bias, c):
    """Indices of the K largest keys, ties to the lowest index (int64)."""
    L, E = logits.shape
    G = c["n_group"]
    z = logits.double()
    dead = (z == -math.inf) | torch.isnan(z)
    value = None
    if bias is not None or (G > 1 and c["group_top"] == 2):
        value = _scores(z, c["scoring"])
        if bias is not None:
            value = value + bias.double()
        value = value.masked_fill(dead, -math.inf)
    key = value if bias is not None else z.masked_fill(dead, -math.inf)
    if G == 1:
        return key.sort(dim=-1, descending=True, stable=True).indices[:, :c["K"]]
    per = (value if c["group_top"] == 2 else key).view(L, G, E // G)
    rank = per.sort(dim=-1, descending=True).values[..., :c["group_top"]].sum(-1)
    kept = rank.sort(dim=-1, descending=True, stable=True).indices
    keep = torch.zeros((L, G), dtype=torch.bool, device=z.device)
    keep.scatter_(1, kept[:, :c["topk_group"]], True)
    keep = keep.repeat_interleave(E // G, 1)
    # inside the kept groups even a masked expert comes before one outside
    key = key.clamp(min=torch.finfo(torch.float64).min)
    key = key.masked_fill(~keep, -math.inf)
    return key.sort(dim=-1, descending=True, stable=True).indices[:, :c["K"]]


def _route_plain(s):
    c = s["case"]
    logits = s["logits"]
    if c["train"]:
        logits = logits.detach().requires_grad_(True)
    experts = _select(s["logits"], s["bias"], c)
    p = _scores(logits.float(), c["scoring"]).gather(1, experts)
    if c["renorm"]:
        t = p.sum(-1, keepdim=True)
        p = torch.where(t == 0, torch.zeros_like(p),
                        p / torch.where(t == 0, torch.ones_like(t), t))
    w = p * c["scale"]
    out = dict(weights=w.detach().to(s["logits"].dtype),
               experts=experts.to(torch.int32))
    if c["train"]:
        out["dlogits"], = torch.autograd.grad(w, logits, s["dweights"].float())
    return out


def _experts_plain(s):
    c = s["case"]
    L, H, E, K = c["L"], c["H"], c["E"], c["K"]
    leaves = [s[k] for k in ("x", "Wg", "Wu", "Wd", "weights")]
    if c["train"]:
        leaves = [t.detach().requires_grad_(True) for t in leaves]
    x, Wg, Wu, Wd, w = (t.float() for t in leaves)
    flat = s["experts"].reshape(-1).long()
    live = flat >= 0
    e = flat.clamp(min=0)  # a dropped slot is computed with weight 0
    w = torch.where(live.view(L, K), w, torch.zeros_like(w))
    order = e.sort(stable=True).indices
    counts = torch.bincount(e, minlength=E)
    first = counts.cumsum(0) - counts
    place = torch.empty_like(e)
    place[order] = torch.arange(L * K, device=e.device) - first[e[order]]
    C = int(counts.max())
    place = e * C + place
    token = torch.arange(L * K, device=e.device) // K
    rows = torch.zeros((E * C, H), device=e.device)
    rows = rows.index_copy(0, place, x[token]).view(E, C, H)
    g = torch.bmm(rows, Wg.transpose(1, 2))
    a = g / (1 + torch.exp(-g)) * torch.bmm(rows, Wu.transpose(1, 2))
    ys = torch.bmm(a, Wd.transpose(1, 2)).view(E * C, H)[place]
    y = (ys.view(L, K, H) * w.unsqueeze(-1)).sum(1)
    out = dict(y=y.detach().to(torch.bfloat16))
    if c["train"]:
        grads = torch.autograd.grad(y, leaves, s["dy"].float())
        out.update(zip(("dx", "dWg", "dWu", "dWd", "dweights"), grads))
    return out


# ---------------------------------------------------------------------------
# this package
# ---------------------------------------------------------------------------
def _route_own(s):
    import chunked_lm_head_gemm_gb300 as lce
    c = s["case"]
    w, experts = lce.route_forward(
        s["logits"], c["K"], scoring=c["scoring"], bias=s["bias"],
        n_group=c["n_group"], topk_group=c["topk_group"],
        group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
    out = dict(weights=w, experts=experts)
    if c["train"]:
        out["dlogits"] = lce.route_backward(
            s["logits"], experts, s["dweights"], scoring=c["scoring"],
            renormalize=c["renorm"], scale=c["scale"])
    return out


def _experts_own(s):
    import chunked_lm_head_gemm_gb300 as lce
    args = [s[k] for k in ("x", "Wg", "Wu", "Wd", "weights", "experts")]
    out = dict(y=lce.experts_forward(*args))
    if s["case"]["train"]:
        grads = lce.experts_backward(*args, s["dy"], grad_dtype=torch.bfloat16)
        out.update(zip(("dx", "dWg", "dWu", "dWd", "dweights"), grads))
    return out


def run(state):
    if state["case"]["op"] == "route":
        if own:
            return _route_own(state)
        return _route_plain(state)
    if own:
        return _experts_own(state)
    return _experts_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    L, E, K = case["L"], case["E"], case["K"]
    if case["op"] == "route":
        b = 2 if case["dtype"] == "bf16" else 4
        moved = L * E * b + L * K * (4 + b)
        if case["train"]:  # the logits are there already; dweights, dlogits
            moved += L * K * b + L * E * b
        return dict(bytes=moved, flops=0)
    H, I = case["H"], case["I"]
    slots = L * K * (1 - case["drop"])
    # experts with a token, as if the slots fell on them evenly
    hit = E * (1 - (1 - 1 / E) ** slots)
    wb = 4 if case["wdtype"] == "f32" else 2
    moved = 2 * L * H * 2 + hit * 3 * H * I * 2 + L * K * (4 + wb)
    flops = slots * 6 * H * I
    if case["train"]:
        moved += 2 * L * H * 2 + E * 3 * H * I * 2 + L * K * wb
        flops *= 3
    return dict(bytes=moved, flops=flops)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)

    def largest(key, n):
        """n largest of each row, ties to the lowest index, one at a time."""
        at = torch.arange(key.shape[1], device=key.device)
        key, found = key.clone(), []
        for _ in range(n):
            top = key == key.amax(1, keepdim=True)
            i = torch.where(top, at, key.shape[1]).amin(1, keepdim=True)
            key.scatter_(1, i, -math.inf)
            found.append(i)
        return torch.cat(found, 1)

    def route(c):
        z = s["logits"].double()
        L, E = z.shape
        if c["scoring"] == "softmax":
            mass = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
            mass = torch.nan_to_num(mass, nan=0.0)
        else:
            mass = torch.sigmoid(z)
        value = mass + (0 if s["bias"] is None else s["bias"].double())
        value = torch.where(z == -math.inf, -math.inf, value)
        key = z if s["bias"] is None else value
        # a rank for each expert, so that what is left out can go below all
        place = torch.empty_like(z)
        order = largest(torch.clamp(key, min=-1e300), E)
        place.scatter_(1, order, -torch.arange(E, dtype=z.dtype,
                                               device=z.device).expand(L, E))
        G = c["n_group"]
        if G > 1:
            per = (value if c["group_top"] == 2 else key).reshape(L, G, -1)
            rank = per.topk(c["group_top"], dim=2).values.sum(2)
            # -inf ranks tie: count them from a value below every other
            kept = largest(torch.clamp(rank, min=-1e300), c["topk_group"])
            keep = torch.zeros_like(rank).scatter_(1, kept, 1.0)
            keep = keep.unsqueeze(2).expand(L, G, E // G).reshape(L, E)
            place = torch.where(keep > 0, place, place - 2 * E)
        chosen = largest(place, c["K"])
        p = torch.gather(mass, 1, chosen)
        q = torch.nan_to_num(p / p.sum(1, keepdim=True), nan=0.0)
        w = c["scale"] * (q if c["renorm"] else p)
        out = dict(weights=w, experts=None)
        if not c["train"]:
            return out
        u = c["scale"] * s["dweights"].double()
        dz = torch.zeros_like(z)
        if c["renorm"]:
            dz.scatter_(1, chosen, q * (u - (u * q).sum(1, keepdim=True)) *
                        (1 if c["scoring"] == "softmax" else 1 - p))
        elif c["scoring"] == "softmax":
            ds = torch.zeros_like(z).scatter_(1, chosen, u)
            dz = mass * (ds - (u * p).sum(1, keepdim=True))
        else:
            dz.scatter_(1, chosen, u * p * (1 - p))
        return dict(out, dlogits=dz)

    def experts(c):
        x, w = s["x"].double(), s["weights"].double()
        y = torch.zeros_like(x)
        if c["train"]:
            dy = s["dy"].double()
            dx, dw = torch.zeros_like(x), torch.zeros_like(w)
            dWg, dWu, dWd = (torch.zeros_like(s[k], dtype=torch.float64)
                             for k in ("Wg", "Wu", "Wd"))
        for i in range(c["E"]):
            t, k = torch.nonzero(s["experts"] == i, as_tuple=True)
            if not len(t):
                continue
            Wg, Wu, Wd = (s[n][i].double() for n in ("Wg", "Wu", "Wd"))
            r, wt = x[t], w[t, k].unsqueeze(1)
            g, u = r @ Wg.T, r @ Wu.T
            sg = torch.sigmoid(g)
            a = g * sg * u
            y.index_add_(0, t, wt * (a @ Wd.T))
            if c["train"]:
                up = dy[t]
                da = up @ Wd
                dw[t, k] = (da * a).sum(1)
                da = wt * da
                dg, du = da * u * sg * (1 + g * (1 - sg)), da * g * sg
                dx.index_add_(0, t, dg @ Wg + du @ Wu)
                dWg[i], dWu[i] = dg.T @ r, du.T @ r
                dWd[i] = up.T @ (wt * a)
        if c["train"]:
            return dict(y=y, dx=dx, dWg=dWg, dWu=dWu, dWd=dWd, dweights=dw)
        return dict(y=y)

    with torch.no_grad():
        return (route if case["op"] == "route" else experts)(case)

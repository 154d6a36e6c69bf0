"""Operators of a training step around the head and the (sparse) MLP, as a
user's program calls them, and what they compute in elementary torch
operations: layer norm and RMS norm (forward alone for serving, forward and
backward for training), the routing's balance loss with its per-expert counts
and gradient, and the global gradient norm with clipping.

A case is a dict of plain values; `prepare` makes its inputs on the GPU from
a seed, `run` makes one pass. With `own` set, `run` calls this package;
otherwise it computes the same in torch, in 32 bits (long sums in 64), rounded
once at the end. `exact` is the definition in 64 bits, written apart from
both.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _named(name, c):
    return dict(c, name=name) if name else c


def _norm(name, kind, L, H, dtype, wdtype, train, *, affine=True, offset=0.0):
    eps = 1e-5 if kind == "layer" else 1e-6
    return _named(name, dict(op="norm", kind=kind, L=L, H=H, dtype=dtype,
                             wdtype=wdtype, train=train, affine=affine,
                             offset=offset, eps=eps))


def _balance(name, L, E, K, scoring, dtype, train, *, padded=0.0, masked=0.0,
             drop=0.0, coef=0.01):
    return _named(name, dict(op="balance", L=L, E=E, K=K, scoring=scoring,
                             dtype=dtype, train=train, padded=padded,
                             masked=masked, drop=drop, coef=coef))


def _clip(name, layers, H, I, E, V, dtype, *, size=4.0, max_norm=1.0):
    return _named(name, dict(op="clip", layers=layers, H=H, I=I, E=E, V=V,
                             dtype=dtype, size=size, max_norm=max_norm))


def listed():
    return [
        # one token of a decode loop: a launch and its latency
        _norm("layer_norm_one_token", "layer", 1, 4096, "bf16", "bf16", False),
        # an odd batch of an odd width, fp32 parameters
        _norm("layer_norm_odd_train", "layer", 2053, 1001, "bf16", "f32", True,
              offset=0.5),
        # a training step whose residual stream is kept in fp32
        _norm("layer_norm_f32_train", "layer", 16384, 2560, "f32", "f32", True),
        # a decode batch in front of the experts
        _norm("rms_norm_decode", "rms", 64, 2048, "bf16", "bf16", False),
        # the norm of every attention head's 128 channels
        _norm("rms_norm_heads_train", "rms", 1 << 20, 128, "bf16", "bf16",
              True),
        # one GPU's shard of a long sequence, before the head
        _norm("rms_norm_long_train", "rms", 131072, 4096, "bf16", "bf16", True),
        # the load of the experts in one decode batch (counts alone)
        _balance("balance_decode_counts", 64, 128, 8, "softmax", "f32", False),
        # an odd, padded batch; some experts masked out, some slots dropped
        _balance("balance_odd_train", 4099, 60, 4, "softmax", "bf16", True,
                 padded=0.2, masked=0.1, drop=0.03),
        # a long training step's router, sigmoid scores
        _balance("balance_long_train", 131072, 256, 8, "sigmoid", "f32", True,
                 padded=0.05),
        # a small layer's gradients: the launches and the host's part
        _clip("clip_one_layer", 1, 64, 32, 4, 0, "f32", size=3.0),
        # many gradients of odd sizes, in two types
        _clip("clip_odd_layers", 24, 1001, 119, 8, 4099, "bf16", size=8.0),
        # sparse-MLP layers under a large head
        _clip("clip_large", 2, 2048, 768, 128, 151936, "bf16", size=30.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "balance", "clip"])
    if op == "norm":
        while True:
            H = _log_int(rng, 16, 16384)
            if rng.random() < 0.6:
                H = 8 * max(2, H // 8)
            L = _log_int(rng, 1, 1 << 20)
            if L * H <= 1 << 28:
                break
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return _norm(None, rng.choice(["layer", "rms"]), L, H, dtype,
                     rng.choice([dtype, "f32"]), rng.random() < 0.6,
                     affine=rng.random() < 0.85,
                     offset=rng.choice([0.0, 0.5]))
    if op == "balance":
        while True:
            E, L = _log_int(rng, 4, 512), _log_int(rng, 2, 131072)
            if L * E <= 131072 * 256:
                break
        return _balance(None, L, E, rng.randint(1, min(8, E)),
                        rng.choice(["softmax", "sigmoid"]),
                        rng.choice(["bf16", "f32"]), rng.random() < 0.75,
                        padded=rng.choice([0.0, 0.3]),
                        masked=rng.choice([0.0, 0.0, 0.1]),
                        drop=rng.choice([0.0, 0.05]))
    while True:
        layers, H = rng.randint(1, 40), _log_int(rng, 32, 4096)
        I, E = _log_int(rng, 16, 4096), _log_int(rng, 1, 64)
        V = rng.choice([0, _log_int(rng, 500, 150000)])
        if layers * 3 * E * I * H + V * H <= 1.2e9:
            break
    # below 1 nothing is clipped
    return _clip(None, layers, H, I, E, V, rng.choice(["bf16", "f32"]),
                 size=rng.choice([0.4, 5.0, 50.0]))


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


def _uniform(shape, seed, k):
    return torch.rand(shape, device="cuda", generator=_gen(seed, k))


def _shapes(c):
    """(shape, type) of every gradient: per layer the norm's weight, the
    router and the experts' three matrices, then the last norm and the head
    (empty where V is 0)."""
    H, I, E, V = c["H"], c["I"], c["E"], c["V"]
    layer = [((H,), "f32"), ((E, H), "f32"), ((E, I, H), c["dtype"]),
             ((E, I, H), c["dtype"]), ((E, H, I), c["dtype"])]
    return layer * c["layers"] + [((H,), "f32"), ((V, H), "f32")]


def _prepare_norm(c, seed):
    L, H = c["L"], c["H"]
    dt, wdt = DTYPES[c["dtype"]], DTYPES[c["wdtype"]]
    x = _normal((L, H), 1.0, seed, 0, dt)
    if c["offset"]:
        x += c["offset"]
    w = b = None
    if c["affine"]:
        w = _normal((H,), 0.2, seed, 1).add_(1.0).to(wdt)
        if c["kind"] == "layer":
            b = _normal((H,), 0.2, seed, 2).to(wdt)
    dy = _normal((L, H), 1.0, seed, 3, dt) if c["train"] else None
    return dict(case=c, x=x, weight=w, bias=b, dy=dy)


def _prepare_balance(c, seed):
    L, E, K = c["L"], c["E"], c["K"]
    # experts differ in popularity, tokens in confidence
    z = _normal((L, E), 1.5, seed, 0) + _normal((E,), 0.4, seed, 1)
    if c["masked"]:
        z = z.masked_fill(_uniform((L, E), seed, 2) < c["masked"], -math.inf)
        z[1] = -math.inf  # and a row whose mask leaves nothing
    experts = torch.topk(z, K, dim=-1).indices.to(torch.int32)
    if c["drop"]:
        off = _uniform((L, K), seed, 3) < c["drop"]
        experts = experts.masked_fill(off, -1)
    mask = None
    if c["padded"]:
        mask = _uniform((L,), seed, 4) >= c["padded"]
        mask[0] = True
    return dict(case=c, logits=z.to(DTYPES[c["dtype"]]), experts=experts,
                mask=mask, dloss=_uniform((), seed, 5) + 0.5)


def _prepare_clip(c, seed):
    shapes = _shapes(c)
    total = sum(math.prod(s) for s, _ in shapes)
    std = c["size"] * c["max_norm"] / math.sqrt(total)
    # tensors differ in the size of their gradients
    spread = [0.7, 1.0, 1.3, 0.5, 1.2]
    grads = [_normal(s, std * spread[i % 5], seed, i, DTYPES[t])
             for i, (s, t) in enumerate(shapes)]
    # the clipped gradients go into one buffer of each type, as an optimizer
    # with flat buffers keeps them
    flat, place, outs = {}, {}, []
    for name, dt in DTYPES.items():
        n = sum(math.prod(s) for s, t in shapes if t == name)
        if n:
            flat[name] = torch.empty(n, dtype=dt, device="cuda")
        place[name] = 0
    for s, t in shapes:
        n = math.prod(s)
        outs.append(flat[t][place[t]:place[t] + n].view(s))
        place[t] += n
    return dict(case=c, grads=grads, outs=outs, flat=flat)


def prepare(case, seed):
    make = dict(norm=_prepare_norm, balance=_prepare_balance,
                clip=_prepare_clip)
    return make[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _norm_plain(s):
    c = s["case"]
    names = [k for k in ("x", "weight", "bias") if s[k] is not None]
    leaves = {k: s[k].detach().requires_grad_(c["train"]) for k in names}
    x = leaves["x"].float()
    if c["kind"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + c["eps"])
    if "weight" in leaves:
        y = y * leaves["weight"].float()
    if "bias" in leaves:
        y = y + leaves["bias"].float()
    out = dict(y=y.detach().to(s["x"].dtype))
    if c["train"]:
        grads = torch.autograd.grad(y, list(leaves.values()), s["dy"].float())
        out.update(("d" + k, g) for k, g in zip(names, grads))
    return out


def _probabilities(z, scoring):
    """Each row's scores, normalised; a row without a finite logit is 0."""
    if scoring == "sigmoid":
        p = torch.sigmoid(z)
    else:
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - torch.where(m == -math.inf, torch.zeros_like(m), m))
    t = p.sum(-1, keepdim=True)
    return p / torch.where(t == 0, torch.ones_like(t), t)


def _counts_plain(s):
    c = s["case"]
    live = s["experts"] >= 0
    if s["mask"] is not None:
        live = live & s["mask"].unsqueeze(1)
    at = torch.where(live, s["experts"], c["E"]).reshape(-1).long()
    counts = torch.zeros(c["E"] + 1, dtype=torch.int32, device=at.device)
    counts.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    return counts[:-1]


def _balance_plain(s):
    c = s["case"]
    counts = _counts_plain(s)
    if not c["train"]:
        return dict(counts=counts)
    logits = s["logits"].detach().requires_grad_(True)
    z = logits.float()
    p = _probabilities(z, c["scoring"])
    if s["mask"] is None:
        n = c["L"]
    else:
        n = s["mask"].sum()
        p = torch.where(s["mask"].unsqueeze(1), p, torch.zeros_like(p))
    share = counts.double() * c["E"] / (n * c["K"])
    mean = p.sum(0, dtype=torch.float64) / n
    loss = c["coef"] * (share * mean).sum()
    dlogits, = torch.autograd.grad(loss, logits, s["dloss"].double())
    return dict(loss=loss.detach().float(), counts=counts, dlogits=dlogits)


def _clip_plain(s):
    c = s["case"]
    every = torch.cat([g.reshape(-1).float() for g in s["grads"]])
    norm = (every * every).sum(dtype=torch.float64).sqrt()
    scale = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0).float()
    out = dict(norm=norm.float())
    for name in s["flat"]:
        dt = DTYPES[name]
        out[name] = torch.cat([(g.reshape(-1).float() * scale).to(dt)
                               for g in s["grads"] if g.dtype == dt])
    return out


# ---------------------------------------------------------------------------
# this package
# ---------------------------------------------------------------------------
def _norm_own(s):
    import chunked_lm_head_gemm_gb300 as lce
    c, x, w, b = s["case"], s["x"], s["weight"], s["bias"]
    train, layer = c["train"], c["kind"] == "layer"
    if layer:
        y, mean, rstd = lce.layer_norm_forward(x, w, b, eps=c["eps"],
                                               save_stats=train)
    else:
        y, rstd = lce.rms_norm_forward(x, w, eps=c["eps"], save_stats=train)
    out = dict(y=y)
    if not train:
        return out
    kw = dict(compute_dweight=c["affine"])
    if c["affine"]:
        kw["grad_dtype"] = w.dtype
    if layer:
        dx, dw, db = lce.layer_norm_backward(x, w, mean, rstd, s["dy"],
                                             compute_dbias=c["affine"], **kw)
    else:
        dx, dw = lce.rms_norm_backward(x, w, rstd, s["dy"], **kw)
        db = None
    out.update((k, g) for k, g in (("dx", dx), ("dweight", dw), ("dbias", db))
               if g is not None)
    return out


def _balance_own(s):
    import chunked_lm_head_gemm_gb300 as lce
    c = s["case"]
    if not c["train"]:
        return dict(counts=lce.expert_counts(s["experts"], c["E"],
                                             mask=s["mask"]))
    loss, counts, slopes = lce.balance_forward(
        s["logits"], s["experts"], scoring=c["scoring"], coef=c["coef"],
        mask=s["mask"])
    dlogits = lce.balance_backward(s["logits"], slopes, s["dloss"],
                                   scoring=c["scoring"], mask=s["mask"])
    return dict(loss=loss, counts=counts, dlogits=dlogits)


def _clip_own(s):
    import chunked_lm_head_gemm_gb300 as lce
    norm = lce.clip_grad_norm(s["grads"], s["case"]["max_norm"],
                              grads_out=s["outs"])
    return dict(s["flat"], norm=norm)


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(norm=_norm_own, balance=_balance_own,
                    clip=_clip_own)[op](state)
    return dict(norm=_norm_plain, balance=_balance_plain,
                clip=_clip_plain)[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "norm":
        b = 2 if case["dtype"] == "bf16" else 4
        wb = 2 if case["wdtype"] == "bf16" else 4
        passes = 4 if case["train"] else 2  # x, y and dy, dx
        params = case["affine"] * (2 if case["kind"] == "layer" else 1)
        moved = passes * case["L"] * case["H"] * b
        moved += params * case["H"] * wb * (2 if case["train"] else 1)
        return dict(bytes=moved, flops=0)
    if case["op"] == "balance":
        L, E, K = case["L"], case["E"], case["K"]
        moved = L * K * 4 + E * 4 + (L if case["padded"] else 0)
        if case["train"]:
            moved += 2 * L * E * (2 if case["dtype"] == "bf16" else 4)
        return dict(bytes=moved, flops=0)
    total = sum(math.prod(s) * (2 if t == "bf16" else 4)
                for s, t in _shapes(case))
    return dict(bytes=2 * total, flops=0)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_norm(s):
    c, H = s["case"], s["case"]["H"]
    w = 1.0 if s["weight"] is None else s["weight"].double()
    out = {"y": torch.empty_like(s["x"], dtype=torch.float64)}
    if c["train"]:
        out["dx"] = torch.empty_like(out["y"])
        if c["affine"]:
            out["dweight"] = 0.0
            if c["kind"] == "layer":
                out["dbias"] = 0.0
    step = max(1, (1 << 27) // H)
    for i in range(0, c["L"], step):
        rows = slice(i, i + step)
        x = s["x"][rows].double()
        if c["kind"] == "layer":
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            r = 1 / torch.sqrt(var + c["eps"])
            n = (x - mean) * r
        else:
            r = 1 / torch.sqrt(x.square().sum(1, keepdim=True) / H + c["eps"])
            n = x * r
        out["y"][rows] = n * w + (0.0 if s["bias"] is None
                                  else s["bias"].double())
        if not c["train"]:
            continue
        dy = s["dy"][rows].double()
        g = dy * w
        dx = g - n * ((g * n).sum(1, keepdim=True) / H)
        if c["kind"] == "layer":
            dx -= g.sum(1, keepdim=True) / H
        out["dx"][rows] = dx * r
        if c["affine"]:
            out["dweight"] = out["dweight"] + torch.einsum("ij,ij->j", dy, n)
            if c["kind"] == "layer":
                out["dbias"] = out["dbias"] + dy.sum(0)
    return out


def _exact_balance(s):
    c = s["case"]
    if not c["train"]:
        return None  # counts alone
    E, K = c["E"], c["K"]
    keep = torch.ones(c["L"], device="cuda", dtype=torch.bool)
    if s["mask"] is not None:
        keep = s["mask"]
    z = s["logits"][keep].double()
    chosen = s["experts"][keep]
    N = z.shape[0]
    load = torch.stack([(chosen == e).sum() for e in range(E)]).double()
    f = load * E / (N * K)
    if c["scoring"] == "softmax":
        p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        slope = torch.ones_like(z)
    else:
        log_s = torch.nn.functional.logsigmoid(z)
        p = torch.exp(log_s - torch.logsumexp(log_s, 1, keepdim=True))
        slope = torch.sigmoid(-z)
    p = torch.nan_to_num(p, nan=0.0)
    loss = c["coef"] * torch.dot(f, p.mean(0))
    dz = p * slope * (f - (p @ f).unsqueeze(1))
    dlogits = torch.zeros(c["L"], E, device="cuda", dtype=torch.float64)
    dlogits[keep] = dz * (c["coef"] / N * s["dloss"].double())
    return dict(loss=loss, counts=None, dlogits=dlogits)


def _exact_clip(s):
    c = s["case"]
    total = math.fsum(float(g.double().square().sum()) for g in s["grads"])
    norm = math.sqrt(total)
    scale = min(1.0, c["max_norm"] / (norm + 1e-6))
    out = dict(norm=torch.tensor(norm, dtype=torch.float64))
    for name in s["flat"]:
        out[name] = torch.cat([g.reshape(-1).double() for g in s["grads"]
                               if g.dtype == DTYPES[name]]) * scale
    return out


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        return dict(norm=_exact_norm, balance=_exact_balance,
                    clip=_exact_clip)[case["op"]](s)

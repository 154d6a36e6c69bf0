"""Plain float64 reference of the norms, the balance loss and the gradient
clipping, in torch on whatever device the inputs are, each gradient by its
formula. What the operators keep in fp32 between their calls (mean, rstd,
slopes, norm) is an input here too, so that each call is checked by itself."""
import math

import torch

U = 2.0 ** -24  # half a step of fp32


def half(dtype):
    return torch.finfo(dtype).eps / 2


def norm(x, weight, bias, eps, layer):
    """(y, mean, rstd), float64."""
    x = x.double()
    mean = x.mean(1) if layer else torch.zeros_like(x[:, 0])
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y, mean, rstd


def norm_grad(x, weight, mean, rstd, dy, layer):
    """(dx, dweight, dbias), float64, from the given statistics."""
    x, dy, r = x.double(), dy.double(), rstd.double()[:, None]
    n = (x - mean.double()[:, None]) * r if layer else x * r
    g = dy if weight is None else dy * weight.double()
    dx = g - n * (g * n).mean(1, keepdim=True)
    if layer:
        dx = dx - g.mean(1, keepdim=True)
    return dx * r, (dy * n).sum(0), dy.sum(0)


def sum_bound(n):
    """Relative to the sum of magnitudes, what a fp32 sum of n terms may lose:
    at most n / 128 + 64 additions follow one another."""
    return (n / 128 + 64) * U


def norm_tolerance(x, weight, bias, eps, layer, dtype):
    """Bound of |y - reference| by the roundings: of the mean (A times the mean
    magnitude), of the variance and its root (A / 2 and the square of the
    mean's error), of the products, and of the result."""
    A = sum_bound(x.shape[1])
    y, mean, rstd = norm(x, weight, bias, eps, layer)
    r = rstd[:, None]
    off = A * x.double().abs().mean(1, keepdim=True) if layer else 0.0
    w = 1.0 if weight is None else weight.double().abs()
    n = (x.double() - mean[:, None]).abs() * r
    rel = A + 8 * U + (off * r) ** 2
    return w * r * off + w * n * rel + y.abs() * (half(dtype) + 2 * U) + 1e-37


def norm_grad_tolerance(x, weight, mean, rstd, dy, layer, dtype, grad_dtype):
    """Bounds for (dx, dweight, dbias) against norm_grad."""
    A, B = sum_bound(x.shape[1]), sum_bound(x.shape[0])
    xd, d, r = x.double(), dy.double().abs(), rstd.double()[:, None]
    n = ((xd - mean.double()[:, None]) if layer else xd).abs() * r
    g = d if weight is None else d * weight.double().abs()
    mg = g.mean(1, keepdim=True) if layer else 0.0
    mgn = (g * n).mean(1, keepdim=True)
    dx, dw, db = norm_grad(x, weight, mean, rstd, dy, layer)
    tx = r * (4 * U * g + (A + 4 * U) * mg + n * (A + 12 * U) * mgn)
    tw = (B + 5 * U) * (d * n).sum(0)
    tb = B * d.sum(0)
    return (tx + dx.abs() * half(dtype) + 1e-37,
            tw + dw.abs() * half(grad_dtype) + 1e-37,
            tb + db.abs() * half(grad_dtype) + 1e-37)


def probabilities(z, scoring):
    """Normalised scores of float64 logits and the factor of the score's
    derivative; a row without a logit above -inf is 0."""
    if scoring == "softmax":
        p = torch.softmax(z, 1)
        d = torch.ones_like(z)
    else:
        p = torch.softmax(torch.nn.functional.logsigmoid(z), 1)
        d = torch.sigmoid(-z)
    dead = (z == -math.inf).all(1, keepdim=True)
    return torch.where(dead, torch.zeros_like(p), p), d


def balance(logits, experts, scoring, coef, mask):
    """(loss, counts, slopes), float64 and int64."""
    L, E = logits.shape
    keep = torch.ones(L, dtype=torch.bool, device=logits.device) \
        if mask is None else mask
    chosen = experts[keep].reshape(-1).long()
    counts = torch.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
    N = int(keep.sum())
    if N == 0:
        zero = torch.zeros(E, dtype=torch.float64, device=logits.device)
        return zero.sum(), counts, zero
    f = counts.double() * E / (N * experts.shape[1])
    p, _ = probabilities(logits[keep].double(), scoring)
    return coef * (f * p.mean(0)).sum(), counts, coef / N * (f - 1)


def balance_grad(logits, slopes, dloss, scoring, mask):
    """dlogits, float64, from the given slopes."""
    p, d = probabilities(logits.double(), scoring)
    c = slopes.double()
    dz = dloss * p * d * (c - (p * c).sum(1, keepdim=True))
    if mask is not None:
        dz = torch.where(mask[:, None], dz, torch.zeros_like(dz))
    return dz


def balance_rel(logits):
    """Relative error of a row's p: the rounding of its argument (that of the
    largest distance from the row's maximum), two exponentials, the division
    and the sum of at most 1024."""
    z = logits.double()
    z = torch.where(torch.isfinite(z), z, torch.zeros_like(z))
    return (4 * z.abs().amax(1, keepdim=True) + 100) * U


def balance_grad_tolerance(logits, slopes, dloss, scoring, mask, dtype):
    p, d = probabilities(logits.double(), scoring)
    c, rel = slopes.double().abs(), balance_rel(logits)
    dot = (p * c).sum(1, keepdim=True)
    t = abs(dloss) * p * d * (2 * rel + 50 * U) * (c + dot)
    dz = balance_grad(logits, slopes, dloss, scoring, mask)
    return t + dz.abs() * half(dtype) + 1e-37


def grad_norm(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum())
                               for g in grads))


def clip(grads, norm, max_norm):
    r = max_norm / (norm + 1e-6)
    scale = 1.0 if r >= 1.0 or max_norm == math.inf else r
    return [g.double() * scale for g in grads]

"""Plain 64-bit forms of the norm, the expert routing and the 8-bit products' epilogue, on the CPU, and how far fp32 may be off."""
import math

import torch

from tests._fp8 import HALF_STEP, SMALLEST

U = 2.0 ** -24  # half a step of fp32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------------------------------ norm
def norm_sum(x, residual):
    """What is normalised: both are exact in fp32's sum but for its one rounding, and one more to x's type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm(r, weight, eps):
    v = r.double()
    rstd = (v.square().mean(1) + eps).rsqrt()
    return v * rstd[:, None] * weight.double(), rstd


def row_adds(h):
    """Additions that a row's sum passes at most: a thread's values (8 of every 8 * 1024), the lanes', the waves'."""
    return 8 * -(-h // 8192) + 6 + 16


def rstd_tolerance(h):
    """Relative: the squares' rounding and sum, halved by the root; the mean, eps, root and reciprocal."""
    return ((row_adds(h) + 1) / 2 + 3) * U


def norm_tolerance(y, h, dtype):
    """y = (r rstd) w: two more products, then half a step of its type."""
    t = (rstd_tolerance(h) + 2 * U) * y.abs()
    return t + HALF_STEP[dtype] * (y.abs() + t) + SMALLEST[dtype]


def norm_backward(dy, x, weight, rstd, dresidual):
    """(dx, dweight) and how far fp32's may be off before the rounding to x's type."""
    v, w, d, s = x.double(), weight.double(), dy.double(), rstd.double()[:, None]
    xn, wd = v * s, w * d
    mean = (wd * xn).mean(1, keepdim=True)
    a, b = s * wd, s * xn * mean
    r = torch.zeros_like(a) if dresidual is None else dresidual.double()
    # each of the three terms passes at most 6 roundings; the mean's sum as row_adds says, of terms with 3 of their own
    err = 6 * U * (a.abs() + b.abs() + r.abs()) + (s * xn).abs() * (row_adds(x.shape[1]) + 4) * U * (wd * xn).abs().mean(1, keepdim=True)
    # a strip's rows, then 8 groups of at most 512 strips
    adds = -(-x.shape[0] // 512) + 64 + 8 + 2
    return (a - b + r, err), ((d * xn).sum(0), adds * U * (d * xn).abs().sum(0))


# ------------------------------------------------------------------------------------------ route
def scores(logits, kind):
    l = logits.double()
    l = torch.where(l.isnan(), -math.inf, l)
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    p = torch.where(l == top, 1.0, torch.exp(l - top))
    p = torch.where(l == -math.inf, 0.0, p)
    return p / p.sum(1, keepdim=True).clamp_min(1e-300)


def route(logits, topk, bias=None, score="softmax", groups=1, topk_groups=None, group_top=2, renormalize=True, scale=1.0):
    """(ids, weights) by lists of whole rows."""
    s = scores(logits, score)
    l = logits.double()
    t, e = l.shape
    key = l.clone() if bias is None and groups == 1 else s + (0 if bias is None else bias.double())
    key = torch.where(key.isnan() | (l.isnan()) | (l == -math.inf), -math.inf, key).tolist()
    size = e // groups
    kept = topk_groups or groups
    ids, weights = [], []
    for i in range(t):
        k = key[i]
        if groups > 1:
            best = []
            for g in range(groups):
                high = [v for v in sorted(k[g * size:(g + 1) * size], reverse=True)[:group_top] if v > -math.inf]
                best.append(sum(high) if high else -math.inf)
            order = sorted(range(groups), key=lambda g: (-best[g], g))[:kept]
            k = [v if j // size in order else -math.inf for j, v in enumerate(k)]
        row = [j for j in sorted(range(e), key=lambda j: (-k[j], j))[:topk] if k[j] > -math.inf]
        w = [s[i, j].item() for j in row]
        total = sum(w) if renormalize else 1.0
        ids.append(row + [-1] * (topk - len(row)))
        weights.append([scale * v / total if total > 0 else 0.0 for v in w] + [0.0] * (topk - len(row)))
    return torch.tensor(ids, dtype=torch.int32).view(t, topk), torch.tensor(weights, dtype=torch.float64).view(t, topk)


def route_weights(logits, ids, score, renormalize, scale):
    """The weights of a given choice, differentiable in 64-bit logits."""
    s = torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)
    w = s.gather(1, ids.long().clamp_min(0)) * (ids >= 0)
    return scale * (w / w.sum(1, keepdim=True) if renormalize else w)


# fp32 exponentials of arguments up to 16 (their rounding, 16 U), and a few roundings more
SCORE_TOLERANCE = 2.0 ** -19


# --------------------------------------------------------------------------------------- epilogue
def phi(v):
    return 0.5 * torch.special.erfc(-v / math.sqrt(2))


def activation(v, act):
    if act == "relu":
        return torch.where(v > 0, v, 0.0)
    return v * phi(v) if act == "gelu" else v * torch.sigmoid(v) if act == "silu" else v


def activation_grad(v, act):
    if act == "relu":
        return (v > 0).double()
    if act == "gelu":
        return phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s)) if act == "silu" else torch.ones_like(v)


def activation_error(v, act):
    """Of the fp32 activation.  GELU: 1.5e-7 of erf's approximation, so 0.75e-7 |v| of v Phi(-|v|) where Phi is not 0 (|v| < 6), and a few roundings;
    SiLU: e^-v by its argument's rounding, |v| 2^-24, the hardware's exp2 and reciprocal, an ulp each, two roundings."""
    if act == "gelu":
        return 0.75e-7 * v.abs().clamp_max(6) + 8 * U * v.abs()
    return v.abs() * torch.sigmoid(v) * (v.abs() * 2 + 8) * U if act == "silu" else torch.zeros_like(v)


def activation_grad_error(v, act):
    """GELU': the same of Phi, and of |v| phi(v) <= 0.25; SiLU': of s (1 + v (1 - s)), whose parts are at most s and |v| s (1 - s)."""
    if act == "gelu":
        return 0.75e-7 + 16 * U * (1 + 0 * v)
    s = torch.sigmoid(v)
    return (s + v.abs() * s * (1 - s)) * (2 * v.abs() + 12) * U if act == "silu" else torch.zeros_like(v)

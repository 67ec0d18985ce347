"""Measured cases of the operators around the 8-bit products: the root-mean-square norm with the residual's addition, routing
to experts, and the products' epilogue (bias, activation, residual), each with its gradients.

listed() names the cases, draw(rng) gives more of the same ranges, prepare(case, seed) makes what a
program has in hand before the call, run(state) is one call, exact(case, seed) the same result in
64 bits and work(case) the bytes and operations a pass cannot do without.  `own` selects between
the operators' plain form (elementary torch operations, the default) and the library's.

Sizes: hidden size 5120, up to 8192 tokens and the 17408-wide intermediate of the library's SwiGLU-MLP workload; 64 experts,
8 per token, as a generic sparse layer, or 256 in 8 groups; single tokens for serving.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
AMAX_MIN = 2.0 ** -90  # the smallest block maximum a scale is made from
B = 128                # scale block
EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # before every product of one new token: the layer's output joins the residual stream, 8-bit rows leave
        {"name": "norm_1x5120_fp8", "op": "norm", "m": 1, "h": 5120, "dtype": "bf16", "wide_weight": False, "residual": True, "fp8": True},
        # the same in a training step or for a long prompt
        {"name": "norm_8192x5120_fp8", "op": "norm", "m": 8192, "h": 5120, "dtype": "bf16", "wide_weight": False, "residual": True, "fp8": True},
        # a ragged batch of prompts, a row length that is no multiple of anything, the norm's output for a 16-bit product
        {"name": "norm_777x5003", "op": "norm", "m": 777, "h": 5003, "dtype": "fp16", "wide_weight": True, "residual": True, "fp8": False},
        # a training step's gradients, with the one that comes down the residual stream
        {"name": "norm_backward_8192x5120", "op": "norm_backward", "m": 8192, "h": 5120, "dtype": "bf16", "wide_weight": False, "residual": True},
        # the same in full precision, at sizes that are no multiples
        {"name": "norm_backward_777x5003_fp32", "op": "norm_backward", "m": 777, "h": 5003, "dtype": "fp32", "wide_weight": True, "residual": False},
        # one new token routed
        {"name": "route_1_token", "op": "route", "t": 1, "e": 64, "topk": 8, "score": "softmax", "bias": False, "groups": 1,
         "topk_groups": 1, "group_top": 1, "renorm": True, "dtype": "bf16"},
        # a training step's tokens, balanced by a bias, each restricted to half of the groups
        {"name": "route_8192_tokens_256_experts", "op": "route", "t": 8192, "e": 256, "topk": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_top": 2, "renorm": True, "dtype": "fp32"},
        # the gradients of a softmax router whose weights are the probabilities themselves
        {"name": "route_backward_8192_tokens_64_experts", "op": "route_backward", "t": 8192, "e": 64, "topk": 8, "score": "softmax",
         "renorm": False, "dtype": "fp32"},
        # a down projection for one new token, added to the residual stream
        {"name": "linear_1x5120x17408", "op": "linear", "m": 1, "n": 5120, "k": 17408, "dtype": "bf16", "act": "none", "bias": True,
         "residual": True, "pre": False},
        # a ragged batch of prompts against sizes that are no multiples of a tile or a scale block
        {"name": "linear_777x5003x4112_gelu", "op": "linear", "m": 777, "n": 5003, "k": 4112, "dtype": "fp16", "act": "gelu", "bias": True,
         "residual": True, "pre": False},
        # an up projection of a training step, which keeps the pre-activation for its gradient
        {"name": "linear_8192x17408x5120_gelu", "op": "linear", "m": 8192, "n": 17408, "k": 5120, "dtype": "bf16", "act": "gelu",
         "bias": True, "residual": False, "pre": True},
        # the gradient of that epilogue, as the operands of the two products that follow
        {"name": "linear_backward_8192x17408_gelu", "op": "linear_backward", "m": 8192, "n": 17408, "dtype": "bf16", "act": "gelu"},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number from lo to hi, even over its logarithm, a multiple of step."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(step, min(hi, v) // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "route", "route", "route_backward", "linear", "linear", "linear_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    yes = lambda p=0.5: rng.random() < p  # noqa: E731
    if op in ("norm", "norm_backward"):
        c = {"op": op, "m": _log(rng, 1, 8192), "h": _log(rng, 64, 8192), "dtype": dtype, "wide_weight": yes(), "residual": yes(0.7)}
        if op == "norm":
            c["fp8"] = yes()
        return c
    if op in ("route", "route_backward"):
        e = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        c = {"op": op, "t": _log(rng, 1, 16384), "e": e, "topk": rng.choice([1, 2, 4, 6, 8]), "score": rng.choice(["softmax", "sigmoid"]),
             "renorm": yes(), "dtype": dtype}
        if op == "route":
            groups = rng.choice([1, 1, 4, 8]) if e >= 64 and e % 8 == 0 else 1
            c.update(bias=yes(), groups=groups, topk_groups=max(1, groups // 2), group_top=rng.choice([1, 2]))
        elif c["topk"] == 1:
            c["renorm"] = False  # (a single weight brought to 1 has no gradient but rounding)
        return c
    act = rng.choice(["none", "relu", "gelu", "silu"])
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 16384), "k": _log(rng, 128, 5120, 16), "dtype": dtype, "act": act,
                "bias": yes(0.7), "residual": yes(), "pre": yes(0.4)}
    return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 16384), "dtype": dtype, "act": act}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _values(shape, g, dtype):
    """Activations: normal, with some features (columns) a dozen times larger."""
    x = torch.randn(shape, generator=g, device="cuda")
    big = torch.rand(shape[-1], generator=g, device="cuda") < 0.01
    return (x * (1 + 11 * big)).to(dtype)


def _operand(shape, g):
    """e4m3 values as a quantised normal matrix has them: its block's largest at 448."""
    return (torch.randn(shape, generator=g, device="cuda") * 120.0).clamp_(-F8_MAX, F8_MAX).to(F8)


def _scales(shape, g, size):
    return (torch.rand(shape, generator=g, device="cuda") + 0.5) * size


def _blocks(n):
    return -(-n // B)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    dtype = DT[case["dtype"]]
    r = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    if op in ("norm", "norm_backward"):
        m, h = case["m"], case["h"]
        s["x"] = _values((m, h), g, dtype)
        s["w"] = (1 + 0.1 * r(h)).to(torch.float32 if case["wide_weight"] else dtype)
        s["residual"] = _values((m, h), g, dtype) if case["residual"] else None
        if op == "norm_backward":
            s["dy"] = r(m, h).to(dtype)
            s["rstd"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
    elif op in ("route", "route_backward"):
        t, e = case["t"], case["e"]
        # some experts more popular than others
        s["logits"] = (r(t, e) + 0.5 * r(1, e)).to(dtype)
        if op == "route":
            s["bias"] = 0.05 * r(e) if case["bias"] else None
        else:
            s["ids"] = torch.rand((t, e), generator=g, device="cuda").topk(case["topk"], dim=1).indices.to(torch.int32)
            s["dweights"] = r(t, case["topk"])
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s.update(a=_operand((m, k), g), sa=_scales((_blocks(k), m), g, 0.01).t(), b=_operand((n, k), g),
                 sb=_scales((_blocks(n), _blocks(k)), g, 1e-4), bias=(0.5 * r(n)).to(dtype) if case["bias"] else None,
                 residual=_values((m, n), g, dtype) if case["residual"] else None)
    else:
        m, n = case["m"], case["n"]
        s.update(dout=r(m, n).to(dtype), pre=r(m, n).to(dtype) if case["act"] != "none" else None)
    return s


# -------------------------------------------------------------------------------- plain forms
def _quantize(x):
    """e4m3 values and scales of x's blocks of 1 x 128; the last ones may be partly filled."""
    m, k = x.shape
    kb = _blocks(k)
    v = torch.nn.functional.pad(x.float(), (0, kb * B - k)).view(m, kb, B)
    finite = v.isfinite()
    amax = torch.where(finite, v.abs(), 0.0).amax(2, keepdim=True).clamp_min(AMAX_MIN)
    top = torch.full_like(amax, F8_MAX)  # (divided as tensors: with a number, torch multiplies by a reciprocal)
    q = torch.where(finite, v * (top / amax), float("nan")).to(F8)
    return q.view(m, kb * B)[:, :k], (amax / top).view(m, kb)


def _rows_fp32(q, scale):
    """The values that e4m3 rows and their scales of 128 features stand for."""
    return q.float() * scale.repeat_interleave(B, -1)[..., :q.shape[-1]]


def _blocks_fp32(q, scale):
    """The same for scales of 128 x 128."""
    return _rows_fp32(q, scale.repeat_interleave(B, -2)[..., :q.shape[-2], :])


def _activate(v, act):
    if act == "relu":
        return torch.where(v > 0, v, 0.0)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v / (1 + torch.exp(-v)) if act == "silu" else v


def _activate_grad(v, act):
    if act == "relu":
        return (v > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    p = 1 / (1 + torch.exp(-v))
    return p * (1 + v * (1 - p))


def _scores(logits, kind):
    """Router scores in 64 bits: values next to each other decide which expert is taken."""
    l = logits.double()
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    p = torch.exp(l - l.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _order(key):
    """Indices by falling key, the lowest index first among equal ones."""
    return key.sort(dim=1, descending=True, stable=True).indices


def _route(s):
    c = s["case"]
    t, e, groups = c["t"], c["e"], c["groups"]
    scores = _scores(s["logits"], c["score"])
    key = s["logits"].double()
    if s["bias"] is not None or groups > 1:
        key = scores if s["bias"] is None else scores + s["bias"].double()
    if groups > 1:
        in_group = key.view(t, groups, e // groups)
        best = in_group.sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        kept = torch.zeros((t, groups), dtype=torch.bool, device="cuda").scatter_(1, _order(best)[:, :c["topk_groups"]], True)
        key = in_group.masked_fill(~kept[:, :, None], -math.inf).view(t, e)
    ids = _order(key)[:, :c["topk"]]
    w = scores.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), w.float()


def _route_backward(s):
    c = s["case"]
    scores = _scores(s["logits"], c["score"])
    ids = s["ids"].long()
    g = s["dweights"].double()
    if c["renorm"]:
        chosen = scores.gather(1, ids)
        total = chosen.sum(1, keepdim=True)
        g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(scores).scatter_add_(1, ids, g)
    if c["score"] == "sigmoid":
        d = ds * scores * (1 - scores)
    else:
        d = scores * (ds - (ds * scores).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _plain(s):
    c = s["case"]
    op = c["op"]
    dtype = DT[c["dtype"]]
    if op == "norm":
        x = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dtype)
        v = x.float()
        rstd = (v.square().mean(1) + EPS).rsqrt()
        y = v * rstd[:, None] * s["w"].float()
        return (_quantize(y) if c["fp8"] else (y.to(dtype),)) + (x, rstd)
    if op == "norm_backward":
        x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        xn = x * rstd
        wdy = dy * s["w"].float()
        dx = rstd * (wdy - xn * (wdy * xn).mean(1, keepdim=True))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        return dx.to(dtype), (dy * xn).sum(0)
    if op == "route":
        return _route(s)
    if op == "route_backward":
        return _route_backward(s)
    if op == "linear":
        p = _rows_fp32(s["a"], s["sa"]) @ _blocks_fp32(s["b"], s["sb"]).t()
        if s["bias"] is not None:
            p = p + s["bias"].float()
        d = _activate(p, c["act"])
        if s["residual"] is not None:
            d = d + s["residual"].float()
        return (d.to(dtype), p.to(dtype)) if c["pre"] else d.to(dtype)
    d = s["dout"].float()
    if s["pre"] is not None:
        d = d * _activate_grad(s["pre"].float(), c["act"])
    return _quantize(d) + _quantize(d.t()) + (d.sum(0),)


# ------------------------------------------------------------------------------ library calls
def _own(s):
    import dense_gemm_epilogues_amd as ep

    c = s["case"]
    op = c["op"]
    dtype = DT[c["dtype"]]
    if op == "norm":
        out = ep.rms_norm(s["x"], s["w"], residual=s["residual"], eps=EPS, quantize=c["fp8"])
        return ((out.y, out.scale) if c["fp8"] else (out.y,)) + (out.residual, out.rstd)
    if op == "norm_backward":
        return ep.rms_norm_backward(s["dy"], s["x"], s["w"], s["rstd"], dresidual=s["residual"])
    if op == "route":
        return ep.expert_route(s["logits"], c["topk"], bias=s["bias"], score=c["score"], groups=c["groups"], topk_groups=c["topk_groups"],
                               group_top=c["group_top"], renormalize=c["renorm"])
    if op == "route_backward":
        return ep.expert_route_backward(s["dweights"], s["logits"], s["ids"], score=c["score"], renormalize=c["renorm"])
    act = None if c["act"] == "none" else c["act"]
    if op == "linear":
        return ep.matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=dtype, bias=s["bias"], activation=act, residual=s["residual"],
                             save_pre=c["pre"])
    d = ep.epilogue_backward_fp8(s["dout"], activation=act, pre=s["pre"])
    return d.q, d.scale, d.q_t, d.scale_t, d.dbias


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------- 64-bit results
def _e4m3(x):
    """float64 values rounded to the nearest e4m3 value, ties to even, as float64 (|x| <= 464)."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -60))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_quantize(x):
    """(q, scale) of float64 rows, by the definition in 64 bits."""
    m, k = x.shape
    kb = _blocks(k)
    size = torch.nn.functional.pad(x.abs(), (0, kb * B - k))
    amax = size.view(m, kb, B).amax(2).clamp_min(AMAX_MIN)
    return _e4m3(x * (448.0 / amax).repeat_interleave(B, 1)[:, :k]), amax / 448.0


def _f64(q, scale, rows=1):
    s = scale.double()
    if rows > 1:
        s = s.repeat_interleave(rows, 0)[:q.shape[0]]
    return q.double() * s.repeat_interleave(B, 1)[:, :q.shape[1]]


def _phi(v):
    """The normal distribution function, by its complement."""
    return 0.5 * torch.special.erfc(-v / math.sqrt(2.0))


def _exact_route(s):
    """Row by row on the host, by numpy's stable sort of negated keys."""
    import numpy as np

    c = s["case"]
    l = s["logits"].double().cpu().numpy()
    if c["score"] == "sigmoid":
        score = np.reciprocal(1.0 + np.exp(-l))
    else:
        score = np.exp(l - l.max(1, keepdims=True))
        score /= score.sum(1, keepdims=True)
    biased = s["bias"] is not None
    key = score.copy() if biased or c["groups"] > 1 else l
    if biased:
        key += s["bias"].double().cpu().numpy()
    size = c["e"] // c["groups"]
    if c["groups"] > 1:
        best = np.stack([np.sort(key[:, i * size:(i + 1) * size], 1)[:, ::-1][:, :c["group_top"]].sum(1) for i in range(c["groups"])], 1)
        gone = np.argsort(-best, axis=1, kind="stable")[:, c["topk_groups"]:]
        for j in range(gone.shape[1]):
            for i in range(c["groups"]):
                key[gone[:, j] == i, i * size:(i + 1) * size] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :c["topk"]]
    w = np.take_along_axis(score, ids, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(w)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"] if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
        v = x.double()
        rstd = 1 / torch.sqrt((v * v).sum(1) / case["h"] + EPS)
        y = v * rstd[:, None] * s["w"].double()
        return (_exact_quantize(y) if case["fp8"] else (y,)) + (v, rstd)
    if op == "norm_backward":
        x, dy, w, rstd = s["x"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()
        along = ((dy * w) * x).sum(1) / case["h"]
        dx = rstd[:, None] * dy * w - (rstd ** 3 * along)[:, None] * x
        if s["residual"] is not None:
            dx += s["residual"].double()
        return dx, torch.matmul(rstd[None, :], dy * x)[0]
    if op == "route":
        return _exact_route(s)
    if op == "route_backward":
        # through torch's own differentiation of the weights in 64 bits
        l = s["logits"].double().requires_grad_()
        score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        w = torch.gather(score, 1, s["ids"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return torch.autograd.grad(w, l, s["dweights"].double())[0]
    if op == "linear":
        p = _f64(s["a"], s["sa"]) @ _f64(s["b"], s["sb"], B).t()
        if s["bias"] is not None:
            p += s["bias"].double()
        act = case["act"]
        d = p.clamp_min(0) if act == "relu" else p * _phi(p) if act == "gelu" else p * torch.sigmoid(p) if act == "silu" else p
        if s["residual"] is not None:
            d = d + s["residual"].double()
        return (d, p) if case["pre"] else d
    d = s["dout"].double()
    if s["pre"] is not None:
        v, act = s["pre"].double(), case["act"]
        if act == "relu":
            d = torch.where(v > 0, d, 0.0)
        elif act == "gelu":
            d = d * (_phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi))
        else:
            p = torch.sigmoid(v)
            d = d * (p + v * p * torch.sigmoid(-v))
    return _exact_quantize(d) + _exact_quantize(d.t()) + (d.sum(0),)


# --------------------------------------------------------------------------------------- work
def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op in ("norm", "norm_backward"):
        m, h = case["m"], case["h"]
        w = h * (4 if case["wide_weight"] else size)
        if op == "norm":
            out = m * (h + 4 * _blocks(h)) if case["fp8"] else m * h * size
            return {"bytes": m * h * size * (3 if case["residual"] else 1) + out + w + 4 * m, "flops": 6 * m * h}
        return {"bytes": m * h * size * (4 if case["residual"] else 3) + w + 4 * h + 4 * m, "flops": 11 * m * h}
    if op in ("route", "route_backward"):
        t, e, k = case["t"], case["e"], case["topk"]
        if op == "route":
            return {"bytes": t * (e * size + 8 * k) + (4 * e if case["bias"] else 0), "flops": 4 * t * e}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": t * (e * size * (2 if dense else 1) + k * (8 if dense else 8 + size)), "flops": 4 * t * e}
    m, n = case["m"], case["n"]
    if op == "linear":
        k = case["k"]
        outs = 1 + case["residual"] + case["pre"]
        return {"bytes": (m + n) * k + 4 * _blocks(k) * (m + _blocks(n)) + m * n * size * outs + n * size * case["bias"], "flops": 2 * m * n * k}
    reads = 1 if case["act"] == "none" else 2
    return {"bytes": m * n * (size * reads + 2) + 4 * (m * _blocks(n) + n * _blocks(m) + n), "flops": 12 * m * n}

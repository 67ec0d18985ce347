"""Measured cases of the 8-bit block-scaled products and the expert (mixture-of-experts) operators.

listed() names the cases, draw(rng) gives more of the same ranges, prepare(case, seed) makes what a
program has in hand before the call, run(state) is one call, exact(case, seed) the same result in
64 bits and work(case) the bytes and operations a pass cannot do without.  `own` selects between
the operators' plain form (elementary torch operations in fp32, the default) and the library's.

Sizes: hidden size 5120, 2048 to 16384 tokens and the 17408-wide intermediate of the library's
SwiGLU-MLP workload; 64 experts, 8 per token, as a generic sparse layer; single tokens for serving.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
AMAX_MIN = 2.0 ** -90  # the smallest block maximum a scale is made from
B = 128                # scale block


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a training step's activations, quantised along their features for the forward product
        {"name": "quantize_rows_8192x5120", "op": "quantize", "m": 8192, "k": 5120, "dtype": "bf16",
         "rows": 1, "transpose": False},
        # the same activations for the weight gradient: 128 x 128 blocks of the transpose
        {"name": "quantize_blocks_transposed_8192x5120", "op": "quantize", "m": 8192, "k": 5120, "dtype": "bf16",
         "rows": 128, "transpose": True},
        # a down projection for one new token
        {"name": "matmul_1x5120x17408", "op": "matmul", "m": 1, "n": 5120, "k": 17408, "dtype": "bf16"},
        # a ragged batch of prompts against sizes that are no multiples of a tile or a scale block
        {"name": "matmul_777x5003x4112", "op": "matmul", "m": 777, "n": 5003, "k": 4112, "dtype": "fp16"},
        # an up projection of a training step
        {"name": "matmul_8192x17408x5120", "op": "matmul", "m": 8192, "n": 17408, "k": 5120, "dtype": "bf16"},
        # experts' gate and up projections for one new token
        {"name": "grouped_1_token", "op": "grouped", "t": 1, "topk": 8, "e": 64, "n": 4096, "k": 5120,
         "align": 1, "dtype": "bf16"},
        # the same for a prompt or a training step
        {"name": "grouped_4096_tokens", "op": "grouped", "t": 4096, "topk": 8, "e": 64, "n": 4096, "k": 5120,
         "align": 128, "dtype": "bf16"},
        # the experts' weight gradients in a training step
        {"name": "wgrad_4096_tokens", "op": "wgrad", "t": 4096, "topk": 8, "e": 64, "m": 4096, "n": 5120,
         "dtype": "bf16"},
        # one new token routed: order and 8-bit rows
        {"name": "route_1_token_fp8", "op": "route", "t": 1, "topk": 8, "e": 64, "h": 5120, "align": 1,
         "dtype": "bf16", "fp8": True, "dropped": 0.0},
        # a training step's tokens routed; some are padding and go to no expert
        {"name": "route_8192_tokens", "op": "route", "t": 8192, "topk": 8, "e": 64, "h": 5120, "align": 128,
         "dtype": "bf16", "fp8": False, "dropped": 0.03},
        # their rows brought back and weighted
        {"name": "combine_8192_tokens", "op": "combine", "t": 8192, "topk": 8, "e": 64, "h": 5120, "align": 128,
         "dtype": "bf16", "dropped": 0.03},
        # and the gradients of that
        {"name": "combine_backward_8192_tokens", "op": "combine_backward", "t": 8192, "topk": 8, "e": 64, "h": 5120,
         "align": 128, "dtype": "bf16", "dropped": 0.03},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number from lo to hi, even over its logarithm, a multiple of step."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(step, min(hi, v) // step * step)


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "grouped", "grouped", "wgrad", "route", "combine",
                     "combine_backward"])
    half = rng.choice(["bf16", "bf16", "fp16"])
    if op == "quantize":
        rows = rng.choice([1, 128])
        return {"op": op, "m": _log(rng, 1, 8192), "k": _log(rng, 16, 5120), "rows": rows,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "transpose": rng.random() < 0.4}
    if op == "matmul":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 16384), "k": _log(rng, 128, 5120, 16),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    e = rng.choice([8, 16, 32, 60, 64])
    topk = rng.choice([1, 2, 4, 6, 8])
    if op == "grouped":
        return {"op": op, "t": _log(rng, 1, 4096), "topk": topk, "e": e, "n": _log(rng, 256, 4096),
                "k": _log(rng, 256, 5120, 16), "align": rng.choice([1, 128]), "dtype": half}
    if op == "wgrad":
        return {"op": op, "t": _log(rng, 16, 4096), "topk": topk, "e": e, "m": _log(rng, 256, 4096),
                "n": _log(rng, 256, 5120), "dtype": rng.choice(["bf16", "fp32"])}
    c = {"op": op, "t": _log(rng, 1, 8192), "topk": topk, "e": e, "h": _log(rng, 64, 5120),
         "align": rng.choice([1, 128]), "dtype": rng.choice(["bf16", "fp16", "fp32"] if op != "route" else ["bf16", "fp16"]),
         "dropped": rng.choice([0.0, 0.1])}
    if op == "route":
        c["fp8"] = rng.random() < 0.5
        if c["fp8"]:
            c["h"] = max(64, c["h"] // 16 * 16)
    return c


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


def _row_scales(m, k, g):
    """One scale for each row and 128 features, features outermost in memory."""
    return _scales((_blocks(k), m), g, 0.01).t()


def _expert_ids(case, g):
    """topk different experts for each token, some experts more popular than others."""
    t, e, k = case["t"], case["e"], case["topk"]
    score = torch.rand((t, e), generator=g, device="cuda") + 0.3 * torch.rand((1, e), generator=g, device="cuda")
    ids = score.topk(k, dim=1).indices.to(torch.int32)
    gone = torch.rand((t, 1), generator=g, device="cuda") < case.get("dropped", 0.0)
    return ids.masked_fill(gone, -1)


def _capacity(t, topk, e, align):
    """Rows the sorted tokens take at most: each group padded to a multiple of align."""
    rows = t * topk
    return rows if align == 1 else -(-(rows + min(e, rows) * (align - 1)) // align) * align


def _order(ids, e, align):
    """pos [T, k]: the row of each (token, choice) in expert order, -1 for a dropped one;
    src [capacity]: the flat (token, choice) of each row, -1 for padding; offsets [E + 1]."""
    t, topk = ids.shape
    flat = ids.reshape(-1).long()
    slot = torch.arange(flat.numel(), device=flat.device)
    kept = (flat >= 0) & (flat < e)
    key = torch.where(kept, flat, e)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=flat.device).index_add_(0, key, torch.ones_like(key))
    padded = (counts[:e] + align - 1) // align * align
    ends = padded.cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    by_expert = key.sort(stable=True).indices
    before = counts.cumsum(0) - counts  # kept rows of the experts before, without padding
    skey = key[by_expert]
    row = torch.where(skey < e, slot - before[skey] + offsets[skey], -1)
    pos = torch.empty_like(flat)
    pos[by_expert] = row
    cap = _capacity(t, topk, e, align)
    src = torch.full((cap + 1,), -1, dtype=torch.int64, device=flat.device)
    src[torch.where(row < 0, cap, row)] = torch.where(row < 0, -1, by_expert)
    return pos.view(t, topk).int(), src[:cap].int(), offsets.int()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    dtype = DT[case["dtype"]]
    if op == "quantize":
        s["x"] = _values((case["m"], case["k"]), g, dtype)
    elif op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        s.update(a=_operand((m, k), g), sa=_row_scales(m, k, g), b=_operand((n, k), g),
                 sb=_scales((_blocks(n), _blocks(k)), g, 1e-4))
    elif op == "grouped":
        e, n, k = case["e"], case["n"], case["k"]
        _, src, offsets = _order(_expert_ids(case, g), e, case["align"])
        rows = src.numel()
        pad = (src < 0)[:, None]
        a = _operand((rows, k), g).view(torch.uint8).masked_fill_(pad, 0).view(F8)
        s.update(a=a, sa=_row_scales(rows, k, g), offsets=offsets, b=_operand((e, n, k), g),
                 sb=_scales((e, _blocks(n), _blocks(k)), g, 1e-4), cap=int((offsets[1:] - offsets[:-1]).max()))
    elif op == "wgrad":
        e, m, n = case["e"], case["m"], case["n"]
        _, src, offsets = _order(_expert_ids(case, g), e, B)
        rows = src.numel()
        pad = (src < 0)[None, :]
        a = _operand((m, rows), g).view(torch.uint8).masked_fill_(pad, 0).view(F8)
        b = _operand((n, rows), g).view(torch.uint8).masked_fill_(pad, 0).view(F8)
        s.update(a=a, sa=_row_scales(m, rows, g), offsets=offsets, b=b, sb=_scales((_blocks(n), _blocks(rows)), g, 1e-2),
                 cap=int((offsets[1:] - offsets[:-1]).max()))
    else:
        ids = _expert_ids(case, g)
        t, h = case["t"], case["h"]
        if op == "route":
            s.update(ids=ids, x=_values((t, h), g, dtype))
        else:
            pos, src, offsets = _order(ids, case["e"], case["align"])
            w = torch.rand((t, case["topk"]), generator=g, device="cuda")
            s.update(pos=pos, src=src, offsets=offsets, w=w / w.sum(1, keepdim=True),
                     y=_values((src.numel(), h), g, dtype))
            if op == "combine_backward":
                s["dout"] = _values((t, h), g, dtype)
    return s


# -------------------------------------------------------------------------------- plain forms
def _pad_to(x, rows, cols):
    """x with zeros up to the given last two sizes."""
    return torch.nn.functional.pad(x, (0, cols - x.shape[-1], 0, rows - x.shape[-2]))


def _quantize(x, rows):
    """e4m3 values and scales of x's blocks of rows x 128; the last ones may be partly filled."""
    m, k = x.shape
    mb, kb = -(-m // rows), _blocks(k)
    v = _pad_to(x.float(), mb * rows, kb * B).view(mb, rows, kb, B)
    finite = v.isfinite()
    amax = torch.where(finite, v.abs(), 0.0).amax((1, 3), keepdim=True).clamp_min(AMAX_MIN)
    top = torch.full_like(amax, F8_MAX)  # (divided as tensors: with a number, torch multiplies by a reciprocal)
    q = torch.where(finite, v * (top / amax), float("nan")).to(F8)
    return q.view(mb * rows, kb * B)[:m, :k], (amax / top).view(mb, kb)


def _rows_fp32(q, scale):
    """The values that e4m3 rows and their scales of 128 features stand for."""
    return q.float() * scale.repeat_interleave(B, -1)[..., :q.shape[-1]]


def _blocks_fp32(q, scale):
    """The same for scales of 128 x 128."""
    return _rows_fp32(q, scale.repeat_interleave(B, -2)[..., :q.shape[-2], :])


def _segments(offsets, cap, rows):
    """[E, cap]: the rows of each group, `rows` past its end."""
    i = offsets[:-1, None].long() + torch.arange(cap, device=offsets.device)
    return torch.where(i < offsets[1:, None], i, rows)


def _plain(s):
    c = s["case"]
    op = c["op"]
    dtype = DT[c["dtype"]]
    if op == "quantize":
        return _quantize(s["x"].t() if c["transpose"] else s["x"], c["rows"])
    if op == "matmul":
        return (_rows_fp32(s["a"], s["sa"]) @ _blocks_fp32(s["b"], s["sb"]).t()).to(dtype)
    if op == "grouped":
        rows = s["a"].shape[0]
        seg = _segments(s["offsets"], s["cap"], rows)
        a = _pad_to(_rows_fp32(s["a"], s["sa"]), rows + 1, c["k"])[seg]
        d = torch.bmm(a, _blocks_fp32(s["b"], s["sb"]).transpose(1, 2))
        out = d.new_zeros((rows + 1, c["n"]))
        out[seg] = d
        out[rows] = 0
        return out[:rows].to(dtype)
    if op == "wgrad":
        rows = s["a"].shape[1]
        seg = _segments(s["offsets"], s["cap"], rows)
        a = _pad_to(_rows_fp32(s["a"], s["sa"]), c["m"], rows + 1)[:, seg].transpose(0, 1)
        b = _pad_to(_blocks_fp32(s["b"], s["sb"]), c["n"], rows + 1)[:, seg].permute(1, 2, 0)
        return torch.bmm(a, b).to(dtype)
    if op == "route":
        pos, src, offsets = _order(s["ids"], c["e"], c["align"])
        x = s["x"]
        pad = (src < 0)[:, None]
        token = src.clamp_min(0).long() // c["topk"]
        if c["fp8"]:
            q, scale = _quantize(x, 1)
            q = q.view(torch.uint8)[token].masked_fill(pad, 0).view(F8)
            return pos, src, offsets, q, scale[token].masked_fill(pad, AMAX_MIN / F8_MAX)
        return pos, src, offsets, x[token].masked_fill(pad, 0)
    kept = (s["pos"] >= 0)[..., None]
    row = s["pos"].clamp_min(0).long()
    w = s["w"][..., None]
    if op == "combine":
        return torch.where(kept, s["y"][row].float() * w, 0.0).sum(1).to(dtype)
    dout = s["dout"].float()[:, None]
    dw = torch.where(kept, s["y"][row].float() * dout, 0.0).sum(2)
    rows = s["y"].shape[0]
    dy = torch.zeros((rows + 1, c["h"]), device="cuda")
    dy[torch.where(kept[..., 0], row, rows)] = w * dout
    return dy[:rows].to(dtype), dw


# ------------------------------------------------------------------------------ library calls
def _own(s):
    import dense_gemm_epilogues_amd as ep

    c = s["case"]
    op = c["op"]
    dtype = DT[c["dtype"]]
    if op == "quantize":
        return ep.quantize_fp8(s["x"], block=(c["rows"], B), transpose=c["transpose"])
    if op == "matmul":
        return ep.matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=dtype)
    if op == "grouped":
        return ep.grouped_matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], out_dtype=dtype)
    if op == "wgrad":
        return ep.grouped_wgrad_fp8(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], out_dtype=dtype)
    if op == "route":
        order = ep.expert_order(s["ids"], c["e"], align=c["align"])
        rows = ep.expert_dispatch(s["x"], order, quantize=c["fp8"])
        return (order.pos, order.src, order.offsets) + (rows if c["fp8"] else (rows,))
    order = ep.ExpertOrder(s["pos"], s["src"], s["offsets"])
    if op == "combine":
        return ep.expert_combine(s["y"], order, s["w"])
    return ep.expert_combine_backward(s["dout"], s["y"], order, s["w"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------- 64-bit results
def _e4m3(x):
    """float64 values rounded to the nearest e4m3 value, ties to even, as float64 (|x| <= 464)."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -60))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_quantize(x, rows):
    """By the definition: both the reciprocal of a block's scale and its product with a value
    are rounded to fp32 before the value is rounded to e4m3."""
    m, k = x.shape
    kb, mb = _blocks(k), -(-m // rows)
    size = torch.where(x.isfinite(), x.double().abs(), 0.0)
    size = torch.nn.functional.pad(size, (0, kb * B - k, 0, mb * rows - m))
    amax = size.view(mb, rows, kb, B).amax(3).amax(1).clamp_min(AMAX_MIN)
    inv = (448.0 / amax).float().double().repeat_interleave(B, 1)[:, :k].repeat_interleave(rows, 0)[:m]
    q = _e4m3((x.double() * inv).float().double())
    return torch.where(x.isfinite(), q, float("nan")), amax / 448.0


def _f64(q, scale, rows=1):
    s = scale.double()
    if rows > 1:
        s = s.repeat_interleave(rows, 0)[:q.shape[0]]
    return q.double() * s.repeat_interleave(B, 1)[:, :q.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s["x"].t() if case["transpose"] else s["x"], case["rows"])
    if op == "matmul":
        return _f64(s["a"], s["sa"]) @ _f64(s["b"], s["sb"], B).t()
    if op in ("grouped", "wgrad"):
        ends = s["offsets"].tolist()
        if op == "grouped":
            out = torch.zeros((s["a"].shape[0], case["n"]), dtype=torch.float64, device="cuda")
            a = _f64(s["a"], s["sa"])
            for i in range(case["e"]):
                out[ends[i]:ends[i + 1]] = a[ends[i]:ends[i + 1]] @ _f64(s["b"][i], s["sb"][i], B).t()
            return out
        a, b = _f64(s["a"], s["sa"]), _f64(s["b"], s["sb"], B)
        return torch.stack([a[:, ends[i]:ends[i + 1]] @ b[:, ends[i]:ends[i + 1]].t() for i in range(case["e"])])
    if op == "route":
        ids = s["ids"].reshape(-1).tolist()
        topk, e, align = case["topk"], case["e"], case["align"]
        lists = [[] for _ in range(e)]
        for i, x in enumerate(ids):
            if 0 <= x < e:
                lists[x].append(i)
        pos, src, offsets = [-1] * len(ids), [], [0]
        for one in lists:
            for i in one:
                pos[i] = len(src)
                src.append(i)
            src += [-1] * (-len(src) % align)
            offsets.append(len(src))
        src += [-1] * (_capacity(case["t"], topk, e, align) - len(src))
        pos = torch.tensor(pos, dtype=torch.int32).view(case["t"], topk)
        token = torch.tensor(src, device="cuda")
        pad, token = (token < 0)[:, None], token.clamp_min(0) // topk
        whole = (pos, torch.tensor(src, dtype=torch.int32), torch.tensor(offsets, dtype=torch.int32))
        if case["fp8"]:
            q, scale = _exact_quantize(s["x"], 1)
            return whole + (q[token].masked_fill(pad, 0), scale[token].masked_fill(pad, AMAX_MIN / 448.0))
        return whole + (s["x"].double()[token].masked_fill(pad, 0),)
    t, h, topk = case["t"], case["h"], case["topk"]
    pos, w, y = s["pos"].long(), s["w"].double(), s["y"]
    if op == "combine":
        out = torch.zeros((t, h), dtype=torch.float64, device="cuda")
        for j in range(topk):
            on = pos[:, j] >= 0
            out[on] += w[on, j, None] * y[pos[on, j]].double()
        return out
    dout = s["dout"].double()
    dy = torch.zeros(y.shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros((t, topk), dtype=torch.float64, device="cuda")
    for j in range(topk):
        on = pos[:, j] >= 0
        dy[pos[on, j]] = w[on, j, None] * dout[on]
        dw[on, j] = (y[pos[on, j]].double() * dout[on]).sum(1)
    return dy, dw


# --------------------------------------------------------------------------------------- work
def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op == "quantize":
        m, k, r = case["m"], case["k"], case["rows"]
        if case["transpose"]:
            m, k = k, m
        return {"bytes": m * k * (size + 1) + 4 * -(-m // r) * _blocks(k), "flops": 3 * m * k}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k + 4 * _blocks(k) * (m + _blocks(n)) + m * n * size, "flops": 2 * m * n * k}
    t, topk, e = case["t"], case["topk"], case["e"]
    slots = t * topk
    if op == "grouped":
        n, k = case["n"], case["k"]
        used = min(e, slots) if slots <= e else e  # experts that rows go to, about
        return {"bytes": slots * (k + 4 * _blocks(k) + n * size) + used * (n * k + 4 * _blocks(n) * _blocks(k)),
                "flops": 2 * slots * n * k}
    if op == "wgrad":
        m, n = case["m"], case["n"]
        return {"bytes": slots * (m + n) + 4 * _blocks(slots) * (m + _blocks(n)) + e * m * n * size,
                "flops": 2 * slots * m * n}
    h = case["h"]
    kept = slots * (1 - case["dropped"])
    if op == "route":
        out = h + 4 * _blocks(h) if case["fp8"] else h * size
        return {"bytes": t * h * size + 12 * slots + kept * out, "flops": 3 * t * h}
    if op == "combine":
        return {"bytes": kept * h * size + t * h * size + 8 * slots, "flops": 2 * kept * h}
    return {"bytes": 2 * kept * h * size + t * h * size + 12 * slots, "flops": 3 * kept * h}

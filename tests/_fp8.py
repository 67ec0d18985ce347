"""Plain 64-bit forms of the 8-bit block-scaled products and the expert operators, on the CPU."""
import torch

F8 = torch.float8_e4m3fn
AMAX_MIN = 2.0 ** -90
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SMALLEST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # half the subnormal step


def blocks(n):
    return -(-n // 128)


def quantize(x, rows, transpose):
    """q (as float32 values) and scale by the definition: quotients and products rounded to fp32."""
    v = (x.t() if transpose else x).float().contiguous()
    m, k = v.shape
    q = torch.empty_like(v)
    scale = torch.empty((-(-m // rows), blocks(k)))
    for i in range(scale.shape[0]):
        for c in range(scale.shape[1]):
            at = (slice(i * rows, (i + 1) * rows), slice(c * 128, (c + 1) * 128))
            b = v[at]
            fin = b.isfinite()
            amax = torch.where(fin, b.abs(), torch.zeros(())).max().clamp_min(AMAX_MIN)
            top = torch.tensor(448.0)
            q[at] = torch.where(fin, b * (top / amax), torch.tensor(float("nan"))).to(F8).float()
            scale[i, c] = amax / top
    return q, scale


def dequantized(q, scale, rows=1):
    s = scale.double().repeat_interleave(rows, -2)[..., :q.shape[-2], :]
    return q.double() * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def product(a, sa, b, sb):
    """(exact D, sum of the products' magnitudes) of a (M x K) and b (N x K), CPU e4m3."""
    x, y = dequantized(a, sa), dequantized(b, sb, 128)
    return x @ y.t(), x.abs() @ y.abs().t()


def product_tolerance(exact, mags, k, dtype):
    """How far a product may be off: fp32 sums of 128 exact products (an ulp, 2^-23, for each of their
    additions, whatever their order), two roundings for the factor, one multiply-add a block, a few more to
    join K ranges, all relative to the sum of magnitudes; then half a step of the output type."""
    gamma = (128 + 2 + 2 * blocks(k) + 16) * 2.0 ** -23
    return gamma * mags + HALF_STEP[dtype] * (exact.abs() + gamma * mags) + SMALLEST[dtype]


def assert_within(got, exact, tol, what=""):
    got = got.double().cpu()
    bad = (got - exact).abs() > tol
    assert got.shape == exact.shape, f"{what}: shape {tuple(got.shape)}, want {tuple(exact.shape)}"
    assert not bad.any() and not got.isnan().any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - exact).abs() / tol).nan_to_num(1e30).max()):.3g} tolerances")


def operand(g, *shape):
    return (torch.randn(shape, generator=g) * 120).clamp(-448, 448).to(F8)


def scales(g, *shape):
    return (torch.rand(shape, generator=g) + 0.5) * 2.0 ** -8


def order(ids, experts, align):
    """(pos, src, offsets) as lists of whole numbers."""
    slots = ids.reshape(-1).tolist()
    lists = [[] for _ in range(experts)]
    for i, e in enumerate(slots):
        if 0 <= e < experts:
            lists[e].append(i)
    pos, src, offsets = [-1] * len(slots), [], [0]
    for one in lists:
        for i in one:
            pos[i] = len(src)
            src.append(i)
        src += [-1] * (-len(src) % align)
        offsets.append(len(src))
    padded = len(slots) + min(experts, len(slots)) * (align - 1)
    src += [-1] * (-(-padded // align) * align - len(src))
    return torch.tensor(pos, dtype=torch.int32).view(ids.shape), torch.tensor(src, dtype=torch.int32), torch.tensor(offsets, dtype=torch.int32)

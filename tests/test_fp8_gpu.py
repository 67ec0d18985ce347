"""8-bit block-scaled products on the GPU against plain 64-bit forms: values bit for bit where the
definition fixes every rounding (quantisation), within derived bounds elsewhere."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 16), (3, 130), (9, 640), (129, 127), (200, 391), (256, 512)])
def test_quantize(dtype, rows, transpose, m, k):
    g = gen(m * 1000 + k)
    x = torch.randn((m, k), generator=g) * torch.exp2(torch.randint(-6, 7, (m, k), generator=g).float())
    x = x.to(dtype)
    q, s = ep.quantize_fp8(x.cuda(), block=(rows, 128), transpose=transpose)
    wq, ws = R.quantize(x, rows, transpose)
    assert q.dtype == R.F8 and s.dtype == torch.float32
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.float().cpu(), wq)
    if rows == 1:
        assert s.stride() == (1, s.shape[0]) or 1 in s.shape


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quantize_special_values(dtype, rows, transpose):
    """Zeros, infinities, NaN, subnormals and the type's largest values; rows of a wider buffer."""
    wide = torch.randn((140, 300), generator=gen(5)).to(dtype)
    x = wide[:, 3:260]
    x[0] = 0
    x[1, 5], x[1, 6], x[1, 140] = float("inf"), float("-inf"), float("nan")
    x[2] = float("nan")
    x[3] = torch.finfo(dtype).tiny / 4
    x[4, 7], x[4, 200] = torch.finfo(dtype).max, -torch.finfo(dtype).max
    x[5] = float("-inf")
    dev = wide.cuda()[:, 3:260]
    q, s = ep.quantize_fp8(dev, block=(rows, 128), transpose=transpose)
    wq, ws = R.quantize(x, rows, transpose)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.float().cpu().isnan(), wq.isnan())
    assert torch.equal(q.float().cpu().nan_to_num(0), wq.nan_to_num(0))


def test_quantize_empty():
    q, s = ep.quantize_fp8(torch.empty((0, 256), device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    q, s = ep.quantize_fp8(torch.empty((5, 0), device="cuda"), block=(128, 128), transpose=True)
    assert q.shape == (0, 5) and s.shape == (0, 1)


# ------------------------------------------------------------------------------------ plain product
SHAPES = [(1, 5, 16), (1, 64, 128), (1, 1000, 1424), (16, 130, 272), (17, 33, 400), (32, 48, 8208), (33, 257, 144),
          (64, 100, 4096), (130, 300, 1040), (257, 513, 2064), (300, 1000, 128), (513, 129, 5008)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul(dtype, m, n, k):
    g = gen(m + n + k)
    a, b = R.operand(g, m, k), R.operand(g, n, k)
    sa, sb = R.scales(g, m, R.blocks(k)), R.scales(g, R.blocks(n), R.blocks(k))
    d = ep.matmul_fp8(a.cuda(), sa.t().contiguous().cuda().t(), b.cuda(), sb.cuda(), out_dtype=dtype)
    exact, mags = R.product(a, sa, b, sb)
    assert d.dtype == dtype
    R.assert_within(d, exact, R.product_tolerance(exact, mags, k, dtype), f"{m} x {n} x {k}")


@pytest.mark.parametrize("m", [3, 200])
def test_matmul_strides(m):
    """Operands, scales and output as parts of larger buffers; row-major scales; what lies around the
    output stays."""
    g, n, k = gen(7), 150, 400
    a, b = R.operand(g, m, 528).cuda()[:, 64:64 + k], R.operand(g, n + 4, 432).cuda()[4:, 32:]
    sa, sb = R.scales(g, m, 9).cuda()[:, 2:6], R.scales(g, 4, 2).cuda().t()
    buf = torch.full((m, n + 11), 7.0, dtype=torch.bfloat16, device="cuda")
    d = ep.matmul_fp8(a, sa, b, sb, out=buf[:, 5:5 + n])
    exact, mags = R.product(a.cpu(), sa.cpu(), b.cpu(), sb.cpu())
    R.assert_within(d, exact, R.product_tolerance(exact, mags, k, torch.bfloat16))
    assert (buf[:, :5] == 7).all() and (buf[:, 5 + n:] == 7).all()


@pytest.mark.parametrize("m", [2, 100])
def test_matmul_nan_stays_in_its_row(m):
    g, n, k = gen(8), 70, 144
    a, b = R.operand(g, m, k), R.operand(g, n, k)
    a.view(torch.uint8)[1, 143] = 0x7f
    sa, sb = R.scales(g, m, 2), R.scales(g, 1, 2)
    d = ep.matmul_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda()).cpu()
    assert d[1].isnan().all() and not d[torch.arange(m) != 1].isnan().any()


def test_matmul_empty():
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    f = lambda *s: z(*s).to(R.F8)  # noqa: E731
    assert ep.matmul_fp8(f(0, 32), z(0, 1), f(8, 32), z(1, 1)).shape == (0, 8)
    d = ep.matmul_fp8(f(4, 0), z(4, 0), f(8, 0), z(1, 0))
    assert d.shape == (4, 8) and not d.any()


# ---------------------------------------------------------------------------------- grouped products
def offsets_of(counts, align=1):
    padded = [-(-c // align) * align for c in counts]
    return torch.tensor([0] + torch.tensor(padded).cumsum(0).tolist(), dtype=torch.int32)


GROUPS = [([1], 1, 0), ([0, 1, 0, 3, 0], 1, 2), ([5, 0, 40, 1], 1, 0), ([200, 0, 1, 300, 17], 1, 30),
          ([128, 0, 256, 384], 128, 128), ([600, 1], 1, 0), ([1] * 70, 1, 5), ([3, 0] * 40 + [700], 1, 0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(130, 272), (300, 1040)])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped(dtype, n, k, case):
    counts, align, tail = GROUPS[case]
    g = gen(case)
    off = offsets_of(counts, align)
    rows, e = int(off[-1]) + tail, len(counts)
    a, b = R.operand(g, rows, k), R.operand(g, e, n, k)
    sa, sb = R.scales(g, rows, R.blocks(k)), R.scales(g, e, R.blocks(n), R.blocks(k))
    d = ep.grouped_matmul_fp8(a.cuda(), sa.t().contiguous().cuda().t(), b.cuda(), sb.cuda(), off.cuda(), out_dtype=dtype)
    for i in range(e):
        at = slice(int(off[i]), int(off[i + 1]))
        exact, mags = R.product(a[at], sa[at], b[i], sb[i])
        R.assert_within(d[at], exact, R.product_tolerance(exact, mags, k, dtype), f"expert {i}")
    assert not d[int(off[-1]):].any()


def test_grouped_strides():
    """Experts' matrices, scales and outputs as parts of larger buffers."""
    g, n, k, e = gen(9), 70, 160, 3
    off = offsets_of([40, 3, 60])
    for rows in (103, 110):
        a = R.operand(g, rows, 256).cuda()[:, 48:48 + k]
        b = R.operand(g, e, n + 2, 208).cuda()[:, 1:1 + n, 16:16 + k]
        sa, sb = R.scales(g, rows, 5).cuda()[:, 1:3], R.scales(g, 2, 1, e).cuda().permute(2, 1, 0)
        buf = torch.full((rows, n + 3), 7.0, dtype=torch.float32, device="cuda")
        d = ep.grouped_matmul_fp8(a, sa, b, sb, off.cuda(), out_dtype=torch.float32, out=buf[:, 2:2 + n])
        for i in range(e):
            at = slice(int(off[i]), int(off[i + 1]))
            exact, mags = R.product(a[at].cpu(), sa[at].cpu(), b[i].cpu(), sb[i].cpu())
            R.assert_within(d[at], exact, R.product_tolerance(exact, mags, k, torch.float32), f"expert {i}")
        assert not d[103:].any() and (buf[:, :2] == 7).all() and (buf[:, 2 + n:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n", [(40, 50), (130, 272), (300, 521)])
@pytest.mark.parametrize("counts,extra", [([128], 0), ([0, 256, 0, 128, 640, 0], 0), ([128, 384], 128)])
def test_wgrad(dtype, m, n, counts, extra):
    g = gen(m + n)
    off = offsets_of(counts, 128)
    rows, e = int(off[-1]) + extra, len(counts)
    a, b = R.operand(g, m, rows), R.operand(g, n, rows)
    sa, sb = R.scales(g, m, R.blocks(rows)), R.scales(g, R.blocks(n), R.blocks(rows))
    d = ep.grouped_wgrad_fp8(a.cuda(), sa.t().contiguous().cuda().t(), b.cuda(), sb.cuda(), off.cuda(), out_dtype=dtype)
    assert d.shape == (e, m, n)
    x, y = R.dequantized(a, sa), R.dequantized(b, sb, 128)
    for i in range(e):
        at = slice(int(off[i]), int(off[i + 1]))
        exact, mags = x[:, at] @ y[:, at].t(), x[:, at].abs() @ y[:, at].abs().t()
        R.assert_within(d[i], exact, R.product_tolerance(exact, mags, counts[i], dtype), f"expert {i}")


def test_wgrad_group_off_the_blocks_is_nan():
    """A group that does not start and end on scale blocks has no defined scales: its gradient is NaN, the
    others' are whole."""
    g, m, n = gen(3), 48, 80
    a, b = R.operand(g, m, 512), R.operand(g, n, 512)
    sa, sb = R.scales(g, m, 4), R.scales(g, 1, 4)
    off = torch.tensor([0, 128, 200, 256, 512], dtype=torch.int32)
    d = ep.grouped_wgrad_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), off.cuda(), out_dtype=torch.float32).cpu()
    assert d[1].isnan().all() and d[2].isnan().all()
    x, y = R.dequantized(a, sa), R.dequantized(b, sb, 128)
    for i, at in ((0, slice(0, 128)), (3, slice(256, 512))):
        exact, mags = x[:, at] @ y[:, at].t(), x[:, at].abs() @ y[:, at].abs().t()
        R.assert_within(d[i], exact, R.product_tolerance(exact, mags, 256, torch.float32))


@pytest.mark.parametrize("off", [[0, 500, 90, 2000000000, 96], [-5, 3, -2147483648, 7, 96], [0, 0, 0, 0, 0], [96] * 5])
@pytest.mark.parametrize("rows,e", [(96, 4), (40, 4)])
def test_grouped_offsets_outside_the_rows_stay_inside_the_buffers(off, rows, e):
    """Offsets that do not ascend or pass the rows give some values; nothing outside the output is written."""
    g = gen(4)
    for n, pad in ((48, 3), (300, 5)):
        a, b = R.operand(g, rows, 128).cuda(), R.operand(g, e, n, 128).cuda()
        buf = torch.full((rows + 2 * pad, n), 7.0, dtype=torch.bfloat16, device="cuda")
        ep.grouped_matmul_fp8(a, R.scales(g, rows, 1).cuda(), b, R.scales(g, e, R.blocks(n), 1).cuda(),
                              torch.tensor(off, dtype=torch.int32, device="cuda"), out=buf[pad:pad + rows])
        assert (buf[:pad] == 7).all() and (buf[pad + rows:] == 7).all()


# ------------------------------------------------------------------------------- streams, graphs, size
def test_side_stream_and_graph():
    """On a side stream, and captured: every replay equals the eager result for the inputs of that time."""
    g, m, n, k, e = gen(11), 200, 300, 1040, 4
    x = torch.randn((m, k), generator=g).bfloat16().cuda()
    w = torch.randn((e, n, k), generator=g).bfloat16().cuda()
    wq, ws = ep.quantize_fp8(w.view(e * n, k), block=(1, 128))
    wq = wq.view(e, n, k)
    ws = R.scales(g, e, R.blocks(n), R.blocks(k)).cuda()
    off = offsets_of([50, 0, 120, 30]).cuda()

    def step(x):
        q, s = ep.quantize_fp8(x)
        return ep.matmul_fp8(q, s, wq[0], ws[0]), ep.grouped_matmul_fp8(q, s, wq, ws, off), ep.quantize_fp8(x, transpose=True)[0]

    want = step(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s = ep.quantize_fp8(x, stream=side)
    d = ep.matmul_fp8(q, s, wq[0], ws[0], stream=side)
    side.synchronize()
    assert torch.equal(d, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    for r in range(4):
        x.copy_(torch.randn((m, k), generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(x)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {r}"


def test_products_past_2_31_output_elements():
    """Outputs whose element offsets pass 32 bits: the last rows are right."""
    g, n, k = gen(12), 16384, 32
    m = (1 << 31) // n + 300
    b, sb = R.operand(g, n, k), R.scales(g, R.blocks(n), 1)
    tail = R.operand(g, 64, k)
    a = torch.zeros((m, k), dtype=R.F8, device="cuda")
    a[-64:] = tail.cuda()
    sa = torch.full((1, m), 0.5, device="cuda").t()
    exact, mags = R.product(tail, torch.full((64, 1), 0.5), b, sb)
    tol = R.product_tolerance(exact, mags, k, torch.bfloat16)
    d = ep.matmul_fp8(a, sa, b.cuda(), sb.cuda())
    R.assert_within(d[-64:], exact, tol, "matmul")
    assert not d[-200:-64].any()
    del d
    d = ep.grouped_matmul_fp8(a, sa, b.cuda()[None], sb.cuda()[None], torch.tensor([0, m], dtype=torch.int32, device="cuda"))
    R.assert_within(d[-64:], exact, tol, "grouped")

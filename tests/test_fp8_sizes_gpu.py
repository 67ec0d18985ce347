"""Outputs and inputs of more than 2^31 elements through the kernels that large products and quantisations take:
the last ones are right, on operands whose sums are exact in every step."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
K = 272  # (past the short sums, which have a kernel of their own)


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of device memory")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def whole(g, *shape):
    return torch.randint(-2, 3, shape, generator=g, device="cuda").float().to(R.F8)


def powers(g, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())


def rows_and_matrix():
    """Operands of (2^31 / 16384 + 300) x 16384 outputs; all rows but the last 500 and the first are zeros."""
    g, n = gen(1), 16384
    m = (1 << 31) // n + 300
    a = torch.zeros((m, K), dtype=R.F8, device="cuda")
    a[-500:], a[0] = whole(g, 500, K), whole(g, K)
    sa, b, sb = torch.full((R.blocks(K), m), 0.5, device="cuda").t(), whole(g, n, K), powers(g, R.blocks(n), R.blocks(K))
    return a, sa, b, sb


def check(d, a, sa, b, sb):
    at = torch.cat([torch.zeros(1, dtype=torch.long), torch.arange(d.shape[0] - 500, d.shape[0])])
    want = R.dequantized(a[at], sa[at]) @ R.dequantized(b, sb, 128).t()
    assert torch.equal(d[at], want.to(d.dtype))
    assert not d[1:-500].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_matmul(dtype):
    a, sa, b, sb = rows_and_matrix()
    check(ep.matmul_fp8(a, sa, b, sb, out_dtype=dtype), a, sa, b, sb)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("experts", [1, 1500])
def test_grouped(experts, dtype):
    """One expert's rows in large tiles; 1500 groups, of one matrix, in small ones."""
    a, sa, b, sb = rows_and_matrix()
    off = torch.arange(experts + 1, device="cuda") * a.shape[0] // experts
    d = ep.grouped_matmul_fp8(a, sa, b.expand(experts, -1, -1), sb.expand(experts, -1, -1), off.int(), out_dtype=dtype)
    check(d, a, sa, b, sb)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradients(dtype):
    g, e, m, n = gen(2), 131, 4096, 4100
    assert (e - 1) * m * n > 1 << 31
    rows = e * 128
    a, b, sa, sb = whole(g, m, rows), whole(g, n, rows), powers(g, m, e), powers(g, R.blocks(n), e)
    d = ep.grouped_wgrad_fp8(a, sa, b, sb, torch.arange(e + 1, dtype=torch.int32, device="cuda") * 128, out_dtype=dtype)
    for i in (0, 1, e // 2, e - 2, e - 1):
        at = slice(i * 128, i * 128 + 128)
        want = R.dequantized(a[:, at], sa[:, i:i + 1]) @ R.dequantized(b[:, at], sb[:, i:i + 1], 128).t()
        assert torch.equal(d[i], want.to(dtype)), f"expert {i}"


@pytest.mark.parametrize("rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quantize(rows, transpose):
    m, k = (1 << 21) + 9, 1040
    last = 128 + m % 128
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 31
    tail = torch.randn((last, k), generator=gen(3), device="cuda").bfloat16()
    x[-last:] = tail
    q, s = ep.quantize_fp8(x, block=(rows, 128), transpose=transpose)
    wq, ws = R.quantize(tail.cpu(), rows, transpose)
    if transpose:
        q, s = q.t(), s.t()
        wq, ws = wq.t(), ws.t()
    assert torch.equal(q[-last:].float().cpu(), wq) and torch.equal(s[-ws.shape[0]:].cpu(), ws)
    rest = q.view(torch.uint8).t()[:, :-last] if transpose else q.view(torch.uint8)[:-last]
    assert not rest.any()

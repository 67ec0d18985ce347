"""8-bit products whose operands and scales lie in buffers full of NaN: nothing around them reaches a result, in any
kernel; and a NaN among an operand's values reaches its row or column alone.  Operands are exact in every step."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
# few rows; 128 x 128 tiles; K ranges; 256 x 256 tiles; short sums
SHAPES = [(5, 130, 400), (100, 300, 400), (64, 256, 5136), (4400, 4300, 400), (100, 300, 240)]
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def whole(g, *shape):
    """Small whole numbers as a view of a wider e4m3 buffer of NaN: 16 columns and 2 rows on every side."""
    buf = torch.full((*shape[:-2], shape[-2] + 4, shape[-1] + 32), 0x7f, dtype=torch.uint8, device="cuda").view(R.F8)
    view = buf[..., 2:-2, 16:-16]
    view.view(torch.uint8).copy_(torch.randint(-2, 3, shape, generator=g, device="cuda").float().to(R.F8).view(torch.uint8))
    return view


def powers(g, *shape):
    buf = torch.full((*shape[:-2], shape[-2] + 2, shape[-1] + 2), float("nan"), device="cuda")
    view = buf[..., 1:-1, 1:-1]
    view.copy_(torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float()))
    return view


def exact(a, sa, b, sb):
    return R.dequantized(a.contiguous(), sa) @ R.dequantized(b.contiguous(), sb, 128).t()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul(m, n, k, dtype):
    g = gen(m + k)
    a, b, sa, sb = whole(g, m, k), whole(g, n, k), powers(g, m, R.blocks(k)), powers(g, R.blocks(n), R.blocks(k))
    assert torch.equal(ep.matmul_fp8(a, sa, b, sb, out_dtype=dtype), exact(a, sa, b, sb).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_nan_operands(m, n, k, dtype):
    g = gen(m + k + 1)
    a, b, sa, sb = whole(g, m, k), whole(g, n, k), powers(g, m, R.blocks(k)), powers(g, R.blocks(n), R.blocks(k))
    want = exact(a, sa, b, sb).to(dtype)
    for row, at in ((0, 0), (m // 2, 129), (m - 1, k - 1)):
        a.view(torch.uint8)[row, at] = 0x7f
        want[row] = float("nan")
    for col, at in ((1, k - 16), (n - 1, 77)):
        b.view(torch.uint8)[col, at] = 0xff
        want[:, col] = float("nan")
    d = ep.matmul_fp8(a, sa, b, sb, out_dtype=dtype)
    assert torch.equal(d.isnan(), want.isnan()) and torch.equal(d.nan_to_num(0), want.nan_to_num(0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,n,k", [([3, 0, 1, 2], 130, 400), ([70, 0, 129, 40], 300, 400), ([2300, 0, 2150], 4300, 400), ([70, 0, 129], 300, 240)])
def test_grouped(counts, n, k, dtype):
    g, e, rows = gen(n + k), len(counts), sum(counts) + 3
    off = torch.tensor([0] + counts).cumsum(0).tolist()
    a, b, sa, sb = whole(g, rows, k), whole(g, e, n, k), powers(g, rows, R.blocks(k)), powers(g, e, R.blocks(n), R.blocks(k))
    a.view(torch.uint8)[off[-1]:] = 0x7f  # (rows of no group are not read)
    d = ep.grouped_matmul_fp8(a, sa, b, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=dtype)
    for i in range(e):
        at = slice(off[i], off[i + 1])
        assert torch.equal(d[at], exact(a[at], sa[at], b[i], sb[i]).to(dtype)), f"expert {i}"
    assert not d[off[-1]:].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,m,n", [([128, 0, 384], 130, 300), ([256, 0, 128, 128], 2100, 2060)])
def test_weight_gradients(counts, m, n, dtype):
    g, rows = gen(m), sum(counts) + 128
    off = torch.tensor([0] + counts).cumsum(0).tolist()
    a, b, sa, sb = whole(g, m, rows), whole(g, n, rows), powers(g, m, R.blocks(rows)), powers(g, R.blocks(n), R.blocks(rows))
    a.view(torch.uint8)[:, off[-1]:] = 0x7f
    sa[:, -1], sb[:, -1] = float("nan"), float("nan")
    d = ep.grouped_wgrad_fp8(a, sa, b, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=dtype)
    for i in range(len(counts)):
        at, kb = slice(off[i], off[i + 1]), slice(off[i] // 128, off[i + 1] // 128)
        want = exact(a[:, at], sa[:, kb], b[:, at], sb[:, kb]).to(dtype) if counts[i] else torch.zeros((m, n), dtype=dtype, device="cuda")
        assert torch.equal(d[i], want), f"expert {i}"

"""Largest sizes and strides of the 8-bit and expert operators.  On the CPU: the C ABI's refusals, which come
before any HIP call (pointers are fake and never read)."""
import ctypes

import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _fp8 as R
from tests._gpu import require_gpu

INVALID, UNSUPPORTED, HIP = 1, 2, 4
P = 0x100000


@pytest.fixture
def no_gpu():
    """A call that is accepted would be launched on its fake pointers: without a GPU it ends at the first HIP call."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is here")


def matmul(**kw):
    base = dict(m=64, n=256, k=256, a=P, lda=256, sa=P, sam=1, sak=64, b=P, ldb=256, sb=P, sbn=2, sbk=1, d=P, ldd=256, out=1, ws=None,
                wsb=0, st=None)
    assert not set(kw) - set(base)
    return ep.lib().ep_matmul_fp8(*{**base, **kw}.values())


def test_row_stride_of_b_scales():
    """The second scale of a 256-column tile lies whole in the 2^31 - 1 bytes of its window, or is refused."""
    assert matmul(sbn=2 ** 29 - 1) == UNSUPPORTED
    assert matmul(sbn=2 ** 29) == UNSUPPORTED


def test_row_stride_of_b_scales_below_the_limit(no_gpu):
    assert 4 * (2 ** 29 - 2) + 4 <= 2 ** 31 - 1
    assert matmul(sbn=2 ** 29 - 2) == HIP


def dispatch(h, elt, scale=None):
    return ep.lib().ep_expert_dispatch(P, 4, h, h, elt, P, 2, P, 8, P, h, scale, None)


def test_row_length_of_dispatched_fp32():
    """Rows of fp32 values are copied as twice as many 16-bit pieces, 2048 a workgroup, 65535 workgroups at most."""
    assert dispatch(65535 * 1024 + 1, 2) == UNSUPPORTED
    assert all(dispatch(2 ** 26, elt, s) == UNSUPPORTED for elt in (0, 1, 2) for s in (None, P))


def test_row_length_of_dispatched_rows_below_the_limits(no_gpu):
    assert dispatch(65535 * 1024, 2) == HIP
    assert all(dispatch(2 ** 26 - 1, *a) == HIP for a in ((0,), (1,), (2, P)))


def grouped(rows, n, e):
    return ep.lib().ep_grouped_matmul_fp8(rows, n, 256, e, P, P, 256, P, 1, rows, P, n * 256, 256, P, n, 2, 1, P, n, 1, None)


def wgrad(m, n, e):
    return ep.lib().ep_grouped_wgrad_fp8(m, n, 256, e, P, P, 256, P, 1, m, P, 256, P, 2, 1, P, n, 1, None)


TILES = 2 ** 24


def test_more_tiles_than_one_launch_takes():
    """2^24 tiles of 128 x 128 and more are refused; a product of their counts does not overflow."""
    assert matmul(m=2 ** 18, n=2 ** 20, ldd=2 ** 20) == UNSUPPORTED
    assert matmul(m=2 ** 30, n=2 ** 30, ldd=2 ** 30) == UNSUPPORTED
    assert grouped(2 ** 18, 128 * (TILES // (2 ** 11 + 65) + 1), 64) == UNSUPPORTED
    assert wgrad(128 * 64, 128 * 64, TILES // 4096) == UNSUPPORTED
    assert wgrad(2 ** 31 - 8192, 2 ** 31 - 8192, 65534) == UNSUPPORTED


def test_most_tiles_one_launch_takes(no_gpu):
    assert matmul(m=2 ** 18, n=2 ** 20 - 128, ldd=2 ** 20) == HIP
    assert grouped(2 ** 18, 128 * (TILES // (2 ** 11 + 65)), 64) == HIP
    assert wgrad(128 * 64, 128 * 64, TILES // 4096 - 1) == HIP


@pytest.mark.gpu
def test_product_of_many_tiles():
    """More than 2^22 tiles, one a workgroup."""
    require_gpu()
    g = torch.Generator()
    g.manual_seed(1)
    m, n, k = 2 ** 29 + 1000, 8, 16
    tail, b = R.operand(g, 200, k), R.operand(g, n, k)
    a = torch.zeros((m, k), dtype=R.F8, device="cuda")
    a[-200:] = tail.cuda()
    sa, sb = torch.full((1, 1), 0.5), R.scales(g, 1, 1)
    d = ep.matmul_fp8(a, sa.cuda().expand(m, 1), b.cuda(), sb.cuda())
    exact, mags = R.product(tail, sa.expand(200, 1), b, sb)
    R.assert_within(d[-200:], exact, R.product_tolerance(exact, mags, k, torch.bfloat16))
    assert not d[:-200].any()


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["matmul", "grouped"])
@pytest.mark.parametrize("n", [2 ** 28 - 16, 2 ** 28 + 5])
def test_few_rows_by_many_columns(call, n):
    """The longest output rows of the kernel that streams b past a few rows, and longer ones."""
    require_gpu()
    g = torch.Generator()
    g.manual_seed(2)
    m, k = 3, 16
    a, tail = R.operand(g, m, k), R.operand(g, 200, k)
    b = torch.zeros((n, k), dtype=R.F8, device="cuda")
    b[-200:] = tail.cuda()
    sa, sb = R.scales(g, m, 1), torch.full((1, 1), 0.5)
    ops = (a.cuda(), sa.cuda(), b, sb.cuda().expand(R.blocks(n), 1))
    if call == "matmul":
        d = ep.matmul_fp8(*ops)
    else:
        d = ep.grouped_matmul_fp8(*ops[:2], b[None], ops[3][None], torch.tensor([0, m], dtype=torch.int32, device="cuda"))
    exact, mags = R.product(a, sa, tail, sb.expand(2, 1))
    R.assert_within(d[:, -200:], exact, R.product_tolerance(exact, mags, k, torch.bfloat16))
    assert not d[:, :-200].any()


def quantize(m, k, rows, transpose):
    return ep.lib().ep_quantize_fp8(P, m, k, k, 1, rows, transpose, P, m if transpose else k, P, None)


# (rows of a block, transposed), and what a workgroup takes: 8 rows by 4 blocks, or 128 x 128 values
WORKGROUPS = [(1, 0, 8, 512), (1, 1, 128, 128), (128, 0, 128, 128), (128, 1, 128, 128)]


@pytest.mark.parametrize("rows,transpose,by_m,by_k", WORKGROUPS)
def test_more_blocks_than_one_launch_quantises(rows, transpose, by_m, by_k):
    assert quantize(by_m * 4096, by_k * 4096, rows, transpose) == UNSUPPORTED
    assert quantize(by_m * 5000, by_k * 4000, rows, transpose) == UNSUPPORTED
    assert quantize(2 ** 31 - 8192, 2 ** 31 - 8192, rows, transpose) == UNSUPPORTED


@pytest.mark.parametrize("rows,transpose,by_m,by_k", WORKGROUPS)
def test_most_blocks_one_launch_quantises(no_gpu, rows, transpose, by_m, by_k):
    """All the workgroups that a launch takes, whatever the kind of block."""
    assert quantize(by_m * 4096, by_k * 4095, rows, transpose) == HIP
    assert quantize(by_m * 4095, by_k * 4096, rows, transpose) == HIP
    assert quantize(2 ** 26 + 9, 16, rows, transpose) == HIP  # (narrow, with 2^23 times 8 rows)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,transpose,by_m,by_k", WORKGROUPS)
def test_quantise_of_many_rows(rows, transpose, by_m, by_k):
    """2^26 narrow rows: the last ones are right, and where the rows before them are zeros, so are their values."""
    require_gpu()
    g = torch.Generator()
    g.manual_seed(3)
    m, k = 2 ** 26 + 9, 16
    last = 128 + m % 128
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((last, k), generator=g).bfloat16()
    x[-last:] = tail.cuda()
    q, s = ep.quantize_fp8(x, block=(rows, 128), transpose=bool(transpose))
    wq, ws = R.quantize(tail, rows, bool(transpose))
    cut = (slice(None), slice(-last, None)) if transpose else (slice(-last, None),)
    assert torch.equal(q[cut].float().cpu(), wq)
    n = ws.shape[1] if transpose else ws.shape[0]
    assert torch.equal((s[:, -n:] if transpose else s[-n:]).cpu(), ws)
    rest = (slice(None), slice(None, -last)) if transpose else (slice(None, -last),)
    assert not q[rest].contiguous().view(torch.uint8).any()


@pytest.mark.parametrize("m,n,k,parts", [(128, 5120, 17408, 8), (64, 5120, 5120, 5), (1024, 4096, 5120, 0), (777, 5003, 4112, 0), (8, 5120, 17408, 0)])
def test_k_ranges(m, n, k, parts):
    """How many K ranges a product takes, by its workspace; none where that is no gain, or b streams past few rows."""
    need = ctypes.c_size_t()
    assert ep.lib().ep_matmul_fp8_workspace(m, n, k, ctypes.byref(need)) == 0
    assert need.value == parts * m * n * 4

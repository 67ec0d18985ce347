"""Largest sizes and strides of the 8-bit and expert operators.  On the CPU: the C ABI's refusals, which come
before any HIP call (pointers are fake and never read)."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep

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

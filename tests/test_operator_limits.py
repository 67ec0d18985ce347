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

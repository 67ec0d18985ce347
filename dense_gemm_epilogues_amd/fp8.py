"""8-bit block-scaled products: quantisation to e4m3 and the products of what it gives.

A matrix in this form is a pair (q, scale): q e4m3 values, scale one fp32 number for each block of 1 x 128
(activations) or 128 x 128 (weights) values; the last blocks may be partly filled.

    xq, xs = quantize_fp8(x)                              # 1 x 128 blocks along the features
    wq, ws = quantize_fp8(w, block=(128, 128))
    y = matmul_fp8(xq, xs, wq, ws)                        # x w^T

Every function only enqueues kernels (libep.so, `ep_*_fp8` in include/ep.h) on torch's current stream, or
on `stream`, as under torch.cuda.stream(stream).  All are outside autograd: results carry no gradient, and a call
that autograd would be expected to follow warns.  The gradients of y = x w^T are products of the transposes:
dy w by matmul_fp8 and grouped_matmul_fp8, dy^T x by grouped_wgrad_fp8 (one expert: matmul_fp8).
"""
import ctypes
from functools import lru_cache

import torch

from . import _check, lib
from ._operators import (BLOCK, E4M3, ELT, blocks, check, check_out, contiguous, current_stream, no_gradient, on_device,
                         streamed, unit_columns)

__all__ = ["quantize_fp8", "matmul_fp8", "grouped_matmul_fp8", "grouped_wgrad_fp8"]


@streamed
def quantize_fp8(x, block=(1, BLOCK), transpose=False):
    """(q, scale) of x (M x K; float16, bfloat16 or float32, unit column stride), or with transpose of its
    K x M transpose.  block (1, 128): scale has shape (rows, ceil(columns / 128)), features outermost in
    memory; (128, 128): (ceil(rows / 128), ceil(columns / 128)).  For a block's largest finite magnitude
    amax (at least 2^-90), scale = amax / 448 and q = e4m3(x * (448 / amax)); infinities and NaN become
    NaN."""
    check("x", x, ELT, (None, None))
    if tuple(block) not in ((1, BLOCK), (BLOCK, BLOCK)):
        raise ValueError(f"block must be (1, 128) or (128, 128), got {block}")
    no_gradient("quantize_fp8", x)
    ld = unit_columns("x", x)
    on_device(x)
    m, k = x.shape
    rows, cols = (k, m) if transpose else (m, k)
    q = torch.empty((rows, cols), dtype=E4M3, device=x.device)
    if block[0] == 1:
        scale = torch.empty((blocks(cols), rows), dtype=torch.float32, device=x.device)
    else:
        scale = torch.empty((blocks(rows), blocks(cols)), dtype=torch.float32, device=x.device)
    if m and k:
        _check(lib().ep_quantize_fp8(x.data_ptr(), m, k, ld, ELT[x.dtype], block[0], int(bool(transpose)), q.data_ptr(),
                                     cols, scale.data_ptr(), current_stream(x)))
    return q, (scale.t() if block[0] == 1 else scale)


def _out(out, dtype, shape, t, inputs):
    if dtype not in ELT:
        raise ValueError(f"out_dtype must be float16, bfloat16 or float32, got {dtype}")
    if out is None:
        return torch.empty(shape, dtype=dtype, device=t.device), shape[-1]
    return out, check_out(out, dtype, shape, t.device, inputs)


def _operand(name, t, shape, device=None):
    check(name, t, E4M3, shape, device)
    ld = unit_columns(name, t)
    if t.numel() and (t.data_ptr() % 16 or (ld % 16 and t.shape[-2] > 1)):
        raise ValueError(f"{name} must be 16-byte aligned with a row stride that is a multiple of 16, got stride {t.stride()}")
    return (ld + 15) // 16 * 16


def _contracted(k):
    if k % 16:
        raise ValueError(f"the contracted length must be a multiple of 16, got {k}")


@lru_cache(maxsize=256)
def _workspace(m, n, k):
    """Bytes of a product's workspace, which depend on its sizes alone."""
    need = ctypes.c_size_t()
    _check(lib().ep_matmul_fp8_workspace(m, n, k, ctypes.byref(need)))
    return need.value


@streamed
def matmul_fp8(a, a_scale, b, b_scale, out_dtype=torch.bfloat16, out=None):
    """(a a_scale) (b b_scale)^T: a (M x K) with scales (M, ceil(K / 128)), b (N x K) with scales
    (ceil(N / 128), ceil(K / 128)); K a multiple of 16.  Summed in fp32, rounded once to out_dtype.

    16-bit outputs of more than 8 rows and K over 256 pass the e4m3 matrix instruction, which adds the products of 8
    neighbouring k in fixed point before fp32: each loses less than 2^-13 of the largest of the 8 (of normal
    operands; include/ep.h has the bound).  Measured, 1.5e-5 of the result's norm with normally distributed operands,
    2.2e-5 with outlier features.  Where large products cancel among 8 neighbours, take float32 outputs, which are
    summed in fp32 throughout, at half the rate."""
    check("a", a, E4M3, (None, None))
    m, k = a.shape
    check("b", b, E4M3, (None, k), a.device)
    n = b.shape[0]
    _contracted(k)
    lda, ldb = _operand("a", a, (m, k)), _operand("b", b, (n, k))
    check("a_scale", a_scale, torch.float32, (m, blocks(k)), a.device)
    check("b_scale", b_scale, torch.float32, (blocks(n), blocks(k)), a.device)
    no_gradient("matmul_fp8", a, a_scale, b, b_scale)
    on_device(a)
    out, ldd = _out(out, out_dtype, (m, n), a, (a, a_scale, b, b_scale))
    if not m or not n:
        return out
    if not k:
        return out.zero_()
    need = _workspace(m, n, k)
    ws = torch.empty(need, dtype=torch.uint8, device=a.device) if need else None
    _check(lib().ep_matmul_fp8(m, n, k, a.data_ptr(), lda, a_scale.data_ptr(), *a_scale.stride(), b.data_ptr(), ldb,
                           b_scale.data_ptr(), *b_scale.stride(), out.data_ptr(), ldd, ELT[out_dtype],
                           ws.data_ptr() if need else None, need, current_stream(a)))
    return out


def _offsets(offsets, experts, device):
    check("offsets", offsets, torch.int32, (None if experts is None else experts + 1,), device)
    if offsets.shape[0] < 2:
        raise ValueError("offsets must hold at least one expert's two ends")
    contiguous("offsets", offsets)
    return offsets.shape[0] - 1


@streamed
def grouped_matmul_fp8(a, a_scale, b, b_scale, offsets, out_dtype=torch.bfloat16, out=None):
    """matmul_fp8 of each expert's rows with its own matrix: a (rows x K) sorted by expert, b (E x N x K) with
    scales (E, ceil(N / 128), ceil(K / 128)), offsets (E + 1 int32 on the device, ascending from 0): expert e
    has rows offsets[e] to offsets[e + 1].  Rows from offsets[E] on become zeros.  (Summed as matmul_fp8 does; with up
    to 4 rows an expert on average in fp32 throughout.)"""
    check("a", a, E4M3, (None, None))
    rows, k = a.shape
    check("b", b, E4M3, (None, None, k), a.device)
    e, n = b.shape[:2]
    _contracted(k)
    lda, ldb = _operand("a", a, (rows, k)), _operand("b", b, (e, n, k))
    if b.stride(0) % 16 and e > 1:
        raise ValueError(f"the expert stride of b must be a multiple of 16, got stride {b.stride()}")
    check("a_scale", a_scale, torch.float32, (rows, blocks(k)), a.device)
    check("b_scale", b_scale, torch.float32, (e, blocks(n), blocks(k)), a.device)
    _offsets(offsets, e, a.device)
    no_gradient("grouped_matmul_fp8", a, a_scale, b, b_scale)
    on_device(a)
    out, ldd = _out(out, out_dtype, (rows, n), a, (a, a_scale, b, b_scale, offsets))
    if not rows or not n:
        return out
    if not k:
        return out.zero_()
    _check(lib().ep_grouped_matmul_fp8(
        rows, n, k, e, offsets.data_ptr(), a.data_ptr(), lda, a_scale.data_ptr(), *a_scale.stride(), b.data_ptr(),
        b.stride(0) if e > 1 else 0, ldb, b_scale.data_ptr(), *b_scale.stride(), out.data_ptr(), ldd, ELT[out_dtype],
        current_stream(a)))
    return out


@streamed
def grouped_wgrad_fp8(a, a_scale, b, b_scale, offsets, out_dtype=torch.bfloat16, out=None):
    """The experts' weight gradients, (E, M, N): for expert e the product of columns offsets[e] to
    offsets[e + 1] of a (M x rows, scales (M, ceil(rows / 128))) with the same columns of b (N x rows, scales
    (ceil(N / 128), ceil(rows / 128))): transposed quantisations of rows sorted by expert.  Groups start and
    end on multiples of 128 (the gradient of one that does not is NaN); an empty one's gradient is zero.  16-bit
    outputs are summed as matmul_fp8's of many rows, of groups of any size."""
    check("a", a, E4M3, (None, None))
    m, rows = a.shape
    check("b", b, E4M3, (None, rows), a.device)
    n = b.shape[0]
    _contracted(rows)
    lda, ldb = _operand("a", a, (m, rows)), _operand("b", b, (n, rows))
    check("a_scale", a_scale, torch.float32, (m, blocks(rows)), a.device)
    check("b_scale", b_scale, torch.float32, (blocks(n), blocks(rows)), a.device)
    e = _offsets(offsets, None, a.device)
    no_gradient("grouped_wgrad_fp8", a, a_scale, b, b_scale)
    on_device(a)
    out, ldd = _out(out, out_dtype, (e, m, n), a, (a, a_scale, b, b_scale, offsets))
    if e > 1 and m and out.stride(0) != m * ldd:
        raise ValueError(f"out must hold the experts one behind another, got stride {out.stride()}")
    if not m or not n:
        return out
    if not rows:
        return out.zero_()
    _check(lib().ep_grouped_wgrad_fp8(
        m, n, rows, e, offsets.data_ptr(), a.data_ptr(), lda, a_scale.data_ptr(), *a_scale.stride(), b.data_ptr(), ldb,
        b_scale.data_ptr(), *b_scale.stride(), out.data_ptr(), ldd, ELT[out_dtype], current_stream(a)))
    return out

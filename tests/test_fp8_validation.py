"""CPU tests of the 8-bit and expert operators' refusals: the binding's checks of tensors, and the C ABI's
checks, which all come before any HIP call (pointers are fake and never read)."""
import ctypes

import pytest
import torch

import dense_gemm_epilogues_amd as ep

F8 = torch.float8_e4m3fn
INVALID, UNSUPPORTED = 1, 2
P = 0x100000


def z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


def f8(*s):
    return torch.zeros(s).to(F8)


def raises(match, f, *a, **k):
    with pytest.raises(ValueError, match=match):
        f(*a, **k)


def test_quantize_refusals():
    q = ep.quantize_fp8
    raises("CUDA", q, z(4, 8))
    raises("must be torch.float16 or", q, z(4, 8, dtype=torch.float64))
    raises("shape", q, z(4))
    raises("block must be", q, z(4, 8), block=(1, 64))
    raises("unit column stride", q, z(8, 4).t())
    raises("below the row length", q, z(1, 8).expand(4, 8))
    raises("torch.Tensor", q, [1.0])


def test_matmul_refusals():
    mm = ep.matmul_fp8
    ok = dict(a=f8(4, 256), a_scale=z(4, 2), b=f8(130, 256), b_scale=z(2, 2))
    call = lambda **kw: mm(*{**ok, **kw}.values())  # noqa: E731
    raises("CUDA", call)
    raises("a must be torch.float8", call, a=z(4, 256))
    raises("b must have shape", call, b=f8(130, 128))
    raises("a_scale must have shape", call, a_scale=z(4, 1))
    raises("b_scale must have shape", call, b_scale=z(1, 2))
    raises("a_scale must be torch.float32", call, a_scale=z(4, 2, dtype=torch.float64))
    raises("multiple of 16", mm, f8(4, 24), z(4, 1), f8(8, 24), z(1, 1))
    raises("row stride that is a multiple of 16", call, a=f8(4, 264)[:, :256])
    raises("16-byte aligned", call, a=f8(4, 272)[:, 8:264])
    raises("unit column stride", call, b=f8(256, 130).t())
    raises("out must have shape", mm, *ok.values(), out=z(4, 128, dtype=torch.bfloat16)) if torch.cuda.is_available() else None


def test_grouped_refusals():
    g = ep.grouped_matmul_fp8
    ok = dict(a=f8(40, 128), a_scale=z(40, 1), b=f8(3, 16, 128), b_scale=z(3, 1, 1), offsets=z(4, dtype=torch.int32))
    call = lambda **kw: g(*{**ok, **kw}.values())  # noqa: E731
    raises("CUDA", call)
    raises("offsets must have shape", call, offsets=z(3, dtype=torch.int32))
    raises("offsets must be torch.int32", call, offsets=z(4, dtype=torch.int64))
    raises("offsets must be contiguous", call, offsets=z(8, dtype=torch.int32)[::2])
    raises("b must have shape", call, b=f8(16, 128))
    raises("b_scale must have shape", call, b_scale=z(3, 2, 1))
    w = ep.grouped_wgrad_fp8
    ok2 = dict(a=f8(8, 256), a_scale=z(8, 2), b=f8(16, 256), b_scale=z(1, 2), offsets=z(3, dtype=torch.int32))
    call2 = lambda **kw: w(*{**ok2, **kw}.values())  # noqa: E731
    raises("CUDA", call2)
    raises("b must have shape", call2, b=f8(16, 128))
    raises("a_scale must have shape", call2, a_scale=z(8, 3))
    raises("at least one expert", call2, offsets=z(1, dtype=torch.int32))


def test_expert_refusals():
    i32 = torch.int32
    raises("CUDA", ep.expert_order, z(4, 2, dtype=i32), 8)
    raises("ids must be", ep.expert_order, z(4, 2), 8)
    raises("contiguous", ep.expert_order, z(4, 4, dtype=i32)[:, :2], 8)
    order = ep.ExpertOrder(z(4, 2, dtype=i32), z(16, dtype=i32), z(4, dtype=i32))
    raises("CUDA", ep.expert_dispatch, z(4, 8), order)
    raises("order.pos must have shape", ep.expert_dispatch, z(5, 8), order)
    raises("must be an ExpertOrder", ep.expert_dispatch, z(4, 8), (1, 2, 3))
    raises("x must be", ep.expert_dispatch, z(4, 8, dtype=torch.float64), order)
    raises("CUDA", ep.expert_combine, z(16, 8), order, z(4, 2))
    raises("the order's 16 rows", ep.expert_combine, z(15, 8), order)
    raises("weights must have shape", ep.expert_combine, z(16, 8), order, z(4, 3))
    raises("weights must be torch.float32", ep.expert_combine, z(16, 8), order, z(4, 2, dtype=torch.float16))
    raises("CUDA", ep.expert_combine_backward, z(4, 8), z(16, 8), order, z(4, 2))
    raises("y must be torch.float32", ep.expert_combine_backward, z(4, 8), z(16, 8, dtype=torch.float16), order)
    raises("y must have shape", ep.expert_combine_backward, z(4, 8), z(16, 9), order)


def test_quantize_abi():
    q = ep.lib().ep_quantize_fp8
    base = dict(x=P, m=4, k=8, ldx=8, elt=1, rows=1, t=0, q=P, ldq=8, s=P, st=None)
    call = lambda **kw: q(*{**base, **kw}.values())  # noqa: E731
    for kw, want in (({"m": 0}, INVALID), ({"k": 2 ** 31}, UNSUPPORTED), ({"x": None}, INVALID), ({"s": None}, INVALID),
                     ({"elt": 3}, UNSUPPORTED), ({"rows": 64}, UNSUPPORTED), ({"x": P + 1}, INVALID), ({"ldx": 7}, INVALID),
                     ({"ldq": 7}, INVALID), ({"t": 1, "ldq": 3}, INVALID), ({"m": 2 ** 30, "k": 2 ** 20, "ldx": 2 ** 20, "ldq": 2 ** 20}, UNSUPPORTED)):
        assert call(**kw) == want, kw
        assert ep.lib().ep_last_error()


def test_matmul_abi():
    L = ep.lib()
    base = dict(m=4, n=8, k=32, a=P, lda=32, sa=P, sam=1, sak=4, b=P, ldb=32, sb=P, sbn=1, sbk=1, d=P, ldd=8, out=1, ws=None,
                wsb=0, st=None)
    call = lambda **kw: L.ep_matmul_fp8(*{**base, **kw}.values())  # noqa: E731
    for kw, want in (({"m": 0}, INVALID), ({"k": 24}, UNSUPPORTED), ({"a": None}, INVALID), ({"sb": None}, INVALID), ({"a": P + 8}, INVALID),
                     ({"lda": 16}, INVALID), ({"ldb": 40}, INVALID), ({"lda": 2 ** 23}, UNSUPPORTED), ({"sam": -1}, INVALID),
                     ({"sam": 2 ** 23}, UNSUPPORTED), ({"ldd": 7}, INVALID), ({"out": 3}, UNSUPPORTED), ({"d": P + 1}, INVALID),
                     ({"n": 2 ** 31}, UNSUPPORTED)):
        assert call(**kw) == want, kw
    need = ctypes.c_size_t(77)
    assert L.ep_matmul_fp8_workspace(1, 5120, 17408, ctypes.byref(need)) == 0 and need.value == 0
    assert L.ep_matmul_fp8_workspace(1, 1, 1, None) == INVALID


def test_grouped_abi():
    L = ep.lib()
    base = dict(rows=4, n=8, k=32, e=2, off=P, a=P, lda=32, sa=P, sam=1, sak=4, b=P, be=256, ldb=32, sb=P, sbe=1, sbn=1, sbk=1, d=P,
                ldd=8, out=1, st=None)
    call = lambda **kw: L.ep_grouped_matmul_fp8(*{**base, **kw}.values())  # noqa: E731
    for kw, want in (({"e": 0}, INVALID), ({"off": None}, INVALID), ({"off": P + 2}, INVALID), ({"be": 8}, INVALID), ({"e": 65535}, UNSUPPORTED),
                     ({"rows": 0}, INVALID), ({"k": 8}, UNSUPPORTED)):
        assert call(**kw) == want, kw
    base = dict(m=4, n=8, rows=128, e=2, off=P, a=P, lda=128, sa=P, sam=1, sak=4, b=P, ldb=128, sb=P, sbn=1, sbk=1, d=P, ldd=8, out=1,
                st=None)
    call = lambda **kw: L.ep_grouped_wgrad_fp8(*{**base, **kw}.values())  # noqa: E731
    for kw, want in (({"e": 0}, INVALID), ({"off": None}, INVALID), ({"rows": 120}, UNSUPPORTED), ({"lda": 112}, INVALID), ({"ldd": 7}, INVALID)):
        assert call(**kw) == want, kw


def test_expert_abi():
    L = ep.lib()
    cap, need = ctypes.c_int64(), ctypes.c_size_t()
    sizes = lambda *a: L.ep_expert_order_sizes(*a, ctypes.byref(cap), ctypes.byref(need))  # noqa: E731
    assert sizes(65536, 64, 128) == 0 and cap.value == 65536 + 64 * 127 + (-(65536 + 64 * 127) % 128) and need.value > 0
    assert sizes(8, 64, 1) == 0 and cap.value == 8 and need.value == 0
    assert sizes(0, 4, 128) == 0 and cap.value == 0
    assert sizes(8, 1025, 1) == UNSUPPORTED and sizes(8, 0, 1) == INVALID and sizes(-1, 4, 1) == INVALID and sizes(8, 4, 8192) == UNSUPPORTED
    assert sizes(2 ** 31 - 5000, 1024, 128) == UNSUPPORTED
    order = lambda **kw: L.ep_expert_order(*{**dict(ids=P, b=4, s=8, e=4, al=1, pos=P, src=P, off=P, ws=None, wsb=0, st=None), **kw}.values())  # noqa: E731
    for kw, want in (({"b": 2}, UNSUPPORTED), ({"ids": None}, INVALID), ({"off": None}, INVALID), ({"ids": P + 2}, INVALID), ({"s": 65536}, INVALID)):
        assert order(**kw) == want, kw
    disp = lambda **kw: L.ep_expert_dispatch(*{**dict(x=P, t=4, h=8, ldx=8, elt=1, pos=P, k=2, src=P, rows=8, out=P, ldo=8, s=None, st=None), **kw}.values())  # noqa: E731
    for kw, want in (({"h": 0}, INVALID), ({"x": None}, INVALID), ({"src": None}, INVALID), ({"elt": 7}, UNSUPPORTED), ({"ldo": 7}, INVALID),
                     ({"out": P + 1}, INVALID), ({"t": 2 ** 23}, UNSUPPORTED), ({"k": 0}, INVALID)):
        assert disp(**kw) == want, kw
    comb = lambda **kw: L.ep_expert_combine(*{**dict(y=P, rows=8, h=8, ldy=8, elt=1, pos=P, t=4, k=2, w=P, ldw=2, out=P, ldo=8, st=None), **kw}.values())  # noqa: E731
    for kw, want in (({"t": 0}, INVALID), ({"y": None}, INVALID), ({"ldw": 1}, INVALID), ({"ldy": 4}, INVALID), ({"w": P + 2}, INVALID)):
        assert comb(**kw) == want, kw
    back = lambda **kw: L.ep_expert_combine_backward(*{**dict(g=P, t=4, h=8, ldg=8, elt=1, y=P, rows=8, ldy=8, pos=P, k=2, src=P, w=P, ldw=2, dy=P, lddy=8, dw=P, st=None), **kw}.values())  # noqa: E731
    for kw, want in (({"g": None}, INVALID), ({"dw": None}, INVALID), ({"dy": None}, INVALID), ({"lddy": 4}, INVALID), ({"elt": -1}, UNSUPPORTED)):
        assert back(**kw) == want, kw


def test_matmul_workspace():
    """K ranges of a product with few tiles need the workspace that is asked for."""
    L = ep.lib()
    need = ctypes.c_size_t(7)
    assert L.ep_matmul_fp8_workspace(8192, 8192, 4096, ctypes.byref(need)) == 0 and need.value == 0
    assert L.ep_matmul_fp8_workspace(8, 512, 8192, ctypes.byref(need)) == 0 and need.value == 0
    assert L.ep_matmul_fp8_workspace(128, 512, 8192, ctypes.byref(need)) == 0
    parts, rest = divmod(need.value, 128 * 512 * 4)
    assert rest == 0 and 2 <= parts <= 64 // 4
    args = lambda ws, size: (128, 512, 8192, P, 8192, P, 1, 128, P, 8192, P, 64, 1, P, 512, 1, ws, size, None)  # noqa: E731
    for ws, size in ((None, 0), (None, need.value), (P, need.value - 1), (P + 8, need.value)):
        assert L.ep_matmul_fp8(*args(ws, size)) == INVALID
    assert b"workspace" in L.ep_last_error()


def test_scale_stride_limits():
    L = ep.lib()
    ok = [64, 64, 256, P, 256, P, 1, 64, P, 256, P, 2, 1, P, 64, 1, None, 0, None]
    for at, value in ((6, 1 << 21), (11, 1 << 29)):
        args = list(ok)
        args[at] = value
        assert L.ep_matmul_fp8(*args) == UNSUPPORTED

"""CPU tests of the refusals of the norm, the expert routing and the 8-bit products' epilogue: the binding's checks of tensors, the
C ABI's checks, which all come before any HIP call (pointers are fake and never read), and how the functions can be called."""
import ctypes
import inspect
import warnings
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import dense_gemm_epilogues_amd as ep

F8 = torch.float8_e4m3fn
H, I32 = torch.float16, torch.int32
INVALID, UNSUPPORTED = 1, 2
P = 0x100000


def z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


def f8(*s):
    return torch.zeros(s).to(F8)


def raises(match, f, *a, **k):
    with pytest.raises(ValueError, match=match):
        f(*a, **k)


def calls():
    return {
        ep.rms_norm: dict(x=z(4, 8), weight=z(8), residual=z(4, 8), eps=1e-5, quantize=True),
        ep.rms_norm_backward: dict(dy=z(4, 8), x=z(4, 8), weight=z(8), rstd=z(4), dresidual=z(4, 8)),
        ep.expert_route: dict(logits=z(4, 16), topk=2, bias=z(16), score="sigmoid", groups=4, topk_groups=2, group_top=1, renormalize=False, scale=2.0),
        ep.expert_route_backward: dict(dweights=z(4, 2), logits=z(4, 16), ids=z(4, 2, dtype=I32), score="sigmoid", renormalize=False, scale=2.0),
        ep.matmul_fp8: dict(a=f8(4, 256), a_scale=z(4, 2), b=f8(130, 256), b_scale=z(2, 2), out_dtype=torch.float32, out=None, bias=z(130),
                            activation="gelu", residual=z(4, 130), save_pre=True),
        ep.epilogue_backward_fp8: dict(dout=z(4, 8), activation="gelu", pre=z(4, 8)),
    }


names = lambda f: f.__name__  # noqa: E731


@pytest.mark.parametrize("f", calls(), ids=names)
def test_arguments_by_name(f):
    """Reaches the operator's own checks, whose last one tensors on the CPU do not pass."""
    kw = calls()[f]
    raises("CUDA", f, **kw)
    raises("CUDA", f, *kw.values(), stream=None)
    first = next(iter(kw))
    with pytest.raises(TypeError, match=first):
        f(**{k: v for k, v in kw.items() if k != first})
    params = inspect.signature(f).parameters
    assert [n for n in params if n != "stream"] == list(kw)
    assert params["stream"].kind is inspect.Parameter.KEYWORD_ONLY and params["stream"].default is None


@pytest.mark.parametrize("f", calls(), ids=names)
def test_stream_of_another_device_is_refused(f):
    with FakeTensorMode(allow_non_fake_inputs=True):  # (tensors of device 0 without a GPU)
        first, *rest = calls()[f].items()
        on_gpu = torch.empty(first[1].shape, dtype=first[1].dtype, device="cuda:0")
        raises("the stream is on cuda:1", f, **{first[0]: on_gpu}, **dict(rest), stream=SimpleNamespace(device=torch.device("cuda", 1)))


@pytest.mark.parametrize("f", calls(), ids=names)
def test_a_lost_gradient_warns(f):
    kw = calls()[f]
    for name, t in kw.items():
        if not (isinstance(t, torch.Tensor) and t.is_floating_point()):
            continue
        some = {**kw, name: t.clone().requires_grad_()}
        if name == "rstd":
            continue
        with pytest.warns(UserWarning, match=f"{f.__name__} is outside autograd") as seen, pytest.raises(ValueError, match="CUDA"):
            f(**some)
        assert seen[0].filename == __file__  # (points at the call)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with pytest.raises(ValueError, match="CUDA"), torch.no_grad():
                f(**some)
            raises("CUDA", f, **kw)


def varied(f):
    return lambda **kw: f(**{**calls()[f], **kw})


def test_norm_refusals():
    n, b = varied(ep.rms_norm), varied(ep.rms_norm_backward)
    raises("x must be torch.float16 or", n, x=z(4, 8, dtype=torch.float64))
    raises("x must have shape", n, x=z(8))
    raises("weight must have shape", n, weight=z(7))
    raises("weight must be", n, weight=z(8, dtype=H))
    raises("weight must be contiguous", n, weight=z(16)[::2])
    raises("residual must have shape", n, residual=z(4, 9))
    raises("residual must be torch.float32", n, residual=z(4, 8, dtype=H))
    raises("unit column stride", n, x=z(8, 4).t())
    raises("below the row length", n, residual=z(1, 8).expand(4, 8))
    for eps in (-1e-6, float("nan"), float("inf")):
        raises("eps must be", n, eps=eps)
    raises("CUDA", n, x=z(4, 8, dtype=H), residual=z(4, 8, dtype=H), weight=z(8))
    raises("x must have shape", b, x=z(5, 8))
    raises("x must be torch.float32", b, x=z(4, 8, dtype=H))
    raises("rstd must have shape", b, rstd=z(4, 1))
    raises("rstd must be torch.float32", b, rstd=z(4, dtype=H))
    raises("rstd must be contiguous", b, rstd=z(8)[::2])
    raises("dresidual must have shape", b, dresidual=z(4, 7))
    raises("weight must have shape", b, weight=z(4))


def test_route_refusals():
    r, b = varied(ep.expert_route), varied(ep.expert_route_backward)
    raises("logits must be", r, logits=z(4, 16, dtype=I32))
    raises("score must be softmax or sigmoid", r, score="tanh")
    raises("bias must have shape", r, bias=z(15))
    raises("bias must be torch.float32", r, bias=z(16, dtype=H))
    raises("bias must be contiguous", r, bias=z(32)[::2])
    raises("unit column stride", r, logits=z(16, 4).t())
    raises("topk must be", r, topk=0)
    raises("topk must be", r, topk=2.0)
    raises("topk must be", r, topk=-3)
    raises("dweights must be torch.float32", b, dweights=z(4, 2, dtype=H))
    raises("logits must have shape", b, logits=z(5, 16))
    raises("ids must have shape", b, ids=z(4, 3, dtype=I32))
    raises("ids must be torch.int32", b, ids=z(4, 2, dtype=torch.int64))
    raises("ids must be contiguous", b, ids=z(4, 4, dtype=I32)[:, :2])
    raises("score must be", b, score=None)


def test_epilogue_refusals():
    m, b = varied(ep.matmul_fp8), varied(ep.epilogue_backward_fp8)
    raises("activation must be None, relu, gelu or silu", m, activation="tanh")
    raises("bias must have shape", m, bias=z(4))
    raises("bias must be", m, bias=z(130, dtype=H))
    raises("bias must be contiguous", m, bias=z(260)[::2])
    raises("residual must be torch.float32", m, residual=z(4, 130, dtype=H))
    raises("residual must have shape", m, residual=z(4, 131))
    raises("unit column stride", m, residual=z(130, 4).t())
    raises("CUDA", m, out_dtype=H, bias=z(130), residual=z(4, 130, dtype=H))
    raises("pre is given with an activation", b, pre=None)
    raises("pre is given with an activation", b, activation=None)
    raises("pre must have shape", b, pre=z(4, 9))
    raises("pre must be torch.float32", b, pre=z(4, 8, dtype=H))
    raises("dout must be", b, dout=f8(4, 8))
    raises("activation must be", b, activation="swish")


def abi(name, base):
    return lambda **kw: getattr(ep.lib(), name)(*{**base, **kw}.values())


def refused(call, cases):
    for kw, want in cases:
        assert call(**kw) == want, kw
        assert ep.lib().ep_last_error()


def test_norm_abi():
    refused(abi("ep_rms_norm", dict(x=P, m=4, h=8, ldx=8, elt=1, res=P, ldr=8, w=P, welt=1, eps=1e-5, sum=P, lds=8, y=P, ldy=8, s=None, rstd=P, st=None)), (
        ({"m": 0}, INVALID), ({"h": 0}, INVALID), ({"m": 2 ** 31}, UNSUPPORTED), ({"h": 2 ** 26}, UNSUPPORTED), ({"elt": 3}, UNSUPPORTED),
        ({"welt": 0}, UNSUPPORTED), ({"w": None}, INVALID), ({"x": None}, INVALID), ({"y": None}, INVALID), ({"rstd": None}, INVALID), ({"sum": None}, INVALID),
        ({"x": P + 1}, INVALID), ({"w": P + 2, "welt": 2}, INVALID), ({"s": P + 2}, INVALID), ({"y": P + 1}, INVALID), ({"ldx": 7}, INVALID), ({"ldr": 7}, INVALID),
        ({"lds": 7}, INVALID), ({"ldy": 7}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"eps": 1e40}, INVALID),
        ({"m": 2 ** 22, "h": 520, "ldx": 520, "ldr": 520, "lds": 520, "ldy": 520}, UNSUPPORTED)))
    need = ctypes.c_size_t(7)
    L = ep.lib()
    assert L.ep_rms_norm_backward_workspace(9000, 5003, ctypes.byref(need)) == 0 and need.value % (5003 * 4) == 0 and need.value >= 5003 * 4
    assert L.ep_rms_norm_backward_workspace(1, 5003, ctypes.byref(need)) == 0 and need.value == 0
    assert L.ep_rms_norm_backward_workspace(1, 1, None) == INVALID
    assert L.ep_rms_norm_backward_workspace(4, 8, ctypes.byref(need)) == 0
    size = need.value
    refused(abi("ep_rms_norm_backward", dict(dy=P, m=4, h=8, ld=8, elt=1, x=P, ldx=8, w=P, welt=1, rstd=P, dr=P, ldr=8, dx=P, ldo=8, dw=P, ws=P, n=size, st=None)), (
        ({"m": 0}, INVALID), ({"dy": None}, INVALID), ({"x": None}, INVALID), ({"rstd": None}, INVALID), ({"dx": None}, INVALID), ({"dw": None}, INVALID),
        ({"w": None}, INVALID), ({"welt": 0}, UNSUPPORTED), ({"ld": 7}, INVALID), ({"ldx": 7}, INVALID), ({"ldr": 7}, INVALID), ({"ldo": 7}, INVALID),
        ({"ws": None}, INVALID), ({"n": size - 1}, INVALID), ({"ws": P + 8}, INVALID), ({"elt": -1}, UNSUPPORTED), ({"dw": P + 2}, INVALID)))


def test_route_abi():
    r = abi("ep_expert_route", dict(l=P, t=4, e=16, ld=16, elt=1, bias=None, score=0, groups=1, tg=1, top=2, k=2, renorm=1, scale=1.0, ids=P, w=P, st=None))
    refused(r, (
        ({"t": -1}, INVALID), ({"e": 0}, INVALID), ({"k": 0}, INVALID), ({"e": 1025, "ld": 1025}, UNSUPPORTED), ({"k": 65, "e": 100, "ld": 100}, UNSUPPORTED),
        ({"k": 17}, INVALID), ({"t": 2 ** 26}, UNSUPPORTED), ({"score": 2}, UNSUPPORTED), ({"elt": 3}, UNSUPPORTED), ({"ld": 15}, INVALID), ({"l": None}, INVALID),
        ({"ids": None}, INVALID), ({"w": P + 2}, INVALID), ({"bias": P + 2}, INVALID), ({"groups": 0}, INVALID), ({"groups": 3}, INVALID), ({"tg": 0}, INVALID),
        ({"tg": 2}, INVALID), ({"groups": 8, "k": 3}, INVALID), ({"top": 3}, UNSUPPORTED), ({"scale": float("inf")}, INVALID),
        ({"e": 130, "ld": 130, "groups": 65}, UNSUPPORTED)))
    assert r(t=0, l=None, ids=None, w=None) == 0
    b = abi("ep_expert_route_backward", dict(g=P, ldg=2, t=4, k=2, l=P, e=16, ld=16, elt=1, ids=P, score=0, renorm=1, scale=1.0, d=P, ldd=16, st=None))
    refused(b, (({"g": None}, INVALID), ({"ldg": 1}, INVALID), ({"ld": 15}, INVALID), ({"ldd": 15}, INVALID), ({"ids": P + 2}, INVALID), ({"d": None}, INVALID),
                ({"score": -1}, UNSUPPORTED), ({"scale": float("nan")}, INVALID), ({"k": 17}, INVALID)))
    assert b(t=0, g=None, l=None, ids=None, d=None) == 0


def test_epilogue_abi():
    refused(abi("ep_matmul_fp8_epilog", dict(m=4, n=8, k=32, a=P, lda=32, sa=P, sam=1, sak=4, b=P, ldb=32, sb=P, sbn=1, sbk=1, d=P, ldd=8, out=1, bias=P, belt=1,
                                             act=2, res=P, ldr=8, pre=P, ldp=8, ws=None, wsb=0, st=None)), (
        ({"m": 0}, INVALID), ({"k": 24}, UNSUPPORTED), ({"out": 3}, UNSUPPORTED), ({"act": 4}, UNSUPPORTED), ({"act": -1}, UNSUPPORTED), ({"belt": 0}, UNSUPPORTED),
        ({"bias": P + 2, "belt": 2}, INVALID), ({"res": P + 1}, INVALID), ({"pre": P + 1}, INVALID), ({"ldr": 7}, INVALID), ({"ldp": 7}, INVALID),
        ({"ldr": 2 ** 23}, UNSUPPORTED), ({"a": P + 8}, INVALID), ({"ldd": 7}, INVALID), ({"m": 128, "n": 512, "k": 8192, "lda": 8192, "ldb": 8192, "ldd": 512,
                                                                                          "ldr": 512, "ldp": 512, "sak": 128}, INVALID)))
    need = ctypes.c_size_t(7)
    assert ep.lib().ep_epilogue_backward_fp8_workspace(300, 70, ctypes.byref(need)) == 0 and need.value == 3 * 70 * 4
    assert ep.lib().ep_epilogue_backward_fp8_workspace(128, 70, ctypes.byref(need)) == 0 and need.value == 0
    assert ep.lib().ep_epilogue_backward_fp8_workspace(300, 70, None) == INVALID
    refused(abi("ep_epilogue_backward_fp8", dict(g=P, m=200, n=8, ld=8, elt=1, act=1, pre=P, ldp=8, q=P, ldq=8, s=P, qt=P, ldqt=200, st_=P, db=P, ws=P, wsb=64, st=None)), (
        ({"m": 0}, INVALID), ({"n": 2 ** 31}, UNSUPPORTED), ({"elt": 3}, UNSUPPORTED), ({"act": 4}, UNSUPPORTED), ({"pre": None}, INVALID), ({"act": 0}, INVALID),
        ({"g": None}, INVALID), ({"q": None}, INVALID), ({"s": None}, INVALID), ({"qt": None}, INVALID), ({"st_": None}, INVALID), ({"db": None}, INVALID),
        ({"ld": 7}, INVALID), ({"ldp": 7}, INVALID), ({"ldq": 7}, INVALID), ({"ldqt": 199}, INVALID), ({"ws": None}, INVALID), ({"wsb": 63}, INVALID),
        ({"ws": P + 8}, INVALID), ({"pre": P + 1}, INVALID), ({"m": 2 ** 20, "n": 2 ** 20, "ld": 2 ** 20, "ldp": 2 ** 20, "ldq": 2 ** 20, "ldqt": 2 ** 20}, UNSUPPORTED)))


def test_launch_limits():
    """The largest launches have fewer than 2^32 threads: refused at the limit, and not (but for the missing or unsuitable
    stream, HIP's own error) below it."""
    L = ep.lib()
    need = ctypes.c_size_t()
    back = lambda m, n: L.ep_epilogue_backward_fp8(P, m, n, n, 1, 0, None, 0, P, n, P, P, m, P, P, P, 1 << 62, ctypes.c_void_p(0))  # noqa: E731
    assert back(1 << 18, 1 << 19) == UNSUPPORTED and b"blocks" in L.ep_last_error()  # 2^11 x 2^12 blocks of 512 threads
    norm = lambda m, h: L.ep_rms_norm(P, m, h, h, 1, None, 0, P, 1, 1e-5, None, 0, P, h, None, P, None)  # noqa: E731
    for m, h in ((1 << 22, 513), (1 << 26, 512), (1 << 28, 128)):
        assert norm(m, h) == UNSUPPORTED and b"launch" in L.ep_last_error()
    assert L.ep_epilogue_backward_fp8_workspace(1 << 18, 1 << 18, ctypes.byref(need)) == 0 and need.value == 4 << 29
    if not torch.cuda.is_available():
        assert back(1 << 18, (1 << 19) - 128) == 4
        for m, h in (((1 << 22) - 1, 513), ((1 << 26) - 4, 512), ((1 << 28) - 16, 128)):
            assert norm(m, h) == 4

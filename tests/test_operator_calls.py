"""How the 8-bit and expert operators can be called (CPU): every argument by its name, `stream` among them."""
import inspect
import warnings
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import dense_gemm_epilogues_amd as ep

F8 = torch.float8_e4m3fn


def z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


def calls():
    order = ep.ExpertOrder(z(4, 2, dtype=torch.int32), z(16, dtype=torch.int32), z(4, dtype=torch.int32))
    f8 = lambda *s: z(*s).to(F8)  # noqa: E731
    off = z(4, dtype=torch.int32)
    return {
        ep.quantize_fp8: dict(x=z(4, 8), block=(1, 128), transpose=True),
        ep.matmul_fp8: dict(a=f8(4, 256), a_scale=z(4, 2), b=f8(130, 256), b_scale=z(2, 2), out_dtype=torch.float32, out=None),
        ep.grouped_matmul_fp8: dict(a=f8(40, 128), a_scale=z(40, 1), b=f8(3, 16, 128), b_scale=z(3, 1, 1), offsets=off, out=None),
        ep.grouped_wgrad_fp8: dict(a=f8(8, 256), a_scale=z(8, 2), b=f8(16, 256), b_scale=z(1, 2), offsets=off, out=None),
        ep.expert_order: dict(ids=z(4, 2, dtype=torch.int32), experts=8, align=16),
        ep.expert_dispatch: dict(x=z(4, 8), order=order, quantize=True, out=None),
        ep.expert_combine: dict(y=z(16, 8), order=order, weights=z(4, 2), out=None),
        ep.expert_combine_backward: dict(dout=z(4, 8), y=z(16, 8), order=order, weights=z(4, 2)),
    }


@pytest.mark.parametrize("f", calls(), ids=lambda f: f.__name__)
def test_arguments_by_name(f):
    """Reaches the operator's own checks, whose last one tensors on the CPU do not pass."""
    kw = calls()[f]
    with pytest.raises(ValueError, match="CUDA"):
        f(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        f(**kw, stream=None)
    first = next(iter(kw))
    with pytest.raises(TypeError, match=first):
        f(**{k: v for k, v in kw.items() if k != first})


@pytest.mark.parametrize("f", calls(), ids=lambda f: f.__name__)
def test_signature_names_the_stream(f):
    params = inspect.signature(f).parameters
    assert [n for n in params if n in calls()[f]] == list(calls()[f])
    assert params["stream"].kind is inspect.Parameter.KEYWORD_ONLY and params["stream"].default is None


@pytest.mark.parametrize("f", calls(), ids=lambda f: f.__name__)
def test_stream_of_another_device_is_refused(f):
    """Work on it would run on the wrong GPU, and unordered with the operands' stream."""
    with FakeTensorMode(allow_non_fake_inputs=True):  # (tensors of device 0 without a GPU)
        first, *rest = calls()[f].items()
        on_gpu = torch.empty(first[1].shape, dtype=first[1].dtype, device="cuda:0")
        with pytest.raises(ValueError, match="the stream is on cuda:1"):
            f(**{first[0]: on_gpu}, **dict(rest), stream=SimpleNamespace(device=torch.device("cuda", 1)))


@pytest.mark.parametrize("f", [f for f in calls() if f is not ep.expert_order], ids=lambda f: f.__name__)
def test_a_lost_gradient_warns(f):
    """The operators are outside autograd: where it would be expected to follow an argument, they say so."""
    kw = calls()[f]
    for name, t in kw.items():
        if not (isinstance(t, torch.Tensor) and t.is_floating_point()):
            continue
        some = {**kw, name: t.clone().requires_grad_()}
        with pytest.warns(UserWarning, match=f"{f.__name__} is outside autograd") as seen, pytest.raises(ValueError, match="CUDA"):
            f(**some)
        assert seen[0].filename == __file__  # (points at the call)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with pytest.raises(ValueError, match="CUDA"), torch.no_grad():
                f(**some)
            with pytest.raises(ValueError, match="CUDA"):
                f(**kw)

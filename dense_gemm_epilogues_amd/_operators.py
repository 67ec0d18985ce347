"""What the 8-bit and expert operators share: the C ABI's signatures, argument checks, streams."""
import ctypes
import inspect
import warnings
from functools import wraps

import torch

P, I64, INT, SIZE = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t

SIGNATURES = {
    "ep_quantize_fp8": [P, I64, I64, I64, INT, INT, INT, P, I64, P, P],
    "ep_matmul_fp8_workspace": [I64, I64, I64, P],
    "ep_matmul_fp8": [I64, I64, I64, P, I64, P, I64, I64, P, I64, P, I64, I64, P, I64, INT, P, SIZE, P],
    "ep_grouped_matmul_fp8": [I64, I64, I64, I64, P, P, I64, P, I64, I64, P, I64, I64, P, I64, I64, I64, P, I64, INT, P],
    "ep_grouped_wgrad_fp8": [I64, I64, I64, I64, P, P, I64, P, I64, I64, P, I64, P, I64, I64, P, I64, INT, P],
    "ep_expert_order_sizes": [I64, I64, I64, P, P],
    "ep_expert_order": [P, INT, I64, I64, I64, P, P, P, P, SIZE, P],
    "ep_expert_dispatch": [P, I64, I64, I64, INT, P, I64, P, I64, P, I64, P, P],
    "ep_expert_combine": [P, I64, I64, I64, INT, P, I64, I64, P, I64, P, I64, P],
    "ep_expert_combine_backward": [P, I64, I64, I64, INT, P, I64, I64, P, I64, P, P, I64, P, I64, P, P],
}

ELT = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
E4M3 = torch.float8_e4m3fn
BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def check(name, t, dtypes, shape, device=None):
    """Raise ValueError unless t is a tensor of one of dtypes (one, or a container) with this shape
    (None: any size) on `device`."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    dtype = t.dtype
    if dtype is not dtypes and (isinstance(dtypes, torch.dtype) or dtype not in dtypes):
        want = dtypes if isinstance(dtypes, torch.dtype) else " or ".join(str(d) for d in dtypes)
        raise ValueError(f"{name} must be {want}, got {dtype}")
    s = t.shape
    fits = len(s) == len(shape)
    if fits:
        for w, g in zip(shape, s):
            if w is not None and w != g:
                fits = False
    if not fits:
        want = tuple("any" if w is None else w for w in shape)
        raise ValueError(f"{name} must have shape {want}, got {tuple(s)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands are on {device}")


def no_gradient(f, *tensors):
    """Warn where autograd would be expected to follow an argument of f, whose results it does not follow."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            warnings.warn(f"{f} is outside autograd: its result carries no gradient to an argument that requires one", stacklevel=4)
            return


def unit_columns(name, t):
    """Row stride of a matrix whose rows are contiguous and apart (ValueError otherwise)."""
    rows, cols = t.shape[-2:]
    ld, step = t.stride()[-2:]
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride, got stride {t.stride()}")
    if rows <= 1:
        return max(ld, cols)
    if ld < cols:
        raise ValueError(f"{name}: row stride {ld} is below the row length {cols}")
    return ld


def contiguous(name, t):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, got stride {t.stride()}")


def on_device(t):
    if not t.is_cuda:
        raise ValueError(f"operands must be on a CUDA (HIP) device, got {t.device}")


def overlaps(a, b):
    """Whether two tensors' storage ranges meet (an output must not lie over an input)."""
    if not a.numel() or not b.numel():
        return False
    ends = [t.data_ptr() + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size() for t in (a, b)]
    return a.data_ptr() < ends[1] and b.data_ptr() < ends[0]


def check_out(out, dtype, shape, device, inputs):
    """Row stride of a given output; it may lie over no input."""
    check("out", out, dtype, shape, device)
    for t in inputs:
        if overlaps(out, t):
            raise ValueError("out lies over an input")
    return unit_columns("out", out)


def streamed(f):
    """Adds `stream=None`: with a torch stream, the call's kernels and the tensors it allocates go to
    that stream, which must be on the first tensor's device.  The launches run with that device current."""
    sig = inspect.signature(f)
    params = list(sig.parameters.values())
    name = params[0].name

    @wraps(f)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            return f(*args, **kw)  # (which refuses it)
        if stream is not None:
            if stream.device != first.device:
                raise ValueError(f"the stream is on {stream.device}, {name} is on {first.device}")
            with torch.cuda.stream(stream):
                return f(*args, **kw)
        if first.get_device() != torch.cuda.current_device():
            with torch.cuda.device(first.device):
                return f(*args, **kw)
        return f(*args, **kw)
    call.__signature__ = sig.replace(parameters=params + [inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def current_stream(t):
    return torch._C._cuda_getCurrentRawStream(t.get_device())

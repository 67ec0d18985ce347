"""The MLP half of a transformer layer on a residual stream, in 8-bit block-scaled products, with its training step: a dense
GELU-MLP, and the sparse (mixture-of-experts) SwiGLU-MLP of sparse_mlp.py behind a router.

    dense:   s = stream + delta,  y = s + W2 gelu(W1 norm(s) + b1) + b2
    sparse:  s = stream + delta,  y = sum_j w_j expert_j(norm(s)),  (ids, w) = route(Wr norm(s))

    python examples/mlp_block.py [--tokens 4096 --hidden 5120 --inter 17408 --experts 64 --topk 8 --expert-inter 2048]

Without sizes given, prints how far outputs and gradients are from the same blocks in float32.
"""
import argparse
import os
import sys
from typing import NamedTuple

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_epilogues_amd as ep  # noqa: E402
from examples import sparse_mlp  # noqa: E402

EPS = 1e-5
ROUTE = {"score": "sigmoid", "renormalize": True, "scale": 1.0}


class Linear(NamedTuple):
    """A matrix (N, K) for x W^T and, transposed, for the data gradient dy W; its bias (N,) or None."""
    q: torch.Tensor
    scale: torch.Tensor
    q_t: torch.Tensor
    scale_t: torch.Tensor
    bias: torch.Tensor


def quantized_linear(w, bias=None):
    """Laid out once a weight update."""
    return Linear(*ep.quantize_fp8(w, block=(128, 128)), *ep.quantize_fp8(w, block=(128, 128), transpose=True), bias)


# ------------------------------------------------------------------------------------------ dense
def dense_forward(delta, stream, norm, up, down):
    """(y, saved): delta and stream (T, h), the layer's output so far and the residual stream; y is the stream behind the block."""
    n = ep.rms_norm(delta, norm, residual=stream, eps=EPS, quantize=True)
    act, pre = ep.matmul_fp8(n.y, n.scale, up.q, up.scale, out_dtype=delta.dtype, bias=up.bias, activation="gelu", save_pre=True)
    y = ep.matmul_fp8(*ep.quantize_fp8(act), down.q, down.scale, out_dtype=delta.dtype, bias=down.bias, residual=n.residual)
    return y, (n, act, pre)


def dense_backward(dy, saved, norm, up, down):
    """(dx, dnorm, dup, dup_bias, ddown, ddown_bias): dx is the gradient of both delta and stream.  T a multiple of 16."""
    n, act, pre = saved
    d = ep.epilogue_backward_fp8(dy)
    dact = ep.matmul_fp8(d.q, d.scale, down.q_t, down.scale_t, out_dtype=dy.dtype)
    ddown = ep.matmul_fp8(d.q_t, d.scale_t, *ep.quantize_fp8(act, block=(128, 128), transpose=True), out_dtype=dy.dtype)
    g = ep.epilogue_backward_fp8(dact, activation="gelu", pre=pre)
    dn = ep.matmul_fp8(g.q, g.scale, up.q_t, up.scale_t, out_dtype=dy.dtype)
    x = ep.rms_norm(n.residual, norm, eps=EPS).y  # (again: kept, it would be a second copy of the activations)
    dup = ep.matmul_fp8(g.q_t, g.scale_t, *ep.quantize_fp8(x, block=(128, 128), transpose=True), out_dtype=dy.dtype)
    dx, dnorm = ep.rms_norm_backward(dn, n.residual, norm, n.rstd, dresidual=dy)
    return dx, dnorm, dup, g.dbias, ddown, d.dbias


# ----------------------------------------------------------------------------------------- sparse
def sparse_forward(delta, stream, norm, router, balance, gate_up, down, topk, align=sparse_mlp.ALIGN):
    """(y, stream, saved): y (T, h) joins the returned stream at the next norm.  router (E, h); balance (E,) float32 moves
    tokens between the experts and has no gradient."""
    n = ep.rms_norm(delta, norm, residual=stream, eps=EPS)
    logits = F.linear(n.y, router)
    ids, weights = ep.expert_route(logits, topk, bias=balance, **ROUTE)
    y, experts = sparse_mlp.forward(n.y, ids, weights, gate_up, down, align=align)
    return y, n.residual, (n, logits, ids, experts)


def sparse_backward(dy, dstream, saved, norm, router, gate_up, down):
    """(dx, dnorm, drouter, dgate_up, ddown) of a forward with align 128: dy and dstream are the gradients of what it returned."""
    n, logits, ids, experts = saved
    dn, dweights, dgate_up, ddown = sparse_mlp.backward(dy, experts, gate_up, down)
    dlogits = ep.expert_route_backward(dweights, logits, ids, **ROUTE)
    dn = dn + dlogits @ router
    dx, dnorm = ep.rms_norm_backward(dn, n.residual, norm, n.rstd, dresidual=dstream)
    return dx, dnorm, dlogits.t() @ n.y, dgate_up, ddown


# -------------------------------------------------------------------------------------- reference
def reference_norm(x, w):
    return x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * w


def reference_dense(delta, stream, norm, up, up_bias, down, down_bias):
    s = delta + stream
    return s + F.gelu(reference_norm(s, norm) @ up.t() + up_bias) @ down.t() + down_bias


def reference_sparse(delta, stream, norm, router, ids, gate_up, down):
    """With the choice of experts given."""
    s = delta + stream
    x = reference_norm(s, norm)
    p = torch.sigmoid(x @ router.t()).gather(1, ids.long())
    return sparse_mlp.reference(x, ids, p / p.sum(1, keepdim=True), gate_up, down), s


def inputs(tokens, hidden, inter, experts, topk, expert_inter, dtype=torch.bfloat16, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    v = {"delta": r(tokens, hidden), "stream": r(tokens, hidden), "norm": 1 + 0.1 * r(hidden), "up": r(inter, hidden) / hidden ** 0.5,
         "up_bias": 0.1 * r(inter), "down": r(hidden, inter) / inter ** 0.5, "down_bias": 0.1 * r(hidden), "dy": r(tokens, hidden),
         "router": r(experts, hidden) / hidden ** 0.5, "gate_up": r(experts, 2 * expert_inter, hidden) / hidden ** 0.5,
         "experts_down": r(experts, hidden, expert_inter) / expert_inter ** 0.5, "dstream": r(tokens, hidden)}
    v = {n: t.to(dtype) for n, t in v.items()}
    v.update(balance=0.05 * r(experts), topk=topk)
    return v


def dense_step(v, up, down):
    y, saved = dense_forward(v["delta"], v["stream"], v["norm"], up, down)
    return (y,) + dense_backward(v["dy"], saved, v["norm"], up, down)


def sparse_step(v, gate_up, down):
    y, stream, saved = sparse_forward(v["delta"], v["stream"], v["norm"], v["router"], v["balance"], gate_up, down, v["topk"])
    return (y,) + sparse_backward(v["dy"], v["dstream"], saved, v["norm"], v["router"], gate_up, down), stream, saved[2]


def weights(v):
    """(up, down) of the dense block and of the sparse one."""
    return ((quantized_linear(v["up"], v["up_bias"]), quantized_linear(v["down"], v["down_bias"])),
            (sparse_mlp.quantized_weights(v["gate_up"]), sparse_mlp.quantized_weights(v["experts_down"])))


def distances(v):
    """{name: relative Frobenius distance from float32} of the outputs and every gradient of both blocks."""
    apart = lambda a, b: ((a.float() - b).norm() / b.norm()).item()  # noqa: E731
    leaf = lambda *names: [v[n].float().requires_grad_() for n in names]  # noqa: E731
    dense, sparse = weights(v)
    got = dense_step(v, *dense)
    leaves = leaf("delta", "stream", "norm", "up", "up_bias", "down", "down_bias")
    y = reference_dense(*leaves)
    want = (y.detach(),) + torch.autograd.grad(y, leaves[:1] + leaves[2:], v["dy"].float())
    out = {n: apart(a, b) for n, a, b in zip(("y", "dx", "dnorm", "dup", "dup_bias", "ddown", "ddown_bias"), got, want)}
    got, stream, ids = sparse_step(v, *sparse)
    leaves = leaf("delta", "stream", "norm", "router", "gate_up", "experts_down")
    y, s = reference_sparse(*leaves[:4], ids, *leaves[4:])
    want = (y.detach(),) + torch.autograd.grad((y, s), leaves[:1] + leaves[2:], (v["dy"].float(), v["dstream"].float()))
    out.update({"sparse " + n: apart(a, b) for n, a, b in zip(("y", "dx", "dnorm", "drouter", "dgate_up", "ddown"), got, want)})
    out["sparse stream"] = apart(stream, s.detach())
    return out


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", None), ("hidden", 5120), ("inter", 17408), ("experts", 64), ("topk", 8), ("expert-inter", 2048), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    if a.tokens is None:
        for n, d in distances(inputs(304, 512, 640, 8, 2, 384)).items():
            print(f"{n}: {d:.4f} from float32")
        return
    v = inputs(a.tokens, a.hidden, a.inter, a.experts, a.topk, a.expert_inter)
    dense, sparse = weights(v)
    one = {n: v[n][:1] for n in ("delta", "stream")}
    runs = {f"dense training step of {a.tokens} tokens": lambda: dense_step(v, *dense),
            f"sparse training step of {a.tokens} tokens": lambda: sparse_step(v, *sparse),
            "one token through the dense block": lambda: dense_forward(one["delta"], one["stream"], v["norm"], *dense),
            "one token through the sparse block": lambda: sparse_forward(one["delta"], one["stream"], v["norm"], v["router"], v["balance"],
                                                                         *sparse, a.topk, align=1)}
    for name, step in runs.items():
        for _ in range(3):
            step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.steps):
            step()
        end.record()
        end.synchronize()
        print(f"{name}: {start.elapsed_time(end) / a.steps:.3f} ms")


if __name__ == "__main__":
    main()

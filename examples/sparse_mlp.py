"""A sparse (mixture-of-experts) SwiGLU-MLP layer in 8-bit block-scaled products: a training step and
a single token's forward, on the library's public operators.

    out[t] = sum_j w[t][j] Wd_e (silu(Wg_e x_t) * (Wu_e x_t)),  e = ids[t][j]

    python examples/sparse_mlp.py [--tokens 4096 --experts 64 --topk 8 --hidden 5120 --inter 2048]

Activations and their gradients are quantised along what each product contracts, with one scale for
1 x 128 values; weights with one for 128 x 128.  Without sizes given, prints how far the layer's output
and gradients are from the same layer in float32.
"""
import argparse
import os
import sys
from typing import NamedTuple

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_epilogues_amd as ep  # noqa: E402

ALIGN = 128  # rows an expert's group is padded to: the scale block of its weight gradients


class Weights(NamedTuple):
    """One projection of all experts, (E, N, K), for x W^T and for the data gradient dy W."""
    q: torch.Tensor         # (E, N, K) e4m3
    scale: torch.Tensor     # (E, N / 128, K / 128)
    q_t: torch.Tensor       # (E, K, N)
    scale_t: torch.Tensor   # (E, K / 128, N / 128)


def quantized_weights(w):
    """Weights of w (E, N, K; N and K multiples of 128), laid out once a weight update."""
    e, n, k = w.shape
    if n % 128 or k % 128:
        raise ValueError(f"expert matrices must have sizes that are multiples of 128, got {n} x {k}")
    flat = w.reshape(e * n, k)
    q, s = ep.quantize_fp8(flat, block=(128, 128))
    qt, st = ep.quantize_fp8(flat, block=(128, 128), transpose=True)
    return Weights(q.view(e, n, k), s.view(e, n // 128, k // 128),
                   qt.view(k, e, n).transpose(0, 1), st.view(k // 128, e, n // 128).transpose(0, 1))


def forward(x, ids, weights, gate_up, down, align=ALIGN):
    """(out, saved): x (T, h), ids and weights (T, k); gate_up holds [Wg | Wu] (E, 2 i, h), down (E, h, i)."""
    order = ep.expert_order(ids, gate_up.q.shape[0], align=align)
    xq, xs = ep.expert_dispatch(x, order, quantize=True)
    gu = ep.grouped_matmul_fp8(xq, xs, gate_up.q, gate_up.scale, order.offsets, out_dtype=x.dtype)
    g, u = gu.chunk(2, dim=1)
    act = F.silu(g) * u
    aq, a_s = ep.quantize_fp8(act)
    y = ep.grouped_matmul_fp8(aq, a_s, down.q, down.scale, order.offsets, out_dtype=x.dtype)
    return ep.expert_combine(y, order, weights), (x, weights, order, gu, act, y)


def backward(dout, saved, gate_up, down):
    """(dx, dweights, dgate_up, ddown) of a forward with align 128."""
    x, weights, order, gu, act, y = saved
    dy, dweights = ep.expert_combine_backward(dout, y, order, weights)
    dyq, dys = ep.quantize_fp8(dy)
    dact = ep.grouped_matmul_fp8(dyq, dys, down.q_t, down.scale_t, order.offsets, out_dtype=dout.dtype)
    ddown = ep.grouped_wgrad_fp8(*ep.quantize_fp8(dy, transpose=True),
                                 *ep.quantize_fp8(act, block=(128, 128), transpose=True), order.offsets, out_dtype=dout.dtype)
    g, u = gu.chunk(2, dim=1)
    s = torch.sigmoid(g.float())
    dgu = torch.cat([dact * u * s * (1 + g * (1 - s)), dact * g * s], dim=1).to(dout.dtype)
    dguq, dgus = ep.quantize_fp8(dgu)
    drows = ep.grouped_matmul_fp8(dguq, dgus, gate_up.q_t, gate_up.scale_t, order.offsets, out_dtype=dout.dtype)
    dgate_up = ep.grouped_wgrad_fp8(*ep.quantize_fp8(dgu, transpose=True),
                                    *ep.quantize_fp8(ep.expert_dispatch(x, order), block=(128, 128), transpose=True),
                                    order.offsets, out_dtype=dout.dtype)
    return ep.expert_combine(drows, order), dweights, dgate_up, ddown


def reference(x, ids, weights, gate_up, down):
    """The layer in float32 (matrices as given, unquantised), expert by expert."""
    out = x.new_zeros(x.shape)
    for e in range(gate_up.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            g, u = (x[t] @ gate_up[e].t()).chunk(2, dim=1)
            out = out.index_add(0, t, (F.silu(g) * u) @ down[e].t() * weights[t, j, None])
    return out


def inputs(tokens, experts, topk, hidden, inter, dtype=torch.bfloat16, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    logits, ids = r(tokens, experts).topk(topk, dim=1)
    return {"x": r(tokens, hidden).to(dtype), "ids": ids.int(), "weights": logits.softmax(1),
            "gate_up": (r(experts, 2 * inter, hidden) / hidden ** 0.5).to(dtype),
            "down": (r(experts, hidden, inter) / inter ** 0.5).to(dtype), "dout": r(tokens, hidden).to(dtype)}


def distances(v):
    """{name: relative Frobenius distance from float32} of the output and every gradient."""
    gate_up, down = quantized_weights(v["gate_up"]), quantized_weights(v["down"])
    out, saved = forward(v["x"], v["ids"], v["weights"], gate_up, down)
    got = (out,) + backward(v["dout"], saved, gate_up, down)
    leaves = [v[n].float().requires_grad_() for n in ("x", "weights", "gate_up", "down")]
    ref = reference(leaves[0], v["ids"], leaves[1], leaves[2], leaves[3])
    want = (ref,) + torch.autograd.grad(ref, leaves, v["dout"].float())
    names = ("out", "dx", "dweights", "dgate_up", "ddown")
    return {n: ((a.float() - b).norm() / b.norm()).item() for n, a, b in zip(names, got, (w.detach() for w in want))}


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", None), ("experts", 64), ("topk", 8), ("hidden", 5120), ("inter", 2048), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    if a.tokens is None:
        for n, d in distances(inputs(300, 8, 2, 512, 384)).items():
            print(f"{n}: {d:.4f} from float32")
        return
    v = inputs(a.tokens, a.experts, a.topk, a.hidden, a.inter)
    gate_up, down = quantized_weights(v["gate_up"]), quantized_weights(v["down"])
    one = {n: v[n][:1] for n in ("x", "ids", "weights")}

    def train():
        _, saved = forward(v["x"], v["ids"], v["weights"], gate_up, down)
        backward(v["dout"], saved, gate_up, down)

    def token():
        forward(one["x"], one["ids"], one["weights"], gate_up, down, align=1)

    for name, step in ((f"training step of {a.tokens} tokens", train), ("one token's forward", token)):
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

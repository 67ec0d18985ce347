"""The sparse SwiGLU-MLP example next to itself on plain 64-bit forms of the library's operators, so that what is
quantised is quantised on both sides, and single tokens next to the batch."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep
from examples import sparse_mlp as M
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

# Relative Frobenius distance of two runs whose products differ by 1.5e-5 of the norm (fixed point; far less in fp32).
# A change of mean size d before a rounding with steps s comes out of it as sqrt(d s): 16-bit steps are about 5.6e-3
# (bf16), e4m3 steps 0.09 of a value.  act: d = 3e-5, e4m3: 1.6e-3; y and out, rounded: 2.7e-3 and 3.5e-3.  dgu: d = 1e-4,
# e4m3: 3e-3; its products and their sums, rounded: up to 4.7e-3.  Three times that:
CLOSE = 2.0 ** -6


class Plain:
    """The library's operators, as the example calls them, in 64 bits with one rounding."""

    @staticmethod
    def quantize_fp8(x, block=(1, 128), transpose=False):
        q, s = R.quantize(x.cpu(), block[0], transpose)
        return q.to(R.F8).cuda(), s.cuda()

    @staticmethod
    def grouped_matmul_fp8(a, a_scale, b, b_scale, offsets, out_dtype):
        ends = offsets.tolist()
        x = R.dequantized(a, a_scale)
        out = torch.zeros((a.shape[0], b.shape[1]), dtype=torch.float64, device=a.device)
        for e in range(b.shape[0]):
            at = slice(ends[e], ends[e + 1])
            out[at] = x[at] @ R.dequantized(b[e], b_scale[e], 128).t()
        return out.to(out_dtype)

    @staticmethod
    def grouped_wgrad_fp8(a, a_scale, b, b_scale, offsets, out_dtype):
        ends = offsets.tolist()
        x, y = R.dequantized(a, a_scale), R.dequantized(b, b_scale, 128)
        return torch.stack([x[:, i:j] @ y[:, i:j].t() for i, j in zip(ends, ends[1:])]).to(out_dtype)

    @staticmethod
    def expert_order(ids, experts, align):
        return ep.ExpertOrder(*(t.cuda() for t in R.order(ids.cpu(), experts, align)))

    @staticmethod
    def expert_dispatch(x, order, quantize=False):
        token = order.src.long().clamp_min(0) // order.pos.shape[1]
        rows = torch.where((order.src < 0)[:, None], torch.zeros((), dtype=x.dtype, device=x.device), x[token])
        return Plain.quantize_fp8(rows) if quantize else rows

    @staticmethod
    def expert_combine(y, order, weights=None):
        w = torch.ones(order.pos.shape, device=y.device) if weights is None else weights
        kept = (order.pos >= 0)[..., None]
        return torch.where(kept, y[order.pos.long().clamp_min(0)].double() * w.double()[..., None], 0.0).sum(1).to(y.dtype)

    @staticmethod
    def expert_combine_backward(dout, y, order, weights):
        dy = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
        dw = torch.zeros(weights.shape, dtype=torch.float64, device=y.device)
        for j in range(order.pos.shape[1]):
            on = order.pos[:, j] >= 0
            at = order.pos[on, j].long()
            dy[at] = weights[on, j, None].double() * dout[on].double()
            dw[on, j] = (y[at].double() * dout[on].double()).sum(1)
        return dy.to(y.dtype), dw.float()


def distance(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,experts,topk,hidden,inter", [(1, 4, 2, 512, 384), (200, 8, 2, 512, 384), (77, 16, 4, 384, 640)])
def test_layer_against_its_plain_forms(tokens, experts, topk, hidden, inter, dtype, monkeypatch):
    require_gpu()
    v = M.inputs(tokens, experts, topk, hidden, inter, dtype)

    def step():
        gate_up, down = M.quantized_weights(v["gate_up"]), M.quantized_weights(v["down"])
        out, saved = M.forward(v["x"], v["ids"], v["weights"], gate_up, down)
        return (out,) + M.backward(v["dout"], saved, gate_up, down)

    got = step()
    monkeypatch.setattr(M, "ep", Plain)
    for name, a, b in zip(("out", "dx", "dweights", "dgate_up", "ddown"), got, step()):
        assert a.dtype == b.dtype and a.shape == b.shape
        assert distance(a, b) < CLOSE, f"{name}: {distance(a, b)}"


def test_single_tokens_are_the_batch_rows():
    """Padded as the batch is, a token's rows pass the same sums: equal bit for bit.  Unpadded they pass the few-row
    kernel, whose sums are in fp32."""
    require_gpu()
    v = M.inputs(64, 8, 3, 512, 256)
    gate_up, down = M.quantized_weights(v["gate_up"]), M.quantized_weights(v["down"])
    whole, _ = M.forward(v["x"], v["ids"], v["weights"], gate_up, down)

    def alone(align):
        return torch.cat([M.forward(v["x"][t:t + 1], v["ids"][t:t + 1], v["weights"][t:t + 1], gate_up, down, align=align)[0]
                          for t in range(64)])

    assert torch.equal(alone(128), whole)
    assert distance(alone(1), whole) < CLOSE

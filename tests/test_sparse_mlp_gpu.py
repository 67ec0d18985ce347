"""The sparse SwiGLU-MLP example: its output and gradients next to the same layer in float32."""
import pytest
import torch

from examples import sparse_mlp as M
from tests._gpu import require_gpu

# Each e4m3 operand of a product is off by at most half a step, 2^-4 of its value; over many independent
# roundings the relative error of a sum of products is below 2^-4 for each operand, and those of a chain of
# products add as squares.  Operands on the way: x, Wgu, act, Wd (out and dweights); dy, Wd, then the forward's
# x and Wgu through g and u, dgu, Wgu (dx); the same with x a second time in place of Wgu (dgate_up); dy, act
# with x and Wgu behind it (ddown).
OPERANDS = {"out": 4, "dweights": 4, "dx": 6, "dgate_up": 6, "ddown": 4}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,experts,topk,hidden,inter", [(1, 4, 2, 256, 128), (300, 8, 2, 512, 384), (77, 16, 4, 384, 256)])
def test_layer_against_float32(dtype, tokens, experts, topk, hidden, inter):
    require_gpu()
    got = M.distances(M.inputs(tokens, experts, topk, hidden, inter, dtype))
    for name, d in got.items():
        assert d < OPERANDS[name] ** 0.5 * 2.0 ** -4, f"{name}: {d}"


@pytest.mark.gpu
@pytest.mark.parametrize("align", [1, 128])
def test_single_token_is_the_batch_row(align):
    """One token alone gives what it gives in a batch, but for the order of fp32 sums and their rounding."""
    require_gpu()
    v = M.inputs(64, 8, 3, 512, 256)
    gate_up, down = M.quantized_weights(v["gate_up"]), M.quantized_weights(v["down"])
    whole, _ = M.forward(v["x"], v["ids"], v["weights"], gate_up, down)
    one, _ = M.forward(v["x"][5:6], v["ids"][5:6], v["weights"][5:6], gate_up, down, align=align)
    assert float((one.float() - whole[5:6].float()).norm() / whole[5:6].float().norm()) < 2 * 2.0 ** -4


def test_weights_refuse_ragged_sizes():
    with pytest.raises(ValueError, match="multiples of 128"):
        M.quantized_weights(torch.zeros((2, 130, 128)))

"""The transformer-MLP example: a run of the norm, the router, the 8-bit products with their epilogues and all gradients, next to
float32, captured in a graph, and single tokens next to the batch."""
import pytest
import torch

from examples import mlp_block as M
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

# As for the sparse layer: each e4m3 operand of a product is off by at most half a step, 2^-4 of its value, and those on the way
# to a result add as squares.  Dense: norm rows, W1, act, W2 (y); dy, W2, then W1 and norm rows through P, g, W1 (dx, dnorm); dy, W2,
# W1 and norm rows through P, g, norm rows (dup, without the last two its bias); dy, act with norm rows and W1 behind it (ddown); the
# stream and dy pass to y and dx unquantised, which only brings these nearer.  ddown_bias: a sum of dy, no product (and bf16's steps of the reference).
# Sparse: as there, with the norm's output rounded to 16 bits; drouter by way of dweights (4 operands); dnorm and dx as its dx.
OPERANDS = {"y": 4, "dx": 6, "dnorm": 6, "dup": 6, "dup_bias": 4, "ddown": 4, "ddown_bias": 1, "sparse y": 4, "sparse dx": 6, "sparse dnorm": 6,
            "sparse drouter": 4, "sparse dgate_up": 6, "sparse ddown": 4, "sparse stream": 1}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", [(16, 128, 256, 4, 1, 128), (304, 512, 640, 8, 2, 384), (80, 384, 528, 16, 4, 256)])
def test_blocks_against_float32(dtype, sizes):
    v = M.inputs(*sizes, dtype=dtype)
    for name, d in M.distances(v).items():
        if name == "sparse drouter" and v["topk"] == 1:  # (one weight over itself is 1 whatever the router says: the gradient is 0 but for
            assert M.sparse_step(v, *M.weights(v)[1])[0][3].abs().max().item() < 2.0 ** -40  # the rounding of doubles)
            continue
        assert d < OPERANDS[name] ** 0.5 * 2.0 ** -4, f"{name}: {d}"


def test_single_tokens_are_the_batch_rows():
    """But for the order of fp32 sums, their rounding, and what that does to e4m3 roundings behind them."""
    v = M.inputs(64, 512, 640, 8, 3, 256)
    dense, sparse = M.weights(v)
    whole, _ = M.dense_forward(v["delta"], v["stream"], v["norm"], *dense)
    args = (v["norm"], v["router"], v["balance"], *sparse, v["topk"])
    rows, stream, saved = M.sparse_forward(v["delta"], v["stream"], *args)
    for t in (0, 5, 63):
        d, s = v["delta"][t:t + 1], v["stream"][t:t + 1]
        one, _ = M.dense_forward(d, s, v["norm"], *dense)
        assert float((one.float() - whole[t].float()).norm() / whole[t].float().norm()) < 2.0 ** -5
        for align in (1, 128):
            y, st, sv = M.sparse_forward(d, s, *args, align=align)
            assert torch.equal(st[0], stream[t]) and torch.equal(sv[2][0].sort().values, saved[2][t].sort().values)
            assert float((y.float() - rows[t].float()).norm() / rows[t].float().norm()) < 2.0 ** -4


def test_training_step_in_a_graph():
    """Both blocks' steps captured, replayed between eager ones: the same bits each time."""
    v = M.inputs(144, 256, 384, 8, 2, 128)
    dense, sparse = M.weights(v)
    step = lambda: M.dense_step(v, *dense) + M.sparse_step(v, *sparse)[0]  # noqa: E731
    step()
    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = step()
    for _ in range(3):
        again = step()
        for t in got:
            t.fill_(9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, again):
            assert torch.equal(a, b) and torch.equal(c, b)

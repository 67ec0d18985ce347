"""8-bit products over several tiles a workgroup, K ranges and the borders between kernels, on operands whose
products and sums are exact in every step (small whole numbers, scales that are powers of two): outputs equal
the exact result rounded once, bit for bit."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def whole(g, *shape):
    """Whole numbers from -2 to 2: products up to 4, whose sums stay exact in fixed point and in fp32."""
    return torch.randint(-2, 3, shape, generator=g, device="cuda").float().to(R.F8)


def powers(g, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())


def exact(a, sa, b, sb):
    return R.dequantized(a, sa) @ R.dequantized(b, sb, 128).t()


def same(got, want, what=""):
    want = want.to(got.dtype)
    bad = got != want
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


# few rows and their border; one tile; K ranges, also of unequal length and with a partly filled last block; 128 x 128
# tiles, several a workgroup; 256 x 256 tiles, several a workgroup, with ragged edges; the shortest sums in tiles
SHAPES = [(1, 1, 16), (2, 17, 384), (8, 130, 8208), (9, 130, 8208), (64, 512, 5120), (128, 640, 17408), (100, 1000, 4240),
          (33, 4099, 1936), (300, 1300, 272), (3000, 3100, 400), (4400, 4300, 400), (4353, 4609, 656), (8200, 8200, 272)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul_exact(dtype, m, n, k):
    g = gen(m + n + k)
    a, b = whole(g, m, k), whole(g, n, k)
    sa, sb = powers(g, R.blocks(k), m).t(), powers(g, R.blocks(n), R.blocks(k))
    same(ep.matmul_fp8(a, sa, b, sb, out_dtype=dtype), exact(a, sa, b, sb), f"{m} x {n} x {k}")


@pytest.mark.parametrize("m,n,k", [(9, 257, 2064), (300, 515, 400), (4400, 4300, 272)])
def test_matmul_into_a_wider_buffer(m, n, k):
    """Rows of odd length at odd addresses; what lies around them stays."""
    g = gen(1)
    a, b = whole(g, m, k), whole(g, n, k)
    sa, sb = powers(g, m, R.blocks(k)), powers(g, R.blocks(n), R.blocks(k))
    buf = torch.full((m + 2, n + 7), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.matmul_fp8(a, sa, b, sb, out=buf[1:m + 1, 3:3 + n])
    same(buf[1:m + 1, 3:3 + n], exact(a, sa, b, sb))
    buf[1:m + 1, 3:3 + n] = 7
    assert (buf == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", [[1] * 64, [5] * 60, [0, 17, 3, 0, 8, 9, 1, 0], [90] * 16, [300, 0, 1, 257, 600, 255] * 4,
                                    [0] * 100 + [2000, 0, 129] + [0] * 30, [4000, 3000]])
def test_grouped_exact(dtype, counts):
    """Groups of every kind of size, more tiles than workgroups, rows behind the last group."""
    g, e, n, k = gen(len(counts)), len(counts), 1300, 400
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    rows = sum(counts) + 5
    a, b = whole(g, rows, k), whole(g, e, n, k)
    sa, sb = powers(g, R.blocks(k), rows).t(), powers(g, e, R.blocks(n), R.blocks(k))
    d = ep.grouped_matmul_fp8(a, sa, b, sb, off, out_dtype=dtype)
    ends = off.tolist()
    for i in range(e):
        at = slice(ends[i], ends[i + 1])
        same(d[at], exact(a[at], sa[at], b[i], sb[i]), f"expert {i}")
    assert not d[ends[-1]:].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,counts", [(1024, 1030, [128] * 30), (1040, 1024, [0, 128, 0, 0, 256, 640] * 6), (260, 4100, [1024, 0, 128] * 4),
                                        (128, 130, [0] * 5), (5, 9, [128, 384])])
def test_wgrad_exact(dtype, m, n, counts):
    """Sums of a single block, empty groups between others, more tiles than workgroups."""
    g, e = gen(m), len(counts)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    rows = max(sum(counts), 128)
    a, b = whole(g, m, rows), whole(g, n, rows)
    sa, sb = powers(g, R.blocks(rows), m).t(), powers(g, R.blocks(n), R.blocks(rows))
    d = ep.grouped_wgrad_fp8(a, sa, b, sb, off, out_dtype=dtype)
    x, y = R.dequantized(a, sa), R.dequantized(b, sb, 128)
    ends = off.tolist()
    for i in range(e):
        at = slice(ends[i], ends[i + 1])
        same(d[i], x[:, at] @ y[:, at].t(), f"expert {i}")


def test_infinite_and_nan_scales_stay_in_their_rows():
    """A row whose scale is infinite or NaN does not reach the tiles worked on before or after it."""
    g, m, n, k = gen(2), 4400, 4300, 400
    a, b = whole(g, m, k), whole(g, n, k)
    sa, sb = powers(g, m, R.blocks(k)), powers(g, R.blocks(n), R.blocks(k))
    sa[255, 3], sa[300, 0], sa[-1, 1] = float("inf"), float("nan"), float("-inf")
    d = ep.matmul_fp8(a, sa, b, sb)
    rest = torch.ones(m, dtype=torch.bool, device="cuda")
    rest[[255, 300, m - 1]] = False
    same(d[rest], exact(a[rest], sa[rest], b, sb))
    assert d[300].isnan().all() and not d[255].isfinite().any() and not d[-1].isfinite().any()


def test_calls_repeat_bit_for_bit_and_in_graphs():
    """K ranges and many tiles: equal results from call to call, on a side stream, and from graph replays."""
    g = gen(3)
    shapes = [(128, 512, 8192), (4400, 4300, 400), (3, 1000, 4096)]
    ops = [((torch.randn((m, k), generator=g, device="cuda") * 100).clamp(-448, 448).to(R.F8), powers(g, m, R.blocks(k)),
            (torch.randn((n, k), generator=g, device="cuda") * 100).clamp(-448, 448).to(R.F8), powers(g, R.blocks(n), R.blocks(k)))
           for m, n, k in shapes]

    def step():
        return [ep.matmul_fp8(*o) for o in ops]

    want = step()
    for a, b in zip(step(), want):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [ep.matmul_fp8(*o, stream=side) for o in ops]
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for r in range(3):
        for o in ops:
            o[0].view(torch.uint8).copy_(o[0].view(torch.uint8).roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b), f"replay {r}"

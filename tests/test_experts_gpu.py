"""Expert order, dispatch, combine and its gradients on the GPU against plain forms: whole numbers and
copied values exactly, sums against 64 bits within derived bounds."""
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
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def random_ids(g, t, k, e, dtype=torch.int32):
    """Ids with repeats, dropped choices and whole dropped tokens."""
    ids = torch.randint(-1, e + 1, (t, k), generator=g)
    ids[torch.rand((t,), generator=g) < 0.1] = -1
    return ids.to(dtype)


def check_order(ids, e, align):
    got = ep.expert_order(ids.cuda(), e, align=align)
    for name, a, b in zip(("pos", "src", "offsets"), got, R.order(ids, e, align)):
        assert a.dtype == torch.int32 and torch.equal(a.cpu(), b), name
    return got


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("t,k,e,align", [(0, 2, 3, 1), (1, 1, 1, 1), (1, 8, 64, 1), (1, 8, 64, 128), (5, 3, 7, 16), (63, 4, 9, 128),
                                         (128, 8, 60, 1), (129, 8, 60, 128), (700, 6, 1024, 4), (3000, 2, 300, 128),
                                         (9001, 8, 64, 128)])
def test_order(dtype, t, k, e, align):
    check_order(random_ids(gen(t + k), t, k, e, dtype), e, align)


@pytest.mark.parametrize("t,k", [(1, 1), (300, 4), (5000, 3)])
def test_order_extremes(t, k):
    """Every slot at one expert; every slot dropped; ids far outside."""
    check_order(torch.full((t, k), 5, dtype=torch.int32), 9, 128)
    check_order(torch.full((t, k), -1, dtype=torch.int32), 9, 128)
    check_order(torch.full((t, k), 2 ** 40 + 3, dtype=torch.int64), 9, 1)
    check_order(torch.full((t, k), -2 ** 31, dtype=torch.int32), 9, 1)


ROWS = [(1, 1, 1, 64, 1), (1, 8, 64, 5120, 1), (3, 2, 4, 1, 128), (17, 4, 8, 77, 1), (65, 3, 5, 200, 16), (40, 9, 12, 2056, 1),
        (100, 8, 16, 2500, 128)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h,align", ROWS)
def test_dispatch(dtype, t, k, e, h, align):
    g = gen(h)
    ids = random_ids(g, t, k, e)
    order = check_order(ids, e, align)
    x = torch.randn((t, h + 3), generator=g).to(dtype)[:, 1:1 + h]
    x[0, 0] = float("nan")
    dev = x.cuda()
    assert dev.stride(0) == h or t == 1 or dev.is_contiguous()
    wide = torch.randn((t, h + 5), generator=g).to(dtype).cuda()
    wide[:, 2:2 + h] = dev
    src = order.src.cpu().long()
    want = torch.where((src < 0)[:, None], torch.zeros((), dtype=dtype), x[src.clamp_min(0) // k])
    for xs in (dev, wide[:, 2:2 + h]):
        got = ep.expert_dispatch(xs, order).cpu()
        assert torch.equal(got.nan_to_num(9), want.nan_to_num(9)) and torch.equal(got.isnan(), want.isnan())
        q, s = ep.expert_dispatch(xs, order, quantize=True)
        wq, ws = R.quantize(x, 1, False)
        pad = (src < 0)[:, None]
        wq, ws = wq[src.clamp_min(0) // k].masked_fill(pad, 0), ws[src.clamp_min(0) // k].masked_fill(pad, R.AMAX_MIN / 448)
        assert torch.equal(s.cpu(), ws)
        assert torch.equal(q.float().cpu().nan_to_num(9), wq.nan_to_num(9)) and torch.equal(q.float().cpu().isnan(), wq.isnan())


def combine64(y, pos, w):
    """(sum, sum of magnitudes) in 64 bits; w None: ones."""
    t, k = pos.shape
    out, mags = torch.zeros((t, y.shape[1]), dtype=torch.float64), torch.zeros((t, y.shape[1]), dtype=torch.float64)
    for j in range(k):
        on = pos[:, j] >= 0
        v = y[pos[on, j].long()].double() * (1.0 if w is None else w[on, j, None].double())
        out[on] += v
        mags[on] += v.abs()
    return out, mags


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h,align", ROWS)
def test_combine(dtype, t, k, e, h, align, weighted):
    g = gen(h + 1)
    order = check_order(random_ids(g, t, k, e), e, align)
    rows = order.src.shape[0]
    y = torch.randn((rows, h), generator=g).to(dtype)
    y[order.src.cpu() < 0] = float("nan")  # padding rows are not read
    w = torch.rand((t, k + 2), generator=g)[:, 1:1 + k] if weighted else None
    buf = torch.full((t, h + 4), 7.0, dtype=dtype, device="cuda")
    got = ep.expert_combine(y.cuda(), order, w.cuda() if weighted else None, out=buf[:, 2:2 + h])
    exact, mags = combine64(y, order.pos.cpu(), w)
    # fp32: a product and an addition for each choice; then half a step of the type
    gamma = 2 * k * 2.0 ** -24 * 1.01
    R.assert_within(got, exact, gamma * mags + R.HALF_STEP[dtype] * (exact.abs() + gamma * mags) + R.SMALLEST[dtype])
    assert (buf[:, :2] == 7).all() and (buf[:, 2 + h:] == 7).all()
    none = (order.pos.cpu() < 0).all(1)
    assert not got.cpu()[none].any()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h,align", ROWS)
def test_combine_backward(dtype, t, k, e, h, align, weighted):
    g = gen(h + 2)
    order = check_order(random_ids(g, t, k, e), e, align)
    pos, src = order.pos.cpu(), order.src.cpu()
    y = torch.randn((src.shape[0], h), generator=g).to(dtype)
    y[src < 0] = float("nan")
    dout = torch.randn((t, h), generator=g).to(dtype)
    w = torch.rand((t, k), generator=g) if weighted else None
    dy, dw = ep.expert_combine_backward(dout.cuda(), y.cuda(), order, w.cuda() if weighted else None)
    assert dy.dtype == dtype and dw.dtype == torch.float32
    want_y = torch.zeros(y.shape, dtype=torch.float64)
    want_w, mags = torch.zeros((t, k), dtype=torch.float64), torch.zeros((t, k), dtype=torch.float64)
    for j in range(k):
        on = pos[:, j] >= 0
        at = pos[on, j].long()
        want_y[at] = dout[on].double() * (1.0 if w is None else w[on, j, None].double())
        p = y[at].double() * dout[on].double()
        want_w[on, j], mags[on, j] = p.sum(1), p.abs().sum(1)
    # dy: one fp32 product, half a step of the type
    R.assert_within(dy, want_y, (2.0 ** -24 + R.HALF_STEP[dtype]) * 1.01 * want_y.abs() + R.SMALLEST[dtype], "dy")
    # dw: fp32 products and h additions at most
    R.assert_within(dw, want_w, (h + 1) * 2.0 ** -24 * 1.01 * mags + 2.0 ** -149, "dw")


def test_gradients_against_differences():
    """The forward functions are linear in y, in the weights and in x: central differences of the kernels'
    own forward in fp32 give the gradients' inner products, up to the forward's rounding."""
    g, t, k, e, h = gen(21), 50, 3, 6, 96
    order = check_order(random_ids(g, t, k, e), e, 16)
    rows = order.src.shape[0]
    r = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    y, w, dout, vy, vw = r(rows, h), r(t, k), r(t, h), r(rows, h), r(t, k)
    dy, dw = ep.expert_combine_backward(dout, y, order, w)
    inner = lambda a, b: float((a.double() * b.double()).sum())  # noqa: E731
    f = lambda yy, ww: ep.expert_combine(yy, order, ww)  # noqa: E731
    # each forward value is off by less than 8 2^-24 of magnitudes below 60; t h values weighted by dout
    tol = 2 * 8 * 2.0 ** -24 * 60 * t * h
    assert abs(inner(f(y + vy, w) - f(y - vy, w), dout) / 2 - inner(dy, vy)) < tol
    assert abs(inner(f(y, w + vw) - f(y, w - vw), dout) / 2 - inner(dw, vw)) < tol
    x, vx, drows = r(t, h), r(t, h), r(rows, h)
    dx = ep.expert_combine(drows, order)
    assert abs(inner(ep.expert_dispatch(x + vx, order) - ep.expert_dispatch(x - vx, order), drows) / 2 - inner(dx, vx)) < tol


def test_side_stream_and_graph():
    g, t, k, e, h = gen(22), 300, 4, 16, 520
    ids, x, w = random_ids(g, t, k, e).cuda(), torch.randn((t, h), generator=g).bfloat16().cuda(), torch.rand((t, k), generator=g).cuda()

    def step():
        order = ep.expert_order(ids, e, align=16)
        rows = ep.expert_dispatch(x, order)
        q, s = ep.expert_dispatch(x, order, quantize=True)
        out = ep.expert_combine(rows, order, w)
        return (*order, rows, q.view(torch.uint8), s, out, *ep.expert_combine_backward(x, rows, order, w))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for r in range(4):
        ids.copy_(random_ids(g, t, k, e))
        x.copy_(torch.randn((t, h), generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, step())):
            assert torch.equal(a, b), f"replay {r}, output {i}"


def test_rows_past_2_31_elements():
    """Expert rows whose element offsets pass 32 bits."""
    t, k, h = 33000, 8, 8200
    assert t * k * h > 2 ** 31
    ids = torch.arange(k, dtype=torch.int32, device="cuda").repeat(t, 1)
    order = ep.expert_order(ids, k)
    x = torch.arange(t, device="cuda").remainder(251)[:, None].expand(t, h).to(torch.bfloat16)
    rows = ep.expert_dispatch(x, order)
    assert torch.equal(rows[-t:], x)
    out = ep.expert_combine(rows, order, torch.full((t, k), 0.125, device="cuda"))
    assert torch.equal(out, x)
    dy, dw = ep.expert_combine_backward(x, rows, order)
    assert torch.equal(dy[-t:], x)
    v = x[:, 0].double()
    assert torch.allclose(dw[:, -1].double(), v * v * h, rtol=h * 2.0 ** -24, atol=0)

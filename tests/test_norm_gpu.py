"""The root-mean-square norm and its gradients on the GPU against 64 bits: every type, lengths from 1 to past what registers
hold, strides, special values, graphs and streams."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _block as B
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# the kernels' borders: 16 and 64 lanes a row, a workgroup of 1, 2 and 4 times 8 values a thread, rows read twice
SHAPES = [(1, 1), (3, 7), (5, 8), (33, 64), (17, 127), (16, 128), (9, 129), (6, 511), (4, 512), (3, 513), (7, 1000), (2, 4099), (300, 640),
          (3, 8192), (2, 8200), (2, 8205), (2, 20003), (2, 32768), (2, 32776), (2, 40001)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def inputs(m, h, dtype, seed, wide=False):
    g = B.gen(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = (r(m, h) * torch.exp2(torch.randint(-3, 4, (1, h), generator=g).float())).to(dtype)
    return x, (1 + 0.3 * r(h)).to(torch.float32 if wide else dtype), r(m, h).to(dtype)


def check_norm(out, x, w, res, eps, quantize):
    m, h = x.shape
    r = B.norm_sum(x, res)
    assert torch.equal(out.residual.cpu(), r)
    y, rstd = B.norm(r, w, eps)
    assert ((out.rstd.cpu().double() - rstd).abs() <= B.rstd_tolerance(h) * rstd).all()
    if not quantize:
        assert out.scale is None and out.y.dtype == x.dtype
        R.assert_within(out.y, y, B.norm_tolerance(y, h, x.dtype))
        return
    t = B.rstd_tolerance(h) + 2 * B.U
    pad = torch.nn.functional.pad(y.abs(), (0, R.blocks(h) * 128 - h)).view(m, R.blocks(h), 128)
    amax = pad.amax(2).clamp_min(R.AMAX_MIN)
    scale = out.scale.cpu().double()
    assert out.y.dtype == R.F8 and ((scale - amax / 448).abs() <= (t + B.U) * amax / 448).all()
    # a rounding to e4m3: half a step, 2^-4 of a normal value, half the subnormal step 2^-9 of the scale; the factor and product before it
    wide = scale.repeat_interleave(128, 1)[:, :h]
    R.assert_within(out.y.double().cpu() * wide, y, (2.0 ** -4 + t + 4 * B.U) * y.abs() * 1.01 + 2.0 ** -10 * wide * 1.01)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,h", SHAPES)
def test_norm(dtype, m, h):
    for i, (with_res, quantize) in enumerate(((False, False), (True, False), (False, True), (True, True))):
        x, w, res = inputs(m, h, dtype, m * 7 + h + i, wide=i % 2 == 1)
        res = res if with_res else None
        out = ep.rms_norm(x.cuda(), w.cuda(), residual=None if res is None else res.cuda(), eps=1e-5, quantize=quantize)
        check_norm(out, x, w, res, 1e-5, quantize)


@pytest.mark.parametrize("h", [100, 640, 1003, 8200, 40001])
def test_quantised_rows_are_those_of_the_unquantised(h):
    """fp32 rows are not rounded: quantising them is what the norm does, bit for bit."""
    x, w, res = (t.cuda() for t in inputs(11, h, torch.float32, h))
    a, b = ep.rms_norm(x, w, residual=res), ep.rms_norm(x, w, residual=res, quantize=True)
    q, s = ep.quantize_fp8(a.y)
    assert torch.equal(q.view(torch.uint8), b.y.view(torch.uint8)) and torch.equal(s, b.scale) and torch.equal(a.rstd, b.rstd)
    assert s.stride() == b.scale.stride()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,h", SHAPES + [(1100, 72), (700, 1032)])
def test_norm_backward(dtype, m, h):
    for with_res in (False, True):
        x, w, dy = inputs(m, h, dtype, m * 5 + h, wide=with_res)
        dres = inputs(m, h, dtype, m + h)[2] if with_res else None
        rstd = (x.double().square().mean(1) + 1e-6).rsqrt().float()
        dx, dw = ep.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), rstd.cuda(), dresidual=None if dres is None else dres.cuda())
        (wx, ex), (ww, ew) = B.norm_backward(dy, x, w, rstd, dres)
        assert dx.dtype == dtype and dw.dtype == torch.float32
        R.assert_within(dx, wx, ex + R.HALF_STEP[dtype] * (wx.abs() + ex) + R.SMALLEST[dtype], "dx")
        R.assert_within(dw, ww, ew + 2.0 ** -140, "dweight")


def test_gradients_against_differences():
    """Along random directions: (f(v + d) - f(v - d)) / 2 of f = sum of dy y + dres r, in 64 bits."""
    m, h = 9, 523
    x, w, dy = inputs(m, h, torch.float32, 3, wide=True)
    res, dres = inputs(m, h, torch.float32, 4)[2], inputs(m, h, torch.float32, 5)[2]
    out = ep.rms_norm(x.cuda(), w.cuda(), residual=res.cuda())
    dx, dw = (t.double().cpu() for t in ep.rms_norm_backward(dy.cuda(), out.residual, w.cuda(), out.rstd, dresidual=dres.cuda()))
    r = out.residual.cpu().double()

    def f(r, w):
        y, _ = B.norm(r, w, 1e-6)
        return (y * dy.double()).sum() + (r * dres.double()).sum()

    g = B.gen(6)
    for _ in range(4):
        v, u = torch.randn((m, h), generator=g).double(), torch.randn(h, generator=g).double()
        e = 1e-4
        want = (f(r + e * v, w.double()) - f(r - e * v, w.double())) / (2 * e)
        # the third derivative's part, e^2, and fp32's part of the sum
        assert abs((dx * v).sum() - want) <= 1e-5 * (dx * v).abs().sum()
        want = (f(r, w.double() + e * u) - f(r, w.double() - e * u)) / (2 * e)
        assert abs((dw * u).sum() - want) <= 1e-5 * (dw * u).abs().sum()


@pytest.mark.parametrize("h", [100, 1000, 1003])
def test_strides(h):
    """Rows of wider buffers, at any alignment."""
    wide = [t.cuda() for t in inputs(7, h + 9, torch.bfloat16, 1)]
    x, res, dy = wide[0][:, 3:3 + h], wide[2][:, 1:1 + h], wide[2][:, 5:5 + h]
    w = wide[1][:h]
    out = ep.rms_norm(x, w, residual=res)
    ref = ep.rms_norm(x.contiguous(), w, residual=res.contiguous())
    for a, b in zip(out, ref):
        assert a is None and b is None or torch.equal(a, b)
    got = ep.rms_norm_backward(dy, x, w, out.rstd, dresidual=res)
    want = ep.rms_norm_backward(dy.contiguous(), x.contiguous(), w, out.rstd, dresidual=res.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("h", [96, 1000, 1003, 40001])
def test_special_values(h):
    """A row of zeros, one with NaN, one with an infinity: other rows keep their values."""
    x, w, res = inputs(8, h, torch.bfloat16, 2)
    plain = ep.rms_norm(x.cuda(), w.cuda(), residual=res.cuda())
    x[1], res[1] = 0, 0
    x[3, h - 1] = float("nan")
    x[5, 0] = float("inf")
    out = ep.rms_norm(x.cuda(), w.cuda(), residual=res.cuda(), eps=1e-6)
    assert not out.y[1].any() and out.rstd[1].item() == pytest.approx(1e3, rel=1e-6)
    assert out.y[3].isnan().all() and out.rstd[3].isnan()
    assert out.rstd[5] == 0 and out.y[5, 0].isnan() and not out.y[5, 1:].any()
    for i in (0, 2, 4, 6, 7):
        assert torch.equal(out.y[i], plain.y[i]) and torch.equal(out.rstd[i], plain.rstd[i])
    q = ep.rms_norm(x.cuda(), w.cuda(), residual=res.cuda(), quantize=True)
    assert q.y[3].float().isnan().all() and (q.scale[1] == R.AMAX_MIN / 448).all() and not q.y[1].float().any()


def test_empty():
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    out = ep.rms_norm(z(0, 16), z(16), quantize=True)
    assert out.y.shape == (0, 16) and out.scale.shape == (0, 1) and out.rstd.shape == (0,)
    out = ep.rms_norm(z(3, 0), z(0), eps=0.25)
    assert out.y.shape == (3, 0) and (out.rstd == 2).all()
    dx, dw = ep.rms_norm_backward(z(0, 5), z(0, 5), z(5), z(0))
    assert dx.shape == (0, 5) and not dw.any() and dw.shape == (5,)


def test_graph_and_streams():
    """Captured on a stream of its own, replayed between eager calls, and twice in flight at once."""
    x, w, res = (t.cuda() for t in inputs(300, 1000, torch.bfloat16, 8))
    want = ep.rms_norm(x, w, residual=res, quantize=True)
    grads = ep.rms_norm_backward(res, want.residual, w, want.rstd, dresidual=x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = ep.rms_norm(x, w, residual=res, quantize=True)
        back = ep.rms_norm_backward(res, out.residual, w, out.rstd, dresidual=x)
    for _ in range(3):
        other = ep.rms_norm_backward(x, res, w, want.rstd)
        torch.cuda.synchronize()
        for t in (out.residual, out.rstd, *back):
            t.fill_(7)
        g.replay()
        side = ep.rms_norm_backward(x, res, w, want.rstd, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        assert torch.equal(out.y.view(torch.uint8), want.y.view(torch.uint8)) and torch.equal(out.scale, want.scale)
        assert torch.equal(out.residual, want.residual) and all(torch.equal(a, b) for a, b in zip(back, grads))
        assert all(torch.equal(a, b) for a, b in zip(side, other))


@pytest.mark.parametrize("m,h", [(257, 7000), (300, 8192), (513, 8200), (767, 1032), (769, 1032), (1500, 2048), (4100, 72), (9000, 264)])
def test_norm_backward_by_the_number_of_workgroups(m, h):
    """1 to 8 rows a workgroup, 256 to 2048 workgroups.  A thread of the parts' sum adds at most 2048 / 32 of them and 5 lanes' sums, a
    workgroup ceil(m / 256) rows of 7000 and more, ceil(m / 512) of others: fewer adds than the bound counts."""
    test_norm_backward(torch.bfloat16, m, h)
    test_norm_backward(torch.float32, m, h)

"""The norm, the routing and the epilogues on inputs that lie in buffers full of NaN, into outputs whose surroundings stay, past 2^31
elements, and several at once: through the binding and, for output strides and outputs over inputs, through the C ABI."""
import ctypes

import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _block as B
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
ELT = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def amid(t, fill=float("nan"), left=5, rows=2):
    """t as a view of a wider buffer of `fill`: some values and rows on every side."""
    if t.dim() == 1:
        buf = torch.full((t.shape[0] + 2 * left,), fill, dtype=t.dtype, device="cuda")
        view = buf[left:-left]
    else:
        buf = torch.full((t.shape[0] + 2 * rows, t.shape[1] + 2 * left), fill, dtype=t.dtype, device="cuda")
        view = buf[rows:-rows, left:-left]
    view.copy_(t)
    return buf, view


def untouched(buf, view, fill):
    inside = torch.zeros_like(buf, dtype=torch.bool)
    at = (view.data_ptr() - buf.data_ptr()) // buf.element_size()
    inside.as_strided(view.shape, view.stride(), at).fill_(True)
    return bool((buf[~inside] == fill).all())


def same(a, b):
    return all(x is None and y is None or torch.equal(x.flatten().view(torch.uint8), y.flatten().view(torch.uint8)) for x, y in zip(a, b))


def rand(g, *s, dtype=torch.float32):
    return torch.randn(s, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,h", [(5, 3), (7, 100), (6, 129), (9, 400), (5, 1003), (4, 2048), (3, 8200), (2, 12001), (2, 33000)])
def test_norm_amid_nan(dtype, m, h):
    g = B.gen(h)
    x, res, dy, w = rand(g, m, h, dtype=dtype), rand(g, m, h, dtype=dtype), rand(g, m, h, dtype=dtype), rand(g, h, dtype=dtype)
    nx, nr, nd, nw = (amid(t)[1] for t in (x, res, dy, w))
    for quantize in (False, True):
        out = ep.rms_norm(x, w, residual=res, quantize=quantize)
        assert same(ep.rms_norm(nx, nw, residual=nr, quantize=quantize), out)
    assert same(ep.rms_norm_backward(nd, nx, nw, out.rstd, dresidual=nr), ep.rms_norm_backward(dy, x, w, out.rstd, dresidual=res))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,h", [(5, 3), (7, 100), (9, 400), (5, 1003), (4, 2048), (2, 33000)])
def test_norm_output_strides_and_in_place(dtype, m, h):
    """The C ABI's own strides: rows of wider buffers, whose other values stay; r written over x or over the residual."""
    L = ep.lib()
    g = B.gen(h + 1)
    x, res, dy, w = rand(g, m, h, dtype=dtype), rand(g, m, h, dtype=dtype), rand(g, m, h, dtype=dtype), rand(g, h, dtype=dtype)
    stream = torch.cuda.current_stream().cuda_stream
    want = ep.rms_norm(x, w, residual=res, eps=1e-5)
    quant = ep.rms_norm(x, w, residual=res, eps=1e-5, quantize=True)
    for over in ("nothing", "x", "res"):
        xb, rb = x.clone(), res.clone()
        sbuf, s = amid(torch.zeros_like(x), 7.0)
        ybuf, y = amid(torch.zeros_like(x), 7.0)
        total = {"nothing": s, "x": xb, "res": rb}[over]
        rstd = torch.empty(m, device="cuda")
        e = ELT[dtype]
        assert L.ep_rms_norm(xb.data_ptr(), m, h, h, e, rb.data_ptr(), h, w.data_ptr(), e, 1e-5, total.data_ptr(), total.stride(0) if m > 1 else h + 10,
                             y.data_ptr(), y.stride(0), None, rstd.data_ptr(), stream) == 0
        assert torch.equal(y, want.y) and torch.equal(total, want.residual) and torch.equal(rstd, want.rstd)
        assert untouched(ybuf, y, 7.0) and untouched(sbuf, s, 7.0)
    qbuf = torch.full((m, h + 9), 0x55, dtype=torch.uint8, device="cuda")
    q, scale = qbuf[:, 4:4 + h], torch.empty((R.blocks(h), m), device="cuda")
    assert L.ep_rms_norm(x.data_ptr(), m, h, h, e, res.data_ptr(), h, w.data_ptr(), e, 1e-5, s.data_ptr(), s.stride(0), q.data_ptr(), h + 9, scale.data_ptr(),
                         rstd.data_ptr(), stream) == 0
    assert torch.equal(q, quant.y.view(torch.uint8)) and torch.equal(scale.t(), quant.scale) and (qbuf[:, :4] == 0x55).all() and (qbuf[:, 4 + h:] == 0x55).all()
    dx, dw = ep.rms_norm_backward(dy, x, w, want.rstd, dresidual=res)
    need = ctypes.c_size_t()
    assert L.ep_rms_norm_backward_workspace(m, h, ctypes.byref(need)) == 0
    ws = torch.full((need.value + 64,), 0xff, dtype=torch.uint8, device="cuda")
    dbuf, d = amid(torch.zeros_like(x), 7.0)
    wbuf, dweight = amid(torch.zeros(h), 7.0)
    assert L.ep_rms_norm_backward(dy.data_ptr(), m, h, h, e, x.data_ptr(), h, w.data_ptr(), e, want.rstd.data_ptr(), res.data_ptr(), h, d.data_ptr(),
                                  d.stride(0), dweight.data_ptr(), ws.data_ptr(), need.value, stream) == 0
    assert torch.equal(d, dx) and torch.equal(dweight, dw) and untouched(dbuf, d, 7.0) and untouched(wbuf, dweight, 7.0) and (ws[need.value:] == 0xff).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,topk", [(3, 5, 2), (9, 64, 8), (5, 130, 4), (7, 300, 5), (2, 1000, 9), (4100, 60, 6), (4097, 250, 8)])
def test_route_amid_nan(dtype, t, e, topk):
    g = B.gen(t + e)
    logits, bias, dw = rand(g, t, e, dtype=dtype), rand(g, e), rand(g, t, topk)
    nl, nb, nd = (amid(v)[1] for v in (logits, bias, dw))
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, w = ep.expert_route(logits, topk, bias=bias, score=score, renormalize=renorm)
            assert same(ep.expert_route(nl, topk, bias=nb, score=score, renormalize=renorm), (ids, w))
            d = ep.expert_route_backward(dw, logits, ids, score=score, renormalize=renorm)
            assert same((ep.expert_route_backward(nd, nl, ids, score=score, renormalize=renorm),), (d,))
            buf, out = amid(torch.zeros_like(logits), 7.0)
            assert ep.lib().ep_expert_route_backward(dw.data_ptr(), topk, t, topk, logits.data_ptr(), e, e, ELT[dtype], ids.data_ptr(), int(score == "sigmoid"),
                                                     int(renorm), 1.0, out.data_ptr(), out.stride(0), torch.cuda.current_stream().cuda_stream) == 0
            assert torch.equal(out, d) and untouched(buf, out, 7.0)


# few rows; K ranges; 128 x 128 tiles; fewer than 8 columns; short sums; 256 x 256 tiles
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(5, 130, 400), (64, 257, 4112), (100, 301, 400), (70, 7, 400), (100, 300, 240), (4200, 4099, 272)])
def test_epilogue_amid_nan(dtype, m, n, k):
    g = B.gen(m + n)
    a, b = R.operand(g, m, k).cuda(), R.operand(g, n, k).cuda()
    sa, sb = R.scales(g, m, R.blocks(k)).cuda(), R.scales(g, R.blocks(n), R.blocks(k)).cuda()
    bias, res = rand(g, n, dtype=dtype), rand(g, m, n, dtype=dtype)
    d, p = ep.matmul_fp8(a, sa, b, sb, out_dtype=dtype, bias=bias, activation="gelu", residual=res, save_pre=True)
    nb, nr = amid(bias)[1], amid(res)[1]
    assert same(ep.matmul_fp8(a, sa, b, sb, out_dtype=dtype, bias=nb, activation="gelu", residual=nr, save_pre=True), (d, p))
    obuf, out = amid(torch.zeros_like(res), 7.0)
    pbuf, pre = amid(torch.zeros_like(res), 7.0)
    need = ctypes.c_size_t()
    assert ep.lib().ep_matmul_fp8_workspace(m, n, k, ctypes.byref(need)) == 0
    ws = torch.empty(need.value + 16, dtype=torch.uint8, device="cuda")
    assert ep.lib().ep_matmul_fp8_epilog(m, n, k, a.data_ptr(), k, sa.data_ptr(), *sa.stride(), b.data_ptr(), k, sb.data_ptr(), *sb.stride(), out.data_ptr(),
                                         out.stride(0), ELT[dtype], nb.data_ptr(), ELT[dtype], 2, nr.data_ptr(), nr.stride(0), pre.data_ptr(), pre.stride(0),
                                         ws.data_ptr(), need.value, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, d) and torch.equal(pre, p) and untouched(obuf, out, 7.0) and untouched(pbuf, pre, 7.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n", [(3, 5), (128, 256), (130, 300), (257, 128), (500, 1001)])
def test_epilogue_gradient_amid_nan(dtype, m, n):
    g = B.gen(m + n)
    dout, pre = rand(g, m, n, dtype=dtype), rand(g, m, n, dtype=dtype)
    nd, np_ = amid(dout)[1], amid(pre)[1]
    for act in (None, "relu", "gelu", "silu"):
        want = ep.epilogue_backward_fp8(dout, act, pre if act else None)
        assert same(ep.epilogue_backward_fp8(nd, act, np_ if act else None), want)
    bytes_amid = lambda r, c: (lambda b: (b, b[1:-1, 3:-5]))(torch.full((r + 2, c + 8), 0x55, dtype=torch.uint8, device="cuda"))  # noqa: E731
    (qb, q), (tb, qt) = bytes_amid(m, n), bytes_amid(n, m)
    (sb, s), (ub, st), (db, dbias) = (amid(torch.zeros(k), 7.0) for k in (m * R.blocks(n), n * R.blocks(m), n))
    need = ctypes.c_size_t()
    assert ep.lib().ep_epilogue_backward_fp8_workspace(m, n, ctypes.byref(need)) == 0
    ws = torch.full((need.value + 64,), 0xff, dtype=torch.uint8, device="cuda")
    assert ep.lib().ep_epilogue_backward_fp8(dout.data_ptr(), m, n, n, ELT[dtype], 3, pre.data_ptr(), n, q.data_ptr(), n + 8, s.data_ptr(), qt.data_ptr(), m + 8,
                                             st.data_ptr(), dbias.data_ptr(), ws.data_ptr(), need.value, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(q, want.q.view(torch.uint8)) and torch.equal(qt, want.q_t.view(torch.uint8)) and torch.equal(dbias, want.dbias)
    assert torch.equal(s.view(-1, m).t(), want.scale) and torch.equal(st.view(-1, n).t(), want.scale_t)
    assert untouched(qb, q, 0x55) and untouched(tb, qt, 0x55) and untouched(sb, s, 7.0) and untouched(ub, st, 7.0) and untouched(db, dbias, 7.0)
    assert (ws[need.value:] == 0xff).all()


def spread(rows, cols):
    """bf16 values that repeat every 4096 rows, more than 2^31 of them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    part = torch.randn((4096, cols), generator=g, device="cuda").bfloat16()
    return part.repeat(-(-rows // 4096), 1)[:rows]


def test_norm_past_32_bits():
    m, h = 70000, 32768
    x = spread(m, h)
    w = torch.ones(h, device="cuda")
    out = ep.rms_norm(x, w, residual=x, quantize=True)
    dx, dw = ep.rms_norm_backward(x, out.residual, w, out.rstd, dresidual=x)
    for lo in (0, m - 37):
        part = ep.rms_norm(x[lo:lo + 37], w, residual=x[lo:lo + 37], quantize=True)
        assert same((part.y, part.residual, part.rstd, part.scale), (out.y[lo:lo + 37], out.residual[lo:lo + 37], out.rstd[lo:lo + 37], out.scale[lo:lo + 37]))
        assert torch.equal(ep.rms_norm_backward(x[lo:lo + 37], part.residual, w, part.rstd, dresidual=x[lo:lo + 37])[0], dx[lo:lo + 37])
    # dy r rstd, every 4096 rows the same
    r = out.residual[:4096].double()
    rows = torch.full((4096, 1), m // 4096, dtype=torch.float64, device="cuda")
    rows[:m % 4096] += 1
    terms = x[:4096].double() * r * out.rstd[:4096].double()[:, None] * rows
    adds = -(-m // 512) + 64 + 10
    assert ((dw.double() - terms.sum(0)).abs() <= adds * B.U * terms.abs().sum(0)).all()


def test_route_past_32_bits():
    t, e = (1 << 25) - 5, 72
    logits = spread(t, e)
    ids, w = ep.expert_route(logits, 3, score="sigmoid")
    d = ep.expert_route_backward(w, logits, ids, score="sigmoid")
    for lo in (0, t - 4097):
        i, v = ep.expert_route(logits[lo:lo + 4097], 3, score="sigmoid")
        assert torch.equal(i, ids[lo:lo + 4097]) and torch.equal(v, w[lo:lo + 4097])
        assert torch.equal(ep.expert_route_backward(v, logits[lo:lo + 4097], i, score="sigmoid"), d[lo:lo + 4097])


@pytest.mark.parametrize("k", [32, 272])
def test_epilogue_past_32_bits(k):
    m, n = 140000, 16384
    g = B.gen(k)
    a, b = R.operand(g, 4096, k).cuda().view(torch.uint8).repeat(-(-m // 4096), 1)[:m].view(R.F8), R.operand(g, n, k).cuda()
    sa, sb = torch.full((m, R.blocks(k)), 2.0 ** -10, device="cuda"), torch.full((R.blocks(n), R.blocks(k)), 2.0 ** -4, device="cuda")
    res, bias = spread(m, n), rand(B.gen(1), n)
    d, p = ep.matmul_fp8(a, sa, b, sb, bias=bias, activation="silu", residual=res, save_pre=True)
    back = ep.epilogue_backward_fp8(res, "silu", p)
    for lo in (0, m - 300):
        at = slice(lo, lo + 300)
        e, q = ep.matmul_fp8(a[at], sa[at], b, sb, bias=bias, activation="silu", residual=res[at], save_pre=True)
        assert torch.equal(e, d[at]) and torch.equal(q, p[at])
        part = ep.epilogue_backward_fp8(res[at], "silu", p[at])
        assert same((part.q, part.scale), (back.q[at], back.scale[at]))
    last = m // 128 * 128
    part = ep.epilogue_backward_fp8(res[last:], "silu", p[last:])
    assert same((part.q_t, part.scale_t), (back.q_t[:, last:], back.scale_t[:, last // 128:]))


def test_several_at_once():
    """Two streams, each with its own calls in flight, give what they give alone."""
    g = B.gen(3)
    x, res, w = rand(g, 2000, 1500, dtype=torch.bfloat16), rand(g, 2000, 1500, dtype=torch.bfloat16), rand(g, 1500)
    logits = rand(g, 6000, 256)
    pre = rand(g, 2000, 1500, dtype=torch.bfloat16)

    def work(i):
        n = ep.rms_norm(x, w, residual=res * (i + 1), quantize=True)
        ids, v = ep.expert_route(logits * (i + 1), 8, groups=8, topk_groups=4)
        return (*n, *ep.rms_norm_backward(res, n.residual, w, n.rstd), ids, v, ep.expert_route_backward(v, logits, ids), *ep.epilogue_backward_fp8(n.residual, "gelu", pre))
    alone = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append([work(i) for _ in range(3)])
        torch.cuda.synchronize()
        for i in range(2):
            assert all(same(run, alone[i]) for run in got[i])

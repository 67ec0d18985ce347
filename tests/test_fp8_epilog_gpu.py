"""The 8-bit products' epilogue (bias, activation, residual, saved pre-activation) in every kernel that carries it, and its
gradient, on the GPU against 64 bits."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _block as B
from tests import _fp8 as R
from tests._gpu import require_gpu
from tests.test_fp8_sums_gpu import cut_off

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# few rows; K ranges joined; 128 x 128 tiles; sums of at most 256 values and fewer than 8 columns (widened operands); 256 x 256 tiles
SHAPES = [(1, 5, 16), (1, 1000, 1424), (8, 257, 400), (9, 4, 528), (130, 7, 272), (64, 100, 4096), (33, 257, 4112), (300, 1000, 128), (129, 131, 256),
          (257, 513, 2064), (513, 129, 528), (777, 1003, 1040), (40, 8, 272), (4100, 4099, 272), (4096, 4352, 400)]
OPTIONS = [dict(bias=True), dict(act="relu", bias=True, pre=True), dict(act="gelu", bias=True, res=True), dict(act="silu", res=True, pre=True),
           dict(res=True), dict(act="gelu", bias=True, wide_bias=True, res=True, pre=True)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def operands(m, n, k, seed):
    g = B.gen(seed)
    a, b = R.operand(g, m, k), R.operand(g, n, k)
    return [t.cuda() for t in (a, R.scales(g, m, R.blocks(k)) * 2.0 ** -8, b, R.scales(g, R.blocks(n), R.blocks(k)) * 2.0 ** -2)]


def extras(m, n, dtype, seed, bias=False, wide_bias=False, res=False, act=None, pre=False):
    g = B.gen(seed)
    kw = {"activation": act, "save_pre": pre}
    if bias:
        kw["bias"] = torch.randn(n, generator=g).to(torch.float32 if wide_bias else dtype).cuda()
    if res:
        kw["residual"] = torch.randn((m, n), generator=g).to(dtype).cuda()
    return kw


def exact_on_gpu(a, sa, b, sb):
    x, y = R.dequantized(a, sa), R.dequantized(b, sb, 128)
    return (x @ y.t()).cpu(), (x.abs() @ y.abs().t()).cpu()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_epilogue(dtype, m, n, k):
    ops = operands(m, n, k, m + n + k)
    prod, mags = exact_on_gpu(*ops)
    for i, o in enumerate(OPTIONS if m < 1000 else OPTIONS[2:4] + OPTIONS[5:]):
        kw = extras(m, n, dtype, i, **o)
        got = ep.matmul_fp8(*ops, out_dtype=dtype, **kw)
        d, pre = got if kw["save_pre"] else (got, None)
        bias = kw["bias"].double().cpu() if "bias" in kw else torch.zeros(n, dtype=torch.float64)
        p = prod + bias
        # of P before a rounding: the product's, and the bias's addition to any of its partial sums
        err = R.product_tolerance(prod, mags + bias.abs(), k, dtype) - R.HALF_STEP[dtype] * prod.abs() + B.U * p.abs()
        if pre is not None:
            R.assert_within(pre, p, err + R.HALF_STEP[dtype] * (p.abs() + err) + R.SMALLEST[dtype], f"pre {o}")
        want = B.activation(p, kw["activation"])
        # |act'| <= 1.13
        err = 1.13 * err + B.activation_error(p, kw["activation"])
        if "residual" in kw:
            want = want + kw["residual"].double().cpu()
        err = err + B.U * want.abs()
        assert d.dtype == dtype
        R.assert_within(d, want, err + R.HALF_STEP[dtype] * (want.abs() + err) + R.SMALLEST[dtype], f"{o}")


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_fp32_results_follow_their_pre_activation(m, n, k):
    """fp32's P is not rounded: D is act(P) + residual of what is returned, to the activation's own error."""
    ops = operands(m, n, k, m + n + k)
    for act in ("relu", "gelu", "silu", None):
        kw = extras(m, n, torch.float32, 5, bias=True, res=True, act=act, pre=True)
        d, p = ep.matmul_fp8(*ops, out_dtype=torch.float32, **kw)
        p, r = p.double().cpu(), kw["residual"].double().cpu()
        want = B.activation(p, act) + r
        R.assert_within(d, want, B.activation_error(p, act) + 2 * B.U * (want.abs() + r.abs()) + 2.0 ** -140, str(act))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_an_epilogue_of_nothing_is_the_product(dtype, m, n, k):
    """Zeros as bias and residual, and the saved P, change no bit.  In fp16 a value's last multiply-add can be rounded
    to fp16 at once (v_fma_mixlo_f16) where nothing follows it, and to fp32 first where something does: both are roundings
    of values within 2^-24 of each other, so they are the same or neighbours, a step of 2^-10 (subnormal 2^-24) apart."""
    ops = operands(m, n, k, 3)
    want = ep.matmul_fp8(*ops, out_dtype=dtype)
    z = lambda *s: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    d, p = ep.matmul_fp8(*ops, out_dtype=dtype, bias=z(n), residual=z(m, n), save_pre=True)
    assert torch.equal(d, p)
    if dtype == torch.float16:
        assert ((p.double() - want.double()).abs() <= 2.0 ** -10 * want.double().abs() + 2.0 ** -24).all()
    else:
        assert torch.equal(p, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(3, 70, 400), (64, 150, 4096), (200, 150, 272), (200, 151, 528), (4096, 4104, 272)])
def test_strides_and_the_residual_as_output(dtype, m, n, k):
    """Residual and output as parts of larger buffers; the residual overwritten by the result; what lies around stays."""
    ops = operands(m, n, k, 9)
    kw = extras(m, n, dtype, 2, bias=True, res=True, act="gelu")
    want = ep.matmul_fp8(*ops, out_dtype=dtype, **kw)
    buf = torch.full((m, n + 11), 7.0, dtype=dtype, device="cuda")
    part = buf[:, 5:5 + n]
    got = ep.matmul_fp8(*ops, out_dtype=dtype, out=part, **kw)
    assert got is part and torch.equal(part, want)
    part.copy_(kw["residual"])
    ep.matmul_fp8(*ops, out_dtype=dtype, out=part, **{**kw, "residual": part})
    assert torch.equal(part, want) and (buf[:, :5] == 7).all() and (buf[:, 5 + n:] == 7).all()
    with pytest.raises(ValueError, match="out lies over an input"):
        ep.matmul_fp8(*ops, out_dtype=dtype, out=buf[:, 4:4 + n], **{**kw, "residual": part})


@pytest.mark.parametrize("m,n,k", [(2, 70, 144), (64, 150, 4096), (100, 70, 144), (300, 200, 528)])
def test_special_values(m, n, k):
    """NaN in an operand's row, infinities and NaN in the bias and the residual stay in their rows and columns; relu takes
    NaN to 0, as the 16-bit epilogues do."""
    ops = operands(m, n, k, 4)
    ops[0].view(torch.uint8)[1, k - 1] = 0x7f
    kw = extras(m, n, torch.bfloat16, 2, bias=True, res=True)
    kw["bias"][3], kw["bias"][9] = float("inf"), float("-inf")
    kw["residual"][0, 5] = float("nan")
    d = ep.matmul_fp8(*ops, **kw)
    assert d[1].isnan().all() and d[0, 5].isnan()
    rest = torch.ones((m, n), dtype=torch.bool, device="cuda")
    rest[1], rest[:, 3], rest[:, 9], rest[0, 5] = False, False, False, False
    assert d[rest].isfinite().all() and d[0, 3] == float("inf") and d[0, 9] == float("-inf")
    d, p = ep.matmul_fp8(*ops, bias=kw["bias"], activation="relu", save_pre=True)
    assert p[1].isnan().all() and not d[1].any() and d[0, 3] == float("inf") and d[0, 9] == 0
    d = ep.matmul_fp8(*ops, bias=kw["bias"], activation="gelu")
    assert d[1].isnan().all() and d[0, 3] == float("inf") and d[0, 9] == 0


# ------------------------------------------------------------------------------------- gradients
GRAD_SHAPES = [(1, 1), (1, 300), (5, 128), (16, 16), (127, 129), (128, 128), (130, 1003), (300, 72), (700, 640), (1100, 5)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n", GRAD_SHAPES)
def test_gradient_operands_of_exact_gradients(dtype, m, n):
    """Without an activation, and with relu, the gradient has no rounding: both quantisations are quantize_fp8's, bit for bit."""
    g = B.gen(m + n)
    dout = (torch.randn((m, n), generator=g) * torch.exp2(torch.randint(-6, 7, (m, n), generator=g).float())).to(dtype).cuda()
    pre = torch.randn((m, n), generator=g).to(dtype).cuda()
    for act in (None, "relu"):
        got = ep.epilogue_backward_fp8(dout, activation=act, pre=pre if act else None)
        d = dout if act is None else torch.where(pre > 0, dout, torch.zeros((), dtype=dtype, device="cuda"))
        for (q, s), (wq, ws) in ((got[:2], ep.quantize_fp8(d)), (got[2:4], ep.quantize_fp8(d, transpose=True))):
            assert torch.equal(q.view(torch.uint8) & 0x7f, wq.view(torch.uint8) & 0x7f) and torch.equal(q.float(), wq.float())
            assert torch.equal(s, ws) and s.stride() == ws.stride()
        x = d.double().cpu()
        # 4 rows of a thread, the lanes', the waves', 8 groups of the blocks of 128 rows
        adds = 4 + 3 + 2 + -(-R.blocks(m) // 8) + 8
        R.assert_within(got.dbias, x.sum(0), adds * B.U * x.abs().sum(0) + 2.0 ** -140)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("m,n", GRAD_SHAPES)
def test_gradient_operands(dtype, act, m, n):
    g = B.gen(m * 3 + n)
    dout, pre = torch.randn((m, n), generator=g).to(dtype), (2 * torch.randn((m, n), generator=g)).to(dtype)
    got = ep.epilogue_backward_fp8(dout.cuda(), activation=act, pre=pre.cuda())
    d = dout.double() * B.activation_grad(pre.double(), act)
    err = dout.double().abs() * B.activation_grad_error(pre.double(), act) + B.U * d.abs()
    for q, s, x, e in ((got.q, got.scale, d, err), (got.q_t, got.scale_t, d.t(), err.t())):
        rows, cols = x.shape
        split = lambda v: torch.nn.functional.pad(v, (0, R.blocks(cols) * 128 - cols)).view(rows, -1, 128)  # noqa: E731
        amax = split(x.abs()).amax(2).clamp_min(R.AMAX_MIN)
        s = s.double().cpu()
        assert ((s - amax / 448).abs() <= (split(e).amax(2) + B.U * amax) / 448 * 1.01).all()
        wide = s.repeat_interleave(128, 1)[:, :cols]
        R.assert_within(q.double().cpu() * wide, x, 1.01 * (2.0 ** -4 * x.abs() + 2.0 ** -10 * wide) + 2 * e + 8 * B.U * x.abs())
    adds = 4 + 3 + 2 + -(-R.blocks(m) // 8) + 8
    R.assert_within(got.dbias, d.sum(0), adds * B.U * d.abs().sum(0) + 1.01 * err.sum(0))


def test_gradient_strides_and_special_values():
    g = B.gen(1)
    wide, wide_pre = torch.randn((150, 310), generator=g).bfloat16().cuda(), torch.randn((150, 310), generator=g).bfloat16().cuda()
    dout, pre = wide[:, 3:260], wide_pre[:, 7:264]
    for a, b in zip(ep.epilogue_backward_fp8(dout, "gelu", pre), ep.epilogue_backward_fp8(dout.contiguous(), "gelu", pre.contiguous())):
        assert torch.equal(a.float(), b.float())
    clean = ep.epilogue_backward_fp8(dout, "relu", pre.abs())
    dout[5, 9], dout[7, 200] = float("nan"), float("inf")
    pre2 = pre.abs()
    pre2[20, 30], pre2[21, 31] = float("nan"), -1.0
    dout[21, 31] = float("inf")  # (behind relu's zero)
    d = ep.epilogue_backward_fp8(dout, "relu", pre2)
    q = d.q.float()
    assert q[5, 9].isnan() and q[7, 200].isnan() and q[20, 30] == 0 and q[21, 31] == 0 and int(q.isnan().sum()) == 2
    assert torch.equal(d.q_t.float().isnan(), q.isnan().t()) and d.scale.isfinite().all() and d.scale_t.isfinite().all()
    keep = [c for c in range(257) if c not in (9, 200, 30, 31)]
    assert torch.equal(d.dbias[keep], clean.dbias[keep]) and d.dbias[9].isnan() and d.dbias[31].isfinite()


def test_gradients_against_differences():
    """dbias of f = sum of dout (act(p + bias) + residual), along every column, in 64 bits."""
    g = B.gen(2)
    dout, pre = torch.randn((140, 60), generator=g), torch.randn((140, 60), generator=g)
    for act in ("gelu", "silu"):
        db = ep.epilogue_backward_fp8(dout.cuda(), act, pre.cuda()).dbias.double().cpu()
        f = lambda e: (dout.double() * B.activation(pre.double() + e, act)).sum(0)  # noqa: E731
        want = (f(1e-4) - f(-1e-4)) / 2e-4
        assert ((db - want).abs() <= 1e-6 * dout.double().abs().sum(0)).all()


def test_gradient_empty():
    d = ep.epilogue_backward_fp8(torch.zeros((0, 40), device="cuda"))
    assert d.q.shape == (0, 40) and d.q_t.shape == (40, 0) and d.scale.shape == (0, 1) and d.scale_t.shape == (40, 0) and not d.dbias.any()


def test_graph_and_streams():
    m, n, k = 300, 520, 4112
    ops = operands(m, n, k, 6)
    kw = extras(m, n, torch.bfloat16, 2, bias=True, res=True, act="silu", pre=True)
    few = operands(4, n, k, 7)
    fkw = extras(4, n, torch.bfloat16, 2, bias=True, res=True, act="silu")
    d, p = ep.matmul_fp8(*ops, **kw)
    f = ep.matmul_fp8(*few, **fkw)
    e = ep.epilogue_backward_fp8(d, "silu", p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        d2, p2 = ep.matmul_fp8(*ops, **kw)
        f2 = ep.matmul_fp8(*few, **fkw)
        e2 = ep.epilogue_backward_fp8(d2, "silu", p2)
    for _ in range(3):
        for t in (d2, p2, f2, e2.dbias, e2.scale_t):
            t.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        d3, p3 = ep.matmul_fp8(*ops, stream=torch.cuda.Stream(), **kw)
        torch.cuda.synchronize()
        assert torch.equal(d2, d) and torch.equal(p2, p) and torch.equal(f2, f) and torch.equal(d3, d) and torch.equal(p3, p)
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(e2, e))


@pytest.mark.parametrize("dtype", DTYPES[:2])
@pytest.mark.parametrize("m,n,k", [(300, 640, 528), (2049, 320, 272), (129, 64, 400), (4100, 4160, 272)])
def test_whole_lines_and_shared_ones(dtype, m, n, k):
    """Rows of whole 128-byte lines, which are stored in another way than rows that share lines: right, and the same bits.

    16-bit tiles take the matrix instruction's sums: in each group of 8 neighbouring k at most 7 products are cut off, each by
    less than 2^(E - 13), 2^E the group's largest product of powers of two.  That is in none of product_tolerance's terms, which count
    fp32 roundings, and among 17 million cancelling sums one is seen: 1.4e-5 of magnitudes 1.5e-2 is off by 3.6e-7, where
    (128 + 2 + 6 + 16) 2^-23 of 1.5e-2 is 2.8e-7, and the plain product's value is the same.  So cut_off is added."""
    ops = operands(m, n, k, m + n + k)
    prod, mags = exact_on_gpu(*ops)
    cut = cut_off(*ops).cpu()
    for i, o in enumerate(OPTIONS[2:4] + OPTIONS[5:]):
        kw = extras(m, n, dtype, i, **o)
        got = ep.matmul_fp8(*ops, out_dtype=dtype, **kw)
        d, pre = got if kw["save_pre"] else (got, None)
        bias = kw["bias"].double().cpu() if "bias" in kw else torch.zeros(n, dtype=torch.float64)
        p = prod + bias
        err = R.product_tolerance(prod, mags + bias.abs(), k, dtype) - R.HALF_STEP[dtype] * prod.abs() + B.U * p.abs() + cut
        if pre is not None:
            R.assert_within(pre, p, err + R.HALF_STEP[dtype] * (p.abs() + err) + R.SMALLEST[dtype], f"pre {o}")
        want = B.activation(p, kw["activation"]) + kw["residual"].double().cpu()
        err = 1.13 * err + B.activation_error(p, kw["activation"]) + B.U * want.abs()
        R.assert_within(d, want, err + R.HALF_STEP[dtype] * (want.abs() + err) + R.SMALLEST[dtype], f"{o}")
    ops = operands(m, n, k, 5)
    kw = extras(m, n, dtype, 1, bias=True, res=True, act="silu", pre=True)
    d, p = ep.matmul_fp8(*ops, out_dtype=dtype, **kw)
    for step, at in ((n + 8, 0), (n + 64, 8), (n + 5, 3), (n + 64, 64)):
        buf = torch.full((m, step), 7.0, dtype=dtype, device="cuda")
        out = buf[:, at:at + n] if at + n <= step else buf[:, :n]
        e, q = ep.matmul_fp8(*ops, out_dtype=dtype, out=out, **kw)
        assert torch.equal(e, d) and torch.equal(q, p)
        out.fill_(7.0)
        assert (buf == 7.0).all()

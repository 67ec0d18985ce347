"""Routing to experts on the GPU against lists in 64 bits: choices exactly, weights and gradients within fp32's bounds."""
import math

import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _block as B
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def check_route(logits, topk, **kw):
    ids, w = ep.expert_route(logits.cuda(), topk, **{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
    want, ww = B.route(logits, topk, **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32 and ids.shape == w.shape == (logits.shape[0], topk)
    assert torch.equal(ids.cpu(), want)
    R.assert_within(w, ww, B.SCORE_TOLERANCE * ww.abs() + 2.0 ** -140)
    return ids, w


CASES = [  # T, E, topk, options
    (1, 1, 1, {}), (1, 64, 8, {}), (7, 8, 8, {}), (3, 60, 6, {}), (65, 64, 2, {"renormalize": False}), (33, 100, 64, {}), (9, 128, 4, {"score": "sigmoid"}),
    (5, 130, 3, {"score": "sigmoid", "renormalize": False, "scale": 2.5}), (17, 256, 8, {"bias": 1}),
    (17, 256, 8, {"score": "sigmoid", "bias": 1, "groups": 8, "topk_groups": 4}), (11, 160, 6, {"groups": 8, "topk_groups": 3, "group_top": 1}),
    (6, 300, 5, {"groups": 3, "topk_groups": 2, "bias": 1}), (4, 512, 7, {"bias": 1, "score": "sigmoid", "renormalize": False}), (3, 1000, 10, {"scale": -1.0}),
    (2, 1024, 64, {"groups": 64, "topk_groups": 9, "score": "sigmoid"}), (5, 96, 4, {"groups": 96 // 3 // 4, "topk_groups": 1}), (8, 64, 8, {"groups": 64, "topk_groups": 8})]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,topk,kw", CASES)
def test_route(dtype, t, e, topk, kw):
    g = B.gen(t * 31 + e + topk)
    logits = (2 * torch.randn((t, e), generator=g)).clamp(-8, 8).to(dtype)
    kw = dict(kw)
    if "bias" in kw:
        kw["bias"] = 0.1 * torch.randn(e, generator=g)
    check_route(logits, topk, **kw)


@pytest.mark.parametrize("kw", [{}, {"score": "sigmoid"}, {"groups": 4, "topk_groups": 2}, {"score": "sigmoid", "groups": 8, "topk_groups": 3, "group_top": 1}])
def test_equal_keys_go_to_the_lowest_index(kw):
    logits = torch.randint(-1, 2, (200, 96), generator=B.gen(1)).to(torch.bfloat16)
    check_route(logits, 7, **kw)
    check_route(torch.zeros((3, 96)), 12, **kw)


@pytest.mark.parametrize("kw", [{}, {"renormalize": False}, {"score": "sigmoid"}, {"bias": 1}, {"score": "sigmoid", "bias": 1, "groups": 4, "topk_groups": 2},
                                {"groups": 4, "topk_groups": 3, "group_top": 1}])
def test_masked_experts(kw):
    """Logits of -infinity and NaN: whole tokens, whole groups, all but a few; infinite ones and the types' ends."""
    g = B.gen(2)
    logits = torch.randn((12, 64), generator=g)
    kw = dict(kw)
    if "bias" in kw:
        kw["bias"] = 0.1 * torch.randn(64, generator=g)
        kw["bias"][7], kw["bias"][20], kw["bias"][21] = -math.inf, math.nan, 3.0
    logits[0] = -math.inf
    logits[1] = math.nan
    logits[2, 5:] = -math.inf
    logits[3, ::2] = -math.inf
    logits[4, :16] = math.nan
    logits[5, 1:] = -math.inf
    logits[6, 9] = math.nan
    logits[7, 3] = math.inf
    logits[8, 40], logits[8, 3] = math.inf, math.inf
    logits[9] = torch.finfo(torch.float32).min
    logits[10, 30] = torch.finfo(torch.float32).max
    logits[11, 16:32] = -math.inf
    ids, w = check_route(logits, 6, **kw)
    assert (ids[:2] == -1).all() and not w[:2].any() and w.isfinite().all()
    order = ep.expert_order(ids, 64)
    assert (order.pos[:2] == -1).all()


@pytest.mark.parametrize("t,e,topk,kw", [(5, 900, 7, {"groups": 3, "topk_groups": 2}), (4, 1023, 9, {"groups": 33, "topk_groups": 5, "score": "sigmoid", "bias": 1}),
                                         (3, 770, 3, {"groups": 5, "topk_groups": 1, "group_top": 1}), (4100, 300, 4, {"groups": 3, "topk_groups": 1})])
def test_groups_that_do_not_divide_a_wave(t, e, topk, kw):
    """Up to 32 experts a lane; equal and masked ones among them."""
    g = B.gen(e)
    logits = (2 * torch.randn((t, e), generator=g)).clamp(-8, 8)
    logits[1] = logits[1].round()
    logits[2, ::3] = -math.inf
    kw = dict(kw)
    if "bias" in kw:
        kw["bias"] = 0.1 * torch.randn(e, generator=g)
    check_route(logits, topk, **kw)


@pytest.mark.parametrize("t", [3, 5000])
def test_zeros_of_either_sign_are_equal(t):
    logits = torch.zeros((t, 40))
    logits[:, ::2] = -0.0
    ids, _ = check_route(logits, 5)
    assert (ids.cpu() == torch.arange(5)).all()
    ids, _ = check_route(logits, 5, score="sigmoid", bias=-0.5 * torch.ones(40))  # (keys of 0)
    assert (ids.cpu() == torch.arange(5)).all()


@pytest.mark.parametrize("t", [6, 4200])
def test_keys_that_fp32_makes_equal(t):
    """Neighbours far closer than fp32's step, in every order, inside and at the end of the choice: decided in double."""
    logits = torch.full((t, 48), 20.0)  # sigmoid: 1 - 2e-9, the others' differences are below 2e-9
    for i in range(t):
        logits[i, torch.randperm(48, generator=B.gen(i))] = 18 + 6 * torch.arange(48) / 48
    check_route(logits, 6, score="sigmoid", bias=torch.zeros(48))
    check_route(logits, 6, score="sigmoid", groups=4, topk_groups=2)
    check_route(logits, 48, score="sigmoid", bias=torch.zeros(48))


def test_far_logits():
    """Scores that underflow in fp32 still decide: keys are in double, and no weight is NaN."""
    logits = torch.tensor([[-200.0, -201.0, -199.0, -300.0], [30.0, 31.0, 32.0, 29.0], [200.0, -200.0, 0.0, 1.0], [-4000.0, -4001.0, -3999.0, -4002.0]])
    for kw in ({"score": "sigmoid"}, {}, {"score": "sigmoid", "bias": torch.zeros(4)}):
        ids, w = ep.expert_route(logits.cuda(), 2, **{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
        want, ww = B.route(logits, 2, **kw)
        assert torch.equal(ids.cpu(), want) and not w.isnan().any()
        assert ((w.cpu() - ww).abs() <= 2.0 ** -15 * ww + 2.0 ** -140).all()  # (e^200: the argument's rounding, 200 2^-24)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e,topk,kw", [
    (8, 2, {}), (60, 6, {"score": "sigmoid"}), (64, 16, {"bias": 1}), (64, 17, {}), (128, 4, {"score": "sigmoid", "groups": 8, "topk_groups": 3}),
    (160, 6, {"groups": 8, "topk_groups": 4, "group_top": 1}), (256, 8, {"score": "sigmoid", "bias": 1, "groups": 8, "topk_groups": 4}), (256, 33, {"bias": 1}),
    (200, 20, {"score": "sigmoid", "renormalize": False}), (384, 8, {"groups": 8, "topk_groups": 4})])
def test_many_tokens(dtype, e, topk, kw):
    """As many as share a wave, the last one not full; among them tokens of equal, masked and infinite logits."""
    t = 4099
    g = B.gen(e + topk)
    logits = (2 * torch.randn((t, e), generator=g)).clamp(-8, 8)
    logits[::7] = logits[::7].round()
    logits[5::50, e // 3:] = -math.inf
    logits[6::90] = math.nan
    logits[7::90, 3] = math.inf
    logits = logits.to(dtype)
    kw = dict(kw)
    if "bias" in kw:
        kw["bias"] = 0.1 * torch.randn(e, generator=g)
    ids, w = check_route(logits, topk, **kw)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    few = [ep.expert_route(logits[i:i + 1000].cuda(), topk, **dev) for i in range(0, t, 1000)]
    assert torch.equal(torch.cat([f[0] for f in few]), ids)


def test_rows_of_wider_buffers():
    wide = torch.randn((9, 80), generator=B.gen(3)).to(torch.float16).cuda()
    x = wide[:, 5:65]
    for a, b in zip(ep.expert_route(x, 4), ep.expert_route(x.contiguous(), 4)):
        assert torch.equal(a, b)
    ids, w = ep.expert_route(x, 4)
    dw = torch.randn((9, 6), generator=B.gen(4)).cuda()[:, 1:5]
    assert torch.equal(ep.expert_route_backward(dw, x, ids), ep.expert_route_backward(dw.contiguous(), x.contiguous(), ids))


def test_empty():
    ids, w = ep.expert_route(torch.zeros((0, 8), device="cuda"), 2)
    assert ids.shape == w.shape == (0, 2)
    assert ep.expert_route_backward(w, torch.zeros((0, 8), device="cuda"), ids).shape == (0, 8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,topk,kw", [c for c in CASES])
def test_route_backward(dtype, t, e, topk, kw):
    g = B.gen(t * 17 + e)
    logits = (2 * torch.randn((t, e), generator=g)).clamp(-8, 8).to(dtype)
    dw = torch.randn((t, topk), generator=g)
    kw = {k: v for k, v in kw.items() if k in ("score", "renormalize", "scale")}
    kw = {"score": "softmax", "renormalize": True, "scale": 1.0, **kw}
    ids, _ = B.route(logits, topk, score=kw["score"])
    if t > 2 and topk > 1:
        ids[1, 1] = -1  # a choice that was dropped
    d = ep.expert_route_backward(dw.cuda(), logits.cuda(), ids.cuda(), **kw)
    l = logits.double().requires_grad_()
    want, = torch.autograd.grad(B.route_weights(l, ids, **kw), l, dw.double())
    # what the terms of a gradient add up to: |w_j| |s| |dw| of every pair
    w = B.route_weights(logits.double(), ids, **kw).abs()
    size = torch.zeros_like(want).scatter_add_(1, ids.long().clamp_min(0), w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True) / abs(kw["scale"])))
    size = size + B.scores(logits, kw["score"]) * (w * dw.abs()).sum(1, keepdim=True) * (not kw["renormalize"])
    assert d.dtype == dtype
    tol = B.SCORE_TOLERANCE * size + R.HALF_STEP[dtype] * want.abs() * 1.01 + R.SMALLEST[dtype]
    tol = tol + 2.0 ** -45 * dw.abs().sum(1, keepdim=True)  # (the 64-bit form's own)
    R.assert_within(d, want, tol)


@pytest.mark.parametrize("kw", [{"score": s, "renormalize": r} for s in ("softmax", "sigmoid") for r in (False, True)])
def test_gradient_against_differences(kw):
    g = B.gen(9)
    logits = torch.randn((13, 70), generator=g)
    ids, _ = ep.expert_route(logits.cuda(), 5, **kw)
    dw = torch.randn((13, 5), generator=g)
    d = ep.expert_route_backward(dw.cuda(), logits.cuda(), ids, scale=1.5, **kw).double().cpu()
    f = lambda l: (B.route_weights(l, ids.cpu(), kw["score"], kw["renormalize"], 1.5) * dw.double()).sum()  # noqa: E731
    for _ in range(4):
        v = torch.randn(logits.shape, generator=g).double()
        want = (f(logits.double() + 1e-4 * v) - f(logits.double() - 1e-4 * v)) / 2e-4
        assert abs((d * v).sum() - want) <= 1e-5 * (d * v).abs().sum()


def test_gradient_of_masked_and_repeated_choices():
    """A token of dropped choices has none; masked experts have zeros; an expert given twice counts twice."""
    logits = torch.randn((4, 20), generator=B.gen(5))
    logits[0] = -math.inf
    logits[1, 3:9] = -math.inf
    logits[2, 4] = math.nan
    ids = torch.tensor([[-1, -1, -1], [0, 12, 25], [7, 7, 1], [2, -5, 2]], dtype=torch.int32)
    dw = torch.randn((4, 3), generator=B.gen(6))
    for score in ("softmax", "sigmoid"):
        d = ep.expert_route_backward(dw.cuda(), logits.cuda(), ids.cuda(), score=score, renormalize=False).cpu()
        assert not d[0].any() and not d[1, 3:9].any() and d[2, 4] == 0 and d.isfinite().all()
        l = torch.where(logits.isnan(), -math.inf, logits)[1:].double().requires_grad_()
        inside = torch.where((ids >= 0) & (ids < 20), ids, -1)[1:]
        want, = torch.autograd.grad(B.route_weights(l, inside, score, False, 1.0), l, dw[1:].double())
        R.assert_within(d[1:], want, B.SCORE_TOLERANCE * (want.abs() + dw.abs().sum(1)[1:, None] * B.scores(logits, score)[1:]) + 2.0 ** -140)


def test_graph_and_streams():
    g0 = B.gen(7)
    logits, dw = torch.randn((500, 256), generator=g0).cuda(), torch.randn((500, 8), generator=g0).cuda()
    kw = dict(score="sigmoid", groups=8, topk_groups=4, bias=(0.1 * torch.randn(256, generator=g0)).cuda())
    ids, w = ep.expert_route(logits, 8, **kw)
    d = ep.expert_route_backward(dw, logits, ids, score="sigmoid")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        i2, w2 = ep.expert_route(logits, 8, **kw)
        d2 = ep.expert_route_backward(dw, logits, i2, score="sigmoid")
    for _ in range(3):
        i2.fill_(5)
        d2.fill_(5)
        torch.cuda.synchronize()
        g.replay()
        i3, w3 = ep.expert_route(logits, 8, stream=torch.cuda.Stream(), **kw)
        torch.cuda.synchronize()
        assert torch.equal(i2, ids) and torch.equal(w2, w) and torch.equal(d2, d) and torch.equal(i3, ids) and torch.equal(w3, w)

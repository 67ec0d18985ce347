"""Grouped 8-bit products whose offsets do not ascend or leave the rows: an offset outside the rows counts as the
nearer end and one below an earlier one as that one, in every kernel, so each row has one group at most and nothing
outside the output is written.  Operands are exact in every step (small whole numbers, scales that are powers of
two): outputs equal the exact result rounded once, bit for bit."""
import pytest
import torch

import dense_gemm_epilogues_amd as ep
from tests import _fp8 as R
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

# rows, experts, columns: few rows; 128 x 128 tiles, one and several columns of them; 256 x 256 tiles
KERNELS = {"rows": (250, 130, 100), "tiles_128": (4000, 130, 100), "tiles_128_wide": (1500, 70, 700), "tiles_256": (6000, 5, 4300)}


def offsets(kind, rows, experts, g):
    if kind == "alternating":  # every second group would be the whole of the rows
        off = [0 if i % 2 == 0 else rows for i in range(experts + 1)]
    elif kind == "falling":
        off = [rows - i * rows // experts for i in range(experts + 1)]
    elif kind == "outside":
        off = [(-5, 2 ** 31 - 1, -2 ** 31, rows + 7)[i % 4] for i in range(experts + 1)]
    else:  # ascending but for some
        off = (torch.arange(experts + 1) * (rows - 3) // experts)
        at = torch.randint(1, experts + 1, (max(experts // 6, 2),), generator=g)
        off[at] = torch.randint(-9, rows + 9, (at.numel(),), generator=g)
        off = off.tolist()
    return off


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["mixed", "falling", "outside", "alternating"])
@pytest.mark.parametrize("kernel", KERNELS)
def test_each_row_has_one_group_at_most(kernel, kind, dtype):
    require_gpu()
    rows, e, n = KERNELS[kernel]
    k, pad = 384, 40
    g = torch.Generator()
    g.manual_seed(rows)
    off = offsets(kind, rows, e, g)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g).float().to(R.F8)  # noqa: E731
    powers = lambda *s: torch.exp2(torch.randint(-1, 2, s, generator=g).float())  # noqa: E731
    a, b = whole(rows, k).cuda(), whole(e, n, k).cuda()
    sa, sb = powers(rows, 3).cuda(), powers(e, R.blocks(n), 3).cuda()
    buf = torch.full((rows + 2 * pad, n), 7.0, dtype=dtype, device="cuda")
    ep.grouped_matmul_fp8(a, sa, b, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=dtype, out=buf[pad:pad + rows])
    assert (buf[:pad] == 7).all() and (buf[pad + rows:] == 7).all()
    ends = torch.tensor(off).clamp(0, rows).cummax(0).values.tolist()
    x = R.dequantized(a, sa)
    for i in range(e):
        at = slice(ends[i], ends[i + 1])
        if at.start < at.stop:
            want = (x[at] @ R.dequantized(b[i], sb[i], 128).t()).to(dtype)
            assert torch.equal(buf[pad:pad + rows][at], want), f"expert {i}, rows {at.start} to {at.stop}"
    assert not buf[pad + ends[-1]:pad + rows].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n", [(48, 80), (1100, 4100)])
def test_empty_group_off_the_blocks_has_a_zero_gradient(m, n, dtype):
    """Next to groups whose gradient is NaN because they start or end off the scale blocks."""
    require_gpu()
    g = torch.Generator()
    g.manual_seed(m)
    rows, off = 512, [0, 0, 128, 200, 200, 200, 256, 512, 512, 300]
    operand = lambda *s: R.operand(g, *s).cuda()  # noqa: E731
    d = ep.grouped_wgrad_fp8(operand(m, rows), R.scales(g, m, 4).cuda(), operand(n, rows), R.scales(g, R.blocks(n), 4).cuda(),
                             torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=dtype)
    for i in (0, 3, 4, 7, 8):
        assert not d[i].any(), f"group {i}"
    assert d[2].isnan().all() and d[5].isnan().all()
    assert d[1].isfinite().all() and d[1].any() and d[6].isfinite().all() and d[6].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("experts", [64, 300])
def test_few_rows_all_on_one_expert(experts, dtype):
    """As many rows as the few-row kernel takes (4 an expert), on the first, one in the middle or the last expert."""
    require_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(experts)
    rows, n, k = 4 * experts, 130, 656
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float().to(R.F8)  # noqa: E731
    a, b = whole(rows, k), whole(experts, n, k)
    sa, sb = torch.full((rows, 6), 0.5, device="cuda"), torch.full((experts, 2, 6), 2.0, device="cuda")
    for one in (0, experts // 2, experts - 1):
        off = torch.tensor([0] * (one + 1) + [rows] * (experts - one), dtype=torch.int32, device="cuda")
        d = ep.grouped_matmul_fp8(a, sa, b, sb, off, out_dtype=dtype)
        assert torch.equal(d, (R.dequantized(a, sa) @ R.dequantized(b[one], sb[one], 128).t()).to(dtype)), f"expert {one}"

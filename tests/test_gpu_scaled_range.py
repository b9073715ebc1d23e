"""The block-scaled product at the ends of its scales' range: products of two
scales beyond fp32, where the results are not; one scale huge, the other tiny;
products below fp32's normal numbers.

Bound: the sums' (2 k + 8) u of the terms' sizes (and, on the 8-bit matrix
instruction, its cuts), C's rounding, and 2^-124 per block, which the header
allows for products of scales below 2^-126.
"""
import pytest
import torch

import all_gather_gemm_agmm_amd as agmm
from test_gpu_scaled import HALF_ULP, operand, spread64
from test_gpu_scaled_sums import cuts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


M, K, N = 150, 520, 140     # five blocks of k


def keep_one(x, block, column):
    """Block `block` of x: zeros but for `column`."""
    part = x.values[:, 128 * block:128 * block + 128]
    one = part[:, column].clone()
    part.zero_()
    part[:, column] = one


def operands(kind, fmt, block):
    a, b = operand(M, K, fmt, 1, 71), operand(N, K, "e4m3", block, 72)
    sa, sb = a.scales, b.scales
    if kind == "nothing meets":             # scales of 2^100 and 2^60 where every product is 0
        keep_one(a, 1, 3)
        keep_one(b, 1, 4)
        sa[1, ::3], sb[1] = 2.0 ** 100, 2.0 ** 60
    elif kind == "smallest values meet":    # 2^70 * 2^70 * 2^-18 (e5m2: 2^-25)
        keep_one(a, 2, 9)
        keep_one(b, 2, 9)
        a.values.view(torch.uint8)[:, 2 * 128 + 9] = 1
        b.values.view(torch.uint8)[:, 2 * 128 + 9] = 1
        sa[2, 1::2], sb[2] = 2.0 ** 70, 2.0 ** 70
    elif kind == "lopsided":                # 2^-60 and 2^119; 2^110 and 2^-100
        sa[0], sb[0] = 2.0 ** -60, 2.0 ** 119
        sa[3, ::2], sb[3] = 2.0 ** 110, 2.0 ** -100
    else:                                   # sums near 2^-120 of products of scales near 2^-140
        sa[:], sb[:] = 2.0 ** -70 * (sa * 8).clamp(0.5, 1), 2.0 ** -70
    return a, b


@pytest.mark.parametrize("kind", ["nothing meets", "smallest values meet", "lopsided", "small"])
@pytest.mark.parametrize("tile", [0, 1, 2, 3])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("c_dtype", [agmm.AGMM_BF16, agmm.AGMM_FP32])
def test_ends_of_the_range(kind, tile, splits, fmt, block, c_dtype):
    a, b = operands(kind, fmt, block)
    with agmm.ScaledPlan(1, M, K, N, fmt, block, c_dtype, tile=tile, splits=splits) as plan:
        C = plan.run([a], b)
        torch.cuda.synchronize()
    x, y = spread64(a), spread64(b)
    ref, size = x @ y.t(), x.abs() @ y.abs().t()
    bound = (2 * K + 8) * 2.0 ** -24 * size + 5 * 2.0 ** -124
    if tile == 0:
        bound = bound + cuts(a, b, fmt)
    bound = bound + HALF_ULP[c_dtype] * (ref.abs() + bound) * (1 + 2.0 ** -7)
    assert ref.abs().max() < 2.0 ** 127
    assert torch.isfinite(C).all()
    err = (C.cpu().double() - ref).abs()
    assert (err <= bound).all(), ((err - bound).max().item(), err.max().item())


@pytest.mark.parametrize("tile", [0, 1, 2, 3])
@pytest.mark.parametrize("block", [1, 128])
def test_results_without_a_number_stay_so(tile, block):
    """NaN values and infinite scales still give NaN, results beyond fp32 an
    infinity, beside elements that are computed anew."""
    a, b = operands("nothing meets", "e4m3", block)
    a.values.view(torch.uint8)[7, 300] = 0x7F          # NaN
    a.scales[3, 9] = float("inf")
    a.scales[4], b.scales[4] = 2.0 ** 90, 2.0 ** 90    # the last block, of 8: every result beyond fp32
    a.values.view(torch.uint8)[:, 512:520] = 0x38      # 1.0
    b.values.view(torch.uint8)[:, 512:520] = 0x38
    a.scales[4, 100:] = 1.0                            # but for these rows
    b.scales[4] = 2.0 ** 90
    with agmm.ScaledPlan(1, M, K, N, "e4m3", block, agmm.AGMM_FP32, tile=tile) as plan:
        C = plan.run([a], b).cpu()
    assert torch.isnan(C[7]).all()
    assert (torch.isnan(C[9]) | torch.isinf(C[9])).all()
    keep = torch.ones(M, dtype=torch.bool)
    keep[[7, 9]] = False
    assert (C[:100][keep[:100]] == float("inf")).all()
    assert torch.isfinite(C[100:]).all() and (C[100:] > 2.0 ** 92).all()

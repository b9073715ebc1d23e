"""Sizes whose products pass 64 bits, on the host: refused, not wrapped."""
import pytest

import all_gather_gemm_agmm_amd as agmm


@pytest.mark.parametrize("ms", [1 << 30, 1 << 57, 1 << 58, (1 << 58) + 1, (1 << 63) - 1])
def test_matmul_plan(ms):
    """64 * 2^58 is 0 in 64 bits, 64 * (2^58 + 1) is 64."""
    lib = agmm.load_library()
    assert lib.agmm_plan_validate(64, ms, 8, 8, agmm.AGMM_BF16, 0) == agmm.AGMM_ERR_UNSUPPORTED
    assert "too large" in agmm.agmm_last_error()
    assert lib.agmm_plan_validate(1, 8, ms, 8, agmm.AGMM_BF16, 0) == agmm.AGMM_ERR_UNSUPPORTED
    assert lib.agmm_plan_validate(1, 8, 8, ms, agmm.AGMM_FP32, 1) == agmm.AGMM_ERR_UNSUPPORTED

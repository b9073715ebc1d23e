"""Host-only checks of the feed-forward block and layer norm (no GPU): refusals
before the device is touched, the kept pre-activations' container, and the rules
of the inline assembly in the kernels built around the GEMM's main loop."""
import ctypes

import pytest
import torch

import asm_rules
import all_gather_gemm_agmm_amd as agmm
from test_asm_rules import _device_asm

INVALID, UNSUPPORTED = agmm.AGMM_ERR_INVALID_ARG, agmm.AGMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("args,status,fragment", [
    ((0, 4, 8, 8, 0, 0, 0), INVALID, "num_shards"),
    ((65, 4, 8, 8, 0, 0, 0), UNSUPPORTED, "maximum"),
    ((2, 4, 0, 8, 0, 0, 0), INVALID, "sizes"),
    ((2, 4, 8, 8, 2, 0, 0), UNSUPPORTED, "bf16 or fp16"),
    ((2, 4, 8, 8, 9, 0, 0), INVALID, "dtype"),
    ((2, 4, 8, 8, 0, 5, 0), INVALID, "activation"),
    ((2, 4, 8, 8, 0, -1, 0), INVALID, "activation"),
    ((2, 4, 8, 8, 0, 0, 2), INVALID, "gated"),
    ((1, 1 << 27, 8, 8, 0, 0, 0), UNSUPPORTED, "too large"),
    ((1, 8, 8, 1 << 27, 0, 0, 0), UNSUPPORTED, "too large"),
    ((1, 8, 8, 1 << 26, 0, 0, 1), UNSUPPORTED, "too large"),
    ((1, 1 << 20, 8, 1 << 16, 0, 0, 0), UNSUPPORTED, "too large"),
    ((1, 8, 1 << 26, 1 << 10, 0, 0, 0), UNSUPPORTED, "too large"),
    ((64, (1 << 58) + 1, 8, 8, 0, 0, 0), UNSUPPORTED, "too large"),
    ((1, 8, (1 << 63) - 1, 8, 0, 0, 0), UNSUPPORTED, "too large"),
])
def test_feed_forward_rejects(args, status, fragment):
    assert agmm.load_library().agmm_ff_plan_validate(*args) == status
    assert agmm.agmm_last_status() == status and fragment in agmm.agmm_last_error()


def test_feed_forward_accepts():
    lib = agmm.load_library()
    for args in ((1, 1, 1, 1, 0, 0, 0), (64, 3, 1001, 77, 1, 4, 1), (8, 4096, 8192, 7168, 0, 2, 1)):
        assert lib.agmm_ff_plan_validate(*args) == agmm.AGMM_OK, agmm.agmm_last_error()
        assert agmm.agmm_last_error() == ""


@pytest.mark.parametrize("args,status,fragment", [
    ((0, 8, 0, 0), INVALID, "sizes"), ((8, -1, 0, 0), INVALID, "sizes"), ((8, 8, 3, 0), INVALID, "dtype"),
    ((8, 8, 0, 3), INVALID, "weight dtype"), ((8, 8, 0, 1), UNSUPPORTED, "weights have"), ((8, 8, 2, 0), UNSUPPORTED, "weights have"),
    ((1 << 28, 8, 0, 0), UNSUPPORTED, "too large"), ((8, 1 << 26, 0, 0), UNSUPPORTED, "too large"),
    ((1 << 20, 1 << 17, 0, 0), UNSUPPORTED, "too large"), ((1 << 62, 1 << 62, 0, 0), UNSUPPORTED, "too large"),
])
def test_norm_rejects(args, status, fragment):
    assert agmm.load_library().agmm_norm_plan_validate(*args) == status
    assert agmm.agmm_last_status() == status and fragment in agmm.agmm_last_error()


def test_norm_accepts():
    lib = agmm.load_library()
    for args in ((1, 1, 0, 0), (8192, 8192, 0, 2), (7, 100003, 2, 2), (1 << 27, 1000, 1, 1)):
        assert lib.agmm_norm_plan_validate(*args) == agmm.AGMM_OK, agmm.agmm_last_error()


def test_null_handles_are_rejected():
    lib = agmm.load_library()
    v = ctypes.c_int64(0)
    assert lib.agmm_ff_forward(None, None, None, None, None, None, None, None, None) == INVALID
    assert lib.agmm_ff_backward(None, None, None, None, None, None, None, None, None, None) == INVALID
    assert lib.agmm_ff_recompute(None, None, None, None, None) == INVALID
    assert lib.agmm_ff_plan_set_int(None, b"tile", 0) == INVALID
    assert lib.agmm_ff_plan_get_int(None, b"tile", ctypes.byref(v)) == INVALID
    assert lib.agmm_ff_plan_workspace_bytes(None) == 0
    lib.agmm_ff_plan_destroy(None)
    assert lib.agmm_norm_forward(None, None, None, None, 1e-5, None, None, None, None) == INVALID
    assert lib.agmm_norm_backward(None, None, None, None, None, None, None, None, None, None) == INVALID
    assert lib.agmm_norm_plan_set_int(None, b"ldx", 0) == INVALID
    assert lib.agmm_norm_plan_get_int(None, b"ldx", ctypes.byref(v)) == INVALID
    assert lib.agmm_norm_plan_workspace_bytes(None) == 0
    lib.agmm_norm_plan_destroy(None)


def test_dequantize():
    values = torch.randn((3, 2, 64)).to(torch.float8_e4m3fn)
    codes = torch.tensor([[[127, 130], [120, 127]]], dtype=torch.uint8).repeat(3, 1, 1)
    got = agmm.Checkpoint(values, codes.view(torch.float8_e8m0fnu), 40).dequantize()
    assert got.shape == (3, 80)
    want = values.float()
    assert torch.equal(got[:, :32], want[:, 0, :32]) and torch.equal(got[:, 32:40], want[:, 0, 32:40] * 8)
    assert torch.equal(got[:, 40:72], want[:, 1, :32] / 128) and torch.equal(got[:, 72:], want[:, 1, 32:40])
    half = torch.randn((3, 1, 32)).half()
    assert torch.equal(agmm.Checkpoint(half, None, 5).dequantize(), half[:, 0, :5].float())


@pytest.mark.parametrize("source", ["feed_tiles.hip", "feed_grads.hip"])
def test_kernels_keep_the_inline_asm_rules(source):
    """The tied MFMAs' rules and the M0 rule (test_asm_rules.py) on each kernel."""
    mfmas = loads = 0
    for sym, lines in asm_rules.functions(_device_asm(source)):
        n, bad = asm_rules.check_function(lines)
        assert bad == [], f"{sym}: {bad[:5]}"
        mfmas += n
        n, bad = asm_rules.check_m0(lines)
        assert bad == [], f"{sym}: {bad[:5]}"
        loads += n
    assert loads > 0 and mfmas > 0, "nothing found: the check would be vacuous"

"""Block-scaled 8-bit quantiser and product on the GPU.

The quantiser's definition fixes every rounding (fp32 quotients, one fp32
product, one rounding to 8 bits), so its outputs are compared bit for bit with
the same steps on the CPU.
"""
import numpy as np
import pytest
import torch

import all_gather_gemm_agmm_amd as agmm

pytestmark = pytest.mark.gpu

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


def to8(v, fmt):
    """fp32 -> the format's values, nearest even, on the CPU in 64 bits; NaN
    and infinities as the quantiser documents them."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    v = v.astype(np.float64)
    fin = np.isfinite(v)
    w = np.where(fin, v, 0.0)
    _, e = np.frexp(w)
    step = np.ldexp(1.0, np.maximum(e - 1, low) - bits)
    out = np.round(w / step) * step
    return np.where(fin, out, np.nan if fmt == "e4m3" else v)


def quantize_ref(x, fmt, block):
    """(values as float64 [rows, cols16], scales float32 [kb, rb]) of a CPU tensor."""
    x = x.float().numpy()
    rows, cols = x.shape
    kb, rb = -(-cols // 128), -(-rows // block)
    values = np.zeros((rows, -(-cols // 16) * 16))
    scales = np.zeros((kb, rb), np.float32)
    with np.errstate(all="ignore"):
        for b in range(kb):
            for r in range(rb):
                part = x[r * block:(r + 1) * block, b * 128:(b + 1) * 128]
                size = np.where(np.isfinite(part), np.abs(part), np.float32(0)).max()
                s = max(np.float32(size) / np.float32(TOP[fmt]), np.float32(2.0 ** -126))
                scales[b, r] = s
                values[r * block:(r + 1) * block, b * 128:b * 128 + part.shape[1]] = \
                    to8(part * (np.float32(1) / s), fmt)
    return values, scales


def check_quantized(got, x, fmt, block):
    values, scales = quantize_ref(x, fmt, block)
    assert got.k == x.shape[1] and got.block_rows == block
    assert np.array_equal(got.scales.cpu().numpy(), scales)
    assert np.array_equal(got.values.cpu().float().numpy().astype(np.float64), values, equal_nan=True)


def draw(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-6, 7, (1, cols), generator=g).float())
    return x.to(TYPES[dtype])


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (7, 17), (16, 512), (127, 129), (128, 128), (129, 1000),
                                       (130, 513), (260, 1040)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize(rows, cols, dtype, fmt, block):
    x = draw(rows, cols, dtype, rows * 1000 + cols)
    xd = x.cuda()
    check_quantized(agmm.quantize(xd, fmt, block), x, fmt, block)
    check_quantized(agmm.quantize(xd, fmt, block, out="cols"), x.t(), fmt, block)
    a, b = agmm.quantize(xd, fmt, block, out="both")
    check_quantized(a, x, fmt, block)
    check_quantized(b, x.t(), fmt, block)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_deep_rows(dtype):
    """Enough rows for the form that takes 8 rows per wave, with a ragged end."""
    x = draw(8195, 2056, dtype, 5)
    check_quantized(agmm.quantize(x.cuda(), "e4m3", 1), x, "e4m3", 1)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_special_values(fmt, block):
    x = draw(140, 300, "fp32", 3)
    x[3, 5] = float("inf")
    x[3, 6] = -float("inf")
    x[4, 200] = float("nan")
    x[10, :] = 0.0
    x[11, :] = float("nan")                  # a row with nothing finite
    x[12, 128:256] = 1e-44                   # subnormals: the scale stops at 2^-126
    x[13, :128] = 3.0e38                     # the largest scale
    x[14, :] = -0.0
    x[128:, 256:] = 0.0                      # a tile of zeros
    for got, want in zip(agmm.quantize(x.cuda(), fmt, block, out="both"), (x, x.t())):
        check_quantized(got, want, fmt, block)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("block,out", [(1, "rows"), (1, "cols"), (128, "both")])
def test_quantize_strided_and_unaligned(dtype, block, out):
    """A view with a row stride, and one that starts at an odd element."""
    base = draw(140, 421, dtype, 9)
    for view in (base[:, :256], base[:, 3:260], base[1:, 1:2]):
        dev = base.cuda()
        if view.shape[1] == 256:
            d = dev[:, :256]
        elif view.shape[1] == 257:
            d = dev[:, 3:260]
        else:
            d = dev[1:, 1:2]
        got = agmm.quantize(d, "e4m3", block, out=out)
        got = got if out == "both" else (got,)
        for g, want in zip(got, {"rows": (view,), "cols": (view.t(),), "both": (view, view.t())}[out]):
            check_quantized(g, want, "e4m3", block)


def test_quantize_writes_its_own_bytes_only():
    """Row strides beyond the padded row: the bytes between rows stay."""
    rows, cols = 131, 150
    x = draw(rows, cols, "bf16", 1).cuda()
    q = torch.full((rows, 208), 0x5A, dtype=torch.uint8, device="cuda")
    qt = torch.full((cols, 160), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((2, rows + 1), -1.0, device="cuda")
    st = torch.full((2 * cols + 3,), -1.0, device="cuda")
    agmm.agmm_quantize(x.data_ptr(), agmm.AGMM_BF16, rows, cols, cols, agmm.AGMM_E4M3, 1, q.data_ptr(), 208,
                       s.data_ptr(), qt.data_ptr(), 160, st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert (q[:, 160:] == 0x5A).all() and (q[:, 150:160] == 0).all()
    assert (qt[:, 144:] == 0x5A).all() and (qt[:, 131:144] == 0).all()
    assert (s.flatten()[2 * rows:] == -1).all() and (st[2 * cols:] == -1).all()


def test_quantize_on_another_stream():
    x = draw(300, 700, "bf16", 2)
    xd = x.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = agmm.quantize(xd, "e4m3", 1, stream=side)
    side.synchronize()
    check_quantized(got, x, "e4m3", 1)


def test_quantize_refusals():
    x = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="format"):
        agmm.quantize(x, "e3m4")
    with pytest.raises(ValueError, match="block_rows"):
        agmm.quantize(x, block_rows=64)
    with pytest.raises(ValueError, match="out"):
        agmm.quantize(x, out="rowwise")
    with pytest.raises(ValueError, match="row-major"):
        agmm.quantize(x.t())
    with pytest.raises(TypeError, match="dtype"):
        agmm.quantize(x.double())
    with pytest.raises(ValueError, match="GPU"):
        agmm.quantize(x.cpu())

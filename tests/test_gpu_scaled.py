"""Block-scaled 8-bit quantiser and product on the GPU.

The quantiser's definition fixes every rounding (fp32 scales, the nearest
8-bit value of the real quotient), so its outputs are compared bit for bit with
the same steps on the CPU, the quotient in 64 bits.
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
                    to8(part.astype(np.float64) / np.float64(s), fmt)
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


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_special_values_of_16_bits(fmt, dtype, block):
    x = draw(140, 300, dtype, 4)
    x[3, 5], x[3, 6], x[4, 200] = float("inf"), -float("inf"), float("nan")
    x[10, :] = 0.0
    x[11, :] = float("nan")
    x[12, 128:256] = 6e-8 if dtype == "fp16" else 1e-39
    x[13, :128] = 6.5e4
    for got, want in zip(agmm.quantize(x.cuda(), fmt, block, out="both"), (x, x.t())):
        check_quantized(got, want, fmt, block)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_midpoints(fmt, dtype, block):
    """Every pair of a maximum and an element whose quotient is a midpoint or
    next to one: multiples of the maximum by midpoints of the format over its
    largest value (exact in 16 bits for maxima that are multiples of 7), and
    in fp32 their neighbours; results below the smallest normal value among them."""
    top = TOP[fmt]
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    rows, cols = 256, 128
    x = torch.zeros((rows, cols), dtype=torch.float64)
    step = 2.0 ** (low - bits)
    mids = [(2 * j + 1) / 2 * step for j in range(2 ** bits)]                               # below the smallest normal
    mids += [2.0 ** e * (1 + (2 * j + 1) / 2 ** (bits + 1)) for e in range(-5, 8) for j in range(2 ** bits)]
    for r in range(rows):
        big = (128 + r % 128) * 2.0 ** (r // 128 * 3 - 4)
        x[r, 0] = big
        for c in range(1, cols):
            x[r, c] = (-1) ** c * mids[(c + 31 * r) % len(mids)] * big / top
    x = x.float() if dtype == "fp32" else x.to(TYPES[dtype])
    if dtype == "fp32":
        x[::3] = torch.nextafter(x[::3], torch.full_like(x[::3], float("inf")))
        x[1::3] = torch.nextafter(x[1::3], torch.full_like(x[1::3], -float("inf")))
        x[:, 0] = x.abs().amax(1)
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


# ---------------------------------------------------------------- product
#
# Tolerance.  The 8-bit products are exact in fp32; the sum of n of them with
# any order of fp32 additions is off by at most (n - 1) u sum |terms|, u =
# 2^-24, and a truncating adder at most twice that.  Each scaling adds u per
# block, C's rounding half a unit of its type.  So
#   |C - ref| <= (2 k + 8) u * sum |a b|  +  half ulp(ref) (+ its spacing at 0).
HALF_ULP = {agmm.AGMM_BF16: 2.0 ** -8, agmm.AGMM_FP16: 2.0 ** -11, agmm.AGMM_FP32: 2.0 ** -24}
FLOOR = {agmm.AGMM_BF16: 0.0, agmm.AGMM_FP16: 2.0 ** -25, agmm.AGMM_FP32: 0.0}


def operand(rows, k, fmt, block, seed, device="cuda"):
    """A Scaled made on the CPU with scales of its own (not from a quantiser):
    random 8-bit values and fp32 scales, zeros past k."""
    g = torch.Generator().manual_seed(seed)
    values = torch.zeros((rows, -(-k // 16) * 16))
    values[:, :k] = torch.randn((rows, k), generator=g) * 8
    scales = torch.exp2(torch.rand((-(-k // 128), -(-rows // block)), generator=g) * 12 - 9)
    return agmm.Scaled(values.to(F8[fmt]).to(device), scales.to(device), k, block)


def spread64(x):
    v = x.values[:, :x.k].cpu().float().double()
    s = x.scales.cpu().double().t().repeat_interleave(128, dim=1)[:, :x.k]
    return v * s.repeat_interleave(x.block_rows, dim=0)[:x.rows]


def check_product(got, a, b, c_dtype):
    ref = a @ b.t()
    size = a.abs() @ b.abs().t()
    k = a.shape[1]
    bound = (2 * k + 8) * 2.0 ** -24 * size + HALF_ULP[c_dtype] * ref.abs() * (1 + 2.0 ** -7) + FLOOR[c_dtype]
    got = got.cpu().double()
    if c_dtype == agmm.AGMM_FP16:   # beyond fp16's range: an infinity of the right sign, within the bound of its edge
        over = torch.isinf(got)
        assert (ref[over].abs() + bound[over] >= 65520).all() and torch.equal(got[over].sign(), ref[over].sign())
        assert (over | (ref.abs() - bound < 65520)).all()
        got, ref, bound = got[~over], ref[~over], bound[~over]
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    worst = (err - bound).max().item()
    assert worst <= 0, (worst, err.max().item())


def run_product(N, ms, k, n, fmt="e4m3", block=128, c_dtype=agmm.AGMM_BF16, seed=0, **settings):
    shards = [operand(ms, k, fmt, 1, seed * 100 + r) for r in range(N)]
    B = operand(n, k, "e4m3", block, seed * 100 + 99)
    with agmm.ScaledPlan(N, ms, k, n, fmt, block, c_dtype, **settings) as plan:
        C = plan.run(shards, B)
        torch.cuda.synchronize()
        used = plan.get("tile"), plan.get("splits")
    check_product(C, torch.cat([spread64(s) for s in shards]), spread64(B), c_dtype)
    return C, shards, B, used


@pytest.mark.parametrize("N,ms,k,n", [
    (1, 1, 1, 1), (1, 1, 128, 16), (8, 1, 512, 48), (3, 5, 130, 33), (2, 8, 1000, 100), (1, 16, 2048, 64),
    (4, 16, 272, 96), (1, 129, 128, 128), (2, 100, 256, 200), (3, 337, 404, 261), (1, 256, 640, 256),
    (2, 256, 128, 512), (5, 103, 1160, 515), (64, 5, 144, 140), (2, 512, 4096, 256)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", [1, 128])
def test_product(N, ms, k, n, fmt, block):
    run_product(N, ms, k, n, fmt, block, agmm.AGMM_BF16, seed=ms + k)


@pytest.mark.parametrize("tile", [0, 1, 2, 3])
@pytest.mark.parametrize("c_dtype", [agmm.AGMM_BF16, agmm.AGMM_FP16, agmm.AGMM_FP32])
@pytest.mark.parametrize("N,ms,k,n", [(2, 20, 700, 70), (1, 300, 1300, 301), (2, 256, 512, 512)])
def test_product_every_tile(tile, c_dtype, N, ms, k, n):
    for splits in (1, 2, 3):
        _, _, _, used = run_product(N, ms, k, n, c_dtype=c_dtype, tile=tile, splits=splits, seed=7)
        kb = -(-k // 128)
        assert used == (tile, -(-kb // -(-kb // splits)))   # ranges of equal whole blocks


@pytest.mark.parametrize("fmt,k,c_dtype", [("e5m2", 300, agmm.AGMM_FP32), ("e4m3", 300, agmm.AGMM_FP32),
                                           ("e5m2", 2048, agmm.AGMM_BF16), ("e4m3", 2048, agmm.AGMM_BF16)])
@pytest.mark.parametrize("ms", [3, 200])
def test_product_of_the_smallest_values(fmt, k, c_dtype, ms):
    """Operands that are subnormal numbers of their formats count like others."""
    a, b = operand(ms, k, fmt, 1, 61), operand(140, k, "e4m3", 128, 62)
    for x, bits in ((a, 3 if fmt == "e5m2" else 7), (b, 7)):
        bytes_ = x.values.view(torch.uint8)
        bytes_ &= 0x80 | bits          # sign and mantissa only
    with agmm.ScaledPlan(1, ms, k, 140, fmt, 128, c_dtype) as plan:
        C = plan.run([a], b)
        torch.cuda.synchronize()
    check_product(C, spread64(a), spread64(b), c_dtype)
    assert (C != 0).any()


def test_product_strides():
    """Operands and C as views with row strides; bytes between C's rows stay."""
    N, ms, k, n = 2, 70, 300, 90
    shards = [operand(ms, k, "e4m3", 1, r) for r in range(N)]
    B = operand(n, k, "e4m3", 128, 9)

    def wide(x, ld):
        buf = torch.full((x.rows, ld), 127, dtype=torch.uint8, device="cuda").view(x.values.dtype)   # NaN
        buf[:, :x.values.shape[1]] = x.values
        return agmm.Scaled(buf[:, :x.values.shape[1]], x.scales, x.k, x.block_rows)

    buf = torch.full((N * ms, 101), -7.0, dtype=torch.bfloat16, device="cuda")
    with agmm.ScaledPlan(N, ms, k, n, "e4m3", 128, agmm.AGMM_BF16, lda=336, ldb=320, ldc=101) as plan:
        C = plan.run([wide(s, 336) for s in shards], wide(B, 320), buf[:, :n])
    torch.cuda.synchronize()
    check_product(C, torch.cat([spread64(s) for s in shards]), spread64(B), agmm.AGMM_BF16)
    assert (buf[:, n:] == -7).all()


def test_product_keeps_rows_and_columns_apart():
    """NaN in one row of A and one row of B reaches that row and column only."""
    N, ms, k, n = 2, 150, 256, 140
    shards = [operand(ms, k, "e4m3", 1, r) for r in range(N)]
    B = operand(n, k, "e4m3", 128, 9)
    with agmm.ScaledPlan(N, ms, k, n) as plan:
        want = plan.run(shards, B)
        shards[1].values.view(torch.uint8)[7, 200] = 0x7F
        B.values.view(torch.uint8)[33, 3] = 0x7F
        got = plan.run(shards, B)
    torch.cuda.synchronize()
    bad = torch.isnan(got)
    assert bad[ms + 7].all() and bad[:, 33].all()
    bad[ms + 7] = False
    bad[:, 33] = False
    assert not bad.any()
    keep = torch.ones_like(bad)
    keep[ms + 7] = False
    keep[:, 33] = False
    assert torch.equal(got[keep], want[keep])


def test_product_calls_share_a_plan_across_streams():
    """A plan that splits k (its partial sums are shared), called on two
    streams with other inputs each: every result is that of its inputs."""
    N, ms, k, n = 1, 16, 8192, 64
    with agmm.ScaledPlan(N, ms, k, n, splits=8) as plan:
        sets = [([operand(ms, k, "e4m3", 1, 10 + i)], operand(n, k, "e4m3", 128, 20 + i)) for i in range(2)]
        want = [plan.run(*s) for s in sets]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [[], []]
        for _ in range(20):
            for i in range(2):
                got[i].append(plan.run(*sets[i], stream=streams[i]))
        torch.cuda.synchronize()
    for i in range(2):
        check_product(want[i], spread64(sets[i][0][0]), spread64(sets[i][1]), agmm.AGMM_BF16)
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_product_calls_that_overlap_keep_their_operands():
    """A call that another one of the same plan overtakes, as one of another
    thread can, between the reading of its shards: both are right."""
    N, ms, k, n = 2, 5, 200, 40
    sets = [([operand(ms, k, "e4m3", 1, 30 + 2 * i), operand(ms, k, "e4m3", 1, 31 + 2 * i)], operand(n, k, "e4m3", 128, 40 + i))
            for i in range(2)]
    other = []
    with agmm.ScaledPlan(N, ms, k, n) as plan:
        want = [plan.run(*s) for s in sets]

        class Overtaken(list):
            def __iter__(self):
                yield self[0]
                yield self[1]
                other.append(plan.run(*sets[1]))

        got = plan.run(Overtaken(sets[0][0]), sets[0][1])
        torch.cuda.synchronize()
    assert torch.equal(got, want[0]) and torch.equal(other[0], want[1])


def test_product_in_a_graph():
    N, ms, k, n = 2, 8, 2048, 96
    shards = [operand(ms, k, "e4m3", 1, r) for r in range(N)]
    B = operand(n, k, "e4m3", 128, 5)
    with agmm.ScaledPlan(N, ms, k, n) as plan:
        C = torch.empty((N * ms, n), dtype=torch.bfloat16, device="cuda")
        want = plan.run(shards, B).clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.run(shards, B, C)
        for _ in range(4):
            C.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(C, want)
        with pytest.raises(agmm.AgmmError) as ei:
            plan.set("splits", 1)
        assert ei.value.status == agmm.AGMM_ERR_UNSUPPORTED
        del graph


def test_product_of_quantised_operands():
    """Quantise and multiply: against the product of the unquantised matrices,
    within the formats' half spacing (2^-4 relative for e4m3) per factor."""
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn((200, 1000), generator=g), torch.randn((150, 1000), generator=g) / 30
    shards = [agmm.quantize(s.bfloat16().cuda()) for s in x.split(100)]
    W = agmm.quantize(w.cuda(), block_rows=128)
    with agmm.ScaledPlan(2, 100, 1000, 150, c_dtype=agmm.AGMM_FP32) as plan:
        C = plan.run(shards, W)
    torch.cuda.synchronize()
    ref = x.double() @ w.double().t()
    rel = (C.cpu().double() - ref).norm() / ref.norm()
    assert rel < 2.0 ** -4
    check_product(C, torch.cat([spread64(s) for s in shards]), spread64(W), agmm.AGMM_FP32)


def test_product_training_identities():
    """dx and dW of y = x W^T through the same product on transposed
    operands, against their formulas on the quantised values."""
    g = torch.Generator().manual_seed(1)
    m, k, n = 260, 300, 200
    x, dy, w = (torch.randn(s, generator=g).cuda() for s in ((m, k), (m, n), (n, k)))
    xq, xt = agmm.quantize(x, out="both")
    dq, dt = agmm.quantize(dy, "e5m2", out="both")
    wq, wt = agmm.quantize(w, block_rows=128, out="both")
    assert torch.equal(wq.dequantize(), wt.dequantize().t())
    with agmm.ScaledPlan(1, m, n, k, "e5m2", 128, agmm.AGMM_FP32) as plan:
        dx = plan.run([dq], wt)
    with agmm.ScaledPlan(1, n, m, k, "e5m2", 1, agmm.AGMM_FP32) as plan:
        dw = plan.run([dt], xt)
    torch.cuda.synchronize()
    check_product(dx, spread64(dq), spread64(wt), agmm.AGMM_FP32)
    check_product(dw, spread64(dt), spread64(xt), agmm.AGMM_FP32)


def test_product_refusals():
    a, b = operand(8, 64, "e4m3", 1, 0), operand(16, 64, "e4m3", 128, 1)
    with agmm.ScaledPlan(1, 8, 64, 16) as plan:
        with pytest.raises(ValueError, match="shards"):
            plan.run([a, a], b)
        with pytest.raises(TypeError, match="Scaled"):
            plan.run([a.values], b)
        with pytest.raises(ValueError, match="block_rows"):
            plan.run([a], operand(16, 64, "e4m3", 1, 1))
        with pytest.raises(TypeError, match="dtype"):
            plan.run([operand(8, 64, "e5m2", 1, 0)], b)
        with pytest.raises(ValueError, match="shape"):
            plan.run([operand(9, 64, "e4m3", 1, 0)], b)
        with pytest.raises(ValueError, match="GPU"):
            plan.run([operand(8, 64, "e4m3", 1, 0, "cpu")], b)
        with pytest.raises(ValueError, match="row-major"):
            plan.run([a], b, torch.empty((16, 8), dtype=torch.bfloat16, device="cuda").t())
        for key, val in (("lda", 48), ("lda", 72), ("ldc", 8), ("tile", 4), ("splits", -1), ("nothing", 1)):
            with pytest.raises(agmm.AgmmError) as ei:
                plan.set(key, val)
            assert ei.value.status == agmm.AGMM_ERR_INVALID_ARG
        with pytest.raises(ValueError, match="row-major"):
            plan.set("lda", 80)
            plan.run([a], b)


def test_product_out_of_memory_is_an_error(monkeypatch):
    monkeypatch.setenv("AGMM_TEST_FAIL_ALLOC", "1")
    with pytest.raises(agmm.AgmmError) as ei:
        agmm.ScaledPlan(1, 16, 8192, 64)
    assert ei.value.status == agmm.AGMM_ERR_OOM
    with agmm.ScaledPlan(1, 512, 512, 65536) as plan:
        assert plan.workspace_bytes() == 0      # no k split: nothing to allocate

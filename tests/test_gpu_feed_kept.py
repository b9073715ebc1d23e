"""Kept pre-activations through the C ABI, in buffers filled beforehand: every
column of them is written, up to the padded width, and nothing behind them; and
the feed-forward checks of 256 x 224 tiles that test_gpu_feed.py runs on the
other forms only."""
import ctypes

import pytest
import torch

import all_gather_gemm_agmm_amd as agmm
import feed_reference as R
from test_gpu_feed import BF16, FP16, TYPE, kept_matches, make

pytestmark = pytest.mark.gpu

UNTOUCHED = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


def filled(shape, dtype):
    """A tensor whose bytes are all ones (NaN in every type here), and the bytes behind it."""
    size = torch.Size(shape).numel() * dtype.itemsize
    flat = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    flat[size:] = UNTOUCHED
    return flat[:size].view(dtype).view(shape), flat[size:]


def forward(plan, shards, w, b, keep, act_dtype):
    """agmm_ff_forward into filled buffers: y and the Checkpoint."""
    m, parts, n, wide = plan.m, plan.parts, plan.n_local, plan.get("saved_cols")
    y, behind_y = filled((m, n), act_dtype)
    values, behind_v = filled((m, parts, wide), act_dtype if keep == 16 else torch.float8_e4m3fn)
    scales, behind_s = filled((m, parts, wide // 32), torch.float8_e8m0fnu) if keep == 8 else (None, None)
    table = (ctypes.c_void_p * len(shards))(*[s.data_ptr() for s in shards])
    status = agmm.load_library().agmm_ff_forward(plan.handle, table, w.data_ptr(), None if b is None else b.data_ptr(), None, y.data_ptr(),
                                                 values.data_ptr(), None if scales is None else scales.data_ptr(),
                                                 torch.cuda.current_stream().cuda_stream)
    assert status == agmm.AGMM_OK, agmm.agmm_last_error()
    torch.cuda.synchronize()
    for behind in (behind_y, behind_v, behind_s):
        assert behind is None or (behind == UNTOUCHED).all()
    return y, agmm.Checkpoint(values, scales, n)


# columns that end inside a block of 32 in every way that 112, the columns of a gated 256 x 224 tile, leaves, and beside it
COLUMNS = (1, 31, 32, 33, 95, 96, 97, 100, 111, 112, 113, 128, 208, 209, 223, 224, 225, 321, 335, 336, 337, 545, 560, 575, 784)


@pytest.mark.parametrize("tile", [-1, 64, 128, 224, 256])
@pytest.mark.parametrize("n", COLUMNS)
@pytest.mark.parametrize("gated", [False, True])
def test_every_kept_column_is_written(gated, n, tile):
    parts = 2 if gated else 1
    for ms, k, dtype in ((150, 128, FP16), (129, 72, BF16), (11, 640, BF16)):
        shards, w, b, _ = make(2, ms, k, n, dtype, parts)
        with agmm.FeedForwardPlan(2, ms, k, n, dtype, activation="silu", gated=gated, with_gradient=False, tile=tile) as plan:
            want, bound, p, e = R.forward("silu", gated, torch.cat(shards), w, b, None, TYPE[dtype])
            for keep in (16, 8):
                y, saved = forward(plan, shards, w, b, keep, TYPE[dtype])
                R.check(y, want, bound, "y")
                kept_matches(saved, p, e, n, parts, TYPE[dtype])
                if keep == 8:   # blocks of nothing but padding cannot exist: every scale is a finite power of two
                    assert torch.isfinite(saved.scales.float()).all()


@pytest.mark.parametrize("keep", [16, 8])
@pytest.mark.parametrize("N,ms,k,n", [(8, 256, 8192, 3472), (4, 512, 4096, 3696), (8, 128, 8192, 1008)])
def test_every_kept_column_of_large_products(N, ms, k, n, keep):
    """Hidden sizes at which the automatic choice takes large tiles, 16 columns short of whole blocks."""
    g = torch.Generator(device="cuda").manual_seed(n)
    shards = [torch.randn((ms, k), generator=g, device="cuda").bfloat16() for _ in range(N)]
    w = (torch.randn((2 * n, k), generator=g, device="cuda") / k ** 0.5).bfloat16()
    with agmm.FeedForwardPlan(N, ms, k, n, BF16, activation="silu", gated=True, with_gradient=False) as plan:
        _, saved = forward(plan, shards, w, None, keep, torch.bfloat16)
    assert (saved.values[:, :, n:].float() == 0).all()
    assert torch.isfinite(saved.values.float()).all()


@pytest.mark.parametrize("gated", [False, True])
def test_exact_sums_by_224(gated):
    """Small whole numbers: p, both kept forms and y are exact."""
    g = torch.Generator().manual_seed(0)
    parts = 2 if gated else 1
    for m, k, n in ((130, 64, 300), (270, 200, 112), (7, 64, 230)):
        a = torch.randint(-4, 5, (m, k), generator=g).bfloat16().cuda()
        w = torch.randint(-3, 4, (parts * n, k), generator=g).bfloat16().cuda()
        w[::7] = 0
        p = a.double() @ w.double().t()
        full = torch.nn.functional.pad(p.view(m, parts, n), (0, -n % 32))
        want = p[:, :n].clamp(min=0) * (p[:, n:] if gated else 1)
        with agmm.FeedForwardPlan(1, m, k, n, BF16, activation="relu", gated=gated, with_gradient=False, tile=224) as plan:
            y, saved = forward(plan, [a], w, None, 8, torch.bfloat16)
            y16, saved16 = forward(plan, [a], w, None, 16, torch.bfloat16)
        s, _ = R.scales_of(p, n, parts)
        assert torch.equal(saved.scales.double(), s)
        assert torch.equal(saved.values.float(), (full / s.repeat_interleave(32, dim=2)).float().to(torch.float8_e4m3fn).float())
        assert torch.equal(saved16.values, full.bfloat16())
        assert torch.equal(y, want.bfloat16()) and torch.equal(y16, y)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("gated", [False, True])
def test_nan_and_infinity_by_224(gated, bad):
    """They reach their row alone, in both kept forms."""
    m, k, n, parts = 40, 64, 112, 2 if gated else 1
    shards, w, b, _ = make(1, m, k, n, BF16, parts)
    w[:, 3] = w[:, 3].abs() + 0.25                     # infinity times a positive number
    rows = [i for i in range(m) if i != 7]
    with agmm.FeedForwardPlan(1, m, k, n, BF16, activation="gelu", gated=gated, with_gradient=False, tile=224) as plan:
        for keep in (8, 16):
            clean = forward(plan, shards, w, b, keep, torch.bfloat16)
            a = shards[0].clone()
            a[7, 3] = bad
            y, saved = forward(plan, [a], w, b, keep, torch.bfloat16)
            assert torch.equal(y[rows], clean[0][rows])
            assert torch.equal(saved.values[rows].float(), clean[1].values[rows].float())
            assert (torch.isnan(y[7]) if bad != bad else torch.isinf(y[7])).all()
            got = saved.values[7, :, :n].float()
            assert (torch.isinf(got) if keep == 16 and bad == bad else torch.isnan(got)).all()
            assert (saved.values[7, :, n:].float() == 0).all()


def test_one_infinite_pre_activation_by_224():
    """It becomes NaN in e4m3 and does not enter the block's scale."""
    m, k, n = 3, 16, 64
    a = torch.zeros((m, k)).half().cuda()
    a[:, 0] = 1
    w = torch.zeros((n, k)).half().cuda()
    w[:, 0] = torch.linspace(-3, 3, n).half()
    w[5, 0] = float("inf")
    with agmm.FeedForwardPlan(1, m, k, n, FP16, with_gradient=False, tile=224) as plan:
        y, saved = forward(plan, [a], w, None, 8, torch.float16)
    got = saved.dequantize()
    assert torch.isnan(got[:, 5]).all() and torch.isfinite(got[:, :5]).all() and torch.isfinite(got[:, 6:]).all()
    want = w[:, 0].double()
    want[5] = 0
    assert torch.equal(saved.scales.double(), R.scales_of(want.expand(m, n).contiguous(), n, 1)[0])
    assert torch.isinf(y[:, 5]).all()


def test_residual_in_place_by_224():
    m, k, n = 300, 128, 256
    shards, w, b, r = make(1, m, k, n, BF16, 1, residual=True)
    with agmm.FeedForwardPlan(1, m, k, n, BF16, with_gradient=False, tile=224) as plan:
        want = plan.forward(shards, w, b, r)
        plan.forward(shards, w, b, r, out=r)
    assert torch.equal(r, want)

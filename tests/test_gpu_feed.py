"""Product with an epilogue, gated product, their kept pre-activations and their
gradients on the GPU, against the formulas in 64 bits (feed_reference.py)."""
import pytest
import torch

import all_gather_gemm_agmm_amd as agmm
import feed_reference as R

pytestmark = pytest.mark.gpu

BF16, FP16 = agmm.AGMM_BF16, agmm.AGMM_FP16
TYPE = {BF16: torch.bfloat16, FP16: torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


def make(N, ms, k, n, dtype, parts, bias=True, residual=False, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * k + n)
    t = TYPE[dtype]
    shards = [torch.randn((ms, k), generator=g).to(t).cuda() for _ in range(N)]
    w = (torch.randn((parts * n, k), generator=g) * (1.5 / k ** 0.5)).to(t).cuda()
    b = (torch.randn(parts * n, generator=g) * 0.5).to(t).cuda() if bias else None
    r = torch.randn((N * ms, n), generator=g).to(t).cuda() if residual else None
    return shards, w, b, r


def kept_matches(saved, p, e, n, parts, dtype):
    """What was kept against p and its error; zeros past n."""
    got = saved.dequantize().double()
    assert (saved.values[:, :, n:].float() == 0).all()
    if saved.scales is None:
        R.check(got, p, e * (1 + R.EPS[dtype]) + R.EPS[dtype] * p.abs() + R.TINY[dtype], "kept, 16 bits")
        return
    want, size = R.scales_of(p, n, parts)
    s = saved.scales.double()
    slack = torch.nn.functional.pad(e.view(len(p), parts, n), (0, -n % 32)).view(s.shape + (32,)).amax(3)
    # another power of two only where p's error reaches 448 times one
    near = ((size + slack) / 448 > want) | (((size - slack) / 448) <= want / 2)
    assert ((s == want) | near).all()
    each = s.repeat_interleave(32, dim=2)[:, :, :n].reshape(len(p), -1)
    R.check(got, p, e * (1 + 2.0 ** -4) + 2.0 ** -4 * p.abs() + each * 2.0 ** -10, "kept, 8 bits")


SHAPES = [  # N, m_per_shard, k, n
    (1, 1, 1, 1), (1, 1, 64, 16), (2, 3, 100, 33), (8, 1, 512, 96), (1, 16, 130, 48), (3, 7, 71, 65), (2, 40, 256, 160),
    (5, 13, 257, 31), (1, 64, 1024, 256), (3, 100, 192, 200), (2, 129, 320, 130), (1, 257, 72, 257), (4, 128, 256, 384),
    (3, 64, 128, 224), (1, 300, 4040, 240), (7, 20, 1100, 500)]


@pytest.mark.parametrize("tile", [-1, 64, 128, 224, 256])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("gated", [False, True])
def test_forward(shape, gated, tile):
    """Every tile at every shape; activations, types, epilogues and kept forms in turn."""
    N, ms, k, n = shape
    for i, (name, dtype, keep) in enumerate([("silu", BF16, 8), ("gelu", FP16, 16), ("gelu_tanh", BF16, 0), ("relu", FP16, 8),
                                             ("none", BF16, 16)]):
        parts = 2 if gated else 1
        shards, w, b, r = make(N, ms, k, n, dtype, parts, bias=i % 2 == 0, residual=not gated and i % 3 != 1, seed=i)
        with agmm.FeedForwardPlan(N, ms, k, n, dtype, activation=name, gated=gated, with_gradient=False, tile=tile) as plan:
            got = plan.forward(shards, w, b, r, keep=keep)
            y, saved = got if keep else (got, None)
            want, bound, p, e = R.forward(name, gated, torch.cat(shards), w, b, r, TYPE[dtype])
            R.check(y, want, bound, f"{name} y")
            if keep:
                kept_matches(saved, p, e, n, parts, TYPE[dtype])
                again = plan.recompute(saved)
                v = saved.dequantize().double()
                x, _ = R.act(name, v[:, :n])
                off = x.abs() * (R.act_error(name, v[:, :n]) + 2.0 ** -22)
                if gated:
                    x, off = x * v[:, n:], off * v[:, n:].abs()
                R.check(again, x, off * 1.01 + R.EPS[TYPE[dtype]] * x.abs() + R.TINY[TYPE[dtype]], f"{name} recomputed")


@pytest.mark.parametrize("tile", [-1, 128, 256])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("gated", [False, True])
def test_backward(shape, gated, tile):
    N, ms, k, n = shape
    for i, (name, dtype, keep) in enumerate([("silu", BF16, 8), ("gelu", FP16, 16), ("gelu_tanh", FP16, 8), ("relu", BF16, 16),
                                             ("none", BF16, 16), ("none", FP16, 0)]):
        if keep == 0 and gated:
            continue
        parts = 2 if gated else 1
        shards, w, b, _ = make(N, ms, k, n, dtype, parts, seed=i)
        dy = (torch.randn((N * ms, n), generator=torch.Generator().manual_seed(i)) / 8).to(TYPE[dtype]).cuda()
        with agmm.FeedForwardPlan(N, ms, k, n, dtype, activation=name, gated=gated, tile=tile) as plan:
            saved = plan.forward(shards, w, b, keep=keep)[1] if keep else None
            da, dw, db = plan.backward(shards, w, saved, dy, need_dbias=True)
            p = saved.dequantize() if keep else torch.zeros((N * ms, n), device="cuda")
            _, *want = R.gradient(name, gated, p, dy, torch.cat(shards), w, TYPE[dtype])
            for got, (exact, bound), what in zip((da, dw, db), want, ("dA", "dW", "dbias")):
                R.check(got, exact, bound, f"{name} {what}")


@pytest.mark.parametrize("gated", [False, True])
def test_each_gradient_alone(gated):
    N, ms, k, n, parts = 3, 50, 136, 72, 2 if gated else 1
    shards, w, b, _ = make(N, ms, k, n, BF16, parts)
    dy = torch.randn((N * ms, n), device="cuda").bfloat16()
    with agmm.FeedForwardPlan(N, ms, k, n, BF16, activation="silu", gated=gated) as plan:
        _, saved = plan.forward(shards, w, b, keep=8)
        all3 = plan.backward(shards, w, saved, dy, need_dbias=True)
        for i in range(3):
            only = plan.backward(shards, w, saved, dy, need_dA=i == 0, need_dW=i == 1, need_dbias=i == 2)
            assert [x is None for x in only] == [j != i for j in range(3)]
            assert torch.equal(only[i], all3[i])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(name, gated):
    """The gradient of sum(y * c) against central differences of the 64-bit
    formula at the kernel's own kept (16-bit) pre-activations: the slopes."""
    m, k, n, parts = 5, 8, 24, 2 if gated else 1
    shards, w, b, _ = make(1, m, k, n, FP16, parts, seed=3)
    c = (torch.randn((m, n), generator=torch.Generator().manual_seed(5))).half().cuda()
    with agmm.FeedForwardPlan(1, m, k, n, FP16, activation=name, gated=gated) as plan:
        _, saved = plan.forward(shards, w, b, keep=16)
        db = plan.backward(shards, w, saved, c, need_dA=False, need_dW=False, need_dbias=True)[2].double()
    p = saved.dequantize().double()
    h = 2.0 ** -12
    for col in range(parts * n):
        total = []
        for sign in (1, -1):
            q = p.clone()
            q[:, col] += sign * h
            v, _ = R.act(name, q[:, :n])
            total.append(((v * q[:, n:] if gated else v) * c.double()).sum())
        want = (total[0] - total[1]) / (2 * h)
        # third derivatives of at most 2 times factors of at most 8: h^2 / 6 of their sum; relu's kink lies
        # within h of no p here unless p is 0
        size = (c.double().abs().sum(0)[col % n] * 8).item()
        assert abs(db[col] - want) <= 2 * h * h * size + 2.0 ** -11 * abs(want) + 2.0 ** -17 * size, (col, db[col], want)


def test_exact_sums_and_8_bit_form():
    """Small whole numbers: every sum is exact, so p, its 8-bit form and y are too."""
    g = torch.Generator().manual_seed(0)
    for tile, (m, k, n) in ((64, (19, 40, 70)), (128, (130, 64, 100)), (256, (130, 64, 300))):
        for gated in (False, True):
            parts = 2 if gated else 1
            a = torch.randint(-4, 5, (m, k), generator=g).bfloat16().cuda()
            w = torch.randint(-3, 4, (parts * n, k), generator=g).bfloat16().cuda()
            w[::7] = 0
            with agmm.FeedForwardPlan(1, m, k, n, BF16, activation="relu", gated=gated, with_gradient=False, tile=tile) as plan:
                y, saved = plan.forward([a], w, keep=8)
            p = a.double() @ w.double().t()
            s, _ = R.scales_of(p, n, parts)
            assert torch.equal(saved.scales.double(), s)
            full = torch.nn.functional.pad(p.view(m, parts, n), (0, -n % 32))
            q = (full / s.repeat_interleave(32, dim=2)).float().to(torch.float8_e4m3fn)
            assert torch.equal(saved.values.float(), q.float())
            want = p[:, :n].clamp(min=0) * (p[:, n:] if gated else 1)
            assert torch.equal(y, want.bfloat16())


@pytest.mark.parametrize("tile", [64, 128, 256])
def test_nan_and_infinity(tile):
    """A NaN in a row of A reaches that row alone; infinities follow IEEE arithmetic; the 8-bit form's other blocks keep
    their scales."""
    m, k, n = 40, 64, 96
    shards, w, b, r = make(1, m, k, n, BF16, 1, residual=True)
    clean = None
    for bad in (None, float("nan"), float("inf")):
        a = shards[0].clone()
        if bad is not None:
            a[7, 3] = bad
            w2 = w.clone()
            w2[:, 3] = w[:, 3].abs() + 0.25        # infinity times a positive number
        else:
            w2 = w.clone()
            w2[:, 3] = w[:, 3].abs() + 0.25
        with agmm.FeedForwardPlan(1, m, k, n, BF16, activation="gelu", tile=tile) as plan:
            y, saved = plan.forward([a], w2, b, r, keep=8)
            da, dw, db = plan.backward([a], w2, saved, r, need_dbias=True)
        if bad is None:
            clean = y, saved, da
            continue
        rows = [i for i in range(m) if i != 7]
        assert torch.equal(y[rows], clean[0][rows]) and torch.equal(da[rows], clean[2][rows])
        assert torch.equal(saved.values[rows].float(), clean[1].values[rows].float())
        assert torch.isnan(saved.values[7].float()).all()
        assert torch.isnan(y[7]).all() if bad != bad else torch.isinf(y[7]).all()
        assert torch.isnan(dw).any() and torch.isnan(db).all()


def test_one_infinite_pre_activation_in_a_block():
    """It becomes NaN in e4m3 and does not enter the block's scale."""
    m, k, n = 3, 16, 64
    a = torch.zeros((m, k)).half().cuda()
    a[:, 0] = 1
    w = torch.zeros((n, k)).half().cuda()
    w[:, 0] = torch.linspace(-3, 3, n).half()
    w[5, 0] = float("inf")
    for tile in (64, 128, 256):
        with agmm.FeedForwardPlan(1, m, k, n, FP16, with_gradient=False, tile=tile) as plan:
            y, saved = plan.forward([a], w, keep=8)
            y16, saved16 = plan.forward([a], w, keep=16)
        got = saved.dequantize()
        # 0 * inf is NaN in the sums of A's zero columns times W's infinity only where A is not 1
        assert torch.isnan(got[:, 5]).all() and torch.isfinite(got[:, :5]).all() and torch.isfinite(got[:, 6:]).all()
        want = w[:, 0].double()
        want[5] = 0
        s, _ = R.scales_of(want.expand(m, n).contiguous(), n, 1)
        assert torch.equal(saved.scales.double(), s)
        assert torch.isinf(y[:, 5]).all() and torch.isinf(saved16.dequantize()[:, 5]).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activation_range(act):
    """Pre-activations from the smallest to beyond the exponential's range: values and slopes."""
    x = torch.cat([torch.linspace(-14, 14, 1000), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 60, -60, 88, -88, 200, -200, 3e4, -3e4, 1e30, -1e30])])
    x = x.bfloat16()
    n = len(x)
    a = torch.zeros((2, 16)).bfloat16().cuda()
    a[:, 0] = 1
    w = torch.zeros((n, 16)).bfloat16().cuda()
    w[:, 0] = x.cuda()
    dy = torch.ones((2, n)).bfloat16().cuda()
    with agmm.FeedForwardPlan(1, 2, 16, n, BF16, activation=act) as plan:
        y, saved = plan.forward([a], w, keep=16)
        db = plan.backward([a], w, saved, dy, need_dA=False, need_dW=False, need_dbias=True)[2]
    v, slope = R.act(act, x.double())
    # beyond fp32's exponential the activation is 0: it is below 2^-120 there
    R.check(y[0].cpu(), v, 2.0 ** -8 * v.abs() + R.act_error(act, x.double()) * v.abs() * 1.01 + 1e-36, "value")
    R.check(db.cpu(), 2 * slope, 2.0 ** -8 * 2 * slope.abs() + 2.1 * R.slope_error(act, x.double()) + 1e-36, "slope")


def strided(rows, cols, ld, dtype, fill=float("nan")):
    return torch.full((rows, ld), fill, dtype=dtype, device="cuda")[:, :cols]


@pytest.mark.parametrize("k,n,lda,ldw,ldo,tile", [(64, 96, 72, 80, 104, -1), (64, 96, 65, 67, 97, 64), (130, 75, 131, 133, 77, 128),
                                                 (200, 300, 208, 200, 301, 256), (63, 33, 63, 64, 40, -1)])
@pytest.mark.parametrize("gated", [False, True])
def test_strides_and_rows_behind(k, n, lda, ldw, ldo, tile, gated):
    """Any stride; what lies between and behind the rows of the outputs stays."""
    N, ms, parts = 2, 70, 2 if gated else 1
    m = N * ms
    shards, w, b, r = make(N, ms, k, n, FP16, parts, residual=not gated)
    sh = []
    for s in shards:
        t = strided(ms, k, lda, torch.float16)
        t.copy_(s)
        sh.append(t)
    wt = strided(parts * n, k, ldw, torch.float16)
    wt.copy_(w)
    res = None
    if r is not None:
        res = strided(m, n, n + 5, torch.float16)
        res.copy_(r)
    dy = torch.randn((m, n), device="cuda").half()
    dys = strided(m, n, n + 3, torch.float16)
    dys.copy_(dy)
    with agmm.FeedForwardPlan(N, ms, k, n, FP16, activation="silu", gated=gated) as plain, \
            agmm.FeedForwardPlan(N, ms, k, n, FP16, activation="silu", gated=gated, lda=lda, ldw=ldw, ldr=n + 5, ldy=ldo, lddy=n + 3,
                                 ldda=k + 1, lddw=k + 9, tile=tile) as plan:
        def out(rows, cols, ld):
            whole = torch.full((rows + 1, ld), 7.0, dtype=torch.float16, device="cuda")
            return whole, whole[:rows, :cols]
        wy, y = out(m, n, ldo)
        wa, da = out(m, k, k + 1)
        ww, dw = out(parts * n, k, k + 9)
        _, saved = plan.forward(sh, wt, b, res, out=y, keep=8)
        want, bound, p, e = R.forward("silu", gated, torch.cat(shards), w, b, r, torch.float16)
        R.check(y, want, bound, "y")
        kept_matches(saved, p, e, n, parts, torch.float16)
        plan.backward(sh, wt, saved, dys, dA=da, dW=dw)
        _, *grads = R.gradient("silu", gated, saved.dequantize(), dy, torch.cat(shards), w, torch.float16)
        R.check(da, *grads[0], "dA")
        R.check(dw, *grads[1], "dW")
        for whole, view in ((wy, y), (wa, da), (ww, dw)):
            view.fill_(7.0)
            assert (whole == 7.0).all()
    with pytest.raises(ValueError):
        plain._on(y, plain._ly, "out")     # another stride than the plan's is refused


def test_residual_in_place():
    m, k, n = 300, 128, 256
    for tile in (64, 128, 256):
        shards, w, b, r = make(1, m, k, n, BF16, 1, residual=True)
        with agmm.FeedForwardPlan(1, m, k, n, BF16, with_gradient=False, tile=tile) as plan:
            want = plan.forward(shards, w, b, r)
            plan.forward(shards, w, b, r, out=r)
        assert torch.equal(r, want)


@pytest.mark.parametrize("offset", [1, 2, 7])
def test_element_alignment(offset):
    """Bias, residual, y, dy, dA, dW and dbias at any element."""
    m, k, n = 150, 72, 130

    def at(rows, cols):
        flat = torch.zeros(rows * cols + 8, dtype=torch.bfloat16, device="cuda")
        return flat[offset:offset + rows * cols].view(rows, cols)

    shards, w, b, r = make(1, m, k, n, BF16, 1, residual=True)
    dy = torch.randn((m, n), device="cuda").bfloat16()
    with agmm.FeedForwardPlan(1, m, k, n, BF16, activation="gelu") as plan:
        y, saved = plan.forward(shards, w, b, r, keep=16)
        want = plan.backward(shards, w, saved, dy, need_dbias=True)
        b2, r2, y2, g2 = at(1, n)[0], at(m, n), at(m, n), at(m, n)
        b2.copy_(b), r2.copy_(r), g2.copy_(dy)
        plan.forward(shards, w, b2, r2, out=y2)
        assert torch.equal(y2, y)
        got = plan.backward(shards, w, saved, g2, dA=at(m, k), dW=at(n, k), dbias=at(1, n)[0])
        for x, z in zip(got, want):
            assert torch.equal(x, z)
        assert torch.equal(plan.recompute(saved, out=at(m, n)), plan.recompute(saved))


def test_every_gradient_range_count():
    """Sums cut into ranges (few output tiles) and not: long n with small k and long m with small n."""
    for N, ms, k, n in ((1, 3000, 40, 50), (2, 20, 64, 4000), (1, 2500, 136, 1000), (5, 576, 64, 50), (3, 960, 200, 130)):
        shards, w, b, _ = make(N, ms, k, n, BF16, 1)
        dy = (torch.randn((N * ms, n), device="cuda") / 8).bfloat16()
        for tile in (-1, 128, 256):
            with agmm.FeedForwardPlan(N, ms, k, n, BF16, activation="silu", tile=tile) as plan:
                _, saved = plan.forward(shards, w, b, keep=16)
                got = plan.backward(shards, w, saved, dy, need_dbias=True)
                again = plan.backward(shards, w, saved, dy, need_dbias=True)
            _, *want = R.gradient("silu", False, saved.dequantize(), dy, torch.cat(shards), w, torch.bfloat16)
            for x, z, (exact, bound), what in zip(got, again, want, ("dA", "dW", "dbias")):
                R.check(x, exact, bound, what)
                assert torch.equal(x, z)           # fixed order: the same bits


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape", [(3, 21, 3814, 381), (1, 32, 2231, 36), (1, 63, 2050, 16), (4, 16, 4096, 17), (2, 100, 1537, 50),
                                   (1, 40, 1024, 100)], ids=str)
def test_few_rows_in_ranges_of_k(shape, gated):
    """Short y, long k: the few-row form adds ranges of k in a second launch, with everything that is done there."""
    N, ms, k, n = shape
    parts = 2 if gated else 1
    for i, (name, dtype, keep, pad) in enumerate([("silu", BF16, 8, 0), ("gelu", FP16, 16, 1), ("relu", BF16, 0, 3)]):
        shards, w, b, r = make(N, ms, k, n, dtype, parts, bias=i != 1, residual=not gated, seed=i)
        wide = torch.full((parts * n, k + pad), float("nan"), dtype=TYPE[dtype], device="cuda")
        wide[:, :k] = w
        want, bound, p, e = R.forward(name, gated, torch.cat(shards), w, b, r, TYPE[dtype])
        with agmm.FeedForwardPlan(N, ms, k, n, dtype, activation=name, gated=gated, with_gradient=False, tile=64, ldw=k + pad) as plan:
            assert plan.workspace_bytes() > 0 or k < 1500   # the ranges' sums: this form copies nothing
            first = plan.forward(shards, wide[:, :k], b, r, keep=keep)
            out = torch.full((N * ms, n), float("nan"), dtype=TYPE[dtype], device="cuda") if gated else r.clone()
            again = plan.forward(shards, wide[:, :k], b, None if gated else out, out=out, keep=keep)
            y, saved = first if keep else (first, None)
            R.check(y, want, bound, f"{name} y")
            assert torch.equal(y, out)               # in place and fixed order: the same bits
            if keep:
                kept_matches(saved, p, e, n, parts, TYPE[dtype])
                assert torch.equal(saved.values.view(torch.uint8), again[1].values.view(torch.uint8))


def test_tiles_agree_at_scale():
    """A training step's shapes: tiles of 256 with interior and edge tiles, XCD order and several shards per tile."""
    N, ms, k, n = 3, 700, 1024, 1100
    for gated in (False, True):
        parts = 2 if gated else 1
        shards, w, b, _ = make(N, ms, k, n, BF16, parts)
        dy = (torch.randn((N * ms, n), device="cuda") / 8).bfloat16()
        want = None
        for tile in (128, 224, 256):
            with agmm.FeedForwardPlan(N, ms, k, n, BF16, activation="gelu_tanh", gated=gated, tile=tile) as plan:
                y, saved = plan.forward(shards, w, b, keep=8)
                grads = plan.backward(shards, w, saved, dy, need_dbias=True)
            exact, bound, p, e = R.forward("gelu_tanh", gated, torch.cat(shards), w, b, None, torch.bfloat16)
            R.check(y, exact, bound, "y")
            kept_matches(saved, p, e, n, parts, torch.bfloat16)
            _, *refs = R.gradient("gelu_tanh", gated, saved.dequantize(), dy, torch.cat(shards), w, torch.bfloat16)
            for x, (ex, bo), what in zip(grads, refs, ("dA", "dW", "dbias")):
                R.check(x, ex, bo, what)


def test_captured_into_a_graph():
    """Forward and backward in one graph, replayed with eager calls of the same plan between the replays."""
    N, ms, k, n = 2, 100, 100, 90     # padded copies: the workspace is in use in both passes
    shards, w, b, _ = make(N, ms, k, n, BF16, 2)
    dy = torch.randn((N * ms, n), device="cuda").bfloat16()
    with agmm.FeedForwardPlan(N, ms, k, n, BF16, activation="silu", gated=True, tile=128) as plan:
        y, saved = plan.forward(shards, w, b, keep=8)
        da, dw, db = plan.backward(shards, w, saved, dy, need_dbias=True)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y2, saved2 = plan.forward(shards, w, b, keep=8)
            grads = plan.backward(shards, w, saved2, dy, need_dbias=True)
        for i in range(4):
            for t in (y2, saved2.values.view(torch.uint8), saved2.scales.view(torch.uint8), *grads):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y2, y) and torch.equal(saved2.values.view(torch.uint8), saved.values.view(torch.uint8))
            for a, z in zip(grads, (da, dw, db)):
                assert torch.equal(a, z)
            other = plan.forward([s * 2 for s in shards], w, b)     # eager, on the current stream
            torch.cuda.synchronize()
            assert not torch.equal(other, y)
        with pytest.raises(agmm.AgmmError):
            plan.set("tile", 256)
        del graph


def test_ranges_of_k_captured_into_a_graph():
    """Few rows whose ranges of k use the workspace, with and without kept pre-activations, replayed with eager calls between."""
    N, ms, k, n = 2, 20, 3001, 100
    shards, w, b, _ = make(N, ms, k, n, FP16, 2)
    dy = torch.randn((N * ms, n), device="cuda").half()
    with agmm.FeedForwardPlan(N, ms, k, n, FP16, activation="gelu", gated=True) as plan:
        want = [plan.forward(shards, w, b), *plan.forward(shards, w, b, keep=16)]
        da, dw, _ = plan.backward(shards, w, want[2], dy)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            y0 = plan.forward(shards, w, b)
            y1, saved = plan.forward(shards, w, b, keep=16)
            da1, dw1, _ = plan.backward(shards, w, saved, dy)
        for _ in range(4):
            for t in (y0, y1, saved.values, da1, dw1):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for t, z in ((y0, want[0]), (y1, want[1]), (saved.values, want[2].values), (da1, da), (dw1, dw)):
                assert torch.equal(t, z)
            other = plan.forward([s * 2 for s in shards], w, b)
            torch.cuda.synchronize()
            assert not torch.equal(other, want[0])
        del graph


def test_ranges_of_k_on_two_streams():
    """Calls that share the ranges' sums are ordered across streams."""
    N, ms, k, n = 1, 48, 4096, 60
    shards, w, b, _ = make(N, ms, k, n, BF16, 1)
    twice = [s * 2 for s in shards]
    with agmm.FeedForwardPlan(N, ms, k, n, BF16, activation="silu", with_gradient=False) as plan:
        assert plan.workspace_bytes() > 0
        want = [plan.forward(shards, w, b), plan.forward(twice, w, b)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(8):
            got = [plan.forward(a, w, b, stream=s) for a, s in zip((shards, twice), streams)]
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_outputs_over_operands_are_refused():
    m, k = 8, 32
    shards, w, b, r = make(1, m, k, k, BF16, 1, residual=True)
    with agmm.FeedForwardPlan(1, m, k, k, BF16) as plan:
        with pytest.raises(agmm.AgmmError, match="overlaps"):
            plan.forward(shards, w, b, out=shards[0])
        with pytest.raises(agmm.AgmmError, match="dA overlaps"):
            plan.backward(shards, w, None, r, dA=shards[0])
        with pytest.raises(agmm.AgmmError, match="dA overlaps"):
            plan.backward(shards, w, None, r, dA=r)
        with pytest.raises(agmm.AgmmError, match="dW overlaps"):
            plan.backward(shards, w, None, r, dW=w)
        plan.set("ldy", k + 8)
        wide = torch.zeros((m, k + 8), dtype=torch.bfloat16, device="cuda")
        dense = wide.view(-1)[:m * k].view(m, k)
        with pytest.raises(agmm.AgmmError, match="strides"):
            plan.forward(shards, w, b, dense, out=wide[:, :k])


def test_two_streams_share_a_plan():
    """Calls on two streams are ordered where they share the workspace."""
    N, ms, k, n = 2, 300, 500, 300
    shards, w, b, _ = make(N, ms, k, n, BF16, 2)
    dy = [torch.randn((N * ms, n), device="cuda").bfloat16() for _ in range(2)]
    with agmm.FeedForwardPlan(N, ms, k, n, BF16, activation="silu", gated=True) as plan:
        _, saved = plan.forward(shards, w, b, keep=8)
        want = [plan.backward(shards, w, saved, g) for g in dy]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [None, None]
        for turn in range(6):
            for i, s in enumerate(streams):
                got[i] = plan.backward(shards, w, saved, dy[i], stream=s)
            torch.cuda.synchronize()
            for i in range(2):
                for x, z in zip(got[i][:2], want[i][:2]):
                    assert torch.equal(x, z)


def test_refusals():
    shards, w, b, r = make(2, 8, 32, 16, BF16, 2, residual=True)
    with agmm.FeedForwardPlan(2, 8, 32, 16, BF16, activation="silu", gated=True, with_gradient=False) as plan:
        with pytest.raises(agmm.AgmmError, match="residual"):
            plan.forward(shards, w, b, r)
        with pytest.raises(agmm.AgmmError, match="workspace"):
            plan.backward(shards, w, plan.forward(shards, w, keep=16)[1], r)
        with pytest.raises(ValueError, match="keep"):
            plan.forward(shards, w, keep=4)
        with pytest.raises(ValueError, match="shards"):
            plan.forward(shards[:1], w)
        with pytest.raises(ValueError, match="shape"):
            plan.forward(shards, w[:16])
        with pytest.raises(TypeError, match="dtype"):
            plan.forward(shards, w.half())
    with pytest.raises(ValueError, match="activation"):
        agmm.FeedForwardPlan(1, 8, 32, 16, BF16, activation="tanh")
    with pytest.raises(agmm.AgmmError):
        agmm.FeedForwardPlan(1, 8, 32, 16, agmm.AGMM_FP32)
    with agmm.FeedForwardPlan(2, 8, 32, 16, BF16, activation="silu", gated=True) as plan:
        y, saved = plan.forward(shards, w, keep=8)
        dy = torch.zeros_like(y)
        with pytest.raises(agmm.AgmmError, match="saved is NULL"):
            plan.backward(shards, w, None, dy)
        with pytest.raises(TypeError):
            plan.backward(shards, w, saved.values, dy)
        with pytest.raises(TypeError, match="scales"):
            plan.backward(shards, w, agmm.Checkpoint(saved.values, None, 16), dy)
        with pytest.raises(ValueError, match="contiguous"):
            plan.backward(shards, w, agmm.Checkpoint(saved.values[:8], saved.scales, 16), dy)
        with pytest.raises(ValueError, match="columns"):
            plan.backward(shards, w, agmm.Checkpoint(saved.values, saved.scales, 15), dy)
        with pytest.raises(agmm.AgmmError, match="NULL"):
            plan.backward(shards, w, saved, dy, need_dA=False, need_dW=False)
        with pytest.raises(agmm.AgmmError):
            plan.set("lda", 31)
        with pytest.raises(agmm.AgmmError):
            plan.set("tile", 32)

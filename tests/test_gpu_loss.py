"""Vocabulary loss and its gradient on the GPU, against the formulas in 64 bits.

Tolerances.  u = 2^-24.
Logits: k exact products added in fp32, off by at most 2 k u sum |a w| (an
adder that truncates included) =: ex.  A row's lse then moves by at most the largest
of its logits' errors, plus the exponentials' and the sum's: v_exp and its
argument's rounding, 2^-22 (1 + the spread of the logits) relative each,
the sum's n u, and the last roundings, 4 u (|lse| + 1).
Gradient: p moves by its logit's error, relatively; d is rounded to 16 bits
(half a unit: 2^-9 bf16, 2^-12 fp16, relative to its largest part); the sums
over v (over i) of the sizes |d w| bound everything behind it, with the fp32
sum's 2 n u; the result is rounded once more to 16 bits.
Both 16-bit types end somewhere: a probability below 2^-126 is 0 (bf16 and
fp32 have no smaller normal number), which takes that much from d.
"""
import math

import numpy as np
import pytest
import torch

import all_gather_gemm_agmm_amd as agmm

pytestmark = pytest.mark.gpu

TYPES = {agmm.AGMM_BF16: torch.bfloat16, agmm.AGMM_FP16: torch.float16}
UNIT = {agmm.AGMM_BF16: 2.0 ** -8, agmm.AGMM_FP16: 2.0 ** -11}
FLOOR = {agmm.AGMM_BF16: 0.0, agmm.AGMM_FP16: 2.0 ** -24}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


class Case:
    def __init__(self, N, ms, k, n, dtype, start=0, total=None, seed=0, spread=3.0):
        g = torch.Generator().manual_seed(seed)
        self.N, self.ms, self.k, self.n, self.m = N, ms, k, n, N * ms
        self.dtype, self.start, self.total = dtype, start, start + n if total is None else total
        self.a = (torch.randn((self.m, k), generator=g)).to(TYPES[dtype])
        self.w = (torch.randn((n, k), generator=g) * spread / math.sqrt(k)).to(TYPES[dtype])
        self.labels = torch.randint(0, self.total, (self.m,), generator=g)
        self.gl = torch.rand(self.m, generator=g) / self.m
        self.gz = torch.randn(self.m, generator=g) * 0.01 / self.m

    def shards(self):
        return [s.contiguous().cuda() for s in self.a.split(self.ms)]

    def plan(self, **kw):
        return agmm.LossPlan(self.N, self.ms, self.k, self.n, self.dtype, vocab_start=self.start,
                             vocab_size=self.total, **kw)

    def logits(self):
        return self.a.double() @ self.w.double().t()

    def logit_error(self):
        return 2 * self.k * U * (self.a.double().abs() @ self.w.double().abs().t())

    def target(self, x):
        at = self.labels - self.start
        here = (at >= 0) & (at < self.n)
        return torch.where(here, x.gather(1, at.clamp(0, self.n - 1)[:, None])[:, 0], torch.zeros(self.m).double())


def check_forward(c, got, ignore=-100):
    loss, lse, target = (t.cpu().double() for t in got)
    x, ex = c.logits(), c.logit_error()
    ref, tgt = torch.logsumexp(x, 1), c.target(x)
    spread = (x.amax(1) - x.amin(1)) + 1
    bound = ex.amax(1) + 2.0 ** -22 * spread + c.n * U + 4 * U * (ref.abs() + 1)
    assert ((lse - ref).abs() <= bound).all(), ((lse - ref).abs() - bound).max()
    tb = ex.amax(1) + U * tgt.abs()
    assert ((target - tgt).abs() <= tb).all(), ((target - tgt).abs() - tb).max()
    off = c.labels == ignore
    assert (loss[off] == 0).all()
    bad = ~off & ((c.labels < 0) | (c.labels >= c.total))
    assert torch.isnan(loss[bad]).all()
    keep = ~off & ~bad
    assert ((loss - (ref - tgt)).abs() <= bound + tb + U * (ref - tgt).abs())[keep].all()
    return ref


def gradient_ref(c, lse, gl, gz, ignore=-100):
    """dA, dW in 64 bits and the bounds on their errors."""
    x, ex = c.logits(), c.logit_error()
    gl = torch.where(c.labels == ignore, torch.zeros(c.m).double(), gl.double())
    a = gl + (0 if gz is None else gz.double())
    p = torch.exp(x - lse.double()[:, None])
    d = a[:, None] * p
    at = c.labels - c.start
    hit = ((at >= 0) & (at < c.n)).nonzero()[:, 0]
    one = torch.zeros_like(d)
    one[hit, at[hit]] = gl[hit]
    d = d - one
    size = a.abs()[:, None] * p + one.abs()
    # error of d before the products: its logit's, the exponential's, the rounding to 16 bits
    expo = ex + 2.0 ** -22 * ((x - lse.double()[:, None]).abs() + 1)
    half, low = UNIT[c.dtype], 0.0 if c.dtype == agmm.AGMM_BF16 else 2.0 ** -38
    big = torch.maximum(a.abs(), gl.abs())
    low += 2.0 ** -126                           # where exp ends
    ed_row = a.abs()[:, None] * p * expo + half * size + low * big[:, None]      # fp16's smallest steps, by row ...
    ed_all = a.abs()[:, None] * p * expo + half * size + low * 2 * big.max()     # ... and by the largest row
    A, W = c.a.double(), c.w.double()
    dA, dW = d @ W, d.t() @ A
    bA = ed_row @ W.abs() + 2 * c.n * U * (size @ W.abs())
    bW = ed_all.t() @ A.abs() + 2 * c.m * U * (size.t() @ A.abs())
    bA += UNIT[c.dtype] * (dA.abs() + bA) + FLOOR[c.dtype]
    bW += UNIT[c.dtype] * (dW.abs() + bW) + FLOOR[c.dtype]
    return dA, dW, bA, bW


def check_backward(c, got, lse, gl, gz, ignore=-100):
    dA, dW, bA, bW = gradient_ref(c, lse, gl, gz, ignore)
    for name, g, ref, b in (("dA", got[0], dA, bA), ("dW", got[1], dW, bW)):
        if g is None:
            continue
        err = (g.cpu().double() - ref).abs()
        assert torch.isfinite(g).all(), name
        assert (err <= b).all(), (name, (err - b).max().item())
        # and as a whole well inside: roundings of both signs average out
        assert err.norm() <= 3 * UNIT[c.dtype] * ref.norm() + FLOOR[c.dtype] * math.sqrt(ref.numel()), name


def run_both(c, gz=True, **kw):
    with c.plan(**kw) as plan:
        s, w, lab = c.shards(), c.w.cuda(), c.labels.cuda()
        fwd = plan.forward(s, w, lab)
        ref = check_forward(c, fwd)
        lse = (ref + 0.5 * (c.total > c.n)).float()     # a merged lse is larger than the slice's
        z = c.gz if gz else None
        got = plan.backward(s, w, lab, lse.cuda(), c.gl.cuda(), None if z is None else z.cuda())
        torch.cuda.synchronize()
        check_backward(c, got, lse, c.gl, z)
    return fwd, got


SHAPES = [
    # N, ms, k, n
    (1, 1, 8, 1), (1, 1, 64, 7), (1, 3, 13, 300), (8, 1, 256, 1000), (3, 37, 100, 513), (2, 64, 128, 257),
    (2, 128, 512, 512), (1, 300, 72, 1030), (4, 70, 264, 777), (1, 513, 64, 2050), (64, 2, 40, 130),
]


@pytest.mark.parametrize("N,ms,k,n", SHAPES)
@pytest.mark.parametrize("dtype", [agmm.AGMM_BF16, agmm.AGMM_FP16])
def test_loss_and_gradient(N, ms, k, n, dtype):
    run_both(Case(N, ms, k, n, dtype, seed=n))


@pytest.mark.parametrize("dtype", [agmm.AGMM_BF16, agmm.AGMM_FP16])
@pytest.mark.parametrize("part", [0, 1, 2])
def test_slice_of_a_vocabulary(part, dtype):
    run_both(Case(2, 33, 136, 300, dtype, start=300 * part, total=900, seed=part), gz=False)


@pytest.mark.parametrize("k", [96, 99])
def test_pieces(k):
    """Several pieces, the last one ragged: the same bounds, and the same
    loss whatever the piece."""
    c = Case(2, 70, k, 1400, agmm.AGMM_BF16, seed=4)
    one, _ = run_both(c, piece=4096)
    many, _ = run_both(c, piece=256)
    torch.testing.assert_close(one[1], many[1], rtol=4 * U, atol=4 * U)
    assert torch.equal(one[2], many[2])


@pytest.mark.parametrize("tile", [128, 256])
def test_large_tiles(tile):
    """Rows and columns for rounds of either tile in every pass."""
    c = Case(2, 2048, 512, 8192, agmm.AGMM_BF16, seed=1)
    with c.plan() as plan:
        plan.set("tile", tile)
        assert plan.get("tile") == tile
    run_both(c, tile=tile)


def test_tile_by_the_sum():
    """Long sums over many rows and columns take 256 x 256 tiles, a few rows 128 x 128."""
    with agmm.LossPlan(1, 4096, 4096, 65536, agmm.AGMM_BF16) as plan:
        assert plan.get("tile") == 256
    with agmm.LossPlan(1, 64, 4096, 65536, agmm.AGMM_BF16) as plan:
        assert plan.get("tile") == 128


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("shape", [(1, 1, 8, 3), (3, 45, 203, 777), (2, 129, 72, 258)])
@pytest.mark.parametrize("dt", [agmm.AGMM_BF16, agmm.AGMM_FP16])
def test_each_tile_at_ragged_sizes(shape, dt, tile):
    run_both(Case(*shape, dt, seed=21), tile=tile)


@pytest.mark.parametrize("N,ms,k,n", [
    (1, 1, 1, 1), (1, 1, 64, 15), (1, 16, 333, 4100), (2, 8, 640, 35000), (3, 5, 72, 17), (1, 17, 31, 64), (4, 16, 513, 1025),
    (1, 64, 1030, 70), (5, 13, 257, 300), (1, 150, 96, 33), (8, 3, 2049, 130), (2, 20, 100, 33001)])
@pytest.mark.parametrize("dt", [agmm.AGMM_BF16, agmm.AGMM_FP16])
def test_few_rows(N, ms, k, n, dt):
    """The form for few rows, at every block size: its row, column and k ends."""
    run_both(Case(N, ms, k, n, dt, seed=31), tile=64)


def test_few_rows_with_strides_and_pieces():
    """Rows of any length apart, no copies, several pieces."""
    c = Case(2, 9, 203, 1400, agmm.AGMM_FP16, seed=32)
    fwd, got = run_both(c, tile=64, piece=512)
    shards = [torch.zeros((c.ms, 211), dtype=torch.float16, device="cuda")[:, :203].copy_(s) for s in c.shards()]
    w = torch.zeros((c.n, 205), dtype=torch.float16, device="cuda")[:, :203].copy_(c.w.cuda())
    with c.plan(tile=64, piece=512, lda=211, ldw=205) as plan:
        strided = plan.forward(shards, w, c.labels.cuda())
        back = plan.backward(shards, w, c.labels.cuda(), strided[1], c.gl.cuda(), c.gz.cuda())
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(fwd, strided))
    check_backward(c, back, strided[1].cpu(), c.gl, c.gz)


def test_form_by_the_sizes():
    """An unaligned W is read in place for few rows; long aligned ones by tiles."""
    with agmm.LossPlan(1, 8, 1001, 50000, agmm.AGMM_BF16, with_gradient=False) as plan:
        assert plan.get("tile") == 64 and plan.workspace_bytes() < 1 << 20
    with agmm.LossPlan(1, 4096, 1001, 50000, agmm.AGMM_BF16, with_gradient=False) as plan:
        assert plan.get("tile") > 64


def test_one_pass_of_two():
    c = Case(1, 40, 64, 300, agmm.AGMM_BF16, seed=2)
    with c.plan() as plan:
        s, w, lab = c.shards(), c.w.cuda(), c.labels.cuda()
        lse, gl = torch.logsumexp(c.logits(), 1).float().cuda(), c.gl.cuda()
        dA, none = plan.backward(s, w, lab, lse, gl, need_dW=False)
        assert none is None
        none, dW = plan.backward(s, w, lab, lse, gl, need_dA=False)
        assert none is None
        torch.cuda.synchronize()
        check_backward(c, (dA, dW), lse.cpu(), c.gl, None)


def test_ignored_rows():
    """Ignored rows: loss 0 and no gradient of it; the lse's gradient stays.  All rows ignored: zeros."""
    c = Case(2, 50, 64, 400, agmm.AGMM_BF16, seed=3)
    c.labels[::3] = -100
    run_both(c)
    c.labels[:] = -100
    with c.plan() as plan:
        s, w, lab = c.shards(), c.w.cuda(), c.labels.cuda()
        loss, lse, target = plan.forward(s, w, lab)
        dA, dW = plan.backward(s, w, lab, lse, c.gl.cuda())
        torch.cuda.synchronize()
        assert (loss == 0).all() and (target == 0).all() and (dA == 0).all() and (dW == 0).all()
        plan.set("ignore_index", 7)
        c.labels[:] = 7
        assert (plan.forward(s, w, c.labels.cuda())[0] == 0).all()


def test_labels_outside_the_vocabulary_are_nan():
    c = Case(1, 20, 64, 100, agmm.AGMM_BF16, start=100, total=300, seed=5)
    c.labels[3], c.labels[7] = 300, -5
    with c.plan() as plan:
        s, w, lab = c.shards(), c.w.cuda(), c.labels.cuda()
        fwd = plan.forward(s, w, lab)
        check_forward(c, fwd)
        dA, dW = plan.backward(s, w, lab, fwd[1], c.gl.cuda())
        torch.cuda.synchronize()
    bad = torch.isnan(dA).all(1).cpu()
    assert bad.nonzero()[:, 0].tolist() == [3, 7] and torch.isnan(dW).all()
    assert torch.isfinite(dA[~bad.cuda()]).all()


def test_special_logits():
    """Rows whose logits are infinite or NaN follow log-sum-exp; the others do not notice."""
    c = Case(1, 6, 8, 300, agmm.AGMM_BF16, seed=6)
    c.a[:, 0] = 0.0
    c.w[:, 0] = 0.0
    c.w[5, 0] = 1.0
    inf = float("inf")
    c.a[1, 0], c.a[2, 0] = inf, -inf          # x[1, 5] = inf, the rest inf * 0 = NaN
    c.labels[:] = 9
    with c.plan() as plan:
        loss, lse, target = (t.cpu() for t in plan.forward(c.shards(), c.w.cuda(), c.labels.cuda()))
    assert torch.isnan(lse[1:3]).all() and torch.isnan(loss[1:3]).all()
    assert torch.isfinite(lse[[0, 3, 4, 5]]).all()
    # one column only: a row of -inf gives -inf, a row of +inf gives +inf
    c = Case(1, 4, 8, 1, agmm.AGMM_BF16, seed=6)
    c.a[:, 0], c.w[:, 0] = torch.tensor([inf, -inf, 1.0, 0.0]).bfloat16(), 1.0
    c.labels[:] = 0
    with c.plan() as plan:
        loss, lse, target = (t.cpu() for t in plan.forward(c.shards(), c.w.cuda(), c.labels.cuda()))
    assert lse[0] == inf and lse[1] == -inf and torch.isfinite(lse[2:]).all() and (loss[2:] == 0).all()


@pytest.mark.parametrize("dtype", [agmm.AGMM_BF16, agmm.AGMM_FP16])
def test_large_logits(dtype):
    """Logits of hundreds: exp never overflows, the loss of a certain row is 0."""
    c = Case(1, 30, 64, 500, dtype, seed=8, spread=60.0)
    run_both(c)


def test_gradient_scales():
    """Upstream gradients from 1e-8 to 1, zeros among them: fp16's range does not cut dA's rows."""
    c = Case(1, 64, 64, 300, agmm.AGMM_FP16, seed=9)
    c.gl = torch.pow(10.0, -4 * torch.rand(64, generator=torch.Generator().manual_seed(0)))
    c.gl[::8] = 0.0
    run_both(c, gz=False)


def test_strides():
    c = Case(2, 30, 64, 200, agmm.AGMM_BF16, seed=10)
    for lda, ldw, ldda, lddw in ((72, 80, 66, 68), (65, 67, 64, 65)):
        def wide(x, ld):
            buf = torch.full((x.shape[0], ld), float("nan"), dtype=x.dtype, device="cuda")
            buf[:, :64] = x.cuda()
            return buf[:, :64]
        outA = torch.full((60, ldda), -7.0, dtype=torch.bfloat16, device="cuda")
        outW = torch.full((200, lddw), -7.0, dtype=torch.bfloat16, device="cuda")
        with c.plan(lda=lda, ldw=ldw, ldda=ldda, lddw=lddw) as plan:
            s, w, lab = [wide(x, lda) for x in c.a.split(30)], wide(c.w, ldw), c.labels.cuda()
            fwd = plan.forward(s, w, lab)
            check_forward(c, fwd)
            got = plan.backward(s, w, lab, fwd[1], c.gl.cuda(), c.gz.cuda(), outA[:, :64], outW[:, :64])
            torch.cuda.synchronize()
        check_backward(c, got, fwd[1].cpu(), c.gl, c.gz)
        assert (outA[:, 64:] == -7).all() and (outW[:, 64:] == -7).all()


def test_gradient_against_differences():
    """Central differences of the loss the kernels compute, along random
    directions: (L(x + h d) - L(x - h d)) / 2h against <grad, d>.  W and A move on
    exact steps of their types; L is summed in 64 bits.  The difference's
    truncation is h^2 and its rounding 1e-6 / h: 1% together at the chosen h."""
    c = Case(1, 24, 64, 200, agmm.AGMM_FP16, seed=11)
    g = torch.Generator().manual_seed(12)
    gl = torch.rand(24, generator=g)
    with c.plan() as plan:
        lab = c.labels.cuda()
        _, lse, _ = plan.forward(c.shards(), c.w.cuda(), lab)
        dA, dW = plan.backward(c.shards(), c.w.cuda(), lab, lse, gl.cuda())

        def total(a, w):
            return (plan.forward([a.cuda()], w.cuda(), lab)[0].cpu().double() * gl.double()).sum()

        h = 2.0 ** -5
        for which in range(6):
            base = c.a if which % 2 == 0 else c.w
            d = torch.randn(base.shape, generator=g)
            up, down = (base.float() + h * d).half(), (base.float() - h * d).half()
            step = (up.double() - down.double()) / (2 * h)         # the direction as it was taken
            args = [(up, c.w), (down, c.w)] if which % 2 == 0 else [(c.a, up), (c.a, down)]
            diff = (total(*args[0]) - total(*args[1])) / (2 * h)
            grad = dA if which % 2 == 0 else dW
            want = (grad.cpu().double() * step).sum()
            scale = grad.cpu().double().norm() * step.norm() / math.sqrt(step.numel())
            assert abs(diff - want) <= 0.02 * scale + 0.02 * abs(want), (which, diff.item(), want.item(), scale.item())


def test_slices_merge_to_the_whole():
    """Three slices of one vocabulary, merged, against the whole in one plan; the
    slices' dA add up to the whole's."""
    whole = Case(2, 20, 64, 600, agmm.AGMM_BF16, seed=13)
    with whole.plan() as plan:
        loss, lse, target = plan.forward(whole.shards(), whole.w.cuda(), whole.labels.cuda())
        dA, dW = plan.backward(whole.shards(), whole.w.cuda(), whole.labels.cuda(), lse, whole.gl.cuda())
    parts = []
    for i in range(3):
        c = Case(2, 20, 64, 600, agmm.AGMM_BF16, seed=13)
        c.w, c.n, c.start, c.total = whole.w[200 * i:200 * (i + 1)].clone(), 200, 200 * i, 600
        parts.append((c, c.plan()))
    out = [p.forward(c.shards(), c.w.cuda(), c.labels.cuda()) for c, p in parts]
    merged, mlse = agmm.merge_vocab_slices(torch.stack([o[1] for o in out]), torch.stack([o[2] for o in out]),
                                           whole.labels.cuda(), 600)
    torch.testing.assert_close(mlse, lse, rtol=0, atol=2.0 ** -19)
    torch.testing.assert_close(merged, loss, rtol=0, atol=2.0 ** -18)
    grads = [p.backward(c.shards(), c.w.cuda(), c.labels.cuda(), mlse, whole.gl.cuda()) for c, p in parts]
    total = sum(g[0].double() for g in grads)
    assert ((total - dA.double()).norm() / dA.double().norm()).item() < 3 * 2.0 ** -8
    assert ((torch.cat([g[1] for g in grads]).double() - dW.double()).norm() / dW.double().norm()).item() < 3 * 2.0 ** -8


def test_calls_on_several_streams_and_twice_the_same():
    """One plan on two streams: its workspace is not shared at one time; equal calls give equal bits."""
    sets = [Case(2, 100, 128, 1000, agmm.AGMM_BF16, seed=20 + i) for i in range(2)]
    with sets[0].plan() as plan:
        dev = [(c.shards(), c.w.cuda(), c.labels.cuda(), c.gl.cuda()) for c in sets]
        want = []
        for s, w, lab, gl in dev:
            f = plan.forward(s, w, lab)
            want.append(f + plan.backward(s, w, lab, f[1], gl))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [[], []]
        for _ in range(10):
            for i, (s, w, lab, gl) in enumerate(dev):
                f = plan.forward(s, w, lab, stream=streams[i])
                got[i].append(f + plan.backward(s, w, lab, f[1], gl, stream=streams[i]))
        torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(g, want[i]))


def test_calls_that_overlap_keep_their_operands():
    """A call that another one of the same plan overtakes, as one of another
    thread can, between the reading of its shards: both are right."""
    cases = [Case(2, 30, 72, 300, agmm.AGMM_BF16, seed=51 + i) for i in range(2)]
    sets = [(c.shards(), c.w.cuda(), c.labels.cuda()) for c in cases]
    other = []
    with cases[0].plan() as plan:
        want = [plan.forward(*s) for s in sets]

        class Overtaken(list):
            def __iter__(self):
                yield self[0]
                yield self[1]
                other.append(plan.forward(*sets[1]))

        got = plan.forward(Overtaken(sets[0][0]), *sets[0][1:])
        torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want[0]))
    assert all(torch.equal(g, w) for g, w in zip(other[0], want[1]))


def test_in_a_graph():
    c = Case(2, 60, 128, 900, agmm.AGMM_BF16, seed=14)
    with c.plan() as plan:
        s, w, lab, gl = c.shards(), c.w.cuda(), c.labels.cuda(), c.gl.cuda()
        dA = torch.empty((120, 128), dtype=torch.bfloat16, device="cuda")
        dW = torch.empty((900, 128), dtype=torch.bfloat16, device="cuda")
        f = plan.forward(s, w, lab)
        want = [t.clone() for t in f + plan.backward(s, w, lab, f[1], gl, dA=dA, dW=dW)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = plan.forward(s, w, lab)
            plan.backward(s, w, lab, out[1], gl, dA=dA, dW=dW)
        for _ in range(4):
            dA.zero_()
            dW.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out + (dA, dW), want))
        del graph


def test_refusals(monkeypatch):
    with pytest.raises(agmm.AgmmError) as ei:
        agmm.LossPlan(1, 8, 64, 100, agmm.AGMM_FP32)
    assert ei.value.status == agmm.AGMM_ERR_UNSUPPORTED
    with pytest.raises(agmm.AgmmError, match="vocabulary"):
        agmm.LossPlan(1, 8, 64, 100, vocab_start=50, vocab_size=120)
    c = Case(1, 8, 64, 100, agmm.AGMM_BF16)
    s, w, lab = c.shards(), c.w.cuda(), c.labels.cuda()
    with c.plan(with_gradient=False) as plan:
        lse = plan.forward(s, w, lab)[1]
        with pytest.raises(agmm.AgmmError) as ei:
            plan.backward(s, w, lab, lse, c.gl.cuda())
        assert ei.value.status == agmm.AGMM_ERR_UNSUPPORTED
        with pytest.raises(TypeError, match="dtype"):
            plan.forward(s, w, lab.int())
        with pytest.raises(TypeError, match="dtype"):
            plan.forward(s, w.half(), lab)
        with pytest.raises(ValueError, match="shape"):
            plan.forward(s, w[:50], lab)
        with pytest.raises(ValueError, match="shards"):
            plan.forward(s + s, w, lab)
        with pytest.raises(ValueError, match="GPU"):
            plan.forward(s, w, lab.cpu())
        for key, val in (("lda", 63), ("ldw", -1), ("piece", -1), ("tile", 0)):
            with pytest.raises(agmm.AgmmError) as ei:
                plan.set(key, val)
            assert ei.value.status == agmm.AGMM_ERR_INVALID_ARG
    with c.plan() as plan:
        with pytest.raises(agmm.AgmmError, match="both NULL"):
            plan.backward(s, w, lab, lse, c.gl.cuda(), need_dA=False, need_dW=False)
        monkeypatch.setenv("AGMM_TEST_FAIL_ALLOC", "1")
        before = plan.get("piece")
        with pytest.raises(agmm.AgmmError) as ei:
            plan.set("lda", 65)              # needs padded copies, and with them more workspace
        assert ei.value.status == agmm.AGMM_ERR_OOM
        assert plan.get("lda") == 64 and plan.get("piece") == before
        check_forward(c, plan.forward(s, w, lab))
        with pytest.raises(agmm.AgmmError) as ei:
            c.plan()
        assert ei.value.status == agmm.AGMM_ERR_OOM


def test_example_trains():
    """examples/vocab_head_step.py: the 8-bit projection, the loss and both
    ways back, run together; the loss falls, dx matches the formula on the
    dequantised operands."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "vocab_head_step.py")
    spec = importlib.util.spec_from_file_location("vocab_head_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for rows in (64, 128):
        head = mod.Head(rows=rows)
        first, dx = head.step()
        assert dx.shape == (head.m, 256) and torch.isfinite(dx).all() and dx.float().norm() > 0
        assert (dx[::16] == 0).all()                       # rows without a target
        for _ in range(14):
            last, _ = head.step()
        head.close()
        assert abs(first.item() - math.log(head.vocab)) < 1.0
        assert last.item() < 0.7 * first.item()

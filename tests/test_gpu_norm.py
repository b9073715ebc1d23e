"""Layer norm and its gradient on the GPU, against the formulas in 64 bits (feed_reference.py)."""
import pytest
import torch

import all_gather_gemm_agmm_amd as agmm
import feed_reference as R

pytestmark = pytest.mark.gpu

TYPE = {agmm.AGMM_BF16: torch.bfloat16, agmm.AGMM_FP16: torch.float16, agmm.AGMM_FP32: torch.float32}
KINDS = [(agmm.AGMM_BF16, agmm.AGMM_BF16), (agmm.AGMM_BF16, agmm.AGMM_FP32), (agmm.AGMM_FP16, agmm.AGMM_FP16),
         (agmm.AGMM_FP16, agmm.AGMM_FP32), (agmm.AGMM_FP32, agmm.AGMM_FP32)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


def make(rows, cols, dtype, wtype, offset=0.5, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * rows + cols)
    x = (torch.randn((rows, cols), generator=g) * 1.5 + offset).to(TYPE[dtype]).cuda()
    dy = torch.randn((rows, cols), generator=g).to(TYPE[dtype]).cuda()
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(TYPE[wtype]).cuda()
    b = (0.3 * torch.randn(cols, generator=g)).to(TYPE[wtype]).cuda()
    return x, dy, w, b


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (5, 7), (2, 64), (9, 255), (1, 512), (300, 513), (4, 1025), (17, 2048), (3, 2050),
                                       (70, 4096), (5, 4101), (2, 8192), (6, 8200), (2, 32768), (3, 40003), (1100, 96), (5000, 16)])
def test_norm(rows, cols, kind):
    dtype, wtype = kind
    x, dy, w, b = make(rows, cols, dtype, wtype)
    with agmm.NormPlan(rows, cols, dtype, wtype) as plan:
        for weight, bias in ((w, b), (None, None), (w, None)):
            got = plan.forward(x, weight, bias)
            for t, (want, bound), what in zip(got, R.norm(x, weight, bias, 1e-5, TYPE[dtype]), ("y", "mean", "rstd")):
                R.check(t, want, bound, what)
            _, mean, rstd = got
            grads = plan.backward(x, dy, weight, mean, rstd)
            wants = R.norm_gradient(x, dy, weight, mean, rstd, TYPE[dtype], TYPE[wtype])
            for t, (want, bound), what in zip(grads, wants, ("dx", "dweight", "dbias")):
                R.check(t, want, bound, what)
            again = plan.backward(x, dy, weight, mean, rstd)
            assert all(torch.equal(s, t) for s, t in zip(grads, again))


def test_gradient_against_differences():
    """dx and dweight of sum(y * c) against central differences of the 64-bit formula."""
    rows, cols = 4, 24
    x, dy, w, b = make(rows, cols, agmm.AGMM_FP32, agmm.AGMM_FP32)
    with agmm.NormPlan(rows, cols, agmm.AGMM_FP32) as plan:
        _, mean, rstd = plan.forward(x, w, b)
        dx, dw, db = (t.double().cpu() for t in plan.backward(x, dy, w, mean, rstd))

    def total(x, w):
        mu = x.mean(1, keepdim=True)
        return (((x - mu) / ((x - mu).pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * w + b.double().cpu()) * dy.double().cpu()).sum()

    xd, wd, h = x.double().cpu(), w.double().cpu(), 1e-5
    for i in range(rows):
        for j in range(cols):
            step = torch.zeros_like(xd)
            step[i, j] = h
            assert abs((total(xd + step, wd) - total(xd - step, wd)) / (2 * h) - dx[i, j]) < 1e-5
    for j in range(cols):
        step = torch.zeros_like(wd)
        step[j] = h
        assert abs((total(xd, wd + step) - total(xd, wd - step)) / (2 * h) - dw[j]) < 1e-5
    assert (db - dy.double().cpu().sum(0)).abs().max() < 1e-5


def test_rows_far_from_zero():
    """A mean a thousand times the deviation: the variance is that of the differences."""
    for cols in (100, 4096, 20000):
        x = (1000 + torch.randn((8, cols), generator=torch.Generator().manual_seed(cols))).cuda()
        with agmm.NormPlan(8, cols, agmm.AGMM_FP32) as plan:
            y, mean, rstd = plan.forward(x)
        d = x.double()
        d = d - d.mean(1, keepdim=True)
        want = d / (d.pow(2).mean(1, keepdim=True) + 1e-5).sqrt()
        # x - mean is off by a step of 1000 in 32 bits, 2^-14, relative to a deviation of 1
        assert (y.double() - want).abs().max() < 2.0 ** -13 and (rstd.double() * d.pow(2).mean(1).add(1e-5).sqrt() - 1).abs().max() < 1e-5


def test_constant_rows_and_one_column():
    x = torch.tensor([[3.0] * 40, [0.0] * 40, [-1e4] * 40]).cuda()
    b = torch.randn(40).cuda()
    with agmm.NormPlan(3, 40, agmm.AGMM_FP32) as plan:
        y, mean, rstd = plan.forward(x, None, b)
        assert torch.equal(y, b.expand(3, 40)) and torch.equal(mean.cpu(), torch.tensor([3.0, 0.0, -1e4]))
        assert (rstd - 1e-5 ** -0.5).abs().max() < 1e-2
        dx, dw, db = plan.backward(x, torch.ones_like(x), None, mean, rstd)
        assert (dx.abs() <= 316.3 * 2.0 ** -20).all() and (dw == 0).all() and (db == 3).all()


def test_nan_and_infinity_stay_in_their_row():
    for cols in (60, 4096, 40000):
        x, dy, w, b = make(5, cols, agmm.AGMM_BF16, agmm.AGMM_FP32)
        with agmm.NormPlan(5, cols, agmm.AGMM_BF16, agmm.AGMM_FP32) as plan:
            y, mean, rstd = plan.forward(x, w, b)
            for bad in (float("nan"), float("inf")):
                z = x.clone()
                z[2, cols // 2] = bad
                got, mu, rs = plan.forward(z, w, b)
                keep = [0, 1, 3, 4]
                assert torch.equal(got[keep], y[keep]) and torch.equal(mu[keep], mean[keep]) and torch.equal(rs[keep], rstd[keep])
                assert torch.isnan(got[2]).all()
                dx, dw, db = plan.backward(z, dy, w, mu, rs)
                assert torch.isnan(dx[2]).all() and torch.isfinite(dx[keep]).all() and torch.isnan(dw).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("cols", [96, 1000, 4096, 20000])
@pytest.mark.parametrize("extra", [1, 2, 8])
def test_strides_offsets_and_rows_behind(cols, extra):
    rows = 20
    x, dy, w, b = make(rows, cols, agmm.AGMM_BF16, agmm.AGMM_BF16)
    with agmm.NormPlan(rows, cols, agmm.AGMM_BF16) as dense, \
            agmm.NormPlan(rows, cols, agmm.AGMM_BF16, ldx=cols + extra, ldy=cols + extra, lddy=cols + 3, lddx=cols + extra) as plan:
        def out(ld):
            whole = torch.full((rows * ld + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
            return whole, whole[1:1 + rows * ld].view(rows, ld)[:, :cols]
        xs, gs = out(cols + extra)[1], out(cols + 3)[1]
        xs.copy_(x), gs.copy_(dy)
        wy, y = out(cols + extra)
        wx, dx = out(cols + extra)
        want = dense.forward(x, w, b)
        got = plan.forward(xs, w, b, out=y)
        assert all(torch.equal(s, t) for s, t in zip(got, want))
        ref = dense.backward(x, dy, w, *want[1:])
        grads = plan.backward(xs, gs, w, *want[1:], dx=dx)
        assert all(torch.equal(s, t) for s, t in zip(grads, ref))
        for whole, view in ((wy, y), (wx, dx)):
            view.fill_(7.0)
            assert (whole == 7.0).all()


@pytest.mark.parametrize("cols", [100, 5000, 40000])
def test_in_place(cols):
    """y over x and dx over dy."""
    x, dy, w, b = make(7, cols, agmm.AGMM_FP16, agmm.AGMM_FP16)
    with agmm.NormPlan(7, cols, agmm.AGMM_FP16) as plan:
        y, mean, rstd = plan.forward(x, w, b)
        want = plan.backward(x, dy, w, mean, rstd)
        got = plan.backward(x, dy, w, mean, rstd, dx=dy)
        assert got[0] is dy and all(torch.equal(s, t) for s, t in zip(got, want))
        assert torch.equal(plan.forward(x, w, b, out=x)[0], y)


def test_each_gradient_alone():
    for cols in (100, 40000):
        x, dy, w, b = make(30, cols, agmm.AGMM_BF16, agmm.AGMM_FP32)
        with agmm.NormPlan(30, cols, agmm.AGMM_BF16, agmm.AGMM_FP32) as plan:
            _, mean, rstd = plan.forward(x, w, b)
            all3 = plan.backward(x, dy, w, mean, rstd)
            for i in range(3):
                only = plan.backward(x, dy, w, mean, rstd, need_dx=i == 0, need_dweight=i == 1, need_dbias=i == 2)
                assert [t is None for t in only] == [j != i for j in range(3)] and torch.equal(only[i], all3[i])


def test_captured_into_a_graph():
    x, dy, w, b = make(200, 1000, agmm.AGMM_BF16, agmm.AGMM_FP32)
    with agmm.NormPlan(200, 1000, agmm.AGMM_BF16, agmm.AGMM_FP32) as plan:
        want = plan.forward(x, w, b)
        ref = plan.backward(x, dy, w, *want[1:])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            got = plan.forward(x, w, b)
            grads = plan.backward(x, dy, w, *got[1:])
        for i in range(4):
            for t in (*got, *grads):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(s, t) for s, t in zip((*got, *grads), (*want, *ref)))
            plan.backward(x, x, w, *want[1:])
            torch.cuda.synchronize()
        with pytest.raises(agmm.AgmmError):
            plan.set("ldx", 1008)
        del graph


def test_two_streams_share_a_plan():
    x, dy, w, b = make(3000, 2000, agmm.AGMM_BF16, agmm.AGMM_FP32)
    dys = [dy, (dy * 2).contiguous()]
    with agmm.NormPlan(3000, 2000, agmm.AGMM_BF16, agmm.AGMM_FP32) as plan:
        _, mean, rstd = plan.forward(x, w, b)
        want = [plan.backward(x, g, w, mean, rstd) for g in dys]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for turn in range(6):
            got = [plan.backward(x, g, w, mean, rstd, stream=s) for g, s in zip(dys, streams)]
            torch.cuda.synchronize()
            assert all(torch.equal(s, t) for a, c in zip(got, want) for s, t in zip(a, c))


def test_refusals():
    x, dy, w, b = make(4, 32, agmm.AGMM_BF16, agmm.AGMM_BF16)
    with agmm.NormPlan(4, 32, agmm.AGMM_BF16) as plan:
        for eps in (-1e-5, float("nan"), float("inf")):
            with pytest.raises(agmm.AgmmError, match="eps"):
                plan.forward(x, w, b, eps=eps)
        with pytest.raises(TypeError, match="dtype"):
            plan.forward(x, w.float(), b)
        with pytest.raises(ValueError, match="shape"):
            plan.forward(x[:3], w, b)
        _, mean, rstd = plan.forward(x, w, b)
        with pytest.raises(agmm.AgmmError, match="NULL"):
            plan.backward(x, dy, w, mean, rstd, need_dx=False, need_dweight=False, need_dbias=False)
        with pytest.raises(agmm.AgmmError):
            plan.set("ldx", 31)
    with pytest.raises(agmm.AgmmError, match="weights have"):
        agmm.NormPlan(4, 32, agmm.AGMM_BF16, agmm.AGMM_FP16)


def test_outputs_over_operands_are_refused():
    x, dy, w, b = make(4, 32, agmm.AGMM_BF16, agmm.AGMM_BF16)
    with agmm.NormPlan(4, 32, agmm.AGMM_BF16) as plan:
        _, mean, rstd = plan.forward(x, w, b)
        with pytest.raises(agmm.AgmmError, match="dx overlaps"):
            plan.backward(x, dy, w, mean, rstd, dx=x)
        wide = torch.zeros((4, 40), dtype=torch.bfloat16, device="cuda")
        dense = wide.view(-1)[:128].view(4, 32)
        plan.set("ldy", 40)
        with pytest.raises(agmm.AgmmError, match="strides"):
            plan.forward(dense, w, b, out=wide[:, :32])
        plan.set("lddx", 40)
        with pytest.raises(agmm.AgmmError, match="strides"):
            plan.backward(x, dense, w, mean, rstd, dx=wide[:, :32])

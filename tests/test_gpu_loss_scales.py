"""fp16 gradients of the vocabulary loss over the whole range of row weights,
against the formulas in 64 bits; bounds as in test_gpu_loss.py."""
import pytest
import torch

import all_gather_gemm_agmm_amd as agmm
from test_gpu_loss import Case, check_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


SHAPES = [(1, 64, 64, 300), (3, 70, 203, 520), (2, 300, 72, 300)]


def run_backward(c, tile):
    lse = torch.logsumexp(c.logits(), 1).float()
    with c.plan(tile=tile) as plan:
        got = plan.backward(c.shards(), c.w.cuda(), c.labels.cuda(), lse.cuda(), c.gl.cuda(), c.gz.cuda())
        torch.cuda.synchronize()
    check_backward(c, got, lse, c.gl, c.gz)
    return got


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("gl,gz,largest", [(0.49999, -0.99998, 1.0), (1.9998, -3.9996, 16.0), (-1.9999, 3.9998, 1.0),
                                           (0.99999, -1.99998, 0.99999)])
def test_gradients_of_opposite_sign(gl, gz, largest, tile, shape):
    """Rows whose loss and lse have gradients of opposite sign and p = 1 at the
    label: d there is the sum of both, twice the larger of |gl + gz| and |gl|."""
    c = Case(*shape, agmm.AGMM_FP16, seed=41)
    g = torch.Generator().manual_seed(42)
    c.a[::2] = (8 * c.w[c.labels[::2]].float() / c.w[c.labels[::2]].float().norm(dim=1, keepdim=True) ** 2 * 8).half()
    c.a[::2] += 0.01 * torch.randn(c.a[::2].shape, generator=g).half()
    p = torch.softmax(c.logits(), 1)[torch.arange(c.m), c.labels]
    assert (p[::2] > 0.999).sum() > c.m // 8
    c.gl, c.gz = torch.full((c.m,), gl), torch.full((c.m,), gz)
    c.gl[1], c.gz[1] = largest, 0.0
    run_backward(c, tile)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 10])
def test_small_weights_under_a_loss_scale(scale, tile, shape):
    """Upstream gradients from 1e-8 to 1, zeros among them, times a loss scale
    that makes the smallest rows' parts of dW ordinary numbers of the type.  The
    rows are certain of one column each, so that no large row covers a small
    one's column."""
    c = Case(*shape, agmm.AGMM_FP16, seed=43, spread=40.0)
    c.a, c.w = c.a * 2, c.w / 2          # neither gradient leaves the type's range
    c.gl = scale * torch.pow(10.0, -8 * torch.rand(c.m, generator=torch.Generator().manual_seed(44)))
    c.gl[0], c.gl[1], c.gl[5::8] = scale, scale * 1e-8, 0.0
    c.gz = torch.zeros(c.m)
    c.labels = torch.randperm(c.n, generator=torch.Generator().manual_seed(45)).repeat(3)[:c.m]
    run_backward(c, tile)

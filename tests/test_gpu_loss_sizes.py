"""Copies of rows longer than one sweep of a launch's workgroups (256 MiB)."""
import pytest
import torch

import all_gather_gemm_agmm_amd as agmm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


@pytest.mark.parametrize("shards", [1, 3])
def test_long_copies(shards):
    """A row length that is no multiple of 8: the tiles read a copy of A (350 MB),
    the few-row form reads the rows in place.  Both hold the same sums of 2501
    exact products, each off by at most 2 k u of the terms' sizes, u = 2^-24."""
    m, k, n = 70002, 2501, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    w = (torch.randn((n, k), generator=g, device="cuda") / 50).bfloat16()
    labels = torch.randint(0, n, (m,), generator=g, device="cuda")
    parts = [s.clone() for s in a.split(m // shards)]
    got = []
    for tile in (64, 128):
        with agmm.LossPlan(shards, m // shards, k, n, with_gradient=False, tile=tile) as plan:
            if tile == 128:
                assert plan.workspace_bytes() > m * k * 2
            got.append(plan.forward(parts, w, labels))
            torch.cuda.synchronize()
    bound = 4 * k * 2.0 ** -24 * (a.float().abs() @ w.float().abs().t()).amax(1) + 2.0 ** -20
    for x, y in zip(*got):
        assert ((x - y).abs() <= 2 * bound).all()
    rows = torch.tensor([0, m // 2, m - 1], device="cuda")
    ref = torch.logsumexp(a[rows].double() @ w.double().t(), 1)
    assert ((got[1][1][rows].double() - ref).abs() <= bound[rows]).all()

"""Order of a plan's calls on the GPU: a call captured into a graph between two
eager ones on other streams leaves the second behind the first."""
import pytest
import torch

import all_gather_gemm_agmm_amd as agmm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()


def scaled_calls():
    g = torch.Generator().manual_seed(1)
    plan = agmm.ScaledPlan(1, 16, 8192, 64, splits=8)
    sets = []
    for _ in range(3):
        a, b = torch.randn((16, 8192), generator=g).cuda(), torch.randn((64, 8192), generator=g).cuda()
        c = torch.empty((16, 64), dtype=torch.bfloat16, device="cuda")
        sets.append((lambda s, a=agmm.quantize(a), b=agmm.quantize(b, block_rows=128), c=c: plan.run([a], b, c, stream=s), c))
    return plan, sets


def loss_calls():
    g = torch.Generator().manual_seed(2)
    plan = agmm.LossPlan(1, 200, 128, 1000)
    sets = []
    for _ in range(3):
        a, w = torch.randn((200, 128), generator=g).bfloat16().cuda(), torch.randn((1000, 128), generator=g).bfloat16().cuda()
        lab = torch.randint(0, 1000, (200,), generator=g).cuda()
        lse, gl = torch.logsumexp(a.float() @ w.float().t(), 1), torch.full((200,), 0.005, device="cuda")
        da, dw = torch.empty_like(a), torch.empty_like(w)
        sets.append((lambda s, a=a, w=w, lab=lab, lse=lse, gl=gl, da=da, dw=dw:
                     plan.backward([a], w, lab, lse, gl, dA=da, dW=dw, stream=s), dw))
    return plan, sets


def matmul_calls():
    g = torch.Generator().manual_seed(3)
    plan = agmm.Plan(2, 128, 4096, 256, agmm.AGMM_BF16, True, variant=agmm.AGMM_VARIANT_UNFUSED)
    sets = []
    for _ in range(3):
        a = [torch.randn((128, 4096), generator=g).bfloat16().cuda() for _ in range(2)]
        b = torch.randn((256, 4096), generator=g).bfloat16().cuda()
        c = torch.empty((256, 256), dtype=torch.bfloat16, device="cuda")
        sets.append((lambda s, a=a, b=b, c=c: plan.run(a, b, c, stream=s), c))
    return plan, sets


@pytest.mark.parametrize("calls", [scaled_calls, loss_calls, matmul_calls])
def test_a_captured_call_between_two_eager_ones(calls):
    plan, ((first, out1), (captured, _), (second, out2)) = calls()
    first(None)
    second(None)
    torch.cuda.synchronize()
    want1, want2 = out1.clone(), out2.clone()
    busy = torch.zeros((8192, 8192), dtype=torch.bfloat16, device="cuda")
    torch.mm(busy, busy)
    out1.zero_()
    out2.zero_()
    streams = [torch.cuda.Stream() for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        for _ in range(150):            # about 100 ms ahead of the first call
            torch.mm(busy, busy)
    first(streams[0])
    with torch.cuda.stream(streams[1]):
        graph.capture_begin()
        captured(streams[1])
        graph.capture_end()
    second(streams[2])
    end = streams[2].record_event()
    ahead = streams[0].query()
    done = end.query()
    torch.cuda.synchronize()
    if not ahead:                       # the first call had not run yet: nor may the second have
        assert not done
    assert torch.equal(out1, want1) and torch.equal(out2, want2)
    graph.reset()
    plan.close()

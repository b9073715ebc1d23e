"""The feed-forward block's operators together, as examples/feed_forward_step.py
uses them: the gradients of a whole step against the 64-bit gradient of the
block."""
import importlib.util
import os

import pytest
import torch

import all_gather_gemm_agmm_amd as agmm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    agmm.load_library()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward_step.py")
    spec = importlib.util.spec_from_file_location("feed_forward_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def exact(block, activation):
    """Loss and gradients of the block in 64 bits, on the CPU, from its masters as they are rounded."""
    def leaf(t):
        return t.double().cpu().requires_grad_()

    x = [leaf(s) for s in block.x]
    gain, shift, bias = leaf(block.gain), leaf(block.shift), leaf(block.bias.bfloat16())
    first, last = [leaf(w.bfloat16()) for w in block.first], [leaf(w.bfloat16()) for w in block.last]
    rows = torch.cat(x)
    normed = torch.nn.functional.layer_norm(rows, (block.width,), gain, shift, 1e-5)
    y = rows + bias
    for w, v in zip(first, last):
        p = normed @ w.t()
        g, u = p[:, :block.part], p[:, block.part:]
        a = torch.nn.functional.silu(g) if activation == "silu" else torch.nn.functional.gelu(g)
        y = y + (a * u) @ v.t()
    loss = ((y - block.goal.double().cpu()) ** 2).mean() / 2
    loss.backward()
    return loss.item(), {"x": [t.grad for t in x], "gain": gain.grad, "shift": shift.grad, "bias": bias.grad,
                         "first": [t.grad for t in first], "last": [t.grad for t in last]}


@pytest.mark.parametrize("activation,keep,rows,width,hidden,slices", [
    ("silu", 16, 64, 256, 512, 2), ("silu", 8, 64, 256, 512, 2), ("gelu", 8, 37, 200, 294, 3), ("gelu", 16, 5, 67, 90, 1)])
def test_gradients_of_a_step(example, activation, keep, rows, width, hidden, slices):
    """Relative 2-norms.  A gradient passes at most 10 roundings to bf16 (normed
    rows, p, h, y's parts, dy, dh, d, dA, drows, itself), each off by at most 2^-8
    of a value: 10 * 2^-8 = 0.04.  Pre-activations in 8 bits are off by 2^-4 of
    themselves; d holds the factor and the gate's slope, whose relative change is
    at most that of the gate where it is not near 0: 2 * 2^-4 more."""
    block = example.Block(rows=rows, width=width, hidden=hidden, slices=slices, activation=activation, keep=keep)
    want_loss, want = exact(block, activation)
    loss, got = block.step()
    again, _ = block.step()
    assert torch.equal(loss, again)
    block.close()
    assert abs(loss.item() - want_loss) < 0.02 * want_loss
    most = 0.04 + (0.125 if keep == 8 else 0.0)
    for name, w in want.items():
        for a, b in zip(got[name] if isinstance(w, list) else [got[name]], w if isinstance(w, list) else [w]):
            assert a.shape == b.shape, name
            off = (a.double().cpu() - b).norm() / b.norm()
            assert off <= most, (name, off.item())


def test_example_runs(example):
    block = example.Block()
    for _ in range(3):
        loss, grads = block.step(rate=20.0)
        assert torch.isfinite(loss)
    assert all(torch.isfinite(t).all() for v in grads.values() for t in (v if isinstance(v, list) else [v]))
    block.close()

"""Host-only checks of the block-scaled product and the vocabulary loss (no
GPU): the C entry points reject malformed arguments with the documented
statuses before they touch the device, and the torch helpers do what they say."""
import ctypes
import os

import pytest
import torch

import all_gather_gemm_agmm_amd as agmm

INVALID, UNSUPPORTED = agmm.AGMM_ERR_INVALID_ARG, agmm.AGMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("args,status,fragment", [
    ((0, 4, 8, 8, 0, 128, 0), INVALID, "num_shards"),
    ((65, 4, 8, 8, 0, 128, 0), UNSUPPORTED, "maximum"),
    ((2, 0, 8, 8, 0, 128, 0), INVALID, "sizes"),
    ((2, 4, 8, 8, 2, 128, 0), INVALID, "format"),
    ((2, 4, 8, 8, 0, 64, 0), INVALID, "b_block_rows"),
    ((2, 4, 8, 8, 0, 1, 3), INVALID, "dtype"),
    ((1, 1 << 27, 8, 8, 0, 1, 0), UNSUPPORTED, "too large"),
    ((1, 8, 8, 1 << 27, 0, 1, 0), UNSUPPORTED, "too large"),
    ((1, 1 << 20, 8, 1 << 16, 0, 1, 0), UNSUPPORTED, "too large"),
])
def test_scaled_validate_rejects(args, status, fragment):
    assert agmm.load_library().agmm_scaled_plan_validate(*args) == status
    assert agmm.agmm_last_status() == status and fragment in agmm.agmm_last_error()


def test_scaled_validate_accepts():
    lib = agmm.load_library()
    for args in ((1, 1, 1, 1, 0, 1, 0), (64, 3, 1001, 77, 1, 128, 2), (8, 4096, 8192, 7168, 0, 128, 1),
                 (1, (1 << 27) - 1, 8, 8, 0, 1, 0)):
        assert lib.agmm_scaled_plan_validate(*args) == agmm.AGMM_OK, agmm.agmm_last_error()
        assert agmm.agmm_last_error() == ""


@pytest.mark.parametrize("args,status,fragment", [
    ((0, 4, 8, 8, 0, 0, 8), INVALID, "num_shards"),
    ((2, 4, 0, 8, 0, 0, 8), INVALID, "sizes"),
    ((2, 4, 8, 8, 2, 0, 8), UNSUPPORTED, "bf16 or fp16"),
    ((2, 4, 8, 8, 9, 0, 8), INVALID, "dtype"),
    ((2, 4, 8, 8, 0, -1, 8), INVALID, "vocabulary"),
    ((2, 4, 8, 8, 0, 1, 8), INVALID, "vocabulary"),
    ((2, 4, 8, 8, 0, 0, 1 << 40), INVALID, "vocabulary"),
    ((1, 1 << 27, 8, 8, 0, 0, 8), UNSUPPORTED, "too large"),
])
def test_loss_validate_rejects(args, status, fragment):
    assert agmm.load_library().agmm_loss_plan_validate(*args) == status
    assert agmm.agmm_last_status() == status and fragment in agmm.agmm_last_error()


def test_loss_validate_accepts():
    lib = agmm.load_library()
    for args in ((1, 1, 1, 1, 0, 0, 1), (8, 1024, 4096, 131072, 0, 0, 131072), (3, 37, 1001, 10007, 1, 10007, 40028)):
        assert lib.agmm_loss_plan_validate(*args) == agmm.AGMM_OK, agmm.agmm_last_error()


def test_quantize_rejects():
    """Every refusal of agmm_quantize, on host addresses it never reads."""
    lib = agmm.load_library()
    buf = ctypes.create_string_buffer(4096)
    base = (ctypes.addressof(buf) + 63) // 64 * 64
    good = dict(x=base, dtype=0, rows=4, cols=20, ldx=20, fmt=0, block=1, q=base, ldq=32, s=base, qt=base, ldqt=16, st=base)

    def call(**kw):
        a = dict(good, **kw)
        return lib.agmm_quantize(a["x"], a["dtype"], a["rows"], a["cols"], a["ldx"], a["fmt"], a["block"], a["q"], a["ldq"],
                                 a["s"], a["qt"], a["ldqt"], a["st"], None)

    for kw, status, fragment in [
            (dict(x=None), INVALID, "x is NULL"), (dict(dtype=3), INVALID, "dtype"), (dict(fmt=2), INVALID, "format"),
            (dict(block=2), INVALID, "block_rows"), (dict(rows=0), INVALID, "sizes"), (dict(cols=-1), INVALID, "sizes"),
            (dict(rows=1 << 28), UNSUPPORTED, "too large"), (dict(rows=1 << 20, cols=1 << 17, ldx=1 << 17), UNSUPPORTED, "too large"),
            (dict(ldx=1 << 60), UNSUPPORTED, "row length"), (dict(ldq=1 << 60), UNSUPPORTED, "row length"),
            (dict(ldx=19), INVALID, "ldx"), (dict(q=None, qt=None), INVALID, "both NULL"), (dict(x=base + 1), UNSUPPORTED, "aligned"),
            (dict(ldq=16), INVALID, "ldq"), (dict(ldq=40), UNSUPPORTED, "16-byte"), (dict(q=base + 8), UNSUPPORTED, "16-byte"),
            (dict(s=None), INVALID, "scale"), (dict(ldqt=8), INVALID, "ldqt"), (dict(st=None), INVALID, "scale"),
            (dict(st=base + 2), UNSUPPORTED, "4-byte")]:
        assert call(**kw) == status, (kw, agmm.agmm_last_error())
        assert fragment in agmm.agmm_last_error(), kw


@pytest.mark.parametrize("ms", [1 << 30, 1 << 57, 1 << 58, (1 << 58) + 1, (1 << 63) - 1])
def test_sizes_whose_products_overflow(ms):
    """64 * m_per_shard may pass 2^63: refused, not wrapped."""
    lib = agmm.load_library()
    assert lib.agmm_scaled_plan_validate(64, ms, 8, 8, 0, 1, 0) == UNSUPPORTED
    assert lib.agmm_loss_plan_validate(64, ms, 8, 8, 0, 0, 8) == UNSUPPORTED
    assert lib.agmm_loss_plan_validate(1, 8, ms, 8, 0, 0, 8) == UNSUPPORTED
    assert lib.agmm_loss_plan_validate(1, 8, 8, 8, 0, ms, 1 << 30) == INVALID


def test_null_handles_are_rejected():
    lib = agmm.load_library()
    v = ctypes.c_int64(0)
    assert lib.agmm_scaled_run(None, None, None, None, None, None, None) == INVALID
    assert lib.agmm_scaled_plan_set_int(None, b"tile", 0) == INVALID
    assert lib.agmm_scaled_plan_get_int(None, b"tile", ctypes.byref(v)) == INVALID
    assert lib.agmm_scaled_plan_workspace_bytes(None) == 0
    lib.agmm_scaled_plan_destroy(None)
    assert lib.agmm_loss_forward(None, None, None, None, None, None, None, None) == INVALID
    assert lib.agmm_loss_backward(None, None, None, None, None, None, None, None, None, None) == INVALID
    assert lib.agmm_loss_plan_set_int(None, b"piece", 0) == INVALID
    assert lib.agmm_loss_plan_get_int(None, b"piece", ctypes.byref(v)) == INVALID
    assert lib.agmm_loss_plan_workspace_bytes(None) == 0
    lib.agmm_loss_plan_destroy(None)


def test_dequantize():
    values = torch.zeros((3, 144)).to(torch.float8_e4m3fn)
    values.view(torch.uint8)[:] = torch.randint(0, 120, (3, 144), dtype=torch.uint8)
    scales = torch.tensor([[2.0], [0.5]])
    got = agmm.Scaled(values, scales, 140, 128).dequantize()
    want = values.float()[:, :140].clone()
    want[:, :128] *= 2.0
    want[:, 128:] *= 0.5
    assert torch.equal(got, want)
    rows = torch.tensor([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]])
    got = agmm.Scaled(values, rows, 140, 1).dequantize()
    assert torch.equal(got[1, :128], values.float()[1, :128] * 2) and torch.equal(got[2, 128:], values.float()[2, 128:140] * 6)


def slices(seed=0, parts=3, m=40, n=50):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, parts * n), generator=g, dtype=torch.float64) * 4
    labels = torch.randint(0, parts * n, (m,), generator=g)
    labels[::7] = -100
    lse, target = [], []
    for i in range(parts):
        part = x[:, i * n:(i + 1) * n]
        at = labels - i * n
        here = (at >= 0) & (at < n)
        lse.append(torch.logsumexp(part, 1))
        target.append(torch.where(here, part.gather(1, at.clamp(0, n - 1)[:, None])[:, 0], torch.zeros(m, dtype=torch.float64)))
    want = torch.nn.functional.cross_entropy(x, labels, reduction="none")
    return lse, target, labels, want, torch.logsumexp(x, 1), parts * n


def test_merge_vocab_slices():
    lse, target, labels, want, whole, total = slices()
    loss, merged = agmm.merge_vocab_slices(torch.stack(lse), torch.stack(target), labels, total)
    torch.testing.assert_close(merged, whole, rtol=1e-14, atol=1e-13)
    torch.testing.assert_close(loss, want, rtol=1e-12, atol=1e-12)
    labels[3], labels[4] = total, -1
    loss, _ = agmm.merge_vocab_slices(torch.stack(lse), torch.stack(target), labels, total)
    assert torch.isnan(loss[3:5]).all()
    loss, _ = agmm.merge_vocab_slices(torch.stack(lse), torch.stack(target), labels, total, ignore_index=-1)
    assert loss[4] == 0


def _rank(rank, world, port, out):
    import torch.distributed as dist
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    lse, target, labels, want, _, total = slices(parts=world)
    both = torch.stack([lse[rank], target[rank]])          # what this rank's forward pass returned
    parts = [torch.empty_like(both) for _ in range(world)]
    dist.all_gather(parts, both)
    stacked = torch.stack(parts)
    loss, _ = agmm.merge_vocab_slices(stacked[:, 0], stacked[:, 1], labels, total)
    out.put((rank, (loss - want).abs().max().item()))
    dist.destroy_process_group()


def test_merge_over_two_processes():
    """The slices of two ranks, exchanged by an all-gather (gloo)."""
    import socket
    import torch.multiprocessing as mp
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    out = ctx.Queue()
    procs = [ctx.Process(target=_rank, args=(r, 2, port, out)) for r in range(2)]
    for p in procs:
        p.start()
    got = [out.get(timeout=120) for _ in procs]
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    assert sorted(r for r, _ in got) == [0, 1] and all(e < 1e-12 for _, e in got)

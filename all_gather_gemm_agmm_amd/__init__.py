"""Python binding of libagmm (all-gather fused matmul for MI355X / gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libagmm.so.  There is no CPU or PyTorch fallback; if the library is
missing or fails to load, every entry point raises.

The functions below carry the names of the C ABI in include/agmm.h and take
plain integers (device addresses, sizes, stream handles).  `Plan` is a small
convenience wrapper that takes torch tensors on the GPU and the current torch
stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libagmm.so")

AGMM_BF16, AGMM_FP16, AGMM_FP32 = 0, 1, 2
AGMM_E4M3, AGMM_E5M2 = 0, 1
FORMATS = {"e4m3": AGMM_E4M3, "e5m2": AGMM_E5M2}
SCALE_BLOCK = 128   # elements of k that share one scale
AGMM_OK, AGMM_ERR_INVALID_ARG, AGMM_ERR_UNSUPPORTED, AGMM_ERR_OOM, AGMM_ERR_HIP = 0, 1, 2, 3, 4
(AGMM_VARIANT_AUTO, AGMM_VARIANT_FUSED, AGMM_VARIANT_STAGED, AGMM_VARIANT_UNFUSED,
 AGMM_VARIANT_SKINNY) = 0, 1, 2, 3, 4
VARIANTS = {"auto": 0, "fused": 1, "staged": 2, "unfused": 3, "skinny": 4}
VARIANT_NAMES = {v: k for k, v in VARIANTS.items()}

# Values of the plan key "tile" (include/agmm.h lists what each one is).
TILES = {"256x256": 0, "128x128": 1, "256x128": 2, "128x64": 3, "128x64_s8": 4,
         "256x256_ring": 5, "128x128_ring": 6, "128x64_ring": 7, "256x256_m16": 8,
         "128x128_m16": 9, "skinny": 10, "256x224_m16": 11}
NUM_TILES = len(TILES)
TILE_SKINNY = TILES["skinny"]
TILES_NEED_BT = (TILES["128x64"], TILES["128x64_s8"], TILES["128x64_ring"], TILE_SKINNY,
                 TILES["256x224_m16"])

# (name, restype, argtypes) of every symbol include/agmm.h declares.
_vp, _i64, _ci, _cc = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_char_p
EXPORTS = [
    ("agmm_plan_validate", _ci, [_ci, _i64, _i64, _i64, _ci, _ci]),
    ("agmm_plan_create", _vp, [_ci, _i64, _i64, _i64, _ci, _ci]),
    ("agmm_run", _ci, [_vp, ctypes.POINTER(_vp), _vp, _vp, _vp]),
    ("agmm_gather", _ci, [_vp, ctypes.POINTER(_vp), _vp, _vp]),
    ("agmm_run_gathered", _ci, [_vp, _vp, _vp, _vp, _vp]),
    ("agmm_run_gather_out", _ci, [_vp, ctypes.POINTER(_vp), _vp, _vp, _vp, _vp]),
    ("agmm_plan_autotune", _ci, [_vp, ctypes.POINTER(_vp), _vp, _vp, _vp, _ci,
                                 ctypes.POINTER(ctypes.c_double)]),
    ("agmm_plan_set_int", _ci, [_vp, _cc, _i64]),
    ("agmm_plan_get_int", _ci, [_vp, _cc, ctypes.POINTER(_i64)]),
    ("agmm_plan_workspace_bytes", ctypes.c_size_t, [_vp]),
    ("agmm_plan_slot_ptr", _vp, [_vp, _ci]),
    ("agmm_plan_tile_order", _ci, [_vp, _ci, ctypes.POINTER(ctypes.c_int32), _ci]),
    ("agmm_plan_timing_begin", _ci, [_vp]),
    ("agmm_plan_timing_read", _ci, [_vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64)]),
    ("agmm_plan_timing_end", _ci, [_vp]),
    ("agmm_plan_destroy", None, [_vp]),
    ("agmm_run_noalloc", _ci, [_ci, _i64, _i64, _i64, _ci, _ci, ctypes.POINTER(_vp), _vp, _vp, _vp]),
    ("agmm_quantize", _ci, [_vp, _ci, _i64, _i64, _i64, _ci, _ci, _vp, _i64, _vp, _vp, _i64, _vp, _vp]),
    ("agmm_scaled_plan_validate", _ci, [_ci, _i64, _i64, _i64, _ci, _ci, _ci]),
    ("agmm_scaled_plan_create", _vp, [_ci, _i64, _i64, _i64, _ci, _ci, _ci]),
    ("agmm_scaled_run", _ci, [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp, _vp, _vp, _vp]),
    ("agmm_scaled_plan_set_int", _ci, [_vp, _cc, _i64]),
    ("agmm_scaled_plan_get_int", _ci, [_vp, _cc, ctypes.POINTER(_i64)]),
    ("agmm_scaled_plan_workspace_bytes", ctypes.c_size_t, [_vp]),
    ("agmm_scaled_plan_destroy", None, [_vp]),
    ("agmm_loss_plan_validate", _ci, [_ci, _i64, _i64, _i64, _ci, _i64, _i64]),
    ("agmm_loss_plan_create", _vp, [_ci, _i64, _i64, _i64, _ci, _i64, _i64, _ci]),
    ("agmm_loss_forward", _ci, [_vp, ctypes.POINTER(_vp), _vp, _vp, _vp, _vp, _vp, _vp]),
    ("agmm_loss_backward", _ci, [_vp, ctypes.POINTER(_vp), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    ("agmm_loss_plan_set_int", _ci, [_vp, _cc, _i64]),
    ("agmm_loss_plan_get_int", _ci, [_vp, _cc, ctypes.POINTER(_i64)]),
    ("agmm_loss_plan_workspace_bytes", ctypes.c_size_t, [_vp]),
    ("agmm_loss_plan_destroy", None, [_vp]),
    ("agmm_last_status", _ci, []),
    ("agmm_last_error", _cc, []),
    ("agmm_version", _cc, []),
]

_lib = None


class AgmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"agmm error {status}: {message}")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libagmm.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m all_gather_gemm_agmm_amd._build`; "
            "the all-gather matmul has no CPU fallback")
    lib = ctypes.CDLL(path)
    for name, res, args in EXPORTS:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(status: int) -> int:
    if status != AGMM_OK:
        lib = load_library()
        raise AgmmError(status, lib.agmm_last_error().decode())
    return status


def _ptr_table(ptrs: Sequence[int]):
    return (ctypes.c_void_p * len(ptrs))(*[ctypes.c_void_p(int(p)) for p in ptrs])


# ---------------------------------------------------------------- raw C ABI
def agmm_plan_validate(num_shards, m_per_shard, k, n_local, dtype, rhs_transpose) -> int:
    return load_library().agmm_plan_validate(num_shards, m_per_shard, k, n_local, dtype,
                                             int(bool(rhs_transpose)))


def agmm_plan_create(num_shards, m_per_shard, k, n_local, dtype, rhs_transpose) -> int:
    lib = load_library()
    h = lib.agmm_plan_create(num_shards, m_per_shard, k, n_local, dtype, int(bool(rhs_transpose)))
    if not h:
        raise AgmmError(lib.agmm_last_status(), lib.agmm_last_error().decode())
    return h


def agmm_run(plan, shard_ptrs: Sequence[int], B: int, C: int, stream: int) -> int:
    return _check(load_library().agmm_run(plan, _ptr_table(shard_ptrs), B, C, stream))


def agmm_plan_autotune(plan, shard_ptrs: Sequence[int], B: int, C: int, stream: int,
                       iters: int = 3) -> float:
    best = ctypes.c_double(0.0)
    _check(load_library().agmm_plan_autotune(plan, _ptr_table(shard_ptrs), B, C, stream, iters,
                                             ctypes.byref(best)))
    return best.value


def agmm_gather(plan, shard_ptrs: Sequence[int], gathered: int, stream: int) -> int:
    return _check(load_library().agmm_gather(plan, _ptr_table(shard_ptrs), gathered, stream))


def agmm_run_gathered(plan, gathered: int, B: int, C: int, stream: int) -> int:
    return _check(load_library().agmm_run_gathered(plan, gathered, B, C, stream))


def agmm_run_gather_out(plan, shard_ptrs: Sequence[int], B: int, C: int, gathered: int,
                        stream: int) -> int:
    return _check(load_library().agmm_run_gather_out(plan, _ptr_table(shard_ptrs), B, C, gathered,
                                                     stream))


def agmm_plan_set_int(plan, key: str, value: int) -> int:
    return _check(load_library().agmm_plan_set_int(plan, key.encode(), int(value)))


def agmm_plan_get_int(plan, key: str) -> int:
    v = ctypes.c_int64(0)
    _check(load_library().agmm_plan_get_int(plan, key.encode(), ctypes.byref(v)))
    return int(v.value)


def agmm_plan_workspace_bytes(plan) -> int:
    return int(load_library().agmm_plan_workspace_bytes(plan))


def agmm_plan_slot_ptr(plan, slot: int) -> int:
    return int(load_library().agmm_plan_slot_ptr(plan, slot) or 0)


def agmm_plan_tile_order(plan, chunk: int = 0):
    # Chunk 0 is never smaller than a later (clamped) chunk.
    cap = max(agmm_plan_get_int(plan, "num_row_blocks"), 1)
    buf = (ctypes.c_int32 * cap)()
    got = load_library().agmm_plan_tile_order(plan, chunk, buf, cap)
    if got < 0:
        raise AgmmError(agmm_last_status(), agmm_last_error())
    return [int(buf[i]) for i in range(got)]


def agmm_plan_timing_begin(plan) -> int:
    return _check(load_library().agmm_plan_timing_begin(plan))


def agmm_plan_timing_read(plan):
    ms, n = ctypes.c_double(0.0), ctypes.c_int64(0)
    _check(load_library().agmm_plan_timing_read(plan, ctypes.byref(ms), ctypes.byref(n)))
    return float(ms.value), int(n.value)


def agmm_plan_timing_end(plan) -> int:
    return _check(load_library().agmm_plan_timing_end(plan))


def agmm_plan_destroy(plan) -> None:
    if plan:
        load_library().agmm_plan_destroy(plan)


NOALLOC_SCRATCH_BYTES = 32 << 20


def agmm_run_noalloc(num_shards, m_per_shard, k, n_local, dtype, rhs_transpose,
                     shard_ptrs: Sequence[int], B: int, C: int, stream: int) -> int:
    return _check(load_library().agmm_run_noalloc(num_shards, m_per_shard, k, n_local, dtype,
                                                  int(bool(rhs_transpose)), _ptr_table(shard_ptrs),
                                                  B, C, stream))


def run_noalloc(shards, B, C, rhs_transpose: bool, stream=None):
    """agmm_run_noalloc on torch tensors: dense row-major shards [m_s, k], B
    [k, n] (or [n, k] with rhs_transpose) and a caller-provided C [m, n]."""
    import torch
    if len(shards) == 0:
        raise ValueError("agmm_run_noalloc needs at least one shard")
    tensors = list(shards) + [B, C]
    if not all(isinstance(t, torch.Tensor) for t in tensors):
        raise TypeError("shards, B and C must be torch tensors")
    dtype = {torch.bfloat16: AGMM_BF16, torch.float16: AGMM_FP16,
             torch.float32: AGMM_FP32}.get(B.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {B.dtype}")
    device = B.device
    if device.type != "cuda":
        raise ValueError("B must be on the GPU")
    for t in tensors:
        if t.device != device:
            raise ValueError(f"every tensor must be on {device} (found one on {t.device})")
        if t.dtype != B.dtype:
            raise TypeError(f"every tensor must have dtype {B.dtype} (found {t.dtype})")
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError("agmm_run_noalloc takes dense row-major 2-D tensors")
    m_s, k = shards[0].shape
    if any(tuple(t.shape) != (m_s, k) for t in shards):
        raise ValueError(f"every shard must have shape {(m_s, k)}")
    n = B.shape[0] if rhs_transpose else B.shape[1]
    if (B.shape[1] if rhs_transpose else B.shape[0]) != k:
        raise ValueError(f"B has shape {tuple(B.shape)}, which does not match k = {k}")
    if tuple(C.shape) != (len(shards) * m_s, n):
        raise ValueError(f"C has shape {tuple(C.shape)}, expected {(len(shards) * m_s, n)}")
    agmm_run_noalloc(len(shards), m_s, k, n, dtype, rhs_transpose, [s.data_ptr() for s in shards],
                     B.data_ptr(), C.data_ptr(), _stream_handle(stream, device.index))
    return C


def agmm_quantize(x, dtype, rows, cols, ldx, fmt, block_rows, q, ldq, scale, qt, ldqt, scale_t, stream) -> int:
    return _check(load_library().agmm_quantize(x, dtype, rows, cols, ldx, fmt, block_rows, q, ldq, scale, qt, ldqt,
                                               scale_t, stream))


def agmm_last_status() -> int:
    return int(load_library().agmm_last_status())


def agmm_last_error() -> str:
    return load_library().agmm_last_error().decode()


def agmm_version() -> str:
    return load_library().agmm_version().decode()


# ------------------------------------------------------- torch convenience
def _torch_dtype(dtype: int):
    import torch
    return {AGMM_BF16: torch.bfloat16, AGMM_FP16: torch.float16, AGMM_FP32: torch.float32}[dtype]


def _stream_handle(stream, device_index=None) -> int:
    """The raw hipStream_t of `stream`, or of the current stream of the given
    (else the current) device."""
    import torch
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:   # the pointer alone, without a Stream object
            return int(raw(torch.cuda.current_device() if device_index is None else device_index))
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


class Plan:
    """A plan bound to torch tensors.  All checks here are host-side shape,
    dtype and device checks; the computation is the library's."""

    def __init__(self, num_shards: int, m_per_shard: int, k: int, n_local: int, dtype: int,
                 rhs_transpose: bool, **settings):
        self.num_shards, self.m_per_shard, self.k, self.n_local = num_shards, m_per_shard, k, n_local
        self.dtype, self.rhs_transpose = dtype, bool(rhs_transpose)
        self.handle = agmm_plan_create(num_shards, m_per_shard, k, n_local, dtype, rhs_transpose)
        import torch
        self.device = torch.cuda.current_device()   # the device the library created the plan on
        self._tdt = _torch_dtype(dtype)
        self._ptrs = (ctypes.c_void_p * num_shards)()   # shard pointer table, reused per call
        self._read_strides()
        for key, val in settings.items():
            if val is not None:
                self.set(key, VARIANTS[val] if key == "variant" and isinstance(val, str) else val)

    def _read_strides(self):
        # row strides in use, kept here so that per-call checks need no
        # call into the library
        self._ld = {k: agmm_plan_get_int(self.handle, k) for k in ("lda", "ldb", "ldc")}

    @property
    def m(self) -> int:
        return self.num_shards * self.m_per_shard

    def set(self, key: str, value: int) -> None:
        try:
            agmm_plan_set_int(self.handle, key, value)
        finally:
            self._read_strides()

    def get(self, key: str) -> int:
        return agmm_plan_get_int(self.handle, key)

    def _check_tensor(self, t, shape, name, ld_key=None, index=None):
        """Shape / dtype / device checks.  With `ld_key` ("lda", "ldb", "ldc")
        the tensor may be a row-strided view whose row stride is the plan's
        setting for that key; otherwise it must be dense row-major."""
        ld = self._ld[ld_key] if ld_key else shape[1]
        try:   # the common case in a few attribute reads
            st = t.stride()
            if (t.dtype is self._tdt and t.is_cuda and t.get_device() == self.device and
                    t.shape == shape and st[1] == 1 and (shape[0] <= 1 or st[0] == ld)):
                return
        except (AttributeError, TypeError, IndexError):
            pass
        if index is not None:
            name = f"{name}[{index}]"
        import torch
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on the GPU")
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}; the plan was created on cuda:{self.device}")
        if t.dtype != _torch_dtype(self.dtype):
            raise TypeError(f"{name} has dtype {t.dtype}, plan expects {_torch_dtype(self.dtype)}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.stride(1) != 1 or (shape[0] > 1 and t.stride(0) != ld):
            raise ValueError(f"{name} must be row-major with rows {ld} elements apart "
                             f"(stride {tuple(t.stride())})")

    def _new_c(self, device):
        """A C buffer with the plan's row stride (a view when ldc > n_local)."""
        import torch
        ldc = self._ld["ldc"]
        return torch.empty((self.m, ldc), dtype=_torch_dtype(self.dtype), device=device)[:, :self.n_local]

    def b_shape(self):
        return (self.n_local, self.k) if self.rhs_transpose else (self.k, self.n_local)

    def run(self, shards, B, C=None, stream=None):
        if len(shards) != self.num_shards:
            raise ValueError(f"expected {self.num_shards} shards, got {len(shards)}")
        shape, ptrs = (self.m_per_shard, self.k), self._ptrs
        for r, s in enumerate(shards):
            self._check_tensor(s, shape, "shards", "lda", r)
            ptrs[r] = s.data_ptr()
        self._check_tensor(B, self.b_shape(), "B", "ldb")
        if C is None:
            C = self._new_c(B.device)
        self._check_tensor(C, (self.m, self.n_local), "C", "ldc")
        _check(load_library().agmm_run(self.handle, ptrs, B.data_ptr(), C.data_ptr(),
                                       _stream_handle(stream, B.device.index)))
        return C

    def run_gather_out(self, shards, B, C=None, gathered=None, stream=None):
        """C = concat(shards) @ B and the gathered operand; returns (C, gathered)."""
        import torch
        if len(shards) != self.num_shards:
            raise ValueError(f"expected {self.num_shards} shards, got {len(shards)}")
        for r, s in enumerate(shards):
            self._check_tensor(s, (self.m_per_shard, self.k), "shards", "lda", r)
        self._check_tensor(B, self.b_shape(), "B", "ldb")
        if C is None:
            C = self._new_c(B.device)
        if gathered is None:
            gathered = torch.empty((self.m, self.k), dtype=_torch_dtype(self.dtype), device=B.device)
        self._check_tensor(C, (self.m, self.n_local), "C", "ldc")
        self._check_tensor(gathered, (self.m, self.k), "gathered")
        agmm_run_gather_out(self.handle, [s.data_ptr() for s in shards], B.data_ptr(), C.data_ptr(),
                            gathered.data_ptr(), _stream_handle(stream, B.device.index))
        return C, gathered

    def autotune(self, shards, B, C=None, iters=3, stream=None) -> float:
        """Time candidate settings on these buffers, keep the fastest; returns
        its mean ms per run (C is overwritten with the product)."""
        if len(shards) != self.num_shards:
            raise ValueError(f"expected {self.num_shards} shards, got {len(shards)}")
        for r, s in enumerate(shards):
            self._check_tensor(s, (self.m_per_shard, self.k), "shards", "lda", r)
        self._check_tensor(B, self.b_shape(), "B", "ldb")
        if C is None:
            C = self._new_c(B.device)
        self._check_tensor(C, (self.m, self.n_local), "C", "ldc")
        return agmm_plan_autotune(self.handle, [s.data_ptr() for s in shards], B.data_ptr(),
                                  C.data_ptr(), _stream_handle(stream, B.device.index), iters)

    def gather(self, shards, out=None, stream=None):
        import torch
        if len(shards) != self.num_shards:
            raise ValueError(f"expected {self.num_shards} shards, got {len(shards)}")
        for r, s in enumerate(shards):
            self._check_tensor(s, (self.m_per_shard, self.k), "shards", "lda", r)
        if out is None:
            out = torch.empty((self.m, self.k), dtype=_torch_dtype(self.dtype), device=shards[0].device)
        self._check_tensor(out, (self.m, self.k), "gathered")
        agmm_gather(self.handle, [s.data_ptr() for s in shards], out.data_ptr(),
                    _stream_handle(stream, out.device.index))
        return out

    def run_gathered(self, gathered, B, C=None, stream=None):
        import torch
        self._check_tensor(gathered, (self.m, self.k), "gathered")
        self._check_tensor(B, self.b_shape(), "B", "ldb")
        if C is None:
            C = self._new_c(B.device)
        self._check_tensor(C, (self.m, self.n_local), "C", "ldc")
        agmm_run_gathered(self.handle, gathered.data_ptr(), B.data_ptr(), C.data_ptr(),
                          _stream_handle(stream, B.device.index))
        return C

    def tile_order(self, chunk: int = 0):
        return agmm_plan_tile_order(self.handle, chunk)

    def workspace_bytes(self) -> int:
        return agmm_plan_workspace_bytes(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            agmm_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


# ------------------------------------------------ block-scaled 8-bit operands
class Scaled:
    """A block-scaled 8-bit matrix [rows, k]: `values` (float8, [rows, k
    rounded up to 16], zeros past k), `scales` (fp32, [ceil(k / 128),
    ceil(rows / block_rows)]), the true row length `k` and `block_rows` (1 or
    128).  Element (r, c) stands for values[r, c] * scales[c // 128, r //
    block_rows]."""

    __slots__ = ("values", "scales", "k", "block_rows")

    def __init__(self, values, scales, k: int, block_rows: int = 1):
        self.values, self.scales, self.k, self.block_rows = values, scales, int(k), int(block_rows)

    @property
    def rows(self) -> int:
        return self.values.shape[0]

    def dequantize(self):
        """The fp32 matrix [rows, k] this one stands for (torch operations; for
        checks, not for speed)."""
        s = self.scales.t().repeat_interleave(SCALE_BLOCK, dim=1)[:, :self.k]
        if self.block_rows > 1:
            s = s.repeat_interleave(self.block_rows, dim=0)[:self.rows]
        return self.values[:, :self.k].float() * s


_HERE = contextlib.nullcontext()


def _device_and_stream(index: int, stream):
    """Context in which outputs are allocated and kernels launched: GPU
    `index`, and the caller's torch stream if one was passed (so that the
    allocator hands out memory in that stream's order)."""
    import torch
    if isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)   # sets the stream's device too
    if index != torch.cuda.current_device():
        return torch.cuda.device(index)
    return _HERE


_QUANT_TYPES: dict = {}   # torch's types and this library's codes, filled on first use


def _format(fmt) -> int:
    code = FORMATS.get(fmt, fmt)
    if code != AGMM_E4M3 and code != AGMM_E5M2:
        raise ValueError(f"unknown 8-bit format {fmt!r} (one of {sorted(FORMATS)})")
    return code


def _format_dtype(fmt: int):
    import torch
    return {AGMM_E4M3: torch.float8_e4m3fn, AGMM_E5M2: torch.float8_e5m2}[fmt]


def quantize(x, fmt="e4m3", block_rows: int = 1, out: str = "rows", stream=None):
    """Block-scaled 8-bit copies of x [rows, cols] (bf16, fp16 or fp32, unit
    column stride): agmm_quantize.  `out` is "rows" (x, for a product that
    contracts its columns), "cols" (x transposed, for one that contracts its
    rows) or "both"; returns a Scaled, or the pair for "both"."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if not _QUANT_TYPES:
        _QUANT_TYPES.update({torch.bfloat16: AGMM_BF16, torch.float16: AGMM_FP16, torch.float32: AGMM_FP32,
                             AGMM_E4M3: torch.float8_e4m3fn, AGMM_E5M2: torch.float8_e5m2, None: torch.float32})
    if out != "rows" and out != "cols" and out != "both":
        raise ValueError(f"out must be 'rows', 'cols' or 'both' (got {out!r})")
    code = _QUANT_TYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype}")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be on the GPU")
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    (rows, cols), (ldx, unit) = x.shape, x.stride()
    if unit != 1 and cols > 1:
        raise ValueError("x must be a row-major matrix (unit column stride)")
    fmt = _format(fmt)
    if block_rows != 1 and block_rows != SCALE_BLOCK:
        raise ValueError(f"block_rows must be 1 or {SCALE_BLOCK}")
    f8, f32, empty = _QUANT_TYPES[fmt], _QUANT_TYPES[None], torch.empty
    q = s = qt = st = None
    q_ptr = s_ptr = qt_ptr = st_ptr = None
    ldq, ldqt = (cols + 15) // 16 * 16, (rows + 15) // 16 * 16
    with _device_and_stream(device.index, stream):
        if out != "cols":
            q = empty((rows, ldq), dtype=f8, device=device)
            s = empty(((cols + 127) // 128, -(-rows // block_rows)), dtype=f32, device=device)
            q_ptr, s_ptr = q.data_ptr(), s.data_ptr()
        if out != "rows":
            qt = empty((cols, ldqt), dtype=f8, device=device)
            st = empty(((rows + 127) // 128, -(-cols // block_rows)), dtype=f32, device=device)
            qt_ptr, st_ptr = qt.data_ptr(), st.data_ptr()
        _check(load_library().agmm_quantize(x.data_ptr(), code, rows, cols, ldx if rows > 1 else max(cols, 1), fmt, block_rows,
                                            q_ptr, ldq, s_ptr, qt_ptr, ldqt, st_ptr, _stream_handle(stream, device.index)))
    if out == "rows":
        return Scaled(q, s, cols, block_rows)
    if out == "cols":
        return Scaled(qt, st, rows, block_rows)
    return Scaled(q, s, cols, block_rows), Scaled(qt, st, rows, block_rows)


class _OpPlan:
    """What the plans of the operators share: their handle, its settings and
    its end.  `_prefix` is that of their C functions; `_expect` says what the
    tensors of a call look like."""

    def _make(self, *args):
        import torch
        lib = load_library()
        self.handle = None
        self.device = torch.cuda.current_device()
        self.handle = getattr(lib, self._prefix + "_create")(*args)
        if not self.handle:
            raise AgmmError(lib.agmm_last_status(), lib.agmm_last_error().decode())

    def set(self, key: str, value: int) -> None:
        _check(getattr(load_library(), self._prefix + "_set_int")(self.handle, key.encode(), int(value)))
        self._expect()

    def get(self, key: str) -> int:
        v = ctypes.c_int64(0)
        _check(getattr(load_library(), self._prefix + "_get_int")(self.handle, key.encode(), ctypes.byref(v)))
        return int(v.value)

    def workspace_bytes(self) -> int:
        return int(getattr(load_library(), self._prefix + "_workspace_bytes")(self.handle))

    def _like(self, shape, dtype, ld=None):
        """What `_on` expects of a tensor, for its one-comparison case."""
        import torch
        stride = (1,) if len(shape) == 1 else (shape[1] if ld is None else ld, 1)
        return (dtype, torch.device("cuda", self.device), torch.Size(shape), stride)

    def _on(self, t, like, name):
        """The address of a tensor of this dtype, device and shape, dense or with
        the row stride of `like`."""
        dtype, device, shape, stride = like
        try:
            if t.dtype == dtype and t.device == device and t.shape == shape:
                got = t.stride()
                # a dimension of one element may have any stride
                if (got == stride or (shape[0] <= 1 or got[0] == stride[0]) and
                        (len(shape) == 1 or shape[1] <= 1 or got[1] == stride[1])):
                    return t.data_ptr()
        except AttributeError:
            pass
        import torch
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on the GPU")
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}; the plan was created on cuda:{self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, plan expects {dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{name} must be row-major with rows {stride[0]} elements apart (stride {tuple(t.stride())})")

    def _new(self, like):
        """A new tensor as `like` describes it."""
        import torch
        dtype, device, shape, stride = like
        if len(shape) == 1 or stride[0] == shape[1]:
            return torch.empty(shape, dtype=dtype, device=device)
        return torch.empty((shape[0], stride[0]), dtype=dtype, device=device)[:, :shape[1]]

    @property
    def m(self) -> int:
        return self.num_shards * self.m_per_shard

    def close(self) -> None:
        if getattr(self, "handle", None):
            getattr(load_library(), self._prefix + "_destroy")(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class ScaledPlan(_OpPlan):
    """C = concat_r(shards[r]) @ B^T for block-scaled 8-bit operands
    (agmm_scaled_run): shards are Scaled [m_per_shard, k] with block_rows 1 in
    `a_format`, B a Scaled [n_local, k] in e4m3 with `b_block_rows`, C of
    `c_dtype` (AGMM_BF16, AGMM_FP16 or AGMM_FP32).  Long products to 16 bits use
    the 8-bit matrix instruction, whose sums cut small terms beside large ones;
    `exact_sums=1` asks for fp32 sums instead, at about half the rate."""

    _prefix = "agmm_scaled_plan"

    def __init__(self, num_shards: int, m_per_shard: int, k: int, n_local: int, a_format="e4m3",
                 b_block_rows: int = SCALE_BLOCK, c_dtype: int = AGMM_BF16, **settings):
        a_format = _format(a_format)
        self._make(num_shards, m_per_shard, k, n_local, a_format, b_block_rows, c_dtype)
        self.num_shards, self.m_per_shard, self.k, self.n_local = num_shards, m_per_shard, k, n_local
        self.a_format, self.b_block_rows, self.c_dtype = a_format, b_block_rows, c_dtype
        self._table = ctypes.c_void_p * num_shards   # a new one per call: calls of several threads may overlap
        self._run = load_library().agmm_scaled_run
        self._expect()
        for key, val in settings.items():
            if val is not None:
                self.set(key, val)

    def _expect(self):
        import torch
        k16, kb, f32 = -(-self.k // 16) * 16, -(-self.k // SCALE_BLOCK), torch.float32
        self._la = self._like((self.m_per_shard, k16), _format_dtype(self.a_format), self.get("lda"))
        self._ls = self._like((kb, self.m_per_shard), f32)
        self._lb = self._like((self.n_local, k16), torch.float8_e4m3fn, self.get("ldb"))
        self._lbs = self._like((kb, -(-self.n_local // self.b_block_rows)), f32)
        self._lc = self._like((self.m, self.n_local), _torch_dtype(self.c_dtype), self.get("ldc"))

    def _operand(self, x, block_rows, name):
        if not isinstance(x, Scaled):
            raise TypeError(f"{name} must be a Scaled")
        if x.k != self.k or x.block_rows != block_rows:
            raise ValueError(f"{name} has k {x.k} and block_rows {x.block_rows}, expected {self.k} and {block_rows}")

    def run(self, shards, B, C=None, stream=None):
        if len(shards) != self.num_shards:
            raise ValueError(f"expected {self.num_shards} shards, got {len(shards)}")
        k, la, ls, on, pa, ps = self.k, self._la, self._ls, self._on, self._table(), self._table()
        r = 0
        for x in shards:
            if x.__class__ is not Scaled or x.k != k or x.block_rows != 1:
                self._operand(x, 1, "shards")
            v, s = x.values, x.scales
            # the common case in one comparison each
            pa[r] = v.data_ptr() if (v.dtype, v.device, v.shape, v.stride()) == la else on(v, la, "shards.values")
            ps[r] = s.data_ptr() if (s.dtype, s.device, s.shape, s.stride()) == ls else on(s, ls, "shards.scales")
            r += 1
        self._operand(B, self.b_block_rows, "B")
        b, bs = on(B.values, self._lb, "B.values"), on(B.scales, self._lbs, "B.scales")
        with _device_and_stream(self.device, stream):
            if C is None:
                C = self._new(self._lc)
            _check(self._run(self.handle, pa, ps, b, bs, on(C, self._lc, "C"), _stream_handle(stream, self.device)))
        return C


class LossPlan(_OpPlan):
    """Softmax cross entropy of the vocabulary projection concat_r(shards[r])
    @ W^T without its logits, and its gradient (agmm_loss_forward,
    agmm_loss_backward).  W [n_local, k] holds columns [vocab_start,
    vocab_start + n_local) of a vocabulary of `vocab_size` (default: all of
    it); `merge_vocab_slices` joins the results of several devices."""

    _prefix = "agmm_loss_plan"

    def __init__(self, num_shards: int, m_per_shard: int, k: int, n_local: int, dtype: int = AGMM_BF16,
                 vocab_start: int = 0, vocab_size: Optional[int] = None, with_gradient: bool = True, **settings):
        self._make(num_shards, m_per_shard, k, n_local, dtype, vocab_start,
                   vocab_start + n_local if vocab_size is None else vocab_size, int(bool(with_gradient)))
        self.num_shards, self.m_per_shard, self.k, self.n_local, self.dtype = num_shards, m_per_shard, k, n_local, dtype
        self._table = ctypes.c_void_p * num_shards   # a new one per call: calls of several threads may overlap
        self._fwd, self._bwd = load_library().agmm_loss_forward, load_library().agmm_loss_backward
        self._expect()
        for key, val in settings.items():
            if val is not None:
                self.set(key, val)

    def _expect(self):
        import torch
        t = _torch_dtype(self.dtype)
        self._la = self._like((self.m_per_shard, self.k), t, self.get("lda"))
        self._lw = self._like((self.n_local, self.k), t, self.get("ldw"))
        self._lda = self._like((self.m, self.k), t, self.get("ldda"))
        self._ldw = self._like((self.n_local, self.k), t, self.get("lddw"))
        self._llab = self._like((self.m,), torch.int64)
        self._lrow = self._like((self.m,), torch.float32)

    def _operands(self, shards, W, labels):
        if len(shards) != self.num_shards:
            raise ValueError(f"expected {self.num_shards} shards, got {len(shards)}")
        la, on, pa = self._la, self._on, self._table()
        for r, s in enumerate(shards):
            pa[r] = on(s, la, "shards")
        return pa, on(W, self._lw, "W"), on(labels, self._llab, "labels")

    def forward(self, shards, W, labels, stream=None):
        """(loss, lse, target), fp32 [m] each."""
        a, w, lab = self._operands(shards, W, labels)
        with _device_and_stream(self.device, stream):
            new = self._new
            loss, lse, target = new(self._lrow), new(self._lrow), new(self._lrow)
            _check(self._fwd(self.handle, a, w, lab, loss.data_ptr(), lse.data_ptr(), target.data_ptr(),
                             _stream_handle(stream, self.device)))
        return loss, lse, target

    def backward(self, shards, W, labels, lse, grad_loss, grad_lse=None, dA=None, dW=None, need_dA: bool = True,
                 need_dW: bool = True, stream=None):
        """(dA [m, k], dW [n_local, k]) for upstream gradients of loss and,
        optionally, lse; None in the place of one that is not needed."""
        a, w, lab = self._operands(shards, W, labels)
        on = self._on
        ls, gl = on(lse, self._lrow, "lse"), on(grad_loss, self._lrow, "grad_loss")
        gz = None if grad_lse is None else on(grad_lse, self._lrow, "grad_lse")
        with _device_and_stream(self.device, stream):
            if dA is None and need_dA:
                dA = self._new(self._lda)
            if dW is None and need_dW:
                dW = self._new(self._ldw)
            _check(self._bwd(self.handle, a, w, lab, ls, gl, gz, None if dA is None else on(dA, self._lda, "dA"),
                             None if dW is None else on(dW, self._ldw, "dW"), _stream_handle(stream, self.device)))
        return dA, dW


def merge_vocab_slices(lse, target, labels, vocab_size: int, ignore_index: int = -100):
    """(loss, lse) over a whole vocabulary from the devices' `lse` and
    `target`, [slices, m] each (torch operations on [slices, m] values): the
    log-sum-exp of the slices' and the sum of their targets.  As in LossPlan,
    ignored rows have loss 0, labels outside the vocabulary NaN."""
    import torch
    whole = torch.logsumexp(lse, dim=0)
    loss = whole - target.sum(dim=0)
    bad = (labels < 0) | (labels >= vocab_size)
    loss = torch.where(bad, torch.full_like(loss, float("nan")), loss)
    return torch.where(labels == ignore_index, torch.zeros_like(loss), loss), whole


# ------------------------------------------------ one call, cached plans
_PLAN_CACHE: dict = {}
_PLAN_CACHE_LOCK = None


def all_gather_matmul(shards, B, rhs_transpose: bool = False, C=None, stream=None):
    """C = concat_r(shards[r]) @ B, or @ B^T with rhs_transpose (B stored
    [n_local, k]): the tpu-inference page's `all_gather_matmul` on one GPU,
    with the shards as separate tensors.  The first call for a problem
    shape, dtype and device creates a plan with the automatic settings and
    keeps it (its workspace stays allocated until clear_plan_cache()); later
    calls reuse it.  Returns C [num_shards * m_per_shard, n_local]."""
    import threading
    global _PLAN_CACHE_LOCK
    if _PLAN_CACHE_LOCK is None:
        _PLAN_CACHE_LOCK = threading.Lock()
    if len(shards) == 0:
        raise ValueError("all_gather_matmul needs at least one shard")
    m_s, k = shards[0].shape
    n = B.shape[0] if rhs_transpose else B.shape[1]
    dtype = {"torch.bfloat16": AGMM_BF16, "torch.float16": AGMM_FP16,
             "torch.float32": AGMM_FP32}.get(str(B.dtype))
    if dtype is None:
        raise ValueError(f"unsupported dtype {B.dtype}")
    if B.device.type != "cuda":
        raise ValueError("B must be on the GPU")
    import torch
    key = (len(shards), int(m_s), int(k), int(n), dtype, bool(rhs_transpose), B.device.index)
    with _PLAN_CACHE_LOCK:
        plan = _PLAN_CACHE.get(key)
        if plan is None:
            with torch.cuda.device(B.device):
                plan = Plan(len(shards), int(m_s), int(k), int(n), dtype, bool(rhs_transpose))
            _PLAN_CACHE[key] = plan
    return plan.run(shards, B, C, stream=stream)


def clear_plan_cache() -> None:
    """Destroy the plans all_gather_matmul keeps (after the work queued on
    them has finished: destroying a plan waits for it)."""
    if _PLAN_CACHE_LOCK is None:
        return
    with _PLAN_CACHE_LOCK:
        plans = list(_PLAN_CACHE.values())
        _PLAN_CACHE.clear()
    for p in plans:
        p.close()

"""Python binding of libsq (include/sq.h): argument marshalling only.

Every function has the name and meaning of the C entry point it wraps.  Device
buffers are torch tensors on the GPU (PyTorch supplies device memory and
streams); the arithmetic runs in the library's HIP kernels.  Importing this
module loads ``libsq.so`` from the package directory and raises if it is
missing: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -m quantized_recurrent_state_gated_amd.build`")

_lib = ctypes.CDLL(LIB_PATH)

SQ_OK, SQ_ERR_INVALID, SQ_ERR_UNSUPPORTED, SQ_ERR_HIP, SQ_ERR_NOMEM, SQ_ERR_DEVICE = 0, -1, -2, -3, -4, -5
SQ_F32, SQ_BF16 = 0, 1
EXPORTED = ("sq_pool_bytes", "sq_pool_alloc", "sq_pool_free", "sq_pool_tile_offset",
            "sq_pool_store", "sq_pool_load", "sq_decode_step", "sq_decode_step_kda", "sq_readout",
            "sq_check_slots", "sq_check_slots_noalloc", "sq_pool_last_device_error",
            "sq_status_string", "sq_decode_step_linear", "sq_prefill", "sq_prefill_workspace",
            "sq_block_tables", "sq_kv_append", "sq_paged_attention", "sq_paged_attention_workspace",
            "sq_kvq_append", "sq_kvq_load", "sq_kvq_attention", "sq_kvq_attention_workspace")
SQ_KVQ_INT8, SQ_KVQ_E4M3 = 0, 1
SQ_RULE_DELTA, SQ_RULE_LINEAR = 0, 1


class SqPoolDesc(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("head_bits", ctypes.POINTER(ctypes.c_uint8)),
                ("row_scale", ctypes.c_void_p), ("col_scale", ctypes.c_void_p),
                ("scale_slot_stride", ctypes.c_int64),
                ("state", ctypes.c_void_p), ("state_bytes", ctypes.c_uint64)]


class SqPrefillDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_seq", "n_tokens", "n_heads", "n_k_heads", "d_k",
                                               "d_v", "dtype", "rule")]
                + [(n, ctypes.c_void_p) for n in ("q", "k", "v")]
                + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")]
                + [(n, ctypes.c_void_p) for n in ("alpha", "beta", "cu_seqlens", "S0", "o", "S",
                                                  "workspace")]
                + [("workspace_bytes", ctypes.c_uint64)])


class SqKvCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class SqKvqCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


_vp, _i32 = ctypes.c_void_p, ctypes.c_int32
_i64, _u64 = ctypes.c_int64, ctypes.c_uint64
_lib.sq_pool_bytes.restype = ctypes.c_uint64
_lib.sq_pool_bytes.argtypes = [_i32, _i32, _i32, _i32, ctypes.POINTER(ctypes.c_uint8)]
_lib.sq_pool_alloc.restype = ctypes.c_int
_lib.sq_pool_alloc.argtypes = [ctypes.POINTER(SqPoolDesc), ctypes.POINTER(_vp)]
_lib.sq_pool_free.restype = None
_lib.sq_pool_free.argtypes = [_vp]
_lib.sq_pool_tile_offset.restype = ctypes.c_int
_lib.sq_pool_tile_offset.argtypes = [_vp, _i32, _i32, ctypes.POINTER(ctypes.c_uint64),
                                     ctypes.POINTER(ctypes.c_uint64)]
_lib.sq_pool_store.restype = ctypes.c_int
_lib.sq_pool_store.argtypes = [_vp, _vp, _i32, _vp, _vp]
_lib.sq_pool_load.restype = ctypes.c_int
_lib.sq_pool_load.argtypes = [_vp, _vp, _i32, _vp, _vp]
_lib.sq_decode_step.restype = ctypes.c_int
_lib.sq_decode_step.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.sq_decode_step_kda.restype = ctypes.c_int
_lib.sq_decode_step_kda.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.sq_decode_step_linear.restype = ctypes.c_int
_lib.sq_decode_step_linear.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.sq_prefill_workspace.restype = _u64
_lib.sq_prefill_workspace.argtypes = [_i32] * 7
_lib.sq_prefill.restype = ctypes.c_int
_lib.sq_prefill.argtypes = [ctypes.POINTER(SqPrefillDesc), _vp]
_lib.sq_block_tables.restype = ctypes.c_int
_lib.sq_block_tables.argtypes = [_vp, _vp, _i32, _i32, _vp, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _i64,
                                 _vp, _vp]
_lib.sq_kv_append.restype = ctypes.c_int
_lib.sq_kv_append.argtypes = [ctypes.POINTER(SqKvCacheDesc), _vp, _vp, _i64, _i64, _vp, _i32, _vp]
_lib.sq_paged_attention_workspace.restype = _u64
_lib.sq_paged_attention_workspace.argtypes = [ctypes.POINTER(SqKvCacheDesc), _i32, _i32, _i32]
_lib.sq_paged_attention.restype = ctypes.c_int
_lib.sq_paged_attention.argtypes = [ctypes.POINTER(SqKvCacheDesc), _vp, _i64, _i32, _i32, _vp, _i64, _vp,
                                    _i32, ctypes.c_float, _i32, _vp, _vp, _vp, _u64, _vp]
_lib.sq_kvq_append.restype = ctypes.c_int
_lib.sq_kvq_append.argtypes = [ctypes.POINTER(SqKvqCacheDesc), _vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _i32,
                               _vp, _i64, _vp]
_lib.sq_kvq_load.restype = ctypes.c_int
_lib.sq_kvq_load.argtypes = [ctypes.POINTER(SqKvqCacheDesc), _vp, _vp, _i32, _vp, _i64, _vp, _vp, _i64, _i64, _i32,
                             _i32, _vp]
_lib.sq_kvq_attention_workspace.restype = _u64
_lib.sq_kvq_attention_workspace.argtypes = [ctypes.POINTER(SqKvqCacheDesc), _i32, _i32, _i32, _i32]
_lib.sq_kvq_attention.restype = ctypes.c_int
_lib.sq_kvq_attention.argtypes = [ctypes.POINTER(SqKvqCacheDesc), _vp, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _i64,
                                  _vp, _i32, ctypes.c_float, _i32, _vp, _vp, _vp, _u64, _vp]
_lib.sq_readout.restype = ctypes.c_int
_lib.sq_readout.argtypes = [_vp, _vp, _i32, _vp, _i32, _vp, _vp]
_lib.sq_check_slots.restype = ctypes.c_int
_lib.sq_check_slots.argtypes = [_vp, _vp, _i32, _vp, _vp]
_lib.sq_check_slots_noalloc.restype = ctypes.c_int
_lib.sq_check_slots_noalloc.argtypes = [_vp, _i32, _i32, _vp, _vp]
_lib.sq_pool_last_device_error.restype = ctypes.c_int
_lib.sq_pool_last_device_error.argtypes = [_vp, _vp]
_lib.sq_status_string.restype = ctypes.c_char_p
_lib.sq_status_string.argtypes = [ctypes.c_int]


class SqError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {sq_status_string(status)} ({status})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != SQ_OK:
        raise SqError(status, where)


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_gpu_seen = False  # torch.cuda.is_available() asks the runtime anew on every call
# the current stream's handle without a Stream object around it (torch has no
# public name for this; without it the public call is used)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int | None:
    global _gpu_seen
    if stream is None:
        if _gpu_seen and _raw_stream is not None and _device is not None:
            return _raw_stream(_device())
        if not torch.cuda.is_available():
            return None
        _gpu_seen = True
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SQ_BF16
    if t.dtype == torch.float32:
        return SQ_F32
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


_FLOATS = (torch.float32, torch.bfloat16)
_DEVICE_TYPES = ("cuda",)  # device types a tensor argument may live on


def _arg(x, where: str, name: str, dtypes, numel: int, optional: bool = False) -> None:
    """Host-side check of a device tensor argument: CUDA, contiguous, one of
    `dtypes`, `numel` elements.  A size mismatch is SQ_ERR_INVALID (as the
    library reports for sizes it can check), a wrong dtype a TypeError.  Raw
    integer pointers are passed through unchecked."""
    # the usual argument, in few steps (a call on small tensors takes as long
    # as its checks)
    if (type(x) is torch.Tensor and x.is_cuda and x.dtype in dtypes and x.numel() == numel
            and x.is_contiguous()):
        return
    if x is None:
        if optional:
            return
        raise SqError(SQ_ERR_INVALID, f"{where} ({name} is required)")
    if isinstance(x, int):
        return
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{where}: {name} must be a torch tensor or a device pointer")
    if x.dtype not in dtypes:
        raise TypeError(f"{where}: {name} must be {' or '.join(str(d) for d in dtypes)}, got {x.dtype}")
    if x.numel() and x.device.type not in _DEVICE_TYPES:
        raise SqError(SQ_ERR_INVALID, f"{where} ({name} is not on a GPU)")
    if not x.is_contiguous():
        raise SqError(SQ_ERR_INVALID, f"{where} ({name} is not contiguous)")
    if x.numel() != numel:
        raise SqError(SQ_ERR_INVALID, f"{where} ({name} has {x.numel()} elements, expected {numel})")


def _bits_array(head_bits):
    hb = bytes(int(b) for b in head_bits)
    return (ctypes.c_uint8 * max(len(hb), 1)).from_buffer_copy(hb or b"\0"), len(hb)


def sq_check_slots(pool: SqPool, slot_ids, result, stream=None) -> None:
    """Write into the int32 device tensor `result` 0 for a valid batch, else
    1 (id out of range) | 2 (id repeated)."""
    n_req = 0 if slot_ids is None else int(slot_ids.numel())
    _arg(result, "sq_check_slots", "result", (torch.int32,), 1)
    _check(_lib.sq_check_slots(pool.handle, _ptr(slot_ids), n_req, _ptr(result), _stream(stream)),
           "sq_check_slots")


def sq_check_slots_noalloc(slot_ids, n_slots: int, result, stream=None) -> None:
    """sq_check_slots without a pool and without any allocation: the stamps
    live in a fixed array inside the library (n_slots <= SQ_CHECK_NOALLOC_MAX_SLOTS)."""
    n_req = 0 if slot_ids is None else int(slot_ids.numel())
    _arg(result, "sq_check_slots_noalloc", "result", (torch.int32,), 1)
    _check(_lib.sq_check_slots_noalloc(_ptr(slot_ids), n_req, int(n_slots), _ptr(result),
                                       _stream(stream)), "sq_check_slots_noalloc")


def sq_pool_last_device_error(pool: SqPool, stream=None) -> int:
    """Synchronize the stream, then read and clear the pool's sticky flag:
    SQ_OK, or SQ_ERR_DEVICE if a kernel met a non-finite updated value."""
    st = _lib.sq_pool_last_device_error(pool.handle, _stream(stream))
    if st not in (SQ_OK, SQ_ERR_DEVICE):
        _check(st, "sq_pool_last_device_error")
    return st


def sq_status_string(status: int) -> str:
    return _lib.sq_status_string(int(status)).decode()


def sq_pool_bytes(n_slots: int, n_heads: int, d_k: int, d_v: int, head_bits) -> int:
    arr, _ = _bits_array(head_bits)
    return int(_lib.sq_pool_bytes(n_slots, n_heads, d_k, d_v, arr))


class SqPool:
    """Owner of an sq_pool handle; keeps the borrowed tensors alive."""

    def __init__(self, handle: int, keep: tuple, n_slots: int, n_heads: int, d_k: int, d_v: int,
                 head_bits):
        self.handle = handle
        self._keep = keep
        self._free = _lib.sq_pool_free  # the library that made the handle releases it
        self.n_slots, self.n_heads, self.d_k, self.d_v = n_slots, n_heads, d_k, d_v
        self.head_bits = list(int(b) for b in head_bits)

    @property
    def state(self) -> torch.Tensor:
        return self._keep[0]

    def __del__(self):
        # also runs at interpreter exit, when module globals may already be gone
        handle, free = getattr(self, "handle", None), getattr(self, "_free", None)
        if handle and free is not None:
            try:
                free(handle)
            except Exception:
                pass
        self.handle = None


def sq_pool_alloc(n_slots: int, n_heads: int, d_k: int, d_v: int, head_bits, row_scale,
                  col_scale, state, state_bytes: int | None = None,
                  scale_slot_stride: int = 0) -> SqPool:
    """Wrap sq_pool_alloc; `state` is a uint8 device tensor (the caller's buffer).
    With scale_slot_stride S > 0 the factor tensors hold n_slots * S per-head
    vectors (slot p, head h at vector p * S + h)."""
    arr, nb = _bits_array(head_bits)
    vecs = n_slots * scale_slot_stride if scale_slot_stride > 0 else n_heads
    _arg(row_scale, "sq_pool_alloc", "row_scale", (torch.float32,), vecs * d_k)
    _arg(col_scale, "sq_pool_alloc", "col_scale", (torch.float32,), vecs * d_v)
    if isinstance(state, torch.Tensor):
        _arg(state, "sq_pool_alloc", "state", (state.dtype,), state.numel())
    if state_bytes is None:
        state_bytes = state.numel() * state.element_size() if hasattr(state, "numel") else 0
    desc = SqPoolDesc(n_slots, n_heads, d_k, d_v, arr, _ptr(row_scale), _ptr(col_scale),
                      int(scale_slot_stride), _ptr(state), int(state_bytes))
    h = _vp()
    _check(_lib.sq_pool_alloc(ctypes.byref(desc), ctypes.byref(h)), "sq_pool_alloc")
    return SqPool(h.value, (state, row_scale, col_scale), n_slots, n_heads, d_k, d_v,
                  list(head_bits)[:nb])


def sq_pool_free(pool: SqPool) -> None:
    if pool is not None and getattr(pool, "handle", None):
        pool._free(pool.handle)
        pool.handle = None


def sq_pool_tile_offset(pool: SqPool, slot: int, head: int):
    off, nb = ctypes.c_uint64(), ctypes.c_uint64()
    _check(_lib.sq_pool_tile_offset(pool.handle, slot, head, ctypes.byref(off), ctypes.byref(nb)),
           "sq_pool_tile_offset")
    return int(off.value), int(nb.value)


def _state_elems(pool: SqPool, n_req: int) -> int:
    return n_req * pool.n_heads * pool.d_k * pool.d_v


def sq_pool_store(pool: SqPool, slot_ids, S, stream=None) -> None:
    n_req = 0 if slot_ids is None else int(slot_ids.numel())
    if n_req:
        _arg(slot_ids, "sq_pool_store", "slot_ids", (torch.int32,), n_req)
        _arg(S, "sq_pool_store", "S", (torch.float32,), _state_elems(pool, n_req))
    _check(_lib.sq_pool_store(pool.handle, _ptr(slot_ids), n_req, _ptr(S), _stream(stream)),
           "sq_pool_store")


def sq_pool_load(pool: SqPool, slot_ids, S, stream=None) -> None:
    """Dequantize the slots' states into the fp32 device tensor S [n_req][H][dk][dv]."""
    n_req = 0 if slot_ids is None else int(slot_ids.numel())
    if n_req:
        _arg(slot_ids, "sq_pool_load", "slot_ids", (torch.int32,), n_req)
        _arg(S, "sq_pool_load", "S", (torch.float32,), _state_elems(pool, n_req))
    _check(_lib.sq_pool_load(pool.handle, _ptr(slot_ids), n_req, _ptr(S), _stream(stream)),
           "sq_pool_load")


def _step_args(where, pool, slot_ids, q, k, v, alpha, beta, o, alpha_per_channel):
    n_req = int(slot_ids.numel())
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError(f"{where}: q, k and v must share one dtype")
    H, dk, dv = pool.n_heads, pool.d_k, pool.d_v
    _arg(slot_ids, where, "slot_ids", (torch.int32,), n_req)
    _arg(q, where, "q", _FLOATS, n_req * H * dk)
    _arg(k, where, "k", _FLOATS, n_req * H * dk)
    _arg(v, where, "v", _FLOATS, n_req * H * dv)
    _arg(alpha, where, "alpha", (torch.float32,), n_req * H * (dk if alpha_per_channel else 1))
    _arg(beta, where, "beta", (torch.float32,), n_req * H)
    _arg(o, where, "o", (torch.float32,), n_req * H * dv, optional=True)
    return n_req


def sq_decode_step(pool: SqPool, slot_ids, q, k, v, alpha, beta, o=None, stream=None) -> None:
    n_req = _step_args("sq_decode_step", pool, slot_ids, q, k, v, alpha, beta, o, False)
    _check(_lib.sq_decode_step(pool.handle, _ptr(slot_ids), n_req, _ptr(q), _ptr(k), _ptr(v),
                               _dtype_code(q), _ptr(alpha), _ptr(beta), _ptr(o), _stream(stream)),
           "sq_decode_step")


def sq_decode_step_kda(pool: SqPool, slot_ids, q, k, v, alpha, beta, o=None, stream=None) -> None:
    """Per-key-channel-gate step; alpha is fp32 [n_req][n_heads][d_k]."""
    n_req = _step_args("sq_decode_step_kda", pool, slot_ids, q, k, v, alpha, beta, o, True)
    _check(_lib.sq_decode_step_kda(pool.handle, _ptr(slot_ids), n_req, _ptr(q), _ptr(k), _ptr(v),
                                   _dtype_code(q), _ptr(alpha), _ptr(beta), _ptr(o),
                                   _stream(stream)), "sq_decode_step_kda")


def sq_readout(pool: SqPool, slot_ids, q, o, stream=None) -> None:
    n_req = int(slot_ids.numel())
    _arg(slot_ids, "sq_readout", "slot_ids", (torch.int32,), n_req)
    _arg(q, "sq_readout", "q", _FLOATS, n_req * pool.n_heads * pool.d_k)
    _arg(o, "sq_readout", "o", (torch.float32,), n_req * pool.n_heads * pool.d_v)
    _check(_lib.sq_readout(pool.handle, _ptr(slot_ids), n_req, _ptr(q), _dtype_code(q), _ptr(o),
                           _stream(stream)), "sq_readout")


def sq_decode_step_linear(pool: SqPool, slot_ids, q, k, v, alpha, beta, o=None, stream=None) -> None:
    """The step without the delta correction: S' = alpha S + beta k v^T, o = S'^T q."""
    n_req = _step_args("sq_decode_step_linear", pool, slot_ids, q, k, v, alpha, beta, o, False)
    _check(_lib.sq_decode_step_linear(pool.handle, _ptr(slot_ids), n_req, _ptr(q), _ptr(k), _ptr(v),
                                      _dtype_code(q), _ptr(alpha), _ptr(beta), _ptr(o),
                                      _stream(stream)), "sq_decode_step_linear")


# ---------------------------------------------------------------- prompts, paged cache

def _int32(x, where: str, name: str) -> int:
    """A size that the library takes as 32 bits (ctypes would cut it to them)."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise SqError(SQ_ERR_INVALID, f"{where} ({name} = {x} does not fit 32 bits)")
    return x


def _rows(x, where: str, name: str, dtype, shape) -> int:
    """Check a [tokens][heads][d] tensor whose tokens may lie further apart
    than their elements (a part of a wider buffer); returns that distance."""
    if type(x) is torch.Tensor and x.is_cuda and x.dtype is dtype and x.shape == shape and x.is_contiguous():
        return shape[1] * shape[2]
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{where}: {name} must be a torch tensor")
    if x.dtype != dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, got {x.dtype}")
    if tuple(x.shape) != shape:
        raise SqError(SQ_ERR_INVALID, f"{where} ({name} has shape {tuple(x.shape)}, expected {shape})")
    row = shape[1] * shape[2]
    if not x.numel():
        return row
    if x.device.type not in _DEVICE_TYPES:
        raise SqError(SQ_ERR_INVALID, f"{where} ({name} is not on a GPU)")
    st = x.stride()
    if (shape[2] > 1 and st[2] != 1) or (shape[1] > 1 and st[1] != shape[2]):
        raise SqError(SQ_ERR_INVALID, f"{where} (the heads of a token of {name} are not contiguous)")
    return st[0] if shape[0] > 1 else row


def sq_prefill_workspace(n_seq: int, n_tokens: int, n_heads: int, d_k: int, d_v: int, dtype,
                         rule: int = SQ_RULE_DELTA) -> int:
    """Bytes of workspace of sq_prefill; `dtype` is a torch dtype or an sq_dtype."""
    code = {torch.bfloat16: SQ_BF16, torch.float32: SQ_F32}.get(dtype, dtype)
    if not isinstance(code, int):
        raise TypeError(f"sq_prefill_workspace: dtype must be float32 or bfloat16, got {dtype}")
    sizes = [_int32(x, "sq_prefill_workspace", name) for x, name in (
        (n_seq, "n_seq"), (n_tokens, "n_tokens"), (n_heads, "n_heads"), (d_k, "d_k"), (d_v, "d_v"),
        (code, "dtype"), (rule, "rule"))]
    return int(_lib.sq_prefill_workspace(*sizes))


def sq_prefill(q, k, v, alpha, beta, cu_seqlens, o, S=None, S0=None, rule: int = SQ_RULE_DELTA,
               workspace=None, stream=None) -> None:
    """Packed prompts through the recurrent state.  q, k [N][Hk][dk], v and o
    [N][H][dv] (float32 or bfloat16, tokens may be strided, o contiguous), alpha
    and beta fp32 [N][H], cu_seqlens int32 [n_seq + 1], S0 and S fp32
    [n_seq][H][dk][dv].  `workspace`: uint8, sq_prefill_workspace bytes."""
    w = "sq_prefill"
    if q.dim() != 3 or v.dim() != 3:
        raise SqError(SQ_ERR_INVALID, f"{w} (q, k and v are [tokens][heads][d])")
    code, dt = _dtype_code(q), q.dtype
    N, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    n_seq, rule = int(cu_seqlens.numel()) - 1, _int32(rule, w, "rule")
    _int32(N, w, "n_tokens")
    qs = _rows(q, w, "q", dt, (N, Hk, dk))
    ks = _rows(k, w, "k", dt, (N, Hk, dk))
    vs = _rows(v, w, "v", dt, (N, H, dv))
    _arg(alpha, w, "alpha", (torch.float32,), N * H)
    _arg(beta, w, "beta", (torch.float32,), N * H)
    _arg(cu_seqlens, w, "cu_seqlens", (torch.int32,), n_seq + 1)
    _arg(o, w, "o", (dt,), N * H * dv)
    _arg(S, w, "S", (torch.float32,), n_seq * H * dk * dv, optional=True)
    _arg(S0, w, "S0", (torch.float32,), n_seq * H * dk * dv, optional=True)
    ws, nb = _workspace(workspace, w)
    d = SqPrefillDesc(n_seq, N, H, Hk, dk, dv, code, rule, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                      qs, ks, vs, _ptr(alpha), _ptr(beta), _ptr(cu_seqlens),
                      None if S0 is None else _ptr(S0), _ptr(o), None if S is None else _ptr(S), ws, nb)
    _check(_lib.sq_prefill(ctypes.byref(d), _stream(stream)), w)


def _workspace(ws, where: str):
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor) or not ws.is_contiguous():
        raise TypeError(f"{where}: workspace must be a contiguous torch tensor")
    if ws.numel() and ws.device.type not in _DEVICE_TYPES:
        raise SqError(SQ_ERR_INVALID, f"{where} (workspace is not on a GPU)")
    return ws.data_ptr(), ws.numel() * ws.element_size()


class SqKvCache:
    """A paged key-value cache over two tensors: k [n_pages][n_kv_heads][page_size][head_dim],
    v [n_pages][n_kv_heads][head_dim][page_size], float32 or bfloat16; keeps them alive."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 4:
            raise SqError(SQ_ERR_INVALID, "SqKvCache (k is [n_pages][n_kv_heads][page_size][head_dim])")
        pages, heads, page, d = k.shape
        code = _dtype_code(k)
        _arg(k, "SqKvCache", "k", _FLOATS, k.numel())
        _arg(v, "SqKvCache", "v", (k.dtype,), k.numel())
        if tuple(v.shape) != (pages, heads, d, page):
            raise SqError(SQ_ERR_INVALID, "SqKvCache (v is [n_pages][n_kv_heads][head_dim][page_size])")
        self.k, self.v, self.dtype = k, v, k.dtype
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = pages, page, heads, d
        self.desc = SqKvCacheDesc(k.data_ptr(), v.data_ptr(), pages, page, heads, d, code)
        self.ref = ctypes.byref(self.desc)


def sq_block_tables(ctx_lens, new_lens, page_size: int, free_pages, block_table, seq_lens, cu_new,
                    cu_pages, slot_map, result, stream=None) -> None:
    """Extend the rows of block_table [n_req][stride] by the pages that new_lens
    tokens after ctx_lens need (taken from free_pages in order) and write
    seq_lens, cu_new, cu_pages, the slot of every new token and a result word."""
    w, i32 = "sq_block_tables", (torch.int32,)
    n = int(ctx_lens.numel())
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise SqError(SQ_ERR_INVALID, f"{w} (block_table is [n_req][stride])")
    _arg(ctx_lens, w, "ctx_lens", i32, n)
    _arg(new_lens, w, "new_lens", i32, n)
    _arg(free_pages, w, "free_pages", i32, free_pages.numel())
    _arg(block_table, w, "block_table", i32, block_table.numel())
    _arg(seq_lens, w, "seq_lens", i32, n)
    _arg(cu_new, w, "cu_new", i32, n + 1)
    _arg(cu_pages, w, "cu_pages", i32, n + 1)
    _arg(slot_map, w, "slot_map", (torch.int64,), slot_map.numel())
    _arg(result, w, "result", i32, 1)
    _check(_lib.sq_block_tables(_ptr(ctx_lens), _ptr(new_lens), n, _int32(page_size, w, "page_size"), _ptr(free_pages),
                                free_pages.numel(), _ptr(block_table), block_table.shape[1],
                                _ptr(seq_lens), _ptr(cu_new), _ptr(cu_pages), _ptr(slot_map),
                                slot_map.numel(), _ptr(result), _stream(stream)), w)


def sq_kv_append(cache: SqKvCache, k, v, slot_map, stream=None) -> None:
    """cache[slot_map[t]] = k[t], v[t]; k, v [tokens][n_kv_heads][head_dim],
    tokens may be strided; slots outside the cache are skipped."""
    w, n = "sq_kv_append", int(slot_map.numel())
    shape = (n, cache.n_kv_heads, cache.head_dim)
    ks, vs = _rows(k, w, "k", cache.dtype, shape), _rows(v, w, "v", cache.dtype, shape)
    _arg(slot_map, w, "slot_map", (torch.int64,), n)
    _check(_lib.sq_kv_append(cache.ref, k.data_ptr(), v.data_ptr(), ks, vs, slot_map.data_ptr(), n,
                             _stream(stream)), w)


def sq_paged_attention_workspace(cache: SqKvCache, n_req: int, n_heads: int, max_len: int) -> int:
    w = "sq_paged_attention_workspace"
    return int(_lib.sq_paged_attention_workspace(cache.ref, _int32(n_req, w, "n_req"), _int32(n_heads, w, "n_heads"),
                                                 _int32(max_len, w, "max_len")))


def sq_paged_attention(cache: SqKvCache, q, block_table, seq_lens, max_len: int, o, workspace=None,
                       scale: float | None = None, window: int = 0, lse=None, stream=None) -> None:
    """Attention of one new token per request, q [n_req][n_heads][head_dim], over
    its cached tokens; scale defaults to head_dim ** -0.5, window 0 is no window.
    `workspace`: sq_paged_attention_workspace bytes."""
    w = "sq_paged_attention"
    if q.dim() != 3:
        raise SqError(SQ_ERR_INVALID, f"{w} (q is [n_req][n_heads][head_dim])")
    n, heads, d = q.shape
    qs = _rows(q, w, "q", cache.dtype, (n, heads, cache.head_dim))
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise SqError(SQ_ERR_INVALID, f"{w} (block_table is [n_req][stride])")
    _arg(block_table, w, "block_table", (torch.int32,), block_table.numel())
    _arg(seq_lens, w, "seq_lens", (torch.int32,), n)
    _arg(o, w, "o", (cache.dtype,), n * heads * d)
    _arg(lse, w, "lse", (torch.float32,), n * heads, optional=True)
    ws, nb = _workspace(workspace, w)
    _check(_lib.sq_paged_attention(cache.ref, q.data_ptr(), qs, n, heads, block_table.data_ptr(),
                                   block_table.shape[1], seq_lens.data_ptr(), _int32(max_len, w, "max_len"),
                                   d ** -0.5 if scale is None else float(scale), _int32(window, w, "window"),
                                   o.data_ptr(), _ptr(lse), ws, nb, _stream(stream)), w)


# ---------------------------------------------------------------- 8-bit paged cache

class SqKvqCache:
    """A paged key-value cache of one byte a value over three tensors: k uint8
    [n_pages][n_kv_heads][page_size][head_dim], v uint8 [n_pages][n_kv_heads][page_size / 16][head_dim][16],
    scales fp32 [n_pages][n_kv_heads][page_size / 16][2]; keeps them alive."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, scales: torch.Tensor, format: int = SQ_KVQ_INT8):
        w, u8 = "SqKvqCache", (torch.uint8,)
        if k.dim() != 4:
            raise SqError(SQ_ERR_INVALID, f"{w} (k is [n_pages][n_kv_heads][page_size][head_dim])")
        pages, heads, page, d = k.shape
        _arg(k, w, "k", u8, k.numel())
        _arg(v, w, "v", u8, k.numel())
        _arg(scales, w, "scales", (torch.float32,), pages * heads * (page // 16) * 2)
        if tuple(v.shape) != (pages, heads, page // 16, d, 16):
            raise SqError(SQ_ERR_INVALID, f"{w} (v is [n_pages][n_kv_heads][page_size / 16][head_dim][16])")
        if tuple(scales.shape) != (pages, heads, page // 16, 2):
            raise SqError(SQ_ERR_INVALID, f"{w} (scales is [n_pages][n_kv_heads][page_size / 16][2])")
        if format not in (SQ_KVQ_INT8, SQ_KVQ_E4M3):
            raise SqError(SQ_ERR_INVALID, f"{w} (format {format})")
        self.k, self.v, self.scales, self.format = k, v, scales, format
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = pages, page, heads, d
        self.desc = SqKvqCacheDesc(k.data_ptr(), v.data_ptr(), scales.data_ptr(), pages, page, heads, d, format)
        self.ref = ctypes.byref(self.desc)


def sq_kvq_append(cache: SqKvqCache, k, v, ctx_lens, cu_new, block_table, stream=None) -> None:
    """Quantize and append: tokens cu_new[r] .. cu_new[r + 1] - 1 of k, v [tokens][n_kv_heads][head_dim]
    (float32 or bfloat16, tokens may be strided) go to positions ctx_lens[r] on of request r."""
    w, i32 = "sq_kvq_append", (torch.int32,)
    n, N, code = int(ctx_lens.numel()), k.shape[0], _dtype_code(k)
    shape = (N, cache.n_kv_heads, cache.head_dim)
    ks, vs = _rows(k, w, "k", k.dtype, shape), _rows(v, w, "v", k.dtype, shape)
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise SqError(SQ_ERR_INVALID, f"{w} (block_table is [n_req][stride])")
    _arg(ctx_lens, w, "ctx_lens", i32, n)
    _arg(cu_new, w, "cu_new", i32, n + 1)
    _arg(block_table, w, "block_table", i32, block_table.numel())
    _check(_lib.sq_kvq_append(cache.ref, k.data_ptr(), v.data_ptr(), ks, vs, code, _int32(N, w, "tokens"),
                              ctx_lens.data_ptr(), cu_new.data_ptr(), n, block_table.data_ptr(), block_table.shape[1],
                              _stream(stream)), w)


def sq_kvq_load(cache: SqKvqCache, block_table, cu, k=None, v=None, first=None, stream=None) -> None:
    """Read back: rows cu[r] .. cu[r + 1] - 1 of k and v [tokens][n_kv_heads][head_dim] (float32 or
    bfloat16, tokens may be strided; either may be None) receive positions first[r] (or 0) on of request r."""
    w, i32 = "sq_kvq_load", (torch.int32,)
    if k is None and v is None:
        raise SqError(SQ_ERR_INVALID, f"{w} (k or v is required)")
    n, some = int(cu.numel()) - 1, v if k is None else k
    N, dt, code = some.shape[0], some.dtype, _dtype_code(some)
    shape = (N, cache.n_kv_heads, cache.head_dim)
    ks = 0 if k is None else _rows(k, w, "k", dt, shape)
    vs = 0 if v is None else _rows(v, w, "v", dt, shape)
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise SqError(SQ_ERR_INVALID, f"{w} (block_table is [n_req][stride])")
    _arg(first, w, "first", i32, n, optional=True)
    _arg(cu, w, "cu", i32, n + 1)
    _arg(block_table, w, "block_table", i32, block_table.numel())
    _check(_lib.sq_kvq_load(cache.ref, _ptr(first), cu.data_ptr(), n, block_table.data_ptr(), block_table.shape[1],
                            _ptr(k), _ptr(v), ks, vs, code, _int32(N, w, "tokens"), _stream(stream)), w)


def sq_kvq_attention_workspace(cache: SqKvqCache, n_req: int, n_q: int, n_heads: int, max_len: int) -> int:
    w = "sq_kvq_attention_workspace"
    return int(_lib.sq_kvq_attention_workspace(cache.ref, _int32(n_req, w, "n_req"), _int32(n_q, w, "n_q"),
                                               _int32(n_heads, w, "n_heads"), _int32(max_len, w, "max_len")))


def sq_kvq_attention(cache: SqKvqCache, q, block_table, seq_lens, max_len: int, o, workspace=None, cu_q=None,
                     scale: float | None = None, window: int = 0, lse=None, stream=None) -> None:
    """Attention of q [queries][n_heads][head_dim] over the cached tokens: one query per request, or with
    cu_q the last cu_q[r + 1] - cu_q[r] tokens of each, causal; scale defaults to head_dim ** -0.5, window 0
    is no window.  `workspace`: sq_kvq_attention_workspace bytes."""
    w = "sq_kvq_attention"
    if q.dim() != 3:
        raise SqError(SQ_ERR_INVALID, f"{w} (q is [queries][n_heads][head_dim])")
    nq, heads, d = q.shape
    n, code, dt = int(seq_lens.numel()), _dtype_code(q), q.dtype
    qs = _rows(q, w, "q", dt, (nq, heads, cache.head_dim))
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise SqError(SQ_ERR_INVALID, f"{w} (block_table is [n_req][stride])")
    if cu_q is not None:
        _arg(cu_q, w, "cu_q", (torch.int32,), n + 1)
        cu_q = _ptr(cu_q)
    _arg(block_table, w, "block_table", (torch.int32,), block_table.numel())
    _arg(seq_lens, w, "seq_lens", (torch.int32,), n)
    _arg(o, w, "o", (dt,), nq * heads * d)
    _arg(lse, w, "lse", (torch.float32,), nq * heads, optional=True)
    ws, nb = _workspace(workspace, w)
    _check(_lib.sq_kvq_attention(cache.ref, q.data_ptr(), qs, code, _int32(nq, w, "queries"), heads, cu_q, n,
                                 block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
                                 _int32(max_len, w, "max_len"), d ** -0.5 if scale is None else float(scale),
                                 _int32(window, w, "window"), o.data_ptr(), _ptr(lse), ws, nb, _stream(stream)), w)

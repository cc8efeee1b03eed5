"""Thin ctypes binding of libpva.so (the C ABI in include/pva.h).

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels.  torch is used for device memory and the current stream.  The
library is loaded on first use; if it is missing this raises -- there is no
other code path.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpva.so")

PVA_OK = 0
STATUS_NAMES = {
    0: "PVA_OK", 1: "PVA_ERR_INVALID_ARG", 2: "PVA_ERR_UNSUPPORTED", 3: "PVA_ERR_WORKSPACE_TOO_SMALL",
    4: "PVA_ERR_CUDA", 5: "PVA_ERR_DEVICE_CHECK", 6: "PVA_ERR_NOT_PREPARED",
}
DEVERR = {
    0x01: "PVA_DEVERR_CU_SEQLENS", 0x02: "PVA_DEVERR_Q_GT_KV", 0x04: "PVA_DEVERR_PAGE_ID",
    0x08: "PVA_DEVERR_SLOT", 0x10: "PVA_DEVERR_LIMITS", 0x20: "PVA_DEVERR_TIMEOUT",
    0x40: "PVA_DEVERR_POSITION", 0x80: "PVA_DEVERR_STATE",
}
# Every function include/pva.h declares; the CPU tests check the library exports each one.
EXPORTS = ("attn_abi_version", "attn_status_string", "attn_workspace_size", "attn_prepare_metadata",
           "attn_forward", "attn_store_kvcache", "attn_get_device_status", "attn_debug_plan_counts",
           "attn_set_timing_events", "attn_prepare_metadata_static", "attn_forward_fp8kv", "attn_store_kvcache_fp8kv",
           "attn_debug_set_wait_limit", "attn_forward_mxfp4kv", "attn_store_kvcache_mxfp4kv",
           "attn_load_kvcache_mxfp4kv", "attn_mxfp4_row_bytes", "attn_append_rope", "attn_forward_rope",
           "attn_append_norm_rope", "attn_forward_norm_rope", "attn_norm_rope", "attn_linear_workspace_size",
           "attn_linear_prepare", "attn_linear_forward", "attn_linear_forward_norm_rope")


class PvaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class Config(ctypes.Structure):
    """Mirror of pva_config."""
    _fields_ = [
        ("num_qo_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("sm_scale", ctypes.c_float),
        ("max_batch", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("max_kv_len", ctypes.c_int32),
        ("enable_split_kv", ctypes.c_int32), ("enable_cascade", ctypes.c_int32),
        ("min_cascade_pages", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
    ]


class LinearConfig(ctypes.Structure):
    """Mirror of pva_linear_config."""
    _fields_ = [
        ("num_qo_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("scale", ctypes.c_float), ("num_states", ctypes.c_int64), ("max_batch", ctypes.c_int32),
        ("max_tokens", ctypes.c_int32),
    ]


class Meta(ctypes.Structure):
    """Mirror of pva_meta (opaque, caller-owned, host memory)."""
    _fields_ = [("opaque", ctypes.c_uint64 * 64)]
    batch = None   # what the prepared batch asks of a call's tensors (Batch), made when a call first asks
    _sizes = None

    def of_batch(self):
        """The Batch, or None of a meta that was never prepared."""
        if self.batch is None and self._sizes is not None:
            self.batch = Batch(*self._sizes)
        return self.batch


class Batch:
    """Sizes of a prepared batch, its device, and the element types of a call's tensors."""
    __slots__ = ("tokens", "q_heads", "kv_heads", "head_dim", "nq", "nkv", "nlse", "pool_bytes", "scaled", "device",
                 "bf16", "f32")

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, slots: int, kv_dtype: int, tokens: int, device: int):
        import torch

        self.tokens, self.device = int(tokens), device
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        elems = kv_heads * head_dim
        row = {KV_BF16: 2 * elems, KV_E4M3: elems, _STATES: 4 * elems * head_dim}.get(kv_dtype)
        if row is None:
            row = int(load().attn_mxfp4_row_bytes(self.kv_heads, self.head_dim))
        self.nq, self.nkv = self.tokens * self.q_heads * self.head_dim, self.tokens * elems
        self.nlse = self.tokens * self.q_heads
        self.pool_bytes = slots * row
        self.scaled = kv_dtype == KV_E4M3
        self.bf16, self.f32 = torch.bfloat16, torch.float32

    def lacks(self, x, n: int, dtype) -> bool:
        """Whether x (or None, which the library refuses itself) is not at least n contiguous elements of
        the type on the batch's device."""
        return x is not None and (x.numel() < n or x.dtype is not dtype or x.get_device() != self.device
                                  or not x.is_contiguous())

    def lacks_pools(self, k_pool, v_pool) -> bool:
        n, dev = self.pool_bytes, self.device
        return (k_pool is not None and (k_pool.nbytes < n or k_pool.get_device() != dev or not k_pool.is_contiguous())
                or v_pool is not None and (v_pool.nbytes < n or v_pool.get_device() != dev or not v_pool.is_contiguous()))

    def refusal(self, where: str) -> PvaError:
        return PvaError(1, f"{where} (for {self.tokens} tokens of {self.q_heads} / {self.kv_heads} heads of "
                           f"{self.head_dim}, pools of {self.pool_bytes} bytes: a tensor that is shorter, strided, "
                           "of another type or on another device)")


def _batch_sizes(cfg: Config, total_tokens, device: int):
    return (cfg.num_qo_heads, cfg.num_kv_heads, cfg.head_dim, cfg.num_pages * cfg.page_size, cfg.kv_dtype, total_tokens,
            device)


def _linear_sizes(cfg: LinearConfig, total_tokens, device: int):
    return (cfg.num_qo_heads, cfg.num_kv_heads, cfg.head_dim, cfg.num_states, _STATES, total_tokens, device)


class RopeArgs(ctypes.Structure):
    """Mirror of pva_rope."""
    _fields_ = [
        ("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("ld_q", ctypes.c_int64),
        ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64), ("max_positions", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class QKNormArgs(ctypes.Structure):
    """Mirror of pva_qk_norm."""
    _fields_ = [("q_gain", ctypes.c_void_p), ("k_gain", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class LinearArgs(ctypes.Structure):
    """Mirror of pva_linear_args."""
    _fields_ = [("log_decay", ctypes.c_void_p), ("ld_decay", ctypes.c_int64), ("ld_q", ctypes.c_int64),
                ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64), ("states", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load libpva.so (once).  Raises FileNotFoundError when it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise FileNotFoundError(f"{path} is missing: build it with paged_variable_length_gb300.build.build()")
        lib = ctypes.CDLL(path)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        CP, MP = ctypes.POINTER(Config), ctypes.POINTER(Meta)
        lib.attn_abi_version.argtypes, lib.attn_abi_version.restype = [], i32
        lib.attn_status_string.argtypes, lib.attn_status_string.restype = [ctypes.c_int], ctypes.c_char_p
        lib.attn_workspace_size.argtypes, lib.attn_workspace_size.restype = [CP], sz
        lib.attn_prepare_metadata.argtypes = [CP, P, P, P, i64, P, i32, i32, i32, P, sz, P, MP]
        lib.attn_prepare_metadata.restype = ctypes.c_int
        lib.attn_prepare_metadata_static.argtypes = [CP, P, P, P, i64, P, i32, i32, i32, P, MP]
        lib.attn_prepare_metadata_static.restype = ctypes.c_int
        lib.attn_forward.argtypes = [MP, P, P, P, P, P, P, P, P]
        lib.attn_forward.restype = ctypes.c_int
        lib.attn_store_kvcache.argtypes = [MP, P, P, P, P, P]
        lib.attn_store_kvcache.restype = ctypes.c_int
        lib.attn_forward_fp8kv.argtypes = [MP, P, P, P, P, P, P, P, P, P, P]
        lib.attn_forward_fp8kv.restype = ctypes.c_int
        lib.attn_store_kvcache_fp8kv.argtypes = [MP, P, P, P, P, P, P, P]
        lib.attn_store_kvcache_fp8kv.restype = ctypes.c_int
        lib.attn_forward_mxfp4kv.argtypes = [MP, P, P, P, P, P, P, P, P]
        lib.attn_forward_mxfp4kv.restype = ctypes.c_int
        lib.attn_store_kvcache_mxfp4kv.argtypes = [MP, P, P, P, P, P]
        lib.attn_store_kvcache_mxfp4kv.restype = ctypes.c_int
        lib.attn_load_kvcache_mxfp4kv.argtypes = [MP, P, P, P, P, P]
        lib.attn_load_kvcache_mxfp4kv.restype = ctypes.c_int
        lib.attn_mxfp4_row_bytes.argtypes, lib.attn_mxfp4_row_bytes.restype = [i32, i32], i64
        RP = ctypes.POINTER(RopeArgs)
        lib.attn_append_rope.argtypes = [MP, RP, P, P, P, P, P, P, P, P, P]
        lib.attn_append_rope.restype = ctypes.c_int
        lib.attn_forward_rope.argtypes = [MP, RP, P, P, P, P, P, P, P, P, P, P, P]
        lib.attn_forward_rope.restype = ctypes.c_int
        NP, LP, CL = ctypes.POINTER(QKNormArgs), ctypes.POINTER(LinearArgs), ctypes.POINTER(LinearConfig)
        lib.attn_append_norm_rope.argtypes = [MP, NP, RP, P, P, P, P, P, P, P, P, P]
        lib.attn_append_norm_rope.restype = ctypes.c_int
        lib.attn_forward_norm_rope.argtypes = [MP, NP, RP, P, P, P, P, P, P, P, P, P, P, P]
        lib.attn_forward_norm_rope.restype = ctypes.c_int
        lib.attn_norm_rope.argtypes, lib.attn_norm_rope.restype = [MP, NP, RP, P, P, P, P, P], ctypes.c_int
        lib.attn_linear_workspace_size.argtypes, lib.attn_linear_workspace_size.restype = [CL], sz
        lib.attn_linear_prepare.argtypes = [CL, P, P, P, P, i32, i32, i32, P, sz, P, MP]
        lib.attn_linear_prepare.restype = ctypes.c_int
        lib.attn_linear_forward.argtypes, lib.attn_linear_forward.restype = [MP, LP, P, P, P, P, P], ctypes.c_int
        lib.attn_linear_forward_norm_rope.argtypes = [MP, LP, NP, RP, P, P, P, P, P, P, P]
        lib.attn_linear_forward_norm_rope.restype = ctypes.c_int
        lib.attn_get_device_status.argtypes = [MP, ctypes.POINTER(ctypes.c_uint32)]
        lib.attn_get_device_status.restype = ctypes.c_int
        lib.attn_set_timing_events.argtypes = [MP, ctypes.POINTER(ctypes.c_void_p), i32]
        lib.attn_set_timing_events.restype = ctypes.c_int
        lib.attn_debug_set_wait_limit.argtypes = [MP, i64]
        lib.attn_debug_set_wait_limit.restype = ctypes.c_int
        lib.attn_debug_plan_counts.argtypes = [MP, ctypes.POINTER(ctypes.c_int64), i32]
        lib.attn_debug_plan_counts.restype = i32
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().attn_status_string(int(status)).decode()


def abi_version() -> int:
    return int(load().attn_abi_version())


def _check(status: int, where: str) -> None:
    if status != PVA_OK:
        raise PvaError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


_raw_stream = None


def _current():
    """(handle of a device's current stream, the current device): functions that make no stream
    object (which costs more than the launch it is for)."""
    global _raw_stream
    if _raw_stream is None:
        import torch

        torch.cuda.current_stream()  # initialises CUDA
        _raw_stream = (torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)
    return _raw_stream


def _stream(stream):
    if stream is None:
        handle, device = _raw_stream or _current()
        return handle(device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_on(b, stream, where):
    """The stream's handle for a call of batch b, whose device has to be the current one (the library
    launches there, whatever the stream)."""
    on_gpu = b is not None and b.device >= 0
    if on_gpu or stream is None:
        handle, device = _raw_stream or _current()
        current = device()
        if on_gpu and current != b.device:
            raise PvaError(1, f"{where} (the batch is on GPU {b.device}, which is not the current device)")
        if stream is None:
            return handle(current)
    return _stream(stream)


KV_BF16, KV_E4M3, KV_MXFP4 = 0, 1, 2
_STATES = -1   # in the place of a pool type: states of linear attention


def make_config(num_qo_heads, num_kv_heads, head_dim, page_size, num_pages, max_batch, max_tokens, max_kv_len,
                sm_scale: float = 0.0, enable_split_kv: bool = True, enable_cascade: bool = True,
                min_cascade_pages: int = 8, kv_dtype: int = KV_BF16) -> Config:
    return Config(num_qo_heads, num_kv_heads, head_dim, page_size, num_pages, sm_scale, max_batch, max_tokens,
                  max_kv_len, int(enable_split_kv), int(enable_cascade), int(min_cascade_pages), int(kv_dtype))


def attn_workspace_size(cfg: Config) -> int:
    return int(load().attn_workspace_size(ctypes.byref(cfg)))


def attn_prepare_metadata(cfg: Config, cu_seqlens_q, cache_seqlens, page_table, slot_mapping, batch: int,
                          total_tokens: int, max_q_len: int, workspace, stream=None) -> Meta:
    meta = Meta()
    st = load().attn_prepare_metadata(
        ctypes.byref(cfg), _ptr(cu_seqlens_q), _ptr(cache_seqlens), _ptr(page_table), int(page_table.stride(0)),
        _ptr(slot_mapping), int(batch), int(total_tokens), int(max_q_len), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream(stream), ctypes.byref(meta))
    _check(st, "attn_prepare_metadata")
    meta._sizes = _batch_sizes(cfg, total_tokens, cu_seqlens_q.get_device())
    return meta


def attn_prepare_metadata_static(cfg: Config, cu_seqlens_q, cache_seqlens, page_table, slot_mapping, batch: int,
                                 total_tokens: int, max_q_len: int, stream=None) -> Meta:
    """attn_prepare_metadata with the plan in the library's built-in scratch area (no workspace)."""
    meta = Meta()
    st = load().attn_prepare_metadata_static(
        ctypes.byref(cfg), _ptr(cu_seqlens_q), _ptr(cache_seqlens), _ptr(page_table), int(page_table.stride(0)),
        _ptr(slot_mapping), int(batch), int(total_tokens), int(max_q_len), _stream(stream), ctypes.byref(meta))
    _check(st, "attn_prepare_metadata_static")
    meta._sizes = _batch_sizes(cfg, total_tokens, cu_seqlens_q.get_device())
    return meta


def attn_forward(meta: Meta, q, k, v, k_pool, v_pool, out, lse=None, stream=None) -> None:
    st = load().attn_forward(ctypes.byref(meta), _ptr(q), _ptr(k), _ptr(v), _ptr(k_pool), _ptr(v_pool), _ptr(out),
                             _ptr(lse), _stream(stream))
    _check(st, "attn_forward")


def attn_store_kvcache(meta: Meta, k, v, k_pool, v_pool, stream=None) -> None:
    st = load().attn_store_kvcache(ctypes.byref(meta), _ptr(k), _ptr(v), _ptr(k_pool), _ptr(v_pool),
                                   _stream(stream))
    _check(st, "attn_store_kvcache")


def attn_forward_fp8kv(meta: Meta, q, k, v, k_pool, v_pool, k_scale, v_scale, out, lse=None, stream=None) -> None:
    """attn_forward over E4M3 pools (uint8 tensors) with per-kv-head fp32 scales (device tensors)."""
    st = load().attn_forward_fp8kv(ctypes.byref(meta), _ptr(q), _ptr(k), _ptr(v), _ptr(k_pool), _ptr(v_pool),
                                   _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "attn_forward_fp8kv")


def attn_store_kvcache_fp8kv(meta: Meta, k, v, k_pool, v_pool, k_scale, v_scale, stream=None) -> None:
    st = load().attn_store_kvcache_fp8kv(ctypes.byref(meta), _ptr(k), _ptr(v), _ptr(k_pool), _ptr(v_pool),
                                         _ptr(k_scale), _ptr(v_scale), _stream(stream))
    _check(st, "attn_store_kvcache_fp8kv")


def attn_forward_mxfp4kv(meta: Meta, q, k, v, k_pool, v_pool, out, lse=None, stream=None) -> None:
    """attn_forward over MXFP4 pools (uint8 [slots, mxfp4_row_bytes] tensors)."""
    b = meta.batch or meta.of_batch()
    if b is not None and (b.lacks(q, b.nq, b.bf16) or b.lacks(k, b.nkv, b.bf16) or b.lacks(v, b.nkv, b.bf16)
                          or b.lacks(out, b.nq, b.bf16) or b.lacks(lse, b.nlse, b.f32)
                          or b.lacks_pools(k_pool, v_pool)):
        raise b.refusal("attn_forward_mxfp4kv")
    s = _stream_on(b, stream, "attn_forward_mxfp4kv")
    st = (_lib or load()).attn_forward_mxfp4kv(meta, _ptr(q), _ptr(k), _ptr(v), _ptr(k_pool), _ptr(v_pool), _ptr(out),
                                               _ptr(lse), s)
    if st:
        _check(st, "attn_forward_mxfp4kv")


def attn_store_kvcache_mxfp4kv(meta: Meta, k, v, k_pool, v_pool, stream=None) -> None:
    b = meta.batch or meta.of_batch()
    if b is not None and (b.lacks(k, b.nkv, b.bf16) or b.lacks(v, b.nkv, b.bf16) or b.lacks_pools(k_pool, v_pool)):
        raise b.refusal("attn_store_kvcache_mxfp4kv")
    s = _stream_on(b, stream, "attn_store_kvcache_mxfp4kv")
    st = (_lib or load()).attn_store_kvcache_mxfp4kv(meta, _ptr(k), _ptr(v), _ptr(k_pool), _ptr(v_pool), s)
    if st:
        _check(st, "attn_store_kvcache_mxfp4kv")


def attn_load_kvcache_mxfp4kv(meta: Meta, k_pool, v_pool, k, v, stream=None) -> None:
    """The values the pools hold at the batch's new tokens' slots, into bf16 k / v [T, Hkv, D]."""
    b = meta.batch or meta.of_batch()
    if b is not None and (b.lacks(k, b.nkv, b.bf16) or b.lacks(v, b.nkv, b.bf16) or b.lacks_pools(k_pool, v_pool)):
        raise b.refusal("attn_load_kvcache_mxfp4kv")
    s = _stream_on(b, stream, "attn_load_kvcache_mxfp4kv")
    st = (_lib or load()).attn_load_kvcache_mxfp4kv(meta, _ptr(k_pool), _ptr(v_pool), _ptr(k), _ptr(v), s)
    if st:
        _check(st, "attn_load_kvcache_mxfp4kv")


def mxfp4_row_bytes(num_kv_heads: int, head_dim: int) -> int:
    """Bytes of one slot's row in an MXFP4 pool (pools: uint8 [slots, row_bytes])."""
    n = int(load().attn_mxfp4_row_bytes(int(num_kv_heads), int(head_dim)))
    if n == 0:
        raise PvaError(2, "attn_mxfp4_row_bytes")
    return n


def _token_stride(x, name: str, batch, is_q: bool, device: int) -> int:
    """Elements between x's tokens, checked against the batch it is of (0 without x)."""
    import torch

    if x is None:
        return 0
    T, heads, dim = x.shape
    st, sh, sd = x.stride()
    if sd != 1 or (sh != dim and heads > 1):
        raise ValueError(f"{name} [T, heads, D] has contiguous heads (only the token stride is free)")
    if x.dtype is not torch.bfloat16 or x.get_device() != device:
        raise ValueError(f"{name} is a bf16 tensor on the device of cos_sin, the gains or the batch")
    if batch is not None and (T < batch.tokens or dim != batch.head_dim
                              or heads != (batch.q_heads if is_q else batch.kv_heads)):
        raise batch.refusal(f"{name} {tuple(x.shape)}")
    return st if T > 1 else heads * dim


class Rope:
    """A rotary position rotation: fp32 cos_sin [max_positions, rot_dim] on the device (a position's
    cosines, then its sines; see rope_table), how elements pair, and positions (int32 [T] on the
    device) when they are not the tokens' indices in their requests."""

    def __init__(self, cos_sin, rot_dim: int | None = None, interleaved: bool = False, positions=None):
        import torch

        if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin is a contiguous fp32 [max_positions, rot_dim] tensor")
        if rot_dim is not None and rot_dim != cos_sin.shape[1]:
            raise ValueError(f"cos_sin has {cos_sin.shape[1]} columns, rot_dim is {rot_dim}")
        self.cos_sin = cos_sin
        self.device = cos_sin.get_device()
        self.max_positions, self.rot_dim = (int(n) for n in cos_sin.shape)
        self.interleaved = bool(interleaved)
        self.set_positions(positions)

    def set_positions(self, positions) -> None:
        """Explicit positions of the batch's tokens, or None."""
        import torch

        if positions is not None and (positions.dtype != torch.int32 or not positions.is_contiguous()):
            raise ValueError("positions is a contiguous int32 tensor")
        if positions is not None and positions.get_device() != self.device:
            raise ValueError("positions lie on another device than cos_sin")
        self.positions = positions

    def args(self, q, k, v, batch: Batch | None = None) -> RopeArgs:
        """The C structure for q (or None), k and v [T, heads, D], checked against the batch they are of
        (k and v may be None too, where the call takes them so)."""
        pos, tokens = self.positions, k if k is not None else q
        if pos is not None and pos.numel() != tokens.shape[0]:
            raise ValueError(f"{pos.numel()} positions for {tokens.shape[0]} tokens")
        if batch is not None and self.device != batch.device:
            raise ValueError("cos_sin is not on the batch's device")
        return RopeArgs(self.cos_sin.data_ptr(), None if pos is None else pos.data_ptr(),
                        _token_stride(q, "q", batch, True, self.device), _token_stride(k, "k", batch, False, self.device),
                        _token_stride(v, "v", batch, False, self.device),
                        self.max_positions, self.rot_dim, self.interleaved, 0)


def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """cos_sin of angles p * base^(-2i / rot_dim), formed in 64 bits (a far position's angle has lost
    its fraction in 32), rounded once to fp32 [max_positions, rot_dim]."""
    import torch

    inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    ang = torch.arange(max_positions, dtype=torch.float64)[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), 1).to(torch.float32).to(device)


class QKNorm:
    """The norm of each head of q and k before the rotation: x / sqrt(mean(x^2) + eps) * gain, with fp32 gains
    [D] on the device for every head of q and of k (None: ones)."""

    def __init__(self, q_gain=None, k_gain=None, eps: float = 1e-6):
        import torch

        for g in (q_gain, k_gain):
            if g is not None and (g.dtype != torch.float32 or g.dim() != 1 or not g.is_contiguous()):
                raise ValueError("a gain is a contiguous fp32 [D] tensor")
        given = [g for g in (q_gain, k_gain) if g is not None]
        if len({g.get_device() for g in given}) > 1:
            raise ValueError("the gains lie on different devices")
        if not 0.0 <= eps < float("inf"):
            raise ValueError("eps is finite and not negative")
        self.q_gain, self.k_gain, self.eps = q_gain, k_gain, float(eps)
        self.device = given[0].get_device() if given else None
        self.head_dims = {int(g.numel()) for g in given}

    def args(self, head_dim: int, device: int) -> QKNormArgs:
        if self.device is not None and self.device != device:
            raise ValueError("the gains are on another device than q and k")
        if self.head_dims - {head_dim}:
            raise ValueError(f"gains of {sorted(self.head_dims)} elements for heads of {head_dim}")
        return QKNormArgs(_ptr(self.q_gain), _ptr(self.k_gain), self.eps, 0)


def _rotation(rope: Rope | None, norm: QKNorm | None, q, k, v, batch: Batch | None):
    """The C structures of a rotation (its strides alone without one) and a norm (or None)."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("neither q nor k")
    if rope is None and norm is None:
        raise ValueError("neither a rotation nor a norm")
    device = some.get_device() if batch is None else batch.device
    if rope is not None:
        args = rope.args(q, k, v, batch)
    else:
        args = RopeArgs(None, None, _token_stride(q, "q", batch, True, device), _token_stride(k, "k", batch, False, device),
                        _token_stride(v, "v", batch, False, device), 0, 0, 0, 0)
    return args, None if norm is None else norm.args(some.shape[2], device)


def attn_append_norm_rope(meta: Meta, norm: QKNorm, rope: Rope | None, q, k, v, q_out, k_pool, v_pool, k_scale=None,
                          v_scale=None, stream=None) -> None:
    """attn_append_rope of normed q and k; rope None: the norm alone."""
    b = meta.batch or meta.of_batch()
    rargs, nargs = _rotation(rope, norm, q, k, v, b)
    if b is not None and (b.lacks(q_out, b.nq, b.bf16) or b.lacks_pools(k_pool, v_pool) or b.scaled
                          and (b.lacks(k_scale, b.kv_heads, b.f32) or b.lacks(v_scale, b.kv_heads, b.f32))):
        raise b.refusal("attn_append_norm_rope")
    s = _stream_on(b, stream, "attn_append_norm_rope")
    st = (_lib or load()).attn_append_norm_rope(meta, nargs, rargs, _ptr(q), _ptr(k), _ptr(v), _ptr(q_out), _ptr(k_pool),
                                                _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), s)
    if st:
        _check(st, "attn_append_norm_rope")


def attn_forward_norm_rope(meta: Meta, norm: QKNorm, rope: Rope | None, q, k, v, q_rot, k_pool, v_pool, out, lse=None,
                           k_scale=None, v_scale=None, stream=None) -> None:
    """attn_append_norm_rope, then the attention of the normed and rotated q."""
    b = meta.batch or meta.of_batch()
    rargs, nargs = _rotation(rope, norm, q, k, v, b)
    if b is not None and (b.lacks(q_rot, b.nq, b.bf16) or b.lacks(out, b.nq, b.bf16) or b.lacks(lse, b.nlse, b.f32)
                          or b.lacks_pools(k_pool, v_pool) or b.scaled
                          and (b.lacks(k_scale, b.kv_heads, b.f32) or b.lacks(v_scale, b.kv_heads, b.f32))):
        raise b.refusal("attn_forward_norm_rope")
    s = _stream_on(b, stream, "attn_forward_norm_rope")
    st = (_lib or load()).attn_forward_norm_rope(meta, nargs, rargs, _ptr(q), _ptr(k), _ptr(v), _ptr(q_rot), _ptr(k_pool),
                                                 _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse), s)
    if st:
        _check(st, "attn_forward_norm_rope")


def attn_norm_rope(meta: Meta, norm: QKNorm | None, rope: Rope | None, q, k, q_out, k_out, stream=None) -> None:
    """q normed and rotated into q_out, k into k_out (metas of either kind; q or k may be None)."""
    b = meta.batch or meta.of_batch()
    rargs, nargs = _rotation(rope, norm, q, k, None, b)
    if b is not None and (b.lacks(q_out, b.nq, b.bf16) or b.lacks(k_out, b.nkv, b.bf16)):
        raise b.refusal("attn_norm_rope")
    s = _stream_on(b, stream, "attn_norm_rope")
    st = (_lib or load()).attn_norm_rope(meta, nargs, rargs, _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), s)
    if st:
        _check(st, "attn_norm_rope")


def make_linear_config(num_qo_heads, num_kv_heads, head_dim, num_states, max_batch, max_tokens,
                       scale: float = 0.0) -> LinearConfig:
    return LinearConfig(num_qo_heads, num_kv_heads, head_dim, scale, num_states, max_batch, max_tokens)


def attn_linear_workspace_size(cfg: LinearConfig) -> int:
    return int(load().attn_linear_workspace_size(ctypes.byref(cfg)))


def attn_linear_prepare(cfg: LinearConfig, cu_seqlens_q, cache_seqlens, state_in, state_out, batch: int, total_tokens: int,
                        max_q_len: int, workspace, stream=None) -> Meta:
    import torch

    device = cu_seqlens_q.get_device()
    for name, x, n in (("cu_seqlens_q", cu_seqlens_q, batch + 1), ("cache_seqlens", cache_seqlens, batch),
                       ("state_in", state_in, batch), ("state_out", state_out, batch)):
        if x is not None and (x.dtype != torch.int32 or x.numel() < n or not x.is_contiguous() or x.get_device() != device):
            raise PvaError(1, f"attn_linear_prepare ({name} is a contiguous int32 tensor of {n} on cu_seqlens_q's device)")
    if workspace.get_device() != device:
        raise PvaError(1, "attn_linear_prepare (the workspace is on another device than cu_seqlens_q)")
    meta = Meta()
    meta._sizes = _linear_sizes(cfg, total_tokens, device)
    s = _stream_on(meta.of_batch(), stream, "attn_linear_prepare")
    st = load().attn_linear_prepare(
        ctypes.byref(cfg), _ptr(cu_seqlens_q), _ptr(cache_seqlens), _ptr(state_in), _ptr(state_out), int(batch),
        int(total_tokens), int(max_q_len), _ptr(workspace), int(workspace.numel() * workspace.element_size()), s,
        ctypes.byref(meta))
    _check(st, "attn_linear_prepare")
    return meta


def _linear_args(b: Batch | None, log_decay, states, ld, where: str) -> LinearArgs:
    """The C structure, checked against the batch; ld: token strides of q, k and v."""
    if b is not None:
        f32 = b.f32
        if b.pool_bytes > states.nbytes or states.dtype is not f32 or states.get_device() != b.device or not states.is_contiguous():
            raise b.refusal(where + " states")
        bad = log_decay.dtype is not f32 or log_decay.get_device() != b.device or log_decay.shape[-1] != b.kv_heads
        if log_decay.dim() == 1:
            bad = bad or not log_decay.is_contiguous()
        else:
            bad = bad or log_decay.dim() != 2 or log_decay.shape[0] < b.tokens or log_decay.stride(1) != 1 and b.kv_heads > 1
        if bad:
            raise b.refusal(where + " log_decay")
    step = 0 if log_decay.dim() == 1 else (log_decay.stride(0) if log_decay.shape[0] > 1 else log_decay.shape[1])
    return LinearArgs(log_decay.data_ptr(), step, *ld, states.data_ptr())


def attn_linear_forward(meta: Meta, q, k, v, log_decay, states, out, stream=None) -> None:
    """Linear attention of the batch's new tokens: log_decay fp32 [Hkv] or [T, Hkv], states fp32
    [num_states, Hkv, D, D] (updated in place); q, k, v may be strided by token."""
    b = meta.batch or meta.of_batch()
    device = q.get_device() if b is None else b.device
    ld = (_token_stride(q, "q", b, True, device), _token_stride(k, "k", b, False, device),
          _token_stride(v, "v", b, False, device))
    args = _linear_args(b, log_decay, states, ld, "attn_linear_forward")
    if b is not None and b.lacks(out, b.nq, b.bf16):
        raise b.refusal("attn_linear_forward")
    s = _stream_on(b, stream, "attn_linear_forward")
    st = (_lib or load()).attn_linear_forward(meta, args, _ptr(q), _ptr(k), _ptr(v), _ptr(out), s)
    if st:
        _check(st, "attn_linear_forward")


def attn_linear_forward_norm_rope(meta: Meta, norm: QKNorm | None, rope: Rope | None, q, k, v, q_rot, k_rot, log_decay,
                                  states, out, stream=None) -> None:
    """attn_norm_rope of q and k into q_rot and k_rot, then attn_linear_forward of those.  A token whose position lies
    outside the table is reported, and its q and k count as 0."""
    b = meta.batch or meta.of_batch()
    rargs, nargs = _rotation(rope, norm, q, k, v, b)
    args = _linear_args(b, log_decay, states, (0, 0, 0), "attn_linear_forward_norm_rope")
    if b is not None and (b.lacks(q_rot, b.nq, b.bf16) or b.lacks(k_rot, b.nkv, b.bf16) or b.lacks(out, b.nq, b.bf16)):
        raise b.refusal("attn_linear_forward_norm_rope")
    s = _stream_on(b, stream, "attn_linear_forward_norm_rope")
    st = (_lib or load()).attn_linear_forward_norm_rope(meta, args, nargs, rargs, _ptr(q), _ptr(k), _ptr(v), _ptr(q_rot),
                                                        _ptr(k_rot), _ptr(out), s)
    if st:
        _check(st, "attn_linear_forward_norm_rope")


def attn_append_rope(meta: Meta, rope: Rope, q, k, v, q_out, k_pool, v_pool, k_scale=None, v_scale=None,
                     stream=None) -> None:
    """q rotated into q_out, k rotated and stored, v stored; q, k, v may be strided by token."""
    b = meta.batch or meta.of_batch()
    args = rope.args(q, k, v, b)
    if b is not None and (b.lacks(q_out, b.nq, b.bf16) or b.lacks_pools(k_pool, v_pool) or b.scaled
                          and (b.lacks(k_scale, b.kv_heads, b.f32) or b.lacks(v_scale, b.kv_heads, b.f32))):
        raise b.refusal("attn_append_rope")
    s = _stream_on(b, stream, "attn_append_rope")
    st = (_lib or load()).attn_append_rope(meta, args, _ptr(q), _ptr(k), _ptr(v), _ptr(q_out), _ptr(k_pool),
                                           _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), s)
    if st:
        _check(st, "attn_append_rope")


def attn_forward_rope(meta: Meta, rope: Rope, q, k, v, q_rot, k_pool, v_pool, out, lse=None, k_scale=None,
                      v_scale=None, stream=None) -> None:
    """attn_append_rope, then the attention of the rotated q."""
    b = meta.batch or meta.of_batch()
    args = rope.args(q, k, v, b)
    if b is not None and (b.lacks(q_rot, b.nq, b.bf16) or b.lacks(out, b.nq, b.bf16) or b.lacks(lse, b.nlse, b.f32)
                          or b.lacks_pools(k_pool, v_pool) or b.scaled
                          and (b.lacks(k_scale, b.kv_heads, b.f32) or b.lacks(v_scale, b.kv_heads, b.f32))):
        raise b.refusal("attn_forward_rope")
    s = _stream_on(b, stream, "attn_forward_rope")
    st = (_lib or load()).attn_forward_rope(meta, args, _ptr(q), _ptr(k), _ptr(v), _ptr(q_rot), _ptr(k_pool),
                                            _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse), s)
    if st:
        _check(st, "attn_forward_rope")


def attn_get_device_status(meta: Meta) -> int:
    """Synchronises; returns the device error word (0 = clean)."""
    bits = ctypes.c_uint32(0)
    st = load().attn_get_device_status(ctypes.byref(meta), ctypes.byref(bits))
    if st not in (PVA_OK, 5):
        _check(st, "attn_get_device_status")
    return int(bits.value)


def attn_debug_plan_counts(meta: Meta) -> dict:
    arr = (ctypes.c_int64 * 9)()
    n = load().attn_debug_plan_counts(ctypes.byref(meta), arr, 9)
    keys = ("dec_units", "dec_groups", "pre_tiles", "casc_groups", "casc_tiles", "split_chunk", "partial_slots",
            "kernels_per_forward", "casc_levels")
    return {keys[i]: int(arr[i]) for i in range(n)}


def attn_debug_set_wait_limit(meta: Meta, limit_ns: int) -> None:
    """Tests only: the forward kernels' wait limit for this meta (ns; 0 = give up at once,
    negative = the default 2 s).  Synchronises; the next prepare restores the default."""
    _check(load().attn_debug_set_wait_limit(ctypes.byref(meta), int(limit_ns)), "attn_debug_set_wait_limit")


def attn_set_timing_events(meta: Meta, events) -> None:
    """events: five torch.cuda.Event(enable_timing=True) already recorded once, or None to turn off."""
    if not events:
        _check(load().attn_set_timing_events(ctypes.byref(meta), None, 0), "attn_set_timing_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(load().attn_set_timing_events(ctypes.byref(meta), arr, len(events)), "attn_set_timing_events")


def deverr_names(bits: int) -> list[str]:
    return [name for b, name in DEVERR.items() if bits & b]


def ragged_layout(cu_seqlens_q, cu_seqlens_kv, device=None):
    """Page table and slot mapping that make contiguous (ragged) K/V an ordinary batch.

    With K/V given as [total_kv, Hkv, D] tensors whose rows cu_seqlens_kv[i] ..
    cu_seqlens_kv[i+1]-1 are request i's keys (its cached part, if any, followed by its
    new tokens), a config with page_size 1 and num_pages >= total_kv, and
    page_table[i][j] = cu_seqlens_kv[i] + j address them in place: pass k / v themselves
    as the pools, kv lengths cu_seqlens_kv[i+1] - cu_seqlens_kv[i] as cache_seqlens, and
    this slot mapping (-1 for every new token: nothing is stored, the keys already sit
    where the table points).  Returns (page_table int32 [B, max_kv], slot_mapping int64
    [total_q]) on ``device``.  Host-side arithmetic, once per batch.
    """
    import torch

    cu = torch.as_tensor(cu_seqlens_kv, dtype=torch.int64).cpu()
    lens = cu[1:] - cu[:-1]
    B = int(lens.numel())
    width = max(int(lens.max()) if B else 1, 1)
    j = torch.arange(width, dtype=torch.int64)
    table = torch.where(j[None, :] < lens[:, None], cu[:-1, None] + j[None, :], torch.zeros(1, dtype=torch.int64))
    total_q = int(torch.as_tensor(cu_seqlens_q)[-1])
    dev = device if device is not None else "cpu"
    return table.to(torch.int32).to(dev), torch.full((total_q,), -1, dtype=torch.int64, device=dev)


def _empty(shape, like, stream, dtype=None):
    """A tensor (bf16 unless said) on like's device, of the stream that writes it (so that its memory,
    once let go, is not given to another stream's work while that one still runs)."""
    import torch

    dtype, dev = dtype or torch.bfloat16, like.device
    handle = _stream(stream) if stream is not None else None
    if handle is None or handle == _current()[0](like.get_device()):
        return torch.empty(shape, dtype=dtype, device=dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


class PagedAttention:
    """Owns a config and a torch-allocated workspace; one prepare per batch, one forward per layer."""

    _empty = staticmethod(_empty)

    def __init__(self, num_qo_heads, num_kv_heads, head_dim, page_size, num_pages, max_batch, max_tokens,
                 max_kv_len, sm_scale: float = 0.0, enable_split_kv: bool = True, enable_cascade: bool = True,
                 min_cascade_pages: int = 8, device="cuda", kv_dtype: int = KV_BF16):
        import torch

        self.cfg = make_config(num_qo_heads, num_kv_heads, head_dim, page_size, num_pages, max_batch, max_tokens,
                               max_kv_len, sm_scale, enable_split_kv, enable_cascade, min_cascade_pages, kv_dtype)
        nbytes = attn_workspace_size(self.cfg)
        if nbytes == 0:
            raise PvaError(2, "attn_workspace_size")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.meta = None
        self._keep = None

    def prepare(self, cu_seqlens_q, cache_seqlens, page_table, total_tokens: int, slot_mapping=None,
                max_q_len: int = 0, stream=None) -> Meta:
        """Once per batch.  The index tensors are kept referenced until the next prepare."""
        batch = int(cache_seqlens.numel())
        self._keep = (cu_seqlens_q, cache_seqlens, page_table, slot_mapping)
        self.total_tokens = int(total_tokens)
        self.meta = attn_prepare_metadata(self.cfg, cu_seqlens_q, cache_seqlens, page_table, slot_mapping, batch,
                                          total_tokens, max_q_len, self.workspace, stream)
        return self.meta

    def forward(self, q, k, v, k_pool, v_pool, out=None, lse=None, stream=None, k_scale=None, v_scale=None,
                rope: Rope | None = None, q_rot=None, norm: QKNorm | None = None):
        """One layer.  With an E4M3 config the pools are uint8 and k_scale / v_scale (fp32 [Hkv],
        on the device) are required; with an MXFP4 config they are uint8 [slots, mxfp4_row_bytes].
        With ``rope``, q and k are rotated by position first (q into q_rot, a new tensor when None)
        and q, k, v may be strided by token; with ``norm`` (and ``rope`` or without) each of their
        heads is normed before."""
        if out is None:
            out = _empty(q.shape, q, stream, q.dtype)
        if norm is not None:
            if q_rot is None:
                q_rot = _empty(q.shape, q, stream)
            attn_forward_norm_rope(self.meta, norm, rope, q, k, v, q_rot, k_pool, v_pool, out, lse, k_scale, v_scale, stream)
        elif rope is not None:
            if q_rot is None:
                q_rot = _empty(q.shape, q, stream)
            attn_forward_rope(self.meta, rope, q, k, v, q_rot, k_pool, v_pool, out, lse, k_scale, v_scale, stream)
        elif self.cfg.kv_dtype == KV_E4M3:
            attn_forward_fp8kv(self.meta, q, k, v, k_pool, v_pool, k_scale, v_scale, out, lse, stream)
        elif self.cfg.kv_dtype == KV_MXFP4:
            attn_forward_mxfp4kv(self.meta, q, k, v, k_pool, v_pool, out, lse, stream)
        else:
            attn_forward(self.meta, q, k, v, k_pool, v_pool, out, lse, stream)
        return out

    def append(self, q, k, v, k_pool, v_pool, rope: Rope | None, q_out=None, k_scale=None, v_scale=None, stream=None,
               norm: QKNorm | None = None):
        """attn_append_rope of one layer, or attn_append_norm_rope with ``norm`` (then rope may be None);
        returns the rotated q (q_out, a new tensor when None; None without q)."""
        if q_out is None and q is not None:
            q_out = _empty(q.shape, q, stream)
        if norm is not None:
            attn_append_norm_rope(self.meta, norm, rope, q, k, v, q_out, k_pool, v_pool, k_scale, v_scale, stream)
        else:
            attn_append_rope(self.meta, rope, q, k, v, q_out, k_pool, v_pool, k_scale, v_scale, stream)
        return q_out

    def norm_rope(self, q, k, rope: Rope | None = None, norm: QKNorm | None = None, q_out=None, k_out=None, stream=None):
        """attn_norm_rope: (q, k) normed and rotated, into tensors of their own."""
        return _norm_rope(self.meta, q, k, rope, norm, q_out, k_out, stream)

    def store(self, k, v, k_pool, v_pool, k_scale=None, v_scale=None, stream=None) -> None:
        """store_kvcache of one layer, into pools of the config's type."""
        if self.cfg.kv_dtype == KV_E4M3:
            attn_store_kvcache_fp8kv(self.meta, k, v, k_pool, v_pool, k_scale, v_scale, stream)
        elif self.cfg.kv_dtype == KV_MXFP4:
            attn_store_kvcache_mxfp4kv(self.meta, k, v, k_pool, v_pool, stream)
        else:
            attn_store_kvcache(self.meta, k, v, k_pool, v_pool, stream)

    def load(self, k_pool, v_pool, k=None, v=None, stream=None):
        """What MXFP4 pools hold at the batch's new tokens' slots, as bf16 (k, v) [T, Hkv, D]."""
        shape = (self.total_tokens, self.cfg.num_kv_heads, self.cfg.head_dim)
        k = _empty(shape, k_pool, stream) if k is None else k
        v = _empty(shape, k_pool, stream) if v is None else v
        attn_load_kvcache_mxfp4kv(self.meta, k_pool, v_pool, k, v, stream)
        return k, v


def _norm_rope(meta: Meta, q, k, rope, norm, q_out, k_out, stream):
    if q_out is None and q is not None:
        q_out = _empty(q.shape, q, stream)
    if k_out is None and k is not None:
        k_out = _empty(k.shape, k, stream)
    attn_norm_rope(meta, norm, rope, q, k, q_out, k_out, stream)
    return q_out, k_out


class LinearAttention:
    """Linear attention layers of a model: owns a config and a torch-allocated workspace; one prepare per batch,
    one forward per layer.  Each layer has its own pool of states, fp32 [num_states, Hkv, D, D]."""

    def __init__(self, num_qo_heads, num_kv_heads, head_dim, num_states, max_batch, max_tokens, scale: float = 0.0,
                 device="cuda"):
        import torch

        self.cfg = make_linear_config(num_qo_heads, num_kv_heads, head_dim, num_states, max_batch, max_tokens, scale)
        nbytes = attn_linear_workspace_size(self.cfg)
        if nbytes == 0:
            raise PvaError(2, "attn_linear_workspace_size")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.meta = None
        self._keep = None

    def prepare(self, cu_seqlens_q, cache_seqlens, total_tokens: int, state_in=None, state_out=None, max_q_len: int = 0,
                stream=None) -> Meta:
        """Once per batch.  state_in / state_out (int32 [batch]): the slots that requests go on from and leave their
        new state in (the same tensor: in place; -1: from zero, not kept; None: all of them).  The index tensors
        are kept referenced until the next prepare."""
        self._keep = (cu_seqlens_q, cache_seqlens, state_in, state_out)
        self.total_tokens = int(total_tokens)
        self.meta = attn_linear_prepare(self.cfg, cu_seqlens_q, cache_seqlens, state_in, state_out,
                                        int(cache_seqlens.numel()), total_tokens, max_q_len, self.workspace, stream)
        return self.meta

    def forward(self, q, k, v, log_decay, states, out=None, rope: Rope | None = None, norm: QKNorm | None = None,
                q_rot=None, k_rot=None, stream=None):
        """One layer: out [T, Hq, D] and the states' update.  With ``rope`` or ``norm``, q and k are normed and
        rotated first (into q_rot and k_rot, new tensors when None)."""
        if out is None:
            out = _empty(q.shape, q, stream)
        if rope is not None or norm is not None:
            if q_rot is None:
                q_rot = _empty(q.shape, q, stream)
            if k_rot is None:
                k_rot = _empty(k.shape, k, stream)
            attn_linear_forward_norm_rope(self.meta, norm, rope, q, k, v, q_rot, k_rot, log_decay, states, out, stream)
        else:
            attn_linear_forward(self.meta, q, k, v, log_decay, states, out, stream)
        return out

    def norm_rope(self, q, k, rope: Rope | None = None, norm: QKNorm | None = None, q_out=None, k_out=None, stream=None):
        """attn_norm_rope: (q, k) normed and rotated, into tensors of their own."""
        return _norm_rope(self.meta, q, k, rope, norm, q_out, k_out, stream)

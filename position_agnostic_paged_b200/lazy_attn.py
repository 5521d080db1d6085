"""Thin ctypes binding of liblazy_attn.so (include/lazy_attn.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, passes their data pointers and the current CUDA stream to the
C entry point of the same name, and raises LazyAttnError on a non-zero return
code.  All computation happens in the library's CUDA kernels; there is no CPU
fallback, and importing this module fails loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblazy_attn.so")

LAZY_OK, LAZY_EINVAL, LAZY_ERANGE, LAZY_ESHAPE, LAZY_EWORKSPACE, LAZY_ECUDA = 0, -1, -2, -3, -4, -5
DSTATUS_BAD_BLOCK, DSTATUS_BAD_SLOT, DSTATUS_BAD_ALIGN, DSTATUS_BAD_TABLE, DSTATUS_TIMEOUT = 1, 2, 4, 8, 16

EXPORTED = [
    "lazy_version", "lazy_strerror", "lazy_pack_words", "lazy_kv_write",
    "lazy_decode_workspace_bytes", "lazy_decode_attn",
    "lazy_prefill_workspace_bytes", "lazy_prefill_attn",
    "lazy_materialize_k", "lazy_plain_decode_attn", "lazy_plain_prefill_attn",
    "lazy_debug_decode_table", "lazy_decode_attn_noalloc", "lazy_decode_noalloc_capacity",
    "lazy_cache_create", "lazy_cache_destroy", "lazy_cache_access", "lazy_cache_contains", "lazy_cache_stats",
    "lazy_mixed_attn", "lazy_rope_theta", "lazy_rope_theta_llama31", "lazy_alibi_slopes",
    "lazy_debug_bounded_wait",
    "lazy_kv_write_q8_workspace_bytes", "lazy_kv_write_q8", "lazy_decode_q8_workspace_bytes", "lazy_decode_attn_q8",
    "lazy_prefill_q8_workspace_bytes", "lazy_prefill_attn_q8", "lazy_decode_mass_workspace_bytes",
    "lazy_decode_attn_mass", "lazy_evict_blocks",
]


class LazyAttnError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code}: {strerror(code)}")
        self.code = code


class LazyAttnCfg(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("block_size", ctypes.c_int), ("rope_base", ctypes.c_float), ("softmax_scale", ctypes.c_float),
                ("rope_theta", ctypes.POINTER(ctypes.c_double)),
                ("alibi_slopes", ctypes.POINTER(ctypes.c_double))]


@dataclass(frozen=True)
class Cfg:
    """rope_theta: optional head_dim/2 RoPE frequencies (e.g. rope.llama31_theta()) in place of
    rope_base^(-2i/head_dim).  alibi_slopes: optional num_q_heads ALiBi slopes (e.g.
    rope.alibi_slopes(num_q_heads)) in place of RoPE: keys are stored as given and each score gets
    -slope_h * (query position - key position)."""
    num_q_heads: int
    num_kv_heads: int
    rope_base: float = 500000.0
    head_dim: int = 128
    block_size: int = 16
    softmax_scale: float = 0.0
    rope_theta: tuple | None = None
    alibi_slopes: tuple | None = None

    def c(self) -> LazyAttnCfg:
        st = LazyAttnCfg(self.num_q_heads, self.num_kv_heads, self.head_dim, self.block_size,
                         float(self.rope_base), float(self.softmax_scale), None, None)
        if self.alibi_slopes is not None:
            if len(self.alibi_slopes) != self.num_q_heads:
                raise ValueError("alibi_slopes needs one slope per query head")
            sl = (ctypes.c_double * len(self.alibi_slopes))(*[float(x) for x in self.alibi_slopes])
            st._alibi_keepalive = sl
            st.alibi_slopes = ctypes.cast(sl, ctypes.POINTER(ctypes.c_double))
        if self.rope_theta is not None:
            if len(self.rope_theta) < 64 and self.head_dim == 128:   # (other head sizes are refused before it is read)
                raise ValueError("rope_theta needs head_dim / 2 = 64 frequencies")
            arr = (ctypes.c_double * len(self.rope_theta))(*[float(x) for x in self.rope_theta])
            st._theta_keepalive = arr
            st.rope_theta = ctypes.cast(arr, ctypes.POINTER(ctypes.c_double))
        return st

    def _shared_c(self) -> LazyAttnCfg:
        """c(), made once where no field can change; to be read only."""
        if type(self.rope_theta) not in (tuple, type(None)) or type(self.alibi_slopes) not in (tuple, type(None)):
            return self.c()
        st = self.__dict__.get("_c")
        if st is None:
            st = self.c()
            object.__setattr__(self, "_c", st)
        return st

    def __getstate__(self):
        """Without the C structure: its pointers belong to this object."""
        return {k: v for k, v in self.__dict__.items() if k != "_c"}


_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_cfgp = ctypes.POINTER(LazyAttnCfg)


class PrefillBatch(ctypes.Structure):
    """lazy_prefill_batch: the arguments of lazy_prefill_attn for one batch."""
    _fields_ = [("q_raw", _vp), ("cu_q", _vp), ("q_pos0", _vp), ("num_req", _i), ("total_q", _i), ("max_q", _i),
                ("table", _vp), ("table_indptr", _vp), ("max_words", _i), ("out", _vp), ("workspace", _vp),
                ("ws_bytes", _sz)]


class DecodeBatch(ctypes.Structure):
    """lazy_decode_batch: the arguments of lazy_decode_attn for one batch."""
    _fields_ = [("q_raw", _vp), ("q_pos", _vp), ("num_req", _i), ("table", _vp), ("table_indptr", _vp),
                ("max_words", _i), ("out", _vp), ("workspace", _vp), ("ws_bytes", _sz)]


class LazyQ8Pool(ctypes.Structure):
    """lazy_q8_pool: device pointers of an 8-bit pool."""
    _fields_ = [("k_codes", _vp), ("v_codes", _vp), ("k_scale", _vp), ("v_scale", _vp), ("blk_meta", _vp),
                ("num_blocks", _i)]


_q8p = ctypes.POINTER(LazyQ8Pool)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m position_agnostic_paged_b200.build` "
                          "(the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "lazy_version": (_i, []),
        "lazy_strerror": (ctypes.c_char_p, [_i]),
        "lazy_pack_words": (_i, [_vp, _vp, _i64, _vp]),
        "lazy_kv_write": (_i, [_cfgp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp]),
        "lazy_decode_workspace_bytes": (_sz, [_cfgp, _i, _i]),
        "lazy_decode_attn": (_i, [_cfgp, _vp, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _sz, _vp, _vp]),
        "lazy_prefill_workspace_bytes": (_sz, [_cfgp, _i, _i, _i, _i]),
        "lazy_prefill_attn": (_i, [_cfgp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp,
                                   _sz, _vp, _vp]),
        "lazy_materialize_k": (_i, [_cfgp, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp]),
        "lazy_plain_decode_attn": (_i, [_cfgp, _vp, _vp, _i, _vp, _vp, _i, _vp, _vp, _i, _vp, _i, _vp, _vp, _sz,
                                        _vp, _vp]),
        "lazy_plain_prefill_attn": (_i, [_cfgp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _i, _vp, _i,
                                         _vp, _vp, _sz, _vp, _vp]),
        "lazy_debug_decode_table": (_i, [_vp, _i64, _vp, _i, _vp, _vp, _vp, _vp, _vp]),
        "lazy_decode_attn_noalloc": (_i, [_cfgp, _vp, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp]),
        "lazy_decode_noalloc_capacity": (_sz, []),
        "lazy_mixed_attn": (_i, [_cfgp, ctypes.POINTER(PrefillBatch), ctypes.POINTER(DecodeBatch), _vp, _vp, _vp, _i,
                                 _vp, _vp]),
        "lazy_rope_theta": (_i, [ctypes.c_double, _i, _vp]),
        "lazy_rope_theta_llama31": (_i, [ctypes.c_double, _i, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                         ctypes.c_double, _vp]),
        "lazy_alibi_slopes": (_i, [_i, _vp]),
        "lazy_debug_bounded_wait": (_i, [ctypes.c_uint32, _i, _vp, _vp, _vp]),
        "lazy_kv_write_q8_workspace_bytes": (_sz, [_cfgp, _i, _i]),
        "lazy_kv_write_q8": (_i, [_cfgp, _vp, _vp, _i, _vp, _vp, _q8p, _vp, _sz, _vp, _vp]),
        "lazy_decode_q8_workspace_bytes": (_sz, [_cfgp, _i, _i, _i]),
        "lazy_decode_attn_q8": (_i, [_cfgp, _vp, _vp, _i, _vp, _vp, _i, _q8p, _vp, _vp, _vp, _sz, _vp, _vp]),
        "lazy_prefill_q8_workspace_bytes": (_sz, [_cfgp, _i, _i, _i, _i, _i]),
        "lazy_prefill_attn_q8": (_i, [_cfgp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _q8p, _vp, _vp, _sz, _vp, _vp]),
        "lazy_decode_mass_workspace_bytes": (_sz, [_cfgp, _i, _i]),
        "lazy_decode_attn_mass": (_i, [_cfgp, _vp, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp, _sz, _vp,
                                       _vp]),
        "lazy_evict_blocks": (_i, [_vp, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
        "lazy_cache_create": (_vp, [_i64]),
        "lazy_cache_destroy": (None, [_vp]),
        "lazy_cache_access": (_i, [_vp, ctypes.c_uint64, ctypes.c_int32, _vp]),
        "lazy_cache_contains": (_i, [_vp, ctypes.c_uint64]),
        "lazy_cache_stats": (_i, [_vp, _vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


def version() -> int:
    return int(_lib.lazy_version())


def strerror(code: int) -> str:
    return _lib.lazy_strerror(int(code)).decode()


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise LazyAttnError(fn, rc)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return int(t.data_ptr())


class _LazyTorch:
    """What the calls need of torch, imported by the first that does: the codec, the tables and the block cache
    work without it."""

    def __getattr__(self, name):
        import torch
        self.cuda = torch.cuda
        # the current stream's handle without making a Stream object (0.2 us against 3 us), where torch has it
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.bf16, self.f32, self.i32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
        self.word, self.code = (torch.int32, torch.uint32), (torch.uint8, torch.float8_e4m3fn)
        self.torch = torch
        if name not in self.__dict__:
            raise AttributeError(name)
        return self.__dict__[name]


_t = _LazyTorch()


def _stream(stream) -> int | None:
    if stream is None:
        if _t.raw_stream is not None:
            return int(_t.raw_stream(_t.cuda.current_device())) or None
        return int(_t.cuda.current_stream().cuda_stream) or None
    return int(getattr(stream, "cuda_stream", stream)) or None


def pack_words(block: np.ndarray, offset: np.ndarray) -> np.ndarray:
    """Host codec: (block, offset) int32 arrays -> uint32 table words (raises on overflow)."""
    block = np.ascontiguousarray(block, np.int32)
    offset = np.ascontiguousarray(offset, np.int32)
    out = np.empty(block.size, np.uint32)
    _check("lazy_pack_words", _lib.lazy_pack_words(block.ctypes.data, offset.ctypes.data, block.size,
                                                   out.ctypes.data))
    return out


def rope_theta(base: float, head_dim: int) -> tuple[float, ...]:
    """lazy_rope_theta: theta_i = base^(-2i/head_dim)."""
    out = np.empty(max(int(head_dim) // 2, 1), np.float64)
    _check("lazy_rope_theta", _lib.lazy_rope_theta(float(base), int(head_dim), out.ctypes.data))
    return tuple(float(x) for x in out[: int(head_dim) // 2])


def rope_theta_llama31(base: float, head_dim: int, factor: float, low_freq_factor: float,
                       high_freq_factor: float, original_max_position: float) -> tuple[float, ...]:
    """lazy_rope_theta_llama31: frequencies with Llama-3.1 scaling."""
    out = np.empty(max(int(head_dim) // 2, 1), np.float64)
    _check("lazy_rope_theta_llama31", _lib.lazy_rope_theta_llama31(
        float(base), int(head_dim), float(factor), float(low_freq_factor), float(high_freq_factor),
        float(original_max_position), out.ctypes.data))
    return tuple(float(x) for x in out[: int(head_dim) // 2])


def alibi_slopes(num_heads: int) -> tuple[float, ...]:
    """lazy_alibi_slopes: the ALiBi paper's head slopes."""
    out = np.empty(max(int(num_heads), 1), np.float64)
    _check("lazy_alibi_slopes", _lib.lazy_alibi_slopes(int(num_heads), out.ctypes.data))
    return tuple(float(x) for x in out[: int(num_heads)])


def kv_write(cfg: Cfg, k_raw, v_raw, slot, local_j, k_pool, v_pool, blk_meta, d_status=None, stream=None):
    c = cfg.c()
    _check("lazy_kv_write", _lib.lazy_kv_write(
        ctypes.byref(c), _ptr(k_raw), _ptr(v_raw), int(slot.numel()), _ptr(slot), _ptr(local_j),
        _ptr(k_pool), _ptr(v_pool), _ptr(blk_meta), int(k_pool.shape[0]), _ptr(d_status), _stream(stream)))


def decode_workspace_bytes(cfg: Cfg, num_req: int, max_words: int) -> int:
    c = cfg.c()
    return int(_lib.lazy_decode_workspace_bytes(ctypes.byref(c), int(num_req), int(max_words)))


def prefill_workspace_bytes(cfg: Cfg, num_req: int, total_q: int, max_q: int, max_words: int) -> int:
    c = cfg.c()
    return int(_lib.lazy_prefill_workspace_bytes(ctypes.byref(c), int(num_req), int(total_q), int(max_q),
                                                 int(max_words)))


def decode_attn(cfg: Cfg, q_raw, q_pos, table, table_indptr, max_words: int, blk_meta, k_pool, v_pool, out,
                workspace, d_status=None, stream=None):
    c = cfg.c()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("lazy_decode_attn", _lib.lazy_decode_attn(
        ctypes.byref(c), _ptr(q_raw), _ptr(q_pos), int(q_pos.numel()), _ptr(table), _ptr(table_indptr),
        int(max_words), _ptr(blk_meta), _ptr(k_pool), _ptr(v_pool), int(k_pool.shape[0]), _ptr(out),
        _ptr(workspace), ws_bytes, _ptr(d_status), _stream(stream)))


def prefill_attn(cfg: Cfg, q_raw, cu_q, q_pos0, max_q: int, table, table_indptr, max_words: int, blk_meta,
                 k_pool, v_pool, out, workspace=None, d_status=None, stream=None):
    c = cfg.c()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("lazy_prefill_attn", _lib.lazy_prefill_attn(
        ctypes.byref(c), _ptr(q_raw), _ptr(cu_q), _ptr(q_pos0), int(q_pos0.numel()), int(q_raw.shape[0]),
        int(max_q), _ptr(table), _ptr(table_indptr), int(max_words), _ptr(blk_meta), _ptr(k_pool),
        _ptr(v_pool), int(k_pool.shape[0]), _ptr(out), _ptr(workspace), ws_bytes, _ptr(d_status),
        _stream(stream)))


def _nbytes(t) -> int:
    return t.numel() * t.element_size() if t is not None else 0


def mixed_attn(cfg: Cfg, prefill: dict | None, decode: dict | None, blk_meta, k_pool, v_pool, d_status=None,
               stream=None):
    """One serving step with prefill chunks and decodes (lazy_mixed_attn): the results of
    prefill_attn(**prefill) and decode_attn(**decode), both batches validated before either runs,
    then run in that order on `stream`.

    prefill: dict(q_raw, cu_q, q_pos0, max_q, table, table_indptr, max_words, out, workspace);
    decode: dict(q_raw, q_pos, table, table_indptr, max_words, out, workspace).  The two
    workspaces must be distinct."""
    c = cfg.c()
    pf = dc = None
    if prefill is not None:
        b = prefill
        pf = PrefillBatch(_ptr(b["q_raw"]), _ptr(b["cu_q"]), _ptr(b["q_pos0"]), int(b["q_pos0"].numel()),
                          int(b["q_raw"].shape[0]), int(b["max_q"]), _ptr(b["table"]), _ptr(b["table_indptr"]),
                          int(b["max_words"]), _ptr(b["out"]), _ptr(b.get("workspace")), _nbytes(b.get("workspace")))
    if decode is not None:
        b = decode
        dc = DecodeBatch(_ptr(b["q_raw"]), _ptr(b["q_pos"]), int(b["q_pos"].numel()), _ptr(b["table"]),
                         _ptr(b["table_indptr"]), int(b["max_words"]), _ptr(b["out"]), _ptr(b["workspace"]),
                         _nbytes(b["workspace"]))
    _check("lazy_mixed_attn", _lib.lazy_mixed_attn(
        ctypes.byref(c), ctypes.byref(pf) if pf is not None else None, ctypes.byref(dc) if dc is not None else None,
        _ptr(blk_meta), _ptr(k_pool), _ptr(v_pool), int(k_pool.shape[0]), _ptr(d_status), _stream(stream)))


def materialize_k(cfg: Cfg, table, blk_meta, k_pool, k_mat, d_status=None, stream=None):
    c = cfg.c()
    _check("lazy_materialize_k", _lib.lazy_materialize_k(
        ctypes.byref(c), _ptr(table), int(table.numel()), _ptr(blk_meta), _ptr(k_pool), int(k_pool.shape[0]),
        _ptr(k_mat), _ptr(d_status), _stream(stream)))


def plain_decode_attn(cfg: Cfg, q_raw, q_pos, table, table_indptr, max_words: int, blk_meta, k_mat, v_pool, out,
                      workspace, d_status=None, stream=None):
    c = cfg.c()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("lazy_plain_decode_attn", _lib.lazy_plain_decode_attn(
        ctypes.byref(c), _ptr(q_raw), _ptr(q_pos), int(q_pos.numel()), _ptr(table), _ptr(table_indptr),
        int(max_words), _ptr(blk_meta), _ptr(k_mat), int(k_mat.shape[0]), _ptr(v_pool), int(v_pool.shape[0]),
        _ptr(out), _ptr(workspace), ws_bytes, _ptr(d_status), _stream(stream)))


def plain_prefill_attn(cfg: Cfg, q_raw, cu_q, q_pos0, max_q: int, table, table_indptr, max_words: int, blk_meta,
                       k_mat, v_pool, out, workspace=None, d_status=None, stream=None):
    c = cfg.c()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("lazy_plain_prefill_attn", _lib.lazy_plain_prefill_attn(
        ctypes.byref(c), _ptr(q_raw), _ptr(cu_q), _ptr(q_pos0), int(q_pos0.numel()), int(q_raw.shape[0]),
        int(max_q), _ptr(table), _ptr(table_indptr), int(max_words), _ptr(blk_meta), _ptr(k_mat),
        int(k_mat.shape[0]), _ptr(v_pool), int(v_pool.shape[0]), _ptr(out), _ptr(workspace), ws_bytes,
        _ptr(d_status), _stream(stream)))


def debug_decode_table(table, blk_meta, num_blocks: int, out_block, out_slot, out_pos, d_status=None, stream=None):
    _check("lazy_debug_decode_table", _lib.lazy_debug_decode_table(
        _ptr(table), int(table.numel()), _ptr(blk_meta), int(num_blocks), _ptr(out_block), _ptr(out_slot),
        _ptr(out_pos), _ptr(d_status), _stream(stream)))


def debug_bounded_wait(polls: int, complete: bool, result, d_status=None, stream=None):
    """lazy_debug_bounded_wait: a bounded mbarrier wait that runs out (complete=False) or succeeds."""
    _check("lazy_debug_bounded_wait", _lib.lazy_debug_bounded_wait(
        int(polls), 1 if complete else 0, _ptr(result), _ptr(d_status), _stream(stream)))


def decode_noalloc_capacity() -> int:
    """Bytes of the library's built-in scratch array used by decode_attn_noalloc."""
    return int(_lib.lazy_decode_noalloc_capacity())


def decode_attn_noalloc(cfg: Cfg, q_raw, q_pos, table, table_indptr, max_words: int, blk_meta, k_pool, v_pool, out,
                        d_status=None, stream=None):
    """decode_attn without a workspace, for callers that cannot allocate device memory.

    The split partials live in a fixed array inside the library (see
    decode_noalloc_capacity()); calls that may overlap on the GPU must be
    serialised by the caller.  Raises LazyAttnError(LAZY_ERANGE) when the
    batch needs more scratch than the array holds.
    """
    c = cfg.c()
    _check("lazy_decode_attn_noalloc", _lib.lazy_decode_attn_noalloc(
        ctypes.byref(c), _ptr(q_raw), _ptr(q_pos), int(q_pos.numel()), _ptr(table), _ptr(table_indptr),
        int(max_words), _ptr(blk_meta), _ptr(k_pool), _ptr(v_pool), int(k_pool.shape[0]), _ptr(out),
        _ptr(d_status), _stream(stream)))


# ---- the 8-bit pool, block mass and eviction.  These calls check what the C side cannot see: types
# (two-byte and four-byte elements would be read as something else), contiguity, shapes and the device.

def _take(name: str, t, dtypes: tuple, shape: tuple | None = None):
    if t.dtype in dtypes and t.is_contiguous() and (shape is None or t.shape == shape):
        return
    raise ValueError(f"{name} must be a contiguous tensor of {' or '.join(map(str, dtypes))}"
                     + (f" with shape {shape}" if shape is not None else "")
                     + f", not {t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ', not contiguous'}")


def _take_aux(workspace, d_status):
    # (an expanded workspace has fewer bytes than elements)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    if d_status is not None and (d_status.dtype not in _t.word or d_status.numel() < 1):
        raise ValueError(f"d_status must be a tensor of {' or '.join(map(str, _t.word))} with an element, not {d_status.dtype} "
                         f"{tuple(d_status.shape)}")


def _launch(name: str, fn, ts, stream, *args):
    """fn(*args, stream) on the tensors' device, which need not be the current one."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    if dev == _t.cuda.current_device():
        _check(name, fn(*args, _stream(stream)))
        return
    with _t.cuda.device(dev):
        _check(name, fn(*args, _stream(stream)))


class Q8Pool:
    """A pool of e4m3 codes with one float32 scale per (block, KV head) (lazy_q8_pool).

    k_codes, v_codes: one-byte elements [num_blocks, Hkv, 16, 128]; k_scale, v_scale: float32
    [num_blocks, Hkv]; blk_meta: int32 [num_blocks].  The tensors stay the caller's."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, blk_meta):
        nb, hkv = int(k_codes.shape[0]), int(k_codes.shape[1])
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            _take(name, t, _t.code, (nb, hkv, 16, 128))
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _take(name, t, _t.f32, (nb, hkv))
        _take("blk_meta", blk_meta, _t.word, (nb,))
        dev = k_codes.device   # the calls look at k_codes alone
        if not v_codes.device == k_scale.device == v_scale.device == blk_meta.device == dev:
            raise ValueError("all tensors of a pool must be on one device")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale, self.blk_meta = k_codes, v_codes, k_scale, v_scale, blk_meta
        self.num_blocks, self.num_kv_heads = nb, hkv

    @classmethod
    def empty(cls, num_blocks: int, num_kv_heads: int, device="cuda") -> "Q8Pool":
        """A pool whose blocks hold no tokens."""
        torch = _t.torch
        codes = lambda: torch.zeros(num_blocks, num_kv_heads, 16, 128, dtype=torch.uint8, device=device)   # noqa: E731
        scale = lambda: torch.ones(num_blocks, num_kv_heads, dtype=torch.float32, device=device)           # noqa: E731
        return cls(codes(), codes(), scale(), scale(), torch.zeros(num_blocks, dtype=torch.int32, device=device))

    def c(self) -> LazyQ8Pool:
        return LazyQ8Pool(_ptr(self.k_codes), _ptr(self.v_codes), _ptr(self.k_scale), _ptr(self.v_scale),
                          _ptr(self.blk_meta), self.num_blocks)


def _heads(cfg: Cfg, pool: Q8Pool) -> None:
    if pool.num_kv_heads != cfg.num_kv_heads:
        raise ValueError(f"the pool has {pool.num_kv_heads} KV heads, the configuration {cfg.num_kv_heads}")


def kv_write_q8_workspace_bytes(cfg: Cfg, n_tok: int, num_blocks: int) -> int:
    c = cfg._shared_c()
    return int(_lib.lazy_kv_write_q8_workspace_bytes(ctypes.byref(c), int(n_tok), int(num_blocks)))


def kv_write_q8(cfg: Cfg, k_raw, v_raw, slot, local_j, pool: Q8Pool, workspace=None, d_status=None, stream=None):
    """New tokens into an 8-bit pool (lazy_kv_write_q8): scales, codes and metadata of the blocks they fall in."""
    c, q, n = cfg._shared_c(), pool.c(), int(slot.numel())
    _heads(cfg, pool)
    for name, t in (("k_raw", k_raw), ("v_raw", v_raw)):
        _take(name, t, _t.bf16, (n, cfg.num_kv_heads, 128))
    for name, t in (("slot", slot), ("local_j", local_j)):
        _take(name, t, _t.i32)
    if local_j.numel() != n:
        raise ValueError("slot and local_j must have one element per token")
    _take_aux(workspace, d_status)
    _launch("lazy_kv_write_q8", _lib.lazy_kv_write_q8,
            (k_raw, v_raw, slot, local_j, pool.k_codes, workspace, d_status), stream,
            ctypes.byref(c), _ptr(k_raw), _ptr(v_raw), n, _ptr(slot), _ptr(local_j), ctypes.byref(q),
            _ptr(workspace), _nbytes(workspace), _ptr(d_status))


def _decode_args(cfg, q_raw, q_pos, table, table_indptr, out, block_mass):
    n = int(q_pos.numel())
    _take("q_raw", q_raw, _t.bf16, (n, cfg.num_q_heads, 128))
    _take("out", out, _t.bf16, (n, cfg.num_q_heads, 128))
    _take("q_pos", q_pos, _t.i32)
    _take("table", table, _t.word)
    _take("table_indptr", table_indptr, _t.i32)
    if table_indptr.numel() != n + 1:
        raise ValueError("table_indptr must have one element more than q_pos")
    if block_mass is not None:
        _take("block_mass", block_mass, _t.f32)
        if block_mass.numel() != table.numel():
            raise ValueError("block_mass must have one element per table word")
    return n


def decode_q8_workspace_bytes(cfg: Cfg, num_req: int, max_words: int, with_mass: bool = False) -> int:
    c = cfg._shared_c()
    return int(_lib.lazy_decode_q8_workspace_bytes(ctypes.byref(c), int(num_req), int(max_words), 1 if with_mass else 0))


def decode_attn_q8(cfg: Cfg, q_raw, q_pos, table, table_indptr, max_words: int, pool: Q8Pool, out, workspace,
                   block_mass=None, d_status=None, stream=None):
    """One decode step over an 8-bit pool (lazy_decode_attn_q8).  block_mass: optional float32
    accumulators, one per table word, that grow by the words' attention weights."""
    c, q = cfg._shared_c(), pool.c()
    _heads(cfg, pool)
    n = _decode_args(cfg, q_raw, q_pos, table, table_indptr, out, block_mass)
    _take_aux(workspace, d_status)
    _launch("lazy_decode_attn_q8", _lib.lazy_decode_attn_q8,
            (q_raw, q_pos, table, table_indptr, pool.k_codes, out, workspace, block_mass, d_status), stream,
            ctypes.byref(c), _ptr(q_raw), _ptr(q_pos), n, _ptr(table), _ptr(table_indptr), int(max_words),
            ctypes.byref(q), _ptr(out), _ptr(block_mass), _ptr(workspace), _nbytes(workspace), _ptr(d_status))


def decode_mass_workspace_bytes(cfg: Cfg, num_req: int, max_words: int) -> int:
    c = cfg._shared_c()
    return int(_lib.lazy_decode_mass_workspace_bytes(ctypes.byref(c), int(num_req), int(max_words)))


def decode_attn_mass(cfg: Cfg, q_raw, q_pos, table, table_indptr, max_words: int, blk_meta, k_pool, v_pool, out,
                     block_mass, workspace, d_status=None, stream=None):
    """decode_attn over the bf16 pool that also adds each table word's attention weight to block_mass
    (lazy_decode_attn_mass)."""
    c = cfg._shared_c()
    n = _decode_args(cfg, q_raw, q_pos, table, table_indptr, out, block_mass)
    nb = int(k_pool.shape[0])
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
        _take(name, t, _t.bf16, (nb, cfg.num_kv_heads, 16, 128))
    _take("blk_meta", blk_meta, _t.word, (nb,))
    _take_aux(workspace, d_status)
    _launch("lazy_decode_attn_mass", _lib.lazy_decode_attn_mass,
            (q_raw, q_pos, table, table_indptr, blk_meta, k_pool, v_pool, out, block_mass, workspace, d_status), stream,
            ctypes.byref(c), _ptr(q_raw), _ptr(q_pos), n, _ptr(table), _ptr(table_indptr), int(max_words),
            _ptr(blk_meta), _ptr(k_pool), _ptr(v_pool), nb, _ptr(out), _ptr(block_mass), _ptr(workspace),
            _nbytes(workspace), _ptr(d_status))


def prefill_q8_workspace_bytes(cfg: Cfg, num_req: int, total_q: int, max_q: int, max_words: int,
                               total_words: int) -> int:
    c = cfg._shared_c()
    return int(_lib.lazy_prefill_q8_workspace_bytes(ctypes.byref(c), int(num_req), int(total_q), int(max_q),
                                                    int(max_words), int(total_words)))


def prefill_attn_q8(cfg: Cfg, q_raw, cu_q, q_pos0, max_q: int, table, table_indptr, max_words: int, pool: Q8Pool,
                    out, workspace, d_status=None, stream=None):
    """Causal prefill over an 8-bit pool (lazy_prefill_attn_q8)."""
    c, q = cfg._shared_c(), pool.c()
    _heads(cfg, pool)
    n, total_q = int(q_pos0.numel()), int(q_raw.shape[0])
    _take("q_raw", q_raw, _t.bf16, (total_q, cfg.num_q_heads, 128))
    _take("out", out, _t.bf16, (total_q, cfg.num_q_heads, 128))
    for name, t in (("cu_q", cu_q), ("q_pos0", q_pos0), ("table_indptr", table_indptr)):
        _take(name, t, _t.i32)
    _take("table", table, _t.word)
    if cu_q.numel() != n + 1 or table_indptr.numel() != n + 1:
        raise ValueError("cu_q and table_indptr must have one element more than q_pos0")
    _take_aux(workspace, d_status)
    _launch("lazy_prefill_attn_q8", _lib.lazy_prefill_attn_q8,
            (q_raw, cu_q, q_pos0, table, table_indptr, pool.k_codes, out, workspace, d_status), stream,
            ctypes.byref(c), _ptr(q_raw), _ptr(cu_q), _ptr(q_pos0), n, total_q, int(max_q), _ptr(table),
            _ptr(table_indptr), int(max_words), ctypes.byref(q), _ptr(out), _ptr(workspace), _nbytes(workspace),
            _ptr(d_status))


def evict_blocks(table, table_indptr, max_words: int, block_mass, keep, n_first: int, n_last: int, table_out,
                 indptr_out, mass_out, evicted=None, d_status=None, stream=None):
    """Shortens every request's table to the keep[r] words of largest accumulated weight
    (lazy_evict_blocks); the first n_first and last n_last words of a request go last."""
    n, words = int(keep.numel()), int(table.numel())
    for name, t in (("table", table), ("table_out", table_out), ("evicted", evicted)):
        if t is not None:
            _take(name, t, _t.word)
    for name, t in (("block_mass", block_mass), ("mass_out", mass_out)):
        _take(name, t, _t.f32)
    for name, t in (("table_indptr", table_indptr), ("indptr_out", indptr_out), ("keep", keep)):
        _take(name, t, _t.i32)
    if table_indptr.numel() != n + 1 or indptr_out.numel() < n + 1:
        raise ValueError("table_indptr and indptr_out must have one element more than keep")
    if block_mass.numel() != words:
        raise ValueError("block_mass must have one element per table word")
    if min([words] + [t.numel() for t in (table_out, mass_out, evicted) if t is not None]) < words:
        raise ValueError("table_out, mass_out and evicted need room for every table word")
    _take_aux(None, d_status)
    _launch("lazy_evict_blocks", _lib.lazy_evict_blocks,
            (table, table_indptr, block_mass, keep, table_out, indptr_out, mass_out, evicted, d_status), stream,
            _ptr(table), _ptr(table_indptr), n, int(max_words), _ptr(block_mass), _ptr(keep), int(n_first),
            int(n_last), _ptr(table_out), _ptr(indptr_out), _ptr(mass_out), _ptr(evicted), _ptr(d_status))


class BlockCache:
    """Host-side LRU cache of pool blocks (lazy_cache_*): key -> the blocks of one cached entry.

    access(key, n_blocks) returns (hit, block_ids); on a miss the blocks are freshly allocated
    (after evicting least recently used entries) and the caller writes the entry there.  An entry
    larger than the cache is counted as a miss and returns (False, None).
    """

    STAT_NAMES = ("hits", "misses", "hit_blocks", "miss_blocks", "evictions", "used_blocks", "entries",
                  "free_extents")

    def __init__(self, capacity_blocks: int):
        self._h = _lib.lazy_cache_create(int(capacity_blocks))
        if not self._h:
            raise LazyAttnError("lazy_cache_create", LAZY_EINVAL)
        self.capacity = int(capacity_blocks)
        self._buf = (ctypes.c_int32 * 1)()

    def close(self) -> None:
        if self._h:
            _lib.lazy_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    def access(self, key: int, n_blocks: int):
        if len(self._buf) < n_blocks:
            self._buf = (ctypes.c_int32 * max(n_blocks, 2 * len(self._buf)))()
        rc = _lib.lazy_cache_access(self._h, ctypes.c_uint64(int(key) & 0xFFFFFFFFFFFFFFFF), int(n_blocks),
                                    ctypes.cast(self._buf, ctypes.c_void_p))
        if rc == LAZY_ERANGE:
            return False, None
        if rc < 0:
            raise LazyAttnError("lazy_cache_access", rc)
        return rc == 1, np.frombuffer(self._buf, dtype=np.int32, count=n_blocks).copy()

    def contains(self, key: int) -> bool:
        return _lib.lazy_cache_contains(self._h, ctypes.c_uint64(int(key) & 0xFFFFFFFFFFFFFFFF)) == 1

    def stats(self) -> dict:
        out = (ctypes.c_int64 * 8)()
        _check("lazy_cache_stats", _lib.lazy_cache_stats(self._h, ctypes.cast(out, ctypes.c_void_p)))
        return dict(zip(self.STAT_NAMES, [int(x) for x in out]))

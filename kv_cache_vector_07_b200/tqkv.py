"""Python binding of libtqkv: argument marshalling only.

Every function mirrors one C entry point of ``include/tqkv.h`` and passes
torch tensors as raw device pointers plus the current CUDA stream.  All
computation happens in the library's CUDA kernels; there is no fallback: if
``libtqkv.so`` is missing or fails to load, importing this module raises.
Workspaces are allocated here with torch (zero-filled) when the caller does
not pass one; the library itself never allocates device memory outside
``tq_make_params``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
from dataclasses import dataclass

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtqkv.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "tqkv.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libtqkv.so is not built ({LIB_PATH}); run `python -m kv_cache_vector_07_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)

TQ_OK, TQ_EINVAL, TQ_EUNSUPPORTED, TQ_ECUDA, TQ_EDEVICE, TQ_ENOMEM, TQ_ESCRATCH = range(7)
TQ_NOALLOC_SCRATCH_BYTES = 16 << 20
TQ_DEV_SLOT_RANGE, TQ_DEV_BLOCK_RANGE, TQ_DEV_WAIT_TIMEOUT = 0x1, 0x2, 0x4
TQ_DEV_ROW, TQ_DEV_NO_PAGES, TQ_DEV_PAGE_SHARED, TQ_DEV_KEEP_RANGE = 0x8, 0x10, 0x20, 0x40
TQ_DTYPE_BF16, TQ_DTYPE_F32 = 0, 1
TQ_ROT_HADAMARD, TQ_ROT_DENSE = 0, 1
TQ_ROPE_HALF, TQ_ROPE_PAIRS = 0, 1
TQ_BITS_HALF = 16
TQ_BITS_POLAR = 32


def half_bits(rate: float) -> int:
    """Code width of a fractional rate (1.5, 2.5, 3.5): TQ_BITS_HALF | b."""
    b = int(rate - 0.5)
    if rate - 0.5 != b or not 1 <= b <= 3:
        raise ValueError("fractional rates are 1.5, 2.5 and 3.5")
    return TQ_BITS_HALF | b


def _n_levels(bits: int, d: int) -> tuple[int, int]:
    if bits == 8:
        return 0, 0
    if bits == TQ_BITS_POLAR:
        lv = int(np.log2(d))
        return 16 + 4 * (lv - 1), 15 + 3 * (lv - 1)
    if bits & TQ_BITS_HALF:
        b = bits & 7
        return (2 << b) + (1 << b), (2 << b) + (1 << b) - 2
    return 1 << bits, (1 << bits) - 1

_vp, _i32, _i64, _u64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t


class CacheDesc(ctypes.Structure):
    """Mirror of tq_cache_desc."""
    _fields_ = [("d", _i32), ("kbits", _i32), ("kqjl", _i32), ("vbits", _i32), ("page_tokens", _i32),
                ("n_kv_heads", _i32)]

    def __repr__(self):
        return (f"CacheDesc(d={self.d}, kbits={self.kbits}, kqjl={self.kqjl}, vbits={self.vbits}, "
                f"page_tokens={self.page_tokens}, n_kv_heads={self.n_kv_heads})")


class RopeDesc(ctypes.Structure):
    """Mirror of tq_rope_desc."""
    _fields_ = [("d", _i32), ("rot_dim", _i32), ("style", _i32), ("n_axes", _i32), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("pair_axis", ctypes.c_uint8 * 128)]


class _Heads(ctypes.Structure):
    """Mirror of tq_heads."""
    _fields_ = [("x", _vp), ("tok_stride", _i64), ("head_stride", _i64), ("weight", _vp), ("out", _vp),
                ("out_tok_stride", _i64), ("out_head_stride", _i64), ("n_heads", _i32)]


class _PagePool(ctypes.Structure):
    """Mirror of tq_page_pool."""
    _fields_ = [("refs", _vp), ("table", _vp), ("lens", _vp), ("num_blocks", _i64), ("n_rows", _i32),
                ("max_blocks", _i32)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_sig("tq_make_params", _i32, [_i32, _i32, _u64, ctypes.POINTER(_vp)])
_sig("tq_make_params_rot", _i32, [_i32, _i32, _u64, _i32, ctypes.POINTER(_vp)])
_sig("tq_compute_rotation_host", _i32, [_i32, _u64, _i32, _vp])
_sig("tq_params_export_rotation", _i32, [_vp, _vp])
_sig("tq_compute_params_host", _i32, [_i32, _i32, _u64, _vp, _vp, _vp, _vp])
_sig("tq_free_params", None, [_vp])
_sig("tq_params_export", _i32, [_vp, _vp, _vp, _vp, _vp])
_sig("tq_cache_bytes", _i32, [ctypes.POINTER(CacheDesc), ctypes.POINTER(_sz)])
_sig("tq_encode_workspace_bytes", _sz, [ctypes.POINTER(CacheDesc), _i64])
_sig("tq_encode", _i32, [_vp, _vp, ctypes.POINTER(CacheDesc), _vp, _vp, _i32, _i64, _vp, _vp, _i64, _vp, _sz,
                         _vp])
_sig("tq_decode_workspace_bytes", _sz, [ctypes.POINTER(CacheDesc), _i32, _i32, _i32])
_sig("tq_decode_attn", _i32, [_vp, _vp, ctypes.POINTER(CacheDesc), _vp, _i32, _i32, _vp, _i32, _vp, _i32, _vp,
                              _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp])
_sig("tq_decode_attn_noalloc", _i32, [_vp, _vp, ctypes.POINTER(CacheDesc), _vp, _i32, _i32, _vp, _i32, _vp, _i32,
                                      _vp, _i64, _vp, _vp, _vp, _i64, _vp])
_sig("tq_decode_step", _i32, [_vp, _vp, ctypes.POINTER(CacheDesc), _vp, _vp, _vp, _vp, _i32, _i32, _vp, _i32, _vp,
                              _i32, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp])
_sig("tq_prefill_workspace_bytes", _sz, [ctypes.POINTER(CacheDesc), _i32, _i32, _i32])
_sig("tq_prefill_attn", _i32, [_vp, _vp, ctypes.POINTER(CacheDesc), _vp, _i32, _i32, _vp, _i32, _i32, _vp, _i64,
                               _vp, _vp, _vp, _sz, _vp])
_sig("tq_score_workspace_bytes", _sz, [ctypes.POINTER(CacheDesc), _i64, _i32, _i32])
_sig("tq_score", _i32, [_vp, ctypes.POINTER(CacheDesc), _vp, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _sz, _vp])
_pool_p, _desc_p, _ptrs = ctypes.POINTER(_PagePool), ctypes.POINTER(CacheDesc), ctypes.POINTER(_vp)
_sig("tq_cross_workspace_bytes", _sz, [_desc_p, _i32, _i32, _i32, _i32, _i32])
_sig("tq_cross_attn", _i32, [_vp, _vp, _desc_p, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _i64, _vp,
                             _vp, _vp, _sz, _vp])
_sig("tq_pages_workspace_bytes", _sz, [_i64, _i32, _i32])
_sig("tq_pages_reserve", _i32, [_desc_p, _pool_p, _vp, _vp, _i64, _vp, _sz, _vp])
_sig("tq_pages_fork", _i32, [_desc_p, _pool_p, _ptrs, _i32, _vp, _vp, _i32, _vp, _sz, _vp])
_sig("tq_pages_compact", _i32, [_desc_p, _pool_p, _ptrs, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _sz, _vp])
_sig("tq_pages_free", _i32, [_desc_p, _pool_p, _vp, _i32, _vp, _sz, _vp])
_sig("tq_qk_norm_rope", _i32, [ctypes.POINTER(RopeDesc), _i32, _i32, _i64, ctypes.POINTER(_Heads),
                               ctypes.POINTER(_Heads), _vp, _i64, _vp, _vp])
_sig("tq_read_status", _i32, [_vp, _vp, ctypes.POINTER(ctypes.c_uint32)])
_sig("tq_status_string", ctypes.c_char_p, [_i32])
_sig("tq_test_stall_next_decode", _i32, [ctypes.c_uint32])
_sig("tq_noalloc_read_status", _i32, [_vp, ctypes.POINTER(ctypes.c_uint32)])


class TQError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_string(code)} ({code})")
        self.code = code


def status_string(code: int) -> str:
    return _lib.tq_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != TQ_OK:
        raise TQError(code, where)


def declared_functions() -> list[str]:
    """Names of the functions declared in include/tqkv.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tq_[a-z0-9_]+)\s*\(", text)))


def exported(name: str) -> bool:
    try:
        getattr(_lib, name)
        return True
    except AttributeError:
        return False


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev_check(*tensors):
    for t in tensors:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libtqkv arguments must be contiguous CUDA tensors")


def _one_device(*tensors) -> int:
    """The index of the one CUDA device that all given tensors are on."""
    dev = None
    for t in tensors:
        if t is not None:
            if dev is None:
                dev = t.get_device()
            elif t.get_device() != dev:
                dev = -1
            if dev < 0:
                raise ValueError("libtqkv arguments must be CUDA tensors of one device")
    return dev


def _call(dev: int, name: str, stream, *args):
    """The C entry point `name` with args and a stream of device dev, which is
    made current for the call where it is not already."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    else:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    f = getattr(_lib, name)
    if dev == torch._C._cuda_getDevice():
        code = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            code = f(*args, stream)
    if code != TQ_OK:
        raise TQError(code, name)


# ---------------------------------------------------------------------------
# parameters
# ---------------------------------------------------------------------------
class Params:
    """Handle of library-owned parameters (tq_make_params)."""

    def __init__(self, d: int, bits: int, seed: int, rotation: int = TQ_ROT_HADAMARD):
        h = _vp()
        _check(_lib.tq_make_params_rot(d, bits, seed, rotation, ctypes.byref(h)), "tq_make_params_rot")
        self._h = h
        self.d, self.bits, self.seed, self.rotation = d, bits, seed, rotation

    def rotation_matrix(self) -> np.ndarray:
        """tq_params_export_rotation: R [d, d] (y = R x), float32."""
        R = np.zeros((self.d, self.d), np.float32)
        _check(_lib.tq_params_export_rotation(self._h, R.ctypes.data), "tq_params_export_rotation")
        return R

    @property
    def handle(self):
        return self._h

    def export(self):
        d = self.d
        signs = np.zeros(d, np.int8)
        S = np.zeros((d, d), np.float32)
        L, NB = _n_levels(self.bits, d)
        lv = np.zeros(max(L, 1), np.float32)
        bd = np.zeros(max(NB, 1), np.float32)
        _check(_lib.tq_params_export(self._h, signs.ctypes.data, S.ctypes.data, lv.ctypes.data, bd.ctypes.data),
               "tq_params_export")
        return signs, S, (lv if L else None), (bd if L else None)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.tq_free_params(h)
            self._h = _vp()


def make_params(d: int, bits: int, seed: int, rotation: int = TQ_ROT_HADAMARD) -> Params:
    return Params(d, bits, seed, rotation)


def compute_rotation_host(d: int, seed: int, rotation: int = TQ_ROT_DENSE) -> np.ndarray:
    """tq_compute_rotation_host: the rotation matrix of (d, seed) on the host."""
    R = np.zeros((d, d), np.float32)
    _check(_lib.tq_compute_rotation_host(d, seed, rotation, R.ctypes.data), "tq_compute_rotation_host")
    return R


def compute_params_host(d: int, bits: int, seed: int):
    signs = np.zeros(d, np.int8)
    S = np.zeros((d, d), np.float32)
    L, NB = _n_levels(bits, d)
    lv = np.zeros(max(L, 1), np.float32)
    bd = np.zeros(max(NB, 1), np.float32)
    _check(_lib.tq_compute_params_host(d, bits, seed, signs.ctypes.data, S.ctypes.data, lv.ctypes.data,
                                       bd.ctypes.data), "tq_compute_params_host")
    return signs, S, (lv if L else None), (bd if L else None)


def free_params(p: Params):
    p.__del__()


# ---------------------------------------------------------------------------
# cache
# ---------------------------------------------------------------------------
def cache_desc(d: int, kbits: int, kqjl: bool, vbits: int, page_tokens: int = 64, n_kv_heads: int = 1) -> CacheDesc:
    return CacheDesc(d, kbits, 1 if kqjl else 0, vbits, page_tokens, n_kv_heads)


def cache_bytes(desc: CacheDesc) -> int:
    out = _sz()
    _check(_lib.tq_cache_bytes(ctypes.byref(desc), ctypes.byref(out)), "tq_cache_bytes")
    return int(out.value)


def _made_on(dev: int, stream):
    """Context for the tensors that a call makes itself: what clears them, and
    the allocator's reuse of them, are ordered by the stream the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        at = int(stream)
        stream = torch.cuda.ExternalStream(at, device=dev) if at else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


@functools.lru_cache(maxsize=256)
def _page_bytes(*fields) -> int:
    return cache_bytes(CacheDesc(*fields))


def _page_of(desc: CacheDesc) -> int:
    """cache_bytes, remembered by the description's values."""
    return _page_bytes(desc.d, desc.kbits, desc.kqjl, desc.vbits, desc.page_tokens, desc.n_kv_heads)


def alloc_cache(desc: CacheDesc, num_blocks: int, device="cuda") -> torch.Tensor:
    """Zeroed cache tensor [num_blocks, n_kv_heads, page_bytes] (uint8)."""
    return torch.zeros((num_blocks, desc.n_kv_heads, cache_bytes(desc)), dtype=torch.uint8, device=device)


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def encode_workspace_bytes(desc: CacheDesc, n_tokens: int) -> int:
    return int(_lib.tq_encode_workspace_bytes(ctypes.byref(desc), n_tokens))


def encode(kp: Params, vp: Params | None, desc: CacheDesc, K: torch.Tensor, V: torch.Tensor | None,
           slot_mapping: torch.Tensor, cache: torch.Tensor, workspace: torch.Tensor | None = None, stream=None):
    """tq_encode: K, V [n_tokens, n_kv_heads, d] (bf16 or fp32) into the cache."""
    _dev_check(K, V, slot_mapping, cache, workspace)
    dt = {torch.bfloat16: TQ_DTYPE_BF16, torch.float32: TQ_DTYPE_F32}.get(K.dtype)
    if dt is None:
        raise ValueError("K must be bf16 or fp32")
    if V is not None and V.dtype != K.dtype:
        raise ValueError("K and V dtypes differ")
    if slot_mapping.dtype != torch.int32:
        raise ValueError("slot_mapping must be int32")
    n_tokens = K.shape[0]
    if workspace is None:
        workspace = _workspace(encode_workspace_bytes(desc, n_tokens), K.device)
    num_blocks = cache.shape[0]
    _check(_lib.tq_encode(kp.handle, vp.handle if vp is not None else None, ctypes.byref(desc), _ptr(K), _ptr(V),
                          dt, n_tokens, _ptr(slot_mapping), _ptr(cache), num_blocks, _ptr(workspace),
                          workspace.numel(), _stream(stream)), "tq_encode")
    return workspace


def decode_workspace_bytes(desc: CacheDesc, B: int, Hq: int, max_seq_len: int) -> int:
    return int(_lib.tq_decode_workspace_bytes(ctypes.byref(desc), B, Hq, max_seq_len))


def decode_attn(kp: Params, vp: Params, desc: CacheDesc, Q: torch.Tensor, block_table: torch.Tensor,
                seq_lens: torch.Tensor, max_seq_len: int, cache: torch.Tensor, out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, logits: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """tq_decode_attn: Q bf16 [B, Hq, d] -> out bf16 [B, Hq, d]."""
    _dev_check(Q, block_table, seq_lens, cache, out, lse, logits, workspace)
    B, Hq, d = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    if workspace is None:
        workspace = _workspace(decode_workspace_bytes(desc, B, Hq, max_seq_len), Q.device)
    stride = logits.shape[-1] if logits is not None else 0
    _check(_lib.tq_decode_attn(kp.handle, vp.handle, ctypes.byref(desc), _ptr(Q), B, Hq, _ptr(block_table),
                               block_table.shape[1], _ptr(seq_lens), max_seq_len, _ptr(cache), cache.shape[0],
                               _ptr(out), _ptr(lse), _ptr(logits), stride, _ptr(workspace), workspace.numel(),
                               _stream(stream)), "tq_decode_attn")
    return out


def decode_step(kp: Params, vp: Params, desc: CacheDesc, K_new: torch.Tensor, V_new: torch.Tensor,
                slot_mapping: torch.Tensor, Q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                max_seq_len: int, cache: torch.Tensor, out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, logits: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """tq_decode_step: write K_new/V_new bf16 [B, n_kv_heads, d] at slot_mapping
    [B], then decode attention of Q bf16 [B, Hq, d] over seq_lens tokens."""
    _dev_check(K_new, V_new, slot_mapping, Q, block_table, seq_lens, cache, out, lse, logits, workspace)
    if K_new.dtype != torch.bfloat16 or V_new.dtype != torch.bfloat16 or slot_mapping.dtype != torch.int32:
        raise ValueError("K_new/V_new must be bf16 and slot_mapping int32")
    B, Hq, d = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    if workspace is None:
        workspace = _workspace(decode_workspace_bytes(desc, B, Hq, max_seq_len), Q.device)
    stride = logits.shape[-1] if logits is not None else 0
    _check(_lib.tq_decode_step(kp.handle, vp.handle, ctypes.byref(desc), _ptr(K_new), _ptr(V_new),
                               _ptr(slot_mapping), _ptr(Q), B, Hq, _ptr(block_table), block_table.shape[1],
                               _ptr(seq_lens), max_seq_len, _ptr(cache), cache.shape[0], _ptr(out), _ptr(lse),
                               _ptr(logits), stride, _ptr(workspace), workspace.numel(), _stream(stream)),
           "tq_decode_step")
    return out


def decode_attn_noalloc(kp: Params, vp: Params, desc: CacheDesc, Q: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, max_seq_len: int, cache: torch.Tensor, out: torch.Tensor | None = None,
                        lse: torch.Tensor | None = None, logits: torch.Tensor | None = None, stream=None):
    """tq_decode_attn_noalloc: tq_decode_attn for callers that cannot allocate
    device memory; the scratch is the library's static device array, shared
    by all calls on the device (calls that overlap on the GPU race)."""
    _dev_check(Q, block_table, seq_lens, cache, out, lse, logits)
    B, Hq, d = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    stride = logits.shape[-1] if logits is not None else 0
    _check(_lib.tq_decode_attn_noalloc(kp.handle, vp.handle, ctypes.byref(desc), _ptr(Q), B, Hq, _ptr(block_table),
                                       block_table.shape[1], _ptr(seq_lens), max_seq_len, _ptr(cache),
                                       cache.shape[0], _ptr(out), _ptr(lse), _ptr(logits), stride, _stream(stream)),
           "tq_decode_attn_noalloc")
    return out


def noalloc_read_status(stream=None) -> int:
    """tq_noalloc_read_status: status flags of the last no-allocation decode
    on the current device (cleared by the read)."""
    flags = ctypes.c_uint32()
    _check(_lib.tq_noalloc_read_status(_stream(stream), ctypes.byref(flags)), "tq_noalloc_read_status")
    return int(flags.value)


def prefill_workspace_bytes(desc: CacheDesc, C: int, Hq: int, seq_len: int) -> int:
    return int(_lib.tq_prefill_workspace_bytes(ctypes.byref(desc), C, Hq, seq_len))


def prefill_attn(kp: Params, vp: Params, desc: CacheDesc, Q: torch.Tensor, block_table: torch.Tensor,
                 seq_len: int, cache: torch.Tensor, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """tq_prefill_attn: chunk queries Q bf16 [C, Hq, d] over one sequence."""
    _dev_check(Q, block_table, cache, out, lse, workspace)
    C, Hq, d = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    if workspace is None:
        workspace = _workspace(prefill_workspace_bytes(desc, C, Hq, seq_len), Q.device)
    _check(_lib.tq_prefill_attn(kp.handle, vp.handle, ctypes.byref(desc), _ptr(Q), C, Hq, _ptr(block_table),
                                block_table.numel(), seq_len, _ptr(cache), cache.shape[0], _ptr(out), _ptr(lse),
                                _ptr(workspace), workspace.numel(), _stream(stream)), "tq_prefill_attn")
    return out


def score_workspace_bytes(desc: CacheDesc, n_db: int, n_q: int, k: int) -> int:
    return int(_lib.tq_score_workspace_bytes(ctypes.byref(desc), n_db, n_q, k))


def score(p: Params, desc: CacheDesc, db_cache: torch.Tensor, n_db: int, Q: torch.Tensor, k: int,
          top_scores: torch.Tensor | None = None, top_idx: torch.Tensor | None = None,
          workspace: torch.Tensor | None = None, stream=None):
    """tq_score: top-k estimated inner products of fp32 queries Q [n_q, d]."""
    _dev_check(db_cache, Q, top_scores, top_idx, workspace)
    n_q = Q.shape[0]
    if top_scores is None:
        top_scores = torch.empty((n_q, k), dtype=torch.float32, device=Q.device)
    if top_idx is None:
        top_idx = torch.empty((n_q, k), dtype=torch.int64, device=Q.device)
    if workspace is None:
        workspace = _workspace(score_workspace_bytes(desc, n_db, n_q, k), Q.device)
    _check(_lib.tq_score(p.handle, ctypes.byref(desc), _ptr(db_cache), n_db, _ptr(Q), n_q, k, _ptr(top_scores),
                         _ptr(top_idx), _ptr(workspace), workspace.numel(), _stream(stream)), "tq_score")
    return top_scores, top_idx


# ---------------------------------------------------------------------------
# cross attention
# ---------------------------------------------------------------------------
def cross_workspace_bytes(desc: CacheDesc, B: int, total_q: int, max_q: int, Hq: int, max_kv_len: int) -> int:
    return int(_lib.tq_cross_workspace_bytes(ctypes.byref(desc), B, total_q, max_q, Hq, max_kv_len))


def cross_attn(kp: Params, vp: Params, desc: CacheDesc, Q: torch.Tensor, cu_q: torch.Tensor, max_q: int,
               block_table: torch.Tensor, kv_lens: torch.Tensor, max_kv_len: int, cache: torch.Tensor,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None):
    """tq_cross_attn: the queries cu_q[b] .. cu_q[b + 1] - 1 of Q bf16 [total_q,
    Hq, d] see all kv_lens[b] tokens of sequence b (block_table [B, max_blocks]).
    Rows of out that belong to no run are not written (zero where out is not
    given).  lse fp32 [total_q, Hq], optional."""
    dev = _one_device(Q, cu_q, block_table, kv_lens, cache, out, lse, workspace)
    for t in (Q, cu_q, block_table, kv_lens, out, lse, workspace):
        if t is not None and not t.is_contiguous():
            raise ValueError("libtqkv arguments must be contiguous CUDA tensors")
    if Q.dim() != 3 or Q.dtype is not torch.bfloat16 or Q.size(2) != desc.d:
        raise ValueError("Q must be bf16 [total_q, Hq, d]")
    total_q, Hq, _ = Q.shape
    B = kv_lens.numel()
    if block_table.dim() != 2 or block_table.size(0) != B or kv_lens.dim() != 1 or cu_q.dim() != 1 or \
            cu_q.numel() != B + 1:
        raise ValueError("block_table must be [B, max_blocks], kv_lens [B] and cu_q [B + 1]")
    if not (cu_q.dtype is block_table.dtype is kv_lens.dtype is torch.int32):
        raise ValueError("cu_q, block_table and kv_lens must be int32")
    if cache.dtype is not torch.uint8 or cache.shape[1:] != (desc.n_kv_heads, _page_of(desc)) or \
            not cache.is_contiguous():
        raise ValueError("cache must be uint8 [num_blocks, n_kv_heads, page bytes]")
    if out is None:
        with _made_on(dev, stream):
            out = torch.zeros_like(Q)
    elif out.shape != Q.shape or out.dtype is not Q.dtype:
        raise ValueError("out must have Q's shape and dtype")
    if lse is not None and (lse.shape != (total_q, Hq) or lse.dtype is not torch.float32):
        raise ValueError("lse must be fp32 [total_q, Hq]")
    if workspace is None:                                # only its header (the status word) starts as zeros
        with _made_on(dev, stream):
            workspace = torch.empty(max(cross_workspace_bytes(desc, B, total_q, max_q, Hq, max_kv_len), 256),
                                    dtype=torch.uint8, device=Q.device)
            workspace[:256].zero_()
    _call(dev, "tq_cross_attn", stream, kp.handle, vp.handle, ctypes.byref(desc), Q.data_ptr(), total_q, max_q, Hq,
          cu_q.data_ptr(), B, block_table.data_ptr(), block_table.size(1), kv_lens.data_ptr(), max_kv_len,
          cache.data_ptr(), cache.size(0), out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel())
    return out


# ---------------------------------------------------------------------------
# pages of a cache
# ---------------------------------------------------------------------------
def pages_workspace_bytes(num_blocks: int, n_rows: int, max_blocks: int) -> int:
    return int(_lib.tq_pages_workspace_bytes(num_blocks, n_rows, max_blocks))


def _pool(desc, refs, table, lens, ints, workspace, stream, caches=None):
    """(device index, tq_page_pool, workspace, cache pointers) of a pages call."""
    dev = _one_device(refs, table, lens, workspace, *ints)
    for t in (refs, table, lens, *ints):
        if t.dtype is not torch.int32 or not t.is_contiguous():
            raise ValueError("refs, table, lens and the requests must be contiguous int32 tensors")
    shape = table.shape
    if len(shape) != 2 or refs.dim() != 1 or lens.shape != shape[:1]:
        raise ValueError("refs must be [num_blocks], table [n_rows, max_blocks] and lens [n_rows]")
    num_blocks, (n_rows, max_blocks) = refs.size(0), shape
    ptrs = None
    if caches is not None:
        layers = [caches] if isinstance(caches, torch.Tensor) else caches
        want = (num_blocks, desc.n_kv_heads, _page_of(desc))
        for c in layers:
            if c.get_device() != dev or c.dtype is not torch.uint8 or c.shape != want or not c.is_contiguous():
                raise ValueError("every cache must be contiguous uint8 [num_blocks, n_kv_heads, page bytes] on the "
                                 "tables' device")
        if not layers:
            raise ValueError("caches must name one cache at least")
        ptrs = (_vp * len(layers))(*[c.data_ptr() for c in layers])
    if workspace is None:
        with _made_on(dev, stream):
            workspace = _workspace(pages_workspace_bytes(num_blocks, n_rows, max_blocks), refs.device)
    elif not workspace.is_contiguous():                  # numel() is what it holds
        raise ValueError("workspace must be contiguous")
    pool = _PagePool(refs.data_ptr(), table.data_ptr(), lens.data_ptr(), num_blocks, n_rows, max_blocks)
    return dev, pool, workspace, ptrs


def pages_reserve(desc: CacheDesc, refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                  new_tokens: torch.Tensor, slot_mapping: torch.Tensor, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """tq_pages_reserve: pages and slots for new_tokens int32 [n_rows] more
    tokens of every row; slot_mapping int32 [n_slots] receives their slots, row
    after row.  refs int32 [num_blocks], table int32 [n_rows, max_blocks] and
    lens int32 [n_rows] are updated.  Returns the workspace (read_status)."""
    dev, pool, workspace, _ = _pool(desc, refs, table, lens, (new_tokens, slot_mapping), workspace, stream)
    if new_tokens.shape != lens.shape or slot_mapping.dim() != 1:
        raise ValueError("new_tokens must be [n_rows] and slot_mapping [n_slots]")
    _call(dev, "tq_pages_reserve", stream, ctypes.byref(desc), ctypes.byref(pool), new_tokens.data_ptr(),
          slot_mapping.data_ptr(), slot_mapping.numel(), workspace.data_ptr(), workspace.numel())
    return workspace


def pages_fork(desc: CacheDesc, caches, refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
               src_rows: torch.Tensor, dst_rows: torch.Tensor, workspace: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """tq_pages_fork: rows dst_rows (empty) become copies of rows src_rows
    (int32 [n]); caches: one cache, or a list with every layer's.  Full pages
    are shared, partly filled ones copied.  Returns the workspace."""
    dev, pool, workspace, ptrs = _pool(desc, refs, table, lens, (src_rows, dst_rows), workspace, stream, caches)
    if src_rows.dim() != 1 or src_rows.shape != dst_rows.shape:
        raise ValueError("src_rows and dst_rows must be [n]")
    _call(dev, "tq_pages_fork", stream, ctypes.byref(desc), ctypes.byref(pool), ptrs, len(ptrs), src_rows.data_ptr(),
          dst_rows.data_ptr(), src_rows.numel(), workspace.data_ptr(), workspace.numel())
    return workspace


def pages_compact(desc: CacheDesc, caches, refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                  rows: torch.Tensor, keep: torch.Tensor, keep_lens: torch.Tensor,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """tq_pages_compact: row rows[i] keeps its tokens keep[i, :keep_lens[i]]
    (int32 [n], [n, most], [n]), in that order; caches as in pages_fork.
    Returns the workspace."""
    dev, pool, workspace, ptrs = _pool(desc, refs, table, lens, (rows, keep, keep_lens), workspace, stream, caches)
    if rows.dim() != 1 or keep.dim() != 2 or keep.size(0) != rows.numel() or keep_lens.shape != rows.shape:
        raise ValueError("rows and keep_lens must be [n] and keep [n, most]")
    _call(dev, "tq_pages_compact", stream, ctypes.byref(desc), ctypes.byref(pool), ptrs, len(ptrs), rows.data_ptr(),
          keep.data_ptr(), keep.size(1), keep_lens.data_ptr(), rows.numel(), workspace.data_ptr(), workspace.numel())
    return workspace


def pages_free(desc: CacheDesc, refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, rows: torch.Tensor,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """tq_pages_free: rows (int32 [n]) give their pages back and become empty.
    Returns the workspace."""
    dev, pool, workspace, _ = _pool(desc, refs, table, lens, (rows,), workspace, stream)
    if rows.dim() != 1:
        raise ValueError("rows must be [n]")
    _call(dev, "tq_pages_free", stream, ctypes.byref(desc), ctypes.byref(pool), rows.data_ptr(), rows.numel(),
          workspace.data_ptr(), workspace.numel())
    return workspace


# ---------------------------------------------------------------------------
# head norms with rotary positions
# ---------------------------------------------------------------------------
def rope_desc(d: int, rot_dim: int | None = None, style: int = TQ_ROPE_HALF, pair_axis=None, n_axes: int = 1,
              eps: float = 1e-6, scale: float = 1.0) -> RopeDesc:
    """The position rotation of one head (tq_rope_desc); pair_axis: the axis of
    each of the rot_dim / 2 pairs (all 0 when omitted)."""
    rot = d if rot_dim is None else rot_dim
    axis = list(pair_axis) if pair_axis is not None else []
    if len(axis) > 128 or (axis and len(axis) != rot // 2) or any(not 0 <= a < n_axes for a in axis):
        raise ValueError("pair_axis holds one axis (0 .. n_axes - 1) for each of the rot_dim / 2 pairs")
    return RopeDesc(d, rot, style, n_axes, eps, scale, (ctypes.c_uint8 * 128)(*axis))


_ROPE_DTYPES = {torch.bfloat16: TQ_DTYPE_BF16, torch.float32: TQ_DTYPE_F32}


def _heads(x, weight, out, d, n, name, dev, stream):
    """(tq_heads, result tensor) of one side of qk_norm_rope."""
    if x is None:
        return None, None
    shape = x.shape
    if len(shape) != 3 or shape[0] != n or shape[2] != d:
        raise ValueError(f"{name} must be [n_tokens, heads, d]")
    if out is None:
        with _made_on(dev, stream):
            out = torch.empty(shape, dtype=x.dtype, device=x.device)
    elif out.shape != shape or out.dtype is not x.dtype:
        raise ValueError(f"{name}_out must have {name}'s shape and dtype")
    xt, xh, xd = x.stride()
    ot, oh, od = out.stride()
    if xd != 1 or od != 1:
        raise ValueError(f"the coordinates of {name} and {name}_out must be adjacent")
    return _Heads(x.data_ptr(), xt, xh, None if weight is None else weight.data_ptr(), out.data_ptr(), ot, oh,
                  shape[1]), out


def qk_norm_rope(desc: RopeDesc, q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor,
                 inv_freq: torch.Tensor, q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """tq_qk_norm_rope: RMS norm (where a weight is given) and position rotation
    of q [n, Hq, d] and k [n, H, d] (bf16 or fp32, strided slices allowed);
    positions int32 [n] or [n_axes, n], inv_freq fp32 [rot_dim / 2].  Returns
    (q_out, k_out), contiguous where not given; q_out may be q itself."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k must be given")
    d, n = desc.d, x.size(0)
    dev = _one_device(q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    dtype, wtype = x.dtype, None
    if dtype not in _ROPE_DTYPES or (k is not None and k.dtype is not dtype):
        raise ValueError("q and k must both be bf16 or both fp32")
    for w in (q_weight, k_weight):
        if w is not None:
            if wtype is not None and w.dtype is not wtype:
                raise ValueError("the weights must both be bf16 or both fp32")
            wtype = w.dtype
            if wtype not in _ROPE_DTYPES or w.shape != (d,) or not w.is_contiguous():
                raise ValueError("weights must be contiguous [d], bf16 or fp32")
    if positions.dtype is not torch.int32 or inv_freq.dtype is not torch.float32:
        raise ValueError("positions must be int32 and inv_freq fp32")
    shape, step = positions.shape, positions.stride()
    if shape != (n,) if desc.n_axes == 1 and len(shape) == 1 else shape != (desc.n_axes, n):
        raise ValueError("positions must be [n_tokens], or [n_axes, n_tokens]")
    if n > 1 and step[-1] != 1:
        raise ValueError("the positions of an axis must be adjacent")
    if inv_freq.numel() != desc.rot_dim // 2 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous [rot_dim / 2]")
    hq, q_out = _heads(q, q_weight, q_out, d, n, "q", dev, stream)
    hk, k_out = _heads(k, k_weight, k_out, d, n, "k", dev, stream)
    _call(dev, "tq_qk_norm_rope", stream, ctypes.byref(desc), _ROPE_DTYPES[dtype], _ROPE_DTYPES[wtype or dtype], n,
          hq and ctypes.byref(hq), hk and ctypes.byref(hk), positions.data_ptr(), step[0] if len(shape) == 2 else n,
          inv_freq.data_ptr())
    return q_out, k_out


def read_status(workspace: torch.Tensor, stream=None) -> int:
    flags = ctypes.c_uint32()
    _check(_lib.tq_read_status(_ptr(workspace), _stream(stream), ctypes.byref(flags)), "tq_read_status")
    return int(flags.value)


def test_stall_next_decode(polls: int) -> None:
    """tq_test_stall_next_decode: the next tensor-core decode launch waits
    `polls` polls on a barrier nothing completes and takes its time-out path
    (a testing aid for the TQ_DEV_WAIT_TIMEOUT flag; 0 cancels)."""
    _check(_lib.tq_test_stall_next_decode(int(polls)), "tq_test_stall_next_decode")

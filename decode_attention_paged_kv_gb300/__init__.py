"""Python binding of libdkv: GB300 decode attention over a paged KV cache.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/dkv.h``.  PyTorch provides the
device memory (outputs and workspace are allocated with torch) and the current
stream.  There is no fallback: if ``libdkv.so`` has not been built, or a call
returns an error status, the call raises.

Public calls (same names as the C ABI, without the ``dkv_`` prefix):
  kv_meta_build(K)                      -> (meta_min, meta_max)
  decode_attn_full(q, K, V)             -> out
  decode_attn_select(q, K, V, meta, k)  -> out (, selected)
  kv_quant4(x) / kv_dequant4(q4)
  kv_append(k, v, K, V, lens)           new tokens into a cache (-> rotated q)
  workspace_bytes(...), read_device_status(workspace)
K and V are dense tensors [B, Hkv, N, d] (bf16 / fp16; any batch / head
strides, token stride d), ``Q4Cache`` tuples in the 4-bit format,
``PagedCache`` pools, or ``Fp8Cache`` / ``Fp8PagedCache`` in the 8-bit format.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import threading
from typing import NamedTuple, Optional

import torch

from . import build as _build_mod

__all__ = [
    "Q4Cache", "PagedCache", "Fp8Cache", "Fp8PagedCache", "Meta8", "DkvError", "lib", "kv_meta_build", "kv_meta8_build",
    "kv_append", "kv_meta_append", "rope_table", "hot_state", "hot_stats", "decode_attn_full",
    "decode_attn_select", "decode_attn_topk_tokens", "kv_quant4", "kv_dequant4",
    "workspace_bytes", "workspace_bytes_tokens", "read_device_status", "status_string",
    "PAGE_SIZE", "DKV_FLAG_GROUP_SELECT",
]

PAGE_SIZE = 16

# enums of include/dkv.h
DKV_OK = 0
DKV_ERR_DEVICE_TIMEOUT = 8
DKV_ERR_DEVICE_CHECK = 9
DKV_BF16, DKV_FP16, DKV_FP32 = 0, 1, 2
DKV_KV_DENSE, DKV_KV_Q4G64, DKV_KV_PAGED, DKV_KV_FP8, DKV_KV_FP8_PAGED = 0, 1, 2, 3, 4
DKV_WORKSPACE_HEADER_BYTES = 256
DKV_FLAG_FORCE_TIMEOUT = 0x1
DKV_FLAG_GROUP_SELECT = 0x2


class DkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: dkv status {status} ({status_string(status)})")


class Q4Cache(NamedTuple):
    """A K or V cache in the 4-bit group-of-64 format.

    codes [B, Hkv, N, d/2] uint8 (channel 2i in the low nibble of byte i);
    gmin, gmax [B, Hkv, N, d/64] fp16 (per-group min / max).
    """
    codes: torch.Tensor
    gmin: torch.Tensor
    gmax: torch.Tensor


class Meta8(NamedTuple):
    """8-bit page metadata (kv_meta8_build): per page a grid
    dec(c) = fmaf(c, step, lo), and per channel the codes of m rounded down
    and of M rounded up on it.  code_min / code_max uint8 [B, Hkv, P, d];
    lo / step float32 [B, Hkv, P]."""
    code_min: torch.Tensor
    code_max: torch.Tensor
    lo: torch.Tensor
    step: torch.Tensor


class PagedCache(NamedTuple):
    """A K or V cache held as a pool of 16-token pages (blocks).

    pool [num_blocks, Hkv, 16, d] bf16 / fp16 (token and channel strides d, 1);
    block_table [B, P] int32: page j of batch entry b is pool block
    block_table[b, j]; seq_len: the N tokens every sequence attends.
    K and V passed to one call must share the block table.
    """
    pool: torch.Tensor
    block_table: torch.Tensor
    seq_len: int


class Fp8Cache(NamedTuple):
    """A K or V cache in the 8-bit format: a value is code * scale.

    codes [B, Hkv, N, d] float8_e4m3fn (any batch / head strides, token stride
    d); scale [B, Hkv, ceil(N / 16)] float32, one per 16 tokens and kv head;
    dtype: the 16-bit type of q, of the tokens appended and of the metadata.
    """
    codes: torch.Tensor
    scale: torch.Tensor
    dtype: torch.dtype = torch.bfloat16


class Fp8PagedCache(NamedTuple):
    """A K or V cache in the 8-bit format, held as a pool of 16-token blocks.

    pool [num_blocks, Hkv, 16, d] float8_e4m3fn; scale [num_blocks, Hkv]
    float32; block_table, seq_len as for PagedCache; dtype as for Fp8Cache.
    """
    pool: torch.Tensor
    scale: torch.Tensor
    block_table: torch.Tensor
    seq_len: int
    dtype: torch.dtype = torch.bfloat16


class _Params(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("seq_len", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("q_stride_b", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
                ("o_stride_b", ctypes.c_int64), ("o_stride_h", ctypes.c_int64),
                ("scale", ctypes.c_float), ("flags", ctypes.c_uint32),
                ("seq_lens", ctypes.c_void_p)]


class _KV(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("data", ctypes.c_void_p), ("gmin", ctypes.c_void_p), ("gmax", ctypes.c_void_p),
                ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("gstride_b", ctypes.c_int64), ("gstride_h", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
                ("num_blocks", ctypes.c_int32), ("scale", ctypes.c_void_p),
                ("sstride_b", ctypes.c_int64), ("sstride_h", ctypes.c_int64)]


class _Append(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in
                 ("batch", "num_q_heads", "num_kv_heads", "head_dim", "seq_len", "new_tokens",
                  "rotary_dim", "rope_len", "interleaved")]
                + [(n, ctypes.c_void_p) for n in ("k", "v", "q", "q_out")]
                + [(f"{t}_stride_{x}", ctypes.c_int64) for t in "kvqo" for x in "bth"]
                + [(n, ctypes.c_void_p) for n in ("cos", "sin", "seq_lens", "new_lens")])


_lib = None
_binding = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """The loaded libdkv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build_mod.LIB
            if not os.path.exists(path):
                raise RuntimeError(
                    f"libdkv.so not found at {path}; build it with "
                    "`python -m decode_attention_paged_kv_gb300.build`")
            L = ctypes.CDLL(path)
            vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            P, KVp = ctypes.POINTER(_Params), ctypes.POINTER(_KV)
            L.dkv_workspace_bytes.argtypes = [P, i32]
            L.dkv_workspace_bytes.restype = sz
            L.dkv_workspace_bytes_fp8.argtypes = [P, i32]
            L.dkv_workspace_bytes_fp8.restype = sz
            L.dkv_kv_append.argtypes = [ctypes.POINTER(_Append), KVp, KVp, vp, vp]
            L.dkv_kv_meta_build.argtypes = [P, KVp, vp, vp, vp]
            L.dkv_decode_attn_full.argtypes = [P, vp, KVp, KVp, vp, i32, vp, sz, vp]
            L.dkv_decode_attn_select.argtypes = [P, vp, KVp, KVp, vp, vp, i32, vp, i32, vp, vp,
                                                 sz, vp]
            L.dkv_decode_attn_topk_tokens.argtypes = [P, vp, KVp, KVp, i32, vp, i32, vp, vp,
                                                      sz, vp]
            L.dkv_kv_meta8_build.argtypes = [P, vp, vp, i32, vp, vp, vp, vp, vp]
            L.dkv_decode_attn_select_meta8.argtypes = [P, vp, KVp, KVp, vp, vp, vp, vp, i32,
                                                       vp, i32, vp, vp, sz, vp]
            L.dkv_workspace_bytes_tokens.argtypes = [P, i32]
            L.dkv_workspace_bytes_tokens.restype = sz
            L.dkv_kv_meta_append.argtypes = [P, KVp, vp, vp, vp]
            L.dkv_kv_meta_append_tokens.argtypes = [P, KVp, i32, vp, vp, vp, vp]
            L.dkv_hot_state_bytes.argtypes = [P]
            L.dkv_hot_state_bytes.restype = sz
            L.dkv_decode_attn_select_hot.argtypes = [P, vp, KVp, KVp, vp, vp, i32, vp, i32, vp,
                                                     vp, sz, i32, vp, sz, vp]
            L.dkv_kv_quant4.argtypes = [i64, i32, vp, vp, vp, vp, vp]
            L.dkv_kv_dequant4.argtypes = [i64, i32, vp, vp, vp, vp, vp]
            L.dkv_read_device_status.argtypes = [vp, vp]
            L.dkv_attn_ctas_per_sm.argtypes = [i32, i32, i32, i32, ctypes.POINTER(i32)]
            L.dkv_status_string.argtypes = [i32]
            L.dkv_status_string.restype = ctypes.c_char_p
            for name in ("dkv_kv_meta_build", "dkv_decode_attn_full", "dkv_decode_attn_select",
                         "dkv_decode_attn_topk_tokens", "dkv_kv_meta8_build",
                         "dkv_decode_attn_select_meta8", "dkv_kv_meta_append",
                         "dkv_kv_meta_append_tokens",
                         "dkv_decode_attn_select_hot", "dkv_kv_append",
                         "dkv_kv_quant4", "dkv_kv_dequant4", "dkv_read_device_status",
                         "dkv_attn_ctas_per_sm"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def _load_binding():
    """The native marshalling of a decode step's calls (csrc/binding.cpp)."""
    global _binding
    lib()
    with _lock:
        if _binding is None:
            path = _build_mod.BINDING
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{os.path.basename(path)} not found at {path}; build it with "
                    "`python -m decode_attention_paged_kv_gb300.build`")
            loader = importlib.machinery.ExtensionFileLoader(f"{__name__}._binding", path)
            spec = importlib.util.spec_from_loader(loader.name, loader)
            m = importlib.util.module_from_spec(spec)
            loader.exec_module(m)
            m.setup(Q4Cache, PagedCache, Fp8Cache, Fp8PagedCache, Meta8, DkvError)
            _binding = m
    return _binding


def status_string(status: int) -> str:
    return lib().dkv_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != DKV_OK:
        raise DkvError(status, where)


def _stream(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


_DTYPE_CODES = {torch.bfloat16: DKV_BF16, torch.float16: DKV_FP16, torch.float32: DKV_FP32}


def _dtype_code(dt: torch.dtype) -> int:
    code = _DTYPE_CODES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    return code


def _kv_struct(kv) -> tuple[_KV, int, int, int, int]:
    """(struct, B, Hkv, N, d) of a dense tensor or a cache tuple."""
    fields, B, H, N, d = (_binding or _load_binding()).describe_cache(kv)
    return _KV(*fields), B, H, N, d


def _params(q: Optional[torch.Tensor], B, Hkv, N, d, out: Optional[torch.Tensor],
            scale: Optional[float], flags: int = 0,
            seq_lens: Optional[torch.Tensor] = None) -> _Params:
    lens = None
    if seq_lens is not None:
        if (seq_lens.dtype != torch.int32 or seq_lens.shape != (B,) or not seq_lens.is_cuda
                or not seq_lens.is_contiguous()):
            raise ValueError("seq_lens must be a contiguous int32 CUDA tensor [B]")
        lens = seq_lens.data_ptr()
    Hq, qsb, qsh, osb, osh = Hkv, 0, 0, 0, 0
    if q is not None:
        qB, Hq, qd = q.shape[:3]
        qsb, qsh, one = q.stride()[:3]
        if qB != B or qd != d or one != 1:
            raise ValueError(f"q shape {tuple(q.shape)} does not match the cache")
    if out is not None:
        # (a row of out may be split into more dimensions, [B, Hq, 1, d] say)
        ok = out.dim() >= 3 and out.shape[0] >= B and out.shape[1] >= Hq
        run = 1  # elements of a row that follow one another
        for n, s in reversed(list(zip(out.shape[2:], out.stride()[2:]))):
            if not ok or run >= d:
                break
            ok = s == run or n == 1
            run *= n
        if not ok or run < d:
            raise ValueError(f"out must hold {(B, Hq, d)} with channel stride 1")
        osb, osh = out.stride()[:2]
    return _Params(B, Hq, Hkv, d, N, PAGE_SIZE, qsb, qsh, osb, osh,
                   1.0 / math.sqrt(d) if scale is None else float(scale), flags, lens)


def workspace_bytes(B: int, Hq: int, Hkv: int, d: int, N: int, top_k: int = 0,
                    page_size: int = PAGE_SIZE, fp8: bool = False) -> int:
    """Workspace bytes dkv_decode_attn_full (top_k = 0) or _select needs (fp8:
    on an 8-bit cache)."""
    p = _Params()
    p.batch, p.num_q_heads, p.num_kv_heads, p.head_dim, p.seq_len = B, Hq, Hkv, d, N
    p.page_size, p.scale = page_size, 1.0
    n = _workspace_need(p, int(top_k), fp8)
    if n == 0:
        raise DkvError(2, "dkv_workspace_bytes")
    return int(n)


def _workspace_need(p: _Params, top_k: int, fp8: bool) -> int:
    f = lib().dkv_workspace_bytes_fp8 if fp8 else lib().dkv_workspace_bytes
    return f(ctypes.byref(p), top_k)


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return workspace
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def kv_meta_build(K, page_size: int = PAGE_SIZE, seq_lens: Optional[torch.Tensor] = None):
    """Page metadata (meta_min, meta_max), each [B, Hkv, P, d]."""
    return (_binding or _load_binding()).kv_meta_build(K, page_size, seq_lens)


def kv_meta_append(K, meta, page_size: int = PAGE_SIZE,
                   seq_lens: Optional[torch.Tensor] = None, new_tokens: Optional[int] = None,
                   new_lens: Optional[torch.Tensor] = None):
    """After an append: rebuild, in place, only the pages of `meta` (from
    kv_meta_build) that the new tokens changed.

    seq_lens: each sequence's length with them (None: the cache length), as
    kv_append took it.  new_tokens: the rows T of that append (None: 1, a decode
    step); new_lens (int32 [B] on the device): how many of them each sequence
    has (None: all).  The other pages must be built already."""
    mn, mx = meta
    (_binding or _load_binding()).kv_meta_append(K, (mn, mx), page_size, seq_lens, new_tokens,
                                                 new_lens)
    return mn, mx


def rope_table(length: int, rotary_dim: int, base: float = 10000.0, device=None):
    """(cos, sin) float32 [length, rotary_dim / 2] of the angles
    p * base^(-2 i / rotary_dim), computed in 64 bits, for kv_append(rope=...).
    Any other table of that shape (scaled or extended positions) serves as well."""
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    a = torch.arange(length, dtype=torch.float64)[:, None] * base ** (-i / rotary_dim)
    return a.cos().float().to(device), a.sin().float().to(device)


def kv_append(k: torch.Tensor, v: torch.Tensor, K, V, seq_lens: Optional[torch.Tensor] = None,
              new_lens: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, rope=None, interleaved: bool = False,
              workspace: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Append new tokens' keys k and values v [B, T, Hkv, d] to the caches K and
    V, in place, rotating keys and queries by their positions; one launch.

    seq_lens (int32 [B] on the device): each sequence's length with its new
    tokens, as the step's other calls take it; None: the caches' whole length.
    new_lens (int32 [B]): how many of the T rows each sequence has; None: all.
    The tokens take the positions seq_lens - new_lens .. seq_lens - 1.
    q [B, T, Hq, d]: queries of the same positions, returned rotated (in q_out
    if given, which may be q itself).
    rope: (cos, sin) float32 [positions, r / 2], r <= d the rotary width, as
    rope_table makes them; None: no rotation.  interleaved: pairs (2i, 2i + 1)
    instead of (i, i + r / 2).
    workspace: where sequences that do not fit, and block-table entries outside
    the pool, are recorded (read_device_status); nothing of them is written.
    K and V: both dense tensors, PagedCache, Fp8Cache or Fp8PagedCache.

    The page metadata of K does not follow by itself: kv_meta_append with
    new_tokens=T and the same seq_lens and new_lens brings it up to date."""
    return (_binding or _load_binding()).kv_append(k, v, K, V, seq_lens, new_lens, q, q_out, rope,
                                                   interleaved, workspace)


def hot_state(B: int, Hkv: int, N: int, device) -> torch.Tensor:
    """A zeroed cross-step reuse state for decode_attn_select(hot=..., step=...)
    on caches of B sequences, Hkv kv heads and N tokens."""
    p = _params(None, B, Hkv, N, 64, None, None)
    n = int(lib().dkv_hot_state_bytes(ctypes.byref(p)))
    if n == 0:
        raise ValueError("invalid shape for a reuse state")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def hot_stats(state: torch.Tensor) -> tuple[int, int]:
    """(cache pages gathered, of them gathered at the previous step too), summed
    over the calls since the state was zeroed."""
    h = state[:16].cpu().view(torch.int64)
    return int(h[0]), int(h[1])


def kv_meta8_build(meta, page_size: int = PAGE_SIZE,
                   seq_lens: Optional[torch.Tensor] = None) -> Meta8:
    """8-bit page metadata from (meta_min, meta_max) [B, Hkv, P, d] (bf16 or
    fp16, as kv_meta_build returns it)."""
    mn, mx = meta
    if mn.dtype not in (torch.bfloat16, torch.float16) or mx.dtype != mn.dtype:
        raise ValueError("meta must be bf16 or fp16")
    if not mn.is_contiguous() or not mx.is_contiguous() or mn.shape != mx.shape:
        raise ValueError("meta must be two contiguous [B, Hkv, P, d] tensors")
    B, H, P, d = mn.shape
    m8 = Meta8(torch.empty(B, H, P, d, dtype=torch.uint8, device=mn.device),
               torch.empty(B, H, P, d, dtype=torch.uint8, device=mn.device),
               torch.empty(B, H, P, dtype=torch.float32, device=mn.device),
               torch.empty(B, H, P, dtype=torch.float32, device=mn.device))
    # N only sets P here: the largest N with ceil(N / S) = P
    p = _params(None, B, H, P * page_size, d, None, None, seq_lens=seq_lens)
    p.page_size = page_size
    _check(lib().dkv_kv_meta8_build(ctypes.byref(p), mn.data_ptr(), mx.data_ptr(),
                                    _dtype_code(mn.dtype), m8.code_min.data_ptr(),
                                    m8.code_max.data_ptr(), m8.lo.data_ptr(),
                                    m8.step.data_ptr(), _stream(mn)), "dkv_kv_meta8_build")
    return m8


def decode_attn_full(q, K, V, scale: Optional[float] = None,
                     out_dtype: torch.dtype = torch.float32,
                     out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, flags: int = 0,
                     seq_lens: Optional[torch.Tensor] = None):
    """Exact decode attention; returns out [B, Hq, d] (seq_lens: int32 [B] on the
    device, tokens each sequence attends; None: all N)."""
    return (_binding or _load_binding()).decode_attn_full(q, K, V, scale, out_dtype, out, workspace,
                                                          flags, seq_lens)


def decode_attn_select(q, K, V, meta, top_k: int, scale: Optional[float] = None,
                       out_dtype: torch.dtype = torch.float32,
                       out: Optional[torch.Tensor] = None, return_selected: bool = False,
                       selected: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, flags: int = 0,
                       group_select: bool = False, seq_lens: Optional[torch.Tensor] = None,
                       page_size: int = PAGE_SIZE, hot: Optional[torch.Tensor] = None,
                       step: int = 0):
    """Query-aware page-sparse decode attention over the top_k pages per q-head
    (group_select: one selection per kv head group, by the summed bound scores;
    page_size: tokens per metadata / selection page, as meta was built with;
    meta: (meta_min, meta_max), or a Meta8 from kv_meta8_build; hot, step: one
    step (1, 2, ...) of a decode loop keeping hot pages in L2, with a state
    from hot_state())."""
    if group_select:
        flags |= DKV_FLAG_GROUP_SELECT
    if not isinstance(meta, (tuple, list)):
        meta = tuple(meta)
    return (_binding or _load_binding()).decode_attn_select(
        q, K, V, meta, top_k, scale, out_dtype, out, return_selected, selected, workspace, flags,
        seq_lens, page_size, hot, step)


def decode_attn_topk_tokens(q, K, V, top_k: int, scale: Optional[float] = None,
                            out_dtype: torch.dtype = torch.float32,
                            out: Optional[torch.Tensor] = None, return_selected: bool = False,
                            selected: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None):
    """Token-level sparse decode attention: per q-head, the top_k tokens by the
    exact score q . k and attention over them only (K contiguous [B, Hkv, N, d])."""
    ks, B, H, N, d = _kv_struct(K)
    vs, B2, H2, N2, d2 = _kv_struct(V)
    if (B, H, N, d) != (B2, H2, N2, d2):
        raise ValueError("K and V shapes differ")
    if isinstance(K, torch.Tensor) and q.dtype != K.dtype:
        raise ValueError("q must have the cache's dtype")
    if out is None:
        out = torch.empty(B, q.shape[1], d, dtype=out_dtype, device=q.device)
    kk = min(int(top_k), N)
    if return_selected and selected is None:
        selected = torch.empty(B, q.shape[1], kk, dtype=torch.int32, device=q.device)
    p = _params(q, B, H, N, d, out, scale)
    nbytes = lib().dkv_workspace_bytes_tokens(ctypes.byref(p), int(top_k))
    ws = _workspace(nbytes, q.device, workspace)
    sel_ptr = selected.data_ptr() if selected is not None else None
    _check(lib().dkv_decode_attn_topk_tokens(ctypes.byref(p), q.data_ptr(), ctypes.byref(ks),
                                             ctypes.byref(vs), int(top_k), out.data_ptr(),
                                             _dtype_code(out.dtype), sel_ptr, ws.data_ptr(),
                                             nbytes, _stream(q)),
           "dkv_decode_attn_topk_tokens")
    return (out, selected) if return_selected else out


def workspace_bytes_tokens(B: int, Hq: int, Hkv: int, d: int, N: int, top_k: int) -> int:
    """Workspace bytes dkv_decode_attn_topk_tokens needs."""
    p = _Params()
    p.batch, p.num_q_heads, p.num_kv_heads, p.head_dim, p.seq_len = B, Hq, Hkv, d, N
    p.page_size, p.scale = PAGE_SIZE, 1.0
    n = lib().dkv_workspace_bytes_tokens(ctypes.byref(p), int(top_k))
    if n == 0:
        raise DkvError(2, "dkv_workspace_bytes_tokens")
    return int(n)


def kv_quant4(x: torch.Tensor) -> Q4Cache:
    """4-bit group-of-64 quantisation of an fp16 tensor [..., d] (contiguous)."""
    if x.dtype != torch.float16 or not x.is_contiguous():
        raise ValueError("kv_quant4 wants a contiguous fp16 tensor")
    d = x.shape[-1]
    rows = x.numel() // d
    codes = torch.empty(*x.shape[:-1], d // 2, dtype=torch.uint8, device=x.device)
    gmin = torch.empty(*x.shape[:-1], d // 64, dtype=torch.float16, device=x.device)
    gmax = torch.empty_like(gmin)
    _check(lib().dkv_kv_quant4(rows, d, x.data_ptr(), codes.data_ptr(), gmin.data_ptr(),
                               gmax.data_ptr(), _stream(x)), "dkv_kv_quant4")
    return Q4Cache(codes, gmin, gmax)


def kv_dequant4(q4: Q4Cache) -> torch.Tensor:
    codes, gmin, gmax = q4
    d = codes.shape[-1] * 2
    rows = codes.numel() // (d // 2)
    x = torch.empty(*codes.shape[:-1], d, dtype=torch.float16, device=codes.device)
    _check(lib().dkv_kv_dequant4(rows, d, codes.data_ptr(), gmin.data_ptr(), gmax.data_ptr(),
                                 x.data_ptr(), _stream(x)), "dkv_kv_dequant4")
    return x


def attn_ctas_per_sm(head_dim: int, dtype: torch.dtype = torch.bfloat16, q4: bool = False,
                     sparse: bool = False) -> int:
    """Resident CTAs per SM of the persistent attention kernel (a diagnostic)."""
    n = ctypes.c_int32(0)
    _check(lib().dkv_attn_ctas_per_sm(int(head_dim), _dtype_code(dtype),
                                      DKV_KV_Q4G64 if q4 else DKV_KV_DENSE, int(sparse),
                                      ctypes.byref(n)), "dkv_attn_ctas_per_sm")
    return int(n.value)


def read_device_status(workspace: torch.Tensor) -> int:
    """Synchronise and return (then clear) the device status word of a workspace.

    After a device error the workspace's merge counters may be left mid-count,
    so the whole workspace is zero-filled again, ready for the next call.
    """
    st = int(lib().dkv_read_device_status(workspace.data_ptr(), _stream(workspace)))
    if st != DKV_OK:
        workspace.zero_()
    return st

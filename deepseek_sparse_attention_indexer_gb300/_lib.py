"""ctypes binding of libdsa_gb300.so (the C ABI in include/dsa.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (PyTorch provides device memory and
streams); bf16 tensors may be torch.bfloat16 or 16-bit integer views of the
same bits.  If the library is missing or the device is not sm_103, calls raise
instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

import torch

from . import _build

DSA_OK = 0
DSA_OUT_F32 = 0     # attention output element types (include/dsa.h)
DSA_OUT_BF16 = 1
STATUS_NAMES = {
    0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED_SHAPE", 3: "DSA_ERR_MISALIGNED",
    4: "DSA_ERR_WORKSPACE_TOO_SMALL", 5: "DSA_ERR_CUDA", 6: "DSA_ERR_DEVICE_TIMEOUT",
    7: "DSA_ERR_DEVICE_BOUNDS", 8: "DSA_ERR_UNSUPPORTED_DEVICE", 9: "DSA_ERR_SCRATCH_TOO_SMALL",
}

# every symbol include/dsa.h declares, with (restype, argtypes)
_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
SIGNATURES = {
    "dsa_status_string": (ctypes.c_char_p, [ctypes.c_int32]),
    "dsa_abi_version": (ctypes.c_int, []),
    "dsa_indexer_scores": (ctypes.c_int32, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _I64, _P]),
    "dsa_topk_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "dsa_topk": (ctypes.c_int32, [_P, _I64, _P, _P, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "mla_sparse_attn_prefill": (ctypes.c_int32, [_P, _P, _P, _I, _I, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "mla_sparse_attn_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "mla_sparse_attn_decode": (ctypes.c_int32, [_P, _P, _P, _P, _I, _I, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "mla_sparse_attn_decode_noalloc": (ctypes.c_int32, [_P, _P, _P, _P, _I, _I, _I, _F, _P, _I, _P, _P]),
    "dsa_indexer_scores_paged": (ctypes.c_int32, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I64, _P]),
    "mla_sparse_attn_decode_paged": (ctypes.c_int32, [_P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _F, _P, _I, _P,
                                                      _P, _SZ, _P]),
    "mla_sparse_attn_prefill_paged": (ctypes.c_int32, [_P, _P, _P, _I, _I, _P, _I, _I, _I, _F, _P, _I, _P, _P, _SZ,
                                                       _P]),
    "mla_cache_write_q8": (ctypes.c_int32, [_P, _I64, _P, _F, _P, _I, _I, _P, _P, _I, _P, _P, _I64, _P]),
    "mla_cache_read_q8": (ctypes.c_int32, [_P, _P, _I64, _P, _I, _P, _P]),
    "mla_cache_read_q8_paged": (ctypes.c_int32, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "mla_sparse_attn_q8_workspace_size": (_SZ, [_I, _I]),
    "mla_sparse_attn_prefill_q8": (ctypes.c_int32, [_P, _P, _P, _P, _I, _I, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "mla_sparse_attn_prefill_q8_paged": (ctypes.c_int32, [_P, _P, _P, _P, _I, _I, _P, _I, _I, _I, _F, _P, _I, _P, _P,
                                                          _SZ, _P]),
    "mla_sparse_attn_decode_q8": (ctypes.c_int32, [_P, _P, _P, _P, _P, _I, _I, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "mla_sparse_attn_decode_q8_paged": (ctypes.c_int32, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _F, _P, _I,
                                                         _P, _P, _SZ, _P]),
    "dsa_indexer_norm_rope": (ctypes.c_int32, [_P, _I64, _P, _I64, _I, _P, _P, _P, _P, _F, _P, _I, _I, _P, _P, _I, _P,
                                               _P, _I64, _P]),
    "mla_value_up_proj": (ctypes.c_int32, [_P, _P, _I, _P, _P]),
    "dsa_indexer_source_layer": (ctypes.c_int, [_I, _I, _I]),
    "dsa_device_status": (ctypes.c_int32, [_P, ctypes.POINTER(ctypes.c_int32), _I]),
    "dsa_selftest_wait_timeout": (ctypes.c_int32, [_I, ctypes.c_uint64, _P]),
    "dsa_selftest_poll_timeout": (ctypes.c_int32, [_I, ctypes.c_uint32, _P]),
}

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


class DsaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)} ({status_string(code)})")


def lib_path() -> str:
    return _build.LIB_PATH


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the library (it must have been built: see __graft_entry__.build())."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or _build.LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"{p} is missing: build the CUDA library first "
                                   "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(p)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(lib, name)
                f.restype = res
                f.argtypes = args
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().dsa_status_string(code).decode()


def _check(fn: str, code: int):
    if code != DSA_OK:
        raise DsaError(fn, code)


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _is16(t: torch.Tensor) -> bool:
    return t.dtype in (torch.bfloat16, torch.int16, torch.uint16)


def _out_dtype(out: torch.Tensor) -> int:
    """The C ABI's out_dtype for an attention output tensor: float32, or bf16 (or a 16-bit view of it)."""
    if out.dtype == torch.float32:
        return DSA_OUT_F32
    if _is16(out):
        return DSA_OUT_BF16
    raise ValueError(f"attention output must be float32 or bf16, got {out.dtype}")


def _new_out(rows: int, device, dtype) -> torch.Tensor:
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"attention output must be float32 or bf16, got {dtype}")
    return torch.empty((rows, 64, 512), dtype=dtype, device=device)


# ----------------------------------------------------------------------------- entry points

def indexer_scores(q_idx: torch.Tensor, k_idx: torch.Tensor, w: torch.Tensor, q_pos0: torch.Tensor,
                   kv_len: torch.Tensor, scores: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """scores [B, L, ld] f32 from q_idx [B,L,32,128], k_idx [B,Nmax,128] (bf16), w [B,L,32] f32."""
    B, L, Hi, Di = q_idx.shape
    Nmax = k_idx.shape[1]
    assert _is16(q_idx) and _is16(k_idx) and w.dtype == torch.float32
    if scores is None:
        ld = (Nmax + 3) // 4 * 4
        scores = torch.empty((B, L, ld), dtype=torch.float32, device=q_idx.device)
    ld = scores.shape[-1]
    rc = load().dsa_indexer_scores(_ptr(q_idx), _ptr(k_idx), _ptr(w), _ptr(q_pos0), _ptr(kv_len),
                                   B, L, Nmax, _ptr(scores), ld, _stream(stream))
    _check("dsa_indexer_scores", rc)
    return scores


def topk(scores: torch.Tensor, q_pos0: torch.Tensor, kv_len: torch.Tensor, Nmax: int, top_k: int,
         idx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """idx [B, L, top_k] int32 (ascending key order, -1 padded)."""
    B, L, ld = scores.shape
    if idx is None:
        idx = torch.empty((B, L, top_k), dtype=torch.int32, device=scores.device)
    rc = load().dsa_topk(_ptr(scores), ld, _ptr(q_pos0), _ptr(kv_len), B, L, Nmax, top_k, _ptr(idx),
                         None, 0, _stream(stream))
    _check("dsa_topk", rc)
    return idx


def mla_sparse_attn_prefill(q: torch.Tensor, kv: torch.Tensor, idx: torch.Tensor, scale: float,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            want_lse: bool = False, stream=None, out_dtype=torch.float32):
    """out [L, 64, 512] (float32 by default, or bf16: the float32 result rounded; a given `out`
    decides) and lse [L, 64] f32, for q [L,64,576], kv [N,576], idx [L,top_k]."""
    L = q.shape[0]
    N = kv.shape[0]
    top_k = idx.shape[-1]
    assert _is16(q) and _is16(kv) and idx.dtype == torch.int32
    if out is None:
        out = _new_out(L, q.device, out_dtype)
    if lse is None and want_lse:
        lse = torch.empty((L, 64), dtype=torch.float32, device=q.device)
    rc = load().mla_sparse_attn_prefill(_ptr(q), _ptr(kv), _ptr(idx), L, N, top_k, float(scale), _ptr(out),
                                        _out_dtype(out), _ptr(lse), None, 0, _stream(stream))
    _check("mla_sparse_attn_prefill", rc)
    return (out, lse) if want_lse else out


def attn_workspace_size(B: int, top_k: int, is_decode: bool = True) -> int:
    return int(load().mla_sparse_attn_workspace_size(B, 1, top_k, 1 if is_decode else 0))


def mla_sparse_attn_decode(q: torch.Tensor, kv: torch.Tensor, kv_len: torch.Tensor, idx: torch.Tensor,
                           scale: float, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, want_lse: bool = False, stream=None,
                           out_dtype=torch.float32):
    """out [B, 64, 512] (float32 by default, or bf16) for q [B,64,576], kv [B,Nmax,576], kv_len [B],
    idx [B,top_k]."""
    B = q.shape[0]
    Nmax = kv.shape[1]
    top_k = idx.shape[-1]
    if out is None:
        out = _new_out(B, q.device, out_dtype)
    if lse is None and want_lse:
        lse = torch.empty((B, 64), dtype=torch.float32, device=q.device)
    ws_bytes = attn_workspace_size(B, top_k)
    if workspace is None:
        workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=q.device)
    rc = load().mla_sparse_attn_decode(_ptr(q), _ptr(kv), _ptr(kv_len), _ptr(idx), B, Nmax, top_k, float(scale),
                                       _ptr(out), _out_dtype(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                       _stream(stream))
    _check("mla_sparse_attn_decode", rc)
    return (out, lse) if want_lse else out


def mla_sparse_attn_decode_noalloc(q: torch.Tensor, kv: torch.Tensor, kv_len: torch.Tensor, idx: torch.Tensor,
                                   scale: float, out: Optional[torch.Tensor] = None,
                                   lse: Optional[torch.Tensor] = None, want_lse: bool = False, stream=None,
                                   out_dtype=torch.float32):
    """Decode attention without a workspace, for callers that may not allocate
    device memory: the library keeps the split partials in its own fixed device
    scratch (B <= 63).  Pass preallocated `out` (and `lse`) to allocate nothing
    here either.  Calls that overlap on the GPU share that scratch and race."""
    B = q.shape[0]
    Nmax = kv.shape[1]
    top_k = idx.shape[-1]
    if out is None:
        out = _new_out(B, q.device, out_dtype)
    if lse is None and want_lse:
        lse = torch.empty((B, 64), dtype=torch.float32, device=q.device)
    rc = load().mla_sparse_attn_decode_noalloc(_ptr(q), _ptr(kv), _ptr(kv_len), _ptr(idx), B, Nmax, top_k,
                                               float(scale), _ptr(out), _out_dtype(out), _ptr(lse), _stream(stream))
    _check("mla_sparse_attn_decode_noalloc", rc)
    return (out, lse) if want_lse else out


def indexer_scores_paged(q_idx: torch.Tensor, k_pool: torch.Tensor, w: torch.Tensor, q_pos0: torch.Tensor,
                         kv_len: torch.Tensor, block_table: torch.Tensor, page_size: int, Nmax: int,
                         scores: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """indexer_scores over a paged key cache: k_pool [num_pages * page_size, 128] bf16,
    block_table [B, bt_stride] int32 (pool page of each logical page of a sequence)."""
    B, L, Hi, Di = q_idx.shape
    assert _is16(q_idx) and _is16(k_pool) and w.dtype == torch.float32 and block_table.dtype == torch.int32
    num_pages = k_pool.shape[0] // page_size
    if scores is None:
        ld = (Nmax + 3) // 4 * 4
        scores = torch.empty((B, L, ld), dtype=torch.float32, device=q_idx.device)
    ld = scores.shape[-1]
    rc = load().dsa_indexer_scores_paged(_ptr(q_idx), _ptr(k_pool), _ptr(w), _ptr(q_pos0), _ptr(kv_len),
                                         _ptr(block_table), block_table.shape[1], page_size, num_pages,
                                         B, L, Nmax, _ptr(scores), ld, _stream(stream))
    _check("dsa_indexer_scores_paged", rc)
    return scores


def mla_sparse_attn_decode_paged(q: torch.Tensor, kv_pool: torch.Tensor, kv_len: torch.Tensor,
                                 block_table: torch.Tensor, page_size: int, idx: torch.Tensor, scale: float,
                                 Nmax: int, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, want_lse: bool = False, stream=None,
                                 out_dtype=torch.float32):
    """mla_sparse_attn_decode over a paged cache: kv_pool [num_pages * page_size, 576] bf16,
    block_table [B, bt_stride] int32; idx holds logical key positions."""
    B = q.shape[0]
    top_k = idx.shape[-1]
    assert _is16(q) and _is16(kv_pool) and idx.dtype == torch.int32 and block_table.dtype == torch.int32
    num_pages = kv_pool.shape[0] // page_size
    if out is None:
        out = _new_out(B, q.device, out_dtype)
    if lse is None and want_lse:
        lse = torch.empty((B, 64), dtype=torch.float32, device=q.device)
    ws_bytes = attn_workspace_size(B, top_k)
    if workspace is None:
        workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=q.device)
    rc = load().mla_sparse_attn_decode_paged(_ptr(q), _ptr(kv_pool), _ptr(kv_len), _ptr(block_table),
                                             block_table.shape[1], page_size, num_pages, _ptr(idx), B, Nmax,
                                             top_k, float(scale), _ptr(out), _out_dtype(out), _ptr(lse),
                                             _ptr(workspace),
                                             workspace.numel(), _stream(stream))
    _check("mla_sparse_attn_decode_paged", rc)
    return (out, lse) if want_lse else out


def mla_sparse_attn_prefill_paged(q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor,
                                  page_size: int, idx: torch.Tensor, scale: float, N: int,
                                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                  want_lse: bool = False, stream=None, out_dtype=torch.float32):
    """mla_sparse_attn_prefill over one sequence's paged cache: kv_pool [num_pages * page_size, 576]
    bf16, block_table int32 with ceil(N / page_size) entries; idx holds logical key positions < N."""
    L = q.shape[0]
    top_k = idx.shape[-1]
    assert _is16(q) and _is16(kv_pool) and idx.dtype == torch.int32 and block_table.dtype == torch.int32
    num_pages = kv_pool.shape[0] // page_size
    if out is None:
        out = _new_out(L, q.device, out_dtype)
    if lse is None and want_lse:
        lse = torch.empty((L, 64), dtype=torch.float32, device=q.device)
    rc = load().mla_sparse_attn_prefill_paged(_ptr(q), _ptr(kv_pool), _ptr(block_table), page_size, num_pages,
                                              _ptr(idx), L, N, top_k, float(scale), _ptr(out), _out_dtype(out),
                                              _ptr(lse), None, 0, _stream(stream))
    _check("mla_sparse_attn_prefill_paged", rc)
    return (out, lse) if want_lse else out


# ----------------------------------------------------------------------------- the 8-bit latent cache

Q8_ROW = 640        # bytes of a cache row: 512 e4m3 latent dims | 64 bf16 rope dims
NORMS = {"rms": 0, "layer": 1}


# The checks below are a few attribute reads a tensor: a decode step calls these functions once a layer and
# token, and a call that takes longer on the host than on the device bounds the step.
_BITS16 = frozenset((torch.bfloat16, torch.int16, torch.uint16))
_F32 = frozenset((torch.float32,))
_I32 = frozenset((torch.int32,))
_U8 = frozenset((torch.uint8,))


@functools.lru_cache(maxsize=4096)
def _q8_workspace_bytes(dev: int, rows: int, top_k: int) -> int:
    """The library's answer for a device and two sizes."""
    return int(load().mla_sparse_attn_q8_workspace_size(rows, top_k))


def _current_device() -> int:
    return torch.cuda.current_device()


def _bad(what: str):
    raise ValueError(what)


def _p(t: torch.Tensor, dev: int, dtypes, n: int, what: str) -> int:
    """Device pointer of a contiguous tensor of n elements on the current device, where the kernels launch."""
    if t.dtype in dtypes and t.numel() == n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what}: expected a contiguous tensor of {n} elements of {'/'.join(map(str, sorted(dtypes, key=str)))} "
                     f"on the current CUDA device, got {tuple(t.shape)} {t.dtype} on {t.device}")


def _opt(t: Optional[torch.Tensor], dev: int, dtypes, n: int, what: str) -> Optional[int]:
    return None if t is None else _p(t, dev, dtypes, n, what)


def _rows(t: torch.Tensor, dev: int, inner, what: str):
    """(pointer, row stride in elements) of a 16-bit tensor whose rows, one a token, are contiguous but may lie
    apart: a slice of a wider projection's output.  inner: the strides inside a row."""
    s = t.stride()
    if t.dtype in _BITS16 and s[1:] == inner and t.get_device() == dev:
        return t.data_ptr(), s[0]
    raise ValueError(f"{what}: expected 16-bit rows of strides {inner} on the current CUDA device, got {tuple(t.shape)} "
                     f"{t.dtype} of strides {s} on {t.device}")


def _stream_on(dev: int, stream) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """A tensor for a call on `stream`, from that stream's memory: neither its earlier nor its next user
    overlaps the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))):
        return torch.empty(shape, dtype=dtype, device=device)


def _q8_rows(cache: torch.Tensor) -> int:
    """Rows of an 8-bit cache (uint8, last dim 640)."""
    if cache.shape[-1] != Q8_ROW:
        _bad("the cache is uint8 with rows of 640 bytes")
    return cache.numel() // Q8_ROW


def _max_pos(cos_sin: torch.Tensor) -> int:
    if cos_sin.dim() != 2 or cos_sin.shape[1] != 64:
        _bad("cos_sin is float32 [max_pos, 64]")
    return cos_sin.shape[0]


def mla_cache_write_q8(kv_a: torch.Tensor, norm_w: torch.Tensor, eps: float, cos_sin: torch.Tensor, pos: torch.Tensor,
                       slots: torch.Tensor, cache: torch.Tensor, cache_scale: torch.Tensor, interleave: bool = True,
                       stream=None) -> None:
    """Latent rows of new tokens into the 8-bit cache: norm, rotation, quantisation and scatter.

    kv_a [R, 576] bf16 (rows may be strided), norm_w [512] f32, cos_sin [max_pos, 64] f32 (32 cosines |
    32 sines a position), pos and slots [R] int32 (a negative slot skips the token; slots differ), cache
    uint8 [..., 640], cache_scale f32 [...]."""
    dev = _current_device()
    R, width = kv_a.shape
    if width != 576:
        _bad("kv_a is [R, 576]")
    p, ld = _rows(kv_a, dev, (1,), "kv_a")
    rows, n_pos = _q8_rows(cache), _max_pos(cos_sin)
    rc = (_lib or load()).mla_cache_write_q8(
        p, ld if R > 1 else 576, _p(norm_w, dev, _F32, 512, "norm_w"), eps, _p(cos_sin, dev, _F32, n_pos * 64, "cos_sin"), n_pos,
        1 if interleave else 0, _p(pos, dev, _I32, R, "pos"), _p(slots, dev, _I32, R, "slots"), R,
        _p(cache, dev, _U8, rows * Q8_ROW, "cache"), _p(cache_scale, dev, _F32, rows, "cache_scale"), rows,
        _stream_on(dev, stream))
    if rc:
        raise DsaError("mla_cache_write_q8", rc)


def mla_cache_read_q8(cache: torch.Tensor, cache_scale: torch.Tensor, slots: torch.Tensor,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [R, 576] bf16: the rows `slots` [R] int32 of the 8-bit cache (zeros for a negative slot)."""
    dev = _current_device()
    R, rows = slots.numel(), _q8_rows(cache)
    if out is None:
        out = _new((R, 576), torch.bfloat16, cache.device, stream)
    rc = (_lib or load()).mla_cache_read_q8(
        _p(cache, dev, _U8, rows * Q8_ROW, "cache"), _p(cache_scale, dev, _F32, rows, "cache_scale"), rows,
        _p(slots, dev, _I32, R, "slots"), R, _p(out, dev, _BITS16, R * 576, "out"), _stream_on(dev, stream))
    if rc:
        raise DsaError("mla_cache_read_q8", rc)
    return out


def _table(block_table: torch.Tensor, B: int) -> int:
    """Pages a sequence of a [B, pages] table."""
    if block_table.dim() != 2 or block_table.shape[0] != B:
        _bad("block_table is int32 [B, pages]")
    return block_table.shape[1]


def mla_cache_read_q8_paged(cache: torch.Tensor, cache_scale: torch.Tensor, kv_len: torch.Tensor,
                            block_table: torch.Tensor, page_size: int, Nmax: int,
                            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [B, Nmax, 576] bf16: the kv_len[b] rows of each sequence of a paged 8-bit cache; later rows
    of a given `out` stay as they are (a new one has zeros there)."""
    dev = _current_device()
    B, rows = kv_len.numel(), _q8_rows(cache)
    stride = _table(block_table, B)
    if out is None:
        out = _new((B, Nmax, 576), torch.bfloat16, cache.device, stream)
        with torch.cuda.stream(torch.cuda.ExternalStream(_stream_on(dev, stream))):
            out.zero_()
    rc = (_lib or load()).mla_cache_read_q8_paged(
        _p(cache, dev, _U8, rows * Q8_ROW, "cache"), _p(cache_scale, dev, _F32, rows, "cache_scale"),
        _p(kv_len, dev, _I32, B, "kv_len"), _p(block_table, dev, _I32, B * stride, "block_table"), stride, page_size,
        rows // page_size if page_size > 0 else 0, B, Nmax, _p(out, dev, _BITS16, B * Nmax * 576, "out"),
        _stream_on(dev, stream))
    if rc:
        raise DsaError("mla_cache_read_q8_paged", rc)
    return out


def _attn_q8(q, cache, cache_scale, idx, out, lse, want_lse, out_dtype, stream):
    """Checks and output buffers the 8-bit attention calls share: the device, the sizes, the tensors to return
    and the pointers of q, cache, cache_scale, idx, out, lse."""
    dev = _current_device()
    rows, heads, width = q.shape
    if heads != 64 or width != 576:
        _bad("q is bf16 [rows, 64, 576]")
    top_k, n = idx.shape[-1], _q8_rows(cache)
    if out is None:
        if out_dtype not in (torch.float32, torch.bfloat16):
            _bad(f"attention output must be float32 or bf16, got {out_dtype}")
        out = _new((rows, 64, 512), out_dtype, q.device, stream)
    if lse is None and want_lse:
        lse = _new((rows, 64), torch.float32, q.device, stream)
    f32 = out.dtype is torch.float32
    return (dev, rows, top_k, n, out, lse, DSA_OUT_F32 if f32 else DSA_OUT_BF16, _p(q, dev, _BITS16, rows * 36864, "q"),
            _p(cache, dev, _U8, n * Q8_ROW, "cache"), _p(cache_scale, dev, _F32, n, "cache_scale"),
            _p(idx, dev, _I32, rows * top_k, "idx"), _p(out, dev, _F32 if f32 else _BITS16, rows * 32768, "out"),
            _opt(lse, dev, _F32, rows * 64, "lse"))


def attn_q8_workspace_size(rows: int, top_k: int) -> int:
    """Bytes an attention call of so many queries over an 8-bit cache takes on the current device (0: none)."""
    return _q8_workspace_bytes(_current_device(), rows, top_k)


# Workspaces of the attention by (device, stream), a set for each thread: calls that one thread makes on one stream run in
# order, so they may share one; a call is several kernels, and another thread's may come between them.  Not used while a
# graph is being captured (its buffers live in the graph's own pool, one for each call) nor for a given stream.
class _Workspaces(threading.local):
    def __init__(self):
        self.by_stream = {}


_workspaces = _Workspaces()


def _q8_workspace(workspace, rows, top_k, dev, device, stream):
    """(tensor to keep until the call, pointer, bytes)."""
    if workspace is None:
        need = _q8_workspace_bytes(dev, rows, top_k)
        if need == 0:
            return None, None, 0
        if stream is None and not torch.cuda.is_current_stream_capturing():
            key = (dev, torch._C._cuda_getCurrentRawStream(dev))
            by_stream = _workspaces.by_stream
            workspace = by_stream.get(key)
            if workspace is None or workspace.nbytes < need:
                workspace = by_stream[key] = torch.empty((need,), dtype=torch.uint8, device=device)
        else:
            workspace = _new((need,), torch.uint8, device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _bad("the workspace is contiguous on the current CUDA device")
    return workspace, workspace.data_ptr(), workspace.nbytes


def mla_sparse_attn_prefill_q8(q: torch.Tensor, cache: torch.Tensor, cache_scale: torch.Tensor, idx: torch.Tensor,
                               scale: float, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                               want_lse: bool = False, stream=None, out_dtype=torch.float32,
                               workspace: Optional[torch.Tensor] = None):
    """mla_sparse_attn_prefill over an 8-bit cache: cache uint8 [N, 640], cache_scale f32 [N]."""
    dev, L, top_k, N, out, lse, od, pq, pc, ps, pi, po, pl = _attn_q8(q, cache, cache_scale, idx, out, lse, want_lse,
                                                                      out_dtype, stream)
    workspace, pw, n_ws = _q8_workspace(workspace, L, top_k, dev, q.device, stream)
    rc = (_lib or load()).mla_sparse_attn_prefill_q8(pq, pc, ps, pi, L, N, top_k, scale, po, od, pl, pw, n_ws,
                                                     _stream_on(dev, stream))
    if rc:
        raise DsaError("mla_sparse_attn_prefill_q8", rc)
    return (out, lse) if want_lse else out


def mla_sparse_attn_prefill_q8_paged(q: torch.Tensor, cache: torch.Tensor, cache_scale: torch.Tensor,
                                     block_table: torch.Tensor, page_size: int, idx: torch.Tensor, scale: float, N: int,
                                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                     want_lse: bool = False, stream=None, out_dtype=torch.float32,
                                     workspace: Optional[torch.Tensor] = None):
    """mla_sparse_attn_prefill_paged over an 8-bit pool: cache uint8 [num_pages * page_size, 640]."""
    dev, L, top_k, n, out, lse, od, pq, pc, ps, pi, po, pl = _attn_q8(q, cache, cache_scale, idx, out, lse, want_lse,
                                                                      out_dtype, stream)
    pages = block_table.numel()
    if page_size > 0 and pages < -(-N // page_size):
        _bad("block_table holds ceil(N / page_size) pages")
    workspace, pw, n_ws = _q8_workspace(workspace, L, top_k, dev, q.device, stream)
    rc = (_lib or load()).mla_sparse_attn_prefill_q8_paged(
        pq, pc, ps, _p(block_table, dev, _I32, pages, "block_table"), page_size, n // page_size if page_size > 0 else 0, pi,
        L, N, top_k, scale, po, od, pl, pw, n_ws, _stream_on(dev, stream))
    if rc:
        raise DsaError("mla_sparse_attn_prefill_q8_paged", rc)
    return (out, lse) if want_lse else out


def mla_sparse_attn_decode_q8(q: torch.Tensor, cache: torch.Tensor, cache_scale: torch.Tensor, kv_len: torch.Tensor,
                              idx: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
                              lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                              want_lse: bool = False, stream=None, out_dtype=torch.float32):
    """mla_sparse_attn_decode over an 8-bit cache: cache uint8 [B, Nmax, 640], cache_scale f32 [B, Nmax]."""
    dev, B, top_k, n, out, lse, od, pq, pc, ps, pi, po, pl = _attn_q8(q, cache, cache_scale, idx, out, lse, want_lse,
                                                                      out_dtype, stream)
    if cache.dim() != 3 or cache.shape[0] != B:
        _bad("the cache is uint8 [B, Nmax, 640]")
    workspace, pw, n_ws = _q8_workspace(workspace, B, top_k, dev, q.device, stream)
    rc = (_lib or load()).mla_sparse_attn_decode_q8(
        pq, pc, ps, _p(kv_len, dev, _I32, B, "kv_len"), pi, B, cache.shape[1], top_k, scale, po, od, pl,
        pw, n_ws, _stream_on(dev, stream))
    if rc:
        raise DsaError("mla_sparse_attn_decode_q8", rc)
    return (out, lse) if want_lse else out


def mla_sparse_attn_decode_q8_paged(q: torch.Tensor, cache: torch.Tensor, cache_scale: torch.Tensor,
                                    kv_len: torch.Tensor, block_table: torch.Tensor, page_size: int, idx: torch.Tensor,
                                    scale: float, Nmax: int, out: Optional[torch.Tensor] = None,
                                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                    want_lse: bool = False, stream=None, out_dtype=torch.float32):
    """mla_sparse_attn_decode_paged over an 8-bit pool: cache uint8 [num_pages * page_size, 640]."""
    dev, B, top_k, n, out, lse, od, pq, pc, ps, pi, po, pl = _attn_q8(q, cache, cache_scale, idx, out, lse, want_lse,
                                                                      out_dtype, stream)
    stride = _table(block_table, B)
    workspace, pw, n_ws = _q8_workspace(workspace, B, top_k, dev, q.device, stream)
    rc = (_lib or load()).mla_sparse_attn_decode_q8_paged(
        pq, pc, ps, _p(kv_len, dev, _I32, B, "kv_len"), _p(block_table, dev, _I32, B * stride, "block_table"), stride,
        page_size, n // page_size if page_size > 0 else 0, pi, B, Nmax, top_k, scale, po, od, pl, pw, n_ws, _stream_on(dev, stream))
    if rc:
        raise DsaError("mla_sparse_attn_decode_q8_paged", rc)
    return (out, lse) if want_lse else out


def indexer_norm_rope(q: torch.Tensor, k: torch.Tensor, k_w: Optional[torch.Tensor], k_b: Optional[torch.Tensor],
                      eps: float, cos_sin: torch.Tensor, pos: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                      q_w: Optional[torch.Tensor] = None, q_b: Optional[torch.Tensor] = None, norm: str = "layer",
                      interleave: bool = True, q_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The indexer's queries and keys of new tokens: norm and rotation of each head, the queries
    returned as [R, 32, 128] bf16, the keys scattered to k_cache.

    q [R, 32, 128] and k [R, 128] bf16 (rows may be strided), weights and biases f32 [128] or None (not
    normalised / nothing added), cos_sin [max_pos, 64] f32, pos and slots [R] int32 (a negative slot
    writes no key; slots differ), k_cache bf16 [..., 128], norm "rms" or "layer"."""
    dev = _current_device()
    R, heads, width = q.shape
    if heads != 32 or width != 128 or k.shape != (R, 128) or k_cache.shape[-1] != 128:
        _bad("q is [R, 32, 128], k [R, 128], k_cache [..., 128]")
    kind = NORMS.get(norm, -1)
    if kind < 0:
        _bad(f"norm is one of {sorted(NORMS)}")
    qp, q_ld = _rows(q, dev, (128, 1), "q")
    kp, k_ld = _rows(k, dev, (1,), "k")
    n_pos, rows = _max_pos(cos_sin), k_cache.numel() // 128
    if q_out is None:
        q_out = _new((R, 32, 128), torch.bfloat16, q.device, stream)
    rc = (_lib or load()).dsa_indexer_norm_rope(
        qp, q_ld if R > 1 else 4096, kp, k_ld if R > 1 else 128, kind, _opt(q_w, dev, _F32, 128, "q_w"),
        _opt(q_b, dev, _F32, 128, "q_b"), _opt(k_w, dev, _F32, 128, "k_w"), _opt(k_b, dev, _F32, 128, "k_b"), eps,
        _p(cos_sin, dev, _F32, n_pos * 64, "cos_sin"), n_pos, 1 if interleave else 0, _p(pos, dev, _I32, R, "pos"),
        _p(slots, dev, _I32, R, "slots"), R, _p(q_out, dev, _BITS16, R * 4096, "q_out"),
        _p(k_cache, dev, _BITS16, rows * 128, "k_cache"), rows, _stream_on(dev, stream))
    if rc:
        raise DsaError("dsa_indexer_norm_rope", rc)
    return q_out


def mla_value_up_proj(o: torch.Tensor, wv_b: torch.Tensor, v: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """v [R, 64, 256] bf16 = per head o[r, h, :] (512 latent dims) times wv_b[h]^T,
    for o [R, 64, 512] and wv_b [64, 256, 512] (bf16)."""
    R = o.shape[0]
    assert _is16(o) and _is16(wv_b)
    assert tuple(o.shape[1:]) == (64, 512) and tuple(wv_b.shape) == (64, 256, 512)
    if v is None:
        v = torch.empty((R, 64, 256), dtype=torch.bfloat16, device=o.device)
    rc = load().mla_value_up_proj(_ptr(o), _ptr(wv_b), R, _ptr(v), _stream(stream))
    _check("mla_value_up_proj", rc)
    return v


def indexer_source_layer(layer: int, topk_freq: int = 4, skip_offset: int = 3) -> int:
    """The layer whose top-k selection `layer` attends with (itself if it runs the
    indexer); GLM-5.x shares the indexer with index_topk_freq 4, index_skip_topk_offset 3."""
    r = load().dsa_indexer_source_layer(layer, topk_freq, skip_offset)
    if r < 0:
        raise ValueError(f"invalid layer schedule arguments ({layer}, {topk_freq}, {skip_offset})")
    return r


def selftest_wait_timeout(spin: bool = False, limit_ns: int = 1_000_000, stream=None) -> None:
    """Launch the failure-detection self-test: one thread waits, with the kernels' bounded wait
    (spin: the polling form), on an mbarrier nothing arrives on; the wait gives up after limit_ns
    and the timeout shows in device_status()."""
    rc = load().dsa_selftest_wait_timeout(1 if spin else 0, ctypes.c_uint64(int(limit_ns)), _stream(stream))
    _check("dsa_selftest_wait_timeout", rc)


def selftest_poll_timeout(warp: bool = False, polls: int = 1 << 16, stream=None) -> None:
    """The same for the waits of the 8-bit attention, which give up after a number of polls: one
    thread's, or (warp) a warp's look at several barriers at once."""
    rc = load().dsa_selftest_poll_timeout(1 if warp else 0, int(polls), _stream(stream))
    _check("dsa_selftest_poll_timeout", rc)


def device_status(reset: bool = True, stream=None) -> int:
    code = ctypes.c_int32(0)
    rc = load().dsa_device_status(_stream(stream), ctypes.byref(code), 1 if reset else 0)
    _check("dsa_device_status", rc)
    return code.value

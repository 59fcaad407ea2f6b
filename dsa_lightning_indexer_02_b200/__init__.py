"""Python binding of libdsa.so (the C ABI in include/dsa.h): argument marshalling only.

Every function here takes torch CUDA tensors, checks their dtype/shape/contiguity, and passes
raw device pointers, sizes and the current CUDA stream to the C entry point of the same name.
All computation runs in the library's CUDA kernels; there is no fallback of any kind: if the
library is missing this module raises at import time.

Shapes follow the C header (bf16 unless stated; every shape is checked before the call):
  dsa_index(qI [Lq,HI,64], kI [Lk,64], w [Lq,HI], q_pos0, scores fp32 [Lq, ld])
  dsa_topk(scores fp32 [Lq, ld], q_pos0, k, idx int32 [Lq,k], window=0)
  dsa_sparse_attn(q [Lq,Hq,128], k/v [Lk,Hkv,128], idx int32 [Lq,topk], q_pos0, scale, out [Lq,Hq,128],
                  lse fp32 [Lq,Hq] = None)
  dsa_prefill(q [L,Hq,128], k/v [>=L,Hkv,128], qI [L,HI,64], kI [>=L,64], w [L,HI], topk, scale,
              out [L,Hq,128], idx_out int32 [L,topk] = None, ws=None, window=0)
  dsa_prefill_rows(q_rows [R,..], k, v, qI_rows [R,..], kI, w_rows [R,HI], row0, topk, scale, out_rows,
                   idx_rows=None, ws=None, window=0)      (k/v/kI cover rows 0 .. row0+R-1)
  dsa_indexer_kl(q [L,Hq,128], k [>=L,Hkv,128], qI [L,HI,64], kI [>=L,64], w [L,HI], scale, kl fp32 [>=L])
  dsa_decode(q [B,Hq,128], qI [B,HI,64], w [B,HI], k_new/v_new [B,Hkv,128], kI_new [B,64],
             k_cache/v_cache [B,Lmax,Hkv,128], kI_cache [B,Lmax,64], ctx_len int32 [B], topk, scale,
             out [B,Hq,128], idx_out int32 [B,topk] = None, ws=None, update_ctx=False)
  dsa_rope(x [T,H,D] bf16 or fp32, out [T,H,D], inv_freq fp64 [R/2], pos int32 [T] = None, pos0=0,
           rot_offset=0, interleaved=False, mscale=1.0, inverse=False)      (x, out: strides free)
  dsa_kv_append(k_new/v_new [N,Hkv,128] (strides free), k_pages/v_pages float8_e4m3fn or int8
                [pages,page,Hkv,128], k_scale/v_scale fp32 [pages,Hkv], page_table int32 [B,max_pages],
                ctx_len int32 [B], cu_new int32 [B+1] = None, inv_freq fp64 [R/2] = None,
                rope_pos int32 [N] = None, rot_offset=0, interleaved=False, mscale=1.0)
  dsa_paged_attn(q [T,Hq,128], k_pages, v_pages, k_scale, v_scale, page_table, n_keys int32 [T], scale,
                 out [T,Hq,128], seq int32 [T] = None, idx int32 [T,topk] = None, lse fp32 [T,Hq] = None, ws=None)
Every tensor must be on the current CUDA device, and contiguous where "strides free" does not stand.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "dsa.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; g.build()'` "
                      "or `python dsa_lightning_indexer_02_b200/build.py` (needs nvcc)")

_lib = ctypes.CDLL(LIB_PATH)

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_WORKSPACE, DSA_ERR_CUDA, DSA_ERR_TIMEOUT, \
    DSA_ERR_DEVICE_INPUT = range(7)
DSA_OP_INDEX, DSA_OP_TOPK, DSA_OP_SPARSE_ATTN, DSA_OP_PREFILL, DSA_OP_DECODE, DSA_OP_INDEXER_KL, \
    DSA_OP_PAGED_ATTN = range(7)
DSA_BF16, DSA_FP32 = range(2)
DSA_ROPE_HALF, DSA_ROPE_INTERLEAVED = range(2)
DSA_KV_E4M3, DSA_KV_INT8 = range(2)
ROPE_SCALINGS = ("plain", "linear", "ntk", "yarn")
PROFILE_KINDS = ("indexer", "topk", "sparse_attn", "combine", "decode_append", "advance", "selftest", "kl", "rope",
                 "kv_append", "paged_attn")

_p, _i, _i64, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_d = ctypes.c_double
_SIGS = {
    "dsa_status_string": (ctypes.c_char_p, [_i]),
    "dsa_version": (_i, []),
    "dsa_index": (_i, [_p, _p, _p, _i, _i64, _i, _i, _i64, _p, _i64, _p]),
    "dsa_topk": (_i, [_p, _i64, _i, _i64, _i, _p, _p, _sz, _p]),
    "dsa_topk_window": (_i, [_p, _i64, _i, _i64, _i, _i64, _p, _p]),
    "dsa_sparse_attn": (_i, [_p, _p, _p, _p, _i, _i64, _i64, _i, _i, _i, _i, _f, _p, _p, _p]),
    "dsa_sparse_attn_dedup": (_i, [_p, _p, _p, _p, _i, _i64, _i64, _i, _i, _i, _i, _f, _p, _p, _p]),
    "dsa_prefill": (_i, [_p, _p, _p, _p, _p, _p, _i64, _i, _i, _i, _i, _i, _i, _f, _p, _p, _p, _sz, _p]),
    "dsa_prefill_rows": (_i, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i, _i, _i, _i, _i, _i, _i64, _f, _p, _p, _p,
                              _sz, _p]),
    "dsa_prefill_window": (_i, [_p, _p, _p, _p, _p, _p, _i64, _i, _i, _i, _i, _i, _i, _i64, _f, _p, _p, _p, _sz,
                                _p]),
    "dsa_decode": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i64, _i, _i, _i, _i, _i, _i, _f, _i,
                        _p, _p, _p, _sz, _p]),
    "dsa_decode_noalloc": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i64, _i, _i, _i, _i, _i, _i, _f, _i,
                                _p, _p, _p]),
    "dsa_decode_noalloc_scratch_bytes": (_sz, []),
    "dsa_indexer_kl": (_i, [_p, _p, _p, _p, _p, _i64, _i, _i, _i, _i, _i, _f, _p, _p, _sz, _p]),
    "dsa_rope": (_i, [_p, _i, _i64, _i, _i, _i64, _i64, _p, _i64, _p, _i, _i, _i, _f, _i, _p, _i64, _i64, _p]),
    "dsa_rope_freqs": (_i, [_i, _d, _i, _d, _d, _d, _d, _p, _p]),
    "dsa_kv_append": (_i, [_p, _p, _i64, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _i, _i, _i, _f, _i, _p, _p, _p, _p,
                           _p, _i, _i, _i, _i, _i, _i, _p]),
    "dsa_paged_attn": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f, _p, _p,
                            _p, _sz, _p]),
    "dsa_workspace_size": (_sz, [_i, _i64, _i, _i, _i, _i]),
    "dsa_sync_status": (_i, [_p]),
    "dsa_error_site": (ctypes.c_uint, []),
    "dsa_profile_begin": (None, []),
    "dsa_profile_end": (_i, [_p, _p]),
    "dsa_profile_end_kinds": (_i, [_i, _p, _p]),
    "dsa_launch_count": (_i64, []),
    "dsa_read_counters": (_i, [_p, _i, _i]),
    "dsa_selftest_timeout": (_i, [_i64, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def header_symbols() -> list[str]:
    """Function names declared in include/dsa.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dsa_[a-z_]+)\s*\(", text)))


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def status_string(status: int) -> str:
    return _lib.dsa_status_string(int(status)).decode()


def version() -> int:
    return int(_lib.dsa_version())


def _check(status: int, where: str) -> None:
    if status != DSA_OK:
        raise DSAError(status, where)


def _stream(stream=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_fast = None


class _Ctypes:
    """Stands in for the marshalling module: declines every call, which is then made through ctypes."""
    rope = kv_append = paged_attn = staticmethod(lambda *operands: None)


def _native():
    """The marshalling module: the checks below and the C call in one step, for operands that need no error
    message (None otherwise).  Loaded with the first call that uses it, since it needs torch; where it was not
    built for this interpreter and torch, calls go through ctypes, with a warning."""
    global _fast
    import importlib.util
    import warnings
    from . import build
    path = build.marshal_path()
    try:
        spec = importlib.util.spec_from_file_location(__name__ + "._marshal", path)
        _fast = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_fast)
    except ImportError as e:
        warnings.warn(f"{path} is not built ({e}): calls go through ctypes, some 10 us slower each", RuntimeWarning)
        _fast = _Ctypes
    return _fast


def _need(t, dtype, name, shape):
    """One tensor argument: its type, dtype, shape (None: any extent) and contiguity.  The
    library reads every size from the leading operand, so an operand whose shape disagrees would
    let a kernel read or write past it: refuse it here."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(e is not None and int(e) != n for e, n in zip(shape, t.shape)):
        want = ", ".join("*" if e is None else str(int(e)) for e in shape)
        raise ValueError(f"{name} must have shape [{want}], got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _at_least(t, name, dim, n):
    if t.shape[dim] < n:
        raise ValueError(f"{name}.shape[{dim}] must be >= {n}, got {t.shape[dim]}")


def _on_device(**tensors):
    """Every tensor argument on the current CUDA device (where the library launches)."""
    import torch
    ts = {k: t for k, t in tensors.items() if t is not None}
    for k, t in ts.items():
        if not t.is_cuda:
            raise ValueError(f"{k} must be a CUDA tensor")
    dev = torch.cuda.current_device()
    for k, t in ts.items():
        if t.device.index != dev:
            raise ValueError(f"{k} is on {t.device}, the current device is cuda:{dev}")


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def workspace_size(op: int, L: int, B: int = 1, Hq: int = 32, HI: int = 32, topk: int = 2048) -> int:
    return int(_lib.dsa_workspace_size(op, L, B, Hq, HI, topk))


def _workspace(ws, op, L, B, Hq, HI, topk, like):
    import torch
    if ws is None:
        return torch.empty(workspace_size(op, L, B, Hq, HI, topk), dtype=torch.uint8, device=like.device)
    if not isinstance(ws, torch.Tensor) or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous torch.Tensor")
    return ws


def dsa_index(qI, kI, w, q_pos0: int, scores, stream=None) -> None:
    """scores[i, s] for the Lq rows of qI (positions q_pos0 + i) and every causal key s."""
    import torch
    bf = torch.bfloat16
    _need(qI, bf, "qI", (None, None, None))
    Lq, HI, dI = qI.shape
    _need(kI, bf, "kI", (None, dI)), _need(w, bf, "w", (Lq, HI)), _need(scores, torch.float32, "scores", (Lq, None))
    _on_device(qI=qI, kI=kI, w=w, scores=scores)
    st = _lib.dsa_index(_ptr(qI), _ptr(kI), _ptr(w), Lq, kI.shape[0], HI, dI, q_pos0, _ptr(scores),
                        scores.shape[1], _stream(stream))
    _check(st, "dsa_index")


def dsa_topk(scores, q_pos0: int, k: int, idx, window: int = 0, stream=None) -> None:
    """idx[i] = the top-k keys of score row i (row i holds q_pos0 + i + 1 valid scores)."""
    import torch
    _need(scores, torch.float32, "scores", (None, None))
    Lq = scores.shape[0]
    _need(idx, torch.int32, "idx", (Lq, k))
    _on_device(scores=scores, idx=idx)
    if window:
        st = _lib.dsa_topk_window(_ptr(scores), scores.shape[1], Lq, q_pos0, k, window, _ptr(idx), _stream(stream))
        _check(st, "dsa_topk_window")
        return
    st = _lib.dsa_topk(_ptr(scores), scores.shape[1], Lq, q_pos0, k, _ptr(idx), None, 0, _stream(stream))
    _check(st, "dsa_topk")


def dsa_sparse_attn(q, k, v, idx, q_pos0: int, scale: float, out, lse=None, stream=None) -> None:
    """Attention of the Lq rows of q over the keys that idx selects for each row."""
    import torch
    bf = torch.bfloat16
    _need(q, bf, "q", (None, None, None))
    Lq, Hq, D = q.shape
    _need(k, bf, "k", (None, None, D))
    _need(v, bf, "v", tuple(k.shape)), _need(idx, torch.int32, "idx", (Lq, None)), _need(out, bf, "out", (Lq, Hq, D))
    if lse is not None:
        _need(lse, torch.float32, "lse", (Lq, Hq))
    _on_device(q=q, k=k, v=v, idx=idx, out=out, lse=lse)
    st = _lib.dsa_sparse_attn(_ptr(q), _ptr(k), _ptr(v), _ptr(idx), Lq, k.shape[0], q_pos0, Hq, k.shape[1], D,
                              idx.shape[1], float(scale), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "dsa_sparse_attn")


def dsa_sparse_attn_dedup(q, k, v, idx, q_pos0: int, scale: float, out, lse=None, stream=None) -> None:
    """dsa_sparse_attn computed per block of adjacent rows over the union of their index sets."""
    import torch
    bf = torch.bfloat16
    _need(q, bf, "q", (None, None, None))
    Lq, Hq, D = q.shape
    _need(k, bf, "k", (None, None, D))
    _need(v, bf, "v", tuple(k.shape)), _need(idx, torch.int32, "idx", (Lq, None)), _need(out, bf, "out", (Lq, Hq, D))
    if lse is not None:
        _need(lse, torch.float32, "lse", (Lq, Hq))
    _on_device(q=q, k=k, v=v, idx=idx, out=out, lse=lse)
    st = _lib.dsa_sparse_attn_dedup(_ptr(q), _ptr(k), _ptr(v), _ptr(idx), Lq, k.shape[0], q_pos0, Hq, k.shape[1], D,
                                    idx.shape[1], float(scale), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "dsa_sparse_attn_dedup")


def _prefill_operands(q, k, v, qI, kI, w, out, idx, topk, key_rows, names):
    """Shapes shared by the prefill entry points: q/qI/w/out/idx hold the same query rows, k/v/kI
    at least `key_rows` key rows."""
    import torch
    bf = torch.bfloat16
    nq, nk, nv, nqI, nkI, nw, nout, nidx = names
    _need(q, bf, nq, (None, None, None))
    rows, Hq, D = q.shape
    _need(k, bf, nk, (None, None, D))
    _at_least(k, nk, 0, key_rows)
    _need(v, bf, nv, tuple(k.shape)), _need(qI, bf, nqI, (rows, None, None))
    HI, dI = qI.shape[1], qI.shape[2]
    _need(kI, bf, nkI, (None, dI))
    _at_least(kI, nkI, 0, key_rows)
    _need(w, bf, nw, (rows, HI)), _need(out, bf, nout, (rows, Hq, D))
    if idx is not None:
        _need(idx, torch.int32, nidx, (rows, topk))
    return Hq, D, HI, dI


def dsa_prefill(q, k, v, qI, kI, w, topk: int, scale: float, out, idx_out=None, ws=None, window: int = 0,
                stream=None) -> None:
    """Indexer, top-k and sparse attention for every row of one causal sequence of q.shape[0] tokens."""
    L = q.shape[0] if hasattr(q, "shape") else 0
    Hq, D, HI, dI = _prefill_operands(q, k, v, qI, kI, w, out, idx_out, topk, L,
                                      ("q", "k", "v", "qI", "kI", "w", "out", "idx_out"))
    _on_device(q=q, k=k, v=v, qI=qI, kI=kI, w=w, out=out, idx_out=idx_out, ws=ws)
    ws = _workspace(ws, DSA_OP_PREFILL, L, 1, Hq, HI, topk, q)
    if window:
        st = _lib.dsa_prefill_window(_ptr(q), _ptr(k), _ptr(v), _ptr(qI), _ptr(kI), _ptr(w), L, Hq, k.shape[1], D,
                                     HI, dI, topk, window, float(scale), _ptr(out), _ptr(idx_out), _ptr(ws),
                                     _nbytes(ws), _stream(stream))
        _check(st, "dsa_prefill_window")
        return
    st = _lib.dsa_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(qI), _ptr(kI), _ptr(w), L, Hq, k.shape[1], D, HI, dI,
                          topk, float(scale), _ptr(out), _ptr(idx_out), _ptr(ws), _nbytes(ws), _stream(stream))
    _check(st, "dsa_prefill")


def dsa_prefill_rows(q_rows, k, v, qI_rows, kI, w_rows, row0: int, topk: int, scale: float, out_rows,
                     idx_rows=None, ws=None, window: int = 0, stream=None) -> None:
    """Prefill of query rows row0 .. row0+len(q_rows)-1; k, v, kI cover at least those rows."""
    rows = q_rows.shape[0] if hasattr(q_rows, "shape") else 0
    Hq, D, HI, dI = _prefill_operands(q_rows, k, v, qI_rows, kI, w_rows, out_rows, idx_rows, topk, row0 + rows,
                                      ("q_rows", "k", "v", "qI_rows", "kI", "w_rows", "out_rows", "idx_rows"))
    _on_device(q_rows=q_rows, k=k, v=v, qI_rows=qI_rows, kI=kI, w_rows=w_rows, out_rows=out_rows, idx_rows=idx_rows,
               ws=ws)
    ws = _workspace(ws, DSA_OP_PREFILL, row0 + rows, 1, Hq, HI, topk, q_rows)
    st = _lib.dsa_prefill_rows(_ptr(q_rows), _ptr(k), _ptr(v), _ptr(qI_rows), _ptr(kI), _ptr(w_rows), row0, rows, Hq,
                               k.shape[1], D, HI, dI, topk, window, float(scale), _ptr(out_rows), _ptr(idx_rows),
                               _ptr(ws), _nbytes(ws), _stream(stream))
    _check(st, "dsa_prefill_rows")


def dsa_indexer_kl(q, k, qI, kI, w, scale: float, kl, ws=None, stream=None) -> None:
    """Indexer warm-up target KL(P_t || Q_t) for every query row of one causal sequence into kl
    (float32 [L]); see dsa_indexer_kl in include/dsa.h."""
    import torch
    bf = torch.bfloat16
    _need(q, bf, "q", (None, None, None))
    L, Hq, D = q.shape
    _need(k, bf, "k", (None, None, D)), _at_least(k, "k", 0, L), _need(qI, bf, "qI", (L, None, None))
    HI, dI = qI.shape[1], qI.shape[2]
    _need(kI, bf, "kI", (None, dI)), _at_least(kI, "kI", 0, L), _need(w, bf, "w", (L, HI))
    _need(kl, torch.float32, "kl", (None,)), _at_least(kl, "kl", 0, L)
    _on_device(q=q, k=k, qI=qI, kI=kI, w=w, kl=kl, ws=ws)
    ws = _workspace(ws, DSA_OP_INDEXER_KL, L, 1, Hq, HI, 1, q)
    st = _lib.dsa_indexer_kl(_ptr(q), _ptr(k), _ptr(qI), _ptr(kI), _ptr(w), L, Hq, k.shape[1], D, HI, dI,
                             float(scale), _ptr(kl), _ptr(ws), _nbytes(ws), _stream(stream))
    _check(st, "dsa_indexer_kl")


def dsa_decode(q, qI, w, k_new, v_new, kI_new, k_cache, v_cache, kI_cache, ctx_len, topk: int, scale: float, out,
               idx_out=None, ws=None, update_ctx: bool = False, stream=None) -> None:
    """One decode step for B sequences: append the new token at ctx_len[b], then indexer, top-k
    and sparse attention over positions 0 .. ctx_len[b]."""
    import torch
    bf = torch.bfloat16
    _need(q, bf, "q", (None, None, None))
    B, Hq, D = q.shape
    _need(k_cache, bf, "k_cache", (B, None, None, D))
    Lmax, Hkv = k_cache.shape[1], k_cache.shape[2]
    _need(v_cache, bf, "v_cache", (B, Lmax, Hkv, D)), _need(qI, bf, "qI", (B, None, None))
    HI, dI = qI.shape[1], qI.shape[2]
    _need(w, bf, "w", (B, HI)), _need(kI_cache, bf, "kI_cache", (B, Lmax, dI))
    _need(k_new, bf, "k_new", (B, Hkv, D)), _need(v_new, bf, "v_new", (B, Hkv, D)), _need(kI_new, bf, "kI_new", (B, dI))
    _need(ctx_len, torch.int32, "ctx_len", (B,)), _need(out, bf, "out", (B, Hq, D))
    if idx_out is not None:
        _need(idx_out, torch.int32, "idx_out", (B, topk))
    _on_device(q=q, qI=qI, w=w, k_new=k_new, v_new=v_new, kI_new=kI_new, k_cache=k_cache, v_cache=v_cache,
               kI_cache=kI_cache, ctx_len=ctx_len, out=out, idx_out=idx_out, ws=ws)
    ws = _workspace(ws, DSA_OP_DECODE, Lmax, B, Hq, HI, topk, q)
    st = _lib.dsa_decode(_ptr(q), _ptr(qI), _ptr(w), _ptr(k_new), _ptr(v_new), _ptr(kI_new), _ptr(k_cache),
                         _ptr(v_cache), _ptr(kI_cache), _ptr(ctx_len), B, Lmax, Hq, Hkv, D, HI, dI, topk,
                         float(scale), int(bool(update_ctx)), _ptr(out), _ptr(idx_out), _ptr(ws), _nbytes(ws),
                         _stream(stream))
    _check(st, "dsa_decode")


def _heads(t, dtype, name, shape):
    """A [tokens, heads, dims] operand whose tokens and heads may lie any distance apart: checks it like
    _need and returns its strides between tokens and heads (those of an axis of one entry are free)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or any(e is not None and int(e) != n for e, n in zip(shape, t.shape)):
        want = ", ".join("*" if e is None else str(int(e)) for e in shape)
        raise ValueError(f"{name} must have shape [{want}], got {list(t.shape)}")
    T, H, D = t.shape
    ts, hs, ds = t.stride()
    if ds != 1 and D != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    if H == 1:
        hs = (D + 7) // 8 * 8
    if T == 1:
        ts = H * hs
    return ts, hs


def rope_freqs(rot_dim: int, theta: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
               orig_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(frequencies, mscale) for dsa_rope and dsa_kv_append: a float64 CPU tensor [rot_dim / 2], to be moved
    to the GPU once, and the factor that goes with them; scaling is one of ROPE_SCALINGS."""
    import torch
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {ROPE_SCALINGS}, got {scaling!r}")
    f = torch.empty(max(0, int(rot_dim)) // 2, dtype=torch.float64)
    m = ctypes.c_float()
    _check(_lib.dsa_rope_freqs(int(rot_dim), float(theta), ROPE_SCALINGS.index(scaling), float(factor),
                               float(orig_len), float(beta_fast), float(beta_slow), _ptr(f),
                               ctypes.cast(ctypes.byref(m), ctypes.c_void_p)), "dsa_rope_freqs")
    return f, m.value


def dsa_rope(x, out, inv_freq, pos=None, pos0: int = 0, rot_offset: int = 0, interleaved: bool = False,
             mscale: float = 1.0, inverse: bool = False, stream=None) -> None:
    """Rotary positions of x's heads into out (which may be x); inverse gives the gradient of the same."""
    if stream is None:
        st = (_fast or _native()).rope(x, out, inv_freq, pos, pos0, rot_offset, interleaved, mscale, inverse)
        if st is not None:
            return _check(st, "dsa_rope")
    import torch
    if getattr(x, "dtype", None) not in (torch.bfloat16, torch.float32):
        raise TypeError(f"x must be a bfloat16 or float32 tensor, got {getattr(x, 'dtype', type(x))}")
    x_ts, x_hs = _heads(x, x.dtype, "x", (None, None, None))
    T, H, D = x.shape
    out_ts, out_hs = _heads(out, x.dtype, "out", (T, H, D))
    _need(inv_freq, torch.float64, "inv_freq", (None,))
    if pos is not None:
        _need(pos, torch.int32, "pos", (T,))
    _on_device(x=x, out=out, inv_freq=inv_freq, pos=pos)
    st = _lib.dsa_rope(_ptr(x), DSA_BF16 if x.dtype == torch.bfloat16 else DSA_FP32, T, H, D, x_ts, x_hs, _ptr(pos),
                       pos0, _ptr(inv_freq), rot_offset, 2 * inv_freq.shape[0], int(bool(interleaved)), float(mscale),
                       int(bool(inverse)), _ptr(out), out_ts, out_hs, _stream(stream))
    _check(st, "dsa_rope")


def _cache_operands(k_pages, v_pages, k_scale, v_scale, page_table):
    """Format and sizes of a paged cache: (kv_format, num_pages, page_size, Hkv, D, B, max_pages)."""
    import torch
    formats = {torch.float8_e4m3fn: DSA_KV_E4M3, torch.int8: DSA_KV_INT8}
    if getattr(k_pages, "dtype", None) not in formats:
        raise TypeError(f"k_pages must be a float8_e4m3fn or int8 tensor, got {getattr(k_pages, 'dtype', type(k_pages))}")
    _need(k_pages, k_pages.dtype, "k_pages", (None, None, None, None))
    num_pages, page, Hkv, D = k_pages.shape
    _need(v_pages, k_pages.dtype, "v_pages", k_pages.shape)
    _need(k_scale, torch.float32, "k_scale", (num_pages, Hkv))
    _need(v_scale, torch.float32, "v_scale", (num_pages, Hkv))
    _need(page_table, torch.int32, "page_table", (None, None))
    return formats[k_pages.dtype], num_pages, page, Hkv, D, page_table.shape[0], page_table.shape[1]


def dsa_kv_append(k_new, v_new, k_pages, v_pages, k_scale, v_scale, page_table, ctx_len, cu_new=None, inv_freq=None,
                  rope_pos=None, rot_offset: int = 0, interleaved: bool = False, mscale: float = 1.0,
                  stream=None) -> None:
    """Append tokens to a paged 8-bit cache at positions ctx_len[b].., keys rotated where inv_freq is given."""
    if stream is None:
        st = (_fast or _native()).kv_append(k_new, v_new, k_pages, v_pages, k_scale, v_scale, page_table, ctx_len,
                                               cu_new, inv_freq, rope_pos, rot_offset, interleaved, mscale)
        if st is not None:
            return _check(st, "dsa_kv_append")
    import torch
    fmt, num_pages, page, Hkv, D, B, max_pages = _cache_operands(k_pages, v_pages, k_scale, v_scale, page_table)
    k_ts, k_hs = _heads(k_new, torch.bfloat16, "k_new", (None, Hkv, D))
    N = k_new.shape[0]
    v_ts, v_hs = _heads(v_new, torch.bfloat16, "v_new", (N, Hkv, D))
    _need(ctx_len, torch.int32, "ctx_len", (B,))
    if cu_new is not None:
        _need(cu_new, torch.int32, "cu_new", (B + 1,))
    elif N != B:
        raise ValueError(f"k_new must have one token for each of page_table's {B} sequences where cu_new is not given, "
                         f"got {N}")
    if inv_freq is not None:
        _need(inv_freq, torch.float64, "inv_freq", (None,))
    if rope_pos is not None:
        _need(rope_pos, torch.int32, "rope_pos", (N,))
    _on_device(k_new=k_new, v_new=v_new, k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale,
               page_table=page_table, ctx_len=ctx_len, cu_new=cu_new, inv_freq=inv_freq, rope_pos=rope_pos)
    st = _lib.dsa_kv_append(_ptr(k_new), _ptr(v_new), k_ts, k_hs, v_ts, v_hs, N, _ptr(cu_new), _ptr(ctx_len),
                            _ptr(rope_pos), _ptr(inv_freq), rot_offset,
                            0 if inv_freq is None else 2 * inv_freq.shape[0], int(bool(interleaved)), float(mscale), fmt,
                            _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), B, num_pages,
                            page, max_pages, Hkv, D, _stream(stream))
    _check(st, "dsa_kv_append")


def dsa_paged_attn(q, k_pages, v_pages, k_scale, v_scale, page_table, n_keys, scale: float, out, seq=None, idx=None,
                   lse=None, ws=None, stream=None) -> None:
    """Attention of q's rows over a paged 8-bit cache: the first n_keys[t] keys of each row's sequence, or
    those of them that idx names."""
    if stream is None:
        st = (_fast or _native()).paged_attn(q, k_pages, v_pages, k_scale, v_scale, page_table, n_keys, scale, out, seq,
                                                idx, lse, ws)
        if st is not None:
            return _check(st, "dsa_paged_attn")
    import torch
    bf = torch.bfloat16
    fmt, num_pages, page, Hkv, D, B, max_pages = _cache_operands(k_pages, v_pages, k_scale, v_scale, page_table)
    _need(q, bf, "q", (None, None, D))
    T, Hq = q.shape[0], q.shape[1]
    _need(out, bf, "out", (T, Hq, D)), _need(n_keys, torch.int32, "n_keys", (T,))
    if seq is not None:
        _need(seq, torch.int32, "seq", (T,))
    elif T != B:
        raise ValueError(f"q must have one row for each of page_table's {B} sequences where seq is not given, got {T}")
    if idx is not None:
        _need(idx, torch.int32, "idx", (T, None))
    if lse is not None:
        _need(lse, torch.float32, "lse", (T, Hq))
    _on_device(q=q, k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale, page_table=page_table,
               n_keys=n_keys, out=out, seq=seq, idx=idx, lse=lse, ws=ws)
    if ws is None and stream is not None:
        with torch.cuda.stream(stream):  # memory that is in order with the kernels' stream
            ws = _workspace(None, DSA_OP_PAGED_ATTN, 1, T, Hq, 1, 1, q)
    else:
        ws = _workspace(ws, DSA_OP_PAGED_ATTN, 1, T, Hq, 1, 1, q)
    st = _lib.dsa_paged_attn(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
                             _ptr(seq), _ptr(n_keys), _ptr(idx), fmt, T, B, num_pages, page, max_pages, Hq, Hkv, D,
                             0 if idx is None else idx.shape[1], float(scale), _ptr(out), _ptr(lse), _ptr(ws),
                             _nbytes(ws), _stream(stream))
    _check(st, "dsa_paged_attn")


def sync_status(stream=None) -> int:
    return int(_lib.dsa_sync_status(_stream(stream)))


def error_site() -> int:
    """Site code (and loop index) of the last device error recorded; 0 if none."""
    return int(_lib.dsa_error_site())


def profile_begin() -> None:
    _lib.dsa_profile_begin()


def profile_end() -> dict:
    launches = (ctypes.c_int64 * len(PROFILE_KINDS))()
    ms = (ctypes.c_double * len(PROFILE_KINDS))()
    _check(_lib.dsa_profile_end_kinds(len(PROFILE_KINDS), launches, ms), "dsa_profile_end")
    return {k: {"launches": int(launches[i]), "ms": float(ms[i])} for i, k in enumerate(PROFILE_KINDS)}


def read_counters(reset: bool = False) -> dict:
    """Device path counters: top-k rows and sampled-threshold fallbacks (see dsa.h)."""
    buf = (ctypes.c_int64 * 8)()
    _check(_lib.dsa_read_counters(buf, 8, int(bool(reset))), "dsa_read_counters")
    return {"topk_rows": buf[0], "topk_retry": buf[1], "topk_global": buf[4], "topk_cluster_rows": buf[2],
            "topk_cluster_retry": buf[3], "topk_cluster_global": buf[5]}


def launch_count() -> int:
    return int(_lib.dsa_launch_count())


def selftest_timeout(wait_ns: int, stream=None) -> None:
    _check(_lib.dsa_selftest_timeout(int(wait_ns), _stream(stream)), "dsa_selftest_timeout")


def lib() -> ctypes.CDLL:
    """The loaded C library (raw ctypes access for callers that marshal pointers themselves)."""
    return _lib

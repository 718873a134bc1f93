"""Thin ctypes binding of libsparsepool (include/sparse_pool.h) on torch tensors.

Argument marshalling only: every function checks dtype/device/shape/contiguity of
the tensors it is given, passes their data pointers and the current CUDA stream to
the C entry point of the same name, and raises ``SparsePoolError`` on a non-zero
status.  Every step of the computation runs in the CUDA kernels; there is no CPU
fallback, and a missing library raises at the first call.  The paged cache's calls
are marshalled by csrc/marshal.cpp, the same way: they are short enough that checking their
tensors in Python takes longer than they do.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsparsepool.so")
MARSHAL_PATH = os.path.join(_PKG, f"_marshal_{torch.__version__}.so")
_lock = threading.Lock()
_lib = None
_marshal = None   # csrc/marshal.cpp, which passes the paged cache's tensors on; loaded by its first call

D = 128
BLK = 64

SPARSE_OK = 0
SPARSE_ERR_INVALID_ARG = -1
SPARSE_ERR_UNSUPPORTED = -2
SPARSE_ERR_CUDA = -3
SPARSE_ERR_TIMEOUT = -4
SPARSE_ERR_NOT_READY = -5
SPARSE_ERR_BAD_INDEX = -6
SPARSE_ERR_NO_PAGES = -7
SPARSE_ATTN_BLOCKS_READY = 1
SPARSE_ATTN_STREAM_K = 2
SPARSE_ATTN_TENSOR_MEMORY = 16
SPARSE_NSA_BRANCH_GRID = 4
SPARSE_SELECT_KEYS_READY = 8

# (name, restype, argtypes) of every entry point declared in include/sparse_pool.h
_P, _I, _LL, _F, _U = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_uint
_SZ = ctypes.c_size_t
SIGNATURES = {
    "sparse_status_string": (ctypes.c_char_p, [_I]),
    "sparse_last_error": (ctypes.c_char_p, []),
    "sparse_version": (_I, []),
    "sparse_pool_append": (_I, [_P, _P, _P, _P, _P, _I, _I, _LL, _I, _LL, _I, _P]),
    "sparse_pool_append_kv": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _LL, _I, _LL, _I, _P]),
    "sparse_select_topk": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P]),
    "sparse_select_topk_ex": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _I, _U, _P, _P]),
    "sparse_select_topk_heads": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _I, _I, _I, _P, _P, _I, _P, _P]),
    "sparse_prefill_select": (_I, [_P, _LL, _P, _I, _P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P]),
    "sparse_decode_attn": (_I, [_P, _P, _P, _LL, _P, _P, _P, _I, _P, _I, _I, _I, _F, _P, _P, _I, _U, _P, _SZ,
                                _P, _P]),
    "sparse_decode_attn_ex": (_I, [_P, _P, _P, _LL, _P, _P, _P, _I, _P, _I, _I, _I, _F, _P, _P, _I, _U, _P, _SZ,
                                   _P, _U, _LL, _P, _P]),
    "sparse_decode_attn_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "sparse_decode_attn_noalloc": (_I, [_P, _P, _P, _LL, _P, _P, _P, _I, _P, _I, _I, _I, _F, _P, _P, _I, _U, _P,
                                        _P]),
    "sparse_decode_attn_forecast": (_I, [_P, _P, _P, _LL, _P, _P, _I, _P, _I, _I, _I, _F, _P, _P, _P, _P, _I, _I,
                                         _I, _I, _P, _P, _I, _I, _U, _P, _P]),
    "sparse_verify_attn_grouped": (_I, [_P, _P, _P, _LL, _P, _I, _I, _I, _I, _P, _I, _I, _I, _F, _P, _P, _I,
                                        _U, _P, _P]),
    "sparse_verify_attn_shared": (_I, [_P, _P, _P, _LL, _P, _I, _I, _I, _I, _P, _I, _I, _I, _F, _P, _P, _I,
                                       _U, _P, _P]),
    "sparse_gather_offloaded": (_I, [_P, _P, _LL, _P, _P, _I, _I, _I, _P, _P, _P, _I, _P, _P]),
    "sparse_decode_attn_nsa": (_I, [_P, _P, _P, _LL, _P, _P, _I, _I, _I, _P, _P, _I, _P, _I, _I, _I, _LL, _P, _F,
                                    _P, _P, _SZ, _I, _U, _P, _P]),
    "sparse_nsa_compress": (_I, [_P, _P, _LL, _I, _I, _LL, _I, _I, _I, _P, _P, _I, _P]),
    "sparse_nsa_select": (_I, [_P, _P, _I, _I, _I, _P, _I, _I, _I, _I, _F, _I, _I, _I, _P, _P, _I, _P, _P]),
    "sparse_decode_attn_nsa_workspace_size": (_SZ, [_I, _I, _I]),
    "sparse_page_plan": (_I, [_P, _P, _I, _P, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P]),
    "sparse_paged_append_f8": (_I, [_P, _P, _I, _I, _P, _P, _LL, _LL, _P, _I, _P, _I, _I, _P, _P, _P, _P]),
    "sparse_paged_decode_attn_f8": (_I, [_P, _P, _P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _I, _F, _P, _P, _P, _SZ,
                                         _P, _P]),
    "sparse_paged_decode_attn_f8_workspace_size": (_SZ, [_I, _I, _I]),
    "sparse_paged_chunk_attn_f8": (_I, [_P, _LL, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P, _P]),
    "sparse_paged_chunk_attn_f8_workspace_size": (_SZ, [_I, _I, _I]),
    "sparse_rope": (_I, [_P, _LL, _I, _P, _LL, _I, _P, _I, _P, _I, _I, _F, _P, _LL, _P, _LL, _P]),
    "sparse_page_fork": (_I, [_P, _P, _I, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, _SZ, _P, _P]),
    "sparse_page_fork_workspace_size": (_SZ, [_I, _I]),
    "sparse_paged_copy_f8": (_I, [_P, _P, _I, _I, _P, _P, _I, _P, _I, _I, _P, _P, _P, _P]),
}


class SparsePoolError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def load(path: str = LIB_PATH):
    """Load libsparsepool.so (built in-tree by ``block_sparse_long_pool_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built; run `python -m block_sparse_long_pool_gb300.build` "
                               "(there is no CPU fallback)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _load_marshal():
    """The module of the paged cache's calls, which reads this torch version's tensor objects; the
    other calls do without it."""
    global _marshal
    lib = load()
    with _lock:
        if _marshal is None:
            if not os.path.exists(MARSHAL_PATH):
                raise RuntimeError(f"{MARSHAL_PATH} is not built for this torch; run "
                                   "`python -m block_sparse_long_pool_gb300.build`")
            spec = importlib.util.spec_from_file_location("_marshal", MARSHAL_PATH)
            marshal = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(marshal)
            marshal.setup(*(ctypes.cast(getattr(lib, f"sparse_{name}"), ctypes.c_void_p).value
                            for name in ("page_plan", "paged_append_f8", "paged_decode_attn_f8",
                                         "paged_chunk_attn_f8", "rope", "page_fork", "paged_copy_f8")))
            _marshal = marshal


def status_string(status: int) -> str:
    return load().sparse_status_string(int(status)).decode()


def _check(rc: int, name: str):
    if rc != SPARSE_OK:
        raise SparsePoolError(rc, f"{name}: {load().sparse_last_error().decode()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, device_ok=True, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device_ok and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def sparse_pool_append(k_cache, v_cache, ktil, k_new, v_new, len_before: int, stream=None):
    """Append k_new/v_new [B][H_kv][n_new][128] at len_before and update ktil."""
    B, H_kv, T_cap, _ = k_cache.shape
    n_new = k_new.shape[2]
    N_cap = ktil.shape[2]
    _need(k_cache, "k_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(v_cache, "v_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(ktil, "ktil", torch.float32, shape=(B, H_kv, N_cap, D))
    _need(k_new, "k_new", torch.bfloat16, shape=(B, H_kv, n_new, D))
    _need(v_new, "v_new", torch.bfloat16, shape=(B, H_kv, n_new, D))
    rc = load().sparse_pool_append(_ptr(k_cache), _ptr(v_cache), _ptr(ktil), _ptr(k_new), _ptr(v_new), B, H_kv,
                                   T_cap, N_cap, int(len_before), n_new, _stream(stream))
    _check(rc, "sparse_pool_append")


def sparse_pool_append_kv(k_cache, v_cache, ktil, vtil, k_new, v_new, len_before: int, khat=None, vhat=None,
                          stream=None):
    """Append k_new/v_new [B][H_kv][n_new][128] at len_before, update the pooled keys
    ktil and values vtil (fp32) and, when given, their bf16 copies khat / vhat."""
    B, H_kv, T_cap, _ = k_cache.shape
    n_new = k_new.shape[2]
    N_cap = ktil.shape[2]
    _need(k_cache, "k_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(v_cache, "v_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(ktil, "ktil", torch.float32, shape=(B, H_kv, N_cap, D))
    _need(vtil, "vtil", torch.float32, shape=(B, H_kv, N_cap, D))
    for t, n in ((khat, "khat"), (vhat, "vhat")):
        if t is not None:
            _need(t, n, torch.bfloat16, shape=(B, H_kv, N_cap, D))
    _need(k_new, "k_new", torch.bfloat16, shape=(B, H_kv, n_new, D))
    _need(v_new, "v_new", torch.bfloat16, shape=(B, H_kv, n_new, D))
    rc = load().sparse_pool_append_kv(_ptr(k_cache), _ptr(v_cache), _ptr(ktil), _ptr(vtil), _ptr(khat), _ptr(vhat),
                                      _ptr(k_new), _ptr(v_new), B, H_kv, T_cap, N_cap, int(len_before), n_new,
                                      _stream(stream))
    _check(rc, "sparse_pool_append_kv")


def sparse_select_topk(F, ktil, seq_len, n_init: int, n_local: int, k: int, idx_out, count_out,
                       status=None, stream=None, flags: int = 0):
    """Fill idx_out [B][H_kv][k_tot] and count_out [B][H_kv] from F [B][H_kv][128] and ktil.
    flags (SPARSE_SELECT_KEYS_READY) calls sparse_select_topk_ex."""
    B, H_kv, N_cap, _ = ktil.shape
    k_tot = idx_out.shape[2]
    _need(F, "F", torch.bfloat16, shape=(B, H_kv, D))
    _need(ktil, "ktil", torch.float32)
    _need(seq_len, "seq_len", torch.int32, shape=(B,))
    _need(idx_out, "idx_out", torch.int32, shape=(B, H_kv, k_tot))
    _need(count_out, "count_out", torch.int32, shape=(B, H_kv))
    if status is not None:
        _need(status, "status", torch.int32)
    if flags:
        rc = load().sparse_select_topk_ex(_ptr(F), _ptr(ktil), _ptr(seq_len), B, H_kv, N_cap, n_init, n_local, k,
                                          _ptr(idx_out), _ptr(count_out), k_tot, int(flags), _ptr(status),
                                          _stream(stream))
        _check(rc, "sparse_select_topk_ex")
        return
    rc = load().sparse_select_topk(_ptr(F), _ptr(ktil), _ptr(seq_len), B, H_kv, N_cap, n_init, n_local, k,
                                   _ptr(idx_out), _ptr(count_out), k_tot, _ptr(status), _stream(stream))
    _check(rc, "sparse_select_topk")


def sparse_select_topk_heads(Q, ktil, seq_len, n_init: int, n_local: int, k: int, idx_out, count_out,
                             scale: float = 0.0, status=None, stream=None):
    """Multi-head (InfLLM-V2) selection: Q [B][H_q][128] bf16, ktil [B][H_kv][N_cap][128]
    fp32 -> idx_out [B][H_kv][k_tot], count_out [B][H_kv]."""
    B, H_kv, N_cap, _ = ktil.shape
    H_q = Q.shape[1]
    k_tot = idx_out.shape[2]
    _need(Q, "Q", torch.bfloat16, shape=(B, H_q, D))
    _need(ktil, "ktil", torch.float32)
    _need(seq_len, "seq_len", torch.int32, shape=(B,))
    _need(idx_out, "idx_out", torch.int32, shape=(B, H_kv, k_tot))
    _need(count_out, "count_out", torch.int32, shape=(B, H_kv))
    if status is not None:
        _need(status, "status", torch.int32)
    rc = load().sparse_select_topk_heads(_ptr(Q), _ptr(ktil), _ptr(seq_len), B, H_q, H_kv, N_cap, float(scale),
                                         n_init, n_local, k, _ptr(idx_out), _ptr(count_out), k_tot, _ptr(status),
                                         _stream(stream))
    _check(rc, "sparse_select_topk_heads")


def _decode_args(Q, k_base, v_base, blk_logical, count, seq_len, O, lse, blk_slot):
    B, H_q, _ = Q.shape
    n_pairs, k_tot = blk_logical.shape[0] * blk_logical.shape[1], blk_logical.shape[2]
    H_kv = blk_logical.shape[1]
    pair_stride = k_base.numel() // (n_pairs * D)
    _need(Q, "Q", torch.bfloat16, shape=(B, H_q, D))
    _need(k_base, "k_base", torch.bfloat16)
    _need(v_base, "v_base", torch.bfloat16, shape=tuple(k_base.shape))
    if k_base.numel() != n_pairs * pair_stride * D:
        raise ValueError("k_base must hold B*H_kv pair regions of pair_stride x 128")
    _need(blk_logical, "blk_logical", torch.int32, shape=(B, H_kv, k_tot))
    if blk_slot is not None:
        _need(blk_slot, "blk_slot", torch.int32, shape=(B, H_kv, k_tot))
    _need(count, "count", torch.int32, shape=(B, H_kv))
    _need(seq_len, "seq_len", torch.int32, shape=(B,))
    _need(O, "O", torch.bfloat16, shape=(B, H_q, D))
    if lse is not None:
        _need(lse, "lse", torch.float32, shape=(B, H_q))
    return B, H_q, H_kv, k_tot, pair_stride


def sparse_decode_attn_workspace_size(B: int, H_q: int, H_kv: int, k_tot: int, n_split: int = 0) -> int:
    """Bytes of the workspace of sparse_decode_attn (split and stream-K paths; 0: sizes
    that no workspace path serves)."""
    return int(load().sparse_decode_attn_workspace_size(B, H_q, H_kv, k_tot, n_split))


def decode_workspace(B: int, H_q: int, H_kv: int, k_tot: int, n_split: int = 0, device="cuda"):
    """A zeroed workspace tensor for sparse_decode_attn, or None when not needed."""
    n = sparse_decode_attn_workspace_size(B, H_q, H_kv, k_tot, n_split)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n > 0 else None


def _ws(workspace):
    if workspace is None:
        return None, 0
    _need(workspace, "workspace", torch.uint8)
    return _ptr(workspace), workspace.numel()


def sparse_decode_attn(Q, k_base, v_base, blk_logical, count, seq_len, O, lse=None, blk_slot=None,
                       scale: float = 0.0, n_split: int = 0, flags: int = 0, workspace=None, status=None,
                       stream=None):
    """O [B][H_q][128] = attention of Q over the listed blocks of k_base/v_base.

    k_base/v_base hold B*H_kv pair regions of pair_stride x 128 rows (a cache
    [B][H_kv][T_cap][128] or a ring slot [B][H_kv][k_tot][64][128]).  ``flags`` may be
    SPARSE_ATTN_BLOCKS_READY: the block list and K/V are not written by the previous
    kernel on ``stream`` (they are already complete while it runs), so K/V streaming may
    start while it drains; SPARSE_ATTN_TENSOR_MEMORY: both contractions as tcgen05.mma
    with tensor-memory accumulators (cluster path, no workspace)."""
    B, H_q, H_kv, k_tot, pair_stride = _decode_args(Q, k_base, v_base, blk_logical, count, seq_len, O, lse,
                                                    blk_slot)
    ws, ws_bytes = _ws(workspace)
    rc = load().sparse_decode_attn(_ptr(Q), _ptr(k_base), _ptr(v_base), pair_stride, _ptr(blk_slot),
                                   _ptr(blk_logical), _ptr(count), k_tot, _ptr(seq_len), B, H_q, H_kv,
                                   float(scale), _ptr(O), _ptr(lse), n_split, int(flags), ws, ws_bytes,
                                   _ptr(status), _stream(stream))
    _check(rc, "sparse_decode_attn")


def sparse_decode_attn_noalloc(Q, k_base, v_base, blk_logical, count, seq_len, O, lse=None, blk_slot=None,
                               scale: float = 0.0, n_split: int = 0, flags: int = 0, status=None, stream=None):
    """sparse_decode_attn without a workspace argument and without allocating: for
    callers that cannot allocate device memory (a host without a caching allocator, an
    engine whose device memory is planned up front).  The library's fixed 4 MiB device
    array serves as scratch; calls sharing it must not overlap on the GPU."""
    B, H_q, H_kv, k_tot, pair_stride = _decode_args(Q, k_base, v_base, blk_logical, count, seq_len, O, lse,
                                                    blk_slot)
    rc = load().sparse_decode_attn_noalloc(_ptr(Q), _ptr(k_base), _ptr(v_base), pair_stride, _ptr(blk_slot),
                                           _ptr(blk_logical), _ptr(count), k_tot, _ptr(seq_len), B, H_q, H_kv,
                                           float(scale), _ptr(O), _ptr(lse), n_split, int(flags), _ptr(status),
                                           _stream(stream))
    _check(rc, "sparse_decode_attn_noalloc")


def sparse_decode_attn_ex(Q, k_base, v_base, blk_logical, count, seq_len, O, ready_flag, ready_target: int,
                          timeout_ns: int, lse=None, blk_slot=None, scale: float = 0.0, n_split: int = 0,
                          flags: int = 0, workspace=None, status=None, stream=None):
    """sparse_decode_attn after a bounded check of a staging-ready word."""
    B, H_q, H_kv, k_tot, pair_stride = _decode_args(Q, k_base, v_base, blk_logical, count, seq_len, O, lse,
                                                    blk_slot)
    _need(ready_flag, "ready_flag", torch.int32)
    rc = load().sparse_decode_attn_ex(_ptr(Q), _ptr(k_base), _ptr(v_base), pair_stride, _ptr(blk_slot),
                                      _ptr(blk_logical), _ptr(count), k_tot, _ptr(seq_len), B, H_q, H_kv,
                                      float(scale), _ptr(O), _ptr(lse), n_split, int(flags), *_ws(workspace),
                                      _ptr(ready_flag),
                                      int(ready_target), int(timeout_ns), _ptr(status), _stream(stream))
    _check(rc, "sparse_decode_attn_ex")


def sparse_decode_attn_forecast(Q, k_cache, v_cache, blk_idx, count, seq_len, O, lse=None, F=None, ktil_next=None,
                                n_init: int = 1, n_local: int = 2, k: int = 0, idx_next=None, count_next=None,
                                scale: float = 0.0, n_split: int = 0, flags: int = 0, status=None, stream=None):
    """One decode layer in one kernel: O = attention of Q over blocks blk_idx of the
    resident cache k_cache / v_cache [B][H_kv][T_cap][128], and (when F is given) the
    Forecast selection of the next layer from ktil_next [B][H_kv][N_cap][128] into
    idx_next [B][H_kv][k_tot_next] / count_next [B][H_kv]."""
    B, H_q, H_kv, k_tot, T_cap = _decode_args(Q, k_cache, v_cache, blk_idx, count, seq_len, O, lse, None)
    _need(k_cache, "k_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    N_cap = k_tot_next = 0
    if F is not None:
        if ktil_next is None or idx_next is None or count_next is None:
            raise ValueError("F needs ktil_next, idx_next and count_next")
        N_cap = ktil_next.shape[2]
        k_tot_next = idx_next.shape[2]
        _need(F, "F", torch.bfloat16, shape=(B, H_kv, D))
        _need(ktil_next, "ktil_next", torch.float32, shape=(B, H_kv, N_cap, D))
        _need(idx_next, "idx_next", torch.int32, shape=(B, H_kv, k_tot_next))
        _need(count_next, "count_next", torch.int32, shape=(B, H_kv))
    if status is not None:
        _need(status, "status", torch.int32)
    rc = load().sparse_decode_attn_forecast(_ptr(Q), _ptr(k_cache), _ptr(v_cache), T_cap, _ptr(blk_idx), _ptr(count),
                                            k_tot, _ptr(seq_len), B, H_q, H_kv, float(scale), _ptr(O), _ptr(lse),
                                            _ptr(F), _ptr(ktil_next), N_cap, n_init, n_local, k, _ptr(idx_next),
                                            _ptr(count_next), k_tot_next, n_split, int(flags), _ptr(status),
                                            _stream(stream))
    _check(rc, "sparse_decode_attn_forecast")


def sparse_verify_attn_grouped(Q, k_cache, v_cache, idx_q, C: int, window_blocks: int, seq_len, O,
                               blocks_loaded=None, scale: float = 0.0, n_split: int = 0, status=None,
                               stream=None, shared: bool = False, flags: int = 0):
    """Grouped verification: Q [B][N_q][H_q][128], idx_q [B][H_kv][N_q][n_sel].  Mode A
    (each query over its own set), or with ``shared`` mode B (sparse_verify_attn_shared:
    every query over its group's first query's set)."""
    B, N_q, H_q, _ = Q.shape
    _, H_kv, T_cap, _ = k_cache.shape
    n_sel = idx_q.shape[3]
    _need(Q, "Q", torch.bfloat16, shape=(B, N_q, H_q, D))
    _need(k_cache, "k_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(v_cache, "v_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(idx_q, "idx_q", torch.int32, shape=(B, H_kv, N_q, n_sel))
    _need(seq_len, "seq_len", torch.int32, shape=(B,))
    _need(O, "O", torch.bfloat16, shape=(B, N_q, H_q, D))
    if blocks_loaded is not None:
        _need(blocks_loaded, "blocks_loaded", torch.int64)
    fn = load().sparse_verify_attn_shared if shared else load().sparse_verify_attn_grouped
    rc = fn(_ptr(Q), _ptr(k_cache), _ptr(v_cache), T_cap, _ptr(idx_q), n_sel, N_q, C, window_blocks, _ptr(seq_len), B,
            H_q, H_kv, float(scale), _ptr(O), _ptr(blocks_loaded), n_split, int(flags), _ptr(status),
            _stream(stream))
    _check(rc, "sparse_verify_attn_shared" if shared else "sparse_verify_attn_grouped")


def sparse_gather_offloaded(k_host, v_host, idx, count, k_ring, v_ring, ready_flag=None, n_ctas: int = 0,
                            status=None, stream=None):
    """Stage blocks idx [B][H_kv][k_tot] of pinned host K/V [B][H_kv][T_host][128]
    into ring slots [B][H_kv][k_tot][64][128]."""
    B, H_kv, T_host, _ = k_host.shape
    k_tot = idx.shape[2]
    _need(k_host, "k_host", torch.bfloat16, device_ok=False, shape=(B, H_kv, T_host, D))
    _need(v_host, "v_host", torch.bfloat16, device_ok=False, shape=(B, H_kv, T_host, D))
    for t, n in ((k_host, "k_host"), (v_host, "v_host")):
        if not t.is_cuda and not t.is_pinned():
            raise ValueError(f"{n} must be pinned host memory (or device memory)")
    _need(idx, "idx", torch.int32, shape=(B, H_kv, k_tot))
    _need(count, "count", torch.int32, shape=(B, H_kv))
    _need(k_ring, "k_ring", torch.bfloat16, shape=(B, H_kv, k_tot, BLK, D))
    _need(v_ring, "v_ring", torch.bfloat16, shape=(B, H_kv, k_tot, BLK, D))
    if ready_flag is not None:
        _need(ready_flag, "ready_flag", torch.int32)
    rc = load().sparse_gather_offloaded(_ptr(k_host), _ptr(v_host), T_host, _ptr(idx), _ptr(count), k_tot, B,
                                        H_kv, _ptr(k_ring), _ptr(v_ring), _ptr(ready_flag), n_ctas, _ptr(status),
                                        _stream(stream))
    _check(rc, "sparse_gather_offloaded")


def sparse_decode_attn_nsa_workspace_size(B: int, H_q: int, H_kv: int) -> int:
    """Bytes of the sparse_decode_attn_nsa workspace (0: invalid sizes)."""
    return int(load().sparse_decode_attn_nsa_workspace_size(B, H_q, H_kv))


def nsa_workspace(B: int, H_q: int, H_kv: int, device="cuda"):
    """A zeroed workspace tensor for sparse_decode_attn_nsa."""
    return torch.zeros(sparse_decode_attn_nsa_workspace_size(B, H_q, H_kv), dtype=torch.uint8, device=device)


def sparse_decode_attn_nsa(Q, k_cache, v_cache, khat, vhat, blk_idx, count, seq_len, window_tokens: int, gates, O,
                           workspace, scale: float = 0.0, n_split: int = 0, flags: int = 0, status=None,
                           stream=None, cmp: tuple = (0, 0)):
    """NSA gated three-branch decode: Q [B][H_q][128], K/V [B][H_kv][T_cap][128],
    compressed rows khat/vhat [B][H_kv][N_cap][128] (one per 64-token block, or with
    ``cmp = (l, s)`` the complete overlapping windows), selected blocks blk_idx
    [B][H_kv][k_tot] with count [B][H_kv], gates [B][H_q][3] = (g_c, g_s, g_w) fp32;
    writes O [B][H_q][128] = g_c o_c + g_s o_s + g_w o_w."""
    B, H_q, _ = Q.shape
    _, H_kv, T_cap, _ = k_cache.shape
    N_cap = khat.shape[2]
    k_tot = blk_idx.shape[2]
    _need(Q, "Q", torch.bfloat16, shape=(B, H_q, D))
    _need(k_cache, "k_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(v_cache, "v_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(khat, "khat", torch.bfloat16, shape=(B, H_kv, N_cap, D))
    _need(vhat, "vhat", torch.bfloat16, shape=(B, H_kv, N_cap, D))
    _need(blk_idx, "blk_idx", torch.int32, shape=(B, H_kv, k_tot))
    _need(count, "count", torch.int32, shape=(B, H_kv))
    _need(seq_len, "seq_len", torch.int32, shape=(B,))
    _need(gates, "gates", torch.float32, shape=(B, H_q, 3))
    _need(O, "O", torch.bfloat16, shape=(B, H_q, D))
    ws, ws_bytes = _ws(workspace)
    rc = load().sparse_decode_attn_nsa(_ptr(Q), _ptr(k_cache), _ptr(v_cache), T_cap, _ptr(khat), _ptr(vhat), N_cap,
                                       int(cmp[0]), int(cmp[1]), _ptr(blk_idx), _ptr(count), k_tot, _ptr(seq_len), B, H_q, H_kv,
                                       int(window_tokens), _ptr(gates), float(scale), _ptr(O), ws, ws_bytes,
                                       n_split, int(flags), _ptr(status), _stream(stream))
    _check(rc, "sparse_decode_attn_nsa")


def sparse_nsa_compress(k_cache, v_cache, khat, vhat, len_before: int, n_new: int, cmp=(32, 16), stream=None):
    """Rows of the overlapping windows completed by tokens [len_before, len_before + n_new)."""
    B, H_kv, T_cap, _ = k_cache.shape
    R = khat.shape[2]
    _need(k_cache, "k_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(v_cache, "v_cache", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(khat, "khat", torch.bfloat16, shape=(B, H_kv, R, D))
    _need(vhat, "vhat", torch.bfloat16, shape=(B, H_kv, R, D))
    rc = load().sparse_nsa_compress(_ptr(k_cache), _ptr(v_cache), T_cap, B, H_kv, int(len_before), int(n_new),
                                    int(cmp[0]), int(cmp[1]), _ptr(khat), _ptr(vhat), R, _stream(stream))
    _check(rc, "sparse_nsa_compress")


def sparse_nsa_select(Q, khat, seq_len, n_init: int, n_local: int, k: int, idx_out, count_out, cmp=(32, 16),
                      scale: float = 0.0, status=None, stream=None):
    """NSA routing: per-head softmax over the compressed rows khat [B][H_kv][R][128],
    summed over the group, max-pooled onto the 64-token blocks, top-k.  Q [B][H_q][128]
    (idx_out [B][H_kv][k_tot], count_out [B][H_kv]) or, for several queries per batch
    element, Q [B][N_q][H_q][128] (idx_out [B][H_kv][N_q][k_tot], count_out [B][H_kv][N_q])."""
    if Q.dim() == 3:
        B, H_q, _ = Q.shape
        N_q = 1
    else:
        B, N_q, H_q, _ = Q.shape
    _, H_kv, R, _ = khat.shape
    k_tot = idx_out.shape[-1]
    _need(Q, "Q", torch.bfloat16, shape=(B, H_q, D) if Q.dim() == 3 else (B, N_q, H_q, D))
    _need(khat, "khat", torch.bfloat16, shape=(B, H_kv, R, D))
    _need(seq_len, "seq_len", torch.int32, shape=(B,))
    _need(idx_out, "idx_out", torch.int32, shape=(B, H_kv, k_tot) if Q.dim() == 3 else (B, H_kv, N_q, k_tot))
    _need(count_out, "count_out", torch.int32, shape=(B, H_kv) if Q.dim() == 3 else (B, H_kv, N_q))
    rc = load().sparse_nsa_select(_ptr(Q), _ptr(khat), R, int(cmp[0]), int(cmp[1]), _ptr(seq_len), B, N_q, H_q, H_kv,
                                  float(scale), n_init, n_local, k, _ptr(idx_out), _ptr(count_out), k_tot,
                                  _ptr(status), _stream(stream))
    _check(rc, "sparse_nsa_select")


def sparse_prefill_select(F, ktil, seq_len, n_init: int, n_local: int, k: int, idx_out, count_out, status=None,
                          stream=None):
    """Forecast selection of every prefill position: F [B][H_kv][T_cap][128] bf16, ktil
    [B][H_kv][N_cap][128] fp32 -> idx_out [B][H_kv][T_cap][k_tot], count_out [B][H_kv][T_cap]."""
    B, H_kv, T_cap, _ = F.shape
    N_cap = ktil.shape[2]
    k_tot = idx_out.shape[3]
    _need(F, "F", torch.bfloat16, shape=(B, H_kv, T_cap, D))
    _need(ktil, "ktil", torch.float32, shape=(B, H_kv, N_cap, D))
    _need(seq_len, "seq_len", torch.int32, shape=(B,))
    _need(idx_out, "idx_out", torch.int32, shape=(B, H_kv, T_cap, k_tot))
    _need(count_out, "count_out", torch.int32, shape=(B, H_kv, T_cap))
    rc = load().sparse_prefill_select(_ptr(F), T_cap, _ptr(ktil), N_cap, _ptr(seq_len), B, H_kv, n_init, n_local, k,
                                      _ptr(idx_out), _ptr(count_out), k_tot, _ptr(status), _stream(stream))
    _check(rc, "sparse_prefill_select")


# ---------------------------------------------------------------- the paged 8-bit cache

_F8 = torch.float8_e4m3fn


# The calls of this cache are short: a decode step's plan or append takes 4 to 6 us on the
# device.  So their tensors are checked and passed on by csrc/marshal.cpp; what is wrong is
# looked for here, only when something is.


def _explain(idx, dtype, shape, **tensors):
    """Raises for the first tensor that is not of this type and shape, contiguous, on device ``idx``."""
    for name, t in tensors.items():
        _need(t, name, dtype, shape=shape)
        if t.get_device() != idx:
            raise ValueError(f"{name} is on {t.device}, expected device {idx}")


def _passed(name, idx, stream, *args) -> bool:
    """Calls ``name`` on device ``idx``, which need not be the current one; false where marshal.cpp
    refused a tensor, and nothing was called."""
    if _marshal is None:
        _load_marshal()
    call = getattr(_marshal, name)
    if idx == torch._C._cuda_getDevice():
        rc = call(idx, torch._C._cuda_getCurrentRawStream(idx) if stream is None else stream.cuda_stream, *args)
    else:
        with torch.cuda.device(idx):
            rc = call(idx, torch._C._cuda_getCurrentRawStream(idx) if stream is None else stream.cuda_stream, *args)
    if rc is None:
        return False
    if rc != SPARSE_OK:
        _check(rc, "sparse_" + name)
    return True


def _device_index(t, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _shape(t, name, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {dims} extents")
    return t.shape


def _refused(name):
    return ValueError(f"{name}: an extent does not fit 32 bits")


def sparse_page_plan(seq_len, n_new, block_table, free_pages, n_free, cu_new, start, seq_len_out, n_free_out, slot_map,
                     tok_req, tok_pos, status=None, stream=None):
    """Block tables and slot maps on the GPU, all int32: requests of seq_len [B] tokens get
    n_new [B] more (negative: the request ends and its pages are returned); pages go from
    the list free_pages [n_pages] (the first n_free [1]) into block_table [B][max_blocks].
    Writes cu_new [B + 1], start [B] (-1: not granted), seq_len_out [B], n_free_out [1] (the
    last two may be seq_len and n_free themselves) and slot_map, tok_req, tok_pos [n_tok]."""
    idx = _device_index(block_table, "block_table")
    if _passed("page_plan", idx, stream, seq_len, n_new, block_table, free_pages, n_free, cu_new, start, seq_len_out,
               n_free_out, slot_map, tok_req, tok_pos, status):
        return
    i32 = torch.int32
    B, max_blocks = _shape(block_table, "block_table", 2)
    _explain(idx, i32, (B, max_blocks), block_table=block_table)
    _explain(idx, i32, (B,), seq_len=seq_len, n_new=n_new, start=start, seq_len_out=seq_len_out)
    _explain(idx, i32, (1,), n_free=n_free, n_free_out=n_free_out, **({} if status is None else {"status": status}))
    _explain(idx, i32, (B + 1,), cu_new=cu_new)
    _explain(idx, i32, tuple(_shape(free_pages, "free_pages", 1)), free_pages=free_pages)
    _explain(idx, i32, tuple(_shape(slot_map, "slot_map", 1)), slot_map=slot_map, tok_req=tok_req, tok_pos=tok_pos)
    raise _refused("sparse_page_plan")


def _explain_rows(t, name, idx, n_tok, H_kv):
    """Rows [n_tok][H_kv][128], whose tokens may be apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != (n_tok, H_kv, D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n_tok, H_kv, D)}")
    if t.get_device() != idx:
        raise ValueError(f"{name} is on {t.device}, expected device {idx}")
    _, head, dim = t.stride()
    if dim != 1 or (head != D and H_kv > 1):
        raise ValueError(f"{name}: the values of a token must be contiguous")


def sparse_paged_append_f8(kv_pages, kv_scale, k_new, v_new, slot_map, ktil=None, tok_req=None, tok_pos=None,
                           status=None, stream=None):
    """Round k_new / v_new [n_tok][H_kv][128] bf16 (parts of wider rows are taken as they are)
    to e4m3 and write them to slot_map [n_tok] of kv_pages [n_pages][H_kv][2][64][128]
    (torch.float8_e4m3fn), with kv_scale [n_pages][H_kv][2] fp32; with ktil
    [B][H_kv][N_cap][128], tok_req and tok_pos [n_tok], update the compressed keys."""
    idx = _device_index(kv_pages, "kv_pages")
    if ktil is not None and (tok_req is None or tok_pos is None):
        raise ValueError("ktil needs tok_req and tok_pos")
    if _passed("paged_append_f8", idx, stream, kv_pages, kv_scale, k_new, v_new, slot_map, ktil, tok_req, tok_pos, status):
        return
    i32, f32 = torch.int32, torch.float32
    n_pages, H_kv = _shape(kv_pages, "kv_pages", 5)[:2]
    (n_tok,) = _shape(slot_map, "slot_map", 1)
    _explain(idx, _F8, (n_pages, H_kv, 2, BLK, D), kv_pages=kv_pages)
    _explain(idx, f32, (n_pages, H_kv, 2), kv_scale=kv_scale)
    _explain_rows(k_new, "k_new", idx, n_tok, H_kv)
    _explain_rows(v_new, "v_new", idx, n_tok, H_kv)
    _explain(idx, i32, (n_tok,), slot_map=slot_map)
    if ktil is not None:
        B, _, N_cap, _ = _shape(ktil, "ktil", 4)
        _explain(idx, f32, (B, H_kv, N_cap, D), ktil=ktil)
        _explain(idx, i32, (n_tok,), tok_req=tok_req, tok_pos=tok_pos)
    if status is not None:
        _explain(idx, i32, (1,), status=status)
    raise _refused("sparse_paged_append_f8")


def sparse_paged_decode_attn_f8_workspace_size(B: int, H_q: int, H_kv: int) -> int:
    """Bytes of the workspace of sparse_paged_decode_attn_f8 (0: invalid sizes)."""
    return int(load().sparse_paged_decode_attn_f8_workspace_size(B, H_q, H_kv))


def paged_workspace(B: int, H_q: int, H_kv: int, device="cuda"):
    """A zeroed workspace tensor for sparse_paged_decode_attn_f8."""
    with torch.cuda.device(device):
        n = sparse_paged_decode_attn_f8_workspace_size(B, H_q, H_kv)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def sparse_paged_decode_attn_f8(Q, kv_pages, kv_scale, block_table, seq_len, O, workspace, blk_idx=None, count=None,
                                lse=None, scale: float = 0.0, status=None, stream=None):
    """O [B][H_q][128] = attention of Q over the pages that block_table [B][max_blocks] names:
    every block of each request's seq_len [B] tokens, or the logical blocks blk_idx
    [B][H_kv][k_tot] with count [B][H_kv]."""
    idx = _device_index(kv_pages, "kv_pages")
    if blk_idx is not None and count is None:
        raise ValueError("blk_idx needs count")
    if _passed("paged_decode_attn_f8", idx, stream, Q, kv_pages, kv_scale, block_table, seq_len, O, workspace, blk_idx,
               count, lse, scale, status):
        return
    i32, f32, b16 = torch.int32, torch.float32, torch.bfloat16
    n_pages, H_kv = _shape(kv_pages, "kv_pages", 5)[:2]
    B, max_blocks = _shape(block_table, "block_table", 2)
    H_q = _shape(Q, "Q", 3)[1]
    _explain(idx, _F8, (n_pages, H_kv, 2, BLK, D), kv_pages=kv_pages)
    _explain(idx, f32, (n_pages, H_kv, 2), kv_scale=kv_scale)
    _explain(idx, b16, (B, H_q, D), Q=Q, O=O)
    _explain(idx, i32, (B, max_blocks), block_table=block_table)
    _explain(idx, i32, (B,), seq_len=seq_len)
    _explain(idx, torch.uint8, tuple(_shape(workspace, "workspace", 1)), workspace=workspace)
    if blk_idx is not None:
        k_tot = _shape(blk_idx, "blk_idx", 3)[2]
        _explain(idx, i32, (B, H_kv, k_tot), blk_idx=blk_idx)
        _explain(idx, i32, (B, H_kv), count=count)
    if lse is not None:
        _explain(idx, f32, (B, H_q), lse=lse)
    if status is not None:
        _explain(idx, i32, (1,), status=status)
    raise _refused("sparse_paged_decode_attn_f8")


def sparse_paged_chunk_attn_f8_workspace_size(B: int, H_q: int, H_kv: int) -> int:
    """Bytes of the workspace of sparse_paged_chunk_attn_f8 (0: invalid sizes)."""
    return int(load().sparse_paged_chunk_attn_f8_workspace_size(B, H_q, H_kv))


def paged_chunk_workspace(B: int, H_q: int, H_kv: int, device="cuda"):
    """A workspace tensor for sparse_paged_chunk_attn_f8."""
    with torch.cuda.device(device):
        n = sparse_paged_chunk_attn_f8_workspace_size(B, H_q, H_kv)
    return torch.empty(n, dtype=torch.uint8, device=device)


def sparse_paged_chunk_attn_f8(Q, kv_pages, kv_scale, block_table, cu_new, start, O, workspace, lse=None,
                               scale: float = 0.0, status=None, stream=None):
    """O [n_tok][H_q][128] = attention of a step's new rows Q [n_tok][H_q][128] (a part of wider rows is
    taken as it is) over the pages that block_table [B][max_blocks] names: request b's rows
    cu_new[b] .. cu_new[b + 1] - 1 are at positions start[b], start[b] + 1, ... and see the tokens up to
    their own.  lse [n_tok][H_q]."""
    idx = _device_index(kv_pages, "kv_pages")
    if _passed("paged_chunk_attn_f8", idx, stream, Q, kv_pages, kv_scale, block_table, cu_new, start, O, workspace, lse, scale,
               status):
        return
    i32, f32 = torch.int32, torch.float32
    n_pages, H_kv = _shape(kv_pages, "kv_pages", 5)[:2]
    B, max_blocks = _shape(block_table, "block_table", 2)
    n_tok, H_q, _ = _shape(Q, "Q", 3)
    _explain(idx, _F8, (n_pages, H_kv, 2, BLK, D), kv_pages=kv_pages)
    _explain(idx, f32, (n_pages, H_kv, 2), kv_scale=kv_scale)
    _explain_rows(Q, "Q", idx, n_tok, H_q)
    _explain(idx, torch.bfloat16, (n_tok, H_q, D), O=O)
    _explain(idx, i32, (B, max_blocks), block_table=block_table)
    _explain(idx, i32, (B + 1,), cu_new=cu_new)
    _explain(idx, i32, (B,), start=start)
    _explain(idx, torch.uint8, tuple(_shape(workspace, "workspace", 1)), workspace=workspace)
    if lse is not None:
        _explain(idx, f32, (n_tok, H_q), lse=lse)
    if status is not None:
        _explain(idx, i32, (1,), status=status)
    raise _refused("sparse_paged_chunk_attn_f8")


def sparse_rope(Q, K, pos, inv_freq, Q_out, K_out, interleaved: bool = False, factor: float = 1.0, stream=None):
    """Turns the rows Q [n_tok][H_q][128] and K [n_tok][H_kv][128] bf16 (parts of wider rows are taken as
    they are; K and K_out may be None) by their positions pos [n_tok] int32 into Q_out and K_out, which may be
    the inputs themselves: pair i by pos * inv_freq[i], inv_freq [rot_dim / 2] fp64 (``rope.frequencies``),
    pairs (i, i + rot_dim / 2) or interleaved (2 i, 2 i + 1).  Rows with a negative position are not written."""
    idx = _device_index(Q, "Q")
    if (K is None) != (K_out is None):
        raise ValueError("K and K_out go together")
    if _passed("rope", idx, stream, Q, K, pos, inv_freq, Q_out, K_out, bool(interleaved), factor):
        return
    n_tok, H_q, _ = _shape(Q, "Q", 3)
    _explain_rows(Q, "Q", idx, n_tok, H_q)
    _explain_rows(Q_out, "Q_out", idx, n_tok, H_q)
    if K is not None:
        H_kv = _shape(K, "K", 3)[1]
        _explain_rows(K, "K", idx, n_tok, H_kv)
        _explain_rows(K_out, "K_out", idx, n_tok, H_kv)
    _explain(idx, torch.int32, (n_tok,), pos=pos)
    _explain(idx, torch.float64, tuple(_shape(inv_freq, "inv_freq", 1)), inv_freq=inv_freq)
    raise _refused("sparse_rope")


def sparse_page_fork_workspace_size(B: int, max_blocks: int) -> int:
    """Bytes of the workspace of sparse_page_fork (0: invalid sizes)."""
    return int(load().sparse_page_fork_workspace_size(B, max_blocks))


def page_fork_workspace(B: int, max_blocks: int, device="cuda"):
    """A workspace tensor for sparse_page_fork."""
    return torch.empty(sparse_page_fork_workspace_size(B, max_blocks), dtype=torch.uint8, device=device)


def sparse_page_fork(src, seq_len, block_table, page_extra, free_pages, n_free, copy_src, copy_dst, workspace,
                     fork_len=None, status=None, stream=None):
    """Requests that become copies of others and requests that end, all int32: src [B] is a request's own
    index (it stays), -1 (it ends) or the request that it becomes a copy of, whose full pages it then
    shares (with fork_len [B] the first fork_len tokens, in whole blocks).  Updates seq_len [B],
    block_table [B][max_blocks], page_extra [n_pages] (holders beyond the first), free_pages [n_pages] and
    n_free [1]; writes the page pairs copy_src, copy_dst [B] for sparse_paged_copy_f8."""
    idx = _device_index(block_table, "block_table")
    if _passed("page_fork", idx, stream, src, seq_len, block_table, page_extra, free_pages, n_free, copy_src, copy_dst, workspace,
               fork_len, status):
        return
    i32 = torch.int32
    B, max_blocks = _shape(block_table, "block_table", 2)
    _explain(idx, i32, (B, max_blocks), block_table=block_table)
    _explain(idx, i32, (B,), src=src, seq_len=seq_len, copy_src=copy_src, copy_dst=copy_dst,
             **({} if fork_len is None else {"fork_len": fork_len}))
    _explain(idx, i32, tuple(_shape(free_pages, "free_pages", 1)), free_pages=free_pages, page_extra=page_extra)
    _explain(idx, i32, (1,), n_free=n_free, **({} if status is None else {"status": status}))
    _explain(idx, torch.uint8, tuple(_shape(workspace, "workspace", 1)), workspace=workspace)
    raise _refused("sparse_page_fork")


def sparse_paged_copy_f8(kv_pages, kv_scale, copy_src, copy_dst, ktil=None, src=None, seq_len=None, status=None, stream=None):
    """Copies the pages copy_src [n] of kv_pages (and their scales) to copy_dst [n], both -1 where there is
    nothing to copy; with ktil [B][H_kv][N_cap][128], src and seq_len [B] also the compressed keys of
    request src[b] to request b."""
    idx = _device_index(kv_pages, "kv_pages")
    if ktil is not None and (src is None or seq_len is None):
        raise ValueError("ktil needs src and seq_len")
    if _passed("paged_copy_f8", idx, stream, kv_pages, kv_scale, copy_src, copy_dst, ktil, src, seq_len, status):
        return
    i32, f32 = torch.int32, torch.float32
    n_pages, H_kv = _shape(kv_pages, "kv_pages", 5)[:2]
    _explain(idx, _F8, (n_pages, H_kv, 2, BLK, D), kv_pages=kv_pages)
    _explain(idx, f32, (n_pages, H_kv, 2), kv_scale=kv_scale)
    _explain(idx, i32, tuple(_shape(copy_src, "copy_src", 1)), copy_src=copy_src, copy_dst=copy_dst)
    if ktil is not None:
        B, _, N_cap, _ = _shape(ktil, "ktil", 4)
        _explain(idx, f32, (B, H_kv, N_cap, D), ktil=ktil)
        _explain(idx, i32, (B,), src=src, seq_len=seq_len)
    if status is not None:
        _explain(idx, i32, (1,), status=status)
    raise _refused("sparse_paged_copy_f8")

"""ctypes binding of libdsa_indexer.so (argument marshalling only).

Every function here has the name of the C entry point it calls. Tensors are torch CUDA
tensors; the binding checks dtype, device and contiguity, allocates outputs and workspaces
with torch when the caller does not pass them, and forwards raw pointers and the current
CUDA stream. All computation happens in the library's kernels; if the library is missing
this module raises instead of falling back to anything else.

What the kernels find wrong in device-side inputs (a page, a slot, a length, a value that is not
finite) is recorded in the call's workspace and read with dsa_read_device_status. A call without
a workspace makes one of its own, and its record is lost with it: dsa_latent_attention_prefill
then leaves the rows of a request with bad offsets, or with more than max_q queries, unwritten
without a word.
"""

from __future__ import annotations

import ctypes
import os
from typing import Callable, List, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa_indexer.so")

DSA_OK = 0
DSA_ERR_INVALID = 1
DSA_ERR_UNSUPPORTED = 2
DSA_ERR_CUDA = 3
DSA_ERR_TIMEOUT = 4
DSA_ERR_DEVICE = 5
DSA_MODE_PREFILL = 0
DSA_MODE_DECODE = 1
DSA_WS_HEADER_BYTES = 256
DSA_DTYPE_BF16 = 0
DSA_DTYPE_F16 = 1
DSA_DTYPE_F32 = 2

_i32, _u64, _sz, _vp = ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t, ctypes.c_void_p
_i64, _f32, _f64 = ctypes.c_int64, ctypes.c_float, ctypes.c_double


class dsa_layer_inputs(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_scale", _vp), ("w", _vp), ("k", _vp), ("k_scale", _vp),
                ("out_score", _vp)]


class dsa_indexer_shape(ctypes.Structure):
    _fields_ = [("mode", _i32), ("H", _i32), ("d", _i32), ("topk", _i32),
                ("Lk", _i32), ("q_pos0", _i32), ("Lq", _i32),
                ("n_blocks", _i32), ("block_size", _i32), ("block_table", _vp),
                ("max_blocks", _i32), ("seq_lens", _vp), ("B", _i32)]


AFTER_LAYER_FN = ctypes.CFUNCTYPE(None, _i32, _vp, _vp)

_SIGNATURES = {
    "dsa_abi_version": (_i32, []),
    "dsa_status_string": (ctypes.c_char_p, [_i32]),
    "dsa_workspace_init": (_i32, [_vp, _sz, _vp]),
    "dsa_read_device_status": (_i32, [_vp, _vp, ctypes.POINTER(_i32), ctypes.POINTER(_i32)]),
    "dsa_prefill_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "dsa_indexer_prefill": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                   _vp, _vp, _vp, _sz, _vp]),
    "dsa_decode_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "dsa_indexer_decode": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _i32,
                                  _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "dsa_indexcache_workspace_bytes": (_sz, [ctypes.POINTER(dsa_indexer_shape)]),
    "indexcache_run": (_i32, [ctypes.c_char_p, _i32, ctypes.POINTER(dsa_indexer_shape),
                              ctypes.POINTER(dsa_layer_inputs), ctypes.POINTER(_vp), _i32,
                              ctypes.POINTER(_vp), AFTER_LAYER_FN, _vp, _vp, _sz, _vp]),
    "indexcache_run_lagged": (_i32, [ctypes.c_char_p, _i32, ctypes.POINTER(dsa_indexer_shape),
                                     ctypes.POINTER(dsa_layer_inputs), ctypes.POINTER(_vp), _i32,
                                     ctypes.POINTER(_vp), AFTER_LAYER_FN, _vp, _vp, _sz, _vp, _vp]),
    "topk_overlap": (_i32, [ctypes.POINTER(_vp), _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                            _sz, _vp]),
    "dsa_selftest_wait_timeout": (_i32, [_vp, _sz, _u64, _vp]),
    "dsa_overlap_blocks": (_i32, [_vp, _i32, ctypes.c_double, _vp]),
    "dsa_pattern_from_overlap": (_i32, [_vp, _i32, _i32, ctypes.c_char_p, ctypes.POINTER(ctypes.c_double)]),
    "dsa_topk_merge": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "dsa_indexer_decode_noalloc": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _i32,
                                          _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "dsa_sparse_attention_workspace_bytes": (_sz, [_i32, _i32]),
    "dsa_sparse_attention_decode": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32,
                                           _i32, _i32, ctypes.c_float, _vp, _vp, _sz, _vp]),
    "dsa_rotary": (_i32, [_vp, _i64, _i64, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32,
                          _vp, _i64, _i64, _vp]),
    "dsa_rotary_frequencies": (_i32, [_i32, _f64, _f64, _i32, _f64, _f64, _vp, _vp]),
    "dsa_index_quantise": (_i32, [_vp, _i64, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _i32, _i32, _i32, _f32,
                                  _vp, _vp, _vp, _sz, _vp]),
    "dsa_index_cache_write": (_i32, [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _f32, _vp,
                                     _vp, _i32, _i32, _vp, _sz, _vp]),
    "dsa_index_cache_read": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _i32, _i64, _vp, _vp,
                                    _vp, _i32, _vp, _sz, _vp]),
    "dsa_latent_attention_decode_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "dsa_latent_attention_prefill_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "dsa_latent_attention_decode": (_i32, [_vp, _i64, _i64, _vp, _i32, _i32, _vp, _i32, _vp, _i32, _i32, _i32,
                                           _i32, _i32, _i32, _f32, _vp, _vp, _vp, _sz, _vp]),
    "dsa_latent_attention_prefill": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp,
                                            _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                            _f32, _vp, _vp, _vp, _sz, _vp]),
}

_LIB: Optional[ctypes.CDLL] = None


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Loads libdsa_indexer.so (built in-tree by sparse_attention_token_04_b200.build)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m "
                               "sparse_attention_token_04_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def status_string(status: int) -> str:
    return lib().dsa_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != DSA_OK:
        raise DsaError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype, shape=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor], stream) -> torch.Tensor:
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
        if workspace.numel() < nbytes:
            raise ValueError(f"workspace too small: {workspace.numel()} < {nbytes}")
        return workspace
    ws = torch.empty(max(nbytes, DSA_WS_HEADER_BYTES), dtype=torch.uint8, device=device)
    _check(lib().dsa_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "dsa_workspace_init")
    return ws


def dsa_abi_version() -> int:
    return int(lib().dsa_abi_version())


def dsa_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    _check(lib().dsa_workspace_init(_ptr(workspace), workspace.numel(), _stream(stream)),
           "dsa_workspace_init")


def dsa_read_device_status(workspace: torch.Tensor, stream=None):
    """Returns (status, detail) recorded on the device since the last read, and clears it."""
    st, det = _i32(0), _i32(0)
    _check(lib().dsa_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(st),
                                        ctypes.byref(det)), "dsa_read_device_status")
    return int(st.value), int(det.value)


def dsa_prefill_workspace_bytes(Lq: int, H: int, d: int, topk: int) -> int:
    return int(lib().dsa_prefill_workspace_bytes(Lq, H, d, topk))


def dsa_decode_workspace_bytes(B: int, max_len: int, H: int, d: int, topk: int) -> int:
    return int(lib().dsa_decode_workspace_bytes(B, max_len, H, d, topk))


def dsa_indexer_prefill(q, q_scale, w, k, k_scale, topk: int, q_pos0: int = 0,
                        out_idx=None, out_score=None, want_score: bool = True,
                        workspace=None, stream=None):
    """Prefill indexer: q[Lq][H][d] u8, q_scale[Lq] f32, w[Lq][H] f32, k[Lk][d] u8, k_scale[Lk]
    f32 -> (out_idx[Lq][topk] i32, out_score[Lq][topk] f32 or None)."""
    Lq, H, d = (int(x) for x in q.shape)
    Lk = int(k.shape[0])
    _need(q, "q", torch.uint8)
    _need(q_scale, "q_scale", torch.float32, (Lq,))
    _need(w, "w", torch.float32, (Lq, H))
    _need(k, "k", torch.uint8, (Lk, d))
    _need(k_scale, "k_scale", torch.float32, (Lk,))
    if out_idx is None:
        out_idx = torch.empty(Lq, topk, dtype=torch.int32, device=q.device)
    _need(out_idx, "out_idx", torch.int32, (Lq, topk))
    if out_score is None and want_score:
        out_score = torch.empty(Lq, topk, dtype=torch.float32, device=q.device)
    if out_score is not None:
        _need(out_score, "out_score", torch.float32, (Lq, topk))
    nbytes = dsa_prefill_workspace_bytes(Lq, H, d, topk)
    ws = _workspace(nbytes, q.device, workspace, stream)
    _check(lib().dsa_indexer_prefill(_ptr(q), _ptr(q_scale), _ptr(w), _ptr(k), _ptr(k_scale), Lk,
                                     q_pos0, Lq, H, d, topk, _ptr(out_idx), _ptr(out_score),
                                     _ptr(ws), ws.numel(), _stream(stream)), "dsa_indexer_prefill")
    return out_idx, out_score


def dsa_indexer_decode(q, q_scale, w, k_cache, k_scale_cache, block_table, seq_lens, topk: int,
                       out_idx=None, out_score=None, want_score: bool = True, workspace=None,
                       stream=None):
    """Decode indexer over a paged cache: q[B][H][d] u8, k_cache[n_blocks][block_size][d] u8,
    k_scale_cache[n_blocks][block_size] f32, block_table[B][max_blocks] i32, seq_lens[B] i32
    -> (out_idx[B][topk] i32 logical positions, out_score[B][topk] f32 or None)."""
    B, H, d = (int(x) for x in q.shape)
    n_blocks, block_size = int(k_cache.shape[0]), int(k_cache.shape[1])
    max_blocks = int(block_table.shape[1])
    _need(q, "q", torch.uint8)
    _need(q_scale, "q_scale", torch.float32, (B,))
    _need(w, "w", torch.float32, (B, H))
    _need(k_cache, "k_cache", torch.uint8, (n_blocks, block_size, d))
    _need(k_scale_cache, "k_scale_cache", torch.float32, (n_blocks, block_size))
    _need(block_table, "block_table", torch.int32, (B, max_blocks))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out_idx is None:
        out_idx = torch.empty(B, topk, dtype=torch.int32, device=q.device)
    _need(out_idx, "out_idx", torch.int32, (B, topk))
    if out_score is None and want_score:
        out_score = torch.empty(B, topk, dtype=torch.float32, device=q.device)
    if out_score is not None:
        _need(out_score, "out_score", torch.float32, (B, topk))
    nbytes = dsa_decode_workspace_bytes(B, max_blocks * block_size, H, d, topk)
    ws = _workspace(nbytes, q.device, workspace, stream)
    _check(lib().dsa_indexer_decode(_ptr(q), _ptr(q_scale), _ptr(w), _ptr(k_cache),
                                    _ptr(k_scale_cache), n_blocks, block_size, _ptr(block_table),
                                    max_blocks, _ptr(seq_lens), B, H, d, topk, _ptr(out_idx),
                                    _ptr(out_score), _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_indexer_decode")
    return out_idx, out_score


def _shape_struct(mode: int, H: int, d: int, topk: int, **kw) -> dsa_indexer_shape:
    s = dsa_indexer_shape()
    s.mode, s.H, s.d, s.topk = mode, H, d, topk
    for name in ("Lk", "q_pos0", "Lq", "n_blocks", "block_size", "max_blocks", "B"):
        setattr(s, name, int(kw.get(name, 0)))
    bt, sl = kw.get("block_table"), kw.get("seq_lens")
    s.block_table = bt.data_ptr() if bt is not None else None
    s.seq_lens = sl.data_ptr() if sl is not None else None
    return s


def dsa_indexcache_workspace_bytes(shape: dsa_indexer_shape) -> int:
    return int(lib().dsa_indexcache_workspace_bytes(ctypes.byref(shape)))


def _indexcache_args(pattern, layers, topk, mode, f_bufs, n_bufs_default, q_pos0, block_table,
                     seq_lens):
    n_layers = len(pattern)
    if len(layers) != n_layers:
        raise ValueError("one layer entry per pattern character")
    first = next((layers[l] for l, c in enumerate(pattern) if c == "F" and layers[l] is not None), None)
    if first is None:
        raise ValueError("no Full layer inputs")
    H, d = int(first["q"].shape[1]), int(first["q"].shape[2])
    if mode == DSA_MODE_PREFILL:
        Lq, Lk = int(first["q"].shape[0]), int(first["k"].shape[0])
        shape = _shape_struct(mode, H, d, topk, Lk=Lk, q_pos0=q_pos0, Lq=Lq)
        rows = Lq
    else:
        kc = first["k_cache"]
        B = int(first["q"].shape[0])
        _need(block_table, "block_table", torch.int32)
        _need(seq_lens, "seq_lens", torch.int32, (B,))
        shape = _shape_struct(mode, H, d, topk, n_blocks=int(kc.shape[0]), block_size=int(kc.shape[1]),
                              max_blocks=int(block_table.shape[1]), B=B, block_table=block_table,
                              seq_lens=seq_lens)
        rows = B
    if f_bufs is None:
        f_bufs = [torch.empty(rows, topk, dtype=torch.int32, device=first["q"].device)
                  for _ in range(n_bufs_default)]
    for b in f_bufs:
        _need(b, "f_buf", torch.int32, (rows, topk))
    arr = (dsa_layer_inputs * n_layers)()
    for l, lay in enumerate(layers):
        if lay is None:
            continue
        kk = lay["k"] if mode == DSA_MODE_PREFILL else lay["k_cache"]
        ks = lay["k_scale"] if mode == DSA_MODE_PREFILL else lay["k_scale_cache"]
        arr[l] = dsa_layer_inputs(lay["q"].data_ptr(), lay["q_scale"].data_ptr(), lay["w"].data_ptr(),
                                  kk.data_ptr(), ks.data_ptr(),
                                  lay["out_score"].data_ptr() if lay.get("out_score") is not None else None)
    fb = (_vp * len(f_bufs))(*[b.data_ptr() for b in f_bufs])
    return shape, arr, fb, f_bufs, first["q"].device


def indexcache_run(pattern: str, layers: Sequence[Optional[dict]], topk: int, mode: int = DSA_MODE_PREFILL,
                   f_bufs: Optional[List[torch.Tensor]] = None, keep_all: bool = True,
                   q_pos0: int = 0, block_table=None, seq_lens=None,
                   after_layer: Optional[Callable[[int, int], None]] = None,
                   workspace=None, stream=None):
    """IndexCache driver. `layers[l]` is a dict of the layer's tensors (q, q_scale, w, k,
    k_scale, optional out_score) for prefill, or (q, q_scale, w, k_cache, k_scale_cache) for
    decode; entries of S layers may be None. Returns (f_bufs, out_layer_ptrs) where
    out_layer_ptrs[l] is the device address of the buffer holding layer l's indices."""
    n_full = pattern.count("F")
    shape, arr, fb, f_bufs, dev = _indexcache_args(pattern, layers, topk, mode, f_bufs,
                                                   n_full if keep_all else 1, q_pos0, block_table,
                                                   seq_lens)
    out_ptrs = (_vp * len(pattern))()
    cb = AFTER_LAYER_FN(lambda l, p, u: after_layer(int(l), int(p or 0))) if after_layer else AFTER_LAYER_FN()
    ws = _workspace(dsa_indexcache_workspace_bytes(shape), dev, workspace, stream)
    _check(lib().indexcache_run(pattern.encode(), len(pattern), ctypes.byref(shape), arr, fb, len(f_bufs),
                                out_ptrs, cb, None, _ptr(ws), ws.numel(), _stream(stream)),
           "indexcache_run")
    return f_bufs, [int(p or 0) for p in out_ptrs]


def indexcache_run_lagged(pattern: str, layers: Sequence[Optional[dict]], topk: int,
                          indexer_stream, mode: int = DSA_MODE_PREFILL,
                          f_bufs: Optional[List[torch.Tensor]] = None, keep_all: bool = True,
                          q_pos0: int = 0, block_table=None, seq_lens=None,
                          consume: Optional[Callable[[int, int], None]] = None,
                          workspace=None, stream=None):
    """Multi-layer-indexer variant of indexcache_run: every Full layer's indexer runs on
    `indexer_stream` while layer l's consumer (called as consume(l, ptr), enqueuing on `stream`)
    reads the selection of the last Full layer before l (layer 0: its own). Returns (f_bufs,
    out_layer_ptrs)."""
    n_full = pattern.count("F")
    shape, arr, fb, f_bufs, dev = _indexcache_args(pattern, layers, topk, mode, f_bufs,
                                                   n_full if keep_all else min(2, n_full), q_pos0,
                                                   block_table, seq_lens)
    out_ptrs = (_vp * len(pattern))()
    cb = AFTER_LAYER_FN(lambda l, p, u: consume(int(l), int(p or 0))) if consume else AFTER_LAYER_FN()
    ws = _workspace(dsa_indexcache_workspace_bytes(shape), dev, workspace, stream)
    _check(lib().indexcache_run_lagged(pattern.encode(), len(pattern), ctypes.byref(shape), arr, fb,
                                       len(f_bufs), out_ptrs, cb, None, _ptr(ws), ws.numel(),
                                       _stream(stream), _stream(indexer_stream)),
           "indexcache_run_lagged")
    return f_bufs, [int(p or 0) for p in out_ptrs]


def topk_overlap(layer_idx: Sequence[torch.Tensor], n_keys: int, out_counts=None, out_valid=None,
                 out_overlap=None, workspace=None, stream=None):
    """Overlap of N index tensors [rows][topk] i32 -> (counts[N][N] u64 as int64 tensor,
    valid[1], overlap[N][N] f64)."""
    N = len(layer_idx)
    rows, topk = (int(x) for x in layer_idx[0].shape)
    for t in layer_idx:
        _need(t, "layer_idx", torch.int32, (rows, topk))
    dev = layer_idx[0].device
    if out_counts is None:
        out_counts = torch.empty(N, N, dtype=torch.int64, device=dev)
    if out_valid is None:
        out_valid = torch.empty(1, dtype=torch.int64, device=dev)
    if out_overlap is None:
        out_overlap = torch.empty(N, N, dtype=torch.float64, device=dev)
    ws = _workspace(DSA_WS_HEADER_BYTES, dev, workspace, stream)
    ptrs = (_vp * N)(*[t.data_ptr() for t in layer_idx])
    _check(lib().topk_overlap(ptrs, N, rows, topk, n_keys, _ptr(out_counts), _ptr(out_valid),
                              _ptr(out_overlap), _ptr(ws), ws.numel(), _stream(stream)), "topk_overlap")
    return out_counts, out_valid, out_overlap


def topk_overlap_ptrs(ptrs: Sequence[int], rows: int, topk: int, n_keys: int, out_counts,
                      out_valid, out_overlap=None, workspace=None, stream=None):
    """Same as topk_overlap for raw device addresses (e.g. the aliased layer buffers that
    indexcache_run reports)."""
    N = len(ptrs)
    ws = _workspace(DSA_WS_HEADER_BYTES, out_counts.device, workspace, stream)
    arr = (_vp * N)(*ptrs)
    _check(lib().topk_overlap(arr, N, rows, topk, n_keys, _ptr(out_counts), _ptr(out_valid),
                              _ptr(out_overlap), _ptr(ws), ws.numel(), _stream(stream)), "topk_overlap")
    return out_counts, out_valid, out_overlap


def dsa_selftest_wait_timeout(workspace: torch.Tensor, budget_ns: int, stream=None) -> None:
    _check(lib().dsa_selftest_wait_timeout(_ptr(workspace), workspace.numel(), int(budget_ns),
                                           _stream(stream)), "dsa_selftest_wait_timeout")


def dsa_topk_merge(scores, idx, idx_offset=None, out_idx=None, out_score=None, stream=None):
    """Top-k of the union of n_lists top-k lists per row: scores [n_lists][rows][topk] f32 and
    idx [n_lists][rows][topk] i32 (each row sorted as the indexer writes it), idx_offset
    [n_lists][rows] i32 added to each list row's valid indices (or None) -> (out_idx[rows][topk]
    i32, out_score[rows][topk] f32)."""
    n_lists, rows, topk = (int(x) for x in idx.shape)
    _need(idx, "idx", torch.int32)
    _need(scores, "scores", torch.float32, (n_lists, rows, topk))
    if idx_offset is not None:
        _need(idx_offset, "idx_offset", torch.int32, (n_lists, rows))
    if out_idx is None:
        out_idx = torch.empty(rows, topk, dtype=torch.int32, device=idx.device)
    _need(out_idx, "out_idx", torch.int32, (rows, topk))
    if out_score is None:
        out_score = torch.empty(rows, topk, dtype=torch.float32, device=idx.device)
    _need(out_score, "out_score", torch.float32, (rows, topk))
    _check(lib().dsa_topk_merge(_ptr(scores), _ptr(idx), _ptr(idx_offset), n_lists, rows, topk,
                                _ptr(out_idx), _ptr(out_score), _stream(stream)), "dsa_topk_merge")
    return out_idx, out_score


def _host_overlap(overlap):
    import numpy as np
    o = np.ascontiguousarray(np.asarray(overlap.cpu() if isinstance(overlap, torch.Tensor) else overlap,
                                        dtype=np.float64))
    if o.ndim != 2 or o.shape[0] != o.shape[1]:
        raise ValueError("overlap must be a square [n_layers][n_layers] matrix")
    return o


def dsa_overlap_blocks(overlap, threshold: float):
    """Blocks of layers from an overlap matrix (host): returns (n_blocks, block_of_layer list)."""
    import numpy as np
    o = _host_overlap(overlap)
    n = o.shape[0]
    out = np.zeros(n, dtype=np.int32)
    nb = int(lib().dsa_overlap_blocks(o.ctypes.data, n, float(threshold), out.ctypes.data))
    if nb < 0:
        raise DsaError(DSA_ERR_INVALID, "dsa_overlap_blocks")
    return nb, out.tolist()


def dsa_pattern_from_overlap(overlap, n_full: int):
    """The F/S pattern with n_full Full layers that keeps the most overlap (host): returns
    (pattern, mean overlap kept per layer)."""
    o = _host_overlap(overlap)
    n = o.shape[0]
    buf = ctypes.create_string_buffer(n + 1)
    kept = ctypes.c_double(0.0)
    _check(lib().dsa_pattern_from_overlap(o.ctypes.data, n, int(n_full), buf, ctypes.byref(kept)),
           "dsa_pattern_from_overlap")
    return buf.value.decode(), float(kept.value)


DSA_DECODE_MAX_REQUESTS = 65535
DSA_NOALLOC_MAX_SCORES = 4194304
DSA_NOALLOC_MAX_REQUESTS = 256


def dsa_indexer_decode_noalloc(q, q_scale, w, k_cache, k_scale_cache, block_table, seq_lens,
                               topk: int, out_idx, out_score=None, device_status=None, stream=None):
    """Decode indexer that allocates no device memory: for callers that must not allocate at
    step time. Outputs (and the optional device int32[2] status) are passed in by the caller;
    the library's fixed scratch bounds B * max_blocks * block_size by DSA_NOALLOC_MAX_SCORES."""
    B, H, d = (int(x) for x in q.shape)
    n_blocks, block_size = int(k_cache.shape[0]), int(k_cache.shape[1])
    max_blocks = int(block_table.shape[1])
    _need(q, "q", torch.uint8)
    _need(q_scale, "q_scale", torch.float32, (B,))
    _need(w, "w", torch.float32, (B, H))
    _need(k_cache, "k_cache", torch.uint8, (n_blocks, block_size, d))
    _need(k_scale_cache, "k_scale_cache", torch.float32, (n_blocks, block_size))
    _need(block_table, "block_table", torch.int32, (B, max_blocks))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    _need(out_idx, "out_idx", torch.int32, (B, topk))
    if out_score is not None:
        _need(out_score, "out_score", torch.float32, (B, topk))
    if device_status is not None:
        _need(device_status, "device_status", torch.int32, (2,))
    _check(lib().dsa_indexer_decode_noalloc(_ptr(q), _ptr(q_scale), _ptr(w), _ptr(k_cache),
                                            _ptr(k_scale_cache), n_blocks, block_size,
                                            _ptr(block_table), max_blocks, _ptr(seq_lens), B, H, d,
                                            topk, _ptr(out_idx), _ptr(out_score),
                                            _ptr(device_status), _stream(stream)),
           "dsa_indexer_decode_noalloc")
    return out_idx, out_score


def dsa_sparse_attention_workspace_bytes(B: int, topk: int) -> int:
    return int(lib().dsa_sparse_attention_workspace_bytes(B, topk))


def dsa_sparse_attention_decode(q, latent, block_table, seq_lens, idx, scale: float, block_size: int = 64,
                                out=None, workspace=None, stream=None):
    """Sparse attention of decode queries over their selected latents: q[B][128][576] bf16,
    latent[n_blocks * block_size][576] bf16, block_table[B][max_blocks] i32, seq_lens[B] i32,
    idx[B][topk] i32 -> out[B][128][512] f32."""
    B, Hq, dqk = (int(x) for x in q.shape)
    n_rows = int(latent.shape[0])
    topk = int(idx.shape[1])
    _need(q, "q", torch.bfloat16)
    _need(latent, "latent", torch.bfloat16, (n_rows, dqk))
    _need(block_table, "block_table", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    _need(idx, "idx", torch.int32, (B, topk))
    if n_rows % block_size:
        raise ValueError("latent rows must be whole blocks")
    dv = 512
    if out is None:
        out = torch.empty(B, Hq, dv, dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, (B, Hq, dv))
    ws = _workspace(dsa_sparse_attention_workspace_bytes(B, topk), q.device, workspace, stream)
    _check(lib().dsa_sparse_attention_decode(_ptr(q), _ptr(latent), n_rows // block_size, block_size,
                                             _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
                                             _ptr(idx), B, Hq, dqk, dv, topk, float(scale), _ptr(out),
                                             _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_sparse_attention_decode")
    return out


_DTYPES = {torch.bfloat16: DSA_DTYPE_BF16, torch.float16: DSA_DTYPE_F16, torch.float32: DSA_DTYPE_F32}
_HALF = (torch.bfloat16, torch.float16)


def _rows(t, name: str, dtypes, shape) -> None:
    """A CUDA tensor of one of `dtypes` whose last dimension is contiguous (other strides are free)."""
    if type(t) is torch.Tensor and t.is_cuda and t.dtype in dtypes and t.shape == shape and t.stride(-1) == 1:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _strides(t):
    """Strides in elements; that of a dimension of one entry says nothing and is taken as 8."""
    st, shape = t.stride(), t.shape
    return [8 if n == 1 else k for n, k in zip(shape, st)] if 1 in shape else st


def _fits(t, name: str, dtype, shape) -> None:
    """As _need with a shape; the usual case in one expression."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, shape)


def _addr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it, which takes longer to make than a
# small call's launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _leave(held) -> None:
    while held:
        held.pop().__exit__(None, None, None)


def _enter(stream, first: torch.Tensor, *others):
    """Makes the device of `first` (every tensor's) current and, where a stream other than the current
    one is given, that stream too, so that what the call allocates belongs to the stream that uses it.
    Returns (the stream's handle, contexts for _leave)."""
    device = first.get_device()
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on {first.device} and {t.device}")
    held = []
    if device != torch.cuda.current_device():
        held.append(torch.cuda.device(device))
        held[-1].__enter__()
    now = _raw_stream(device)
    if stream is None:
        return now, held
    raw = int(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream)
    if raw != now:
        if isinstance(stream, torch.cuda.Stream) and stream.device_index != device:
            _leave(held)
            raise ValueError(f"a stream of device {stream.device_index} for tensors on {first.device}")
        held.append(torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                                      else torch.cuda.ExternalStream(raw, device=device)))
        held[-1].__enter__()
    return raw, held


def _rotation(T: int, d: int, positions, inv_freq):
    """rot dims of a call's rotation, 0 where no positions are given."""
    if positions is None:
        if inv_freq is not None:
            raise ValueError("inv_freq without positions")
        return 0
    _fits(positions, "positions", torch.int32, (T,))
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a tensor of shape (rot // 2,)")
    half = inv_freq.shape[0]
    _fits(inv_freq, "inv_freq", torch.float32, (half,))
    return 2 * half


def dsa_rotary_frequencies(rot: int, theta: float = 10000.0, factor: float = 1.0, original_len: int = 4096,
                           beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Rotary frequencies (host): returns (inv_freq[rot // 2] f32 tensor on `device`, mscale), scaled
    for contexts `factor` times as long as original_len where factor > 1."""
    out = torch.empty(max(int(rot) // 2, 0), dtype=torch.float32)
    m = ctypes.c_float(0.0)
    _check(lib().dsa_rotary_frequencies(int(rot), float(theta), float(factor), int(original_len), float(beta_fast),
                                        float(beta_slow), _ptr(out) if out.numel() else None, ctypes.byref(m)),
           "dsa_rotary_frequencies")
    return (out if device is None else out.to(device)), float(m.value)


def dsa_rotary(x, positions, inv_freq, interleaved: bool = False, rot_offset: int = 0, mscale: float = 1.0,
               inverse: bool = False, out=None, stream=None):
    """Rotary positions: x[T][H][d] bf16 / f16 / f32 (last dimension contiguous), positions[T] i32,
    inv_freq[rot // 2] f32 -> out like x, the dims [rot_offset, rot_offset + rot) of every head turned by
    positions * inv_freq. out may be x; inverse turns back (the gradient of the rotation)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a tensor of shape (T, H, d)")
    T, H, d = x.shape
    _rows(x, "x", _DTYPES, x.shape)
    rot = _rotation(T, d, positions, inv_freq)
    if rot == 0:
        raise ValueError("positions and inv_freq are needed")
    s, held = _enter(stream, x, positions, inv_freq, out)
    try:
        if out is None:
            out = x.new_empty((T, H, d))
        else:
            _rows(out, "out", (x.dtype,), x.shape)
        xs, os_ = _strides(x), _strides(out)
        _check(lib().dsa_rotary(x.data_ptr(), xs[0], xs[1], positions.data_ptr(), inv_freq.data_ptr(), T, H, d, rot,
                                int(rot_offset), int(interleaved), int(inverse), mscale, _DTYPES[x.dtype],
                                out.data_ptr(), os_[0], os_[1], s), "dsa_rotary")
    finally:
        _leave(held)
    return out


def dsa_index_quantise(x, positions=None, inv_freq=None, interleaved: bool = False, rot_offset: int = 0,
                       mscale: float = 1.0, codes=None, scale=None, workspace=None, stream=None):
    """E4M3 inputs of the indexer: x[T][H][d] (queries) or x[T][d] (keys) bf16 / f16 / f32, rotated where
    positions are given -> (codes u8 of x's shape, scale[T] f32)."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x must be a tensor of shape (T, H, d) or (T, d)")
    T, d = x.shape[0], x.shape[-1]
    H = x.shape[1] if x.dim() == 3 else 1
    _rows(x, "x", _DTYPES, x.shape)
    rot = _rotation(T, d, positions, inv_freq)
    s, held = _enter(stream, x, positions, inv_freq, codes, scale, workspace)
    try:
        if codes is None:
            codes = x.new_empty((T, H, d) if x.dim() == 3 else (T, d), dtype=torch.uint8)
        else:
            _fits(codes, "codes", torch.uint8, x.shape)
        if scale is None:
            scale = x.new_empty((T,), dtype=torch.float32)
        else:
            _fits(scale, "scale", torch.float32, (T,))
        ws = _workspace(DSA_WS_HEADER_BYTES, x.device, workspace, s)
        xs = _strides(x)
        _check(lib().dsa_index_quantise(x.data_ptr(), xs[0], xs[1] if x.dim() == 3 else 8, T, H, d, _DTYPES[x.dtype],
                                        _addr(positions), _addr(inv_freq), rot, int(rot_offset), int(interleaved),
                                        mscale, codes.data_ptr(), scale.data_ptr(), ws.data_ptr(), ws.numel(), s),
               "dsa_index_quantise")
    finally:
        _leave(held)
    return codes, scale


def dsa_index_cache_write(x, slots, k_cache, k_scale_cache, positions=None, inv_freq=None, interleaved: bool = False,
                          rot_offset: int = 0, mscale: float = 1.0, workspace=None, stream=None):
    """Quantises keys x[T][d] bf16 / f16 / f32 (rotated where positions are given) into the paged cache
    k_cache[n_blocks][block_size][d] u8, k_scale_cache[n_blocks][block_size] f32 at slots[T] i64 (-1: not
    written)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor of shape (T, d)")
    T, d = x.shape
    _rows(x, "x", _DTYPES, x.shape)
    n_blocks, block_size = k_cache.shape[0], k_cache.shape[1]
    _fits(slots, "slots", torch.int64, (T,))
    _fits(k_cache, "k_cache", torch.uint8, (n_blocks, block_size, d))
    _fits(k_scale_cache, "k_scale_cache", torch.float32, (n_blocks, block_size))
    rot = _rotation(T, d, positions, inv_freq)
    s, held = _enter(stream, x, slots, k_cache, k_scale_cache, positions, inv_freq, workspace)
    try:
        ws = _workspace(DSA_WS_HEADER_BYTES, x.device, workspace, s)
        _check(lib().dsa_index_cache_write(x.data_ptr(), _strides(x)[0], T, d, _DTYPES[x.dtype], slots.data_ptr(),
                                           _addr(positions), _addr(inv_freq), rot, int(rot_offset), int(interleaved),
                                           mscale, k_cache.data_ptr(), k_scale_cache.data_ptr(), n_blocks, block_size,
                                           ws.data_ptr(), ws.numel(), s), "dsa_index_cache_write")
    finally:
        _leave(held)


def dsa_index_cache_read(k_cache, k_scale_cache, block_table, cu_rows, total: int, starts=None,
                         want_codes: bool = True, values=None, out_codes=None, out_scale=None, out_values=None,
                         workspace=None, stream=None):
    """Reads request ranges of the paged key cache: rows cu_rows[b] .. cu_rows[b + 1] of the outputs are
    positions starts[b] .. (0 .. without starts) of request b -> (codes[total][d] u8, scale[total] f32,
    values[total][d] of the type `values`), the first two None without want_codes, the last without values."""
    n_blocks, block_size, d = k_cache.shape
    B, max_blocks = block_table.shape
    total = int(total)
    _fits(k_cache, "k_cache", torch.uint8, (n_blocks, block_size, d))
    _fits(k_scale_cache, "k_scale_cache", torch.float32, (n_blocks, block_size))
    _fits(block_table, "block_table", torch.int32, (B, max_blocks))
    _fits(cu_rows, "cu_rows", torch.int32, (B + 1,))
    if starts is not None:
        _fits(starts, "starts", torch.int32, (B,))
    if out_values is not None and values is None:
        values = out_values.dtype
    if values is not None and values not in _DTYPES:
        raise ValueError(f"values must be one of {[str(t) for t in _DTYPES]}, got {values}")
    s, held = _enter(stream, k_cache, k_scale_cache, block_table, cu_rows, starts, out_codes, out_scale,
                      out_values, workspace)
    try:
        if out_codes is not None:
            _fits(out_codes, "out_codes", torch.uint8, (total, d))
        elif want_codes:
            out_codes = k_cache.new_empty((total, d))
        if out_scale is not None:
            _fits(out_scale, "out_scale", torch.float32, (total,))
        elif want_codes:
            out_scale = k_scale_cache.new_empty((total,))
        if out_values is not None:
            _fits(out_values, "out_values", values, (total, d))
        elif values is not None:
            out_values = k_cache.new_empty((total, d), dtype=values)
        ws = _workspace(DSA_WS_HEADER_BYTES, k_cache.device, workspace, s)
        _check(lib().dsa_index_cache_read(k_cache.data_ptr(), k_scale_cache.data_ptr(), n_blocks, block_size, d,
                                          block_table.data_ptr(), max_blocks, _addr(starts), cu_rows.data_ptr(), B,
                                          total, _addr(out_codes), _addr(out_scale), _addr(out_values),
                                          _DTYPES.get(values, DSA_DTYPE_F32), ws.data_ptr(), ws.numel(), s),
               "dsa_index_cache_read")
    finally:
        _leave(held)
    return out_codes, out_scale, out_values


def dsa_latent_attention_decode_workspace_bytes(B: int, q_len: int, Hq: int) -> int:
    return int(lib().dsa_latent_attention_decode_workspace_bytes(B, q_len, Hq))


def dsa_latent_attention_decode(q, latent, block_table, seq_lens, scale: float, block_size: int = 64, out=None,
                                lse=None, want_lse: bool = True, workspace=None, stream=None):
    """Dense latent attention of 1 to 8 new tokens a request over the paged latents (absorbed form):
    q[B][q_len][Hq][576] or q[B][Hq][576] bf16 / f16, latent[n_blocks * block_size][576],
    block_table[B][max_blocks] i32, seq_lens[B] i32 -> (out like q with 512 dims, lse[B][q_len][Hq] or
    [B][Hq] f32)."""
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
        raise ValueError("q must be a tensor of shape (B, q_len, Hq, 576) or (B, Hq, 576)")
    shape = q.shape
    _rows(q, "q", _HALF, shape)
    st = _strides(q)
    B, q_len, Hq, dqk = shape if len(shape) == 4 else (shape[0], 1, shape[1], shape[2])
    if B > 1 and q_len > 1 and st[0] != q_len * st[1]:
        raise ValueError("q's tokens must be evenly spaced over its requests")
    # (..., q_len, Hq) of the outputs, and the stride from one token to the next
    tokens = (B, q_len, Hq) if len(shape) == 4 else (B, Hq)
    q_stride_t = st[1] if q_len > 1 else st[0]
    n_rows, max_blocks, dv = latent.shape[0], block_table.shape[-1], 512
    _fits(latent, "latent", q.dtype, (n_rows, dqk))
    _fits(block_table, "block_table", torch.int32, (B, max_blocks))
    _fits(seq_lens, "seq_lens", torch.int32, (B,))
    if block_size < 1 or n_rows % block_size:
        raise ValueError("latent rows must be whole blocks")
    s, held = _enter(stream, q, latent, block_table, seq_lens, out, lse, workspace)
    try:
        if out is None:
            out = q.new_empty(tokens + (dv,))
        else:
            _fits(out, "out", q.dtype, tokens + (dv,))
        if lse is None and want_lse:
            lse = q.new_empty(tokens, dtype=torch.float32)
        elif lse is not None:
            _fits(lse, "lse", torch.float32, tokens)
        ws = _workspace(dsa_latent_attention_decode_workspace_bytes(B, q_len, Hq), q.device, workspace, s)
        _check(lib().dsa_latent_attention_decode(q.data_ptr(), q_stride_t, st[-2], latent.data_ptr(),
                                                 n_rows // block_size, block_size, block_table.data_ptr(), max_blocks,
                                                 seq_lens.data_ptr(), B, q_len, Hq, dqk, dv, _DTYPES[q.dtype], scale,
                                                 out.data_ptr(), _addr(lse), ws.data_ptr(), ws.numel(), s),
               "dsa_latent_attention_decode")
    finally:
        _leave(held)
    return out, lse


def dsa_latent_attention_prefill_workspace_bytes(B: int, Tq: int, Tk: int, max_q: int, H: int,
                                                 causal: bool = True) -> int:
    return int(lib().dsa_latent_attention_prefill_workspace_bytes(B, Tq, Tk, max_q, H, int(causal)))


def dsa_latent_attention_prefill(q, k_nope, k_pe, v, cu_q, cu_k, max_q: int, scale: float, causal: bool = True,
                                 out=None, lse=None, want_lse: bool = True, workspace=None, stream=None):
    """Latent attention of ragged prefills (expanded form): q[Tq][H][192], k_nope[Tk][H][128], k_pe[Tk][64],
    v[Tk][H][128] bf16 / f16 (last dimensions contiguous), request offsets cu_q, cu_k [B + 1] i32, at most
    max_q queries a request -> (out[Tq][H][128], lse[Tq][H] f32)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor of shape (Tq, H, 192)")
    Tq, H, dqk = q.shape
    _rows(q, "q", _HALF, (Tq, H, dqk))
    Tk, d_nope, d_pe, dv = k_pe.shape[0], k_nope.shape[-1], k_pe.shape[-1], v.shape[-1]
    _rows(k_nope, "k_nope", (q.dtype,), (Tk, H, d_nope))
    _rows(k_pe, "k_pe", (q.dtype,), (Tk, d_pe))
    _rows(v, "v", (q.dtype,), (Tk, H, dv))
    if d_nope + d_pe != dqk:
        raise ValueError("q's heads must be as wide as k_nope's and k_pe together")
    B = cu_q.numel() - 1
    _fits(cu_q, "cu_q", torch.int32, (B + 1,))
    _fits(cu_k, "cu_k", torch.int32, (B + 1,))
    s, held = _enter(stream, q, k_nope, k_pe, v, cu_q, cu_k, out, lse, workspace)
    try:
        if out is None:
            out = q.new_empty((Tq, H, dv))
        else:
            _fits(out, "out", q.dtype, (Tq, H, dv))
        if lse is None and want_lse:
            lse = q.new_empty((Tq, H), dtype=torch.float32)
        elif lse is not None:
            _fits(lse, "lse", torch.float32, (Tq, H))
        if workspace is None:
            workspace = _workspace(dsa_latent_attention_prefill_workspace_bytes(B, Tq, Tk, max_q, H, causal), q.device, None, s)
        ws = _workspace(DSA_WS_HEADER_BYTES, q.device, workspace, s)
        qs, ks, vs = _strides(q), _strides(k_nope), _strides(v)
        _check(lib().dsa_latent_attention_prefill(
            q.data_ptr(), qs[0], qs[1], k_nope.data_ptr(), ks[0], ks[1], k_pe.data_ptr(), _strides(k_pe)[0], v.data_ptr(),
            vs[0], vs[1], cu_q.data_ptr(), cu_k.data_ptr(), B, Tq, Tk, int(max_q), H, d_nope, d_pe, dv, _DTYPES[q.dtype],
            int(causal), scale, out.data_ptr(), _addr(lse), ws.data_ptr(), ws.numel(), s), "dsa_latent_attention_prefill")
    finally:
        _leave(held)
    return out, lse

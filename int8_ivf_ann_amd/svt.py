"""ctypes binding of the C ABI in include/svt.h (argument marshalling only).

Every step of the search runs in the gfx950 kernels of libsvt.so; this module only converts Python
and torch objects into pointers and sizes.  PyTorch provides device memory and streams.  There is no
fallback: if libsvt.so is missing or fails to load, every entry point raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsvt.so")

SVT_OK, SVT_EINVAL, SVT_ENOMEM, SVT_EDEVICE, SVT_EUNSUPPORTED, SVT_ESTATE, SVT_ENOSPACE = 0, -1, -2, -3, -4, -5, -6
SVT_MAX_K = 2048
SVT_MAX_K_LARGE = 16384
SVT_MAX_SIG_WORDS = 2
SVT_PATH_AUTO, SVT_PATH_QUERY, SVT_PATH_TILE, SVT_PATH_EXHAUSTIVE, SVT_PATH_LARGE_K = 0, 1, 2, 3, 4
SVT_OPT_MERGE_FROM_SLOTS, SVT_OPT_FORCE_REDO = 1, 2
SVT_MAX_MASK_GROUPS = 4
SVT_NOALLOC_SCRATCH_BYTES = 256 << 20
SVT_RERANK_MAX_EXPERTS, SVT_RERANK_MAX_UNITS, SVT_RERANK_MAX_CAND, SVT_RERANK_MAX_OUT = 8, 64, 4096, 2048
SVT_F32, SVT_F16, SVT_BF16 = 0, 1, 2
SVT_ACT_NONE, SVT_ACT_RELU, SVT_ACT_SILU, SVT_ACT_GELU = 0, 1, 2, 3
SVT_MAX_EXPERTS, SVT_MAX_TOP = 512, 16
_PATHS = {"auto": SVT_PATH_AUTO, "query": SVT_PATH_QUERY, "tile": SVT_PATH_TILE, "large_k": SVT_PATH_LARGE_K}

#: every symbol include/svt.h declares
EXPORTED = ("svt_index_upload", "svt_index_upload_updatable", "svt_index_insert", "svt_index_delete",
            "svt_index_resign", "svt_index_free", "svt_index_info", "svt_search_workspace_size", "svt_search_path",
            "svt_search", "svt_search_noalloc", "svt_rerank", "svt_route", "svt_route_backward",
            "svt_expert_sort_workspace_size", "svt_expert_sort", "svt_expert_dispatch", "svt_expert_dispatch_backward",
            "svt_expert_combine", "svt_expert_combine_backward", "svt_quant_pack_size", "svt_quant_pack",
            "svt_quant_linear", "svt_embedding", "svt_embedding_backward_workspace_size", "svt_embedding_backward",
            "svt_gated_linear_workspace_size", "svt_gated_linear", "svt_gated_linear_backward_workspace_size", "svt_gated_linear_backward",
            "svt_token_logprobs_workspace_size", "svt_token_logprobs", "svt_token_logprobs_backward", "svt_last_error", "svt_bloom_mask", "svt_bloom_sign", "svt_profile_enable", "svt_profile_read")


class SvtError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"svt error {code}: {msg}")
        self.code = code


class svt_index_desc(ctypes.Structure):
    _fields_ = [
        ("n_items", ctypes.c_int64),
        ("dim", ctypes.c_int32),
        ("sig_words", ctypes.c_int32),
        ("nlist", ctypes.c_int32),
        ("items", ctypes.c_void_p),
        ("sigs", ctypes.c_void_p),
        ("list_of", ctypes.c_void_p),
        ("centroids", ctypes.c_void_p),
        ("item_scale", ctypes.c_float),
    ]


class svt_search_options(ctypes.Structure):
    _fields_ = [
        ("path", ctypes.c_int32),
        ("pool_keys", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("mask_groups", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 4),
    ]


class svt_rerank_net(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("hidden", ctypes.c_int32), ("gate_w", ctypes.c_void_p),
                ("gate_b", ctypes.c_void_p), ("w1", ctypes.c_void_p), ("b1", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("b2", ctypes.c_void_p)]


class svt_quant_weights(ctypes.Structure):
    """Weights in 4 bits (see svt_quant_pack); ``buffer`` keeps the packed tensor alive."""
    _fields_ = [("n_matrices", ctypes.c_int32), ("n_out", ctypes.c_int32), ("n_in", ctypes.c_int32),
                ("group", ctypes.c_int32), ("scale_type", ctypes.c_int32), ("has_zeros", ctypes.c_int32),
                ("packed", ctypes.c_void_p), ("packed_bytes", ctypes.c_size_t)]
    buffer = None


def make_options(path="auto", pool_keys: int = 0, flags: int = 0, mask_groups: int = 0) -> svt_search_options:
    """Search options: path "auto" | "query" | "tile" | "large_k" (or an SVT_PATH_* value), pool_keys (tile path,
    0 = default), flags (OR of SVT_OPT_*), mask_groups (masks per query, 0 or 1: one)."""
    o = svt_search_options()
    o.path = _PATHS[path] if isinstance(path, str) else int(path)
    o.pool_keys = int(pool_keys)
    o.flags = int(flags)
    o.mask_groups = int(mask_groups)
    return o


def _with_groups(opts, G: int):
    """The options to pass for masks of G groups (a copy with mask_groups set; G must agree with it)."""
    if opts is None:
        return make_options(mask_groups=G) if G > 1 else None
    have = max(1, int(opts.mask_groups))
    if have != G:
        raise ValueError(f"masks carry {G} groups per query but the options say mask_groups={opts.mask_groups}")
    return opts


_lib = None


def lib():
    """Load libsvt.so (raises if it is not built: there is no CPU path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.svt_index_upload.argtypes = [ctypes.POINTER(svt_index_desc), vp, ctypes.POINTER(vp)]
    L.svt_index_upload_updatable.argtypes = [ctypes.POINTER(svt_index_desc), i64, i32, ctypes.c_float, vp,
                                             ctypes.POINTER(vp)]
    L.svt_index_insert.argtypes = [vp, i32, vp, vp, vp, vp, vp]
    L.svt_index_delete.argtypes = [vp, i32, vp, vp]
    L.svt_index_resign.argtypes = [vp, i32, vp, vp, vp]
    L.svt_index_free.argtypes = [vp, vp]
    L.svt_index_info.argtypes = [vp, vp, vp, vp, vp]
    L.svt_search_workspace_size.argtypes = [vp, i32, i32, i32, vp]
    L.svt_search_workspace_size.restype = sz
    L.svt_search_path.argtypes = [vp, i32, i32, i32, vp]
    L.svt_search.argtypes = [vp, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.svt_search_noalloc.argtypes = [vp, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.svt_rerank.argtypes = [vp, i32, vp, vp, i32, vp, ctypes.POINTER(svt_rerank_net), i32, vp, vp, vp, vp]
    qw = ctypes.POINTER(svt_quant_weights)
    L.svt_route.argtypes = [i32, i32, i32, i32, vp, i32, vp, vp, vp]
    L.svt_route_backward.argtypes = [i32, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp]
    L.svt_expert_sort_workspace_size.argtypes = [i32, i32, i32]
    L.svt_expert_sort.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.svt_expert_dispatch.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp]
    L.svt_expert_dispatch_backward.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp]
    L.svt_expert_combine.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp]
    L.svt_expert_combine_backward.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.svt_quant_pack_size.argtypes = [qw]
    L.svt_quant_pack.argtypes = [qw, vp, vp, vp, vp]
    L.svt_quant_linear.argtypes = [i32, i32, vp, qw, vp, vp, i32, i32, vp, vp]
    f32 = ctypes.c_float
    L.svt_embedding.argtypes = [i64, i64, i32, i32, vp, vp, f32, vp, vp]
    L.svt_embedding_backward_workspace_size.argtypes = [i64, i64, i32]
    L.svt_embedding_backward.argtypes = [i64, i64, i32, i32, vp, vp, f32, i32, i32, vp, vp, sz, vp]
    L.svt_gated_linear_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    L.svt_gated_linear.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    L.svt_gated_linear_backward_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    L.svt_gated_linear_backward.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz,
                                            vp]
    L.svt_token_logprobs_workspace_size.argtypes = [i32, i32, i32]
    L.svt_token_logprobs.argtypes = [i32, i32, i32, i32, vp, vp, f32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.svt_token_logprobs_backward.argtypes = [i32, i32, i32, vp, vp, f32, vp, vp, vp, vp, vp, vp]
    L.svt_last_error.restype = ctypes.c_char_p
    L.svt_bloom_mask.argtypes = [vp, i32, i32, i32, vp]
    L.svt_bloom_sign.argtypes = [vp, i64, i32, i32, i32, vp, i32]
    L.svt_profile_enable.argtypes = [ctypes.c_int]
    L.svt_profile_read.argtypes = [vp, vp, i32, vp, vp]
    sizes = ("svt_search_workspace_size", "svt_expert_sort_workspace_size", "svt_quant_pack_size",
             "svt_embedding_backward_workspace_size", "svt_gated_linear_workspace_size",
             "svt_gated_linear_backward_workspace_size", "svt_token_logprobs_workspace_size")
    for name in EXPORTED:
        if name in sizes:
            getattr(L, name).restype = sz
        elif name != "svt_last_error":
            getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def svt_last_error() -> str:
    return lib().svt_last_error().decode()


def _check(rc: int) -> None:
    if rc != SVT_OK:
        raise SvtError(rc, svt_last_error())


def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else ctypes.c_void_p(a.ctypes.data)


def _t_ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _opt_ptr(opts):
    return None if opts is None else ctypes.byref(opts)


def _check_tensor(name, t, dtypes, shape, device=None, nullable=False):
    """The C side cannot see dtypes, shapes or strides: a wrong tensor would be read or written out of
    bounds on the device.  Raise ValueError unless t is a contiguous tensor of one of ``dtypes`` with
    exactly ``shape``, on ``device`` (when given)."""
    if t is None:
        if nullable:
            return
        raise ValueError(f"{name}: required")
    if not hasattr(t, "data_ptr") or not hasattr(t, "dtype"):
        raise ValueError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {[str(d) for d in dtypes]}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_cuda:
        raise ValueError(f"{name}: not a device tensor")


# ------------------------------------------------------------------------------------------------
def svt_bloom_mask(token_keys: Sequence[int], n_hashes: int, sig_words: int) -> np.ndarray:
    keys = np.ascontiguousarray(np.asarray(token_keys, dtype=np.uint64))
    out = np.zeros(sig_words, np.uint64)
    _check(lib().svt_bloom_mask(_np_ptr(keys) if keys.size else None, int(keys.size), n_hashes, sig_words,
                                _np_ptr(out)))
    return out


def svt_bloom_sign(token_keys: np.ndarray, n_hashes: int, sig_words: int, n_threads: int = 0) -> np.ndarray:
    keys = np.ascontiguousarray(token_keys, dtype=np.uint64)
    n, t = keys.shape
    out = np.empty((n, sig_words), np.uint64)
    _check(lib().svt_bloom_sign(_np_ptr(keys), n, t, n_hashes, sig_words, _np_ptr(out), n_threads))
    return out


def _desc(items, sigs, list_of, centroids, item_scale):
    items = np.ascontiguousarray(items, np.int8)
    sigs = np.ascontiguousarray(sigs, np.uint64)
    list_of = np.ascontiguousarray(list_of, np.int32)
    centroids = np.ascontiguousarray(centroids, np.int8)
    d = svt_index_desc()
    d.n_items = items.shape[0]
    d.dim = items.shape[1] if items.ndim == 2 else centroids.shape[1]
    d.sig_words = sigs.shape[1] if sigs.ndim == 2 else 1
    d.nlist = centroids.shape[0]
    d.items, d.sigs, d.list_of, d.centroids = (_np_ptr(items), _np_ptr(sigs), _np_ptr(list_of), _np_ptr(centroids))
    d.item_scale = float(item_scale)
    return d, (items, sigs, list_of, centroids)   # the arrays stay alive while d is used


def svt_index_upload(items: np.ndarray, sigs: np.ndarray, list_of: np.ndarray, centroids: np.ndarray,
                     item_scale: float, stream=None) -> ctypes.c_void_p:
    """Host arrays -> device index handle (the current torch device)."""
    d, keep = _desc(items, sigs, list_of, centroids, item_scale)
    h = ctypes.c_void_p()
    _check(lib().svt_index_upload(ctypes.byref(d), _stream_ptr(stream), ctypes.byref(h)))
    return h


def svt_index_upload_updatable(items, sigs, list_of, centroids, item_scale: float, id_capacity: int,
                               slack_min: int = 0, slack_frac: float = 0.0, stream=None) -> ctypes.c_void_p:
    """Host arrays -> an index that takes in-place inserts, deletes and re-signs (free slots per cluster:
    max(slack_min, ceil(slack_frac * size)); later ids in [0, id_capacity))."""
    d, keep = _desc(items, sigs, list_of, centroids, item_scale)
    h = ctypes.c_void_p()
    _check(lib().svt_index_upload_updatable(ctypes.byref(d), int(id_capacity), int(slack_min), float(slack_frac),
                                            _stream_ptr(stream), ctypes.byref(h)))
    return h


def _ids(ids):
    return np.ascontiguousarray(ids, np.int64).reshape(-1)


def svt_index_insert(handle, ids, rows, sigs, list_of, stream=None) -> None:
    """Insert items (host arrays: ids [n], rows [n, dim] int8, sigs [n, W] uint64, list_of [n])."""
    ids = _ids(ids)
    n = ids.shape[0]
    _, dim, W, _ = svt_index_info(handle)
    rows = np.ascontiguousarray(rows, np.int8).reshape(n, dim)
    sigs = np.ascontiguousarray(sigs, np.uint64).reshape(n, W)
    list_of = np.ascontiguousarray(list_of, np.int32).reshape(n)
    _check(lib().svt_index_insert(handle, n, _np_ptr(ids), _np_ptr(rows), _np_ptr(sigs), _np_ptr(list_of),
                                  _stream_ptr(stream)))


def svt_index_delete(handle, ids, stream=None) -> None:
    ids = _ids(ids)
    _check(lib().svt_index_delete(handle, ids.shape[0], _np_ptr(ids), _stream_ptr(stream)))


def svt_index_resign(handle, ids, sigs, stream=None) -> None:
    ids = _ids(ids)
    n = ids.shape[0]
    _, _, W, _ = svt_index_info(handle)
    sigs = np.ascontiguousarray(sigs, np.uint64).reshape(n, W)
    _check(lib().svt_index_resign(handle, n, _np_ptr(ids), _np_ptr(sigs), _stream_ptr(stream)))


def svt_index_free(handle, stream=None) -> None:
    """Free an index after synchronising ``stream`` (the stream its searches ran on)."""
    _check(lib().svt_index_free(handle, _stream_ptr(stream)))


def svt_index_info(handle) -> Tuple[int, int, int, int]:
    n = ctypes.c_int64()
    d, w, nl = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().svt_index_info(handle, ctypes.byref(n), ctypes.byref(d), ctypes.byref(w), ctypes.byref(nl)))
    return n.value, d.value, w.value, nl.value


def svt_search_workspace_size(handle, n_queries: int, nprobe: int, k: int, opts=None) -> int:
    sz = lib().svt_search_workspace_size(handle, n_queries, nprobe, k, _opt_ptr(opts))
    if sz == 0:
        err = svt_last_error()
        if err:
            raise SvtError(SVT_EINVAL, err)
    return int(sz)


def svt_search_path(handle, n_queries: int, nprobe: int, k: int, opts=None) -> str:
    """The path a search of these sizes takes: "query", "tile" or "exhaustive"."""
    rc = lib().svt_search_path(handle, n_queries, nprobe, k, _opt_ptr(opts))
    if rc < 0:
        raise SvtError(rc, svt_last_error())
    return {SVT_PATH_QUERY: "query", SVT_PATH_TILE: "tile", SVT_PATH_EXHAUSTIVE: "exhaustive",
            SVT_PATH_LARGE_K: "large_k"}[rc]


def _search_tensors(handle, queries, masks, k, query_scales, out_ids, out_scores, out_fscores, out_counts,
                    out_stats):
    """Checks the search tensors and allocates the outputs not passed in; returns (B, dev, outputs)."""
    import torch
    n, dim, W, _ = svt_index_info(handle)
    if not hasattr(queries, "shape") or len(queries.shape) != 2:
        raise ValueError("queries: expected a 2-D tensor [B, dim]")
    B = int(queries.shape[0])
    dev = queries.device
    _check_tensor("queries", queries, (torch.int8,), (B, dim))
    if not hasattr(masks, "shape") or len(masks.shape) not in (2, 3):
        raise ValueError("masks: expected a tensor [B, W] or [B, G, W]")
    G = int(masks.shape[1]) if len(masks.shape) == 3 else 1
    if not 1 <= G <= SVT_MAX_MASK_GROUPS:
        raise ValueError(f"masks: {G} groups per query, at most {SVT_MAX_MASK_GROUPS}")
    _check_tensor("masks", masks, (torch.int64, torch.uint64), (B, G, W) if len(masks.shape) == 3 else (B, W), dev)
    _check_tensor("query_scales", query_scales, (torch.float32,), (B,), dev, nullable=True)
    if out_ids is None:
        out_ids = torch.empty((B, k), dtype=torch.int64, device=dev)
    if out_scores is None:
        out_scores = torch.empty((B, k), dtype=torch.int32, device=dev)
    if out_fscores is None:
        out_fscores = torch.empty((B, k), dtype=torch.float32, device=dev)
    if out_counts is None:
        out_counts = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_stats is None:
        out_stats = torch.empty((B, 2), dtype=torch.int64, device=dev)
    _check_tensor("out_ids", out_ids, (torch.int64,), (B, k), dev)
    _check_tensor("out_scores", out_scores, (torch.int32,), (B, k), dev)
    _check_tensor("out_fscores", out_fscores, (torch.float32,), (B, k), dev)
    _check_tensor("out_counts", out_counts, (torch.int32,), (B,), dev)
    _check_tensor("out_stats", out_stats, (torch.int64,), (B, 2), dev)
    return B, dev, G, (out_ids, out_scores, out_fscores, out_counts, out_stats)


def svt_search(handle, queries, masks, nprobe: int, k: int, query_scales=None, out_ids=None, out_scores=None,
               out_fscores=None, out_counts=None, out_stats=None, workspace=None, stream=None, opts=None):
    """queries: int8 [B, d] cuda tensor; masks: uint64 (or int64) [B, W] cuda tensor.
    Returns (ids int64 [B,k], scores int32 [B,k], fscores f32 [B,k], counts int32 [B], stats int64 [B,2]);
    outputs are allocated with torch unless passed in.  Asynchronous on ``stream``.  ``opts``: a
    svt_search_options (see make_options) or None."""
    import torch
    B, dev, G, outs = _search_tensors(handle, queries, masks, k, query_scales, out_ids, out_scores, out_fscores,
                                      out_counts, out_stats)
    opts = _with_groups(opts, G)
    if workspace is None:
        nbytes = svt_search_workspace_size(handle, B, nprobe, k, opts) if B > 0 else 0
        workspace = torch.empty((max(nbytes, 256),), dtype=torch.uint8, device=dev)
    _check_tensor("workspace", workspace, (torch.uint8,), (workspace.numel(),), dev)
    _check(lib().svt_search(handle, B, _t_ptr(queries), _t_ptr(masks), _t_ptr(query_scales), nprobe, k,
                            *[_t_ptr(t) for t in outs], _opt_ptr(opts), _t_ptr(workspace), int(workspace.numel()),
                            _stream_ptr(stream)))
    return outs


def svt_search_noalloc(handle, queries, masks, nprobe: int, k: int, query_scales=None, out_ids=None,
                       out_scores=None, out_fscores=None, out_counts=None, out_stats=None, stream=None, opts=None):
    """svt_search with the library's static scratch as workspace (the C call allocates no device memory;
    outputs not passed in are still allocated here, by torch).  Searches on one GPU must not overlap."""
    B, dev, G, outs = _search_tensors(handle, queries, masks, k, query_scales, out_ids, out_scores, out_fscores,
                                      out_counts, out_stats)
    opts = _with_groups(opts, G)
    _check(lib().svt_search_noalloc(handle, B, _t_ptr(queries), _t_ptr(masks), _t_ptr(query_scales), nprobe, k,
                                    *[_t_ptr(t) for t in outs], _opt_ptr(opts), _stream_ptr(stream)))
    return outs


_NET_KEYS = ("gate_w", "gate_b", "w1", "b1", "w2", "b2")


def svt_rerank(handle, queries, cand_ids, net, k_out: int, query_scales=None, out_ids=None, out_scores=None,
               out_counts=None, stream=None):
    """Re-score each query's candidates with a gated mixture of experts and keep the k_out best.
    queries: int8 [B, d] cuda tensor; cand_ids: int64 [B, n_cand] cuda tensor (e.g. svt_search's ids;
    -1 and ids not in the index are skipped); net: dict of float32 cuda tensors gate_w [E, d],
    gate_b [E], w1 [E, H, d], b1 [E, H], w2 [E, H], b2 [E].  Returns (ids int64 [B, k_out],
    scores float32 [B, k_out], counts int32 [B]); asynchronous on ``stream``."""
    import torch
    n, dim, W, _ = svt_index_info(handle)
    if not hasattr(queries, "shape") or len(queries.shape) != 2:
        raise ValueError("queries: expected a 2-D tensor [B, dim]")
    if not hasattr(cand_ids, "shape") or len(cand_ids.shape) != 2:
        raise ValueError("cand_ids: expected a 2-D tensor [B, n_cand]")
    B, n_cand = int(queries.shape[0]), int(cand_ids.shape[1])
    dev = queries.device
    _check_tensor("queries", queries, (torch.int8,), (B, dim))
    _check_tensor("cand_ids", cand_ids, (torch.int64,), (B, n_cand), dev)
    _check_tensor("query_scales", query_scales, (torch.float32,), (B,), dev, nullable=True)
    if not hasattr(net.get("w1"), "shape") or len(net["w1"].shape) != 3:
        raise ValueError("net['w1']: expected a tensor [E, H, d]")
    E, H = int(net["w1"].shape[0]), int(net["w1"].shape[1])
    shapes = {"gate_w": (E, dim), "gate_b": (E,), "w1": (E, H, dim), "b1": (E, H), "w2": (E, H), "b2": (E,)}
    for key in _NET_KEYS:
        _check_tensor(f"net['{key}']", net.get(key), (torch.float32,), shapes[key], dev)
    if out_ids is None:
        out_ids = torch.empty((B, k_out), dtype=torch.int64, device=dev)
    if out_scores is None:
        out_scores = torch.empty((B, k_out), dtype=torch.float32, device=dev)
    if out_counts is None:
        out_counts = torch.empty((B,), dtype=torch.int32, device=dev)
    _check_tensor("out_ids", out_ids, (torch.int64,), (B, k_out), dev)
    _check_tensor("out_scores", out_scores, (torch.float32,), (B, k_out), dev)
    _check_tensor("out_counts", out_counts, (torch.int32,), (B,), dev)
    cnet = svt_rerank_net(E, H, *[net[key].data_ptr() for key in _NET_KEYS])
    _check(lib().svt_rerank(handle, B, _t_ptr(queries), _t_ptr(query_scales), n_cand, _t_ptr(cand_ids),
                            ctypes.byref(cnet), k_out, _t_ptr(out_ids), _t_ptr(out_scores), _t_ptr(out_counts),
                            _stream_ptr(stream)))
    return out_ids, out_scores, out_counts


# ------------------------------------------------------------------------------------------------
# Routed experts: the calls of include/svt.h on torch tensors.  Inputs and outputs are dense tensors on one
# device; outputs not passed in are allocated on the call's stream.  Gradients are calls of their own: no call
# records history, so a tensor that requires grad is refused where torch would record it (grad mode on).
# Call under torch.no_grad(), from a torch.autograd.Function, or on detached tensors.
_TYPES = None


def _types():
    global _TYPES
    if _TYPES is None:
        import torch
        _TYPES = {torch.float32: SVT_F32, torch.float16: SVT_F16, torch.bfloat16: SVT_BF16}
    return _TYPES


_raw_stream = None


def _current_stream(dev):
    """The handle of the device's current stream, without a Stream object where torch offers that (a
    microsecond and a half of a call that takes seven)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(dev.index)


class _Run:
    """The device and stream of one call: inside, torch allocates on them; enters as the stream's handle.
    Tensors on another device than the current one, and ``stream`` (default: the device's current one),
    are made current for the call."""
    __slots__ = ("ctx", "handle")

    def __init__(self, dev, stream):
        import torch
        self.ctx = None
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream: on {stream.device}, expected {dev}")
            self.ctx = torch.cuda.stream(stream)   # also makes the stream's device current
            self.handle = stream.cuda_stream
            return
        if torch.cuda.current_device() != dev.index:
            self.ctx = torch.cuda.device(dev)
        self.handle = _current_stream(dev)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _check_history(name):
    import torch
    if torch.is_grad_enabled():
        raise ValueError(f"{name}: requires grad, but the call records no history (use torch.no_grad(), an autograd "
                         "function or detach(); gradients are the _backward calls)")


def _rows_of(name, t, dims=2):
    """(shape, element type, device) of a dense float tensor of ``dims`` dimensions on a device."""
    if not hasattr(t, "data_ptr") or t.dim() != dims:
        raise ValueError(f"{name}: expected a {dims}-D tensor")
    code = _types().get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: dtype {t.dtype} not in {[str(d) for d in _types()]}")
    if t.requires_grad:
        _check_history(name)
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: not a device tensor")
    shape = tuple(t.shape)
    if max(shape) >= 2 ** 31:
        raise ValueError(f"{name}: shape {shape} beyond 2^31 - 1")
    return shape, code, t.device


def _check_dense(name, t, dtype, shape, dev):
    """_check_tensor for one dtype, without its formatting on the way to success."""
    if getattr(t, "requires_grad", False):
        _check_history(name)
    if t is not None and getattr(t, "dtype", None) is dtype and t.shape == shape and t.is_contiguous() and \
            t.is_cuda and t.device == dev:
        return
    _check_tensor(name, t, (dtype,), shape, dev)


def _out(name, t, dtype, shape, dev, like):
    """t, checked; or a new tensor, made by ``like`` (a tensor on dev), the quickest way torch has."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _check_dense(name, t, dtype, shape, dev)
    return t


def _entries(name, t, dev=None):
    """(n_tokens, top, device) of an int32 tensor [n_tokens, top]."""
    import torch
    if not hasattr(t, "data_ptr") or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor [n_tokens, top]")
    T, K = t.shape
    _check_dense(name, t, torch.int32, (T, K), t.device if dev is None else dev)
    if T * K > 2 ** 30:
        raise ValueError(f"{name}: {T * K} entries, more than 2^30")
    return T, K, t.device


def svt_route(logits, top: int, renormalise: bool = True, out_experts=None, out_weights=None, stream=None):
    """The ``top`` best experts of each token: logits [T, E] (float32, float16, bfloat16) -> (experts int32
    [T, top], weights float32 [T, top]), by (logit desc, expert asc).  Weights are the softmax over the chosen
    experts (``renormalise``) or over all open ones; -inf and NaN shut an expert; -1 and 0 where fewer than
    ``top`` are open."""
    import torch
    (T, E), code, dev = _rows_of("logits", logits)
    if not 1 <= top <= min(SVT_MAX_TOP, E):
        raise ValueError(f"top: {top} out of [1, min({SVT_MAX_TOP}, {E} experts)]")
    with _Run(dev, stream) as s:
        out_experts = _out("out_experts", out_experts, torch.int32, (T, top), dev, logits)
        out_weights = _out("out_weights", out_weights, torch.float32, (T, top), dev, logits)
        _check(lib().svt_route(T, E, top, code, logits.data_ptr(), int(renormalise), out_experts.data_ptr(),
                               out_weights.data_ptr(), s))
    return out_experts, out_weights


def svt_route_backward(logits, experts, weights, d_weights, renormalise: bool = True, out=None, stream=None):
    """The gradient in the logits of svt_route's weights: logits [T, E], svt_route's experts and weights and
    the weights' gradient d_weights (float32 [T, top]) -> d_logits [T, E] of the logits' dtype."""
    import torch
    (T, E), code, dev = _rows_of("logits", logits)
    if not hasattr(experts, "data_ptr") or experts.dim() != 2:
        raise ValueError("experts: expected a 2-D tensor [n_tokens, top]")
    K = experts.shape[1]
    _check_dense("experts", experts, torch.int32, (T, K), dev)
    _check_dense("weights", weights, torch.float32, (T, K), dev)
    _check_dense("d_weights", d_weights, torch.float32, (T, K), dev)
    with _Run(dev, stream) as s:
        out = _out("out", out, logits.dtype, (T, E), dev, logits)
        _check(lib().svt_route_backward(T, E, K, code, logits.data_ptr(), int(renormalise), experts.data_ptr(),
                                        weights.data_ptr(), d_weights.data_ptr(), out.data_ptr(), s))
    return out


@functools.lru_cache(maxsize=256)
def svt_expert_sort_workspace_size(n_tokens: int, top: int, n_experts: int) -> int:
    """Bytes of workspace that svt_expert_sort needs for these sizes (0: none)."""
    need = lib().svt_expert_sort_workspace_size(n_tokens, top, n_experts)
    if need == 0 and svt_last_error():
        raise SvtError(SVT_EINVAL, svt_last_error())
    return int(need)


def svt_expert_sort(experts, n_experts: int, offsets=None, order=None, position=None, workspace=None, stream=None):
    """Entries grouped by expert, in their own order: experts int32 [T, top] (outside [0, n_experts): dropped)
    -> (offsets int32 [n_experts + 1], order int32 [T * top], position int32 [T, top]).  ``order`` names the
    entry of each sorted row (-1 past offsets[n_experts]), ``position`` the sorted row of each entry (-1:
    dropped)."""
    import torch
    T, K, dev = _entries("experts", experts)
    if not 1 <= n_experts <= SVT_MAX_EXPERTS:
        raise ValueError(f"n_experts: {n_experts} out of [1, {SVT_MAX_EXPERTS}]")
    need = svt_expert_sort_workspace_size(T, K, n_experts)
    with _Run(dev, stream) as s:
        offsets = _out("offsets", offsets, torch.int32, (n_experts + 1,), dev, experts)
        order = _out("order", order, torch.int32, (T * K,), dev, experts)
        position = _out("position", position, torch.int32, (T, K), dev, experts)
        if workspace is not None:
            _check_tensor("workspace", workspace, (torch.uint8,), (workspace.numel(),), dev)
        elif need:
            workspace = experts.new_empty((need,), dtype=torch.uint8)
        _check(lib().svt_expert_sort(T, K, n_experts, experts.data_ptr(), offsets.data_ptr(), order.data_ptr(),
                                 position.data_ptr(), None if workspace is None else workspace.data_ptr(),
                                 0 if workspace is None else workspace.numel(), s))
    return offsets, order, position


def svt_expert_dispatch(x, position, out=None, stream=None):
    """Each token's row to its sorted rows: x [T, D], position int32 [T, top] -> rows [T * top, D].  Rows that
    no entry names (behind the last one) are left as they were."""
    (T, D), code, dev = _rows_of("x", x)
    n, K, _ = _entries("position", position, dev)
    if n != T:
        raise ValueError(f"position: shape {tuple(position.shape)} for {T} tokens")
    with _Run(dev, stream) as s:
        out = _out("out", out, x.dtype, (T * K, D), dev, x)
        _check(lib().svt_expert_dispatch(T, K, D, code, x.data_ptr(), position.data_ptr(), out.data_ptr(), s))
    return out


def _gather_sum(fn, name, rows, position, weights, out, stream):
    import torch
    (R, D), code, dev = _rows_of(name, rows)
    T, K, _ = _entries("position", position, dev)
    if R != T * K:
        raise ValueError(f"{name}: {R} rows for {T} tokens of {K} entries")
    args = ()
    if fn == "svt_expert_combine":
        if weights is not None:
            _check_dense("weights", weights, torch.float32, (T, K), dev)
        args = (None if weights is None else weights.data_ptr(),)
    with _Run(dev, stream) as s:
        out = _out("out", out, rows.dtype, (T, D), dev, rows)
        _check(getattr(lib(), fn)(T, K, D, code, rows.data_ptr(), position.data_ptr(), *args, out.data_ptr(), s))
    return out


def svt_expert_dispatch_backward(d_rows, position, out=None, stream=None):
    """The gradient of svt_expert_dispatch: d_rows [T * top, D], position [T, top] -> dx [T, D], the sum of a
    token's rows."""
    return _gather_sum("svt_expert_dispatch_backward", "d_rows", d_rows, position, None, out, stream)


def svt_expert_combine(rows, position, weights=None, out=None, stream=None):
    """The experts' rows back to their tokens: rows [T * top, D], position int32 [T, top], weights float32 [T,
    top] (None: ones) -> y [T, D], the weighted sum of a token's rows."""
    return _gather_sum("svt_expert_combine", "rows", rows, position, weights, out, stream)


def svt_expert_combine_backward(dy, rows, position, weights, out_rows=None, out_weights=None, stream=None):
    """The gradients of svt_expert_combine: dy [T, D], its rows [T * top, D], position and weights -> (d_rows
    [T * top, D], d_weights float32 [T, top]).  Rows that no entry names are left as they were."""
    import torch
    (T, D), code, dev = _rows_of("dy", dy)
    n, K, _ = _entries("position", position, dev)
    if n != T:
        raise ValueError(f"position: shape {tuple(position.shape)} for {T} tokens")
    _check_dense("rows", rows, dy.dtype, (T * K, D), dev)
    _check_dense("weights", weights, torch.float32, (T, K), dev)
    with _Run(dev, stream) as s:
        out_rows = _out("out_rows", out_rows, dy.dtype, (T * K, D), dev, dy)
        out_weights = _out("out_weights", out_weights, torch.float32, (T, K), dev, dy)
        _check(lib().svt_expert_combine_backward(T, K, D, code, dy.data_ptr(), rows.data_ptr(), position.data_ptr(),
                                                 weights.data_ptr(), out_rows.data_ptr(), out_weights.data_ptr(), s))
    return out_rows, out_weights


def svt_quant_pack(nibbles, scales, zeros, n_in: int, group: int, packed=None, stream=None) -> svt_quant_weights:
    """Weights W[n, k] = scales[n, k // group] * (q[n, k] - zeros[n, k // group]) in the layout svt_quant_linear
    reads.  nibbles uint8 [M, N, (n_in + 1) // 2] (or [N, ..] for one matrix): q of input 2 i in the low half of
    byte i; scales [M, N, ceil(n_in / group)] float32, float16 or bfloat16; zeros uint8 of the same shape, or
    None (every zero point 8).  group: 32, 64 or 128."""
    import torch
    if hasattr(nibbles, "dim") and nibbles.dim() == 2:
        nibbles = nibbles[None]
        scales = scales[None] if hasattr(scales, "dim") else scales
        zeros = zeros[None] if hasattr(zeros, "dim") else zeros
    (M, N, _), code, dev = _rows_of("scales", scales, 3)
    groups = -(-int(n_in) // int(group)) if group > 0 else 0
    _check_tensor("nibbles", nibbles, (torch.uint8,), (M, N, (n_in + 1) // 2), dev)
    _check_tensor("scales", scales, (scales.dtype,), (M, N, groups), dev)
    _check_tensor("zeros", zeros, (torch.uint8,), (M, N, groups), dev, nullable=True)
    w = svt_quant_weights(M, N, n_in, group, code, int(zeros is not None), None, 0)
    need = lib().svt_quant_pack_size(ctypes.byref(w))
    if need == 0:
        raise SvtError(SVT_EUNSUPPORTED if group not in (32, 64, 128) else SVT_EINVAL, svt_last_error())
    with _Run(dev, stream) as s:
        packed = _out("packed", packed, torch.uint8, (need,), dev, nibbles)
        w.packed, w.packed_bytes, w.buffer = packed.data_ptr(), need, packed
        _check(lib().svt_quant_pack(ctypes.byref(w), nibbles.data_ptr(), scales.data_ptr(),
                                    None if zeros is None else zeros.data_ptr(), s))
    return w


_ACTIVATIONS = {"none": SVT_ACT_NONE, "relu": SVT_ACT_RELU}


def svt_quant_linear(x, weights: svt_quant_weights, offsets=None, bias=None, activation: str = "none", out=None,
                     out_dtype=None, stream=None):
    """y = act(x W^T + bias) with svt_quant_pack's weights: x [R, n_in] -> y [R, n_out] of ``out_dtype`` (x's
    dtype, the default, or float32).  Without ``offsets`` the one matrix serves every row; with offsets int32
    [M + 1] (svt_expert_sort's) matrix e serves rows offsets[e] .. offsets[e + 1] - 1 and rows past the last
    stay as they were.  bias: float32 [M, n_out], or None."""
    import torch
    (R, K), code, dev = _rows_of("x", x)
    M, N = weights.n_matrices, weights.n_out
    if K != weights.n_in:
        raise ValueError(f"x: shape {tuple(x.shape)} for weights of {weights.n_in} inputs")
    if weights.buffer is None or weights.buffer.device != dev:
        raise ValueError(f"weights: not packed on {dev}")
    if offsets is not None:
        _check_dense("offsets", offsets, torch.int32, (M + 1,), dev)
    if bias is not None:
        if M == 1 and bias.dim() == 1:
            bias = bias[None]
        _check_dense("bias", bias, torch.float32, (M, N), dev)
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation: {activation!r} not in {sorted(_ACTIVATIONS)}")
    out_dtype = out.dtype if out is not None else x.dtype if out_dtype is None else out_dtype
    if out_dtype not in _types():
        raise ValueError(f"out: dtype {out_dtype} not in {[str(d) for d in _types()]}")
    with _Run(dev, stream) as s:
        out = _out("out", out, out_dtype, (R, N), dev, x)
        _check(lib().svt_quant_linear(R, code, x.data_ptr(), ctypes.byref(weights),
                                      None if offsets is None else offsets.data_ptr(),
                                      None if bias is None else bias.data_ptr(), _ACTIVATIONS[activation],
                                      _types()[out_dtype], out.data_ptr(), s))
    return out


# ------------------------------------------------------------------------------------------------
# A scorer in training: rows of a table for tokens, gated products, log probabilities, and their gradients.  As the
# calls above: dense tensors on one device, no history recorded.

def _token_ids(name, t, dev):
    """(number, device) of an int64 tensor of tokens."""
    import torch
    if not hasattr(t, "data_ptr"):
        raise ValueError(f"{name}: expected a tensor")
    _check_dense(name, t, torch.int64, t.shape, dev)
    return t.numel()


def _workspace(given, need, dev, like):
    """(tensor or None, pointer, bytes) of a workspace: the one given, checked, or a new one of ``need`` bytes."""
    import torch
    if given is not None:
        _check_tensor("workspace", given, (torch.uint8,), (given.numel(),), dev)
    elif need:
        given = like.new_empty((need,), dtype=torch.uint8)
    return (None, None, 0) if given is None else (given, given.data_ptr(), given.numel())


def svt_embedding(table, ids, scale: float = 1.0, out=None, stream=None):
    """Rows of a table for tokens: table [V, D] (float32, float16, bfloat16), ids int64 of any shape -> scale *
    table[ids], [*ids.shape, D] of the table's dtype; a token outside [0, V) gets a row of zeros."""
    (V, D), code, dev = _rows_of("table", table)
    n = _token_ids("ids", ids, dev)
    with _Run(dev, stream) as s:
        out = _out("out", out, table.dtype, (*ids.shape, D), dev, table)
        _check(lib().svt_embedding(n, V, D, code, table.data_ptr(), ids.data_ptr(), scale, out.data_ptr(), s))
    return out


@functools.lru_cache(maxsize=256)
def svt_embedding_backward_workspace_size(n_tokens: int, n_rows: int, width: int) -> int:
    """Bytes of workspace that svt_embedding_backward needs for these sizes."""
    need = lib().svt_embedding_backward_workspace_size(n_tokens, n_rows, width)
    if need == 0 and svt_last_error():
        raise SvtError(SVT_EINVAL, svt_last_error())
    return int(need)


def svt_embedding_backward(d_out, ids, n_rows: int, scale: float = 1.0, out=None, accumulate: bool = False,
                           out_dtype=None, workspace=None, stream=None):
    """The gradient in a table of ``n_rows`` rows: d_out [*ids.shape, D], ids int64 -> d_table [n_rows, D] of
    ``out_dtype`` (d_out's, the default, or float32): row v is scale times the sum of the rows of d_out whose token is
    v.  ``accumulate`` adds them to ``out`` (which has to be given) and touches no other row."""
    import torch
    if not hasattr(d_out, "dim") or d_out.dim() < 1:
        raise ValueError("d_out: expected a tensor [*ids.shape, D]")
    shape, code, dev = _rows_of("d_out", d_out, d_out.dim())
    D = shape[-1]
    n = _token_ids("ids", ids, dev)
    if d_out.shape[:-1] != ids.shape:
        raise ValueError(f"ids: shape {tuple(ids.shape)} for d_out of shape {tuple(d_out.shape)}")
    if accumulate and out is None:
        raise ValueError("out: to be given where the gradient is added to it")
    if out is not None and out_dtype is not None and out_dtype is not out.dtype:
        raise ValueError(f"out: dtype {out.dtype}, expected {out_dtype}")
    out_dtype = out.dtype if out is not None else d_out.dtype if out_dtype is None else out_dtype
    if out_dtype is not d_out.dtype and out_dtype is not torch.float32:
        raise ValueError(f"out: dtype {out_dtype} is neither {d_out.dtype} nor torch.float32")
    need = svt_embedding_backward_workspace_size(n, n_rows, D)
    with _Run(dev, stream) as s:
        out = _out("out", out, out_dtype, (n_rows, D), dev, d_out)
        workspace, at, size = _workspace(workspace, need, dev, d_out)
        _check(lib().svt_embedding_backward(n, n_rows, D, code, d_out.data_ptr(), ids.data_ptr(), scale, int(accumulate),
                                            _types()[out_dtype], out.data_ptr(), at, size, s))
    return out


_GATES = {"none": SVT_ACT_NONE, "relu": SVT_ACT_RELU, "silu": SVT_ACT_SILU, "gelu": SVT_ACT_GELU}


def _gated_shape(x, w_gate, w_up, offsets, activation):
    """(rows, inputs, outputs, matrices, element type, device, activation's code) of a gated product."""
    import torch
    (R, K), code, dev = _rows_of("x", x)
    if not hasattr(w_gate, "dim") or w_gate.dim() != (2 if offsets is None else 3):
        raise ValueError("w_gate: expected a tensor " + ("[N, K]" if offsets is None else "[M, N, K]"))
    M, N = 1 if offsets is None else w_gate.shape[0], w_gate.shape[-2]
    shape = (N, K) if offsets is None else (M, N, K)
    _check_dense("w_gate", w_gate, x.dtype, shape, dev)
    _check_dense("w_up", w_up, x.dtype, shape, dev)
    if offsets is not None:
        _check_dense("offsets", offsets, torch.int32, (M + 1,), dev)
    if activation not in _GATES:
        raise ValueError(f"activation: {activation!r} not in {sorted(_GATES)}")
    return R, K, N, M, code, dev, _GATES[activation]


@functools.lru_cache(maxsize=256)
def svt_gated_linear_workspace_size(n_rows: int, n_in: int, n_out: int, n_matrices: int, dtype: int, by_expert: bool,
                                    aligned: bool) -> int:
    """Bytes of workspace that svt_gated_linear needs (0: none); dtype: SVT_F32, SVT_F16 or SVT_BF16, aligned: whether x and
    the weights are 4-byte aligned."""
    need = lib().svt_gated_linear_workspace_size(n_rows, n_in, n_out, n_matrices, dtype, int(by_expert), int(aligned))
    if need == 0 and svt_last_error():
        raise SvtError(SVT_EINVAL, svt_last_error())
    return int(need)


def svt_gated_linear(x, w_gate, w_up, offsets=None, activation: str = "silu", keep: bool = False, out=None, out_gate=None,
                     out_up=None, workspace=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T): x [R, K] (float32, float16, bfloat16), w_gate and w_up [N, K] of its dtype -> h
    [R, N].  With ``offsets`` int32 [M + 1] (svt_expert_sort's) the weights are [M, N, K], pair e serves rows offsets[e]
    .. offsets[e + 1] - 1, and rows past the last stay as they were.  activation: "silu", "gelu", "relu" or "none".
    ``keep`` also returns what the gradient needs: (h, gate, up)."""
    R, K, N, M, code, dev, act = _gated_shape(x, w_gate, w_up, offsets, activation)
    at_x, at_g, at_u = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    need = svt_gated_linear_workspace_size(R, K, N, M, code, offsets is not None, (at_x | at_g | at_u) % 4 == 0)
    with _Run(dev, stream) as s:
        out = _out("out", out, x.dtype, (R, N), dev, x)
        if keep:
            out_gate = _out("out_gate", out_gate, x.dtype, (R, N), dev, x)
            out_up = _out("out_up", out_up, x.dtype, (R, N), dev, x)
        workspace, at, size = _workspace(workspace, need, dev, x)
        _check(lib().svt_gated_linear(R, K, N, M, code, at_x, at_g, at_u, None if offsets is None else offsets.data_ptr(),
                                      act, out.data_ptr(), out_gate.data_ptr() if keep else None,
                                      out_up.data_ptr() if keep else None, at, size, s))
    return (out, out_gate, out_up) if keep else out


@functools.lru_cache(maxsize=256)
def svt_gated_linear_backward_workspace_size(n_rows: int, n_in: int, n_out: int, n_matrices: int, dtype: int,
                                             by_expert: bool, aligned: bool) -> int:
    """Bytes of workspace that svt_gated_linear_backward needs; arguments as svt_gated_linear_workspace_size."""
    need = lib().svt_gated_linear_backward_workspace_size(n_rows, n_in, n_out, n_matrices, dtype, int(by_expert),
                                                          int(aligned))
    if need == 0 and svt_last_error():
        raise SvtError(SVT_EINVAL, svt_last_error())
    return int(need)


def svt_gated_linear_backward(dh, x, w_gate, w_up, gate, up, offsets=None, activation: str = "silu", out_x=None,
                              out_gate=None, out_up=None, need_x: bool = True, need_weights: bool = True, workspace=None,
                              stream=None):
    """The gradients of svt_gated_linear: dh [R, N], its inputs and what it kept -> (dx [R, K], d_gate and d_up like
    w_gate and w_up).  The gradients of gate and up are rounded to x's dtype before the products.  ``need_x`` and
    ``need_weights`` leave one part out (None in its place).  Rows that no pair of matrices names stay as they were in dx;
    a pair without rows gets zeros."""
    R, K, N, M, code, dev, act = _gated_shape(x, w_gate, w_up, offsets, activation)
    for name, t in (("dh", dh), ("gate", gate), ("up", up)):
        _check_dense(name, t, x.dtype, (R, N), dev)
    at_x, at_g, at_u = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    need = svt_gated_linear_backward_workspace_size(R, K, N, M, code, offsets is not None, (at_x | at_g | at_u) % 4 == 0)
    with _Run(dev, stream) as s:
        out_x = _out("out_x", out_x, x.dtype, (R, K), dev, x) if need_x else None
        out_gate = _out("out_gate", out_gate, x.dtype, w_gate.shape, dev, x) if need_weights else None
        out_up = _out("out_up", out_up, x.dtype, w_gate.shape, dev, x) if need_weights else None
        workspace, at, size = _workspace(workspace, need, dev, x)
        _check(lib().svt_gated_linear_backward(R, K, N, M, code, dh.data_ptr(), at_x, at_g, at_u, gate.data_ptr(),
                                               up.data_ptr(), None if offsets is None else offsets.data_ptr(), act,
                                               *[None if t is None else t.data_ptr() for t in (out_x, out_gate, out_up)],
                                               at, size, s))
    return out_x, out_gate, out_up


@functools.lru_cache(maxsize=256)
def svt_token_logprobs_workspace_size(n_tokens: int, vocab: int, top: int) -> int:
    """Bytes of workspace that svt_token_logprobs needs for these sizes (0: none)."""
    need = lib().svt_token_logprobs_workspace_size(n_tokens, vocab, top)
    if need == 0 and svt_last_error():
        raise SvtError(SVT_EINVAL, svt_last_error())
    return int(need)


def svt_token_logprobs(logits, tokens, top: int = 0, scale: float = 1.0, out_logprobs=None, out_entropy=None,
                       out_norms=None, out_top_tokens=None, out_top_logprobs=None, workspace=None, stream=None):
    """Of p = softmax(scale * logits) for each row: logits [T, V] (float32, float16, bfloat16), tokens int64 [T] ->
    (logprobs float32 [T], entropy float32 [T], norms float32 [T, 2]), and with ``top`` > 0 also (top_tokens int64
    [T, top], top_logprobs float32 [T, top]), by (logit desc, token asc).  -inf and NaN shut a token.  logprobs is 0
    where the token lies outside [0, V); -1 and -inf where fewer than ``top`` are open.  norms is for the gradient; scale lies
    in (0, 2^127]."""
    import torch
    (T, V), code, dev = _rows_of("logits", logits)
    _check_dense("tokens", tokens, torch.int64, (T,), dev)
    if not 0 <= top <= min(SVT_MAX_TOP, V):
        raise ValueError(f"top: {top} out of [0, min({SVT_MAX_TOP}, {V} tokens)]")
    need = svt_token_logprobs_workspace_size(T, V, top)
    with _Run(dev, stream) as s:
        out_logprobs = _out("out_logprobs", out_logprobs, torch.float32, (T,), dev, logits)
        out_entropy = _out("out_entropy", out_entropy, torch.float32, (T,), dev, logits)
        out_norms = _out("out_norms", out_norms, torch.float32, (T, 2), dev, logits)
        best = ()
        if top:
            best = (_out("out_top_tokens", out_top_tokens, torch.int64, (T, top), dev, logits),
                    _out("out_top_logprobs", out_top_logprobs, torch.float32, (T, top), dev, logits))
        workspace, at, size = _workspace(workspace, need, dev, logits)
        _check(lib().svt_token_logprobs(T, V, top, code, logits.data_ptr(), tokens.data_ptr(), scale,
                                        out_logprobs.data_ptr(), out_entropy.data_ptr(), out_norms.data_ptr(),
                                        *([t.data_ptr() for t in best] or (None, None)), at, size, s))
    return (out_logprobs, out_entropy, out_norms, *best)


def svt_token_logprobs_backward(logits, tokens, norms, entropy, d_logprobs, d_entropy=None, scale: float = 1.0, out=None,
                                stream=None):
    """The gradient in the logits of svt_token_logprobs's log probabilities and entropy: its inputs, its norms and
    entropy, the gradients d_logprobs and d_entropy (float32 [T]; None: zeros) -> d_logits [T, V] of the logits'
    dtype."""
    import torch
    (T, V), code, dev = _rows_of("logits", logits)
    _check_dense("tokens", tokens, torch.int64, (T,), dev)
    _check_dense("norms", norms, torch.float32, (T, 2), dev)
    _check_dense("entropy", entropy, torch.float32, (T,), dev)
    _check_dense("d_logprobs", d_logprobs, torch.float32, (T,), dev)
    if d_entropy is not None:
        _check_dense("d_entropy", d_entropy, torch.float32, (T,), dev)
    with _Run(dev, stream) as s:
        out = _out("out", out, logits.dtype, (T, V), dev, logits)
        _check(lib().svt_token_logprobs_backward(T, V, code, logits.data_ptr(), tokens.data_ptr(), scale, norms.data_ptr(),
                                                 entropy.data_ptr(), d_logprobs.data_ptr(),
                                                 None if d_entropy is None else d_entropy.data_ptr(), out.data_ptr(), s))
    return out


def svt_profile_enable(on) -> None:
    """False/0: off; True/1: every stage; 2: the scan stage only (two event records per search)."""
    _check(lib().svt_profile_enable(int(on)))


def svt_profile_read(max_stages: int = 8):
    """Returns ({stage: total ms}, n_searches) over the searches recorded since the last read."""
    ms = (ctypes.c_float * max_stages)()
    names = (ctypes.c_char_p * max_stages)()
    n, ns = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().svt_profile_read(ms, names, max_stages, ctypes.byref(n), ctypes.byref(ns)))
    return {names[i].decode(): float(ms[i]) for i in range(min(n.value, max_stages))}, ns.value


# ------------------------------------------------------------------------------------------------
class Index:
    """Convenience owner of an uploaded index: ``Index(items, sigs, list_of, centroids, scale)``,
    ``search(queries, masks, nprobe, k)`` with torch device tensors, ``close()``."""

    def __init__(self, items, sigs, list_of, centroids, item_scale, stream=None, id_capacity=None, slack_min=0,
                 slack_frac=0.0):
        if id_capacity is None:
            self.handle = svt_index_upload(items, sigs, list_of, centroids, item_scale, stream)
        else:   # updatable
            self.handle = svt_index_upload_updatable(items, sigs, list_of, centroids, item_scale, id_capacity,
                                                     slack_min, slack_frac, stream)
        self.n_items, self.dim, self.sig_words, self.nlist = svt_index_info(self.handle)
        self._ws = None

    def workspace(self, n_queries: int, nprobe: int, k: int, opts=None):
        import torch
        nbytes = max(256, svt_search_workspace_size(self.handle, n_queries, nprobe, k, opts))
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = None
            self._ws = torch.empty((nbytes,), dtype=torch.uint8, device="cuda")
        return self._ws

    def search(self, queries, masks, nprobe: int, k: int, query_scales=None, stream=None, opts=None, **outs):
        B = int(queries.shape[0])
        if hasattr(masks, "shape") and len(masks.shape) == 3:
            opts = _with_groups(opts, int(masks.shape[1]))
        ws = self.workspace(B, nprobe, k, opts) if B > 0 else None
        return svt_search(self.handle, queries, masks, nprobe, k, query_scales=query_scales, workspace=ws,
                          stream=stream, opts=opts, **outs)

    def rerank(self, queries, cand_ids, net, k_out: int, query_scales=None, stream=None, **outs):
        return svt_rerank(self.handle, queries, cand_ids, net, k_out, query_scales=query_scales, stream=stream,
                          **outs)

    def insert(self, ids, rows, sigs, list_of, stream=None):
        svt_index_insert(self.handle, ids, rows, sigs, list_of, stream)
        self.n_items = svt_index_info(self.handle)[0]

    def delete(self, ids, stream=None):
        svt_index_delete(self.handle, ids, stream)
        self.n_items = svt_index_info(self.handle)[0]

    def resign(self, ids, sigs, stream=None):
        svt_index_resign(self.handle, ids, sigs, stream)

    def close(self, stream=None):
        if self.handle is not None:
            svt_index_free(self.handle, stream)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

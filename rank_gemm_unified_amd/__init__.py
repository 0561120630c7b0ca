"""Python binding of liblorapool: the unmerged multi-LoRA projection over a unified page pool.

The functions below carry the C-ABI's names and only marshal arguments (torch tensors become their
device addresses, streams their hipStream_t handles); every step of the projection runs in the
library's HIP kernels.  Importing this package fails loudly when the library has not been built or
was built from sources other than the ones beside it.

``Pool`` is a convenience owner of the device buffers a pool needs (pages and page table),
allocated with torch; torch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblorapool.so")

LORA_OK, LORA_EINVAL, LORA_ENOMEM, LORA_ENOENT = 0, -1, -2, -3
LORA_ERANK, LORA_EBUSY, LORA_EEXIST, LORA_EHIP, LORA_EDEVICE = -4, -5, -6, -7, -8
LORA_F32, LORA_BF16 = 0, 1
LORA_MAX_RANK, LORA_MAX_ADAPTERS, LORA_MAX_TOKENS = 64, 8192, 1 << 22
LORA_VICTIM_LOAD_ORDER, LORA_VICTIM_LRU, LORA_VICTIM_FARTHEST = 0, 1, 2
LORA_MAX_CALL_SLOTS = 4
LORA_NOALLOC_SCRATCH_MB = 32
LORA_MAX_SEQS, LORA_MAX_KV_TOKENS, LORA_MAX_TOKENS_PER_PAGE, LORA_MAX_HEADS = 65535, 1 << 22, 256, 1024
STATUS_NAMES = {0: "ok", -1: "einval", -2: "enomem", -3: "enoent", -4: "erank", -5: "ebusy",
                -6: "eexist", -7: "ehip", -8: "edevice"}

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it first (python rank_gemm_unified_amd/build.py "
                      "or __graft_entry__.build()); there is no fallback path")
# torch ships its own HIP runtime under the same soname as /opt/rocm's.  Whichever is loaded first
# serves the whole process, and a process that loads this library before torch ends up with two
# halves of different runtimes that see no device.  Load torch's first.
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_P64 = ctypes.POINTER(ctypes.c_int64)
_P32 = ctypes.POINTER(ctypes.c_int32)


class lora_pool_stats_t(ctypes.Structure):
    _fields_ = [("num_pages", _i64), ("free_pages", _i64), ("kv_pages", _i64), ("adapter_pages", _i64),
                ("resident_adapters", _i32), ("idle_adapters", _i32), ("kv_requests", _i64),
                ("loads", _i64), ("evictions", _i64), ("bytes_loaded", _i64)]


class lora_profile_t(ctypes.Structure):
    _fields_ = [("calls", _i64), ("ms_group", ctypes.c_double), ("ms_first", ctypes.c_double),
                ("ms_second", ctypes.c_double)]


class lora_kv_layout_t(ctypes.Structure):
    """How heads lie in a page: lora_kv_layout_t(n_heads, n_kv_heads, head_dim, tokens_per_page)."""
    _fields_ = [("n_heads", _i32), ("n_kv_heads", _i32), ("head_dim", _i32), ("tokens_per_page", _i32)]


_f32 = ctypes.c_float
_SIGS = {
    "lora_pool_create": (ctypes.c_int, [_vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp, ctypes.POINTER(_vp)]),
    "lora_pool_free": (ctypes.c_int, [_vp]),
    "lora_pool_load_adapter": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _vp]),
    "lora_pool_release_adapter": (ctypes.c_int, [_vp, _i32]),
    "lora_pool_set_victim_rule": (ctypes.c_int, [_vp, _i32]),
    "lora_pool_set_lookahead": (ctypes.c_int, [_vp, _vp, _i64]),
    "lora_pool_evict_adapter": (ctypes.c_int, [_vp, _i32, _vp]),
    "lora_pool_grow_kv": (ctypes.c_int, [_vp, _i64, _i32, _vp]),
    "lora_pool_free_kv": (ctypes.c_int, [_vp, _i64]),
    "lora_pool_pages_for": (_i64, [_i32, _i32, _i32]),
    "lora_kv_pages_per_token": (_i64, [_i32]),
    "lora_pool_stats": (ctypes.c_int, [_vp, ctypes.POINTER(lora_pool_stats_t)]),
    "lora_pool_page_table": (ctypes.c_int, [_vp, _i32, ctypes.POINTER(_vp), _P32]),
    "lora_pool_adapter_pages": (ctypes.c_int, [_vp, _i32, _vp, _i64, _P64, _P32, _P32]),
    "lora_pool_kv_pages": (ctypes.c_int, [_vp, _i64, _vp, _i64, _P64]),
    "lora_pool_free_list": (ctypes.c_int, [_vp, _vp, _i64, _P64]),
    "lora_pool_resident": (ctypes.c_int, [_vp, _vp, _i32, _P32]),
    "lora_project_workspace_size": (_sz, [_vp, _i64]),
    "lora_project_slots_workspace_size": (_sz, [_vp, _i32, _i64]),
    "lora_project_slots": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "lora_project_slots_x": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "lora_project": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "lora_debug_gather": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "lora_debug_project": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp, _vp, _vp]),
    "lora_project_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "lora_kv_write": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _vp, _i32, _i64, _vp]),
    "lora_kv_attend_workspace_size": (_sz, [_vp, _vp, _i32, _i64, _i32]),
    "lora_kv_attend": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _i32, _vp, _i32, _i64, _f32, _vp, _i64, _vp, _vp,
                                      _vp, _sz, _vp]),
    "lora_kv_attend_chunk_workspace_size": (_sz, [_vp, _vp, _i32, _i64, _i64, _i32]),
    "lora_kv_attend_chunk": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _i32, _vp, _vp, _i32, _i64, _i64, _f32, _vp,
                                            _i64, _vp, _vp, _vp, _sz, _vp]),
    "lora_kv_evict": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp,
                                     _i32, _vp, _vp]),
    "lora_pool_drop_kv": (ctypes.c_int, [_vp, _i64, _vp, _i64]),
    "lora_check_device_errors": (ctypes.c_int, [_vp]),
    "lora_profile_start": (ctypes.c_int, [_vp, _i32]),
    "lora_profile_stop": (ctypes.c_int, [_vp, ctypes.POINTER(lora_profile_t)]),
    "lora_last_error": (ctypes.c_char_p, []),
    "lora_version": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGS.items():
    try:
        _f = getattr(_lib, _name)
    except AttributeError as _e:
        raise ImportError(f"{LIB_PATH} lacks {_name}: it is stale, rebuild it "
                          "(python rank_gemm_unified_amd/build.py)") from _e
    _f.restype, _f.argtypes = _res, _args

EXPORTED = tuple(_SIGS)

# The library carries the hash of the sources it was built from; refuse one built from other sources
# (a stale build whose exports happen to match would otherwise load silently).
from ._srchash import source_hash as _source_hash  # noqa: E402

SOURCE_HASH = _source_hash()
_built = _lib.lora_version().decode()
if SOURCE_HASH is not None and not _built.endswith(" src " + SOURCE_HASH):
    raise ImportError(f"{LIB_PATH} ({_built}) was not built from the sources beside it (hash {SOURCE_HASH}): "
                      "it is stale, rebuild it (python rank_gemm_unified_amd/build.py)")


class LoraError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        self.status = STATUS_NAMES.get(code, str(code))
        msg = _lib.lora_last_error().decode(errors="replace")
        super().__init__(f"{where}: {self.status} ({code}): {msg}")


def _check(rc: int, where: str) -> int:
    if rc != LORA_OK:
        raise LoraError(rc, where)
    return rc


def _ptr(t) -> int | None:
    """Device/host address of a tensor or array (None stays NULL)."""
    if t is None or type(t) is int:
        return t
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(s, int):
        return s
    return s.cuda_stream


# The current stream's handle of a device.  torch's own short way to it where there is one: a stream object costs
# two microseconds, as much as the rest of a call's checks.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda device: torch.cuda.current_stream(device).cuda_stream)


# ---- C-ABI, one wrapper per entry point ----------------------------------------------------------

def lora_pool_create(pages, num_pages, hidden, dtype, max_rank, n_slots, max_adapters, page_table,
                     free_order=None):
    fo = None
    if free_order is not None:
        fo = np.ascontiguousarray(free_order, dtype=np.int64)
    out = _vp()
    _check(_lib.lora_pool_create(_ptr(pages), num_pages, hidden, dtype, max_rank, n_slots, max_adapters,
                                 _ptr(page_table), None if fo is None else fo.ctypes.data, ctypes.byref(out)),
           "lora_pool_create")
    return out.value


def lora_pool_free(pool):
    return _check(_lib.lora_pool_free(pool), "lora_pool_free")


def lora_pool_load_adapter(pool, adapter_id, rank, A_t, B, stream=None, check=True):
    rc = _lib.lora_pool_load_adapter(pool, adapter_id, rank, _ptr(A_t), _ptr(B), _stream(stream))
    return _check(rc, "lora_pool_load_adapter") if check else rc


def lora_pool_set_victim_rule(pool, rule, check=True):
    rc = _lib.lora_pool_set_victim_rule(pool, rule)
    return _check(rc, "lora_pool_set_victim_rule") if check else rc


def lora_pool_set_lookahead(pool, adapter_ids, check=True):
    ids = np.ascontiguousarray(adapter_ids, dtype=np.int32)
    rc = _lib.lora_pool_set_lookahead(pool, ids.ctypes.data if ids.size else None, ids.size)
    return _check(rc, "lora_pool_set_lookahead") if check else rc


def lora_pool_release_adapter(pool, adapter_id, check=True):
    rc = _lib.lora_pool_release_adapter(pool, adapter_id)
    return _check(rc, "lora_pool_release_adapter") if check else rc


def lora_pool_evict_adapter(pool, adapter_id, stream=None, check=True):
    rc = _lib.lora_pool_evict_adapter(pool, adapter_id, _stream(stream))
    return _check(rc, "lora_pool_evict_adapter") if check else rc


def lora_pool_grow_kv(pool, request_id, layers, check=True):
    """Returns the new KV page ids (list), or the status code when check=False and it failed."""
    out = np.zeros(max(2 * layers, 1), np.int64)
    rc = _lib.lora_pool_grow_kv(pool, request_id, layers, out.ctypes.data)
    if rc != LORA_OK:
        return _check(rc, "lora_pool_grow_kv") if check else rc
    return out[: 2 * layers].tolist()


def lora_pool_free_kv(pool, request_id, check=True):
    rc = _lib.lora_pool_free_kv(pool, request_id)
    return _check(rc, "lora_pool_free_kv") if check else rc


def lora_pool_drop_kv(pool, request_id, page_ids, check=True):
    ids = np.ascontiguousarray(page_ids, dtype=np.int64)
    rc = _lib.lora_pool_drop_kv(pool, request_id, ids.ctypes.data if ids.size else None, ids.size)
    return _check(rc, "lora_pool_drop_kv") if check else rc


def lora_pool_pages_for(rank, projections, layers):
    return _lib.lora_pool_pages_for(rank, projections, layers)


def lora_kv_pages_per_token(layers):
    return _lib.lora_kv_pages_per_token(layers)


def lora_pool_stats(pool) -> dict:
    st = lora_pool_stats_t()
    _check(_lib.lora_pool_stats(pool, ctypes.byref(st)), "lora_pool_stats")
    return {name: getattr(st, name) for name, _ in st._fields_}


def lora_pool_page_table(pool, slot):
    ptr, stride = _vp(), _i32()
    _check(_lib.lora_pool_page_table(pool, slot, ctypes.byref(ptr), ctypes.byref(stride)), "lora_pool_page_table")
    return ptr.value, stride.value


def lora_pool_adapter_pages(pool, adapter_id):
    n, rank, users = _i64(), _i32(), _i32()
    rc = _lib.lora_pool_adapter_pages(pool, adapter_id, None, 0, ctypes.byref(n), ctypes.byref(rank),
                                      ctypes.byref(users))
    if rc == LORA_ENOENT:
        raise LoraError(rc, "lora_pool_adapter_pages")
    out = np.zeros(max(n.value, 1), np.int64)
    _check(_lib.lora_pool_adapter_pages(pool, adapter_id, out.ctypes.data, n.value, ctypes.byref(n),
                                        ctypes.byref(rank), ctypes.byref(users)), "lora_pool_adapter_pages")
    return out[: n.value].tolist(), rank.value, users.value


def lora_pool_kv_pages(pool, request_id):
    n = _i64()
    rc = _lib.lora_pool_kv_pages(pool, request_id, None, 0, ctypes.byref(n))
    if rc == LORA_ENOENT:
        raise LoraError(rc, "lora_pool_kv_pages")
    out = np.zeros(max(n.value, 1), np.int64)
    _check(_lib.lora_pool_kv_pages(pool, request_id, out.ctypes.data, n.value, ctypes.byref(n)), "lora_pool_kv_pages")
    return out[: n.value].tolist()


def lora_pool_free_list(pool):
    n = _i64()
    _lib.lora_pool_free_list(pool, None, 0, ctypes.byref(n))
    out = np.zeros(max(n.value, 1), np.int64)
    _check(_lib.lora_pool_free_list(pool, out.ctypes.data, n.value, ctypes.byref(n)), "lora_pool_free_list")
    return out[: n.value].tolist()


def lora_pool_resident(pool):
    n = _i32()
    _lib.lora_pool_resident(pool, None, 0, ctypes.byref(n))
    out = np.zeros(max(n.value, 1), np.int32)
    _check(_lib.lora_pool_resident(pool, out.ctypes.data, n.value, ctypes.byref(n)), "lora_pool_resident")
    return out[: n.value].tolist()


def lora_project_workspace_size(pool, T):
    return _lib.lora_project_workspace_size(pool, T)


def lora_project(pool, x, W, page_table, adapter_ids, ranks, scale, T, y, workspace, workspace_bytes=None,
                 stream=None, check=True):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = _lib.lora_project(pool, _ptr(x), _ptr(W), _ptr(page_table), _ptr(adapter_ids), _ptr(ranks), _ptr(scale),
                           T, _ptr(y), _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "lora_project") if check else rc


def lora_project_slots_workspace_size(pool, n, T):
    return _lib.lora_project_slots_workspace_size(pool, n, T)


def lora_project_slots(pool, slots, x, Ws, adapter_ids, ranks, scale, T, ys, workspace, workspace_bytes=None,
                       stream=None, check=True):
    """slots: sequence of slot indices; Ws, ys: sequences of tensors (or addresses), one per slot."""
    n = len(slots)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    sl = np.ascontiguousarray(slots, dtype=np.int32)
    wp = (ctypes.c_void_p * max(n, 1))(*[_ptr(w) for w in Ws])
    yp = (ctypes.c_void_p * max(n, 1))(*[_ptr(y) for y in ys])
    rc = _lib.lora_project_slots(pool, n, sl.ctypes.data, _ptr(x), ctypes.cast(wp, ctypes.c_void_p),
                                 _ptr(adapter_ids), _ptr(ranks), _ptr(scale), T, ctypes.cast(yp, ctypes.c_void_p),
                                 _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "lora_project_slots") if check else rc


def lora_debug_gather(pool, page_table, adapter_ids, ranks, T, out, stream=None, check=True):
    rc = _lib.lora_debug_gather(pool, _ptr(page_table), _ptr(adapter_ids), _ptr(ranks), T, _ptr(out),
                                _stream(stream))
    return _check(rc, "lora_debug_gather") if check else rc


def lora_project_slots_x(pool, slots, xs, Ws, adapter_ids, ranks, scale, T, ys, workspace, workspace_bytes=None,
                         stream=None, check=True):
    """slots: sequence of slot indices; xs, Ws, ys: sequences of tensors (or addresses), one per slot."""
    n = len(slots)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    sl = np.ascontiguousarray(slots, dtype=np.int32)
    xp = (ctypes.c_void_p * max(n, 1))(*[_ptr(x) for x in xs])
    wp = (ctypes.c_void_p * max(n, 1))(*[_ptr(w) for w in Ws])
    yp = (ctypes.c_void_p * max(n, 1))(*[_ptr(y) for y in ys])
    rc = _lib.lora_project_slots_x(pool, n, sl.ctypes.data, ctypes.cast(xp, ctypes.c_void_p),
                                   ctypes.cast(wp, ctypes.c_void_p), _ptr(adapter_ids), _ptr(ranks), _ptr(scale), T,
                                   ctypes.cast(yp, ctypes.c_void_p), _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "lora_project_slots_x") if check else rc


def lora_debug_project(pool, x, W, page_table, adapter_ids, ranks, scale, T, y, workspace, gather_out, order_out,
                       workspace_bytes=None, stream=None, check=True):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = _lib.lora_debug_project(pool, _ptr(x), _ptr(W), _ptr(page_table), _ptr(adapter_ids), _ptr(ranks),
                                 _ptr(scale), T, _ptr(y), _ptr(workspace), workspace_bytes, _ptr(gather_out),
                                 _ptr(order_out), _stream(stream))
    return _check(rc, "lora_debug_project") if check else rc


def lora_project_noalloc(pool, x, W, page_table, adapter_ids, ranks, scale, T, y, stream=None, check=True):
    rc = _lib.lora_project_noalloc(pool, _ptr(x), _ptr(W), _ptr(page_table), _ptr(adapter_ids), _ptr(ranks),
                                   _ptr(scale), T, _ptr(y), _stream(stream))
    return _check(rc, "lora_project_noalloc") if check else rc


def lora_kv_write(pool, layout, k, ldk, v, ldv, table, max_pages, q_start, lens, n_seq, T, stream=None, check=True):
    rc = _lib.lora_kv_write(pool, ctypes.byref(layout), _ptr(k), ldk, _ptr(v), ldv, _ptr(table), max_pages,
                            _ptr(q_start), _ptr(lens), n_seq, T, _stream(stream))
    return _check(rc, "lora_kv_write") if check else rc


def lora_kv_attend_workspace_size(pool, layout, n_seq, max_len, with_scores=False):
    return _lib.lora_kv_attend_workspace_size(pool, ctypes.byref(layout), n_seq, max_len, int(with_scores))


def lora_kv_attend(pool, layout, q, ldq, table, max_pages, lens, n_seq, max_len, scale, out, ldo, prior=None,
                   scores=None, workspace=None, workspace_bytes=None, stream=None, check=True):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.lora_kv_attend(pool, ctypes.byref(layout), _ptr(q), ldq, _ptr(table), max_pages, _ptr(lens), n_seq,
                             max_len, scale, _ptr(out), ldo, _ptr(prior), _ptr(scores), _ptr(workspace),
                             workspace_bytes, _stream(stream))
    return _check(rc, "lora_kv_attend") if check else rc


def lora_kv_attend_chunk_workspace_size(pool, layout, n_seq, T, max_len, with_scores=False):
    return _lib.lora_kv_attend_chunk_workspace_size(pool, ctypes.byref(layout), n_seq, T, max_len, int(with_scores))


def lora_kv_attend_chunk(pool, layout, q, ldq, table, max_pages, q_start, lens, n_seq, T, max_len, scale, out, ldo,
                         prior=None, scores=None, workspace=None, workspace_bytes=None, stream=None, check=True):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.lora_kv_attend_chunk(pool, ctypes.byref(layout), _ptr(q), ldq, _ptr(table), max_pages, _ptr(q_start),
                                   _ptr(lens), n_seq, T, max_len, scale, _ptr(out), ldo, _ptr(prior), _ptr(scores),
                                   _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "lora_kv_attend_chunk") if check else rc


def lora_kv_evict(pool, layout, layers, n_seq, table, table_out, max_pages, scores, scores_out, lens, lens_out, budget,
                  keep_first, keep_last, dropped, max_drop, n_dropped, stream=None, check=True):
    rc = _lib.lora_kv_evict(pool, ctypes.byref(layout), layers, n_seq, _ptr(table), _ptr(table_out), max_pages,
                            _ptr(scores), _ptr(scores_out), _ptr(lens), _ptr(lens_out), budget, keep_first, keep_last,
                            _ptr(dropped), max_drop, _ptr(n_dropped), _stream(stream))
    return _check(rc, "lora_kv_evict") if check else rc


def lora_check_device_errors(pool, check=True):
    rc = _lib.lora_check_device_errors(pool)
    return _check(rc, "lora_check_device_errors") if check else rc


def lora_profile_start(pool, max_calls):
    return _check(_lib.lora_profile_start(pool, max_calls), "lora_profile_start")


def lora_profile_stop(pool) -> dict:
    pr = lora_profile_t()
    _check(_lib.lora_profile_stop(pool, ctypes.byref(pr)), "lora_profile_stop")
    return {name: getattr(pr, name) for name, _ in pr._fields_}


def lora_last_error() -> str:
    return _lib.lora_last_error().decode(errors="replace")


def lora_version() -> str:
    return _lib.lora_version().decode()


def run_pool_ops(pool, ops, ranks, adapter_weights, stream=None):
    """Apply a list of pool operations (as the workload generators emit them) to a pool handle.

    adapter_weights(aid) -> (A_t, B).  Returns each operation's status code.
    """
    out = []
    for op in ops:
        k = op[0]
        if k == "load":
            aid = op[1]
            at, b = adapter_weights(aid) if int(ranks[aid]) > 0 else (None, None)
            out.append(lora_pool_load_adapter(pool, aid, int(ranks[aid]), at, b, stream, check=False))
        elif k == "kv":
            r = lora_pool_grow_kv(pool, op[1], op[2], check=False)
            out.append(r if isinstance(r, int) else 0)
        elif k == "free_kv":
            out.append(lora_pool_free_kv(pool, op[1], check=False))
        elif k == "release":
            out.append(lora_pool_release_adapter(pool, op[1], check=False))
        elif k == "evict":
            out.append(lora_pool_evict_adapter(pool, op[1], stream, check=False))
        else:
            raise ValueError(k)
    return out


# ---- convenience owner of a pool's device buffers ----------------------------------------------------

class Pool:
    """A pool plus the torch-allocated device memory it runs on (pages, page table, workspace)."""

    def __init__(self, num_pages, hidden, dtype, n_slots=1, max_adapters=1, max_rank=LORA_MAX_RANK,
                 free_order=None, device="cuda"):
        import torch
        self.torch = torch
        self.hidden, self.dtype, self.n_slots = hidden, dtype, n_slots
        self.max_rank, self.max_adapters, self.num_pages = max_rank, max_adapters, num_pages
        self.tdtype = torch.float32 if dtype == LORA_F32 else torch.bfloat16
        if device is None:
            self.pages = self.table = None
        else:
            self.pages = torch.empty((num_pages, hidden), dtype=self.tdtype, device=device)
            self.table = torch.empty((n_slots, max_adapters, 2 * max_rank), dtype=torch.int32, device=device)
        self.handle = lora_pool_create(self.pages, num_pages, hidden, dtype, max_rank, n_slots, max_adapters,
                                       self.table, free_order)
        self._ws = None

    def close(self):
        if self.handle:
            lora_pool_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def slot_table(self, slot):
        return self.table[slot]

    def stats(self):
        return lora_pool_stats(self.handle)

    def workspace(self, T):
        need = lora_project_workspace_size(self.handle, T)
        if self._ws is None or self._ws.numel() < need:
            self._ws = self.torch.empty(max(need, 256), dtype=self.torch.uint8, device=self.pages.device)
        return self._ws

    def run_ops(self, ops, ranks, adapter_weights, stream=None):
        return run_pool_ops(self.handle, ops, ranks, adapter_weights, stream)

    def project_slots(self, slots, x, Ws, adapter_ids, ranks, scale, ys=None, stream=None):
        """x: one tensor every slot reads (lora_project_slots), or a list with one per slot
        (lora_project_slots_x)."""
        per_slot = isinstance(x, (list, tuple))
        x0 = x[0] if per_slot else x
        T = x0.shape[0]
        if ys is None:
            ys = [self.torch.empty_like(x0) for _ in slots]
        need = lora_project_slots_workspace_size(self.handle, len(slots), T)
        if self._ws is None or self._ws.numel() < need:
            self._ws = self.torch.empty(max(need, 256), dtype=self.torch.uint8, device=self.pages.device)
        if per_slot:
            lora_project_slots_x(self.handle, slots, x, Ws, adapter_ids, ranks, scale, T, ys, self._ws, stream=stream)
        else:
            lora_project_slots(self.handle, slots, x, Ws, adapter_ids, ranks, scale, T, ys, self._ws, stream=stream)
        return ys

    def project(self, slot, x, W, adapter_ids, ranks, scale, y=None, stream=None):
        T = x.shape[0]
        if y is None:
            y = self.torch.empty_like(x)
        ws = self.workspace(T)
        lora_project(self.handle, x, W, self.table[slot], adapter_ids, ranks, scale, T, y, ws, stream=stream)
        return y

    # ---- the KV cache ----------------------------------------------------------------------------
    # layout: lora_kv_layout_t.  table: int32 [n_seq, 2, max_pages]; lens: int32 [n_seq]; q_start: int32
    # [n_seq + 1].  Workspace and outputs are allocated per call on the call's stream, so calls on
    # several streams, and calls captured into several graphs, share none.

    def _where(self, stream):
        """(stream handle, whether the call runs on the current stream)."""
        if stream is None:
            return _current_stream(self.pages.get_device()), True
        return (stream if isinstance(stream, int) else stream.cuda_stream), False

    def _empty(self, here, stream, shape, dtype):
        """Memory that belongs to the call's stream, as its allocator sees it."""
        if here:
            return self.pages.new_empty(shape, dtype=dtype)
        torch, dev = self.torch, self.pages.device
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=dev)

    def _like(self, here, stream, t):
        """As _empty, for a contiguous tensor of t's kind (the quickest of torch's calls that allocate)."""
        return self.torch.empty_like(t) if here else self._empty(here, stream, t.shape, t.dtype)

    def _kv_rows(self, what, t, width):
        """Rows of `width` elements of the pool's type: how far they lie apart."""
        shape, stride = t.shape, t.stride()
        if len(shape) != 2 or shape[1] != width or t.dtype is not self.tdtype or not t.is_cuda \
                or t.get_device() != self.pages.get_device() or (stride[1] != 1 and shape[0]):
            raise ValueError(f"{what}: rows of {width} {self.tdtype} elements on {self.pages.device} are wanted, not "
                             f"{tuple(shape)} {t.dtype} on {t.device}, strides {stride}")
        return stride[0]

    def _kv_ints(self, what, t, shape, dtype):
        if t.shape != shape or t.dtype is not dtype or not t.is_cuda or t.get_device() != self.pages.get_device() \
                or not t.is_contiguous():
            raise ValueError(f"{what}: contiguous {dtype} {shape} on {self.pages.device} is wanted, not {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")

    def _kv_pages(self):
        if self.pages is None:
            raise ValueError("a bookkeeping-only pool holds no KV vectors")

    def _kv_table(self, table, lens, q_start):
        self._kv_pages()
        i32 = torch.int32
        n, mp = table.shape[0], table.shape[-1]
        self._kv_ints("table", table, (n, 2, mp), i32)
        self._kv_ints("lens", lens, (n,), i32)
        if q_start is not None:
            self._kv_ints("q_start", q_start, (n + 1,), i32)
        return n, mp

    def kv_write(self, layout, k, v, table, lens, q_start=None, stream=None):
        """K and V rows of new tokens into their pages (lora_kv_write)."""
        n, mp = self._kv_table(table, lens, q_start)
        width = layout.n_kv_heads * layout.head_dim
        ldk, ldv = self._kv_rows("k", k, width), self._kv_rows("v", v, width)
        if k.shape[0] != v.shape[0]:
            raise ValueError(f"k has {k.shape[0]} rows and v {v.shape[0]}")
        lora_kv_write(self.handle, layout, k.data_ptr(), ldk, v.data_ptr(), ldv, table.data_ptr(), mp,
                      None if q_start is None else q_start.data_ptr(), lens.data_ptr(), n, k.shape[0],
                      stream=self._where(stream)[0])

    def _kv_attend(self, layout, q, table, lens, q_start, scale, max_len, out, scores, prior, workspace, stream):
        n, mp = self._kv_table(table, lens, q_start)
        T, width, cap = q.shape[0], layout.n_heads * layout.head_dim, mp * layout.tokens_per_page
        ldq = self._kv_rows("q", q, width)
        if q_start is None and T != n:
            raise ValueError(f"q has {T} rows for {n} sequences")
        if scores is not None:
            self._kv_ints("scores", scores, (n, cap), torch.float32)
        if prior is not None:
            self._kv_ints("prior", prior, (n, cap), torch.float32)
        handle, here = self._where(stream)
        if out is None:
            out, ldo = self._empty(here, stream, (T, width), self.tdtype), width
        else:
            ldo = self._kv_rows("out", out, width)
            if out.shape[0] != T:
                raise ValueError(f"out has {out.shape[0]} rows and q {T}")
        scale = layout.head_dim ** -0.5 if scale is None else scale
        max_len = cap if max_len is None else max_len
        if workspace is None:
            need = lora_kv_attend_workspace_size(self.handle, layout, n, max_len, scores is not None) \
                if q_start is None else \
                lora_kv_attend_chunk_workspace_size(self.handle, layout, n, T, max_len, scores is not None)
            workspace = self._empty(here, stream, (need,), torch.uint8) if need else None
        elif not workspace.is_cuda or workspace.get_device() != self.pages.get_device() or not workspace.is_contiguous():
            raise ValueError(f"workspace: contiguous memory on {self.pages.device} is wanted, not {tuple(workspace.shape)} on "
                             f"{workspace.device}, strides {workspace.stride()}")
        args = (None if prior is None else prior.data_ptr(), None if scores is None else scores.data_ptr(),
                None if workspace is None else workspace.data_ptr(),
                0 if workspace is None else workspace.numel() * workspace.element_size())
        if q_start is None:
            lora_kv_attend(self.handle, layout, q.data_ptr(), ldq, table.data_ptr(), mp, lens.data_ptr(), n, max_len,
                           scale, out.data_ptr(), ldo, *args, stream=handle)
        else:
            lora_kv_attend_chunk(self.handle, layout, q.data_ptr(), ldq, table.data_ptr(), mp, q_start.data_ptr(),
                                 lens.data_ptr(), n, T, max_len, scale, out.data_ptr(), ldo, *args, stream=handle)
        return out

    def kv_attend(self, layout, q, table, lens, scale=None, max_len=None, out=None, scores=None, prior=None,
                  workspace=None, stream=None):
        """Attention of one new token per sequence (lora_kv_attend).  scale None: head_dim ** -0.5; max_len
        None: the table's capacity; scores: float32 [n_seq, max_pages * tokens_per_page], written as
        prior + this call's weights (prior=scores accumulates in place)."""
        return self._kv_attend(layout, q, table, lens, None, scale, max_len, out, scores, prior, workspace, stream)

    def kv_attend_chunk(self, layout, q, table, lens, q_start, scale=None, max_len=None, out=None, scores=None,
                        prior=None, workspace=None, stream=None):
        """Causal attention of many new tokens per sequence (lora_kv_attend_chunk); arguments as kv_attend's."""
        return self._kv_attend(layout, q, table, lens, q_start, scale, max_len, out, scores, prior, workspace, stream)

    def kv_evict(self, layout, table, scores, lens, budget, keep_first=0, keep_last=0, max_drop=None, in_place=False,
                 stream=None):
        """Thin the caches out by accumulated attention (lora_kv_evict).  table: int32 [layers, n_seq, 2,
        max_pages]; scores: float32 [layers, n_seq, max_pages * tokens_per_page].  Returns (table, scores, lens,
        dropped, n_dropped), the first two the tensors passed in if in_place."""
        self._kv_pages()
        layers, n, mp = table.shape[0], table.shape[1], table.shape[-1]
        self._kv_ints("table", table, (layers, n, 2, mp), torch.int32)
        self._kv_ints("scores", scores, (layers, n, mp * layout.tokens_per_page), torch.float32)
        self._kv_ints("lens", lens, (n,), torch.int32)
        max_drop = mp if max_drop is None else max_drop
        handle, here = self._where(stream)
        table_out = table if in_place else self._like(here, stream, table)
        scores_out = scores if in_place else self._like(here, stream, scores)
        lens_out, n_dropped = self._like(here, stream, lens), self._like(here, stream, lens)
        if max_drop == mp:
            dropped = self._like(here, stream, table)
        else:
            dropped = self._empty(here, stream, (layers, n, 2, max_drop), torch.int32)
        lora_kv_evict(self.handle, layout, layers, n, table.data_ptr(), table_out.data_ptr(), mp, scores.data_ptr(),
                      scores_out.data_ptr(), lens.data_ptr(), lens_out.data_ptr(), budget, keep_first, keep_last,
                      dropped.data_ptr(), max_drop, n_dropped.data_ptr(), stream=handle)
        return table_out, scores_out, lens_out, dropped, n_dropped


from .kv_cache import KvCache  # noqa: E402,F401

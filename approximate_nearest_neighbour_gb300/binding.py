"""Thin ctypes binding of libivfpq_gb300.so (include/ivfpq.h).

Argument marshalling only: every function here checks shapes and dtypes of
torch CUDA tensors, passes their device pointers and the current CUDA stream
to the C entry point of the same name, and raises :class:`IVFPQError` on a
non-zero status. No computation happens in Python and there is no CPU
fallback: if the library has not been built, :class:`LibraryMissing` is
raised.
"""

from __future__ import annotations

import ctypes as C
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libivfpq_gb300.so")

IVFPQ_OK = 0
IVFPQ_ERR_INVALID_ARG = -1
IVFPQ_ERR_UNSUPPORTED = -2
IVFPQ_ERR_OOM = -3
IVFPQ_ERR_CUDA = -4
IVFPQ_ERR_DEVICE_CHECK = -5
IVFPQ_ERR_TIMEOUT = -6

LUT_FP32, LUT_FP16, LUT_FP8 = 0, 1, 2
LUT_TYPES = {"fp32": LUT_FP32, "fp16": LUT_FP16, "fp8": LUT_FP8}
MAX_K = 2048
MXFP4, NVFP4 = 0, 1
FP4_FORMATS = {"mxfp4": MXFP4, "nvfp4": NVFP4}
MAX_BEAMS, MAX_BEAM_K = 64, 128
MAX_RANK, MAX_ADAPTERS = 128, 8191

# name -> (restype, argtypes); mirrors include/ivfpq.h
_VP, _I, _I64, _F = C.c_void_p, C.c_int, C.c_int64, C.c_float
SIGNATURES = {
    "ivfpq_index_create": (_I, [_I, _I, _I, _I, _VP, _VP, C.POINTER(_VP)]),
    "ivfpq_index_destroy": (_I, [_VP]),
    "ivfpq_set_lut_type": (_I, [_VP, _I]),
    "ivfpq_add": (_I, [_VP, _VP, _VP, _VP, _I64, _VP]),
    "ivfpq_ntotal": (_I64, [_VP]),
    "ivfpq_search": (_I, [_VP, _VP, _I64, _I, _I, _VP, _VP, _VP]),
    "ivfpq_search_probes": (_I, [_VP, _VP, _I64, _I, _VP, _VP, _VP]),
    "ivfpq_search_preassigned": (_I, [_VP, _VP, _I64, _I, _VP, _I, _VP, _VP, _VP]),
    "ivfpq_set_profiling": (_I, [_VP, _I]),
    "ivfpq_stage_times": (_I, [_VP, C.POINTER(C.c_float), C.POINTER(C.c_int)]),
    "ivfpq_last_scan_kernel": (C.c_char_p, [_VP]),
    "ivfpq_set_precomputed": (_I, [_VP, _I]),
    "ivfpq_set_scan_mode": (_I, [_VP, _I, _I]),
    "ivfpq_uses_precomputed": (_I, [_VP]),
    "ivfpq_kernel_launches": (C.c_uint64, []),
    "ivfpq_workspace_allocations": (C.c_uint64, []),
    "flat_knn": (_I, [_VP, _I64, _I, _VP, _I64, _I, _VP, _VP, _VP]),
    "kselect": (_I, [_VP, _I64, _I64, _I, _VP, _VP, _VP]),
    "kselect_noalloc": (_I, [_VP, _I64, _I64, _I, _VP, _VP, _VP]),
    "knn_merge": (_I, [_VP, _VP, _I64, _I, _I, _I, _VP, _VP, _VP]),
    "kmeans_lloyd": (_I, [_VP, _I64, _I, _I, _I, _VP, _VP, _VP, _VP, _VP]),
    "pq_train": (_I, [_VP, _I64, _I, _I, _I, _VP, _VP, _VP, _VP]),
    "ivfpq_encode": (_I, [_VP, _VP, _I64, _VP, _VP, _VP]),
    "ivfpq_residuals": (_I, [_VP, _I, _I, _VP, _I64, _VP, _VP, _VP]),
    "ivfpq_encode_hinted": (_I, [_VP, _VP, _I64, _VP, _VP, _VP, C.POINTER(_I64), _VP]),
    "ivfpq_repaired_queries": (_I, [_VP, C.POINTER(_I64), _VP]),
    "ivfpq_knn_graph": (_I, [_VP, _VP, _VP, _I64, _I, _I, _VP, _VP, _VP]),
    "fp4_quantize": (_I, [_VP, _I, _I64, _I64, _I64, _I, _VP, _VP, _VP, _VP]),
    "fp4_dequantize": (_I, [_VP, _VP, _I64, _I64, _I, _VP, _VP, _I, _VP]),
    "fp4_product": (_I, [_VP, _VP, _I64, _VP, _VP, _I64, _I64, _I, _VP, _VP, _VP, _I, _VP]),
    "fp4_linear": (_I, [_VP, _I, _I64, _I64, _VP, _VP, _I64, _I64, _I, _VP, _VP, _VP, _I, _VP]),
    "score_adjust": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _I64, _I64, _VP, _VP, _VP, _VP, _VP,
                          _VP, _VP, _I64, _VP, _VP, _I64, _I, _VP, _I, _I64, _VP]),
    "topk_distill_forward": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _VP, _I, _F, _I, _VP, _VP,
                                  _VP]),
    "topk_distill_backward": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _VP, _I, _F, _I, _VP, _VP,
                                   _VP, _I64, _VP]),
    "topk_distill": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _VP, _I, _F, _I, _VP, _VP, _VP, _I64,
                          _VP]),
    "beam_select": (_I, [_VP, _I, _I64, _I, _I64, _I64, _VP, _VP, C.c_int32, _I, _VP, _VP, _VP,
                         _VP]),
    "beam_reorder": (_I, [_VP, _I, _VP, _I64, _I, _I, _VP, _VP]),
    "embedding_lookup": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _I, _I64, _F, _VP, _I, _I64, _VP]),
    "embedding_gradient": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _I, _I64, _F, _I64, _I, _VP, _I,
                                _I64, _VP]),
    "adapter_linear": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _VP, _I, _I, _I64, _VP, _VP, _VP,
                            _I64, _VP, _I, _I64, _VP]),
    "ivfpq_device_check": (_I, [_VP]),
    "ivfpq_selftest_wait_timeout": (_I, [_I, _VP]),
    "ivfpq_last_error": (C.c_char_p, []),
    "ivfpq_status_string": (C.c_char_p, [_I]),
}


class LibraryMissing(RuntimeError):
    pass


class IVFPQError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


_lib = None
_lock = threading.Lock()


def lib():
    """The loaded library (raises LibraryMissing if it was never built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise LibraryMissing(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = C.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def _check(fn, status):
    if status != IVFPQ_OK:
        msg = lib().ivfpq_last_error().decode(errors="replace")
        raise IVFPQError(fn, status, msg)


def _torch():
    import torch
    return torch


def _stream(stream=None):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, dtype, name, ndim=None, device=True):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(t, shape, dtype, name, device):
    """A caller-given output checked against the shape the call writes
    (the library trusts its pointers), or a new tensor."""
    torch = _torch()
    shape = tuple(int(v) for v in shape)
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.device != torch.device(device):
        raise ValueError(f"{name} must be on {device} (the inputs' device), got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _same_device(what, *tensors):
    devs = {t.device for t in tensors if t is not None}
    if len(devs) > 1:
        raise ValueError(f"{what}: tensors on several devices {sorted(map(str, devs))}")


# ---------------------------------------------------------------------------
class Index:
    """Owner of an ivfpq_index handle."""

    def __init__(self, handle, d, nlist, m):
        self.handle = handle
        self.d, self.nlist, self.m = d, nlist, m

    def __del__(self):
        try:
            if self.handle:
                lib().ivfpq_index_destroy(self.handle)
                self.handle = None
        except Exception:
            pass

    @property
    def ntotal(self):
        return int(lib().ivfpq_ntotal(self.handle))


def ivfpq_index_create(centroids, codebooks, nbits=8):
    """centroids: fp32 [nlist, d]; codebooks: fp32 [m, 256, d/m] (CUDA)."""
    torch = _torch()
    _need(centroids, torch.float32, "centroids", 2)
    _need(codebooks, torch.float32, "codebooks", 3)
    nlist, d = centroids.shape
    m = codebooks.shape[0]
    if m < 1 or d % m or tuple(codebooks.shape[1:]) != (256, d // m):
        raise ValueError(f"ivfpq_index_create: codebooks must be [m, 256, d/m] with d = {d}, "
                         f"got {tuple(codebooks.shape)}")
    _same_device("ivfpq_index_create", centroids, codebooks)
    h = C.c_void_p()
    _check("ivfpq_index_create",
           lib().ivfpq_index_create(d, nlist, m, nbits, _ptr(centroids), _ptr(codebooks),
                                    C.byref(h)))
    return Index(h, d, nlist, m)


def ivfpq_index_destroy(index):
    if index.handle:
        _check("ivfpq_index_destroy", lib().ivfpq_index_destroy(index.handle))
        index.handle = None


def ivfpq_set_lut_type(index, lut_type):
    if isinstance(lut_type, str):
        lut_type = LUT_TYPES[lut_type]
    _check("ivfpq_set_lut_type", lib().ivfpq_set_lut_type(index.handle, int(lut_type)))


def ivfpq_add(index, codes, list_ids, ids, stream=None):
    """codes: uint8 [n, m]; list_ids: int32 [n]; ids: int64 [n] (CUDA)."""
    torch = _torch()
    _need(codes, torch.uint8, "codes", 2)
    _need(list_ids, torch.int32, "list_ids", 1)
    _need(ids, torch.int64, "ids", 1)
    n = codes.shape[0]
    if codes.shape[1] != index.m or list_ids.shape[0] != n or ids.shape[0] != n:
        raise ValueError("ivfpq_add: inconsistent shapes")
    _same_device("ivfpq_add", codes, list_ids, ids)
    _check("ivfpq_add", lib().ivfpq_add(index.handle, _ptr(codes), _ptr(list_ids), _ptr(ids), n,
                                         _stream(stream)))


def _queries(fn, index, queries):
    """Checks a [nq, d] fp32 query matrix against the index's d (the kernels
    read d floats per row, so a narrower matrix would be read past its end)
    before checking that it is a contiguous CUDA tensor."""
    torch = _torch()
    _need(queries, torch.float32, "queries", 2, device=False)
    if queries.shape[1] != index.d:
        raise ValueError(f"{fn}: query dimension {queries.shape[1]} does not match the "
                         f"index's d = {index.d}")
    _need(queries, torch.float32, "queries", 2)
    return queries.shape[0]


def ivfpq_search(index, queries, nprobe, k, out_dist=None, out_ids=None, stream=None):
    torch = _torch()
    nq = _queries("ivfpq_search", index, queries)
    out_dist = _out(out_dist, (nq, k), torch.float32, "out_dist", queries.device)
    out_ids = _out(out_ids, (nq, k), torch.int64, "out_ids", queries.device)
    _check("ivfpq_search", lib().ivfpq_search(index.handle, _ptr(queries), nq, nprobe, k,
                                               _ptr(out_dist), _ptr(out_ids), _stream(stream)))
    return out_dist, out_ids


def ivfpq_search_probes(index, queries, nprobe, with_dist=True, stream=None):
    torch = _torch()
    nq = _queries("ivfpq_search_probes", index, queries)
    probes = torch.empty((nq, nprobe), dtype=torch.int32, device=queries.device)
    coarse = (torch.empty((nq, nprobe), dtype=torch.float32, device=queries.device)
              if with_dist else None)
    _check("ivfpq_search_probes",
           lib().ivfpq_search_probes(index.handle, _ptr(queries), nq, nprobe, _ptr(probes),
                                     _ptr(coarse), _stream(stream)))
    return probes, coarse


def ivfpq_search_preassigned(index, queries, probes, k, out_dist=None, out_ids=None,
                             stream=None):
    torch = _torch()
    _need(queries, torch.float32, "queries", 2)
    _need(probes, torch.int32, "probes", 2)
    nq, nprobe = probes.shape
    if tuple(queries.shape) != (nq, index.d):
        raise ValueError(f"ivfpq_search_preassigned: queries must be [{nq}, {index.d}] "
                         f"(one row per probe row), got {tuple(queries.shape)}")
    _same_device("ivfpq_search_preassigned", queries, probes)
    out_dist = _out(out_dist, (nq, k), torch.float32, "out_dist", queries.device)
    out_ids = _out(out_ids, (nq, k), torch.int64, "out_ids", queries.device)
    _check("ivfpq_search_preassigned",
           lib().ivfpq_search_preassigned(index.handle, _ptr(queries), nq, nprobe, _ptr(probes), k,
                                          _ptr(out_dist), _ptr(out_ids), _stream(stream)))
    return out_dist, out_ids


def ivfpq_set_profiling(index, enable=True):
    _check("ivfpq_set_profiling", lib().ivfpq_set_profiling(index.handle, int(bool(enable))))


def ivfpq_stage_times(index):
    """([coarse, plan, scan, merge] milliseconds summed over the searches
    recorded since profiling was enabled, number of searches)."""
    buf = (C.c_float * 4)()
    n = C.c_int(0)
    _check("ivfpq_stage_times", lib().ivfpq_stage_times(index.handle, buf, C.byref(n)))
    return list(buf), n.value


def ivfpq_set_precomputed(index, mode):
    """-1 automatic, 0 off, 1 on (where supported) for the precomputed-term
    lookup tables; returns whether searches now use them."""
    _check("ivfpq_set_precomputed", lib().ivfpq_set_precomputed(index.handle, int(mode)))
    return bool(lib().ivfpq_uses_precomputed(index.handle))


def ivfpq_set_scan_mode(index, mode, group=0):
    """-1 automatic, 0 by query, 1 by list (where its shapes apply); group =
    table sets per by-list item (2 or 3, -1 automatic, 0 keeps it)."""
    _check("ivfpq_set_scan_mode", lib().ivfpq_set_scan_mode(index.handle, int(mode), int(group)))


def ivfpq_uses_precomputed(index):
    return bool(lib().ivfpq_uses_precomputed(index.handle))


def last_scan_kernel(index):
    """Name of the list-scan kernel family the index's last search used."""
    r = lib().ivfpq_last_scan_kernel(index.handle)
    return r.decode() if r else None


def kernel_launches():
    """Kernels launched by the library since it was loaded."""
    return int(lib().ivfpq_kernel_launches())


def workspace_allocations():
    """Temporary device allocations the library has made since it was loaded."""
    return int(lib().ivfpq_workspace_allocations())


def device_check(stream=None):
    """Synchronises the stream and raises IVFPQError (IVFPQ_ERR_TIMEOUT) if a
    kernel of the library gave up a bounded wait since the last check."""
    _check("ivfpq_device_check", lib().ivfpq_device_check(_stream(stream)))


def selftest_wait_timeout(spins=1024, stream=None):
    """Launches a block whose bounded wait is bound to expire (nothing
    completes the barrier phase it waits on); device_check() then reports
    it."""
    _check("ivfpq_selftest_wait_timeout",
           lib().ivfpq_selftest_wait_timeout(int(spins), _stream(stream)))


def flat_knn(db, queries, k, out_dist=None, out_ids=None, stream=None):
    torch = _torch()
    _need(db, torch.float32, "db", 2)
    _need(queries, torch.float32, "queries", 2)
    n, d = db.shape
    nq = queries.shape[0]
    if queries.shape[1] != d:
        raise ValueError("flat_knn: dimension mismatch")
    _same_device("flat_knn", db, queries)
    out_dist = _out(out_dist, (nq, k), torch.float32, "out_dist", queries.device)
    out_ids = _out(out_ids, (nq, k), torch.int64, "out_ids", queries.device)
    _check("flat_knn", lib().flat_knn(_ptr(db), n, d, _ptr(queries), nq, k, _ptr(out_dist),
                                       _ptr(out_ids), _stream(stream)))
    return out_dist, out_ids


def kmeans_lloyd(x, init, niter, stream=None):
    """Lloyd k-means on device fp32 x [n, d] seeded from rows init (int64
    [k]): (centroids [k, d], assignment int32 [n], objective per pass as a
    numpy fp64 array of niter + 1)."""
    import numpy as np
    torch = _torch()
    _need(x, torch.float32, "x", 2)
    _need(init, torch.int64, "init", 1)
    n, d = x.shape
    k = init.shape[0]
    _same_device("kmeans_lloyd", x, init)
    cent = torch.empty((k, d), dtype=torch.float32, device=x.device)
    assign = torch.empty((n,), dtype=torch.int32, device=x.device)
    obj = np.zeros(niter + 1, np.float64)
    _check("kmeans_lloyd", lib().kmeans_lloyd(
        _ptr(x), n, d, k, niter, _ptr(init), _ptr(cent), _ptr(assign),
        obj.ctypes.data_as(C.c_void_p), _stream(stream)))
    return cent, assign, obj


def pq_train(x, m, niter, init, stream=None):
    """Product quantizer codebooks [m, 256, d/m] trained on device fp32 x
    [n, d], seeded from rows init (int64 [256]); returns (codebooks,
    objective per pass, numpy fp64 [niter + 1])."""
    import numpy as np
    torch = _torch()
    _need(x, torch.float32, "x", 2)
    _need(init, torch.int64, "init", 1)
    n, d = x.shape
    if init.shape[0] != 256:
        raise ValueError(f"pq_train: init must hold 256 seed rows, got {init.shape[0]}")
    _same_device("pq_train", x, init)
    cb = torch.empty((m, 256, d // m), dtype=torch.float32, device=x.device)
    obj = np.zeros(niter + 1, np.float64)
    _check("pq_train", lib().pq_train(_ptr(x), n, d, m, niter, _ptr(init), _ptr(cb),
                                       obj.ctypes.data_as(C.c_void_p), _stream(stream)))
    return cb, obj


def ivfpq_knn_graph(index, x, self_ids, nprobe, k, stream=None):
    """k approximate neighbours of every row of x among the index's other
    vectors: ([n, k] fp32 distances, [n, k] int64 ids)."""
    torch = _torch()
    _need(x, torch.float32, "x", 2)
    _need(self_ids, torch.int64, "self_ids", 1)
    n = x.shape[0]
    if x.shape[1] != index.d or self_ids.shape[0] != n:
        raise ValueError(f"ivfpq_knn_graph: x must be [n, {index.d}] and self_ids [n], got "
                         f"{tuple(x.shape)} and {tuple(self_ids.shape)}")
    _same_device("ivfpq_knn_graph", x, self_ids)
    d = torch.empty((n, k), dtype=torch.float32, device=x.device)
    i = torch.empty((n, k), dtype=torch.int64, device=x.device)
    _check("ivfpq_knn_graph", lib().ivfpq_knn_graph(index.handle, _ptr(x), _ptr(self_ids), n,
                                                     nprobe, k, _ptr(d), _ptr(i),
                                                     _stream(stream)))
    return d, i


def ivfpq_encode(index, x, stream=None):
    """(list ids int32 [n], codes uint8 [n, m]) of device fp32 x [n, d]."""
    torch = _torch()
    _need(x, torch.float32, "x", 2)
    n = x.shape[0]
    if x.shape[1] != index.d:
        raise ValueError(f"ivfpq_encode: x must be [n, {index.d}], got {tuple(x.shape)}")
    lists = torch.empty((n,), dtype=torch.int32, device=x.device)
    codes = torch.empty((n, index.m), dtype=torch.uint8, device=x.device)
    _check("ivfpq_encode", lib().ivfpq_encode(index.handle, _ptr(x), n, _ptr(lists),
                                               _ptr(codes), _stream(stream)))
    return lists, codes


def ivfpq_residuals(centroids, x, stream=None):
    """(nearest centroid int32 [n], residual x - centroid fp32 [n, d]) of device
    fp32 x [n, d] against device fp32 centroids [nlist, d]."""
    torch = _torch()
    _need(centroids, torch.float32, "centroids", 2)
    _need(x, torch.float32, "x", 2)
    nlist, d = centroids.shape
    n = x.shape[0]
    if x.shape[1] != d:
        raise ValueError(f"ivfpq_residuals: x must be [n, {d}], got {tuple(x.shape)}")
    _same_device("ivfpq_residuals", centroids, x)
    lists = torch.empty((n,), dtype=torch.int32, device=x.device)
    resid = torch.empty((n, d), dtype=torch.float32, device=x.device)
    _check("ivfpq_residuals", lib().ivfpq_residuals(_ptr(centroids), nlist, d, _ptr(x), n,
                                                     _ptr(lists), _ptr(resid), _stream(stream)))
    return lists, resid


def ivfpq_encode_hinted(index, x, hint, list_ids=None, codes=None, stream=None):
    """ivfpq_encode with a candidate list per row (int32 [n]): (list ids,
    codes, rows that needed the full nearest-centroid search)."""
    torch = _torch()
    _need(x, torch.float32, "x", 2)
    _need(hint, torch.int32, "hint", 1)
    n = x.shape[0]
    if x.shape[1] != index.d or hint.shape[0] != n:
        raise ValueError(f"ivfpq_encode_hinted: x must be [n, {index.d}] and hint [n], got "
                         f"{tuple(x.shape)} and {tuple(hint.shape)}")
    _same_device("ivfpq_encode_hinted", x, hint)
    list_ids = _out(list_ids, (n,), torch.int32, "list_ids", x.device)
    codes = _out(codes, (n, index.m), torch.uint8, "codes", x.device)
    searched = C.c_int64(0)
    _check("ivfpq_encode_hinted",
           lib().ivfpq_encode_hinted(index.handle, _ptr(x), n, _ptr(hint), _ptr(list_ids),
                                     _ptr(codes), C.byref(searched), _stream(stream)))
    return list_ids, codes, int(searched.value)


def ivfpq_repaired_queries(index, stream=None):
    """Queries re-scanned with full-length queues since the previous call."""
    n = C.c_int64(0)
    _check("ivfpq_repaired_queries",
           lib().ivfpq_repaired_queries(index.handle, C.byref(n), _stream(stream)))
    return int(n.value)


def knn_merge(dists, ids, k, out_dist=None, out_ids=None, stream=None):
    """k smallest of S shards' results per query. dists fp32 and ids int64,
    both [S, nq, k_in] on the device; returns ([nq, k] fp32, [nq, k] int64)."""
    torch = _torch()
    _need(dists, torch.float32, "dists", 3)
    _need(ids, torch.int64, "ids", 3)
    if tuple(ids.shape) != tuple(dists.shape):
        raise ValueError("knn_merge: dists and ids must have the same shape")
    S, nq, k_in = dists.shape
    _same_device("knn_merge", dists, ids)
    out_dist = _out(out_dist, (nq, k), torch.float32, "out_dist", dists.device)
    out_ids = _out(out_ids, (nq, k), torch.int64, "out_ids", dists.device)
    _check("knn_merge", lib().knn_merge(_ptr(dists), _ptr(ids), nq, S, k_in, k, _ptr(out_dist),
                                         _ptr(out_ids), _stream(stream)))
    return out_dist, out_ids


def kselect(vals, k, out_vals=None, out_idx=None, stream=None):
    torch = _torch()
    _need(vals, torch.float32, "vals", 2)
    rows, cols = vals.shape
    out_vals = _out(out_vals, (rows, k), torch.float32, "out_vals", vals.device)
    out_idx = _out(out_idx, (rows, k), torch.int64, "out_idx", vals.device)
    _check("kselect", lib().kselect(_ptr(vals), rows, cols, k, _ptr(out_vals), _ptr(out_idx),
                                     _stream(stream)))
    return out_vals, out_idx


def kselect_noalloc(vals, k, out_vals, out_idx, stream=None):
    """kselect through the entry point that allocates no device memory; the
    caller provides the outputs (fp32 and int64, [rows, k])."""
    torch = _torch()
    _need(vals, torch.float32, "vals", 2)
    if out_vals is None or out_idx is None:
        raise ValueError("kselect_noalloc: the caller provides out_vals and out_idx")
    rows, cols = vals.shape
    out_vals = _out(out_vals, (rows, k), torch.float32, "out_vals", vals.device)
    out_idx = _out(out_idx, (rows, k), torch.int64, "out_idx", vals.device)
    _check("kselect_noalloc", lib().kselect_noalloc(_ptr(vals), rows, cols, k, _ptr(out_vals),
                                                     _ptr(out_idx), _stream(stream)))
    return out_vals, out_idx


# ---- 4-bit vectors, score rows and distillation ------------------------------
# These calls take a few microseconds on the device for small inputs, so their
# marshalling stays short: one look-up of the stream, no context managers, and
# the general checks (_need, _out) only where a cheap test does not settle them.
class _Late(dict):
    """torch's names these calls use, looked up once (torch is imported late)."""

    def __missing__(self, key):
        torch = _torch()
        self.update(Tensor=torch.Tensor, empty=torch.empty, f32=torch.float32, i32=torch.int32,
                    i64=torch.int64, u8=torch.uint8, bool=torch.bool,
                    device=torch._C._cuda_getDevice,
                    stream=torch._C._cuda_getCurrentRawStream,
                    codes={torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
        return self[key]


_late = _Late()


def _dtype_code(t, name):
    """ivfpq_dtype of a torch dtype."""
    code = _late["codes"].get(t)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t}")
    return code


def _rows(t, name):
    """(dtype code, rows, cols, row stride) of a floating 2-d CUDA matrix whose
    rows are dense; the rows themselves may be strided or repeated."""
    try:
        code = _dtype_code(t.dtype, name)
        rows, cols = t.shape
        ld, inner = t.stride()
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    except ValueError:
        raise ValueError(f"{name} must have 2 dimensions") from None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must have dense rows (stride 1 along columns)")
    if rows <= 1:
        ld = cols
    elif 0 < ld < cols:
        raise ValueError(f"{name} must not have overlapping rows")
    return code, rows, cols, ld


def _array(t, dtype, shape, name, dev):
    """Address of a contiguous tensor of the given shape and dtype on device
    dev (an index)."""
    if not isinstance(t, _late["Tensor"]):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _need(t, dtype, name, len(shape))
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    return t.data_ptr()


def _out_rows(t, shape, dtype, name, device):
    """A caller-given output whose rows may be strided: its row stride."""
    _, rows, cols, ld = _rows(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if (rows, cols) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (the inputs' device), got {t.device}")
    if rows > 1 and ld < cols:
        raise ValueError(f"{name} must not repeat rows")
    return ld


def _current(dev):
    """Handle of the current stream of device dev (an index), which must be the
    current device: kernels are launched there."""
    if _late["device"]() != dev:
        raise ValueError(f"the tensors are on cuda:{dev} and the current device is another")
    return _late["stream"](dev)


def _on_stream(fn, stream, args, kwargs):
    """fn(*args, **kwargs) with `stream` current: its outputs belong to that
    stream, and the allocator keeps the given tensors until its work is done."""
    torch = _torch()
    for t in (*args, *kwargs.values()):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return fn(*args, **kwargs)


def _fp4_format(fmt):
    f = FP4_FORMATS.get(fmt) if isinstance(fmt, str) else fmt
    if f != MXFP4 and f != NVFP4:
        raise ValueError(f"unknown 4-bit format {fmt!r}: one of {sorted(FP4_FORMATS)}")
    return f


def fp4_shapes(rows, cols, fmt="mxfp4"):
    """Shapes of the packed codes and of the scale tiles of a [rows, cols] matrix."""
    kp = (cols + 31) // 32 * 32
    span = 128 if _fp4_format(fmt) == MXFP4 else 64  # columns of a scale tile
    return (rows, kp // 2), ((rows + 127) // 128, (kp + span - 1) // span, 512)


def _packed(codes, scales, f, name, cols=None):
    """(rows, columns) of packed rows, with the scales' shape checked against the codes'."""
    u8 = _late["u8"]
    try:
        rows, pitch = codes.shape
        shape = scales.shape
        ok = (codes.dtype is u8 and scales.dtype is u8 and codes.is_cuda
              and scales.get_device() == codes.get_device() and codes.is_contiguous()
              and scales.is_contiguous())
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _need(codes, u8, f"{name} codes", 2)
        _need(scales, u8, f"{name} scales", 3)
        raise ValueError(f"{name}: codes and scales on several devices")
    if pitch == 0 or pitch % 16:
        raise ValueError(f"{name} codes must have a multiple of 16 bytes per row, got {pitch}")
    kp = 2 * pitch
    if cols is None:
        cols = kp
    elif not kp - 32 < cols <= kp:
        raise ValueError(f"{name}: {cols} columns do not match codes of {pitch} bytes per row")
    span = 128 if f == MXFP4 else 64
    if shape != ((rows + 127) // 128, (kp + span - 1) // span, 512):
        raise ValueError(f"{name} scales must have shape {fp4_shapes(rows, cols, f)[1]}, got "
                         f"{tuple(shape)}")
    return rows, cols


def fp4_quantize(x, fmt="mxfp4", tensor_scale=None, codes=None, scales=None, stream=None):
    """(codes, scales) of the rows of x in a 4-bit block-scaled format:
    "mxfp4" (a power-of-two scale per 32 columns) or "nvfp4" (an E4M3 scale per
    16 columns beside tensor_scale, fp32 [1] on the device, 1 if not given)."""
    if stream is not None:
        return _on_stream(fp4_quantize, stream, (x, fmt, tensor_scale, codes, scales), {})
    f = _fp4_format(fmt)
    code, rows, cols, ld = _rows(x, "x")
    dev, at = x.device, x.get_device()
    g = (None if tensor_scale is None
         else _array(tensor_scale, _late["f32"], (1,), "tensor_scale", at))
    cs, ss = fp4_shapes(rows, cols, f)
    u8 = _late["u8"]
    codes = (_late["empty"](cs, dtype=u8, device=dev) if codes is None
             else _out(codes, cs, u8, "codes", dev))
    scales = (_late["empty"](ss, dtype=u8, device=dev) if scales is None
              else _out(scales, ss, u8, "scales", dev))
    rc = (_lib or lib()).fp4_quantize(x.data_ptr(), code, rows, cols, ld, f, g, codes.data_ptr(),
                                      scales.data_ptr(), _current(at))
    if rc:
        _check("fp4_quantize", rc)
    return codes, scales


def fp4_dequantize(codes, scales, cols=None, fmt="mxfp4", tensor_scale=None, dtype=None, out=None,
                   stream=None):
    """The values packed rows stand for, [rows, cols] (cols: all packed columns
    if not given) of dtype (float32 if not given)."""
    if stream is not None:
        return _on_stream(fp4_dequantize, stream,
                          (codes, scales, cols, fmt, tensor_scale, dtype, out), {})
    f = _fp4_format(fmt)
    rows, cols = _packed(codes, scales, f, "fp4_dequantize:", cols)
    dev, at = codes.device, codes.get_device()
    if dtype is None:
        dtype = _late["f32"] if out is None else out.dtype
    code = _dtype_code(dtype, "dtype")
    g = (None if tensor_scale is None
         else _array(tensor_scale, _late["f32"], (1,), "tensor_scale", at))
    out = (_late["empty"]((rows, cols), dtype=dtype, device=dev) if out is None
           else _out(out, (rows, cols), dtype, "out", dev))
    rc = (_lib or lib()).fp4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, f, g,
                                        out.data_ptr(), code, _current(at))
    if rc:
        _check("fp4_dequantize", rc)
    return out


def fp4_product(a_codes, a_scales, b_codes, b_scales, fmt="mxfp4", a_tensor_scale=None,
                b_tensor_scale=None, dtype=None, out=None, stream=None):
    """Inner products [m, n] of packed rows a [m, cols] and b [n, cols], in
    dtype (float32 if not given: score rows for kselect, once negated)."""
    if stream is not None:
        return _on_stream(fp4_product, stream, (a_codes, a_scales, b_codes, b_scales, fmt,
                                                a_tensor_scale, b_tensor_scale, dtype, out), {})
    f = _fp4_format(fmt)
    m, cols = _packed(a_codes, a_scales, f, "fp4_product: a")
    n, bcols = _packed(b_codes, b_scales, f, "fp4_product: b")
    if cols != bcols:
        raise ValueError(f"fp4_product: a has {cols} packed columns and b {bcols}")
    dev, at = a_codes.device, a_codes.get_device()
    if b_codes.get_device() != at:
        _same_device("fp4_product", a_codes, b_codes)
    f32 = _late["f32"]
    if dtype is None:
        dtype = f32 if out is None else out.dtype
    code = _dtype_code(dtype, "dtype")
    ga = gb = None
    if a_tensor_scale is not None:
        ga = _array(a_tensor_scale, f32, (1,), "a_tensor_scale", at)
    if b_tensor_scale is not None:
        gb = _array(b_tensor_scale, f32, (1,), "b_tensor_scale", at)
    out = (_late["empty"]((m, n), dtype=dtype, device=dev) if out is None
           else _out(out, (m, n), dtype, "out", dev))
    rc = (_lib or lib()).fp4_product(
        a_codes.data_ptr(), a_scales.data_ptr(), m, b_codes.data_ptr(), b_scales.data_ptr(), n,
        cols, f, ga, gb, out.data_ptr(), code, _current(at))
    if rc:
        _check("fp4_product", rc)
    return out


def fp4_linear(x, w_codes, w_scales, fmt="mxfp4", x_tensor_scale=None, w_tensor_scale=None,
               dtype=None, out=None, stream=None):
    """x [m, cols] quantized row by row, times packed weights w [n, cols]:
    [m, n] in dtype (x's if not given)."""
    if stream is not None:
        return _on_stream(fp4_linear, stream, (x, w_codes, w_scales, fmt, x_tensor_scale,
                                               w_tensor_scale, dtype, out), {})
    f = _fp4_format(fmt)
    xcode, m, cols, ld = _rows(x, "x")
    n, _ = _packed(w_codes, w_scales, f, "fp4_linear: w", cols)
    dev, at = x.device, x.get_device()
    if w_codes.get_device() != at:
        _same_device("fp4_linear", x, w_codes)
    if dtype is None:
        dtype = x.dtype if out is None else out.dtype
    code = xcode if dtype is x.dtype else _dtype_code(dtype, "dtype")
    gx = gw = None
    if x_tensor_scale is not None:
        gx = _array(x_tensor_scale, _late["f32"], (1,), "x_tensor_scale", at)
    if w_tensor_scale is not None:
        gw = _array(w_tensor_scale, _late["f32"], (1,), "w_tensor_scale", at)
    out = (_late["empty"]((m, n), dtype=dtype, device=dev) if out is None
           else _out(out, (m, n), dtype, "out", dev))
    rc = (_lib or lib()).fp4_linear(x.data_ptr(), xcode, m, ld, w_codes.data_ptr(),
                                    w_scales.data_ptr(), n, cols, f, gx, gw, out.data_ptr(), code,
                                    _current(at))
    if rc:
        _check("fp4_linear", rc)
    return out


def score_adjust(scores, history=None, history_len=None, prompt_len=None, repetition=None,
                 presence=None, frequency=None, bias_ids=None, bias_vals=None, temperature=None,
                 mask=None, negate=False, out=None, dtype=None, stream=None):
    """Score rows with penalties for repeated tokens, biases, temperature and a
    bit mask applied (include/ivfpq.h states the order). history: int32
    [rows, length] (rows may be strided) with history_len and prompt_len int32
    [rows]; repetition, presence, frequency, temperature: fp32 [rows];
    bias_ids / bias_vals: int32 / fp32 [rows, nb]; mask: int32 [rows or 1,
    ceil(cols / 32)], set bits are allowed. out (scores itself, or the scores'
    type or float32) is made if not given."""
    if stream is not None:
        return _on_stream(score_adjust, stream,
                          (scores, history, history_len, prompt_len, repetition, presence,
                           frequency, bias_ids, bias_vals, temperature, mask, negate, out, dtype),
                          {})
    i32, f32, Tensor = _late["i32"], _late["f32"], _late["Tensor"]
    code, rows, cols, lds = _rows(scores, "scores")
    dev, at = scores.device, scores.get_device()
    hist = hl = pl = bi = bv = mk = rep = pres = freq = temp = None
    hist_cols = ldh = nb = ldm = 0
    one = (rows,)
    if history is not None:
        if not isinstance(history, Tensor) or history.dtype is not i32:
            raise TypeError("history must be an int32 tensor")
        if history.dim() != 2 or history.shape[0] != rows or history.get_device() != at:
            raise ValueError(f"history must be [{rows}, length] on {dev}")
        hist_cols = history.shape[1]
        ldh, inner = history.stride()
        if hist_cols > 1 and inner != 1:
            raise ValueError("history must have dense rows (stride 1 along its length)")
        if history_len is not None:
            hl = _array(history_len, i32, one, "history_len", at)
        if prompt_len is not None:
            pl = _array(prompt_len, i32, one, "prompt_len", at)
        hist = history.data_ptr()
        if hist_cols == 0:
            hist = hl = pl = None
    elif history_len is not None or prompt_len is not None:
        raise ValueError("history_len and prompt_len need a history")
    if (bias_ids is None) != (bias_vals is None):
        raise ValueError("bias_ids and bias_vals go together")
    if bias_ids is not None:
        if not isinstance(bias_ids, Tensor):
            raise TypeError("bias_ids must be a torch tensor")
        if bias_ids.dim() != 2 or bias_ids.shape[0] != rows:
            raise ValueError(f"bias_ids and bias_vals must both be [{rows}, nb]")
        nb = bias_ids.shape[1]
        bi = _array(bias_ids, i32, (rows, nb), "bias_ids", at)
        bv = _array(bias_vals, f32, (rows, nb), "bias_vals", at)
        if nb == 0:
            bi = bv = None
    if mask is not None:
        words = (cols + 31) // 32
        if not isinstance(mask, Tensor):
            raise TypeError("mask must be a torch tensor")
        mrows = rows if mask.dim() == 2 and mask.shape[0] == rows else 1
        mk = _array(mask, i32, (mrows, words), "mask", at)
        ldm = words if mrows == rows else 0
    if repetition is not None:
        rep = _array(repetition, f32, one, "repetition", at)
    if presence is not None:
        pres = _array(presence, f32, one, "presence", at)
    if frequency is not None:
        freq = _array(frequency, f32, one, "frequency", at)
    if temperature is not None:
        temp = _array(temperature, f32, one, "temperature", at)
    if dtype is None:
        dtype = scores.dtype if out is None else out.dtype
    ocode = code if dtype is scores.dtype else _dtype_code(dtype, "dtype")
    if out is None:
        out, ldo = _late["empty"]((rows, cols), dtype=dtype, device=dev), cols
    else:
        ldo = _out_rows(out, (rows, cols), dtype, "out", dev)
    rc = (_lib or lib()).score_adjust(
        scores.data_ptr(), code, rows, cols, lds, hist, hist_cols, ldh, hl, pl, rep, pres, freq,
        bi, bv, nb, temp, mk, ldm, 1 if negate else 0, out.data_ptr(), ocode, ldo, _current(at))
    if rc:
        _check("score_adjust", rc)
    return out


def _teacher(scores, vals, ids):
    """Checks of a distillation call's inputs: (dtype code, rows, cols, row
    stride, k, addresses of the teacher's values and ids, device index)."""
    code, rows, cols, ld = _rows(scores, "scores")
    try:
        k = vals.shape[1]
    except (AttributeError, IndexError):
        _need(vals, _late["f32"], "teacher_vals", 2)
        raise
    at = scores.get_device()
    return (code, rows, cols, ld, k, _array(vals, _late["f32"], (rows, k), "teacher_vals", at),
            _array(ids, _late["i64"], (rows, k), "teacher_ids", at), at)


def topk_distill_forward(scores, teacher_vals, teacher_ids, temperature=1.0, negated=False,
                         stream=None):
    """(loss fp32 [rows], stats fp32 [rows, 2]) of the student's score rows
    against a teacher's top list, as kselect or a search returns it (fp32
    values and int64 ids, [rows, k]); negated: smaller values are better, as in
    distances. stats is for topk_distill_backward."""
    if stream is not None:
        return _on_stream(topk_distill_forward, stream,
                          (scores, teacher_vals, teacher_ids, temperature, negated), {})
    code, rows, cols, ld, k, tv, ti, at = _teacher(scores, teacher_vals, teacher_ids)
    dev = scores.device
    loss = _late["empty"]((rows,), dtype=_late["f32"], device=dev)
    stats = _late["empty"]((rows, 2), dtype=_late["f32"], device=dev)
    rc = (_lib or lib()).topk_distill_forward(scores.data_ptr(), code, rows, cols, ld, tv, ti, k,
                                              temperature, 1 if negated else 0, loss.data_ptr(),
                                              stats.data_ptr(), _current(at))
    if rc:
        _check("topk_distill_forward", rc)
    return loss, stats


def topk_distill_backward(scores, teacher_vals, teacher_ids, stats, row_grad, temperature=1.0,
                          negated=False, grad=None, stream=None):
    """Gradient of sum(row_grad * loss) with respect to the scores, in their
    type; grad may be scores itself. A row whose row_grad is 0 gets zeros."""
    if stream is not None:
        return _on_stream(topk_distill_backward, stream,
                          (scores, teacher_vals, teacher_ids, stats, row_grad, temperature,
                           negated, grad), {})
    code, rows, cols, ld, k, tv, ti, at = _teacher(scores, teacher_vals, teacher_ids)
    dev = scores.device
    st = _array(stats, _late["f32"], (rows, 2), "stats", at)
    w = _array(row_grad, _late["f32"], (rows,), "row_grad", at)
    if grad is None:
        grad, ldg = _late["empty"]((rows, cols), dtype=scores.dtype, device=dev), cols
    else:
        ldg = _out_rows(grad, (rows, cols), scores.dtype, "grad", dev)
    rc = (_lib or lib()).topk_distill_backward(scores.data_ptr(), code, rows, cols, ld, tv, ti, k,
                                               temperature, 1 if negated else 0, st, w,
                                               grad.data_ptr(), ldg, _current(at))
    if rc:
        _check("topk_distill_backward", rc)
    return grad


def topk_distill(scores, teacher_vals, teacher_ids, row_grad, temperature=1.0, negated=False,
                 grad=None, stream=None):
    """(loss fp32 [rows], gradient of sum(row_grad * loss)) in one call, as a
    training step needs them; grad may be scores itself."""
    if stream is not None:
        return _on_stream(topk_distill, stream,
                          (scores, teacher_vals, teacher_ids, row_grad, temperature, negated,
                           grad), {})
    code, rows, cols, ld, k, tv, ti, at = _teacher(scores, teacher_vals, teacher_ids)
    dev = scores.device
    w = _array(row_grad, _late["f32"], (rows,), "row_grad", at)
    loss = _late["empty"]((rows,), dtype=_late["f32"], device=dev)
    if grad is None:
        grad, ldg = _late["empty"]((rows, cols), dtype=scores.dtype, device=dev), cols
    else:
        ldg = _out_rows(grad, (rows, cols), scores.dtype, "grad", dev)
    rc = (_lib or lib()).topk_distill(scores.data_ptr(), code, rows, cols, ld, tv, ti, k,
                                      temperature, 1 if negated else 0, w, loss.data_ptr(),
                                      grad.data_ptr(), ldg, _current(at))
    if rc:
        _check("topk_distill", rc)
    return loss, grad


# ---- beams, embeddings and adapters ------------------------------------------
def beam_select(scores, totals, k, finished=None, end_id=0, stream=None):
    """(totals fp32, beams int32, ids int32), all [groups, k]: the k best
    continuations of each group's beams, best first (include/ivfpq.h states the
    order). scores: [groups * beams, cols], rows may be strided; totals: fp32
    [groups, beams], -inf for a beam that is not alive; finished: bool or uint8
    [groups, beams], beams whose only continuation is end_id at their own total.
    Fewer than k continuations: (-inf, -1, -1) at the tail."""
    if stream is not None:
        return _on_stream(beam_select, stream, (scores, totals, k, finished, end_id), {})
    code, rows, cols, lds = _rows(scores, "scores")
    at, dev, empty, f32 = scores.get_device(), scores.device, _late["empty"], _late["f32"]
    try:
        groups, beams = totals.shape
    except (AttributeError, ValueError):
        _need(totals, f32, "totals", 2)
        raise
    if groups * beams != rows:
        raise ValueError(f"totals are {groups} x {beams} and scores have {rows} rows")
    t = _array(totals, f32, (groups, beams), "totals", at)
    fin = None
    if finished is not None:
        if not isinstance(finished, _late["Tensor"]):
            raise TypeError("finished must be a torch tensor")
        if finished.dtype is not _late["u8"] and finished.dtype is not _late["bool"]:
            raise TypeError(f"finished must be bool or uint8, got {finished.dtype}")
        fin = _array(finished, finished.dtype, (groups, beams), "finished", at)
        if not 0 <= end_id < cols:
            raise ValueError(f"end_id={end_id} outside [0, {cols})")
    shape, i32 = (groups, k), _late["i32"]
    out = empty(shape, dtype=f32, device=dev)
    which = empty(shape, dtype=i32, device=dev)
    ids = empty(shape, dtype=i32, device=dev)
    rc = (_lib or lib()).beam_select(scores.data_ptr(), code, groups, beams, cols, lds, t, fin,
                                     end_id, k, out.data_ptr(), which.data_ptr(), ids.data_ptr(),
                                     _current(at))
    if rc:
        _check("beam_select", rc)
    return out, which, ids


# ivfpq_state of include/ivfpq.h as nine int64: src, dst, src_row, dst_row, outer,
# src_outer, dst_outer, inner, unit
_STATE = 9


def _dense_tail(shape, stride):
    """Leading dimensions left when the dense trailing ones are one run."""
    run, i = 1, len(shape)
    while i > 1 and (shape[i - 1] == 1 or stride[i - 1] == run):
        run *= shape[i - 1]
        i -= 1
    return i


def _segments(shape, stride, end, name):
    """(number, stride) of the segments that dimensions 1 .. end - 1 count."""
    n, step = 1, 0
    for size, st in zip(shape[end - 1:0:-1], stride[end - 1:0:-1]):
        if size == 1:
            continue
        if n == 1:
            n, step = size, st
        elif st == step * n:
            n *= size
        else:
            raise ValueError(f"{name}: dimensions before the positions must have one stride")
    return n, step


def _state(t, o, axis, groups, width, n, lengths, at, index):
    """The ivfpq_state (nine numbers) of tensor t written to o, positions along
    dimension axis."""
    Tensor = _late["Tensor"]
    if not isinstance(t, Tensor) or not isinstance(o, Tensor):
        raise TypeError(f"states[{index}] must be a torch tensor")
    if t.get_device() != at or o.get_device() != at or not t.is_cuda:
        raise ValueError(f"states[{index}] and its output must be on cuda:{at}")
    shape, so, size = t.shape, o.shape, t.element_size()
    dims = len(shape)
    if dims < 1 or shape[0] != groups * width:
        raise ValueError(f"states[{index}] must have {groups * width} rows, got shape "
                         f"{tuple(shape)}")
    if o is not t and (o.dtype != t.dtype or so[0] != groups * n or so[1:] != shape[1:]):
        raise ValueError(f"the output of states[{index}] must be {t.dtype} with {groups * n} "
                         f"rows of its shape, got {o.dtype} {tuple(so)}")
    if lengths and not 1 <= axis < dims:
        raise ValueError(f"states[{index}]: positions must be one of its dimensions 1 to "
                         f"{dims - 1}")
    st = t.stride()
    sto = st if o is t else o.stride()
    if lengths:
        unit = size
        for v in shape[axis + 1:]:
            unit *= v
        inner = unit * shape[axis]
    if t.is_contiguous() and (o is t or o.is_contiguous()):
        row = size
        for v in shape[1:]:
            row *= v
        if not lengths:
            return (t.data_ptr(), o.data_ptr(), row, row, 1, 0, 0, row, 0)
        return (t.data_ptr(), o.data_ptr(), row, row, row // inner if inner else 0, inner,
                inner, inner, unit)
    first = max(_dense_tail(shape, st), _dense_tail(shape, sto))
    if lengths:
        if first > axis:
            raise ValueError(f"states[{index}]: positions and what follows them must be dense")
        first = axis
    else:
        unit, inner = 0, size
        for v in shape[first:]:
            inner *= v
    outer, src_outer = _segments(shape, st, first, f"states[{index}]")
    _, dst_outer = _segments(shape, sto, first, f"states[{index}]")
    src_row = st[0] if shape[0] > 1 else 0
    dst_row = sto[0] if so[0] > 1 else 0
    return (t.data_ptr(), o.data_ptr(), src_row * size, dst_row * size, outer,
            src_outer * size, dst_outer * size, inner, unit)


def beam_reorder(states, beams, lengths=None, axis=1, out=None, stream=None):
    """The states of the beams (a tensor or a sequence of tensors, each with
    groups * width rows of any dtype) in the order of the selected continuations:
    row g * n + j becomes row g * width + beams[g, j]. beams: int32 [groups, n], as
    beam_select returns them; a beam outside the group leaves its row as it was.
    lengths: int32 [groups], the positions in use along dimension `axis` (one
    number, or one per state); what lies past them stays as it was. In place (n =
    width) unless out, tensors of groups * n rows, is given; returns what was
    written. States must not overlap each other, nor a state an output other than
    its own. A state that repeats memory within its rows is refused in place."""
    if stream is not None:
        flat = [states] if not isinstance(states, (list, tuple)) else list(states)
        flat += ([] if out is None else [out] if not isinstance(out, (list, tuple)) else list(out))
        for t in flat:
            if isinstance(t, _late["Tensor"]) and t.is_cuda:
                t.record_stream(stream)
        return _on_stream(beam_reorder, stream, (states, beams, lengths, axis, out), {})
    one = not isinstance(states, (list, tuple))
    src = [states] if one else states
    dst = src if out is None else [out] if one else out
    if len(dst) != len(src):
        raise ValueError(f"{len(src)} states and {len(dst)} outputs")
    i32 = _late["i32"]
    try:
        groups, n = beams.shape
    except (AttributeError, ValueError):
        _need(beams, i32, "beams", 2)
        raise
    at = beams.get_device()
    b = _array(beams, i32, (groups, n), "beams", at)
    if not beams.is_cuda:
        raise ValueError("beams must be a CUDA tensor")
    length = None if lengths is None else _array(lengths, i32, (groups,), "lengths", at)
    if not src or groups == 0 or n == 0:
        return out if out is not None else states
    axes = axis if isinstance(axis, (list, tuple)) else [axis] * len(src)
    if len(axes) != len(src):
        raise ValueError(f"{len(src)} states and {len(axes)} position dimensions")
    rows = src[0].shape[0] if isinstance(src[0], _late["Tensor"]) and src[0].dim() else -1
    if rows < 0 or rows % groups:
        raise ValueError(f"states[0] must have a multiple of {groups} rows")
    width = rows // groups
    if out is None and width != n:
        raise ValueError(f"in place, {n} continuations need as many rows, not {width}")
    numbers = []
    seen = set()
    for i, (t, o, d) in enumerate(zip(src, dst, axes)):
        st = _state(t, o, d, groups, width, n, length is not None, at, i)
        if st[1] in seen and st[4] and st[7]:  # (empty ones may share an address)
            raise ValueError(f"states[{i}] is written twice")
        seen.add(st[1])
        numbers += st
    array = (C.c_int64 * len(numbers))(*numbers)
    rc = (_lib or lib()).beam_reorder(array, len(src), b, groups, width, n, length, _current(at))
    if rc:
        _check("beam_reorder", rc)
    return out if out is not None else states


def _ids(ids, name, dev):
    """(address, bytes per id, count) of a contiguous int32 or int64 tensor."""
    if not isinstance(ids, _late["Tensor"]):
        raise TypeError(f"{name} must be a torch tensor")
    dtype = ids.dtype
    if dtype is not _late["i32"] and dtype is not _late["i64"]:
        raise TypeError(f"{name} must be int32 or int64, got {dtype}")
    return _array(ids, dtype, ids.shape, name, dev), 4 if dtype is _late["i32"] else 8, ids.numel()


def embedding_lookup(table, ids, scale=1.0, dtype=None, out=None, stream=None):
    """scale * table[ids], [*ids.shape, cols] in dtype (the table's if not given,
    or float32); zeros where an id is outside the table. table: [rows, cols],
    rows may be strided; ids: int32 or int64, any shape; out: 2-d with strided
    rows for 1-d ids, contiguous otherwise, in memory of its own."""
    if stream is not None:
        return _on_stream(embedding_lookup, stream, (table, ids, scale, dtype, out), {})
    code, rows, cols, ldt = _rows(table, "table")
    at = table.get_device()
    p, size, tokens = _ids(ids, "ids", at)
    if dtype is None:
        dtype = table.dtype if out is None else out.dtype
    ocode = code if dtype is table.dtype else _dtype_code(dtype, "dtype")
    ldo = cols
    if out is None:
        out = _late["empty"]((*ids.shape, cols), dtype=dtype, device=table.device)
    elif ids.dim() == 1:
        ldo = _out_rows(out, (tokens, cols), dtype, "out", table.device)
    else:
        out = _out(out, (*ids.shape, cols), dtype, "out", table.device)
    to = out.data_ptr()
    if to == table.data_ptr() and tokens and rows and cols:
        raise ValueError("out must not be the table's memory")
    rc = (_lib or lib()).embedding_lookup(table.data_ptr(), code, rows, cols, ldt, p, size, tokens,
                                          scale, to, ocode, ldo, _current(at))
    if rc:
        _check("embedding_lookup", rc)
    return out


def embedding_gradient(grad, ids, rows, scale=1.0, padding=None, accumulate=False, dtype=None,
                       out=None, stream=None):
    """The gradient [rows, cols] of embedding_lookup's table from grad [tokens,
    cols] (rows may be strided or one repeated) and ids, int32 or int64 of as many
    elements: scale times the sums by token, in dtype (grad's if not given, or
    float32). Ids outside the table and the id `padding` have none. accumulate:
    the sums are added to out, which must be given; rows without a token stay. out
    has memory of its own."""
    if stream is not None:
        return _on_stream(embedding_gradient, stream,
                          (grad, ids, rows, scale, padding, accumulate, dtype, out), {})
    code, tokens, cols, ldg = _rows(grad, "grad")
    at = grad.get_device()
    p, size, count = _ids(ids, "ids", at)
    if count != tokens:
        raise ValueError(f"{count} ids and {tokens} rows of grad")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if dtype is None:
        dtype = grad.dtype if out is None else out.dtype
    ocode = code if dtype is grad.dtype else _dtype_code(dtype, "dtype")
    if out is None:
        out, ldo = _late["empty"]((rows, cols), dtype=dtype, device=grad.device), cols
    else:
        ldo = _out_rows(out, (rows, cols), dtype, "out", grad.device)
    to = out.data_ptr()
    if to == grad.data_ptr() and tokens and rows and cols:
        raise ValueError("out must not be grad's memory")
    rc = (_lib or lib()).embedding_gradient(
        grad.data_ptr(), code, tokens, cols, ldg, p, size, rows, scale,
        -1 if padding is None else padding, 1 if accumulate else 0, to, ocode, ldo, _current(at))
    if rc:
        _check("embedding_gradient", rc)
    return out


def adapter_linear(x, a, b, ids, scales=None, base=None, dtype=None, out=None, stream=None):
    """base[t] + scales[i] * (x[t] @ a[i].T) @ b[i].T with i = ids[t], [tokens, n]:
    low-rank adapters beside a projection that all requests share (base: its
    result; zeros if not given). x: fp16 or bf16 [tokens, cols], rows may be
    strided; a: [adapters, rank, cols], b: [adapters, n, rank] of x's dtype; ids:
    int32 [tokens], outside [0, adapters) for a token without one; scales: fp32
    [adapters]. In base's dtype, or dtype (x's if not given, or float32). out may be
    base itself."""
    if stream is not None:
        return _on_stream(adapter_linear, stream, (x, a, b, ids, scales, base, dtype, out), {})
    code, tokens, cols, ldx = _rows(x, "x")
    at, dev, i32 = x.get_device(), x.device, _late["i32"]
    try:
        adapters, rank, _ = a.shape
        _, n, _ = b.shape
    except (AttributeError, ValueError):
        _need(a, x.dtype, "a", 3)
        _need(b, x.dtype, "b", 3)
        raise
    pa = _array(a, x.dtype, (adapters, rank, cols), "a", at)
    pb = _array(b, x.dtype, (adapters, n, rank), "b", at)
    pi = _array(ids, i32, (tokens,), "ids", at)
    ps = None if scales is None else _array(scales, _late["f32"], (adapters,), "scales", at)
    pbase, ldb = None, 0
    if base is not None:
        if dtype is None:
            dtype = base.dtype if out is None else out.dtype
        _, brows, bcols, ldb = _rows(base, "base")
        if base.dtype != dtype or (brows, bcols) != (tokens, n) or base.get_device() != at:
            raise ValueError(f"base must be {dtype} [{tokens}, {n}] on {dev}, got {base.dtype} "
                             f"{tuple(base.shape)} on {base.device}")
        pbase = base.data_ptr()
    if dtype is None:
        dtype = x.dtype if out is None else out.dtype
    ocode = code if dtype is x.dtype else _dtype_code(dtype, "dtype")
    if out is None:
        out, ldo = _late["empty"]((tokens, n), dtype=dtype, device=dev), n
    else:
        ldo = _out_rows(out, (tokens, n), dtype, "out", dev)
    rc = (_lib or lib()).adapter_linear(x.data_ptr(), code, tokens, cols, ldx, pa, pb, adapters,
                                        rank, n, pi, ps, pbase, ldb, out.data_ptr(), ocode, ldo,
                                        _current(at))
    if rc:
        _check("adapter_linear", rc)
    return out

"""Python binding of the B200 masked attention forward C ABI (include/fa.h).

Argument marshalling only: every step of the computation runs in the CUDA
library ``libfa_b200.so`` (built in-tree by ``masked_attention_fa_b200.build``).
PyTorch is used for device memory and streams. If the library is missing the
import of any entry point fails loudly; there is no fallback.

The C entry points keep their names (``fa_create``, ``fa_fwd``, ...). The
``MaskedAttention`` class wraps a handle for convenience.
"""
from __future__ import annotations

import ctypes
import math
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_b200.so")

FA_BNSD, FA_BSND, FA_TND = 0, 1, 2
LAYOUTS = {"BNSD": FA_BNSD, "BSND": FA_BSND, "TND": FA_TND}
FA_MASK_NONE, FA_MASK_SS, FA_MASK_B1SS, FA_MASK_BNSS = 0, 1, 2, 3
MASK_KINDS = {None: FA_MASK_NONE, "SS": FA_MASK_SS, "B1SS": FA_MASK_B1SS, "BNSS": FA_MASK_BNSS}
STATUS = {0: "FA_OK", 1: "FA_ERR_NULLPTR", 2: "FA_ERR_PARAM_INVALID", 3: "FA_ERR_SHAPE",
          4: "FA_ERR_UNSUPPORTED", 5: "FA_ERR_ALLOC", 6: "FA_ERR_CUDA", 7: "FA_ERR_TIMEOUT",
          8: "FA_ERR_DEVICE"}
FA_TILE_EMPTY, FA_TILE_PARTIAL, FA_TILE_FULL = 0, 1, 2
FA_ALIBI_NONE, FA_ALIBI_RIGHT, FA_ALIBI_SQRT, FA_ALIBI_LEFT = 0, 1, 2, 3
ALIBI = {None: FA_ALIBI_NONE, "right": FA_ALIBI_RIGHT, "sqrt": FA_ALIBI_SQRT,
         "left": FA_ALIBI_LEFT}


class FaError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {message}")


class fa_desc_t(ctypes.Structure):
    _fields_ = [
        ("layout", ctypes.c_int32),
        ("sparse_mode", ctypes.c_int32),
        ("mask_kind", ctypes.c_int32),
        ("alibi", ctypes.c_int32),
        ("B", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("Sq", ctypes.c_int64),
        ("Skv", ctypes.c_int64),
        ("D", ctypes.c_int64),
        ("pre_tokens", ctypes.c_int64),
        ("next_tokens", ctypes.c_int64),
        ("scale", ctypes.c_double),
    ]


class fa_split_part_t(ctypes.Structure):
    _fields_ = [
        ("desc", fa_desc_t),
        ("q_begin", ctypes.c_int64),
        ("q_end", ctypes.c_int64),
        ("kv_begin", ctypes.c_int64),
        ("kv_end", ctypes.c_int64),
    ]


class fa_relbias_t(ctypes.Structure):
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("bucket_of", ctypes.c_void_p),
        ("num_buckets", ctypes.c_int32),
        ("reach", ctypes.c_int32),
    ]


_lib = None


def load_library():
    """Load libfa_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m masked_attention_fa_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    i64p = P  # host int64 arrays, passed as addresses
    dp = ctypes.POINTER(fa_desc_t)
    st = ctypes.c_int32
    lib.fa_create.argtypes = [dp, ctypes.POINTER(P)]
    lib.fa_create.restype = st
    lib.fa_fwd.argtypes = [P, P, P, P, P, i64p, i64p, i64p, P, P, P]
    lib.fa_fwd.restype = st
    lib.fa_fwd_alibi.argtypes = [P, P, P, P, P, i64p, i64p, i64p, P, P, P]
    lib.fa_fwd_alibi.restype = st
    rp = ctypes.POINTER(fa_relbias_t)
    lib.fa_fwd_relbias.argtypes = [P, P, P, P, rp, i64p, i64p, i64p, P, P, P]
    lib.fa_fwd_relbias.restype = st
    lib.fa_bwd.argtypes = [P, P, P, P, P, P, P, P, P, i64p, i64p, i64p, P, P, P, P]
    lib.fa_bwd.restype = st
    lib.fa_bwd_alibi.argtypes = [P, P, P, P, P, P, P, P, P, i64p, i64p, i64p, P, P, P, P]
    lib.fa_bwd_alibi.restype = st
    lib.fa_bwd_relbias.argtypes = [P, P, P, P, rp, P, P, P, P, i64p, i64p, i64p, P, P, P, P, P]
    lib.fa_bwd_relbias.restype = st
    lib.fa_sync_status.argtypes = [P]
    lib.fa_sync_status.restype = st
    lib.fa_destroy.argtypes = [P]
    lib.fa_destroy.restype = st
    lib.fa_last_error.argtypes = []
    lib.fa_last_error.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = ctypes.c_int32
    lib.fa_validate.argtypes = [dp, i64p, i64p, i64p, ctypes.c_int32]
    lib.fa_validate.restype = st
    lib.fa_visible_pairs.argtypes = [dp, i64p, i64p, i64p, ctypes.c_int32, i64p]
    lib.fa_visible_pairs.restype = st
    lib.fa_tile_class.argtypes = [dp, i64p, i64p, i64p, ctypes.c_int32, ctypes.c_int64,
                                  ctypes.c_int64, ctypes.c_int64]
    lib.fa_tile_class.restype = ctypes.c_int32
    lib.fa_plan_stats.argtypes = [dp, i64p, i64p, i64p, ctypes.c_int32, i64p]
    lib.fa_plan_stats.restype = st
    lib.fa_plan_items.argtypes = [dp, i64p, i64p, i64p, ctypes.c_int32, ctypes.c_int64,
                                  ctypes.POINTER(ctypes.c_int32), i64p]
    lib.fa_plan_items.restype = st
    lib.fa_fwd_noalloc.argtypes = [dp, P, P, P, P, i64p, i64p, i64p, P, P, P]
    lib.fa_fwd_noalloc.restype = st
    lib.fa_noalloc_sync_status.argtypes = [P]
    lib.fa_noalloc_sync_status.restype = st
    lib.fa_fwd_paged.argtypes = [P, P, P, P, P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                 i64p, i64p, i64p, P, P, P]
    lib.fa_fwd_paged.restype = st
    lib.fa_mask_occupancy.argtypes = [dp, P, P, P, P]
    lib.fa_mask_occupancy.restype = st
    lib.fa_fwd_with_ranges.argtypes = [P, P, P, P, P, P, P, P, P]
    lib.fa_fwd_with_ranges.restype = st
    lib.fa_split_queries.argtypes = [dp, i64p, i64p, ctypes.c_int32, i64p, ctypes.c_int32,
                                     ctypes.POINTER(fa_split_part_t), i64p, i64p]
    lib.fa_split_queries.restype = st
    _lib = lib
    return lib


EXPORTED = ("fa_create", "fa_fwd", "fa_sync_status", "fa_destroy", "fa_last_error",
            "fa_version", "fa_validate", "fa_visible_pairs", "fa_tile_class", "fa_plan_stats",
            "fa_plan_items", "fa_fwd_noalloc", "fa_split_queries", "fa_mask_occupancy",
            "fa_fwd_with_ranges", "fa_fwd_paged", "fa_noalloc_sync_status", "fa_fwd_alibi",
            "fa_fwd_relbias", "fa_bwd", "fa_bwd_alibi", "fa_bwd_relbias")


def _check(status):
    if status != 0:
        msg = load_library().fa_last_error().decode(errors="replace")
        raise FaError(status, msg)


# Work-list size per SM from which closed-form calls claim their items at
# run time (the library's kClaimMinItemsPerCta; used to name the kernel
# instance a call runs).
CLAIM_MIN_ITEMS_PER_CTA = 8


def make_desc(layout, B, N, Sq, Skv, D, sparse_mode=0, pre_tokens=0, next_tokens=0, scale=None,
              mask_kind=None, alibi=None) -> fa_desc_t:
    lay = LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    mk = MASK_KINDS[mask_kind] if (mask_kind is None or isinstance(mask_kind, str)) else int(mask_kind)
    al = ALIBI[alibi] if (alibi is None or isinstance(alibi, str)) else int(alibi)
    sc = (1.0 / float(D) ** 0.5) if scale is None else float(scale)
    return fa_desc_t(lay, int(sparse_mode), mk, al, int(B), int(N), int(Sq), int(Skv), int(D),
                     int(pre_tokens), int(next_tokens), sc)


class _Arrays:
    """Host int64 arrays for prefix / actual_seq_* kept alive for one call."""

    def __init__(self, prefix, cu_q, cu_kv):
        self.prefix = None if prefix is None else np.ascontiguousarray(prefix, dtype=np.int64)
        self.cu_q = None if cu_q is None else np.ascontiguousarray(cu_q, dtype=np.int64)
        self.cu_kv = None if cu_kv is None else np.ascontiguousarray(cu_kv, dtype=np.int64)

    @staticmethod
    def _p(a):
        return None if a is None else a.__array_interface__["data"][0]

    def ptrs(self):
        return self._p(self.prefix), self._p(self.cu_q), self._p(self.cu_kv)


def _need_lengths(desc, prefix, cu_q, cu_kv):
    """The library reads B entries of every array that the problem takes."""
    takes = []
    if desc.sparse_mode in (5, 6):
        takes.append(("prefix", prefix))
    if desc.layout == FA_TND:
        takes += [("actual_seq_qlen", cu_q), ("actual_seq_kvlen", cu_kv)]
    for name, a in takes:
        n = desc.B if a is None else len(a) if isinstance(a, (list, tuple)) else np.asarray(a).size
        if n < desc.B:
            raise ValueError(f"{name} has {n} entries, the problem {desc.B} batch entries")


# ---------------------------------------------------------------- C names

def fa_version() -> int:
    return int(load_library().fa_version())


def fa_last_error() -> str:
    return load_library().fa_last_error().decode(errors="replace")


def fa_validate(desc, prefix=None, actual_seq_qlen=None, actual_seq_kvlen=None, has_mask=False):
    """Status code of the host-side checks (0 = valid)."""
    _need_lengths(desc, prefix, actual_seq_qlen, actual_seq_kvlen)
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    return int(load_library().fa_validate(ctypes.byref(desc), *a.ptrs(), int(bool(has_mask))))


def fa_visible_pairs(desc, prefix=None, actual_seq_qlen=None, actual_seq_kvlen=None,
                     has_mask=False) -> int:
    _need_lengths(desc, prefix, actual_seq_qlen, actual_seq_kvlen)
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    out = ctypes.c_int64(0)
    _check(load_library().fa_visible_pairs(ctypes.byref(desc), *a.ptrs(), int(bool(has_mask)),
                                           ctypes.byref(out)))
    return int(out.value)


def fa_tile_class(desc, b, qt, kt, prefix=None, actual_seq_qlen=None, actual_seq_kvlen=None,
                  has_mask=False) -> int:
    _need_lengths(desc, prefix, actual_seq_qlen, actual_seq_kvlen)
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    return int(load_library().fa_tile_class(ctypes.byref(desc), *a.ptrs(), int(bool(has_mask)),
                                             int(b), int(qt), int(kt)))


def fa_plan_items(desc, prefix=None, actual_seq_qlen=None, actual_seq_kvlen=None, num_sms=148):
    """The closed-form work list in the kernel's order on a device with
    num_sms SMs: int32 array [n, 4] of (sequence, head, 256-row block, cost
    key)."""
    import numpy as np
    _need_lengths(desc, prefix, actual_seq_qlen, actual_seq_kvlen)
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    n = ctypes.c_int64(0)
    lib = load_library()
    st = lib.fa_plan_items(ctypes.byref(desc), *a.ptrs(), int(num_sms), 0, None, ctypes.byref(n))
    if n.value == 0:
        _check(st)
        return np.zeros((0, 4), dtype=np.int32)
    out = np.zeros((n.value, 4), dtype=np.int32)
    _check(lib.fa_plan_items(ctypes.byref(desc), *a.ptrs(), int(num_sms), n.value,
                             out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), ctypes.byref(n)))
    return out


def fa_plan_stats(desc, prefix=None, actual_seq_qlen=None, actual_seq_kvlen=None,
                  has_mask=False):
    """(work items, EMPTY, PARTIAL, FULL) of the scheduler for one call."""
    _need_lengths(desc, prefix, actual_seq_qlen, actual_seq_kvlen)
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    out = (ctypes.c_int64 * 4)()
    _check(load_library().fa_plan_stats(ctypes.byref(desc), *a.ptrs(), int(bool(has_mask)), out))
    return tuple(int(x) for x in out)


def fa_create(desc) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load_library().fa_create(ctypes.byref(desc), ctypes.byref(h)))
    return h


def fa_destroy(h):
    _check(load_library().fa_destroy(h))


def fa_sync_status(h) -> int:
    """Raw status of the handle's last call (0 = OK)."""
    return int(load_library().fa_sync_status(h))


def _ptr(t):
    return None if t is None else t.data_ptr()


def fa_fwd(h, q, k, v, o, lse, atten_mask=None, prefix=None, actual_seq_qlen=None,
           actual_seq_kvlen=None, stream=None):
    """Enqueue one forward on `stream` (torch.cuda.Stream, raw handle int, or
    None = torch's current stream). Tensors must be CUDA tensors."""
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    _check(load_library().fa_fwd(h, _ptr(q), _ptr(k), _ptr(v), _ptr(atten_mask), *a.ptrs(),
                                 _ptr(o), _ptr(lse), _stream_int(stream, q.device)))


def fa_fwd_alibi(h, q, k, v, slopes, o, lse, prefix=None, actual_seq_qlen=None,
                 actual_seq_kvlen=None, stream=None):
    """fa_fwd for a handle with an ALiBi variant; slopes: fp32 CUDA tensor [N]."""
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    _check(load_library().fa_fwd_alibi(h, _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), *a.ptrs(),
                                       _ptr(o), _ptr(lse),
                                       _stream_int(stream, q.device)))


def _relbias(table, bucket_of):
    """(fa_relbias_t, the int32 array it points into) of a table [num_buckets,
    N] and a bucket map of 2 * reach + 1 entries."""
    m = np.asarray(bucket_of)
    if m.dtype != np.int32:  # a cast would cut fractions off and wrap large numbers
        if m.size and not (m.min() >= 0 and m.max() < 2 ** 31 and (m == np.floor(m)).all()):
            raise ValueError("the bucket map must hold whole numbers in [0, num_buckets)")
    m = np.ascontiguousarray(m, dtype=np.int32)
    if m.ndim != 1 or m.size < 3 or m.size % 2 == 0:
        raise ValueError("the bucket map must have 2 * reach + 1 entries, reach >= 1")
    b = fa_relbias_t(table.data_ptr(), m.__array_interface__["data"][0], table.shape[0],
                     m.size // 2)
    return b, m


def relative_buckets(num_buckets, max_distance, bidirectional=True):
    """Bucket map int32 [2 * max_distance + 1] of the usual logarithmic
    buckets: entry rel + max_distance is the bucket of the distance rel = key
    - query. Two-sided maps give each side half of the buckets (rel > 0 the
    upper half); one-sided maps put every rel > 0 into bucket 0. Half of a
    side's buckets hold one distance each, the others grow with the logarithm
    of the distance up to max_distance (a boundary within 1e-9 of a whole
    number counts as that number)."""
    side = num_buckets // 2 if bidirectional else num_buckets
    single = side // 2
    if single < 1 or max_distance <= single:
        raise ValueError("need two buckets a side and max_distance above its single distances")
    rel = np.arange(-max_distance, max_distance + 1)
    d = np.abs(rel) if bidirectional else np.maximum(-rel, 0)
    grow = np.log(np.maximum(d, single) / single) / np.log(max_distance / single)
    far = single + np.floor(grow * (side - single) + 1e-9).astype(np.int64)
    bucket = np.where(d < single, d, np.minimum(far, side - 1))
    if bidirectional:
        bucket = bucket + side * (rel > 0)
    return bucket.astype(np.int32)


def fa_fwd_relbias(h, q, k, v, table, bucket_of, o, lse, prefix=None, actual_seq_qlen=None,
                   actual_seq_kvlen=None, stream=None):
    """fa_fwd with a learned relative position bias; table: fp32 CUDA tensor
    [num_buckets, N], bucket_of: host int32 [2 * reach + 1]."""
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    b, keep = _relbias(table, bucket_of)
    _check(load_library().fa_fwd_relbias(h, _ptr(q), _ptr(k), _ptr(v), ctypes.byref(b), *a.ptrs(),
                                         _ptr(o), _ptr(lse),
                                         _stream_int(stream, q.device)))


def fa_bwd(h, q, k, v, o, lse, d_o, dq, dk, dv, atten_mask=None, d_lse=None, prefix=None,
           actual_seq_qlen=None, actual_seq_kvlen=None, stream=None):
    """Enqueue one backward (see include/fa.h). Tensors must be CUDA tensors."""
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    _check(load_library().fa_bwd(h, _ptr(q), _ptr(k), _ptr(v), _ptr(atten_mask), _ptr(o),
                                 _ptr(lse), _ptr(d_o), _ptr(d_lse), *a.ptrs(), _ptr(dq), _ptr(dk),
                                 _ptr(dv), _stream_int(stream, q.device)))


def fa_bwd_alibi(h, q, k, v, slopes, o, lse, d_o, dq, dk, dv, d_lse=None, prefix=None,
                 actual_seq_qlen=None, actual_seq_kvlen=None, stream=None):
    """fa_bwd for a handle with an ALiBi variant; slopes: fp32 CUDA tensor [N]."""
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    _check(load_library().fa_bwd_alibi(h, _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(o),
                                       _ptr(lse), _ptr(d_o), _ptr(d_lse), *a.ptrs(), _ptr(dq),
                                       _ptr(dk), _ptr(dv),
                                       _stream_int(stream, q.device)))


def fa_bwd_relbias(h, q, k, v, table, bucket_of, o, lse, d_o, dq, dk, dv, dtable, d_lse=None,
                   prefix=None, actual_seq_qlen=None, actual_seq_kvlen=None, stream=None):
    """fa_bwd after fa_fwd_relbias; dtable: fp32 CUDA tensor [num_buckets, N]."""
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    b, keep = _relbias(table, bucket_of)
    _check(load_library().fa_bwd_relbias(h, _ptr(q), _ptr(k), _ptr(v), ctypes.byref(b), _ptr(o),
                                         _ptr(lse), _ptr(d_o), _ptr(d_lse), *a.ptrs(), _ptr(dq),
                                         _ptr(dk), _ptr(dv), _ptr(dtable),
                                         _stream_int(stream, q.device)))


def _raw_stream(index):
    """Torch's current stream on CUDA device `index`, as an integer."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # a tenth of the public call's time
    return raw(index) if raw else torch.cuda.current_stream(index).cuda_stream


def _stream_int(stream, device):
    import torch
    if type(stream) is int:
        return stream
    if stream is None:
        return _raw_stream(device.index)
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def occupancy_shapes(desc):
    """Shapes of fa_mask_occupancy's outputs: (tile classes, ranges)."""
    planes = {1: 1, 2: int(desc.B), 3: int(desc.B) * int(desc.N)}[int(desc.mask_kind)]
    n_qt = (int(desc.Sq) + 127) // 128
    n_kt = (int(desc.Skv) + 127) // 128
    return (planes, n_qt, n_kt), (planes, n_qt, 4)


def fa_mask_occupancy(desc, atten_mask, tile_class=None, ranges=None, stream=None):
    """The dense-mask pre-pass alone (see include/fa.h): returns the uint8
    tile classes [P, ceil(Sq/128), ceil(Skv/128)] and the int32 ranges
    [P, ceil(Sq/128), 4] as CUDA tensors (allocated unless given)."""
    import torch
    cshape, rshape = occupancy_shapes(desc)
    dev = atten_mask.device
    if tile_class is None:
        tile_class = torch.empty(cshape, dtype=torch.uint8, device=dev)
    if ranges is None:
        ranges = torch.empty(rshape, dtype=torch.int32, device=dev)
    _check(load_library().fa_mask_occupancy(ctypes.byref(desc), _ptr(atten_mask),
                                            _ptr(tile_class), _ptr(ranges),
                                            ctypes.c_void_p(_stream_int(stream, dev))))
    return tile_class, ranges


def fa_fwd_with_ranges(h, q, k, v, o, lse, atten_mask, ranges, stream=None):
    """fa_fwd for a dense-mask handle with the pre-pass's ranges supplied."""
    _check(load_library().fa_fwd_with_ranges(h, _ptr(q), _ptr(k), _ptr(v), _ptr(atten_mask),
                                             _ptr(ranges), _ptr(o), _ptr(lse),
                                             _stream_int(stream, q.device)))


def fa_fwd_paged(h, q, k_cache, v_cache, block_table, o, lse, actual_seq_qlen,
                 actual_seq_kvlen, prefix=None, stream=None):
    """Forward of a TND handle reading K/V from paged caches
    [num_blocks, block_size, N, D] through block_table [B, max_blocks] (int32)."""
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    num_blocks, block_size = int(k_cache.shape[0]), int(k_cache.shape[1])
    max_blocks = int(block_table.shape[1])
    _check(load_library().fa_fwd_paged(h, _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(block_table), num_blocks, block_size, max_blocks,
                                       *a.ptrs(), _ptr(o), _ptr(lse),
                                       _stream_int(stream, q.device)))


def fa_fwd_noalloc(desc, q, k, v, o, lse, atten_mask=None, prefix=None, actual_seq_qlen=None,
                   actual_seq_kvlen=None, stream=None):
    """The allocation-free forward: no handle, the work list lives in the
    library's fixed device array (see include/fa.h). Same arguments as
    fa_fwd plus the descriptor."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    _need_lengths(desc, prefix, actual_seq_qlen, actual_seq_kvlen)
    a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
    _check(load_library().fa_fwd_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(atten_mask), *a.ptrs(), _ptr(o), _ptr(lse),
                                         ctypes.c_void_p(int(stream))))


def fa_noalloc_sync_status(stream=None, raise_on_error=True):
    """Wait for `stream` and read the error word of the allocation-free
    path's fixed array (see include/fa.h); returns the status code, or
    raises FaError for a non-OK status when raise_on_error."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    lib = load_library()
    st = lib.fa_noalloc_sync_status(ctypes.c_void_p(int(stream)))
    if raise_on_error:
        _check(st)
    return st


def fa_split_queries(desc, actual_seq_qlen, actual_seq_kvlen, n_parts, part, cuts=None):
    """Part `part` of the query split of a TND mode-2/3 job (see include/fa.h).

    Returns a dict with the part's descriptor, its query token range
    [q_begin, q_end) and key range [kv_begin, kv_end) in the unsplit tensors,
    and its cumulative length arrays.
    """
    _need_lengths(desc, None, actual_seq_qlen, actual_seq_kvlen)
    a = _Arrays(None, actual_seq_qlen, actual_seq_kvlen)
    c = None if cuts is None else np.ascontiguousarray(cuts, dtype=np.int64)
    out = fa_split_part_t()
    oq = np.zeros(int(desc.B), dtype=np.int64)
    ok = np.zeros(int(desc.B), dtype=np.int64)
    _, pq, pk = a.ptrs()
    _check(load_library().fa_split_queries(
        ctypes.byref(desc), pq, pk, int(n_parts), _Arrays._p(c), int(part), ctypes.byref(out),
        _Arrays._p(oq), _Arrays._p(ok)))
    nb = int(out.desc.B)
    return {"desc": out.desc, "q_begin": int(out.q_begin), "q_end": int(out.q_end),
            "kv_begin": int(out.kv_begin), "kv_end": int(out.kv_end),
            "actual_seq_qlen": oq[:nb].tolist(), "actual_seq_kvlen": ok[:nb].tolist()}


# ---------------------------------------------------------------- helper class

class MaskedAttention:
    """A handle for one problem shape: ``o, lse = attn(q, k, v, ...)``."""

    def __init__(self, layout, B, N, Sq, Skv, D, sparse_mode=0, pre_tokens=0, next_tokens=0,
                 scale=None, mask_kind=None, alibi=None):
        self.layout = layout
        self.desc = make_desc(layout, B, N, Sq, Skv, D, sparse_mode, pre_tokens, next_tokens,
                              scale, mask_kind, alibi)
        self.handle = fa_create(self.desc)
        # What the calls compare and pass, worked out once.
        self._lib = load_library()
        (self._oshape, self._lshape), self._kshape = self.out_shapes(), self.kv_shape()
        self._takes_lengths = self.desc.sparse_mode in (5, 6) or self.desc.layout == FA_TND
        self._room = {s: math.prod(s) for s in (self._oshape, self._lshape, self._kshape)}

    def out_shapes(self):
        d = self.desc
        if self.layout == "BNSD":
            return (d.B, d.N, d.Sq, d.D), (d.B, d.N, d.Sq)
        if self.layout == "BSND":
            return (d.B, d.Sq, d.N, d.D), (d.B, d.N, d.Sq)
        return (d.Sq, d.N, d.D), (d.N, d.Sq)

    def __call__(self, q, k, v, atten_mask=None, prefix=None, actual_seq_qlen=None,
                 actual_seq_kvlen=None, out=None, lse=None, stream=None, ranges=None,
                 slopes=None, rel_bias=None, rel_buckets=None):
        import torch
        if self._takes_lengths:
            _need_lengths(self.desc, prefix, actual_seq_qlen, actual_seq_kvlen)
        if rel_bias is not None:
            return self._relbias_forward(q, k, v, rel_bias, rel_buckets, atten_mask, ranges,
                                         slopes, prefix, actual_seq_qlen, actual_seq_kvlen, out,
                                         lse, stream)
        self._no_mask_beside(slopes, atten_mask, ranges)
        oshape, lshape = self._oshape, self._lshape
        if out is None:
            out = torch.empty(oshape, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(lshape, dtype=torch.float32, device=q.device)
        dev, kshape, bf16, room = q.device, self._kshape, torch.bfloat16, self._need_room
        if not q.is_cuda:
            raise ValueError("q must be a contiguous bf16 CUDA tensor")
        room("q", q, oshape, bf16, dev)
        room("k", k, kshape, bf16, dev)
        room("v", v, kshape, bf16, dev)
        room("out", out, oshape, bf16, dev)
        room("lse", lse, lshape, torch.float32, dev)
        if atten_mask is not None:
            if atten_mask.dtype not in (torch.uint8, torch.bool) or not atten_mask.is_contiguous():
                raise ValueError("atten_mask must be a contiguous uint8/bool tensor")
            if self._mask_shape() is not None:
                room("atten_mask", atten_mask, self._mask_shape(), atten_mask.dtype, dev)
        if slopes is not None:
            room("slopes", slopes, (self.desc.N,), torch.float32, dev)
            fa_fwd_alibi(self.handle, q, k, v, slopes, out, lse, prefix, actual_seq_qlen,
                         actual_seq_kvlen, stream)
        elif ranges is not None:
            if self._mask_shape() is not None:
                room("ranges", ranges, occupancy_shapes(self.desc)[1], torch.int32, dev)
            fa_fwd_with_ranges(self.handle, q, k, v, out, lse, atten_mask, ranges, stream)
        else:
            fa_fwd(self.handle, q, k, v, out, lse, atten_mask, prefix, actual_seq_qlen,
                   actual_seq_kvlen, stream)
        return out, lse

    def kv_shape(self):
        d = self.desc
        if self.layout == "BNSD":
            return (d.B, d.N, d.Skv, d.D)
        if self.layout == "BSND":
            return (d.B, d.Skv, d.N, d.D)
        return (d.Skv, d.N, d.D)

    def _mask_shape(self):
        d = self.desc
        return {FA_MASK_SS: (d.Sq, d.Skv), FA_MASK_B1SS: (d.B, 1, d.Sq, d.Skv),
                FA_MASK_BNSS: (d.B, d.N, d.Sq, d.Skv)}.get(d.mask_kind)

    def _need_room(self, name, t, shape, dtype, device):
        """t must be contiguous, of this dtype and on `device`, with the elements of
        `shape` (or more, such as a buffer for longer calls): the library reads
        and writes that many."""
        if (t.dtype is dtype and t.device == device and t.is_contiguous()
                and (t.shape == shape or t.numel() >= (self._room.get(shape) or math.prod(shape)))):
            return
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {tuple(shape)} "
                         f"on {device}")

    @staticmethod
    def _need(name, t, shape, dtype, device):
        """t must be a contiguous tensor of this shape and dtype on `device`."""
        try:
            if (t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda
                    and t.is_contiguous()):
                return
        except AttributeError:
            pass
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape "
                         f"{tuple(shape)} on {device}")

    def _no_mask_beside(self, slopes, atten_mask, ranges=None):
        """An ALiBi call reads no attenMask: one that sparse mode 0 would read is
        refused (the other modes a handle with slopes can have ignore it)."""
        if slopes is None:
            return
        if ranges is not None or (atten_mask is not None and self.desc.sparse_mode <= 1):
            raise ValueError("slopes go with neither ranges nor, in sparse mode 0, an atten_mask")

    def _need_bias(self, device, rel_bias, rel_buckets):
        import torch
        if rel_buckets is None:
            raise ValueError("rel_bias needs rel_buckets, its bucket map")
        if not isinstance(rel_bias, torch.Tensor) or rel_bias.dim() != 2:
            raise ValueError("rel_bias must be a tensor [num_buckets, N]")
        self._need("rel_bias", rel_bias, (rel_bias.shape[0], self.desc.N), torch.float32, device)

    @staticmethod
    def _on(stream, device, inputs, body):
        """body(raw stream) with the tensors' device current, and `stream`
        (None: torch's current one) current too, so that what is allocated
        belongs to it; tensors of other streams are kept from reuse until this
        stream has read them."""
        import torch
        if stream is None and torch.cuda.current_device() == device.index:
            return body(_raw_stream(device.index))
        with torch.cuda.device(device):
            here = torch.cuda.current_stream(device)
            if stream is None:
                stream = here
            elif not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            with torch.cuda.stream(stream):
                result = body(stream.cuda_stream)
            if stream != here:
                for t in inputs:
                    if t is not None:
                        t.record_stream(stream)
            return result

    def _relbias_forward(self, q, k, v, rel_bias, rel_buckets, atten_mask, ranges, slopes, prefix,
                         actual_seq_qlen, actual_seq_kvlen, out, lse, stream):
        import torch
        if atten_mask is not None or ranges is not None or slopes is not None:
            raise ValueError("rel_bias goes with neither atten_mask, ranges nor slopes")
        bf16, f32, dev, need = torch.bfloat16, torch.float32, q.device, self._need
        oshape, kshape, lshape = self._oshape, self._kshape, self._lshape
        need("q", q, oshape, bf16, dev)
        need("k", k, kshape, bf16, dev)
        need("v", v, kshape, bf16, dev)
        if out is not None:
            need("out", out, oshape, bf16, dev)
        if lse is not None:
            need("lse", lse, lshape, f32, dev)
        self._need_bias(dev, rel_bias, rel_buckets)

        def body(s):
            o = torch.empty_like(q) if out is None else out
            l = torch.empty(lshape, dtype=f32, device=dev) if lse is None else lse
            a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
            b, keep = _relbias(rel_bias, rel_buckets)
            _check(self._lib.fa_fwd_relbias(
                self.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(b), *a.ptrs(),
                o.data_ptr(), l.data_ptr(), s))
            return o, l

        return self._on(stream, dev, (q, k, v, rel_bias, out, lse), body)

    def backward(self, d_o, q, k, v, o, lse, atten_mask=None, prefix=None, actual_seq_qlen=None,
                 actual_seq_kvlen=None, d_lse=None, slopes=None, rel_bias=None, rel_buckets=None,
                 dq=None, dk=None, dv=None, d_rel_bias=None, stream=None):
        """Gradients of ``o, lse = attn(q, k, v, ...)`` called with the same
        arguments: (dq, dk, dv), and d_rel_bias with a learned bias (see
        fa_bwd in include/fa.h). d_o, d_lse: the gradients of o and lse (d_lse
        None: 0)."""
        import torch
        if self._takes_lengths:
            _need_lengths(self.desc, prefix, actual_seq_qlen, actual_seq_kvlen)
        self._no_mask_beside(slopes, atten_mask)
        bf16, f32, dev, need = torch.bfloat16, torch.float32, q.device, self._need
        oshape, kshape, lshape = self._oshape, self._kshape, self._lshape
        need("q", q, oshape, bf16, dev)
        need("o", o, oshape, bf16, dev)
        need("d_o", d_o, oshape, bf16, dev)
        need("k", k, kshape, bf16, dev)
        need("v", v, kshape, bf16, dev)
        need("lse", lse, lshape, f32, dev)
        for name, t, shape, dtype in (("dq", dq, oshape, bf16), ("dk", dk, kshape, bf16),
                                      ("dv", dv, kshape, bf16), ("d_lse", d_lse, lshape, f32)):
            if t is not None:
                need(name, t, shape, dtype, dev)
        if slopes is not None:
            need("slopes", slopes, (self.desc.N,), f32, dev)
        if atten_mask is not None and self._mask_shape() is not None:
            kind = torch.bool if getattr(atten_mask, "dtype", None) is torch.bool else torch.uint8
            need("atten_mask", atten_mask, self._mask_shape(), kind, dev)
        if rel_bias is not None:
            if atten_mask is not None or slopes is not None:
                raise ValueError("rel_bias goes with neither atten_mask nor slopes")
            self._need_bias(dev, rel_bias, rel_buckets)
            if d_rel_bias is not None:
                need("d_rel_bias", d_rel_bias, rel_bias.shape, f32, dev)

        def body(s):
            gq = torch.empty_like(q) if dq is None else dq
            gk = torch.empty_like(k) if dk is None else dk
            gv = torch.empty_like(v) if dv is None else dv
            a = _Arrays(prefix, actual_seq_qlen, actual_seq_kvlen)
            operands = (self.handle, q.data_ptr(), k.data_ptr(), v.data_ptr())
            rest = (o.data_ptr(), lse.data_ptr(), d_o.data_ptr(), _ptr(d_lse), *a.ptrs(),
                    gq.data_ptr(), gk.data_ptr(), gv.data_ptr())
            if rel_bias is not None:
                gt = torch.empty_like(rel_bias) if d_rel_bias is None else d_rel_bias
                b, keep = _relbias(rel_bias, rel_buckets)
                _check(self._lib.fa_bwd_relbias(*operands, ctypes.byref(b), *rest, gt.data_ptr(), s))
                return gq, gk, gv, gt
            if slopes is not None:
                _check(self._lib.fa_bwd_alibi(*operands, slopes.data_ptr(), *rest, s))
            else:
                _check(self._lib.fa_bwd(*operands, _ptr(atten_mask), *rest, s))
            return gq, gk, gv

        return self._on(stream, dev, (d_o, q, k, v, o, lse, atten_mask, d_lse, slopes, rel_bias, dq,
                                      dk, dv, d_rel_bias), body)

    def paged(self, q, k_cache, v_cache, block_table, actual_seq_qlen, actual_seq_kvlen,
              prefix=None, out=None, lse=None, stream=None):
        """O, lse of a TND handle with K/V in paged caches (see fa_fwd_paged)."""
        import torch
        if self._takes_lengths:
            _need_lengths(self.desc, prefix, actual_seq_qlen, actual_seq_kvlen)
        oshape, lshape = self.out_shapes()
        if out is None:
            out = torch.empty(oshape, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(lshape, dtype=torch.float32, device=q.device)
        if not q.is_cuda:
            raise ValueError("q must be a contiguous bf16 CUDA tensor")
        for name, t, shape, dtype in (
                ("q", q, oshape, torch.bfloat16), ("k_cache", k_cache, (), torch.bfloat16),
                ("v_cache", v_cache, (), torch.bfloat16), ("out", out, oshape, torch.bfloat16),
                ("lse", lse, lshape, torch.float32), ("block_table", block_table, (), torch.int32)):
            self._need_room(name, t, shape, dtype, q.device)
        d = self.desc
        if (k_cache.dim() != 4 or tuple(v_cache.shape) != tuple(k_cache.shape)
                or k_cache.shape[2] != d.N or k_cache.shape[3] != d.D):
            raise ValueError("k_cache and v_cache must both be [num_blocks, block_size, N, D]")
        if block_table.dim() != 2 or block_table.shape[0] != d.B:
            raise ValueError("block_table must be [B, max_blocks]")
        if tuple(q.shape) != tuple(oshape):
            raise ValueError(f"q must be {tuple(oshape)}")
        fa_fwd_paged(self.handle, q, k_cache, v_cache, block_table, out, lse, actual_seq_qlen,
                     actual_seq_kvlen, prefix, stream)
        return out, lse

    def occupancy(self, atten_mask, stream=None):
        """Run the dense-mask pre-pass on its own: (tile classes, ranges);
        pass the ranges back as ``attn(..., ranges=ranges)`` to skip it."""
        if self._mask_shape() is not None:
            if not atten_mask.is_cuda or atten_mask.element_size() != 1:
                raise ValueError("atten_mask must be a contiguous uint8/bool CUDA tensor")
            self._need_room("atten_mask", atten_mask, self._mask_shape(), atten_mask.dtype,
                            atten_mask.device)
        return fa_mask_occupancy(self.desc, atten_mask, stream=stream)

    def sync_status(self):
        st = fa_sync_status(self.handle)
        if st != 0:
            raise FaError(st, fa_last_error())

    def close(self):
        if self.handle is not None:
            fa_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

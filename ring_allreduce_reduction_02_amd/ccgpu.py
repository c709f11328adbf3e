"""ctypes binding of libcc.so (include/cc.h), same names as the C ABI.

Argument marshalling only: every step of every collective runs in the HIP
kernels of libcc.so.  PyTorch provides the device memory and the stream.

Rank-strided buffers are 2-D tensors ``t[N, L]`` whose rows are contiguous
(``t.stride(1) == 1``) and whose row stride may exceed L (padding between
ranks), e.g. ``torch.empty(N, L + pad, device="cuda")[:, :L]``.  Rank r's
buffer is row r.

If the library has not been built this module raises on first use: there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
# the library built next to this file; CC_LIB_PATH names another build of it
# (the sanitizer run's)
LIB_PATH = os.environ.get("CC_LIB_PATH") or os.path.join(HERE, "libcc.so")

CC_OK, CC_ERR_INVALID_ARG, CC_ERR_UNSUPPORTED, CC_ERR_NO_DEVICE, CC_ERR_HIP = range(5)
DTYPES = {"int32": 0, "f32": 1, "bf16": 2}
OPS = {"sum": 0, "max": 1, "prod": 2}
ALGOS = {"ring": 0, "hd": 1, "butterfly": 2, "tree": 3, "double_tree": 4, "ring_2port": 5}
COLLS = {"all_reduce": 0, "reduce_scatter": 1, "all_gather": 2, "broadcast": 3, "all_to_all": 4}
ESIZE = {"int32": 4, "f32": 4, "bf16": 2}
MAX_RANKS = 64


class RankBuf(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("rank_stride_bytes", ctypes.c_size_t)]


class Config(ctypes.Structure):
    _fields_ = [("algo", ctypes.c_int), ("fuse_depth", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("blocks_per_cu", ctypes.c_int), ("grid_sync", ctypes.c_int)]


class PlanOp(ctypes.Structure):
    _fields_ = [("step", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("dst", ctypes.c_int32),
                ("in1", ctypes.c_int32), ("in2", ctypes.c_int32), ("lo", ctypes.c_uint64), ("len", ctypes.c_uint64)]


PLAN_FLAGS = {"local_send": 1, "in1": 2, "in1_send": 4, "in2": 8, "in2_send": 16, "final": 32, "both": 64, "copy": 128}


class CCError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


_STATUS = {0: "CC_OK", 1: "CC_ERR_INVALID_ARG", 2: "CC_ERR_UNSUPPORTED", 3: "CC_ERR_NO_DEVICE", 4: "CC_ERR_HIP"}
_lib: Optional[ctypes.CDLL] = None

EXPORTS = {
    "cc_all_reduce": [RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                      ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_reduce_noalloc": [RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                              ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_reduce_scatter": [RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                          ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_gather": [RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                      ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_broadcast": [RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                     ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_to_all": [RankBuf, RankBuf, ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t, ctypes.c_int,
                      ctypes.c_int, ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_reduce_buckets": [RankBuf, RankBuf, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t),
                              ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(Config),
                              ctypes.c_void_p],
    "cc_bucket_plan": [ctypes.POINTER(ctypes.c_size_t), ctypes.c_int, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_size_t,
                       ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t),
                       ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_int)],
    "cc_workspace_size": [ctypes.c_int, ctypes.POINTER(Config), ctypes.c_int, ctypes.c_size_t, ctypes.c_int,
                          ctypes.POINTER(ctypes.c_size_t)],
    "cc_get_traffic": [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_size_t, ctypes.c_int,
                       ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_int)],
    "cc_chunk_bounds": [ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "cc_all_reduce_plan": [ctypes.c_int, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(PlanOp), ctypes.c_size_t,
                           ctypes.POINTER(ctypes.c_size_t)],
    "cc_all_reduce_hierarchical": [RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                   ctypes.POINTER(ctypes.c_int), ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_hierarchical_workspace_size": [ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(Config),
                                       ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "cc_hierarchical_traffic": [ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.c_size_t, ctypes.c_int,
                                ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_int)],
    "cc_hierarchical_plan": [ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.c_size_t, ctypes.POINTER(PlanOp),
                             ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)],
    "cc_moe_capacity": [ctypes.c_int, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                        ctypes.POINTER(ctypes.c_size_t)],
    "cc_moe_dispatch_padded": [RankBuf, RankBuf, ctypes.POINTER(ctypes.c_size_t), ctypes.c_int, ctypes.c_size_t,
                               ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_moe_combine_padded": [RankBuf, RankBuf, ctypes.POINTER(ctypes.c_size_t), ctypes.c_int, ctypes.c_size_t,
                              ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_to_all_hierarchical": [RankBuf, RankBuf, ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t, ctypes.c_int,
                                   ctypes.c_int, ctypes.c_int, ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_to_all_hierarchical_workspace_size": [ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t, ctypes.c_int,
                                                  ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "cc_all_to_all_traffic": [ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                              ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_uint64),
                              ctypes.POINTER(ctypes.c_uint64)],
    "cc_all_to_all_step_bytes": [ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                                 ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)],
    "cc_all_to_all_plan": [ctypes.c_int, RankBuf, RankBuf, ctypes.POINTER(ctypes.c_size_t), ctypes.c_int,
                           ctypes.c_size_t, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                           ctypes.POINTER(Config), ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)],
    "cc_quantize_ef": [RankBuf, RankBuf, RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                       ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_reduce_dequant": [RankBuf, RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                              ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_reduce_int8_ef": [RankBuf, RankBuf, RankBuf, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                              ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_int8_ef_workspace_size": [ctypes.POINTER(Config), ctypes.c_int, ctypes.c_size_t, ctypes.c_int,
                                  ctypes.POINTER(ctypes.c_size_t)],
    "cc_int8_message_bytes": [ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)],
    "cc_embedding": [RankBuf] * 3 + [ctypes.c_size_t] * 3 + [ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                                             ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_embedding_grad": [RankBuf] * 3 + [ctypes.c_size_t] * 3 + [ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                                                  ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_all_reduce_embedding_grad": [RankBuf] * 3 + [ctypes.c_size_t] * 3 + [ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                                                             ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_embedding_grad_workspace_size": [ctypes.c_int, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_size_t,
                                         ctypes.POINTER(ctypes.c_size_t)],
    "cc_moe_route": [RankBuf] * 5 + [ctypes.c_size_t] + [ctypes.c_int] * 5 + [ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_moe_route_workspace_size": [ctypes.c_int, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                                    ctypes.POINTER(ctypes.c_size_t)],
    "cc_moe_route_grad": [RankBuf] * 4 + [ctypes.c_size_t] + [ctypes.c_int] * 5 + [ctypes.POINTER(Config),
                                                                                  ctypes.c_void_p],
    "cc_moe_ffn": [RankBuf] * 5 + [ctypes.POINTER(ctypes.c_size_t), ctypes.c_int] + [ctypes.c_size_t] * 3
                  + [ctypes.c_int] * 3 + [ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_moe_ffn_grad": [RankBuf] * 8 + [ctypes.POINTER(ctypes.c_size_t), ctypes.c_int] + [ctypes.c_size_t] * 3
                       + [ctypes.c_int] * 3 + [ctypes.POINTER(Config), ctypes.c_void_p],
    "cc_moe_ffn_workspace_size": [ctypes.POINTER(ctypes.c_size_t), ctypes.c_int] + [ctypes.c_size_t] * 3
                                 + [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_size_t)],
    "cc_status_string": [ctypes.c_int],
    "cc_last_error": [],
    "cc_version": [],
}


def load() -> ctypes.CDLL:
    """Load libcc.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m ring_allreduce_reduction_02_amd.build_lib`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, args in EXPORTS.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_char_p if name in ("cc_status_string", "cc_last_error", "cc_version") else ctypes.c_int
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != CC_OK:
        raise CCError(status, load().cc_last_error().decode())


def dtype_name(t) -> str:
    import torch
    m = {torch.int32: "int32", torch.float32: "f32", torch.bfloat16: "bf16"}
    if t.dtype not in m:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return m[t.dtype]


def rankbuf(t) -> RankBuf:
    """A [N, L] tensor with contiguous rows -> cc_rankbuf_t."""
    if t.dim() != 2:
        raise ValueError("rank-strided buffers are 2-D tensors [nranks, elements]")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("each rank's row must be contiguous")
    if not t.is_cuda:
        raise ValueError("buffers must be device tensors")
    return RankBuf(t.data_ptr(), t.stride(0) * t.element_size())


def config(algo: str = "ring", fuse_depth: int = 0, workspace=None, blocks_per_cu: int = 0,
           grid_sync: bool = False) -> Config:
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return Config(ALGOS[algo], int(fuse_depth), ws_ptr, ws_bytes, int(blocks_per_cu), int(bool(grid_sync)))


def _stream(stream) -> ctypes.c_void_p:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def workspace_size(coll: str, nranks: int, count: int, dtype: str, algo: str = "ring",
                   fuse_depth: int = 0, grid_sync: bool = False) -> int:
    out = ctypes.c_size_t(0)
    cfg = Config(ALGOS[algo], int(fuse_depth), None, 0, 0, int(bool(grid_sync)))
    _check(load().cc_workspace_size(COLLS[coll], ctypes.byref(cfg), nranks, count, DTYPES[dtype],
                                    ctypes.byref(out)))
    return out.value


def make_workspace(coll: str, nranks: int, count: int, dtype: str, algo: str = "ring",
                   fuse_depth: int = 0, device="cuda", grid_sync: bool = False):
    """Allocate (with torch) the workspace a schedule needs, or None."""
    import torch
    n = workspace_size(coll, nranks, count, dtype, algo, fuse_depth, grid_sync)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def get_traffic(coll: str, nranks: int, count: int, dtype: str, algo: str = "ring"):
    """(max bytes any rank sends, steps) of the simulated network."""
    b = ctypes.c_uint64(0)
    s = ctypes.c_int(0)
    _check(load().cc_get_traffic(COLLS[coll], ALGOS[algo], nranks, count, DTYPES[dtype], ctypes.byref(b),
                                 ctypes.byref(s)))
    return b.value, s.value


def chunk_bounds(count: int, nranks: int):
    arr = (ctypes.c_size_t * (nranks + 1))()
    _check(load().cc_chunk_bounds(count, nranks, arr))
    return list(arr)


def all_reduce(send, recv=None, op: str = "sum", algo: str = "ring", fuse_depth: int = 0,
               workspace=None, stream=None, blocks_per_cu: int = 0, grid_sync: bool = False) -> None:
    """recv[r] = (+)_j send[j] for every rank r; send/recv are [N, M].
    grid_sync: the stepwise ring's passes in one launch, each pass waiting for the previous one."""
    recv = send if recv is None else recv
    N, M = send.shape
    if tuple(recv.shape) != (N, M) or recv.dtype != send.dtype:
        raise ValueError("recv must match send")
    cfg = config(algo, fuse_depth, workspace, blocks_per_cu, grid_sync)
    _check(load().cc_all_reduce(rankbuf(send), rankbuf(recv), M, DTYPES[dtype_name(send)], OPS[op], N,
                                ctypes.byref(cfg), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 16 << 20


def all_reduce_noalloc(send, recv=None, op: str = "sum", algo: str = "ring", fuse_depth: int = 0,
                       stream=None, blocks_per_cu: int = 0, grid_sync: bool = False) -> None:
    """all_reduce with the schedule's staging in the library's fixed scratch
    (cc_all_reduce_noalloc): no workspace argument, nothing allocated."""
    recv = send if recv is None else recv
    N, M = send.shape
    if tuple(recv.shape) != (N, M) or recv.dtype != send.dtype:
        raise ValueError("recv must match send")
    cfg = config(algo, fuse_depth, None, blocks_per_cu, grid_sync)
    _check(load().cc_all_reduce_noalloc(rankbuf(send), rankbuf(recv), M, DTYPES[dtype_name(send)], OPS[op], N,
                                        ctypes.byref(cfg), _stream(stream)))


def all_reduce_plan(algo: str, nranks: int, count: int):
    """The descriptor steps a stepwise AllReduce runs (cc_all_reduce_plan), as
    a list of dicts with keys step, flags, dst, in1, in2, lo, len."""
    L = load()
    n = ctypes.c_size_t(0)
    _check(L.cc_all_reduce_plan(ALGOS[algo], nranks, count, None, 0, ctypes.byref(n)))
    recs = (PlanOp * max(n.value, 1))()
    _check(L.cc_all_reduce_plan(ALGOS[algo], nranks, count, recs, n.value, ctypes.byref(n)))
    return [{f: getattr(recs[i], f) for f, _ in PlanOp._fields_} for i in range(n.value)]


def _dims(dims: Sequence[int]):
    return len(dims), (ctypes.c_int * max(len(dims), 1))(*[int(p) for p in dims])


def hierarchical_workspace_size(dims: Sequence[int], count: int, dtype: str, fuse_depth: int = 0) -> int:
    nd, arr = _dims(dims)
    out = ctypes.c_size_t(0)
    cfg = Config(ALGOS["ring"], int(fuse_depth), None, 0, 0, 0)
    _check(load().cc_hierarchical_workspace_size(nd, arr, ctypes.byref(cfg), count, DTYPES[dtype],
                                                 ctypes.byref(out)))
    return out.value


def make_hierarchical_workspace(dims: Sequence[int], count: int, dtype: str, fuse_depth: int = 0, device="cuda"):
    """Allocate (with torch) the workspace of a hierarchical AllReduce, or None."""
    import torch
    n = hierarchical_workspace_size(dims, count, dtype, fuse_depth)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def all_reduce_hierarchical(send, recv=None, dims: Sequence[int] = (), op: str = "sum", fuse_depth: int = 0,
                            workspace=None, stream=None, blocks_per_cu: int = 0) -> None:
    """Hierarchical AllReduce over the rank grid dims (level 0 innermost,
    prod(dims) = N); send/recv are [N, M]."""
    recv = send if recv is None else recv
    N, M = send.shape
    if tuple(recv.shape) != (N, M) or recv.dtype != send.dtype:
        raise ValueError("recv must match send")
    nd, arr = _dims(dims)
    cfg = config("ring", fuse_depth, workspace, blocks_per_cu)
    _check(load().cc_all_reduce_hierarchical(rankbuf(send), rankbuf(recv), M, DTYPES[dtype_name(send)], OPS[op],
                                             nd, arr, ctypes.byref(cfg), _stream(stream)))


def hierarchical_traffic(dims: Sequence[int], count: int, dtype: str):
    """Per level: (largest bytes any rank sends inside its group, ring steps)."""
    nd, arr = _dims(dims)
    b = (ctypes.c_uint64 * max(nd, 1))()
    st = (ctypes.c_int * max(nd, 1))()
    _check(load().cc_hierarchical_traffic(nd, arr, count, DTYPES[dtype], b, st))
    return [(b[i], st[i]) for i in range(nd)]


def hierarchical_plan(dims: Sequence[int], count: int):
    """The descriptor steps of the stepwise hierarchical AllReduce, as
    all_reduce_plan returns them."""
    L = load()
    nd, arr = _dims(dims)
    n = ctypes.c_size_t(0)
    _check(L.cc_hierarchical_plan(nd, arr, count, None, 0, ctypes.byref(n)))
    recs = (PlanOp * max(n.value, 1))()
    _check(L.cc_hierarchical_plan(nd, arr, count, recs, n.value, ctypes.byref(n)))
    return [{f: getattr(recs[i], f) for f, _ in PlanOp._fields_} for i in range(n.value)]


def bucket_plan(sizes: Sequence[int], elem_bytes: int, cap_bytes: int, align_elems: int = 1):
    """Host bucket plan (cc_bucket_plan): returns (bucket_of, tensor_offset,
    bucket_offset, bucket_count) as Python lists."""
    n = len(sizes)
    cap = max(n, 1)
    sz = (ctypes.c_size_t * cap)(*[int(v) for v in sizes])
    bof = (ctypes.c_int * cap)()
    toff = (ctypes.c_size_t * cap)()
    boff = (ctypes.c_size_t * cap)()
    bcnt = (ctypes.c_size_t * cap)()
    nb = ctypes.c_int(0)
    _check(load().cc_bucket_plan(sz, n, elem_bytes, cap_bytes, align_elems, bof, toff, boff, bcnt, ctypes.byref(nb)))
    k = nb.value
    return list(bof)[:n], list(toff)[:n], list(boff)[:k], list(bcnt)[:k]


def all_reduce_buckets(send, recv, offsets: Sequence[int], counts: Sequence[int], op: str = "sum",
                       algo: str = "ring", fuse_depth: int = 0, workspace=None, stream=None,
                       blocks_per_cu: int = 0) -> None:
    """Independent AllReduces over element ranges [offsets[b], +counts[b]) of
    the [N, L] rank buffers (cc_all_reduce_buckets)."""
    recv = send if recv is None else recv
    N = send.shape[0]
    if tuple(recv.shape) != tuple(send.shape) or recv.dtype != send.dtype:
        raise ValueError("recv must match send")
    nb = len(offsets)
    if len(counts) != nb:
        raise ValueError("offsets and counts differ in length")
    off = (ctypes.c_size_t * max(nb, 1))(*[int(v) for v in offsets])
    cnt = (ctypes.c_size_t * max(nb, 1))(*[int(v) for v in counts])
    cfg = config(algo, fuse_depth, workspace, blocks_per_cu)
    _check(load().cc_all_reduce_buckets(rankbuf(send), rankbuf(recv), off, cnt, nb, DTYPES[dtype_name(send)],
                                        OPS[op], N, ctypes.byref(cfg), _stream(stream)))


def reduce_scatter(send, recv, op: str = "sum", algo: str = "ring", fuse_depth: int = 0,
                   workspace=None, stream=None, blocks_per_cu: int = 0) -> None:
    """send [N, N*S] -> recv [N, S]: rank r gets the reduced chunk r."""
    N, S = recv.shape
    if tuple(send.shape) != (N, N * S) or recv.dtype != send.dtype:
        raise ValueError("send must be [N, N*S] for recv [N, S]")
    cfg = config(algo, fuse_depth, workspace, blocks_per_cu)
    _check(load().cc_reduce_scatter(rankbuf(send), rankbuf(recv), S, DTYPES[dtype_name(send)], OPS[op], N,
                                    ctypes.byref(cfg), _stream(stream)))


def all_gather(send, recv, algo: str = "ring", fuse_depth: int = 0, stream=None, blocks_per_cu: int = 0) -> None:
    """send [N, S] -> recv [N, N*S]: slot r of every rank holds rank r's send."""
    N, S = send.shape
    if tuple(recv.shape) != (N, N * S) or recv.dtype != send.dtype:
        raise ValueError("recv must be [N, N*S] for send [N, S]")
    cfg = config(algo, fuse_depth, None, blocks_per_cu)
    _check(load().cc_all_gather(rankbuf(send), rankbuf(recv), S, DTYPES[dtype_name(send)], N,
                                ctypes.byref(cfg), _stream(stream)))


def broadcast(send, recv=None, root: int = 0, algo: str = "ring", fuse_depth: int = 0, stream=None,
              blocks_per_cu: int = 0) -> None:
    """recv[r] = send[root] for every r; send/recv are [N, M]."""
    recv = send if recv is None else recv
    N, M = recv.shape
    if tuple(send.shape) != (N, M) or recv.dtype != send.dtype:
        raise ValueError("recv must match send")
    cfg = config(algo, fuse_depth, None, blocks_per_cu)
    _check(load().cc_broadcast(rankbuf(send), rankbuf(recv), M, DTYPES[dtype_name(send)], root, N,
                               ctypes.byref(cfg), _stream(stream)))


def all_to_all(send, recv, counts: Sequence[Sequence[int]], elem_per_row: int = 1, fuse_depth: int = 0,
               stream=None, blocks_per_cu: int = 0) -> None:
    """Blocked transpose with per-(source, destination) row counts."""
    N = send.shape[0]
    flat = [int(v) for row in counts for v in row]
    if len(flat) != N * N or recv.shape[0] != N:
        raise ValueError("counts must be N x N")
    arr = (ctypes.c_size_t * (N * N))(*flat)
    cfg = config("ring", fuse_depth, None, blocks_per_cu)
    _check(load().cc_all_to_all(rankbuf(send), rankbuf(recv), arr, elem_per_row, DTYPES[dtype_name(send)], N,
                                ctypes.byref(cfg), _stream(stream)))


def _sizes(rows: Sequence[Sequence[int]], n: int, m: int, what: str):
    flat = [int(v) for row in rows for v in row]
    if len(flat) != n * m or any(len(row) != m for row in rows):
        raise ValueError(f"{what} must be {n} x {m}")
    return (ctypes.c_size_t * max(len(flat), 1))(*flat)


def moe_capacity(nranks: int, tokens: int, topk: int, nexperts: int, factor_num: int, factor_den: int) -> int:
    """ceil(nranks * tokens * topk / nexperts * factor_num / factor_den)."""
    out = ctypes.c_size_t(0)
    _check(load().cc_moe_capacity(nranks, tokens, topk, nexperts, factor_num, factor_den, ctypes.byref(out)))
    return out.value


def moe_dispatch_padded(send, recv, counts: Sequence[Sequence[int]], capacity: int, elem_per_row: int = 1,
                        fuse_depth: int = 0, stream=None, blocks_per_cu: int = 0) -> None:
    """Token side send [N, rows] -> expert side recv [N, E*capacity*elem_per_row];
    counts is N x E (rows per source and expert)."""
    N, E = send.shape[0], len(counts[0]) if len(counts) else 0
    arr = _sizes(counts, N, E, "counts")
    cfg = config("ring", fuse_depth, None, blocks_per_cu)
    _check(load().cc_moe_dispatch_padded(rankbuf(send), rankbuf(recv), arr, E, capacity, elem_per_row,
                                         DTYPES[dtype_name(send)], N, ctypes.byref(cfg), _stream(stream)))


def moe_combine_padded(send, recv, counts: Sequence[Sequence[int]], capacity: int, elem_per_row: int = 1,
                       fuse_depth: int = 0, stream=None, blocks_per_cu: int = 0) -> None:
    """Expert side send -> token side recv, the transpose of moe_dispatch_padded."""
    N, E = send.shape[0], len(counts[0]) if len(counts) else 0
    arr = _sizes(counts, N, E, "counts")
    cfg = config("ring", fuse_depth, None, blocks_per_cu)
    _check(load().cc_moe_combine_padded(rankbuf(send), rankbuf(recv), arr, E, capacity, elem_per_row,
                                        DTYPES[dtype_name(send)], N, ctypes.byref(cfg), _stream(stream)))


def all_to_all_hierarchical_workspace_size(counts: Sequence[Sequence[int]], elem_per_row: int, dtype: str,
                                           local_size: int) -> int:
    N = len(counts)
    out = ctypes.c_size_t(0)
    _check(load().cc_all_to_all_hierarchical_workspace_size(_sizes(counts, N, N, "counts"), elem_per_row,
                                                            DTYPES[dtype], N, local_size, ctypes.byref(out)))
    return out.value


def make_all_to_all_hierarchical_workspace(counts, elem_per_row: int, dtype: str, local_size: int, device="cuda"):
    import torch
    n = all_to_all_hierarchical_workspace_size(counts, elem_per_row, dtype, local_size)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def all_to_all_hierarchical(send, recv, counts: Sequence[Sequence[int]], local_size: int, elem_per_row: int = 1,
                            workspace=None, stream=None, blocks_per_cu: int = 0) -> None:
    """AllToAll(v) as aggregate / exchange / distribute over nodes of
    local_size ranks; same result as all_to_all."""
    N = send.shape[0]
    arr = _sizes(counts, N, N, "counts")
    cfg = config("ring", 0, workspace, blocks_per_cu)
    _check(load().cc_all_to_all_hierarchical(rankbuf(send), rankbuf(recv), arr, elem_per_row,
                                             DTYPES[dtype_name(send)], N, local_size, ctypes.byref(cfg),
                                             _stream(stream)))


def all_to_all_traffic(counts: Sequence[Sequence[int]], elem_per_row: int, dtype: str, local_size: int):
    """[flat, aggregate, exchange, distribute]: (transfers, total bytes, most bytes one rank sends)."""
    N = len(counts)
    f = (ctypes.c_int * 4)()
    t = (ctypes.c_uint64 * 4)()
    m = (ctypes.c_uint64 * 4)()
    _check(load().cc_all_to_all_traffic(_sizes(counts, N, N, "counts"), elem_per_row, DTYPES[dtype], N, local_size,
                                        f, t, m))
    return [(f[k], t[k], m[k]) for k in range(4)]


def all_to_all_step_bytes(counts: Sequence[Sequence[int]], elem_per_row: int, dtype: str):
    """Pairwise steps k = 0..N-1: (max block bytes, total block bytes)."""
    N = len(counts)
    mx = (ctypes.c_uint64 * N)()
    tt = (ctypes.c_uint64 * N)()
    _check(load().cc_all_to_all_step_bytes(_sizes(counts, N, N, "counts"), elem_per_row, DTYPES[dtype], N, mx, tt))
    return list(mx), list(tt)


class CopyOp(ctypes.Structure):
    _fields_ = [("step", ctypes.c_uint32), ("reserved", ctypes.c_uint32), ("src", ctypes.c_uint64),
                ("dst", ctypes.c_uint64), ("bytes", ctypes.c_uint64)]


A2A_KINDS = {"moe_dispatch": 1, "moe_combine": 2, "hierarchical": 3}


def all_to_all_plan(kind: str, send: RankBuf, recv: RankBuf, counts: Sequence[Sequence[int]], nranks: int,
                    elem_per_row: int, dtype: str, nexperts: int = 0, capacity: int = 0, local_size: int = 1,
                    fuse_depth: int = 0, workspace: int = 0, workspace_bytes: int = 0):
    """The copies an AllToAll variant performs (cc_all_to_all_plan), for rank
    buffers given as raw RankBuf addresses: list of (step, src, dst, bytes),
    src 0 meaning a zero fill."""
    L = load()
    flat = [int(v) for row in counts for v in row]
    arr = (ctypes.c_size_t * max(len(flat), 1))(*flat)
    cfg = Config(ALGOS["ring"], int(fuse_depth), workspace or None, workspace_bytes, 0, 0)
    n = ctypes.c_size_t(0)
    args = (A2A_KINDS[kind], send, recv, arr, nexperts, capacity, elem_per_row, DTYPES[dtype], nranks, local_size,
            ctypes.byref(cfg))
    _check(L.cc_all_to_all_plan(*args, None, 0, ctypes.byref(n)))
    recs = (CopyOp * max(n.value, 1))()
    _check(L.cc_all_to_all_plan(*args, ctypes.cast(recs, ctypes.c_void_p), n.value, ctypes.byref(n)))
    return [(recs[i].step, recs[i].src, recs[i].dst, recs[i].bytes) for i in range(n.value)]


QUANT_BLOCK = 128


def quantize_ef(grad, err, q, scales, stream=None, blocks_per_cu: int = 0) -> None:
    """grad [N, M] (f32/bf16), err [N, M] f32 (updated), q [N, M] int8,
    scales [N, ceil(M/128)] f32: the compression step with error feedback."""
    N, M = grad.shape
    cfg = config("ring", 0, None, blocks_per_cu)
    _check(load().cc_quantize_ef(rankbuf(grad), rankbuf(err), rankbuf(q), rankbuf(scales), M,
                                 DTYPES[dtype_name(grad)], N, ctypes.byref(cfg), _stream(stream)))


def all_reduce_dequant(q, scales, recv, stream=None, blocks_per_cu: int = 0) -> None:
    """recv [N, M] (f32/bf16) = ring-order sum of every rank's dequantized message."""
    N, M = recv.shape
    cfg = config("ring", 0, None, blocks_per_cu)
    _check(load().cc_all_reduce_dequant(rankbuf(q), rankbuf(scales), rankbuf(recv), M,
                                        DTYPES[dtype_name(recv)], N, ctypes.byref(cfg), _stream(stream)))


def int8_ef_workspace_size(nranks: int, count: int, dtype: str, fuse_depth: int) -> int:
    out = ctypes.c_size_t(0)
    cfg = Config(ALGOS["ring"], int(fuse_depth), None, 0, 0, 0)
    _check(load().cc_int8_ef_workspace_size(ctypes.byref(cfg), nranks, count, DTYPES[dtype], ctypes.byref(out)))
    return out.value


def all_reduce_int8_ef(grad, err, recv=None, fuse_depth: int = 0, workspace=None, stream=None,
                       blocks_per_cu: int = 0) -> None:
    """Compression with error feedback and the AllReduce of the compressed
    contributions (recv defaults to grad: in place)."""
    recv = grad if recv is None else recv
    N, M = grad.shape
    cfg = config("ring", fuse_depth, workspace, blocks_per_cu)
    _check(load().cc_all_reduce_int8_ef(rankbuf(grad), rankbuf(err), rankbuf(recv), M, DTYPES[dtype_name(grad)], N,
                                        ctypes.byref(cfg), _stream(stream)))


def int8_message_bytes(count: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().cc_int8_message_bytes(count, ctypes.byref(out)))
    return out.value


# ---- the model's side of the exchanges: embedding, routing, expert feed-forward

ACTS = {"silu": 0, "gelu": 1}


class _Call:
    """The operands, stream and config of one call.  Everything belongs to the
    current device, which is asked for once; a call with no workspace and no
    occupancy cap passes no config (NULL is that config)."""

    def __init__(self, stream, workspace=None, blocks_per_cu: int = 0):
        import torch
        dev = self.dev = torch.cuda.current_device() if torch.cuda.is_initialized() else None
        if stream is None:
            self.stream = torch.cuda.current_stream().cuda_stream if dev is not None else None
        else:
            if stream.device_index != dev:
                raise ValueError("the stream belongs to another device")
            self.stream = stream.cuda_stream
        self.cfg = None
        if workspace is not None:
            if not workspace.is_cuda or workspace.get_device() != dev:
                raise ValueError("the workspace must be on the current device")
            if not workspace.is_contiguous():
                raise ValueError("the workspace must be contiguous")
        if workspace is not None or blocks_per_cu:
            self.cfg = ctypes.byref(config("ring", 0, workspace, blocks_per_cu))

    def operand(self, t, name: str, n: int, length: int, dtype=None) -> RankBuf:
        """A rank-strided operand [n, length] on the current device."""
        shape = t.shape
        if len(shape) != 2 or shape[0] != n or shape[1] != length:
            raise ValueError(f"{name} must be [{n}, {length}], got {list(shape)}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name}: buffers must be device tensors")
        if t.get_device() != self.dev:
            raise ValueError(f"{name} is on {t.device}, the current device is {self.dev}")
        stride = t.stride()
        if length > 1 and stride[1] != 1:
            raise ValueError(f"{name}: each rank's row must be contiguous")
        return RankBuf(t.data_ptr(), stride[0] * t.element_size())


def _rows(t, width: int, name: str) -> int:
    if t.dim() != 2 or width < 1 or t.shape[1] % width:
        raise ValueError(f"{name} must be [nranks, rows * {width}]")
    return t.shape[1] // width


def embedding(table, ids, out, width: int, scale: float = 1.0, stream=None, blocks_per_cu: int = 0) -> None:
    """out [N, T * width] = scale * the rows ids [N, T] (int32) of table
    [N, V * width]; zero rows for ids outside [0, V).  A table expanded over
    the ranks (stride 0) is one table that all ranks read."""
    import torch
    (N, T), V, c = ids.shape, _rows(table, width, "table"), _Call(stream, None, blocks_per_cu)
    _check(load().cc_embedding(c.operand(table, "table", N, V * width), c.operand(ids, "ids", N, T, torch.int32),
                               c.operand(out, "out", N, T * width, table.dtype), V, T, width, scale,
                               DTYPES[dtype_name(table)], N, c.cfg, c.stream))


def embedding_grad_workspace_size(nranks: int, vocab: int, tokens: int, width: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().cc_embedding_grad_workspace_size(nranks, vocab, tokens, width, ctypes.byref(out)))
    return out.value


def make_embedding_grad_workspace(nranks: int, vocab: int, tokens: int, width: int, dtype: str = "f32", device="cuda"):
    """Allocate (with torch) the workspace of either embedding gradient, or None."""
    import torch
    n = embedding_grad_workspace_size(nranks, vocab, tokens, width)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _embedding_grad(call: str, grad, ids, dtable, width, scale, workspace, stream, blocks_per_cu) -> None:
    import torch
    (N, T), V, c = ids.shape, _rows(dtable, width, "dtable"), _Call(stream, workspace, blocks_per_cu)
    _check(getattr(load(), call)(c.operand(grad, "grad", N, T * width), c.operand(ids, "ids", N, T, torch.int32),
                                 c.operand(dtable, "dtable", N, V * width, grad.dtype), V, T, width, scale,
                                 DTYPES[dtype_name(grad)], N, c.cfg, c.stream))


def embedding_grad(grad, ids, dtable, width: int, scale: float = 1.0, workspace=None, stream=None,
                   blocks_per_cu: int = 0) -> None:
    """dtable [N, V * width]: each rank's gradient of its table from grad
    [N, T * width] at ids [N, T]; every row is written."""
    _embedding_grad("cc_embedding_grad", grad, ids, dtable, width, scale, workspace, stream, blocks_per_cu)


def all_reduce_embedding_grad(grad, ids, dtable, width: int, scale: float = 1.0, workspace=None, stream=None,
                              blocks_per_cu: int = 0) -> None:
    """dtable [N, V * width]: the gradient summed over all ranks, on every rank."""
    _embedding_grad("cc_all_reduce_embedding_grad", grad, ids, dtable, width, scale, workspace, stream, blocks_per_cu)


def moe_route_workspace_size(nranks: int, tokens: int, nexperts: int, topk: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().cc_moe_route_workspace_size(nranks, tokens, nexperts, topk, ctypes.byref(out)))
    return out.value


def make_moe_route_workspace(nranks: int, tokens: int, nexperts: int, topk: int, device="cuda"):
    """Allocate (with torch) the workspace of moe_route, or None."""
    import torch
    n = moe_route_workspace_size(nranks, tokens, nexperts, topk)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def moe_route(logits, experts, weights, order, counts, topk: int, normalize: bool = False, workspace=None,
              stream=None) -> None:
    """logits [N, T * E] -> experts (int32) and weights (f32) [N, T * topk],
    order (int32) [N, T * topk], counts (int32) [N, E]."""
    import torch
    N, E = counts.shape
    T, c = _rows(logits, E, "logits"), _Call(stream, workspace)
    _check(load().cc_moe_route(c.operand(logits, "logits", N, T * E),
                               c.operand(experts, "experts", N, T * topk, torch.int32),
                               c.operand(weights, "weights", N, T * topk, torch.float32),
                               c.operand(order, "order", N, T * topk, torch.int32),
                               c.operand(counts, "counts", N, E, torch.int32), T, E, topk, 1 if normalize else 0,
                               DTYPES[dtype_name(logits)], N, c.cfg, c.stream))


def moe_route_grad(logits, experts, dweights, dlogits, topk: int, normalize: bool = False, stream=None) -> None:
    """dlogits [N, T * E] from dweights (f32) [N, T * topk] at the experts moe_route chose."""
    import torch
    N, T = experts.shape[0], _rows(experts, topk, "experts")
    E, c = _experts_of(logits, N, T), _Call(stream)
    _check(load().cc_moe_route_grad(c.operand(logits, "logits", N, T * E),
                                    c.operand(experts, "experts", N, T * topk, torch.int32),
                                    c.operand(dweights, "dweights", N, T * topk, torch.float32),
                                    c.operand(dlogits, "dlogits", N, T * E, logits.dtype), T, E, topk,
                                    1 if normalize else 0, DTYPES[dtype_name(logits)], N, c.cfg, c.stream))


def _experts_of(logits, n: int, tokens: int) -> int:
    if logits.dim() != 2 or (tokens and logits.shape[1] % tokens):
        raise ValueError(f"logits must be [{n}, {tokens} * nexperts]")
    return logits.shape[1] // tokens if tokens else 1


def moe_ffn_workspace_size(counts: Sequence[Sequence[int]], capacity: int, width: int, hidden: int, dtype: str,
                           grad: bool = False) -> int:
    N, E = len(counts), len(counts[0]) if len(counts) else 0
    out = ctypes.c_size_t(0)
    _check(load().cc_moe_ffn_workspace_size(_sizes(counts, N, E, "counts"), E, capacity, width, hidden, DTYPES[dtype],
                                            N, int(bool(grad)), ctypes.byref(out)))
    return out.value


def make_moe_ffn_workspace(counts, capacity: int, width: int, hidden: int, dtype: str, grad: bool = False,
                           device="cuda"):
    """Allocate (with torch) the workspace of moe_ffn (or moe_ffn_grad)."""
    import torch
    n = moe_ffn_workspace_size(counts, capacity, width, hidden, dtype, grad)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _ffn_operands(x, w_in, w_out, counts, capacity, width):
    """(N, E, hidden, expert-side length, counts array) of a feed-forward call."""
    N, E = x.shape[0], len(counts[0]) if len(counts) else 0
    arr = _sizes(counts, N, E, "counts")
    if E < N or E % N:
        raise ValueError(f"{E} experts are not a multiple of {N} ranks")
    hidden = _rows(w_out, E // N * width, "w_out")
    return N, E, hidden, E * capacity * width, arr


def moe_ffn(x, w_in, w_out, y, counts: Sequence[Sequence[int]], capacity: int, width: int, pre=None, act: str = "silu",
            workspace=None, stream=None) -> None:
    """Gated feed-forward of the experts on the expert side of
    moe_dispatch_padded: x, y [N, E * capacity * width], w_in
    [N, E/N * 2 * hidden * width], w_out [N, E/N * width * hidden], counts
    N x E; pre [N, E * capacity * 2 * hidden] keeps the pre-activations."""
    N, E, hidden, side, arr = _ffn_operands(x, w_in, w_out, counts, capacity, width)
    per, dt, c = E // N, x.dtype, _Call(stream, workspace)
    args = (c.operand(x, "x", N, side), c.operand(w_in, "w_in", N, per * 2 * hidden * width, dt),
            c.operand(w_out, "w_out", N, per * width * hidden, dt),
            RankBuf(None, 0) if pre is None else c.operand(pre, "pre", N, E * capacity * 2 * hidden, dt),
            c.operand(y, "y", N, side, dt))
    _check(load().cc_moe_ffn(*args, arr, E, capacity, width, hidden, ACTS[act], DTYPES[dtype_name(x)], N, c.cfg,
                             c.stream))


def moe_ffn_grad(x, w_in, w_out, pre, dy, dx, dw_in, dw_out, counts: Sequence[Sequence[int]], capacity: int,
                 width: int, act: str = "silu", workspace=None, stream=None) -> None:
    """The gradients of moe_ffn from dy, with pre as moe_ffn kept it."""
    N, E, hidden, side, arr = _ffn_operands(x, w_in, w_out, counts, capacity, width)
    per, dt, c = E // N, x.dtype, _Call(stream, workspace)
    wi, wo = per * 2 * hidden * width, per * width * hidden
    args = (c.operand(x, "x", N, side), c.operand(w_in, "w_in", N, wi, dt), c.operand(w_out, "w_out", N, wo, dt),
            c.operand(pre, "pre", N, E * capacity * 2 * hidden, dt), c.operand(dy, "dy", N, side, dt),
            c.operand(dx, "dx", N, side, dt), c.operand(dw_in, "dw_in", N, wi, dt),
            c.operand(dw_out, "dw_out", N, wo, dt))
    _check(load().cc_moe_ffn_grad(*args, arr, E, capacity, width, hidden, ACTS[act], DTYPES[dtype_name(x)], N, c.cfg,
                                  c.stream))


def raw(fn: str, *args):
    """Call a C-ABI function with raw ctypes arguments; returns the status."""
    return getattr(load(), fn)(*args)


def grid_sync_timed_out(workspace) -> bool:
    """After a grid_sync call has completed: whether a barrier wait gave up
    (the uint32 at byte offset 4 of the workspace)."""
    import torch
    return int(workspace[4:8].view(torch.int32).item()) != 0

"""ctypes marshalling for libar.so (see ``include/ar.h`` for the contract).

Buffers may be given as torch tensors (their ``data_ptr()`` is used) or as
integer device addresses.  ``stream`` may be a ``torch.cuda.Stream``, an
integer ``hipStream_t`` handle, or None for torch's current stream on the
current device (the NULL stream when torch is absent).
"""
from __future__ import annotations

import ctypes
import os
import weakref
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libar.so")

AR_MAX_RANKS = 128
DTYPES = {"f32": 0, "bf16": 1, "f16": 2, "i32": 3}
OPS = {"sum": 0, "prod": 1, "min": 2, "max": 3, "avg": 4}
SCHEDS = {"auto": 0, "ring": 1, "tree": 2, "fused": 3, "split": 4, "dtree": 5}
COLLS = {"allreduce": 0, "reduce_scatter": 1, "all_gather": 2}
ACCS = {"storage": 0, "fp32": 1}
AVGS = {"prescale": 0, "split": 1}
_SCHED_NAMES = {v: k for k, v in SCHEDS.items()}
_STATUS = {0: "AR_OK", 1: "AR_ERR_INVALID_ARG", 2: "AR_ERR_UNSUPPORTED", 3: "AR_ERR_ALIGNMENT", 4: "AR_ERR_HIP"}

if not os.path.exists(_LIB_PATH):
    raise ImportError("libar.so is not built (expected at %s); build it with `python reduce_scatter_amd/build.py` "
                      "or __graft_entry__.build()" % _LIB_PATH)

# One HIP runtime per process: PyTorch-ROCm ships its own libamdhip64 (same
# SONAME as the system one).  Loading torch first makes libar.so bind to the
# runtime torch already loaded; loading libar.so first would pull in the
# system copy and torch would then load a second, separate runtime, whose
# devices, streams and allocations are not the ones libar.so sees.
try:
    import torch  # noqa: F401
except ImportError:
    pass

_lib = ctypes.CDLL(_LIB_PATH)


class _Numerics(ctypes.Structure):
    _fields_ = [("acc", ctypes.c_int), ("avg", ctypes.c_int)]


class _PlanStruct(ctypes.Structure):
    _fields_ = [("chosen", ctypes.c_int), ("legal_mask", ctypes.c_uint), ("steps", ctypes.c_int * 6),
                ("bytes", ctypes.c_double * 6), ("predicted_us", ctypes.c_double * 6)]


_vpp = ctypes.POINTER(ctypes.c_void_p)
_lib.ar_allreduce.argtypes = [_vpp, _vpp, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                              ctypes.c_void_p]
_lib.ar_reduce_scatter.argtypes = _lib.ar_allreduce.argtypes
_lib.ar_allreduce_ex.argtypes = [_vpp, _vpp, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                 ctypes.c_void_p, ctypes.c_void_p]
_lib.ar_reduce_scatter_ex.argtypes = _lib.ar_allreduce_ex.argtypes
_lib.ar_all_gather.argtypes = [_vpp, _vpp, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                               ctypes.c_void_p]
_lib.ar_plan.argtypes = [ctypes.c_int, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                         ctypes.POINTER(_PlanStruct)]
_lib.ar_tree_parent.argtypes = [ctypes.c_int, ctypes.c_int]
_lib.ar_tree_parent.restype = ctypes.c_int
_lib.ar_dtree_parent.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int]
_lib.ar_dtree_parent.restype = ctypes.c_int
_lib.ar_status_string.argtypes = [ctypes.c_int]
_lib.ar_status_string.restype = ctypes.c_char_p
for _f in (_lib.ar_allreduce, _lib.ar_reduce_scatter, _lib.ar_all_gather, _lib.ar_plan, _lib.ar_allreduce_ex,
           _lib.ar_reduce_scatter_ex):
    _f.restype = ctypes.c_int


def library_path() -> str:
    return _LIB_PATH


class ArError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        self.name = _STATUS.get(status, str(status))
        super().__init__(ar_status_string(status))


@dataclass
class Plan:
    chosen: str
    legal: list
    steps: dict
    bytes: dict
    predicted_us: dict


def ar_status_string(status: int) -> str:
    return _lib.ar_status_string(int(status)).decode()


def _code(table, value, what):
    if isinstance(value, str):
        if value not in table:
            raise ValueError("unknown %s %r (expected one of %s)" % (what, value, sorted(table)))
        return table[value]
    return int(value)


def _dtype_code(dtype):
    try:
        import torch
        tmap = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16", torch.int32: "i32"}
        if dtype in tmap:
            dtype = tmap[dtype]
    except ImportError:
        pass
    return _code(DTYPES, dtype, "dtype")


def _ptr(b):
    if b is None:
        return None
    if isinstance(b, int):
        return b
    return int(b.data_ptr())


class PointerTable:
    """A host array of device pointers built once and reusable across calls
    (a list of tensors costs a ``data_ptr()`` call per buffer on every call;
    at 128 ranks that host time is comparable to a small collective).  The
    table keeps references to the tensors it was built from."""

    def __init__(self, bufs):
        self.n = len(bufs)
        self._checked = None             # the last shape these buffers were checked against
        self.array = (ctypes.c_void_p * max(1, self.n))(*[_ptr(b) for b in bufs])
        self._bufs = list(bufs)          # tensors stay alive (and their memory owned) while the table exists

    def __len__(self):
        return self.n


def pointers(bufs) -> PointerTable:
    """Build a reusable pointer table for ``bufs`` (tensors or integer addresses)."""
    return PointerTable(bufs)


def _ptr_array(bufs):
    if isinstance(bufs, PointerTable):
        return bufs.array
    return (ctypes.c_void_p * max(1, len(bufs)))(*[_ptr(b) for b in bufs])


def _tables(sendbufs, recvbufs):
    send = _ptr_array(sendbufs)
    return send, (send if recvbufs is sendbufs else _ptr_array(recvbufs))


_gpu_state = []     # [current-stream getter] once known; [None] without torch or a GPU


def _current_stream_getter():
    try:
        import torch
    except ImportError:
        return None
    if not torch.cuda.is_available():
        return None
    raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and dev is not None:
        return lambda: raw(dev())                      # the handle of torch's current stream, without a Stream object
    return lambda: int(torch.cuda.current_stream().cuda_stream)


def _stream(stream):
    if stream is None:
        if not _gpu_state:
            _gpu_state.append(_current_stream_getter())
        get = _gpu_state[0]
        return get() if get is not None else 0
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(status):
    if status != 0:
        raise ArError(status)


def ar_allreduce(sendbufs, recvbufs, count, dtype, op, n=None, sched="auto", stream=None):
    """All-reduce ``count`` elements of each of the n rank buffers (in place when recvbufs is sendbufs)."""
    n = len(sendbufs) if n is None else n
    send, recv = _tables(sendbufs, recvbufs)
    _check(_lib.ar_allreduce(send, recv, count, _dtype_code(dtype),
                             _code(OPS, op, "op"), n, _code(SCHEDS, sched, "schedule"), _stream(stream)))


def ar_reduce_scatter(sendbufs, recvbufs, recvcount, dtype, op, n=None, sched="auto", stream=None):
    """Reduce-scatter: each send buffer holds n*recvcount elements; rank r receives slice r."""
    n = len(sendbufs) if n is None else n
    send, recv = _tables(sendbufs, recvbufs)
    _check(_lib.ar_reduce_scatter(send, recv, recvcount, _dtype_code(dtype),
                                  _code(OPS, op, "op"), n, _code(SCHEDS, sched, "schedule"), _stream(stream)))


def _numerics(acc, avg):
    return ctypes.byref(_Numerics(_code(ACCS, acc, "accumulation"), _code(AVGS, avg, "avg route")))


def ar_allreduce_ex(sendbufs, recvbufs, count, dtype, op, n=None, sched="auto", acc="storage", avg="prescale",
                    stream=None):
    """All-reduce with explicit numerics: ``acc`` "storage" | "fp32" (bf16 / fp16
    partials kept in fp32, fused schedule), ``avg`` "prescale" | "split"."""
    n = len(sendbufs) if n is None else n
    send, recv = _tables(sendbufs, recvbufs)
    _check(_lib.ar_allreduce_ex(send, recv, count, _dtype_code(dtype), _code(OPS, op, "op"), n,
                                _code(SCHEDS, sched, "schedule"), _numerics(acc, avg), _stream(stream)))


def ar_reduce_scatter_ex(sendbufs, recvbufs, recvcount, dtype, op, n=None, sched="auto", acc="storage",
                         avg="prescale", stream=None):
    """Reduce-scatter with explicit numerics (as :func:`ar_allreduce_ex`)."""
    n = len(sendbufs) if n is None else n
    send, recv = _tables(sendbufs, recvbufs)
    _check(_lib.ar_reduce_scatter_ex(send, recv, recvcount, _dtype_code(dtype), _code(OPS, op, "op"), n,
                                     _code(SCHEDS, sched, "schedule"), _numerics(acc, avg), _stream(stream)))


def ar_all_gather(sendbufs, recvbufs, sendcount, dtype, n=None, sched="auto", stream=None):
    """All-gather: each rank receives the n pieces of sendcount elements, in rank order."""
    n = len(sendbufs) if n is None else n
    send, recv = _tables(sendbufs, recvbufs)
    _check(_lib.ar_all_gather(send, recv, sendcount, _dtype_code(dtype), n,
                              _code(SCHEDS, sched, "schedule"), _stream(stream)))


def ar_plan(coll, count, dtype, op, n) -> Plan:
    """The cost model's choice for a call (host only; no GPU needed)."""
    p = _PlanStruct()
    _check(_lib.ar_plan(_code(COLLS, coll, "collective"), count, _dtype_code(dtype), _code(OPS, op, "op"), n,
                        ctypes.byref(p)))
    legal = [name for name, s in SCHEDS.items() if s and (p.legal_mask >> s) & 1]
    return Plan(chosen=_SCHED_NAMES[p.chosen], legal=legal,
                steps={s: p.steps[SCHEDS[s]] for s in legal},
                bytes={s: p.bytes[SCHEDS[s]] for s in legal},
                predicted_us={s: p.predicted_us[SCHEDS[s]] for s in legal})


def ar_tree_parent(n: int, v: int) -> int:
    return int(_lib.ar_tree_parent(n, v))


def ar_dtree_parent(n: int, which: int, v: int) -> int:
    return int(_lib.ar_dtree_parent(n, which, v))


# ---------------------------------------------------------------------------
# M-to-N layout reshard (include/ar_reshard.h)
# ---------------------------------------------------------------------------

REPLICATE = -1
ROUTES = {"auto": 0, "flat": 1, "hier": 2, "fused": 3}
_ROUTE_NAMES = {v: k for k, v in ROUTES.items()}


class _Layout(ctypes.Structure):
    _fields_ = [("ndim", ctypes.c_int), ("shape", ctypes.c_longlong * 3), ("mesh_ndim", ctypes.c_int),
                ("mesh", ctypes.c_int * 2), ("placement", ctypes.c_int * 2), ("base_rank", ctypes.c_int)]


class _Transfer(ctypes.Structure):
    _fields_ = [("src_rank", ctypes.c_int), ("dst_rank", ctypes.c_int), ("leader_rank", ctypes.c_int),
                ("lo", ctypes.c_longlong * 3), ("hi", ctypes.c_longlong * 3), ("bytes", ctypes.c_longlong)]


class _ReshardPlanStruct(ctypes.Structure):
    _fields_ = [("chosen", ctypes.c_int), ("n_transfers", ctypes.c_int), ("n_sources", ctypes.c_int),
                ("n_shards", ctypes.c_int), ("max_replicas", ctypes.c_int), ("unique_bytes", ctypes.c_longlong),
                ("bytes", ctypes.c_double * 4), ("launches", ctypes.c_int * 4), ("predicted_us", ctypes.c_double * 4)]


_lib.ar_reshard_plan.argtypes = [ctypes.POINTER(_Layout), ctypes.POINTER(_Layout), ctypes.c_size_t, ctypes.c_int,
                                 ctypes.POINTER(_ReshardPlanStruct), ctypes.POINTER(_Transfer), ctypes.c_int]
_lib.ar_reshard_plan.restype = ctypes.c_int
_lib.ar_reshard.argtypes = [_vpp, _vpp, ctypes.POINTER(_Layout), ctypes.POINTER(_Layout), ctypes.c_size_t,
                            ctypes.c_int, ctypes.c_void_p]
_lib.ar_reshard.restype = ctypes.c_int


@dataclass(frozen=True)
class Layout:
    """An endpoint layout (S, M, p): global ``shape``, ``mesh`` extents, one
    placement per mesh axis (REPLICATE or the sharded tensor dimension) and
    the mesh's ``base_rank``."""
    shape: tuple
    mesh: tuple
    placements: tuple
    base_rank: int = 0


_lib.ar_layout_shard.argtypes = [ctypes.POINTER(_Layout), ctypes.c_int, ctypes.POINTER(ctypes.c_longlong),
                                 ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(ctypes.c_int)]
_lib.ar_layout_shard.restype = ctypes.c_int


def _layout(L):
    """Any object with ``shape``, ``mesh``, ``placements`` (REPLICATE or the
    sharded tensor dimension per mesh axis) and optionally ``base_rank``."""
    s = _Layout()
    shape, mesh, pl = tuple(L.shape), tuple(L.mesh), tuple(L.placements)
    if not (1 <= len(shape) <= 3 and 1 <= len(mesh) <= 2 and len(pl) == len(mesh)):
        raise ValueError("a layout has 1-3 tensor dimensions and 1-2 mesh axes, one placement per axis")
    s.ndim, s.mesh_ndim = len(shape), len(mesh)
    for d, v in enumerate(shape):
        s.shape[d] = int(v)
    for k in range(len(mesh)):
        s.mesh[k] = int(mesh[k])
        s.placement[k] = int(pl[k])
    s.base_rank = int(getattr(L, "base_rank", 0))
    return s


def ar_layout_shard(layout, slot):
    """([(lo, hi)] per tensor dimension, communicator rank) of mesh slot ``slot``."""
    L = _layout(layout)
    lo, hi, rank = (ctypes.c_longlong * 3)(), (ctypes.c_longlong * 3)(), ctypes.c_int()
    _check(_lib.ar_layout_shard(ctypes.byref(L), slot, lo, hi, ctypes.byref(rank)))
    return [(lo[d], hi[d]) for d in range(L.ndim)], rank.value


def local_shape(layout, slot):
    """Shape of mesh slot ``slot``'s local buffer."""
    return tuple(h - l for l, h in ar_layout_shard(layout, slot)[0])


@dataclass
class ReshardPlan:
    chosen: str
    n_transfers: int
    n_sources: int
    n_shards: int
    max_replicas: int
    unique_bytes: int
    bytes: dict
    launches: dict
    predicted_us: dict
    transfers: list        # (src_rank, dst_rank, leader_rank, [(lo, hi)] per tensor dim, bytes)


def ar_reshard_plan(src, dst, elem_size, domains=1) -> ReshardPlan:
    """The layout-derived schedule and route costs (host only)."""
    ls, ld = _layout(src), _layout(dst)
    out = _ReshardPlanStruct()
    _check(_lib.ar_reshard_plan(ctypes.byref(ls), ctypes.byref(ld), elem_size, domains, ctypes.byref(out), None, 0))
    n = out.n_transfers
    arr = (_Transfer * max(1, n))()
    _check(_lib.ar_reshard_plan(ctypes.byref(ls), ctypes.byref(ld), elem_size, domains, ctypes.byref(out), arr, n))
    nd = ls.ndim
    transfers = [(t.src_rank, t.dst_rank, t.leader_rank, [(t.lo[d], t.hi[d]) for d in range(nd)], t.bytes)
                 for t in arr[:n]]
    names = ("flat", "hier", "fused")
    return ReshardPlan(_ROUTE_NAMES[out.chosen], n, out.n_sources, out.n_shards, out.max_replicas,
                       out.unique_bytes, {k: out.bytes[ROUTES[k]] for k in names},
                       {k: out.launches[ROUTES[k]] for k in names},
                       {k: out.predicted_us[ROUTES[k]] for k in names}, transfers)


def ar_reshard(src_bufs, dst_bufs, src, dst, elem_size, route="auto", stream=None):
    """Reshard from layout ``src`` (buffers ``src_bufs``, one per source mesh
    slot; None allowed for replicas that are not the owner of their shard)
    to layout ``dst`` (``dst_bufs``, one per destination slot)."""
    ls, ld = _layout(src), _layout(dst)
    _check(_lib.ar_reshard(_ptr_array(src_bufs), _ptr_array(dst_bufs), ctypes.byref(ls), ctypes.byref(ld),
                           elem_size, _code(ROUTES, route, "route"), _stream(stream)))


# ---------------------------------------------------------------------------
# Reductions over a vocabulary axis split over the ranks (include/ar_vocab.h)
# ---------------------------------------------------------------------------

class _VocabStruct(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("dtype", ctypes.c_int), ("rows", ctypes.c_longlong),
                ("widths", ctypes.POINTER(ctypes.c_longlong)), ("pitches", ctypes.POINTER(ctypes.c_longlong)),
                ("grad_pitches", ctypes.POINTER(ctypes.c_longlong)), ("temperature", ctypes.c_float)]


_vshape, _vp, _int = ctypes.POINTER(_VocabStruct), ctypes.c_void_p, ctypes.c_int
_lib.ar_vocab_workspace.argtypes = [_vshape, _int, ctypes.POINTER(ctypes.c_size_t)]
_lib.ar_logprobs.argtypes = [_vpp, _vshape, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.ar_logprobs_backward.argtypes = [_vpp, _vpp, _vshape, _vp, _vp, _vp, _vp, _vp]
_lib.ar_logprobs_grad.argtypes = [_vpp, _vpp, _vshape, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.ar_distill.argtypes = [_vpp, _vshape, _vp, _vp, _int, _int, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.ar_distill_backward.argtypes = [_vpp, _vpp, _vshape, _vp, _vp, _int, _int, _vp, _vp, _vp]
_lib.ar_distill_grad.argtypes = [_vpp, _vpp, _vshape, _vp, _vp, _int, _int, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
for _f in (_lib.ar_vocab_workspace, _lib.ar_logprobs, _lib.ar_logprobs_backward, _lib.ar_logprobs_grad,
           _lib.ar_distill, _lib.ar_distill_backward, _lib.ar_distill_grad):
    _f.restype = ctypes.c_int


class VocabShape:
    """Rows of logits whose vocabulary axis lies in n rank buffers: rank r
    holds ``widths[r]`` columns of every row, rows ``pitches[r]`` elements
    apart (default: the widths), gradients ``grad_pitches[r]`` (default: the
    pitches).  Built once and reusable across calls."""

    def __init__(self, rows, widths, dtype, pitches=None, grad_pitches=None, temperature=1.0):
        self.rows, self.widths, self.n = int(rows), [int(w) for w in widths], len(widths)
        for p in (pitches, grad_pitches):
            if p is not None and len(p) != self.n:
                raise ValueError("one pitch per rank")
        self.pitches = self.widths if pitches is None else [int(p) for p in pitches]
        self.grad_pitches = self.pitches if grad_pitches is None else [int(p) for p in grad_pitches]
        self.dtype, self.temperature = _dtype_code(dtype), float(temperature)
        self._arrays = [(ctypes.c_longlong * max(1, self.n))(*a)
                        for a in (self.widths, self.pitches, self.grad_pitches)]
        self._struct = _VocabStruct(self.n, self.dtype, self.rows, *self._arrays, self.temperature)
        self.ref = ctypes.byref(self._struct)


def vocab_widths(vocab, n):
    """Columns of each of n ranks under the shard bounds of ``ar_layout_shard``."""
    return [(r + 1) * vocab // n - r * vocab // n for r in range(n)]


def _at_pitch(b, pitch, rows):
    """Whether a tensor's rows (all its dimensions but the last) are packed elements ``pitch`` apart."""
    if b.dim() == 0 or b.numel() == 0 or (b.dim() != 2 and b.is_contiguous()):
        return True
    outer = [(size, stride) for size, stride in zip(b.shape[:-1], b.stride()[:-1]) if size > 1]
    if b.shape[-1] > 1 and b.stride(-1) != 1:
        return False
    if any(a[1] != c[0] * c[1] for a, c in zip(outer, outer[1:])):
        return False
    return not outer or outer[-1][1] == pitch or rows <= 1


def _on_host(t):
    """Whether a tensor lies where no kernel can reach it (pinned memory can be reached)."""
    return not t.is_cuda and t.numel() > 0 and not t.is_pinned()


def _refuse(host, shape):
    """Refuse tensors in host memory by name, once all else about the arguments is right."""
    if host and shape.rows:
        raise ValueError("%s must be on the GPU, not in host memory" % host[0])


def _logit_table(bufs, shape, host, grads=False):
    """Pointer table of rank buffers; tensors must have the shape's type and hold its rows."""
    if not isinstance(bufs, PointerTable):
        bufs = PointerTable(bufs)
    if bufs._checked != (shape, grads):
        if bufs.n != shape.n:
            raise ValueError("%d rank buffers for %d ranks" % (bufs.n, shape.n))
        for b, w, p in zip(bufs._bufs, shape.widths, shape.grad_pitches if grads else shape.pitches):
            if b is None or isinstance(b, int):
                continue
            if _dtype_code(b.dtype) != shape.dtype:
                raise ValueError("rank buffer of %s does not have the shape's dtype" % b.dtype)
            room = b.untyped_storage().nbytes() // b.element_size() - b.storage_offset()
            if shape.rows and w and room < (shape.rows - 1) * p + w:
                raise ValueError("rank buffer holds %d elements; %d rows of %d at pitch %d need more"
                                 % (room, shape.rows, w, p))
            if not _at_pitch(b, p, shape.rows):
                raise ValueError("rank buffer has strides %s; its pitch is %d" % (tuple(b.stride()), p))
            if _on_host(b):
                host.append("grads" if grads else "logits")
        if not host:
            bufs._checked = (shape, grads)
    return bufs.array


def _vector(t, dtype, numel, what, host):
    """Address of a contiguous tensor argument (integer addresses and None pass through); its name goes into ``host``
    if it is in host memory."""
    if t is None or isinstance(t, int):
        return t
    if str(t.dtype) != dtype or t.numel() < numel or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of at least %d elements" % (what, dtype, numel))
    if _on_host(t):
        host.append(what)
    return t.data_ptr()


def _f32(t, numel, what, host):
    return _vector(t, "torch.float32", numel, what, host)


def _i64(t, numel, what, host):
    return _vector(t, "torch.int64", numel, what, host)


def _workspace(w, host):
    if w is None:
        return None, 0
    if _on_host(w):
        host.append("workspace")
    return w.data_ptr() or None, w.numel() * w.element_size()


def ar_vocab_workspace(shape, top_k=0) -> int:
    """Workspace bytes of the calls below on ``shape`` (host only)."""
    n = ctypes.c_size_t()
    _check(_lib.ar_vocab_workspace(shape.ref, top_k, ctypes.byref(n)))
    return n.value


def ar_logprobs(logits, shape, targets, logprobs, entropy=None, top_k=0, top_logprobs=None, top_ids=None, saved=None,
                workspace=None, stream=None):
    """ln p of each row's target; optionally the entropy, the ``top_k`` most
    likely entries, and the statistics ``ar_logprobs_backward`` needs."""
    r, host = shape.rows, []
    ws, wb = _workspace(workspace, host)
    args = (_logit_table(logits, shape, host), shape.ref, _i64(targets, r, "targets", host),
            _f32(logprobs, r, "logprobs", host), _f32(entropy, r, "entropy", host), top_k,
            _f32(top_logprobs, r * top_k, "top_logprobs", host), _i64(top_ids, r * top_k, "top_ids", host),
            _f32(saved, 4 * r, "saved", host))
    _refuse(host, shape)
    _check(_lib.ar_logprobs(*args, ws, wb, _stream(stream)))


def ar_logprobs_backward(logits, grads, shape, targets, saved, grad_logprobs=None, grad_entropy=None, stream=None):
    """Gradient of the logits from the gradients of the log probabilities and entropies."""
    r, host = shape.rows, []
    args = (_logit_table(logits, shape, host), _logit_table(grads, shape, host, True), shape.ref,
            _i64(targets, r, "targets", host), _f32(saved, 4 * r, "saved", host),
            _f32(grad_logprobs, r, "grad_logprobs", host), _f32(grad_entropy, r, "grad_entropy", host))
    _refuse(host, shape)
    _check(_lib.ar_logprobs_backward(*args, _stream(stream)))


def ar_logprobs_grad(logits, grads, shape, targets, logprobs=None, grad_logprobs=None, grad_entropy=None,
                     entropy=None, saved=None, workspace=None, stream=None):
    """Log probabilities (optionally entropies) and the gradient in one call."""
    r, host = shape.rows, []
    ws, wb = _workspace(workspace, host)
    args = (_logit_table(logits, shape, host), _logit_table(grads, shape, host, True), shape.ref,
            _i64(targets, r, "targets", host), _f32(grad_logprobs, r, "grad_logprobs", host),
            _f32(grad_entropy, r, "grad_entropy", host), _f32(logprobs, r, "logprobs", host),
            _f32(entropy, r, "entropy", host), _f32(saved, 4 * r, "saved", host))
    _refuse(host, shape)
    _check(_lib.ar_logprobs_grad(*args, ws, wb, _stream(stream)))


def _teacher(shape, ids, values, k, host):
    """(k, ids address, values address): k from a two-dimensional list of ids unless given."""
    if k is None:
        if ids is None or isinstance(ids, int) or ids.dim() != 2:
            raise ValueError("k is needed unless teacher_ids is a two-dimensional tensor")
        k = ids.shape[1]
    return k, _i64(ids, shape.rows * k, "teacher_ids", host), _f32(values, shape.rows * k, "teacher_values", host)


def ar_distill(logits, shape, teacher_ids, teacher_values, loss, tail=False, k=None, saved=None, workspace=None,
               stream=None):
    """Divergence of the student's distribution from a teacher's top entries
    (``tail``: log probabilities with the remaining mass compared as well;
    otherwise renormalised logits)."""
    r, host = shape.rows, []
    ws, wb = _workspace(workspace, host)
    k, ids, values = _teacher(shape, teacher_ids, teacher_values, k, host)
    args = (_logit_table(logits, shape, host), shape.ref, ids, values, k, int(bool(tail)), _f32(loss, r, "loss", host),
            _f32(saved, 4 * r, "saved", host))
    _refuse(host, shape)
    _check(_lib.ar_distill(*args, ws, wb, _stream(stream)))


def ar_distill_backward(logits, grads, shape, teacher_ids, teacher_values, saved, tail=False, k=None, grad_loss=None,
                        stream=None):
    """Gradient of the logits from the gradients of the rows' losses (None: ones)."""
    r, host = shape.rows, []
    k, ids, values = _teacher(shape, teacher_ids, teacher_values, k, host)
    args = (_logit_table(logits, shape, host), _logit_table(grads, shape, host, True), shape.ref, ids, values, k,
            int(bool(tail)), _f32(saved, 4 * r, "saved", host), _f32(grad_loss, r, "grad_loss", host))
    _refuse(host, shape)
    _check(_lib.ar_distill_backward(*args, _stream(stream)))


def ar_distill_grad(logits, grads, shape, teacher_ids, teacher_values, loss=None, tail=False, k=None, grad_loss=None,
                    saved=None, workspace=None, stream=None):
    """The rows' losses and the gradient in one call."""
    r, host = shape.rows, []
    ws, wb = _workspace(workspace, host)
    k, ids, values = _teacher(shape, teacher_ids, teacher_values, k, host)
    args = (_logit_table(logits, shape, host), _logit_table(grads, shape, host, True), shape.ref, ids, values, k,
            int(bool(tail)), _f32(grad_loss, r, "grad_loss", host), _f32(loss, r, "loss", host),
            _f32(saved, 4 * r, "saved", host))
    _refuse(host, shape)
    _check(_lib.ar_distill_grad(*args, ws, wb, _stream(stream)))


# ---------------------------------------------------------------------------
# Operators around a step's collectives (include/ar_layer.h)
# ---------------------------------------------------------------------------

class _NormStruct(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
                ("rows", ctypes.c_longlong), ("width", ctypes.c_longlong), ("pitches", ctypes.POINTER(ctypes.c_longlong)),
                ("eps", ctypes.c_float), ("offset", ctypes.c_float), ("group", ctypes.c_int)]


class _EmbedStruct(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("tokens", ctypes.c_longlong), ("width", ctypes.c_longlong),
                ("entries", ctypes.POINTER(ctypes.c_longlong)), ("pitches", ctypes.POINTER(ctypes.c_longlong)),
                ("grad_pitches", ctypes.POINTER(ctypes.c_longlong)), ("scale", ctypes.c_float)]


class _GradsStruct(ctypes.Structure):
    _fields_ = [("count", ctypes.c_longlong), ("bufs", ctypes.c_void_p), ("sizes", ctypes.POINTER(ctypes.c_longlong)),
                ("dtypes", ctypes.POINTER(ctypes.c_int))]


_szp, _float = ctypes.POINTER(ctypes.c_size_t), ctypes.c_float
_nshape, _eshape, _glist = ctypes.POINTER(_NormStruct), ctypes.POINTER(_EmbedStruct), ctypes.POINTER(_GradsStruct)
_lib.ar_reduce_norm.argtypes = [_vpp, _nshape, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.ar_norm_workspace.argtypes = [_nshape, _szp]
_lib.ar_reduce_norm_backward.argtypes = [_vp, ctypes.c_longlong, _nshape, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                         ctypes.c_size_t, _vp]
_lib.ar_embedding.argtypes = [_vpp, _eshape, _vp, _vp, _vp]
_lib.ar_embedding_workspace.argtypes = [_eshape, _szp]
_lib.ar_embedding_backward.argtypes = [_vp, _eshape, _vp, _vpp, _int, _vp, ctypes.c_size_t, _vp]
_lib.ar_grad_workspace.argtypes = [_glist, _szp]
_lib.ar_grad_norm.argtypes = [_glist, _float, _vp, _vp, ctypes.c_size_t, _vp]
_lib.ar_clip_grads.argtypes = [_glist, _vpp, _float, _float, _float, _vp, _vp, ctypes.c_size_t, _vp]
for _f in (_lib.ar_reduce_norm, _lib.ar_norm_workspace, _lib.ar_reduce_norm_backward, _lib.ar_embedding,
           _lib.ar_embedding_workspace, _lib.ar_embedding_backward, _lib.ar_grad_workspace, _lib.ar_grad_norm,
           _lib.ar_clip_grads):
    _f.restype = ctypes.c_int

try:
    # torch types of a tensor argument by the shape's type code; none where the call itself refuses the code
    _TYPES = {DTYPES["f32"]: (torch.float32,), DTYPES["bf16"]: (torch.bfloat16,), DTYPES["f16"]: (torch.float16,)}
    _F32, _I64, _BYTES = (torch.float32,), (torch.int64,), (torch.float8_e4m3fn, torch.uint8)
except NameError:
    _TYPES, _F32, _I64, _BYTES = {}, (), (), ()
_CODES = {types[0]: code for code, types in _TYPES.items()}

_device_state = []  # [current-device getter] once known


def _device():
    """torch's current device; -2, which no tensor is on, without torch or a GPU."""
    if not _device_state:
        gpu = bool(_TYPES) and torch.cuda.is_available()
        _device_state.append(torch._C._cuda_getDevice if gpu else lambda: -2)
    return _device_state[0]()


def _longs(values, n, what):
    if values is not None and len(values) != n:
        raise ValueError("one %s per rank" % what)
    return None if values is None else (ctypes.c_longlong * max(1, n))(*[int(v) for v in values])


class NormShape:
    """Rows of ``width`` columns whose sum over n rank buffers is normalised:
    rows of rank r ``pitches[r]`` elements apart (default: the width), the
    weight in ``weight_dtype`` (default: the rows' type; else fp32) around
    ``offset``, and ``group`` columns to a scale of the 8-bit output (0: the
    row).  Built once and reusable across calls."""

    def __init__(self, rows, width, n, dtype, pitches=None, weight_dtype=None, eps=1e-6, offset=0.0, group=0):
        self.rows, self.width, self.n = int(rows), int(width), int(n)
        self.dtype = _dtype_code(dtype)
        self.weight_dtype = self.dtype if weight_dtype is None else _dtype_code(weight_dtype)
        self.eps, self.offset, self.group = float(eps), float(offset), int(group)
        self.pitches = [self.width] * self.n if pitches is None else [int(p) for p in pitches]
        self._pitches = _longs(self.pitches, self.n, "pitch")
        self.groups = -(-self.width // self.group) if self.group > 0 else 1
        self._types, self._weight_types = _TYPES.get(self.dtype, ()), _TYPES.get(self.weight_dtype, ())
        self._key = (object(), "partials")     # one of its own, by which a table knows the shape it was looked over for
        self._struct = _NormStruct(self.n, self.dtype, self.weight_dtype, self.rows, self.width, self._pitches, self.eps,
                                   self.offset, self.group)
        self.ref = ctypes.byref(self._struct)


class EmbedShape:
    """``tokens`` rows of ``width`` columns looked up in a table of which rank r
    holds ``entries[r]`` rows, ``pitches[r]`` elements apart (default: the
    width), its gradient's ``grad_pitches[r]`` (default: the pitches).
    ``dtype`` is the table's and its gradient's type, ``out_dtype`` that of the
    looked-up rows and their gradient (default: the same).  Built once and
    reusable across calls."""

    def __init__(self, tokens, entries, width, dtype, out_dtype=None, pitches=None, grad_pitches=None, scale=1.0):
        self.tokens, self.entries, self.n, self.width = int(tokens), [int(e) for e in entries], len(entries), int(width)
        self.dtype = _dtype_code(dtype)
        self.out_dtype = self.dtype if out_dtype is None else _dtype_code(out_dtype)
        self.pitches = [self.width] * self.n if pitches is None else [int(p) for p in pitches]
        self.grad_pitches = self.pitches if grad_pitches is None else [int(p) for p in grad_pitches]
        self.scale = float(scale)
        self._out_types, self._table_key, self._grads_key = _TYPES.get(self.out_dtype, ()), (object(), "tables"), (object(), "grads")
        self._arrays = (_longs(self.entries, self.n, "entry"), _longs(self.pitches, self.n, "pitch"),
                        _longs(self.grad_pitches, self.n, "pitch"))
        self._struct = _EmbedStruct(self.n, self.dtype, self.out_dtype, self.tokens, self.width, *self._arrays, self.scale)
        self.ref = ctypes.byref(self._struct)


def _dense(t):
    """Whether a tensor's elements fill their stretch of memory, in whatever order of dimensions."""
    if t.is_contiguous() or t.numel() == 0:
        return True
    step = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz > 1):
        if stride != step:
            return False
        step *= size
    return True


class GradList:
    """Gradient buffers of any types, sizes and dense layouts, taken together;
    the list keeps references to its tensors.  Built once and reusable across calls."""

    def __init__(self, tensors):
        self._tensors = list(tensors)
        self.host, self.count, self._layouts, self._alike = [], len(self._tensors), [], None
        self._device, codes = _device(), []
        for t in self._tensors:
            if not t.is_contiguous() and not _dense(t):
                raise ValueError("gradients must fill their memory; got strides %s" % (tuple(t.stride()),))
            self._layouts.append((t.dtype, t.shape, t.stride()))
            if t.get_device() != self._device:
                _reachable(t, "gradients", self.host, self._device)
            code = _CODES.get(t.dtype)
            codes.append(_dtype_code(t.dtype) if code is None else code)
        m = max(1, self.count)
        self.sizes = [t.numel() for t in self._tensors]
        self._bufs = (ctypes.c_void_p * m)(*[t.data_ptr() or None for t in self._tensors])
        self._sizes = (ctypes.c_longlong * m)(*self.sizes)
        self._dtypes = (ctypes.c_int * m)(*codes)
        self._struct = _GradsStruct(self.count, ctypes.cast(self._bufs, ctypes.c_void_p), self._sizes, self._dtypes)
        self.ref = ctypes.byref(self._struct)

    def on_host(self, device):
        """Names of what no kernel of ``device``, the current one, reaches; refuses tensors on another one."""
        if device != self._device:
            host = []
            for t in self._tensors:
                _reachable(t, "gradients", host, device)
            self.host, self._device = host, device
        return self.host

    def like(self, other):
        """Whether ``other`` has the same types, shapes and strides, buffer by buffer."""
        if other is self or (self._alike is not None and self._alike() is other):
            return True
        if self._layouts != other._layouts:
            return False
        self._alike = weakref.ref(other)   # the last one found alike, not kept alive; lists do not change
        return True


def _reachable(t, what, host, device):
    """Notes a tensor in host memory by name (as ``_on_host``) and refuses one on another device than the current one."""
    d = t.get_device()
    if d != device:
        if d >= 0:
            raise ValueError("%s must be on the current device (%d), not on device %d" % (what, device, d))
        if _on_host(t):
            host.append(what)


def _packed(t, dtypes, numel, what, host, device):
    """Address of a contiguous tensor argument of one of ``dtypes`` (integer addresses and None pass through)."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype not in dtypes or t.numel() < numel or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of %s with at least %d elements"
                         % (what, " or ".join(str(d) for d in dtypes), numel))
    if t.get_device() != device:
        _reachable(t, what, host, device)
    return t.data_ptr() or None


def _rank_rows(bufs, key, dtype, rows, width, pitches, host, device):
    """Pointer table of rank buffers; tensors must have the type and hold ``rows[r]`` rows (one number: each) at
    ``pitches[r]``.  A table is looked over once for a shape and device."""
    if not isinstance(bufs, PointerTable):
        bufs = PointerTable(bufs)
    if bufs._checked != (key, device):
        rows = [rows] * len(pitches) if isinstance(rows, int) else rows
        if bufs.n != len(rows):
            raise ValueError("%d rank buffers for %d ranks" % (bufs.n, len(rows)))
        at = len(host)
        for b, r, p in zip(bufs._bufs, rows, pitches):
            if b is None or isinstance(b, int) or r == 0:
                continue
            _rows_at(b, dtype, r, width, p, key[1], host, device)
        if len(host) == at:
            bufs._checked = (key, device)
    return bufs.array


def _rows_at(b, dtype, rows, width, pitch, what, host, device):
    if b.dtype not in _TYPES.get(dtype, ()):
        raise ValueError("%s of %s do not have the shape's dtype" % (what, b.dtype))
    room = b.untyped_storage().nbytes() // b.element_size() - b.storage_offset()
    if room < (rows - 1) * pitch + width:
        raise ValueError("%s: a buffer of %d elements; %d rows of %d at pitch %d need more" % (what, room, rows, width, pitch))
    if not _at_pitch(b, pitch, rows):
        raise ValueError("%s have strides %s; their pitch is %d" % (what, tuple(b.stride()), pitch))
    _reachable(b, what, host, device)


def _pitch_of(x, width):
    """Elements between a tensor's rows (all its dimensions but the last): the innermost stride of those that hold more
    than one; the width where no such dimension is left or a row is divided into several (``_rows_at`` has it packed then)."""
    if x.dim() > 1 and x.shape[-1] >= width:
        for size, stride in zip(x.shape[-2::-1], x.stride()[-2::-1]):
            if size > 1:
                return stride
    return width


def _space(w, host, device):
    if w is None:
        return None, 0
    if not w.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _reachable(w, "workspace", host, device)
    return w.data_ptr() or None, w.numel() * w.element_size()


def _refuse_host(host, anything=True):
    if host and anything:
        raise ValueError("%s must be on the GPU, not in host memory" % host[0])


def ar_reduce_norm(partials, shape, weight, out=None, residual=None, summed=None, rstd=None, out8=None, scales=None,
                   stream=None):
    """Sum of the n rank buffers and the residual (``summed``), and its RMS norm
    (``out``; ``out8`` with ``scales``: e4m3 values, a scale to each row or
    group of columns).  ``rstd`` is what ``ar_reduce_norm_backward`` needs
    beside ``summed``."""
    host, r, w, dt, dev = [], shape.rows, shape.width, shape._types, _device()
    size = r * w
    args = (_rank_rows(partials, shape._key, shape.dtype, r, w, shape.pitches, host, dev), shape.ref,
            _packed(weight, shape._weight_types, w, "weight", host, dev), _packed(residual, dt, size, "residual", host, dev),
            _packed(summed, dt, size, "summed", host, dev), _packed(out, dt, size, "out", host, dev),
            _packed(rstd, _F32, r, "rstd", host, dev), _packed(out8, _BYTES, size, "out8", host, dev),
            _packed(scales, _F32, r * shape.groups, "scales", host, dev))
    _refuse_host(host, r)
    _check(_lib.ar_reduce_norm(*args, _stream(stream)))


def ar_norm_workspace(shape) -> int:
    """Workspace bytes of ``ar_reduce_norm_backward`` with a weight gradient (host only)."""
    n = ctypes.c_size_t()
    _check(_lib.ar_norm_workspace(shape.ref, ctypes.byref(n)))
    return n.value


def ar_reduce_norm_backward(x, shape, weight, rstd, grad_out, grad_x, grad_summed=None, grad_weight=None, workspace=None,
                            stream=None):
    """Gradient of the residual and of every partial (``grad_x``), and of the
    weight, from that of ``out`` and, optionally, of ``summed``.  ``x`` is
    ``summed`` (its rows may be apart), ``rstd`` from ``ar_reduce_norm``."""
    host, r, w, dt, dev = [], shape.rows, shape.width, shape._types, _device()
    pitch, size = 0, r * w
    if x is not None and not isinstance(x, int):
        pitch = _pitch_of(x, w)
        if r > 1 and pitch < w:            # 0 would mean the width to the library
            raise ValueError("x has rows at a pitch of %d elements; they hold %d" % (pitch, w))
        if r:
            _rows_at(x, shape.dtype, r, w, pitch, "x", host, dev)
        x = x.data_ptr() or None
    ws, wb = _space(workspace, host, dev)
    args = (x, pitch, shape.ref, _packed(weight, shape._weight_types, w, "weight", host, dev),
            _packed(rstd, _F32, r, "rstd", host, dev), _packed(grad_out, dt, size, "grad_out", host, dev),
            _packed(grad_summed, dt, size, "grad_summed", host, dev), _packed(grad_x, dt, size, "grad_x", host, dev),
            _packed(grad_weight, _F32, w, "grad_weight", host, dev))
    _refuse_host(host)
    _check(_lib.ar_reduce_norm_backward(*args, ws, wb, _stream(stream)))


def ar_embedding(tables, shape, token_ids, out, stream=None):
    """The tokens' rows of a table split by vocabulary entries over the n rank
    buffers, times the scale; zeros for a token outside the vocabulary."""
    host, t, dev = [], shape.tokens, _device()
    args = (_rank_rows(tables, shape._table_key, shape.dtype, shape.entries, shape.width, shape.pitches, host, dev), shape.ref,
            _packed(token_ids, _I64, t, "token_ids", host, dev),
            _packed(out, shape._out_types, t * shape.width, "out", host, dev))
    _refuse_host(host, t)
    _check(_lib.ar_embedding(*args, _stream(stream)))


def ar_embedding_workspace(shape) -> int:
    """Workspace bytes of ``ar_embedding_backward`` (host only)."""
    n = ctypes.c_size_t()
    _check(_lib.ar_embedding_workspace(shape.ref, ctypes.byref(n)))
    return n.value


def ar_embedding_backward(grad_out, shape, token_ids, grads, accumulate=False, workspace=None, stream=None):
    """Gradient of every rank's part of the table, zeros in the rows of entries
    without a token; or, with ``accumulate``, added to what the buffers hold."""
    host, t, dev = [], shape.tokens, _device()
    ws, wb = _space(workspace, host, dev)
    table = _rank_rows(grads, shape._grads_key, shape.dtype, shape.entries, shape.width, shape.grad_pitches, host, dev)
    args = (_packed(grad_out, shape._out_types, t * shape.width, "grad_out", host, dev), shape.ref,
            _packed(token_ids, _I64, t, "token_ids", host, dev), table, int(bool(accumulate)))
    _refuse_host(host, t or not accumulate)
    _check(_lib.ar_embedding_backward(*args, ws, wb, _stream(stream)))


def ar_grad_workspace(grads) -> int:
    """Workspace bytes of the two calls below (host only)."""
    n = ctypes.c_size_t()
    _check(_lib.ar_grad_workspace(grads.ref, ctypes.byref(n)))
    return n.value


def ar_grad_norm(grads, norm, scale=1.0, workspace=None, stream=None):
    """``scale`` times the 2-norm of all buffers of a ``GradList`` taken together."""
    dev = _device()
    host = list(grads.on_host(dev))
    ws, wb = _space(workspace, host, dev)
    norm = _packed(norm, _F32, 1, "norm", host, dev)
    _refuse_host(host)
    _check(_lib.ar_grad_norm(grads.ref, scale, norm, ws, wb, _stream(stream)))


def ar_clip_grads(grads, outs, norm, max_norm, scale=1.0, eps=1e-6, workspace=None, stream=None):
    """``ar_grad_norm``, and every buffer times ``scale`` and, where the norm is
    above it, ``max_norm / (norm + eps)``, into the buffers of ``outs`` (in place
    when ``outs`` is ``grads``).  An infinite ``max_norm`` never clips."""
    if not grads.like(outs):
        raise ValueError("outs must have the types, shapes and strides of grads")
    dev = _device()
    host = grads.on_host(dev) + outs.on_host(dev)
    ws, wb = _space(workspace, host, dev)
    norm = _packed(norm, _F32, 1, "norm", host, dev)
    _refuse_host(host)
    _check(_lib.ar_clip_grads(grads.ref, outs._bufs, max_norm, scale, eps, norm, ws, wb, _stream(stream)))

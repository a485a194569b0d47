"""Python binding of the per-rank state-sharding engine (libfsstate.so).

Argument marshalling only: every step of the path runs in the HIP kernels
behind the C ABI declared in include/fs.h.  torch supplies device memory and
streams.  There is no fallback: if the library is missing, importing its
functions raises.

    plan = fs_plan(shapes, "bf16", world=8, mode="fsdp2")
    plan.upload()                         # segment/tile tables -> device
    fs_pack(plan, params, gathered)       # all-gather copy-in (all N ranks)
    fs_unpack(plan, gathered, outs)       # all-gather copy-out
    fs_reduce_shard(slices, grad32, world=8, grad_acc=4)
    fs_adamw_step(master, m, v, grad32, p16, lr=1e-3, step=1)

With clipping by the global norm (`total` goes through an all-reduce when the
ranks are processes):

    fs_reduce_shard_norm(slices, grad32, total, world=8, grad_acc=4)
    fs_adamw_step_clip(master, m, v, grad32, p16, total=total, max_norm=1.0, step=1)

With 4-bit communication (microscaled blocks of 32):

    mp = fs_mx4_plan(plan).upload()
    fs_pack_mx4(mp, params, gathered4)    # copy-in; seed=... rounds stochastically
    fs_unpack_mx4(mp, gathered4, outs)    # copy-out
    fs_mx4_quantize(x, xq)                # or read a weight where it was gathered:
    fs_mx4_matmul(xq, mp.matrix(gathered4, i), y)
    fs_reduce_shard_mx4(mp, slices4, grad32, rank=r, grad_acc=4)
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
import threading
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfsstate.so")

FS_OK = 0
FS_E_INVAL, FS_E_UNSUPPORTED, FS_E_DTYPE, FS_E_OVERFLOW, FS_E_ALIGN, FS_E_HIP, FS_E_NOMEM = range(-1, -8, -1)
_CODES = {0: "FS_OK", -1: "FS_E_INVAL", -2: "FS_E_UNSUPPORTED", -3: "FS_E_DTYPE",
          -4: "FS_E_OVERFLOW", -5: "FS_E_ALIGN", -6: "FS_E_HIP", -7: "FS_E_NOMEM"}
FS_BF16, FS_FP32 = 0, 1
NOALLOC_MAX_NUMEL = 16777216   # scratch capacity of fs_reduce_adamw_step_noalloc (fp32 elements)
FS_FSDP1_FLAT, FS_FSDP2_PER_PARAM = 1, 2
FS_NORM_L2, FS_NORM_INF = 1, 2


class FsError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_CODES.get(code, code)}: {msg}")
        self.code = code


class PlanInfo(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("dtype", ctypes.c_int32), ("world", ctypes.c_int32),
                ("use_orig_params", ctypes.c_int32), ("grad_acc", ctypes.c_int32),
                ("n_params", ctypes.c_int32), ("elem_bytes", ctypes.c_int32), ("bopt", ctypes.c_int32),
                ("total_numel", ctypes.c_int64), ("flat_numel", ctypes.c_int64),
                ("shard_numel", ctypes.c_int64), ("gathered_numel", ctypes.c_int64),
                ("align_pad", ctypes.c_int64), ("tail_pad", ctypes.c_int64),
                ("n_segments", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("ledger_ideal_bytes", ctypes.c_double), ("ledger_padded_bytes", ctypes.c_double),
                ("ledger_ddp_bytes", ctypes.c_double), ("ledger_zero1_bytes", ctypes.c_double),
                ("ledger_zero2_bytes", ctypes.c_double), ("peak_full_shard_bytes", ctypes.c_double),
                ("comm_full_shard_bytes", ctypes.c_double), ("comm_shard_grad_op_bytes", ctypes.c_double)]


class Segment(ctypes.Structure):
    _fields_ = [("dst_off", ctypes.c_int64), ("src_off", ctypes.c_int64), ("len", ctypes.c_int64),
                ("param", ctypes.c_int32), ("rank", ctypes.c_int32)]


class ParamLayout(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("start", ctypes.c_int64), ("chunk_rows", ctypes.c_int64),
                ("row", ctypes.c_int64), ("pre", ctypes.c_int64)]


class AdamWHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("step", ctypes.c_int64)]


class Clip(ctypes.Structure):
    _fields_ = [("total", ctypes.c_void_p), ("max_norm", ctypes.c_float), ("eps", ctypes.c_float),
                ("norm_type", ctypes.c_int32)]


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libfsstate.so (built by `python -m fsdp_sharded_state_amd.build`)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m fsdp_sharded_state_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    L.fs_plan.argtypes = [i32, vp, vp, i32, i32, i32, i32, i32, ctypes.POINTER(vp)]
    L.fs_plan_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
    L.fs_plan_param.argtypes = [vp, i32, ctypes.POINTER(ParamLayout)]
    L.fs_plan_segments.argtypes = [vp, vp, i64, ctypes.POINTER(i64)]
    L.fs_plan_upload.argtypes = [vp, vp, sz, vp]
    L.fs_plan_destroy.argtypes = [vp]
    L.fs_plan_destroy.restype = None
    L.fs_plan_twin.argtypes = [vp, i32, ctypes.POINTER(vp)]
    L.fs_pack.argtypes = [vp, vp, vp, i32, vp]
    L.fs_unpack.argtypes = [vp, vp, vp, vp]
    L.fs_reduce_shard.argtypes = [i64, i32, i32, vp, vp, vp]
    L.fs_adamw_step.argtypes = [i64, vp, vp, vp, vp, i32, vp, ctypes.POINTER(AdamWHparams), vp]
    L.fs_reshard_plan.argtypes = [vp, vp, ctypes.POINTER(vp)]
    L.fs_reshard_info.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.fs_reshard_upload.argtypes = [vp, vp, sz, vp]
    L.fs_reshard.argtypes = [vp, vp, vp, vp]
    L.fs_reshard_destroy.argtypes = [vp]
    L.fs_reshard_destroy.restype = None
    L.fs_reduce_shard_ex.argtypes = [i64, i32, i32, i32, vp, vp, vp]
    L.fs_pack_cast.argtypes = [vp, vp, i32, vp, i32, vp]
    L.fs_load_local.argtypes = [vp, i32, vp, vp, vp]
    L.fs_reduce_adamw_step_noalloc.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp, ctypes.POINTER(AdamWHparams), vp]
    L.fs_reduce_adamw_step.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp, vp, ctypes.POINTER(AdamWHparams), vp]
    L.fs_grad_norm.argtypes = [i32, vp, vp, vp, i32, i32, vp, vp, vp, sz, vp]
    L.fs_grad_norm_workspace.argtypes = [i32, vp, vp, ctypes.POINTER(i64)]
    L.fs_clip_grads.argtypes = [i32, vp, vp, vp, ctypes.POINTER(Clip), vp, vp]
    L.fs_reduce_shard_norm.argtypes = [i64, i32, i32, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
    L.fs_reduce_shard_norm_workspace.argtypes = [i64, ctypes.POINTER(i64)]
    L.fs_adamw_step_clip.argtypes = [i64, vp, vp, vp, vp, i32, vp, ctypes.POINTER(AdamWHparams), ctypes.POINTER(Clip),
                                     vp]
    mat = ctypes.POINTER(Mx4MatrixStruct)
    L.fs_mx4_quantize.argtypes = [i64, i64, vp, i32, i64, mat, mat, vp, vp]
    L.fs_mx4_dequantize.argtypes = [mat, vp, i32, i64, vp]
    L.fs_mx4_matmul.argtypes = [mat, mat, vp, i32, i64, vp]
    L.fs_mx4_plan.argtypes = [vp, ctypes.POINTER(vp)]
    L.fs_mx4_plan_info.argtypes = [vp, ctypes.POINTER(Mx4PlanInfo)]
    L.fs_mx4_plan_piece.argtypes = [vp, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.fs_mx4_plan_upload.argtypes = [vp, vp, sz, vp]
    L.fs_mx4_plan_matrix.argtypes = [vp, vp, i32, mat]
    L.fs_mx4_plan_destroy.argtypes = [vp]
    L.fs_mx4_plan_destroy.restype = None
    L.fs_pack_mx4.argtypes = [vp, vp, i32, vp, i32, vp, vp]
    L.fs_unpack_mx4.argtypes = [vp, vp, vp, i32, vp]
    L.fs_reduce_shard_mx4.argtypes = [vp, i32, i32, vp, vp, vp]
    L.fs_copy_bytes.argtypes = [vp, vp, i64, vp]
    L.fs_stream_read.argtypes = [vp, i64, vp, vp]
    L.fs_stream_fill.argtypes = [vp, i64, ctypes.c_uint32, vp]
    L.fs_last_error.argtypes = []
    L.fs_last_error.restype = ctypes.c_char_p
    for name in ("fs_plan", "fs_plan_twin", "fs_plan_info", "fs_plan_param", "fs_plan_segments", "fs_plan_upload",
                 "fs_pack", "fs_unpack", "fs_reduce_shard", "fs_adamw_step", "fs_reduce_adamw_step",
                 "fs_reduce_shard_ex", "fs_pack_cast", "fs_reshard_plan", "fs_reshard_info",
                 "fs_reshard_upload", "fs_reshard", "fs_load_local", "fs_reduce_adamw_step_noalloc",
                 "fs_grad_norm", "fs_grad_norm_workspace", "fs_clip_grads", "fs_reduce_shard_norm",
                 "fs_reduce_shard_norm_workspace", "fs_adamw_step_clip",
                 "fs_mx4_quantize", "fs_mx4_dequantize", "fs_mx4_matmul", "fs_mx4_plan",
                 "fs_mx4_plan_info", "fs_mx4_plan_piece", "fs_mx4_plan_upload", "fs_mx4_plan_matrix", "fs_pack_mx4",
                 "fs_unpack_mx4", "fs_reduce_shard_mx4",
                 "fs_copy_bytes", "fs_stream_read", "fs_stream_fill"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(rc: int):
    if rc != FS_OK:
        raise FsError(rc, lib().fs_last_error().decode())


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(dtype) -> int:
    if dtype in ("bf16", torch.bfloat16, FS_BF16):
        return FS_BF16
    if dtype in ("fp32", torch.float32, FS_FP32):
        return FS_FP32
    raise ValueError(f"unsupported dtype {dtype!r}")


def _mode_code(mode) -> int:
    if mode in ("fsdp1", FS_FSDP1_FLAT):
        return FS_FSDP1_FLAT
    if mode in ("fsdp2", FS_FSDP2_PER_PARAM):
        return FS_FSDP2_PER_PARAM
    raise ValueError(f"unsupported mode {mode!r}")


def _dev_ptr(t: torch.Tensor, what: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _bytes_on(index: int, stream, handle: int, nbytes: int) -> torch.Tensor:
    """Memory of the current GPU, `index`, that belongs to a stream (None: the
    current one): the allocator hands it out again in that stream's order."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=index)
    device = torch.device("cuda", index)
    own = (stream if isinstance(stream, torch.cuda.Stream) else
           torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device))
    with torch.cuda.stream(own):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


class _Table:
    """Device memory that kernels read when they run, not when they are
    enqueued.  The allocator hands it out again in the order of the stream it
    was taken on; every other stream that reads it is recorded, once, so that
    the allocator waits for that one too."""

    __slots__ = ("memory", "index", "known")

    def __init__(self, memory: torch.Tensor, handle: int):
        self.memory, self.index = memory, memory.get_device()
        self.known = {handle} - {_PER_THREAD_STREAM}    # handles of the streams that need no more

    def read_on(self, stream, handle: int) -> bool:
        """A launch on `stream` (None: the current one), whose handle this is,
        reads the memory.  False where the allocator cannot be told: a bare
        handle may be destroyed before the memory is given back, and the
        per-thread default stream is another one in every thread."""
        if handle in self.known:
            return True
        if stream is None:
            stream = torch.cuda.current_stream(self.memory.device)
        if handle == _PER_THREAD_STREAM or not isinstance(stream, torch.cuda.Stream):
            return False
        self.memory.record_stream(stream)
        self.known.add(handle)
        return True


def _read_on(table: Optional[_Table], stream) -> Optional[int]:
    """The handle of the stream of a launch that reads a plan's tables (None: it has none yet, which the call refuses)."""
    handle = _stream(stream)
    if table is not None and handle not in table.known:
        table.read_on(stream, handle)
    return handle


_putting = threading.Lock()


def _put(plan, fn, nbytes: int, device, stream):
    """A plan's tables on a GPU, unless they are there already.  One thread at
    a time, so that the library has the tables that the plan keeps."""
    where = torch.device(device)
    with _putting:
        if plan.workspace is not None and where.type == "cuda" and plan.workspace.get_device() == (
                torch.cuda.current_device() if where.index is None else where.index):
            return
        table = _upload(fn, plan._h, nbytes, where, stream)
        if plan._table is not None:
            plan._earlier.append(plan._table)
        plan._table, plan.workspace = table, table.memory


def _upload(fn, plan, nbytes: int, device, stream) -> _Table:
    """The tables of a plan on a GPU, in memory of the stream that copies them:
    what another stream has under way could still write to memory of its own.
    In place of the per-thread default stream, which the allocator cannot tell
    from other threads', the default one copies; the copy is waited for."""
    where, nbytes = torch.device(device), max(16, nbytes)
    if where.type != "cuda":
        ws = torch.empty(nbytes, dtype=torch.uint8, device=where)
        _check(fn(plan, ws.data_ptr(), nbytes, None))   # refuses host memory
        return _Table(ws, 0)
    index = torch.cuda.current_device() if where.index is None else where.index
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _upload(fn, plan, nbytes, where, stream)
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tables go to {torch.device('cuda', index)}")
    if handle == _PER_THREAD_STREAM:
        stream, handle = torch.cuda.default_stream(index), 0
    ws = _bytes_on(index, stream, handle, nbytes)
    _check(fn(plan, ws.data_ptr(), nbytes, handle))
    return _Table(ws, handle)


# What a call asks of every tensor of a list.
_DATA_PTR, _NUMEL, _IS_CONTIGUOUS = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous
_ELEMENT_SIZE, _GET_DEVICE = torch.Tensor.element_size, torch.Tensor.get_device
_IS_CUDA, _DTYPE = operator.attrgetter("is_cuda"), operator.attrgetter("dtype")


class Plan:
    """An uploaded-or-not layout plan (wraps fs_plan_t).  Keep a plan until the
    work of calls on a bare stream handle is done, and as long as a captured
    graph holds calls on it; for other streams the tables stay as long as
    enqueued work reads them."""

    def __init__(self, handle: int):
        self._h = ctypes.c_void_p(handle)
        self._destroy = lib().fs_plan_destroy   # kept for interpreter shutdown
        info = PlanInfo()
        _check(lib().fs_plan_info(self._h, ctypes.byref(info)))
        self.info = info
        self.workspace: Optional[torch.Tensor] = None
        self._table: Optional[_Table] = None    # the workspace and who reads it
        self._earlier: list = []                # those on other GPUs, which launches and captured graphs may still read
        self._ptr_cache = {}
        self._pinned = set()        # pointer-table keys a captured graph or another stream may still read
        self._pieces = {}           # rank -> local piece element counts
        self.numels = [self.param(i).numel for i in range(info.n_params)]
        self.shapes: Optional[List[tuple]] = None   # set by fs_plan()

    def close(self):
        """Release the plan's host memory (also done on garbage collection)."""
        h = self.__dict__.pop("_h", None)
        if h is not None and h.value:
            self._destroy(h)

    def __del__(self):
        self.close()

    # summary
    def __getattr__(self, name):
        info = self.__dict__.get("info")
        if info is not None and name in dict(PlanInfo._fields_):
            return getattr(info, name)
        raise AttributeError(name)

    def param(self, i: int) -> ParamLayout:
        out = ParamLayout()
        _check(lib().fs_plan_param(self._h, i, ctypes.byref(out)))
        return out

    def segments(self) -> List[tuple]:
        n = ctypes.c_int64()
        _check(lib().fs_plan_segments(self._h, None, 0, ctypes.byref(n)))
        arr = (Segment * max(1, n.value))()
        _check(lib().fs_plan_segments(self._h, arr, n.value, ctypes.byref(n)))
        return [(s.dst_off, s.src_off, s.len, s.param, s.rank) for s in arr[:n.value]]

    def local_pieces(self, rank: int) -> List[Optional[tuple]]:
        """Where each parameter's elements held by `rank` sit: per parameter,
        (offset in the rank's shard, first element of the flattened
        parameter, count), or None when the rank holds none of it.  A
        parameter's elements on one rank are always one contiguous run, in
        both layouts."""
        if not 0 <= rank < self.info.world:
            raise ValueError(f"rank {rank} out of range [0, {self.info.world})")
        c = self.info.shard_numel
        out: List[Optional[tuple]] = [None] * self.info.n_params
        for dst, src, ln, p, r in self.segments():
            if r == rank:
                if out[p] is not None:
                    raise RuntimeError(f"parameter {p} has two runs on rank {rank}")
                out[p] = (dst - r * c, src, ln)
        return out

    def twin(self, dtype) -> "Plan":
        """The plan of `dtype` elements at this plan's element positions
        (fs_plan_twin): lays out the fp32 master, m and v of this plan's bf16
        parameters element for element (not uploaded)."""
        h = ctypes.c_void_p()
        _check(lib().fs_plan_twin(self._h, _dtype_code(dtype), ctypes.byref(h)))
        t = Plan(h.value)
        t.shapes = self.shapes
        return t

    def local_views(self, shard: torch.Tensor, rank: int) -> List[torch.Tensor]:
        """The sharded state dict of `rank`, zero-copy: for each parameter,
        the view of `shard` (that rank's shard buffer, shard_numel elements:
        parameters, gradients or optimizer state laid out by this plan) that
        holds the parameter's local elements.  FSDP2: shaped (rows, *shape[1:])
        -- the rank's dim-0 chunk, empty when it has no rows; FSDP1: 1-D, the
        flattened parameter's elements that fall in the rank's flat shard."""
        if shard.dim() != 1 or shard.numel() != self.info.shard_numel:
            raise ValueError(f"shard must be 1-D with {self.info.shard_numel} elements")
        if shard.element_size() != self.info.elem_bytes:
            raise ValueError(f"shard element size {shard.element_size()} != plan's {self.info.elem_bytes}")
        fsdp2 = self.info.mode == FS_FSDP2_PER_PARAM
        views = []
        for i, piece in enumerate(self.local_pieces(rank)):
            off, _, ln = piece if piece is not None else (0, 0, 0)
            v = shard[off:off + ln]
            tail = tuple(self.shapes[i][1:]) if fsdp2 and self.shapes and self.shapes[i] else ()
            row = math.prod(tail)
            views.append(v.view((ln // row,) + tail) if fsdp2 and row else v)
        return views

    def local_numels(self, rank: int) -> List[int]:
        """Element count of every parameter's local piece on `rank`."""
        if rank not in self._pieces:
            self._pieces[rank] = [0 if pc is None else pc[2] for pc in self.local_pieces(rank)]
        return self._pieces[rank]

    def load_local(self, shard: torch.Tensor, rank: int, tensors: Sequence[torch.Tensor], stream=None):
        """Import a sharded state dict (fs_load_local): write each parameter's
        local tensor (shaped as local_views returns it, or flat) into its place
        in `shard` (that rank's shard buffer on the GPU) and zero the pads."""
        if not 0 <= rank < self.info.world:
            raise ValueError(f"rank {rank} out of range [0, {self.info.world})")
        if shard.dim() != 1 or shard.numel() != self.info.shard_numel:
            raise ValueError(f"shard must be 1-D with {self.info.shard_numel} elements")
        if shard.element_size() != self.info.elem_bytes:
            raise ValueError(f"shard element size {shard.element_size()} != plan's {self.info.elem_bytes}")
        want = self.local_numels(rank)
        if len(tensors) != len(want):
            raise ValueError(f"expected {len(want)} local tensors, got {len(tensors)}")
        for i, (t, n) in enumerate(zip(tensors, want)):
            if t.numel() != n:
                raise ValueError(f"local tensor {i}: {t.numel()} elements, rank {rank} holds {n}")
        tab = self.ptr_table(tensors, "local tensors", numels=want, stream=stream)
        _check(lib().fs_load_local(self._h, int(rank), tab.data_ptr(),
                                   _dev_ptr(shard, "shard") if shard.numel() else 0, _read_on(self._table, stream)))

    def upload(self, device="cuda", stream=None) -> "Plan":
        """Put the tables on a GPU, copied on `stream`, and wait for them.  They do not change, so where they are
        there already they stay."""
        _put(self, lib().fs_plan_upload, self.info.workspace_bytes, device, stream)
        return self

    def ptr_table(self, tensors: Sequence[torch.Tensor], what: str, elem_bytes: Optional[int] = None,
                  numels: Optional[Sequence[int]] = None, stream=None, known: bool = False) -> torch.Tensor:
        """Device array of the tensors' data pointers (cached per pointer set).
        Every tensor must hold `numels[i]` elements (default: its parameter's
        element count) of `elem_bytes` bytes (default: the plan's).  known: the
        caller has checked that they are GPU tensors of that element size.

        The kernels read the table when they run, not when they are enqueued,
        so a table must outlive every launch that uses it.  A few recent sets
        are kept; the oldest is released when a new one is made, which is safe
        for launches on the stream that was current when it was made (the
        allocator reuses its memory in that stream's order); every other torch
        stream that it is used on, given or current, is recorded.  A table used
        while a graph is being captured, with a stream given as a raw handle or
        on the per-thread default stream is pinned for the plan's lifetime.  A new set
        cannot be made during capture (its upload would be a captured copy
        from host memory): run the call once before capturing."""
        if len(tensors) != self.info.n_params:
            raise ValueError(f"{what}: expected {self.info.n_params} tensors, got {len(tensors)}")
        esz = self.info.elem_bytes if elem_bytes is None else elem_bytes
        want = self.numels if numels is None else numels
        ptrs, held = list(map(_DATA_PTR, tensors)), list(map(_NUMEL, tensors))   # in bulk: half the time of a loop's
        if 0 in held:
            ptrs = [p if n else 0 for p, n in zip(ptrs, held)]
        if held != list(want) or not all(map(_IS_CONTIGUOUS, tensors)) or not (
                known or all(map(_IS_CUDA, tensors)) and not set(map(_ELEMENT_SIZE, tensors)) - {esz}):
            for i, t in enumerate(tensors):     # which one it is
                if t.element_size() != esz:
                    raise ValueError(f"{what}[{i}]: element size {t.element_size()} != {esz}")
                if t.numel() != want[i]:
                    raise ValueError(f"{what}[{i}]: numel {t.numel()} != {want[i]}")
                if t.numel():
                    _dev_ptr(t, f"{what}[{i}]")
        key = (tuple(ptrs), tensors[0].get_device() if tensors else -1)
        capturing = ((tensors and tensors[0].is_cuda or torch.cuda.is_available()) and
                     torch.cuda.is_current_stream_capturing())
        tab = self._ptr_cache.get(key)
        if tab is None:
            if capturing:
                raise RuntimeError(f"{what}: a pointer set not seen before, during graph capture; run the same "
                                   "call once before capturing so that its device pointer table exists")
            dev = next((t.device for t in tensors if t.is_cuda), torch.device("cuda"))   # one without elements may be elsewhere
            tab = torch.tensor(ptrs or [0], dtype=torch.int64, device=dev)
            tab = _Table(tab, torch._C._cuda_getCurrentRawStream(tab.get_device()))
            if len(self._ptr_cache) >= 8:          # keep a few pointer sets (pack and unpack sides)
                # (a copy of the keys, and no error without the oldest: another thread may be at the same place)
                old = next((k for k in list(self._ptr_cache) if k not in self._pinned), None)
                if old is not None:
                    self._ptr_cache.pop(old, None)
            self._ptr_cache[key] = tab
        handle = torch._C._cuda_getCurrentRawStream(tab.index) if stream is None else _stream(stream)
        if stream is None and not capturing and handle in tab.known:
            return tab.memory
        bare = stream is not None and not isinstance(stream, torch.cuda.Stream)
        if not tab.read_on(stream, handle) or capturing or bare:
            self._pinned.add(key)
            self._ptr_cache[key] = tab          # another thread may have released it before the pin was there
        return tab.memory


def fs_plan(shapes: Sequence[Sequence[int]], dtype="bf16", world: int = 1, use_orig_params: bool = False,
            mode="fsdp1", grad_acc: int = 1) -> Plan:
    """Plan one FSDP group's shard layout (fs_plan)."""
    n = len(shapes)
    ndim = (ctypes.c_int32 * max(1, n))(*[len(s) for s in shapes])
    flat = [int(d) for s in shapes for d in s]
    dims = (ctypes.c_int64 * max(1, len(flat)))(*flat)
    h = ctypes.c_void_p()
    _check(lib().fs_plan(n, ndim, dims, _dtype_code(dtype), int(world), int(bool(use_orig_params)),
                         _mode_code(mode), int(grad_acc), ctypes.byref(h)))
    plan = Plan(h.value)
    plan.shapes = [tuple(int(d) for d in s) for s in shapes]
    return plan


class Reshard:
    """Relayout plan from one group plan to another (wraps fs_reshard_t)."""

    def __init__(self, src: "Plan", dst: "Plan"):
        h = ctypes.c_void_p()
        _check(lib().fs_reshard_plan(src._h, dst._h, ctypes.byref(h)))
        self._h = h
        self._destroy = lib().fs_reshard_destroy
        self.src_info, self.dst_info = src.info, dst.info
        wb, ns = ctypes.c_int64(), ctypes.c_int64()
        _check(lib().fs_reshard_info(h, ctypes.byref(wb), ctypes.byref(ns)))
        self.workspace_bytes, self.n_segments = wb.value, ns.value
        self.workspace: Optional[torch.Tensor] = None
        self._table: Optional[_Table] = None    # the workspace and who reads it
        self._earlier: list = []                # those on other GPUs, which launches and captured graphs may still read

    def close(self):
        h = self.__dict__.pop("_h", None)
        if h is not None and h.value:
            self._destroy(h)

    def __del__(self):
        self.close()

    def upload(self, device="cuda", stream=None) -> "Reshard":
        """As Plan.upload."""
        _put(self, lib().fs_reshard_upload, self.workspace_bytes, device, stream)
        return self


def fs_reshard_plan(src: "Plan", dst: "Plan") -> Reshard:
    """Plan moving a group's gathered buffer from plan src (N) to plan dst (N')."""
    return Reshard(src, dst)


def fs_reshard(r: Reshard, src_gathered: torch.Tensor, dst_gathered: torch.Tensor, stream=None):
    """dst_gathered <- src_gathered re-laid from the src plan to the dst plan."""
    if src_gathered.numel() != r.src_info.gathered_numel or dst_gathered.numel() != r.dst_info.gathered_numel:
        raise ValueError("fs_reshard: buffer sizes do not match the plans")
    _check(lib().fs_reshard(r._h, _dev_ptr(src_gathered, "src_gathered") if src_gathered.numel() else 0,
                            _dev_ptr(dst_gathered, "dst_gathered") if dst_gathered.numel() else 0,
                            _read_on(r._table, stream)))


def fs_pack(plan: Plan, params: Sequence[torch.Tensor], out: torch.Tensor, rank: int = -1, stream=None):
    """All-gather copy-in: params -> out (whole gathered buffer, or rank's shard)."""
    want = plan.info.gathered_numel if rank < 0 else plan.info.shard_numel
    if out.numel() != want or out.element_size() != plan.info.elem_bytes:
        raise ValueError(f"fs_pack: out must hold {want} elements of {plan.info.elem_bytes} bytes")
    tab = plan.ptr_table(params, "params", stream=stream)
    _check(lib().fs_pack(plan._h, tab.data_ptr(), _dev_ptr(out, "out") if want else 0, int(rank),
                         _read_on(plan._table, stream)))


def fs_pack_cast(plan: Plan, params: Sequence[torch.Tensor], out: torch.Tensor, rank: int = -1, stream=None):
    """Copy-in with the parameter-dtype cast: fp32 params into a bf16 plan's
    gathered buffer (or rank's shard), rounded to nearest even."""
    want = plan.info.gathered_numel if rank < 0 else plan.info.shard_numel
    if out.numel() != want or out.dtype != torch.bfloat16:
        raise ValueError(f"fs_pack_cast: out must be bfloat16 with {want} elements")
    if not params:
        raise ValueError("fs_pack_cast: no parameters")
    dt = params[0].dtype
    if any(p.dtype != dt for p in params):
        raise ValueError("fs_pack_cast: parameters must share one dtype")
    tab = plan.ptr_table(params, "params", elem_bytes=params[0].element_size(), stream=stream)
    _check(lib().fs_pack_cast(plan._h, tab.data_ptr(), _dtype_code(dt), _dev_ptr(out, "out") if want else 0,
                              int(rank), _read_on(plan._table, stream)))


def fs_unpack(plan: Plan, gathered: torch.Tensor, params: Sequence[torch.Tensor], stream=None):
    """All-gather copy-out: gathered -> params."""
    if gathered.numel() != plan.info.gathered_numel or gathered.element_size() != plan.info.elem_bytes:
        raise ValueError("fs_unpack: gathered has the wrong size or element size")
    tab = plan.ptr_table(params, "params", stream=stream)
    _check(lib().fs_unpack(plan._h, _dev_ptr(gathered, "gathered") if gathered.numel() else 0,
                           tab.data_ptr(), _read_on(plan._table, stream)))


def fs_reduce_shard(slices: Sequence[torch.Tensor], out: torch.Tensor, world: int, grad_acc: int = 1, stream=None):
    """Average slices[j*world + k] (bf16, n each) into out (fp32, n)."""
    n = out.numel()
    if out.dtype != torch.float32:
        raise ValueError("fs_reduce_shard: out must be float32")
    if len(slices) != world * grad_acc:
        raise ValueError(f"fs_reduce_shard: need world*grad_acc = {world * grad_acc} slices")
    ptrs = []
    for k, s in enumerate(slices):
        if s.dtype != torch.bfloat16 or s.numel() != n:
            raise ValueError(f"fs_reduce_shard: slice {k} must be bf16 with {n} elements")
        ptrs.append(_dev_ptr(s, f"slices[{k}]") if n else 0)
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    _check(lib().fs_reduce_shard(n, int(world), int(grad_acc), arr, _dev_ptr(out, "out") if n else 0,
                                 _stream(stream)))


def fs_reduce_shard_ex(slices: Sequence[torch.Tensor], out: torch.Tensor, world: int, grad_acc: int = 1,
                       reduce_dtype="fp32", stream=None):
    """fs_reduce_shard with a reduce dtype: "fp32" (same as fs_reduce_shard)
    or "bf16" (each micro-step's average delivered in bf16, accumulated in fp32)."""
    n = out.numel()
    if out.dtype != torch.float32:
        raise ValueError("fs_reduce_shard_ex: out must be float32")
    if len(slices) != world * grad_acc:
        raise ValueError(f"fs_reduce_shard_ex: need world*grad_acc = {world * grad_acc} slices")
    ptrs = []
    for k, s in enumerate(slices):
        if s.dtype != torch.bfloat16 or s.numel() != n:
            raise ValueError(f"fs_reduce_shard_ex: slice {k} must be bf16 with {n} elements")
        ptrs.append(_dev_ptr(s, f"slices[{k}]") if n else 0)
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    _check(lib().fs_reduce_shard_ex(n, int(world), int(grad_acc), _dtype_code(reduce_dtype), arr,
                                    _dev_ptr(out, "out") if n else 0, _stream(stream)))


def fs_adamw_step(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, grad: torch.Tensor,
                  param_bf16: Optional[torch.Tensor] = None, *, lr: float = 1e-3, beta1: float = 0.9,
                  beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01, step: int = 1,
                  stream=None):
    """One AdamW step over the fp32 shard (in place), writing the bf16 copy."""
    n = master.numel()
    for name, t in (("master", master), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
        if t.dtype != torch.float32 or t.numel() != n:
            raise ValueError(f"fs_adamw_step: {name} must be float32 with {n} elements")
    if grad.numel() != n or grad.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("fs_adamw_step: grad must be float32 or bfloat16 with n elements")
    if param_bf16 is not None and (param_bf16.dtype != torch.bfloat16 or param_bf16.numel() != n):
        raise ValueError("fs_adamw_step: param_bf16 must be bfloat16 with n elements")
    hp = AdamWHparams(lr, beta1, beta2, eps, weight_decay, 0, int(step))
    ptr = (lambda t, w: _dev_ptr(t, w) if n else 0)
    _check(lib().fs_adamw_step(n, ptr(master, "master"), ptr(exp_avg, "exp_avg"), ptr(exp_avg_sq, "exp_avg_sq"),
                               ptr(grad, "grad"), FS_BF16 if grad.dtype == torch.bfloat16 else FS_FP32,
                               ptr(param_bf16, "param_bf16") if param_bf16 is not None else None,
                               ctypes.byref(hp), _stream(stream)))


def fs_reduce_adamw_step(slices: Sequence[torch.Tensor], master: torch.Tensor, exp_avg: torch.Tensor,
                         exp_avg_sq: torch.Tensor, param_bf16: Optional[torch.Tensor] = None,
                         grad_out: Optional[torch.Tensor] = None, *, world: int, grad_acc: int = 1,
                         lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                         weight_decay: float = 0.01, step: int = 1, stream=None):
    """Fused reduce + AdamW: average slices[j*world + k] (bf16) and apply one
    AdamW step to the fp32 shard in place; the averaged gradient goes to
    grad_out only if given."""
    n = master.numel()
    for name, t in (("master", master), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
        if t.dtype != torch.float32 or t.numel() != n:
            raise ValueError(f"fs_reduce_adamw_step: {name} must be float32 with {n} elements")
    if len(slices) != world * grad_acc:
        raise ValueError(f"fs_reduce_adamw_step: need world*grad_acc = {world * grad_acc} slices")
    ptrs = []
    for k, s in enumerate(slices):
        if s.dtype != torch.bfloat16 or s.numel() != n:
            raise ValueError(f"fs_reduce_adamw_step: slice {k} must be bf16 with {n} elements")
        ptrs.append(_dev_ptr(s, f"slices[{k}]") if n else 0)
    if param_bf16 is not None and (param_bf16.dtype != torch.bfloat16 or param_bf16.numel() != n):
        raise ValueError("fs_reduce_adamw_step: param_bf16 must be bfloat16 with n elements")
    if grad_out is not None and (grad_out.dtype != torch.float32 or grad_out.numel() != n):
        raise ValueError("fs_reduce_adamw_step: grad_out must be float32 with n elements")
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    hp = AdamWHparams(lr, beta1, beta2, eps, weight_decay, 0, int(step))
    ptr = (lambda t, w: (_dev_ptr(t, w) if n else 0) if t is not None else None)
    _check(lib().fs_reduce_adamw_step(n, int(world), int(grad_acc), arr, ptr(master, "master"),
                                      ptr(exp_avg, "exp_avg"), ptr(exp_avg_sq, "exp_avg_sq"),
                                      ptr(param_bf16, "param_bf16"), ptr(grad_out, "grad_out"),
                                      ctypes.byref(hp), _stream(stream)))


def fs_reduce_adamw_step_noalloc(slices: Sequence[torch.Tensor], master: torch.Tensor, exp_avg: torch.Tensor,
                                 exp_avg_sq: torch.Tensor, param_bf16: Optional[torch.Tensor] = None, *, world: int,
                                 grad_acc: int = 1, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999,
                                 eps: float = 1e-8, weight_decay: float = 0.01, step: int = 1, stream=None):
    """fs_reduce_adamw_step without grad_out, for callers that cannot
    allocate: with more than 32 terms the partial sums go to the library's
    per-GPU scratch array (at most NOALLOC_MAX_NUMEL elements)."""
    n = master.numel()
    for name, t in (("master", master), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
        if t.dtype != torch.float32 or t.numel() != n:
            raise ValueError(f"fs_reduce_adamw_step_noalloc: {name} must be float32 with {n} elements")
    if len(slices) != world * grad_acc:
        raise ValueError(f"fs_reduce_adamw_step_noalloc: need world*grad_acc = {world * grad_acc} slices")
    ptrs = []
    for k, s in enumerate(slices):
        if s.dtype != torch.bfloat16 or s.numel() != n:
            raise ValueError(f"fs_reduce_adamw_step_noalloc: slice {k} must be bf16 with {n} elements")
        ptrs.append(_dev_ptr(s, f"slices[{k}]") if n else 0)
    if param_bf16 is not None and (param_bf16.dtype != torch.bfloat16 or param_bf16.numel() != n):
        raise ValueError("fs_reduce_adamw_step_noalloc: param_bf16 must be bfloat16 with n elements")
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    hp = AdamWHparams(lr, beta1, beta2, eps, weight_decay, 0, int(step))
    ptr = (lambda t, w: (_dev_ptr(t, w) if n else 0) if t is not None else None)
    _check(lib().fs_reduce_adamw_step_noalloc(n, int(world), int(grad_acc), arr, ptr(master, "master"),
                                              ptr(exp_avg, "exp_avg"), ptr(exp_avg_sq, "exp_avg_sq"),
                                              ptr(param_bf16, "param_bf16"), ctypes.byref(hp), _stream(stream)))


_PER_THREAD_STREAM = 2   # hipStreamPerThread's handle

_DTYPE_CODES = {torch.bfloat16: FS_BF16, torch.float32: FS_FP32}
_NORM_CODES = {2: FS_NORM_L2, "2": FS_NORM_L2, math.inf: FS_NORM_INF, "inf": FS_NORM_INF}


def _norm_code(norm_type) -> int:
    code = _NORM_CODES.get(norm_type)
    if code is None:
        raise ValueError(f"unsupported norm_type {norm_type!r}: 2 and inf are defined")
    return code


class GradList:
    """A list of gradient tensors (or of reduce slices) that is handed to
    several calls: their addresses, element counts and types, looked up once.

    The tensors' memory is held, not the tensor objects' identity: a gradient
    that is replaced (`p.grad = other`, `p.data = other`) needs a new list.  A
    storage that has been resized since is noticed and refused."""

    def __init__(self, tensors: Sequence[torch.Tensor]):
        n = len(tensors)
        devices = {t.get_device() for t in tensors}
        if len(devices) > 1 or -1 in devices or not all(t.is_contiguous() for t in tensors):
            for i, t in enumerate(tensors):
                _dev_ptr(t, f"tensor {i}")
                if t.device != tensors[0].device:
                    raise ValueError(f"tensor {i} is on {t.device}, tensor 0 on {tensors[0].device}")
        ptrs, numels = [t.data_ptr() for t in tensors], [t.numel() for t in tensors]
        codes = [_DTYPE_CODES.get(t.dtype) for t in tensors]
        if None in codes:
            _dtype_code(tensors[codes.index(None)].dtype)   # raises
        self._index: Optional[int] = devices.pop() if n else None      # of their GPU; None for an empty list
        self._same = (codes[0], numels[0]) if n and len(set(codes)) == 1 and len(set(numels)) == 1 else None
        storages = {}                                       # holding them keeps the memory
        for t in tensors:
            st = t.untyped_storage()
            storages[st._cdata] = st
        self._storages = [(st, st.data_ptr(), st.nbytes()) for st in storages.values()]
        self._n = n
        self._ptrs = (ctypes.c_void_p * max(1, n))(*ptrs)
        self._numels = (ctypes.c_int64 * max(1, n))(*numels)
        self._codes = (ctypes.c_int32 * max(1, n))(*codes)
        need = ctypes.c_int64()
        _check(lib().fs_grad_norm_workspace(n, self._numels, self._codes, ctypes.byref(need)))
        self._norm_bytes = need.value
        if self._same is not None:
            _check(lib().fs_reduce_shard_norm_workspace(numels[0], ctypes.byref(need)))
        self._reduce_bytes = need.value                 # as the slices of one reduce

    def __len__(self) -> int:
        return self._n

    def _live(self) -> "GradList":
        for st, ptr, nbytes in self._storages:
            if st.data_ptr() != ptr or st.nbytes() != nbytes:
                raise ValueError("a tensor of the list no longer has the memory it had when the list was made")
        return self


def fs_grad_list(tensors: Sequence[torch.Tensor]) -> GradList:
    """A list of bf16 and fp32 gradients on one GPU, for fs_grad_norm,
    fs_clip_grads and (bf16, one size) fs_reduce_shard_norm."""
    return GradList(tensors)


def _grad_list(tensors) -> GradList:
    return tensors._live() if isinstance(tensors, GradList) else GradList(tensors)


def _scalar_ptr(t: Optional[torch.Tensor], dtype: torch.dtype, index: Optional[int], what: str) -> Optional[int]:
    """Address of a one-value tensor on GPU `index` (None: on any GPU)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != 1:
        raise ValueError(f"{what} must be one {dtype} value")
    if t.get_device() != index:
        if index is not None and index >= 0:
            raise ValueError(f"{what} is on {t.device}, the other arguments on cuda:{index}")
        if not t.is_cuda:
            raise ValueError(f"{what} must be a GPU tensor")
    return t.data_ptr()


def _launch(index: int, stream, fn, *args, scratch: int = -1, table: Optional[_Table] = None):
    """Run a launching call with GPU `index` current, on `stream` (default:
    that GPU's current stream).  table: what the call reads of a plan (None
    also where a plan has none yet, which the call refuses).  scratch >= 0:
    that many workspace bytes and their count go before the stream; they
    belong to the stream the kernels run on, so the allocator hands them out again in that stream's order.  The
    per-thread default stream is refused there: it is a stream of its own in
    every host thread, but has one handle, so the allocator would hand one
    thread's workspace to another while it is in use."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _launch(index, stream, fn, *args, scratch=scratch, table=table)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        handle = _stream(stream)
        if isinstance(stream, torch.cuda.Stream) and stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    if table is not None and handle not in table.known:
        table.read_on(stream, handle)
    if scratch < 0:
        return _check(fn(*args, handle))
    if handle == _PER_THREAD_STREAM:
        raise ValueError("the per-thread default stream cannot be used here: make a stream for each thread")
    if scratch == 0:
        return _check(fn(*args, None, 0, handle))
    ws = _bytes_on(index, stream, handle, scratch)
    return _check(fn(*args, ws.data_ptr(), scratch, handle))


def fs_grad_norm(grads, total: torch.Tensor, norm: Optional[torch.Tensor] = None, *, norm_type=2.0,
                 accumulate: bool = False, stream=None):
    """Total (float64, one value: the sum of squares, or with norm_type inf
    the largest magnitude) and norm (float32, one value) of a list of bf16 and
    fp32 gradients: a sequence of tensors or a GradList.  accumulate: joined
    to the total that stands there.  stream: a torch stream or a raw handle,
    which is not to be destroyed before the call's work is done; not the
    per-thread default stream."""
    kind = _norm_code(norm_type)
    gl = _grad_list(grads)
    tot = _scalar_ptr(total, torch.float64, gl._index, "total")
    index = total.get_device()
    _launch(index, stream, lib().fs_grad_norm, gl._n, gl._ptrs, gl._numels, gl._codes, kind, int(accumulate),
            tot, _scalar_ptr(norm, torch.float32, index, "norm"), scratch=gl._norm_bytes)


def fs_clip_grads(grads, total: torch.Tensor, max_norm: float, norm: Optional[torch.Tensor] = None, *, norm_type=2.0,
                  norm_eps: float = 1e-6, stream=None):
    """Scale a list of gradients in place by min(1, max_norm / (norm_of(total)
    + norm_eps)); norm (float32, one value) receives the norm of the total."""
    kind = _norm_code(norm_type)
    gl = _grad_list(grads)
    clip = Clip(_scalar_ptr(total, torch.float64, gl._index, "total"), max_norm, norm_eps, kind)
    index = total.get_device()
    _launch(index, stream, lib().fs_clip_grads, gl._n, gl._ptrs, gl._numels, gl._codes, ctypes.byref(clip),
            _scalar_ptr(norm, torch.float32, index, "norm"))


def fs_reduce_shard_norm(slices, out: torch.Tensor, total: torch.Tensor, norm: Optional[torch.Tensor] = None, *,
                         world: int, grad_acc: int = 1, reduce_dtype="fp32", norm_type=2.0,
                         accumulate: bool = False, stream=None):
    """fs_reduce_shard_ex (slices: a sequence or a GradList), and the total and
    norm of the averaged gradients, as fs_grad_norm gives them for out.
    stream: as there."""
    kind = _norm_code(norm_type)
    n = out.numel()
    if out.dtype is not torch.float32:
        raise ValueError("fs_reduce_shard_norm: out must be float32")
    if len(slices) != world * grad_acc:
        raise ValueError(f"fs_reduce_shard_norm: need world*grad_acc = {world * grad_acc} slices")
    gl = _grad_list(slices)
    if gl._n and gl._same != (FS_BF16, n):
        raise ValueError(f"fs_reduce_shard_norm: every slice must be bf16 with {n} elements")
    index = out.get_device()
    if gl._n and gl._index != index:
        raise ValueError(f"fs_reduce_shard_norm: out is on {out.device}, the slices on cuda:{gl._index}")
    ptr = _dev_ptr(out, "out")
    _launch(index, stream, lib().fs_reduce_shard_norm, n, int(world), int(grad_acc), _dtype_code(reduce_dtype),
            gl._ptrs, ptr if n else 0, kind, int(accumulate), _scalar_ptr(total, torch.float64, index, "total"),
            _scalar_ptr(norm, torch.float32, index, "norm"), scratch=gl._reduce_bytes)


def fs_adamw_step_clip(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, grad: torch.Tensor,
                       param_bf16: Optional[torch.Tensor] = None, *, total: torch.Tensor, max_norm: float,
                       norm_type=2.0, norm_eps: float = 1e-6, lr: float = 1e-3, beta1: float = 0.9,
                       beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01, step: int = 1,
                       stream=None):
    """fs_adamw_step on the gradient times min(1, max_norm / (norm_of(total) +
    norm_eps)), applied as the gradient is read."""
    kind = _norm_code(norm_type)
    n, index = master.numel(), master.get_device()
    f32, bf16 = torch.float32, torch.bfloat16
    gdt = bf16 if grad.dtype is bf16 else f32
    ptrs = []
    for name, t, dt in (("master", master, f32), ("exp_avg", exp_avg, f32), ("exp_avg_sq", exp_avg_sq, f32),
                        ("grad", grad, gdt), ("param_bf16", param_bf16, bf16)):
        if t is None and name == "param_bf16":
            ptrs.append(None)
            continue
        if t.dtype is not dt or t.numel() != n:
            raise ValueError(f"fs_adamw_step_clip: {name} must be {'float32 or bfloat16' if name == 'grad' else dt} "
                             f"with {n} elements")
        if t.get_device() != index:
            raise ValueError(f"fs_adamw_step_clip: {name} is on {t.device}, master on {master.device}")
        ptrs.append(t.data_ptr() if t.is_contiguous() else _dev_ptr(t, name))
    clip = Clip(_scalar_ptr(total, torch.float64, index, "total"), max_norm, norm_eps, kind)
    if index < 0:
        _dev_ptr(master, "master")      # raises
    hp = AdamWHparams(lr, beta1, beta2, eps, weight_decay, 0, int(step))
    _launch(index, stream, lib().fs_adamw_step_clip, n, *ptrs[:4], FS_BF16 if gdt is bf16 else FS_FP32, ptrs[4],
            ctypes.byref(hp), ctypes.byref(clip))


# ------------------------------------------------ microscaled 4-bit shards --

MX4_BLOCK = 32   # elements of a block: 16 bytes of codes and one scale byte


class Mx4MatrixStruct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("code_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("chunk_rows", ctypes.c_int64), ("chunk_stride", ctypes.c_int64)]


class Mx4PlanInfo(ctypes.Structure):
    _fields_ = [("shard_blocks", ctypes.c_int64), ("shard_bytes", ctypes.c_int64),
                ("gathered_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64)]


def _bytes_rows(t: torch.Tensor, width: int, what: str):
    if t.dtype is not torch.uint8 or t.dim() != 2 or t.shape[1] != width:
        raise ValueError(f"{what} must be a uint8 matrix of {width} columns")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor")
    if t.shape[1] > 1 and t.numel() and t.stride(1) != 1:
        raise ValueError(f"{what}: the bytes of a row must follow each other")


class Mx4Matrix:
    """A matrix of 4-bit blocks along its rows: codes (uint8, rows by 16 for
    each block of 32 elements) and scales (uint8, rows by one a block), each
    with any row stride (codes: a multiple of 16 bytes).  `cols` counts
    elements; the last block of a row may be partly filled, with zeros after
    the last element."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        nb = -(-int(cols) // MX4_BLOCK)
        if cols < 0:
            raise ValueError("cols must be >= 0")
        _bytes_rows(codes, 16 * nb, "codes")
        _bytes_rows(scales, nb, "scales")
        if codes.shape[0] != scales.shape[0] or codes.device != scales.device:
            raise ValueError("codes and scales must have the same rows, on the same GPU")
        self.codes: Optional[torch.Tensor] = codes
        self.scales: Optional[torch.Tensor] = scales
        self._hold(Mx4MatrixStruct(codes.data_ptr(), scales.data_ptr(), codes.shape[0], int(cols), codes.stride(0),
                                   scales.stride(0), 0, 0), codes.get_device(), (codes, scales))

    def _hold(self, m: Mx4MatrixStruct, index: int, tensors):
        self._m, self._ref, self._index = m, ctypes.byref(m), index
        self._tensors = [(t, t.data_ptr()) for t in tensors]
        self.shape = (m.rows, m.cols)

    @classmethod
    def _gathered(cls, m: Mx4MatrixStruct, gathered: torch.Tensor) -> "Mx4Matrix":
        self = cls.__new__(cls)
        self.codes = self.scales = None     # in the gathered buffer, chunk by chunk
        self._hold(m, gathered.get_device(), (gathered,))
        return self

    def _on(self, index: int, name: str):
        """The matrix for a call on GPU `index`."""
        if self._index != index:
            raise ValueError(f"{name} is on GPU {self._index}, the other arguments on cuda:{index}")
        for t, ptr in self._tensors:
            if t.data_ptr() != ptr:
                raise ValueError("the matrix's tensors no longer have the memory they had when it was made")
        return self._ref


def fs_mx4_empty(rows: int, cols: int, device="cuda") -> Mx4Matrix:
    """Memory for a (rows, cols) matrix of 4-bit blocks, uninitialized."""
    nb = -(-int(cols) // MX4_BLOCK)
    return Mx4Matrix(torch.empty(rows, 16 * nb, dtype=torch.uint8, device=device),
                     torch.empty(rows, nb, dtype=torch.uint8, device=device), cols)


def _plain_matrix(t: torch.Tensor, what: str) -> tuple:
    """(rows, columns, address, dtype code, row stride, GPU) of a matrix whose rows are contiguous."""
    code, index = _DTYPE_CODES.get(t.dtype), t.get_device()
    if code is None or t.dim() != 2:
        raise ValueError(f"{what} must be a bfloat16 or float32 matrix")
    if index < 0:
        raise ValueError(f"{what} must be a GPU tensor")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if step != 1 and cols > 1 and rows:
        raise ValueError(f"{what}: the elements of a row must follow each other")
    return rows, cols, t.data_ptr(), code, ld, index


def fs_mx4_quantize(x: torch.Tensor, by_row: Optional[Mx4Matrix] = None, by_col: Optional[Mx4Matrix] = None, *,
                    seed: Optional[torch.Tensor] = None, stream=None):
    """Quantise a matrix (bf16 or fp32, any row stride) in blocks along its
    rows into by_row, along its columns into by_col (the transpose's shape),
    or both in one pass.  seed: None rounds to nearest; one int64 on the GPU
    rounds stochastically by it, read when the kernel runs."""
    rows, cols, ptr, code, ld, index = _plain_matrix(x, "x")
    row = col = None
    if by_row is not None:
        row = by_row._on(index, "by_row")
    if by_col is not None:
        col = by_col._on(index, "by_col")
    _launch(index, stream, lib().fs_mx4_quantize, rows, cols, ptr, code, ld, row, col,
            None if seed is None else _scalar_ptr(seed, torch.int64, index, "seed"))


def fs_mx4_dequantize(m: Mx4Matrix, out: torch.Tensor, *, stream=None):
    """The values of a matrix of 4-bit blocks, as bf16 or fp32 (out's type)."""
    rows, cols, ptr, code, ld, index = _plain_matrix(out, "out")
    if (rows, cols) != m.shape:
        raise ValueError(f"fs_mx4_dequantize: out must be {m.shape}")
    _launch(index, stream, lib().fs_mx4_dequantize, m._on(index, "the matrix"), ptr, code, ld)


def fs_mx4_matmul(a: Mx4Matrix, b: Mx4Matrix, out: torch.Tensor, *, stream=None):
    """out = a b^T (bf16 or fp32, any row stride): a is (m, k), b (n, k), out
    (m, n).  Summed in fp32."""
    m, n, ptr, code, ld, index = _plain_matrix(out, "out")
    if a.shape[1] != b.shape[1] or a.shape[0] != m or b.shape[0] != n:
        raise ValueError(f"fs_mx4_matmul: a {a.shape} by b {b.shape} transposed does not give {tuple(out.shape)}")
    _launch(index, stream, lib().fs_mx4_matmul, a._on(index, "a"), b._on(index, "b"), ptr, code, ld)


class Mx4Plan:
    """The layout of a group's quantised shards (wraps fs_mx4_plan_t).  To be
    kept like a Plan."""

    def __init__(self, plan: Plan):
        h = ctypes.c_void_p()
        _check(lib().fs_mx4_plan(plan._h, ctypes.byref(h)))
        self._h = h
        self._destroy = lib().fs_mx4_plan_destroy
        info = Mx4PlanInfo()
        _check(lib().fs_mx4_plan_info(h, ctypes.byref(info)))
        self.plan = plan
        self.shard_blocks, self.shard_bytes = info.shard_blocks, info.shard_bytes
        self.gathered_bytes, self.workspace_bytes = info.gathered_bytes, info.workspace_bytes
        self.workspace: Optional[torch.Tensor] = None
        self._table: Optional[_Table] = None    # the workspace and who reads it
        self._earlier: list = []                # those on other GPUs, which launches and captured graphs may still read

    def close(self):
        h = self.__dict__.pop("_h", None)
        if h is not None and h.value:
            self._destroy(h)

    def __del__(self):
        self.close()

    def upload(self, device="cuda", stream=None) -> "Mx4Plan":
        """As Plan.upload."""
        where = torch.device(device)
        if where.type != "cuda":
            raise ValueError(f"fs_mx4_plan: the tables go to a GPU, not to {where}")
        _put(self, lib().fs_mx4_plan_upload, self.workspace_bytes, where, stream)
        return self

    def piece(self, i: int, rank: int) -> tuple:
        """(first block in the rank's shard, element count) of parameter i."""
        b, n = ctypes.c_int64(), ctypes.c_int64()
        _check(lib().fs_mx4_plan_piece(self._h, int(i), int(rank), ctypes.byref(b), ctypes.byref(n)))
        return b.value, n.value

    def matrix(self, gathered: torch.Tensor, i: int) -> Mx4Matrix:
        """Parameter i where it lies in a gathered buffer (FSDP2, rows of whole blocks)."""
        self._bytes(gathered, self.gathered_bytes, "gathered")
        m = Mx4MatrixStruct()
        _check(lib().fs_mx4_plan_matrix(self._h, gathered.data_ptr(), int(i), ctypes.byref(m)))
        return Mx4Matrix._gathered(m, gathered)

    @staticmethod
    def _bytes(t: torch.Tensor, n: int, what: str) -> int:
        if t.dtype is not torch.uint8 or t.numel() != n:
            raise ValueError(f"{what} must be uint8 with {n} elements")
        return _dev_ptr(t, what)

    def _params(self, tensors, what: str, index: int, stream) -> tuple:
        """(pointer table, its address, dtype code).  The caller holds the table until it has launched: another
        thread's calls may release it from the plan's."""
        if not tensors:
            return None, 0, FS_BF16
        if len(set(map(_DTYPE, tensors))) > 1 or set(map(_GET_DEVICE, tensors)) != {index}:
            raise ValueError(f"{what} must share one dtype, on the buffer's GPU")
        code = _dtype_code(tensors[0].dtype)
        tab = self.plan.ptr_table(tensors, what, elem_bytes=tensors[0].element_size(), stream=stream, known=True)
        return tab, tab.data_ptr(), code


def fs_mx4_plan(plan: Plan) -> Mx4Plan:
    """Lay out the quantised shards of a plan's group (fs_mx4_plan)."""
    return Mx4Plan(plan)


def fs_pack_mx4(mp: Mx4Plan, params: Sequence[torch.Tensor], out: torch.Tensor, rank: int = -1, *,
                seed: Optional[torch.Tensor] = None, stream=None):
    """All-gather copy-in in 4 bits: params (bf16 or fp32) -> out (uint8: the
    whole gathered buffer, or rank's shard).  seed: as in fs_mx4_quantize."""
    ptr = mp._bytes(out, mp.gathered_bytes if rank < 0 else mp.shard_bytes, "out")
    index = out.get_device()
    _held, tab, code = mp._params(params, "params", index, stream)
    _launch(index, stream, lib().fs_pack_mx4, mp._h, tab, code, ptr, int(rank),
            None if seed is None else _scalar_ptr(seed, torch.int64, index, "seed"), table=mp._table)


def fs_unpack_mx4(mp: Mx4Plan, gathered: torch.Tensor, params: Sequence[torch.Tensor], *, stream=None):
    """All-gather copy-out of 4 bits: gathered -> params (bf16 or fp32)."""
    ptr = mp._bytes(gathered, mp.gathered_bytes, "gathered")
    index = gathered.get_device()
    _held, tab, code = mp._params(params, "params", index, stream)
    _launch(index, stream, lib().fs_unpack_mx4, mp._h, ptr, tab, code, table=mp._table)


def fs_reduce_shard_mx4(mp: Mx4Plan, slices, out: torch.Tensor, *, rank: int, grad_acc: int = 1, stream=None):
    """Average slices[j*world + k] (uint8, each rank's quantised shard; a
    sequence, or one tensor of a row a slice) into out (fp32, shard_numel)."""
    n, terms = mp.plan.info.shard_numel, mp.plan.info.world * int(grad_acc)
    if out.dtype is not torch.float32 or out.numel() != n:
        raise ValueError(f"fs_reduce_shard_mx4: out must be float32 with {n} elements")
    if len(slices) != terms:
        raise ValueError(f"fs_reduce_shard_mx4: need world*grad_acc = {terms} slices")
    index, ptr = out.get_device(), _dev_ptr(out, "out")
    if isinstance(slices, torch.Tensor):
        if slices.dim() != 2 or slices.dtype is not torch.uint8 or slices.shape[1] != mp.shard_bytes or (
                slices.numel() and slices.stride(1) != 1):
            raise ValueError(f"fs_reduce_shard_mx4: slices must be uint8 rows of {mp.shard_bytes} bytes")
        if slices.get_device() != index:
            raise ValueError(f"fs_reduce_shard_mx4: out is on {out.device}, the slices on {slices.device}")
        base, step = slices.data_ptr(), slices.stride(0)
        ptrs = [base + k * step for k in range(terms)]
    else:
        ptrs = [mp._bytes(s, mp.shard_bytes, f"slices[{k}]") for k, s in enumerate(slices)]
        if any(s.get_device() != index for s in slices):
            raise ValueError(f"fs_reduce_shard_mx4: a slice is not on {out.device}")
    _launch(index, stream, lib().fs_reduce_shard_mx4, mp._h, int(rank), int(grad_acc),
            (ctypes.c_void_p * max(1, terms))(*ptrs), ptr, table=mp._table)


def fs_copy_bytes(dst: torch.Tensor, src: torch.Tensor, stream=None):
    """Plain streaming copy (measurement aid): src -> dst, same byte size."""
    nb = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nb:
        raise ValueError("fs_copy_bytes: size mismatch")
    _check(lib().fs_copy_bytes(_dev_ptr(dst, "dst"), _dev_ptr(src, "src"), nb, _stream(stream)))


def fs_stream_read(src: torch.Tensor, sink: torch.Tensor, stream=None):
    """Read-only stream over src's bytes (measurement aid); sink: a device
    tensor of at least 4 bytes that may receive an unspecified value."""
    if sink.numel() * sink.element_size() < 4:
        raise ValueError("fs_stream_read: sink needs 4 bytes")
    _check(lib().fs_stream_read(_dev_ptr(src, "src"), src.numel() * src.element_size(), _dev_ptr(sink, "sink"),
                                _stream(stream)))


def fs_stream_fill(dst: torch.Tensor, value: int, stream=None):
    """Write-only stream: every 32-bit word of dst becomes `value` (measurement aid)."""
    _check(lib().fs_stream_fill(_dev_ptr(dst, "dst"), dst.numel() * dst.element_size(), int(value) & 0xFFFFFFFF,
                                _stream(stream)))

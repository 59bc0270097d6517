"""Python binding of libtide (include/tide.h): argument marshalling only.

Every step of the reduce-scatter local stage, the all-gather copy-out and
copy-in, and the stock gradient pack runs in the HIP library; this module turns torch tensors into device pointers and
the current HIP stream, checks that each tensor has the size, dtype, device
and contiguity the plan expects (so that no kernel is launched on a buffer
smaller than the plan assumes), and raises on a non-zero status.  There is no
fallback: without the compiled library, importing this module fails.
"""
import ctypes
import functools
import os

import numpy as np

# PyTorch ships its own HIP runtime under the same soname as the system's, and
# whichever copy a process loads first serves every library in it.  torch is
# imported before the library is loaded, so that torch and this library share
# one runtime (its devices, memory and streams).
import torch  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libtide.so")

TIDE_OK = 0
STATUS_NAMES = {
    0: "TIDE_OK",
    -1: "TIDE_ERR_INVALID",
    -2: "TIDE_ERR_RANGE",
    -3: "TIDE_ERR_ALIGN",
    -4: "TIDE_ERR_NOMEM",
    -5: "TIDE_ERR_HIP",
    -6: "TIDE_ERR_UNSUPPORTED",
}
FLAG_CACHED_LOADS = 0x1
FLAG_CACHED_STORES = 0x2
FLAG_NO_LDS = 0x4
DTYPE_BF16 = 0
DTYPE_F32 = 1
CODE_E4M3 = 0
CODE_INT8 = 1
MAX_WORLD = 256
NOALLOC_SCRATCH_BYTES = 1 << 20

# Every symbol include/tide.h declares.
EXPORTS = (
    "tide_plan_create",
    "tide_plan_layout",
    "tide_plan_sizes",
    "tide_plan_segments",
    "tide_plan_set_options",
    "tide_plan_get_options",
    "tide_plan_launches",
    "tide_plan_paths",
    "tide_reduce_scatter_local",
    "tide_reduce_scatter_local_noalloc",
    "tide_allgather_copyout",
    "tide_allgather_copyin",
    "tide_reduce_scatter_local_f32",
    "tide_stock_chunk_cat",
    "tide_checkpoint_layout",
    "tide_checkpoint_pack",
    "tide_checkpoint_unpack",
    "tide_checkpoint_weight_grad_workspace",
    "tide_checkpoint_weight_grad",
    "tide_vocab_loss_workspace",
    "tide_vocab_loss",
    "tide_vocab_loss_grad",
    "tide_device_info",
    "tide_probe_launch",
    "tide_victim_axpb",
    "tide_stream_create",
    "tide_stream_destroy",
    "tide_plan_destroy",
    "tide_last_error",
)


class TideError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class Options(ctypes.Structure):
    _fields_ = [("cu_budget", ctypes.c_int32), ("wg_per_cu", ctypes.c_int32),
                ("chunk_elems", ctypes.c_int64), ("flags", ctypes.c_uint32), ("wave_chunks", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIBRARY):
        raise ImportError(f"{LIBRARY} is missing: build it with `python param_collectives_amd/build.py` "
                          "(the HIP path has no fallback)")
    lib = ctypes.CDLL(LIBRARY)
    vp, i32, i64, i64p = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)
    lib.tide_plan_create.argtypes = [i32, i32, ctypes.POINTER(i32), i64p, ctypes.POINTER(Options),
                                     ctypes.POINTER(vp)]
    lib.tide_plan_layout.argtypes = [vp, i64p, i64p, i64p]
    lib.tide_plan_sizes.argtypes = [vp, i64p, i64p]
    lib.tide_plan_segments.argtypes = [vp, i32, i64p, i64, i64p]
    lib.tide_plan_set_options.argtypes = [vp, ctypes.POINTER(Options)]
    lib.tide_plan_get_options.argtypes = [vp, i32, ctypes.POINTER(Options)]
    lib.tide_plan_launches.argtypes = [vp, i32, i32, i64p, i64, i64p]
    lib.tide_plan_paths.argtypes = [vp, i32, i64p]
    lib.tide_reduce_scatter_local.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.c_float, i32, vp]
    lib.tide_allgather_copyout.argtypes = [vp, vp, ctypes.POINTER(vp), vp]
    lib.tide_allgather_copyin.argtypes = [vp, ctypes.POINTER(vp), i32, vp, vp]
    lib.tide_reduce_scatter_local_f32.argtypes = lib.tide_reduce_scatter_local.argtypes
    lib.tide_reduce_scatter_local_noalloc.argtypes = lib.tide_reduce_scatter_local.argtypes
    lib.tide_stock_chunk_cat.argtypes = [vp, ctypes.POINTER(vp), vp, vp]
    f32 = ctypes.c_float
    lib.tide_checkpoint_layout.argtypes = [i64, i64p, i64p]
    lib.tide_checkpoint_pack.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, vp]
    lib.tide_checkpoint_unpack.argtypes = [vp, vp, i32, i64, i64, vp, i32, i64, vp]
    lib.tide_checkpoint_weight_grad_workspace.argtypes = [vp, i64, i64, i64, i64, i64p]
    lib.tide_checkpoint_weight_grad.argtypes = [vp, i64, i64, i64, vp, vp, i32, i64, vp, i32, f32, i32, vp, i64, vp]
    lib.tide_vocab_loss_workspace.argtypes = [vp, i64, vp, i64, i64, i64, i64, i32, i32, i64p]
    lib.tide_vocab_loss.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, vp, vp, vp, i64, vp]
    lib.tide_vocab_loss_grad.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, vp, vp, vp, vp, i32, i32, vp, i64, vp]
    i32p = ctypes.POINTER(i32)
    lib.tide_device_info.argtypes = [i32p, i32p, i32p, i32p]
    lib.tide_probe_launch.argtypes = [vp, i32, i32, i64, vp]
    lib.tide_victim_axpb.argtypes = [vp, vp, i64, ctypes.c_float, ctypes.c_float, vp]
    lib.tide_stream_create.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32, ctypes.POINTER(vp)]
    lib.tide_stream_destroy.argtypes = [vp]
    lib.tide_plan_destroy.argtypes = [vp]
    lib.tide_plan_destroy.restype = None
    lib.tide_last_error.argtypes = []
    lib.tide_last_error.restype = ctypes.c_char_p
    for name in EXPORTS[:-2]:
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()


def _check(status):
    if status != TIDE_OK:
        raise TideError(status, lib.tide_last_error().decode(errors="replace"))


def _options(cu_budget=0, wg_per_cu=0, chunk_elems=0, flags=0, wave_chunks=0):
    return Options(int(cu_budget), int(wg_per_cu), int(chunk_elems), int(flags), int(wave_chunks))


def _ptr_array(values):
    return (ctypes.c_void_p * max(len(values), 1))(*[int(v) if v else None for v in values])


class Plan:
    """A shard-layout plan for `world` simulated ranks and the given parameter
    shapes (tide_plan_create)."""

    def __init__(self, world, shapes, cu_budget=0, wg_per_cu=0, chunk_elems=0, flags=0, wave_chunks=0):
        self.world = int(world)
        self.shapes = [tuple(int(d) for d in s) for s in shapes]
        ndims = (ctypes.c_int32 * max(len(self.shapes), 1))(*[len(s) for s in self.shapes])
        flat = [d for s in self.shapes for d in s]
        dims = (ctypes.c_int64 * max(len(flat), 1))(*flat)
        handle = ctypes.c_void_p()
        opt = _options(cu_budget, wg_per_cu, chunk_elems, flags, wave_chunks)
        _check(lib.tide_plan_create(self.world, len(self.shapes), ndims, dims, ctypes.byref(opt),
                                    ctypes.byref(handle)))
        self.handle = handle
        R = np.zeros(len(self.shapes), dtype=np.int64)
        o = np.zeros(len(self.shapes), dtype=np.int64)
        S = np.zeros(1, dtype=np.int64)
        _check(lib.tide_plan_layout(self.handle, R.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                    o.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                    S.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))))
        self.rows_per_rank, self.shard_offset, self.shard_elems = R, o, int(S[0])
        # element counts as the library sizes them: numel[p] of parameter p,
        # n_real[r][p] of rank r's shard of p (its real, non-padding elements)
        numel = np.zeros(len(self.shapes), dtype=np.int64)
        real = np.zeros(self.world * len(self.shapes), dtype=np.int64)
        _check(lib.tide_plan_sizes(self.handle, numel.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                   real.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))))
        self.numel = [int(v) for v in numel]
        self.n_real = real.reshape(self.world, len(self.shapes)).tolist()

    def segments(self, op):
        """The work segments (op 0: reduce-scatter, 1: copy-out, 2: copy-in,
        3: stock pack, 4: reduce-scatter of fp32 gradients) as an int64 array
        of rows (kind, src_idx, dst_idx, src_off, dst_off, len)."""
        count = ctypes.c_int64()
        _check(lib.tide_plan_segments(self.handle, int(op), None, 0, ctypes.byref(count)))
        table = np.zeros((max(count.value, 1), 6), dtype=np.int64)
        _check(lib.tide_plan_segments(self.handle, int(op), table.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                      count.value, ctypes.byref(count)))
        return table[:count.value]

    def launches(self, op=0, cu_count=0):
        """The kernel launches one call of `op` makes under the current
        options, as an int64 array of rows (first chunk, end chunk, first
        segment, end segment, workgroups); cu_count stands for a cu_budget of
        0 (0: the bound device's CU count)."""
        count = ctypes.c_int64()
        _check(lib.tide_plan_launches(self.handle, int(op), int(cu_count), None, 0, ctypes.byref(count)))
        table = np.zeros((max(count.value, 1), 5), dtype=np.int64)
        _check(lib.tide_plan_launches(self.handle, int(op), int(cu_count),
                                      table.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), count.value,
                                      ctypes.byref(count)))
        return table[:count.value]

    def paths(self, op=0):
        """Elements of the latest call of `op` by code path (tide_plan_paths):
        dict of vector, realigned and element-by-element counts, and whether a
        reduce-scatter ran its realigning instance."""
        out = np.zeros(4, dtype=np.int64)
        _check(lib.tide_plan_paths(self.handle, int(op), out.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))))
        return {"vector": int(out[0]), "realigned": int(out[1]), "element": int(out[2]),
                "realigning_instance": bool(out[3])}

    def set_options(self, cu_budget=0, wg_per_cu=0, chunk_elems=0, flags=0, wave_chunks=0):
        opt = _options(cu_budget, wg_per_cu, chunk_elems, flags, wave_chunks)
        _check(lib.tide_plan_set_options(self.handle, ctypes.byref(opt)))

    def options(self, op=0):
        """Effective launch knobs for op 0 (reduce-scatter), 1 (copy-out),
        2 (copy-in), 3 (stock pack) or 4 (reduce-scatter of fp32 gradients)."""
        opt = Options()
        _check(lib.tide_plan_get_options(self.handle, int(op), ctypes.byref(opt)))
        return {"cu_budget": opt.cu_budget, "wg_per_cu": opt.wg_per_cu, "chunk_elems": opt.chunk_elems,
                "flags": opt.flags, "wave_chunks": opt.wave_chunks}

    def destroy(self):
        if getattr(self, "handle", None):
            lib.tide_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    # ------------------------------------------------------------ raw calls

    @staticmethod
    def _lengths(values, n, what):
        # the library reads exactly n entries of each pointer array
        if len(values) != n:
            raise ValueError(f"{what} must hold {n} addresses, got {len(values)}")

    def reduce_scatter_local_raw(self, grad_ptrs, out_ptrs, alpha=1.0, accumulate=0, stream=0, f32=False):
        """tide_reduce_scatter_local (bf16 gradients) or, with f32=True,
        tide_reduce_scatter_local_f32 on raw device addresses: grad_ptrs[u*P+p],
        out_ptrs[r] (ints), stream a hipStream_t handle (int)."""
        self._lengths(grad_ptrs, self.world * len(self.shapes), "grad_ptrs")
        self._lengths(out_ptrs, self.world, "out_ptrs")
        fn = lib.tide_reduce_scatter_local_f32 if f32 else lib.tide_reduce_scatter_local
        _check(fn(self.handle, _ptr_array(grad_ptrs), _ptr_array(out_ptrs), float(alpha), int(accumulate),
                  ctypes.c_void_p(int(stream) or None)))

    def stock_chunk_cat_raw(self, grad_ptrs, packed_ptr, stream=0):
        """tide_stock_chunk_cat on raw device addresses (grad_ptrs[p] of one
        rank, packed_ptr to W*S fp32 elements)."""
        self._lengths(grad_ptrs, len(self.shapes), "grad_ptrs")
        _check(lib.tide_stock_chunk_cat(self.handle, _ptr_array(grad_ptrs), ctypes.c_void_p(int(packed_ptr) or None),
                                        ctypes.c_void_p(int(stream) or None)))

    def allgather_copyin_raw(self, shard_ptrs, shard_dtype, rank_major_ptr, stream=0):
        """tide_allgather_copyin on raw device addresses (shard_ptrs[r*P+p])."""
        self._lengths(shard_ptrs, self.world * len(self.shapes), "shard_ptrs")
        _check(lib.tide_allgather_copyin(self.handle, _ptr_array(shard_ptrs), int(shard_dtype),
                                         ctypes.c_void_p(int(rank_major_ptr) or None),
                                         ctypes.c_void_p(int(stream) or None)))

    def allgather_copyout_raw(self, rank_major_ptr, param_ptrs, stream=0):
        """tide_allgather_copyout on raw device addresses."""
        self._lengths(param_ptrs, len(self.shapes), "param_ptrs")
        _check(lib.tide_allgather_copyout(self.handle, ctypes.c_void_p(int(rank_major_ptr) or None),
                                          _ptr_array(param_ptrs), ctypes.c_void_p(int(stream) or None)))


# The current stream's handle alone (building torch.cuda.current_stream()'s object
# takes longer than a launch) and torch.cuda.current_device() without its check
# that there is one, or the public calls in a torch that lacks these.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_handle(stream):
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return int(stream.cuda_stream)


def _require(t, dtype, numel, what):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what}: expected a GPU tensor, got {t.device}")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{what}: lives on {t.device}, but the kernels run on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    if t.numel() != numel:
        raise ValueError(f"{what}: expected {numel} elements, got {t.numel()}")


class Call:
    """One operation with its tensors checked and its pointer arrays
    marshalled once (the buffers an FSDP2 group reuses every step); calling it
    launches on the given (or current) stream with a single library call.
    It holds references to the tensors, so they outlive it."""

    def __init__(self, fn, args, tensors):
        self._fn = fn
        self._args = args
        self._tensors = tensors

    def __call__(self, stream=None):
        _check(self._fn(*self._args, ctypes.c_void_p(_stream_handle(stream) or None)))


class TensorCall(Call):
    """A Call without a plan, which would be bound to its device: it is launched
    on the device it was made on only."""

    def __init__(self, fn, args, tensors):
        super().__init__(fn, args, tensors)
        self._device = _current_device()

    def __call__(self, stream=None):
        self._on_its_device()
        _check(self._fn(*self._args, _device_stream(stream)))

    def _on_its_device(self):
        if _current_device() != self._device:
            raise ValueError(f"the call was made on cuda:{self._device}, but the current device is "
                             f"cuda:{_current_device()}")


class WorkspaceCall(TensorCall):
    """A TensorCall of an operation with a workspace: the caller's, or one that
    each launch takes for itself on the stream it runs on.  A launch of its own
    workspace may overlap others on other streams, the object may be dropped
    while it runs, and one that is captured takes it from the graph's memory."""

    def __init__(self, fn, args, tensors, nbytes, workspace):
        super().__init__(fn, args, tensors)
        self._bytes = nbytes
        self._workspace = workspace
        if workspace is not None:
            _workspace(nbytes, workspace, None)  # its checks

    def __call__(self, stream=None):
        self._on_its_device()
        handle = _device_stream(stream)
        ws, nbytes, keep = _workspace(self._bytes, self._workspace, stream)
        _check(self._fn(*self._args, ws, nbytes, handle))


def _rs_checked(plan, grads, outs):
    """Checks the tensors of a reduce-scatter; returns (gradient pointers,
    output pointers, whether the gradients are fp32)."""
    import torch

    W, P = plan.world, len(plan.shapes)
    if len(grads) != W or any(len(row) != P for row in grads):
        raise ValueError(f"grads must be {W} lists of {P} tensors")
    if len(outs) != W:
        raise ValueError(f"outs must hold {W} tensors")
    dtypes = {t.dtype for row in grads for t in row}
    if dtypes not in ({torch.float32}, {torch.bfloat16}):
        raise TypeError(f"grads must be all torch.bfloat16 or all torch.float32, got {dtypes}")
    dtype = dtypes.pop()
    ptrs = []
    for u in range(W):
        for p in range(P):
            _require(grads[u][p], dtype, plan.numel[p], f"grads[{u}][{p}]")
            ptrs.append(grads[u][p].data_ptr())
    for r in range(W):
        _require(outs[r], torch.float32, plan.shard_elems, f"outs[{r}]")
    return ptrs, [o.data_ptr() for o in outs], dtype == torch.float32


def reduce_scatter_call(plan, grads, outs, alpha=1.0, accumulate=False):
    """A registered reduce-scatter (see reduce_scatter_local)."""
    g, o, f32 = _rs_checked(plan, grads, outs)
    fn = lib.tide_reduce_scatter_local_f32 if f32 else lib.tide_reduce_scatter_local
    return Call(fn, (plan.handle, _ptr_array(g), _ptr_array(o), ctypes.c_float(alpha), int(bool(accumulate))),
                (plan, grads, outs))


def reduce_scatter_local(plan, grads, outs, alpha=1.0, accumulate=False, stream=None):
    """Reduce-scatter local stage: grads[u][p] (all bf16 or all fp32,
    plan.shapes[p]) for u in [0, W) -> outs[r] (fp32, plan.shard_elems
    elements) for r in [0, W): outs[r] = alpha * (sum over u in rank order),
    added to the old outs[r] when accumulate is true."""
    g, o, f32 = _rs_checked(plan, grads, outs)
    plan.reduce_scatter_local_raw(g, o, alpha, int(bool(accumulate)), _stream_handle(stream), f32=f32)


def reduce_scatter_local_noalloc(plan, grads, outs, alpha=1.0, accumulate=False, stream=None):
    """The allocation-free reduce-scatter (tide_reduce_scatter_local_noalloc):
    the results of reduce_scatter_local from bf16 gradients, with the call's
    tables written to the library's fixed device scratch array instead of
    plan-owned device memory.  Calls that may overlap on one device race for
    that array."""
    g, o, f32 = _rs_checked(plan, grads, outs)
    if f32:
        raise TypeError("the allocation-free reduce-scatter takes bf16 gradients")
    _check(lib.tide_reduce_scatter_local_noalloc(plan.handle, _ptr_array(g), _ptr_array(o), ctypes.c_float(alpha),
                                                 int(bool(accumulate)),
                                                 ctypes.c_void_p(_stream_handle(stream) or None)))


def _pk_checked(plan, grads, packed):
    import torch

    P = len(plan.shapes)
    if len(grads) != P:
        raise ValueError(f"grads must hold {P} tensors (one rank's gradients)")
    for p in range(P):
        _require(grads[p], torch.bfloat16, plan.numel[p], f"grads[{p}]")
    _require(packed, torch.float32, plan.world * plan.shard_elems, "packed")
    return [t.data_ptr() for t in grads], packed.data_ptr()


def stock_chunk_cat_call(plan, grads, packed):
    """A registered stock gradient pack (see stock_chunk_cat)."""
    g, pk = _pk_checked(plan, grads, packed)
    return Call(lib.tide_stock_chunk_cat, (plan.handle, _ptr_array(g), ctypes.c_void_p(pk or None)),
                (plan, grads, packed))


def stock_chunk_cat(plan, grads, packed, stream=None):
    """Stock gradient pack of one rank: grads[p] (bf16, plan.shapes[p]) ->
    packed (fp32, W*S elements: rank r's rows of p at r*S + o_p, widened,
    padding +0)."""
    g, pk = _pk_checked(plan, grads, packed)
    plan.stock_chunk_cat_raw(g, pk, _stream_handle(stream))


def _co_checked(plan, rank_major, params):
    import torch

    P = len(plan.shapes)
    _require(rank_major, torch.bfloat16, plan.world * plan.shard_elems, "rank_major")
    if len(params) != P:
        raise ValueError(f"params must hold {P} tensors")
    for p in range(P):
        _require(params[p], torch.bfloat16, plan.numel[p], f"params[{p}]")
    return rank_major.data_ptr(), [t.data_ptr() for t in params]


def allgather_copyout_call(plan, rank_major, params):
    """A registered copy-out (see allgather_copyout)."""
    rm, ps = _co_checked(plan, rank_major, params)
    return Call(lib.tide_allgather_copyout, (plan.handle, ctypes.c_void_p(rm or None), _ptr_array(ps)),
                (plan, rank_major, params))


def allgather_copyout(plan, rank_major, params, stream=None):
    """All-gather copy-out: rank_major (bf16, W*S elements) -> params[p]
    (bf16, plan.shapes[p])."""
    rm, ps = _co_checked(plan, rank_major, params)
    plan.allgather_copyout_raw(rm, ps, _stream_handle(stream))


def _ci_checked(plan, shards, rank_major):
    import torch

    W, P = plan.world, len(plan.shapes)
    if len(shards) != W or any(len(row) != P for row in shards):
        raise ValueError(f"shards must be {W} lists of {P} tensors")
    dtypes = {t.dtype for row in shards for t in row}
    if dtypes not in ({torch.float32}, {torch.bfloat16}):
        raise TypeError(f"shards must be all torch.float32 or all torch.bfloat16, got {dtypes}")
    dtype = dtypes.pop()
    ptrs = []
    for r in range(W):
        for p in range(P):
            _require(shards[r][p], dtype, plan.n_real[r][p], f"shards[{r}][{p}]")
            ptrs.append(shards[r][p].data_ptr())
    _require(rank_major, torch.bfloat16, W * plan.shard_elems, "rank_major")
    return ptrs, DTYPE_F32 if dtype == torch.float32 else DTYPE_BF16, rank_major.data_ptr()


def allgather_copyin_call(plan, shards, rank_major):
    """A registered copy-in (see allgather_copyin)."""
    ptrs, dt, rm = _ci_checked(plan, shards, rank_major)
    return Call(lib.tide_allgather_copyin, (plan.handle, _ptr_array(ptrs), dt, ctypes.c_void_p(rm or None)),
                (plan, shards, rank_major))


def allgather_copyin(plan, shards, rank_major, stream=None):
    """All-gather copy-in: shards[r][p] (rank r's local shard of parameter p,
    n_real(p, r) elements, all float32 or all bfloat16) -> rank_major (bf16,
    W*S elements; fp32 shards are cast by round to nearest even)."""
    ptrs, dt, rm = _ci_checked(plan, shards, rank_major)
    plan.allgather_copyin_raw(ptrs, dt, rm, _stream_handle(stream))


# ------------------------------------------------------------ activation checkpoints

_BF16 = (torch.bfloat16,)
_FLOATS = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}
_CODES = {torch.float8_e4m3fn: CODE_E4M3, torch.int8: CODE_INT8}


def _device_stream(stream):
    """The handle of a stream (None: the current one) of the current device."""
    if stream is not None and getattr(stream, "device_index", None) not in (None, _current_device()):
        raise ValueError(f"the stream is one of cuda:{stream.device_index}, but the kernels run on the current device "
                         f"cuda:{_current_device()}")
    return _stream_handle(stream)


def _on_device(t, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    device = t.get_device()  # -1 on the host
    if device < 0:
        raise ValueError(f"{what}: expected a GPU tensor, got {t.device}")
    if device != _current_device():
        raise ValueError(f"{what}: lives on {t.device}, but the kernels run on the current device "
                         f"cuda:{_current_device()}")


def _matrix(t, dtypes, what, strided=True):
    """(address, rows, columns, row stride) of a matrix of one of `dtypes`
    whose rows are contiguous; without `strided` they have no gaps."""
    _on_device(t, what)
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a matrix, got {t.dim()} dimensions")
    rows, cols = t.shape
    if t.is_contiguous():
        return t.data_ptr(), rows, cols, cols
    # the stride of a dimension of one element says nothing
    stride = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or stride < cols:
        raise ValueError(f"{what}: expected contiguous, non-overlapping rows, got strides {t.stride()}")
    if not strided:
        raise ValueError(f"{what}: expected rows without gaps, got strides {t.stride()}")
    return t.data_ptr(), rows, cols, stride


def _vector(t, dtype, n, what):
    _on_device(t, what)
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{what}: expected a contiguous tensor of {n} elements, got shape {tuple(t.shape)}, strides "
                         f"{t.stride()}")
    return t.data_ptr()


@functools.lru_cache(maxsize=256)
def checkpoint_layout(cols):
    """(code columns, scale columns) of a checkpoint of rows of `cols` values
    (tide_checkpoint_layout)."""
    codes, scales = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.tide_checkpoint_layout(int(cols), ctypes.byref(codes), ctypes.byref(scales)))
    return codes.value, scales.value


def _packed(codes, scales, rows, cols):
    """(codes address, scales address, TIDE_CODE_*) of a checkpoint of a rows x cols matrix."""
    _on_device(codes, "codes")
    _on_device(scales, "scales")
    if codes.dtype not in _CODES:
        raise TypeError(f"codes: expected torch.float8_e4m3fn or torch.int8, got {codes.dtype}")
    if scales.dtype != torch.uint8:
        raise TypeError(f"scales: expected torch.uint8, got {scales.dtype}")
    c, s = checkpoint_layout(cols)
    if codes.shape != (rows, c) or scales.shape != (rows, s):
        raise ValueError(f"codes and scales of a {rows} x {cols} matrix are {(rows, c)} and {(rows, s)}, got "
                         f"{tuple(codes.shape)} and {tuple(scales.shape)}")
    if not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("codes and scales: expected contiguous tensors")
    return codes.data_ptr(), scales.data_ptr(), _CODES[codes.dtype]


def _pack_args(x, codes, scales):
    p, rows, cols, stride = _matrix(x, _FLOATS, "x")
    c, s, fmt = _packed(codes, scales, rows, cols)
    return p, _FLOATS[x.dtype], rows, cols, stride, fmt, c, s


def checkpoint_pack_call(x, codes, scales):
    """A registered checkpoint pack (see checkpoint_pack)."""
    return TensorCall(lib.tide_checkpoint_pack, _pack_args(x, codes, scales), (x, codes, scales))


def checkpoint_pack(x, codes, scales, stream=None):
    """Pack a matrix into its 8-bit form: x (bf16 or fp32, contiguous rows) ->
    codes (float8_e4m3fn or int8, which chooses the code type) and scales
    (uint8), sized by checkpoint_layout (tide_checkpoint_pack)."""
    _check(lib.tide_checkpoint_pack(*_pack_args(x, codes, scales), _device_stream(stream)))


def _unpack_args(codes, scales, out):
    p, rows, cols, stride = _matrix(out, _FLOATS, "out")
    c, s, fmt = _packed(codes, scales, rows, cols)
    return c, s, fmt, rows, cols, p, _FLOATS[out.dtype], stride


def checkpoint_unpack_call(codes, scales, out):
    """A registered checkpoint restore (see checkpoint_unpack)."""
    return TensorCall(lib.tide_checkpoint_unpack, _unpack_args(codes, scales, out), (codes, scales, out))


def checkpoint_unpack(codes, scales, out, stream=None):
    """Restore a packed matrix, exactly, into out (bf16 or fp32, contiguous
    rows; tide_checkpoint_unpack)."""
    _check(lib.tide_checkpoint_unpack(*_unpack_args(codes, scales, out), _device_stream(stream)))


def _workspace(nbytes, given, stream):
    """(address, bytes, tensor) of a workspace of nbytes: the caller's, or one
    that belongs to the stream the call runs on (once freed it goes back to
    that stream's work only)."""
    if given is None:
        if nbytes == 0:
            return 0, 0, None
        if stream is None:
            given = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        else:
            with torch.cuda.stream(stream):
                given = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    else:
        _on_device(given, "workspace")
        if given.dtype != torch.uint8 or not given.is_contiguous():
            raise TypeError("workspace: expected a contiguous torch.uint8 tensor")
    return given.data_ptr(), given.numel(), given


def _weight_grad_args(dy, codes, scales, dw, alpha, accumulate):
    """(arguments up to the workspace's, bytes of workspace)."""
    y, rows, outs, stride = _matrix(dy, _BF16, "dy")
    w, w_outs, ins, _ = _matrix(dw, _FLOATS, "dw", strided=False)
    if w_outs != outs:
        raise ValueError(f"dw has {w_outs} rows, dy {outs} columns")
    c, s, fmt = _packed(codes, scales, rows, ins)
    need = ctypes.c_int64()
    _check(lib.tide_checkpoint_weight_grad_workspace(y, rows, outs, stride, ins, ctypes.byref(need)))
    return (y, rows, outs, stride, c, s, fmt, ins, w, _FLOATS[dw.dtype], alpha, int(bool(accumulate))), need.value


def checkpoint_weight_grad_workspace(dy, in_features):
    """Bytes of workspace the weight gradient from dy takes
    (tide_checkpoint_weight_grad_workspace)."""
    y, rows, outs, stride = _matrix(dy, _BF16, "dy")
    need = ctypes.c_int64()
    _check(lib.tide_checkpoint_weight_grad_workspace(y, rows, outs, stride, int(in_features), ctypes.byref(need)))
    return need.value


def checkpoint_weight_grad_call(dy, codes, scales, dw, alpha=1.0, accumulate=False, workspace=None):
    """A registered weight gradient (see checkpoint_weight_grad).  With a
    `workspace` of the caller's its launches must not overlap, and a graph that
    records one needs it as long as it is replayed; without one each launch takes
    its own."""
    args, need = _weight_grad_args(dy, codes, scales, dw, alpha, accumulate)
    return WorkspaceCall(lib.tide_checkpoint_weight_grad, args, (dy, codes, scales, dw), need, workspace)


def checkpoint_weight_grad(dy, codes, scales, dw, alpha=1.0, accumulate=False, workspace=None, stream=None):
    """Weight gradient of a linear layer from the checkpoint of its input:
    dw[o][i] = alpha * sum_t dy[t][o] X[t][i], added to the old dw when
    accumulate is true; dy bf16 (tokens x out_features, contiguous rows), dw
    bf16 or fp32 (out_features x in_features).  `workspace` is a uint8 tensor of
    at least checkpoint_weight_grad_workspace bytes; without one the call takes
    its own (tide_checkpoint_weight_grad)."""
    args, need = _weight_grad_args(dy, codes, scales, dw, alpha, accumulate)
    handle = _device_stream(stream)
    ws, nbytes, keep = _workspace(need, workspace, stream)
    _check(lib.tide_checkpoint_weight_grad(*args, ws, nbytes, handle))


# ------------------------------------------------------------ vocabulary loss


def _projection(hidden, weight):
    """The operands' arguments, (tokens, hidden size, vocabulary)."""
    h, tokens, size, h_stride = _matrix(hidden, _BF16, "hidden")
    w, vocab, w_size, w_stride = _matrix(weight, _BF16, "weight")
    if w_size != size:
        raise ValueError(f"weight has {w_size} columns, hidden {size}")
    return (h, h_stride, w, w_stride), (tokens, size, vocab)


def _vocab_loss_bytes(operands, sizes, gradients, dtype):
    need = ctypes.c_int64()
    _check(lib.tide_vocab_loss_workspace(*operands, *sizes, gradients, dtype, ctypes.byref(need)))
    return need.value


def vocab_loss_workspace(hidden, weight, dweight=None):
    """Bytes of workspace of vocab_loss, or of vocab_loss_grad where its
    dweight is given (tide_vocab_loss_workspace)."""
    operands, sizes = _projection(hidden, weight)
    if dweight is None:
        return _vocab_loss_bytes(operands, sizes, 0, DTYPE_F32)
    _matrix(dweight, _FLOATS, "dweight", strided=False)
    return _vocab_loss_bytes(operands, sizes, 1, _FLOATS[dweight.dtype])


def _vocab_loss_args(hidden, weight, targets, loss, lse):
    """(arguments up to the workspace's, bytes of workspace)."""
    operands, sizes = _projection(hidden, weight)
    tokens = sizes[0]
    t = _vector(targets, torch.int64, tokens, "targets")
    out = _vector(loss, torch.float32, tokens, "loss"), None if lse is None else _vector(lse, torch.float32, tokens, "lse")
    return (*operands, t, *sizes, *out), _vocab_loss_bytes(operands, sizes, 0, DTYPE_F32)


def vocab_loss_call(hidden, weight, targets, loss, lse=None, workspace=None):
    """A registered vocabulary loss (see vocab_loss); `workspace` as for
    checkpoint_weight_grad_call."""
    args, need = _vocab_loss_args(hidden, weight, targets, loss, lse)
    return WorkspaceCall(lib.tide_vocab_loss, args, (hidden, weight, targets, loss, lse), need, workspace)


def vocab_loss(hidden, weight, targets, loss, lse=None, workspace=None, stream=None):
    """Cross entropy of the projection hidden @ weight.T (both bf16, contiguous
    rows) against targets (int64): loss[t] and, if given, the log-sum-exp
    lse[t], fp32 per token.  A target outside the vocabulary leaves its token
    out, with 0s.  `workspace` as for checkpoint_weight_grad (tide_vocab_loss)."""
    args, need = _vocab_loss_args(hidden, weight, targets, loss, lse)
    handle = _device_stream(stream)
    ws, nbytes, keep = _workspace(need, workspace, stream)
    _check(lib.tide_vocab_loss(*args, ws, nbytes, handle))


def _vocab_loss_grad_args(hidden, weight, targets, grad_loss, loss, lse, dhidden, dweight, accumulate):
    """(arguments up to the workspace's, bytes of workspace)."""
    operands, sizes = _projection(hidden, weight)
    tokens, size, vocab = sizes
    t = _vector(targets, torch.int64, tokens, "targets")
    g = _vector(grad_loss, torch.float32, tokens, "grad_loss")
    out = _vector(loss, torch.float32, tokens, "loss"), None if lse is None else _vector(lse, torch.float32, tokens, "lse")
    dh, *dh_shape, _ = _matrix(dhidden, _BF16, "dhidden", strided=False)
    dw, *dw_shape, _ = _matrix(dweight, _FLOATS, "dweight", strided=False)
    if dh_shape != [tokens, size] or dw_shape != [vocab, size]:
        raise ValueError(f"dhidden and dweight must be {tokens} x {size} and {vocab} x {size}, got {dh_shape} and "
                         f"{dw_shape}")
    dtype = _FLOATS[dweight.dtype]
    return (*operands, t, g, *sizes, *out, dh, dw, dtype, int(bool(accumulate))), _vocab_loss_bytes(operands, sizes, 1, dtype)


def vocab_loss_grad_call(hidden, weight, targets, grad_loss, loss, lse, dhidden, dweight, accumulate=False,
                         workspace=None):
    """A registered vocabulary loss with gradients (see vocab_loss_grad);
    `workspace` as for checkpoint_weight_grad_call."""
    args, need = _vocab_loss_grad_args(hidden, weight, targets, grad_loss, loss, lse, dhidden, dweight, accumulate)
    return WorkspaceCall(lib.tide_vocab_loss_grad, args,
                         (hidden, weight, targets, grad_loss, loss, lse, dhidden, dweight), need, workspace)


def vocab_loss_grad(hidden, weight, targets, grad_loss, loss, lse, dhidden, dweight, accumulate=False, workspace=None,
                    stream=None):
    """vocab_loss with the gradients of sum_t grad_loss[t] * loss[t]: dhidden
    (bf16) and dweight (bf16 or fp32; added to the old one when accumulate is
    true).  lse may be None (tide_vocab_loss_grad)."""
    args, need = _vocab_loss_grad_args(hidden, weight, targets, grad_loss, loss, lse, dhidden, dweight, accumulate)
    handle = _device_stream(stream)
    ws, nbytes, keep = _workspace(need, workspace, stream)
    _check(lib.tide_vocab_loss_grad(*args, ws, nbytes, handle))


# ------------------------------------------------------------ instruments


def device_info():
    """CU count, largest LDS allocation per workgroup and LDS per CU (bytes),
    and wall-clock rate (kHz) of the current device (tide_device_info)."""
    cu, lds, lds_cu, khz = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib.tide_device_info(ctypes.byref(cu), ctypes.byref(lds), ctypes.byref(lds_cu), ctypes.byref(khz)))
    return {"cu_count": cu.value, "max_lds_per_workgroup": lds.value, "lds_per_cu": lds_cu.value,
            "wall_clock_khz": khz.value}


PROBE_WORDS = 8


def probe(records, grid, lds_bytes, hold_ns, stream=None):
    """Launch the hardware-ID probe (tide_probe_launch): `records` is a GPU
    int32 tensor of at least grid*8 elements; decode it with decode_probe."""
    import torch

    if not isinstance(records, torch.Tensor) or records.device.type != "cuda" or records.dtype != torch.int32:
        raise TypeError("records: expected a GPU torch.int32 tensor")
    if not records.is_contiguous() or records.numel() < int(grid) * PROBE_WORDS:
        raise ValueError(f"records: expected a contiguous tensor of at least {int(grid) * PROBE_WORDS} elements")
    _check(lib.tide_probe_launch(ctypes.c_void_p(records.data_ptr()), int(grid), int(lds_bytes), int(hold_ns),
                                 ctypes.c_void_p(_stream_handle(stream) or None)))


def decode_probe(records):
    """Probe records (any int32/uint32 array of grid*8 words) -> dict of numpy
    arrays: block, wave, simd, cu, sh, se, xcc, ok (LDS read back intact),
    entry, exit (wall-clock ticks)."""
    r = np.asarray(records).reshape(-1, PROBE_WORDS).view(np.uint32).astype(np.int64)
    hw = r[:, 1]
    return {
        "block": r[:, 0], "wave": hw & 0xF, "simd": (hw >> 4) & 0x3, "cu": (hw >> 8) & 0xF, "sh": (hw >> 12) & 0x1,
        "se": (hw >> 13) & 0x7, "xcc": r[:, 2] & 0xF, "ok": r[:, 3] == 0,
        "entry": r[:, 4] | (r[:, 5] << 32), "exit": r[:, 6] | (r[:, 7] << 32),
    }


def victim_axpb(x, y, a, b, stream=None):
    """The elementwise victim y = a * x + b on fp32 GPU tensors of equal size
    (tide_victim_axpb)."""
    import torch

    for t, what in ((x, "x"), (y, "y")):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or t.dtype != torch.float32:
            raise TypeError(f"{what}: expected a GPU torch.float32 tensor")
        if not t.is_contiguous():
            raise ValueError(f"{what}: expected a contiguous tensor")
    if x.numel() != y.numel():
        raise ValueError("x and y must have the same number of elements")
    _check(lib.tide_victim_axpb(ctypes.c_void_p(x.data_ptr() or None), ctypes.c_void_p(y.data_ptr() or None),
                                x.numel(), ctypes.c_float(a), ctypes.c_float(b),
                                ctypes.c_void_p(_stream_handle(stream) or None)))


class Stream:
    """A library-created stream (tide_stream_create), optionally restricted to
    the CUs in `cu_mask` (a sequence of CU indices).  `.torch` is the same
    stream as a torch.cuda.ExternalStream, for events and torch work."""

    def __init__(self, cus=None):
        import torch

        handle = ctypes.c_void_p()
        if cus is None:
            _check(lib.tide_stream_create(None, 0, ctypes.byref(handle)))
        else:
            n = device_info()["cu_count"]
            words = [0] * ((n + 31) // 32)
            for c in cus:
                if not 0 <= int(c) < n:
                    raise ValueError(f"CU index {c} out of range [0, {n})")
                words[int(c) // 32] |= 1 << (int(c) % 32)
            arr = (ctypes.c_uint32 * len(words))(*words)
            _check(lib.tide_stream_create(arr, len(words), ctypes.byref(handle)))
        self.handle = handle.value
        self.torch = torch.cuda.ExternalStream(self.handle)

    def destroy(self):
        if getattr(self, "handle", None):
            self.torch.synchronize()
            _check(lib.tide_stream_destroy(ctypes.c_void_p(self.handle)))
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

"""Python binding of the GB300 variable-size all-to-all (``liba2av.so``).

The functions below carry the C ABI's names (``include/a2av.h``) and only
marshal arguments: every step of the exchange -- reading the device splits,
the scans, ``out_splits_offsets``, the copies -- runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams; nothing here falls back
to a CPU or PyTorch implementation, and every call raises if the compiled
library is missing.
"""
from __future__ import annotations

import ctypes
import os
import threading

from ._build import LIBRARY, build

__all__ = [
    "A2av", "A2avError", "load", "build",
    "a2av_create", "a2av_run", "a2av_combine", "a2av_status", "a2av_destroy", "a2av_set_path",
    "a2av_set_grid", "a2av_last_launch", "a2av_last_dispatch", "a2av_error_string", "a2av_version", "a2av_run_noalloc",
    "a2av_dispatch", "a2av_dispatch_workspace_bytes", "ERR_BAD_INDEX", "MAX_DISPATCH_KEYS",
    "a2av_run_multi", "A2avExchange", "MAX_EXCHANGES", "BoundCall", "a2av_combine_items",
    "COMBINE_WORKSPACE_BYTES",
    "OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED", "ERR_CUDA", "ERR_BAD_SPLITS", "ERR_TIMEOUT",
    "PATH_AUTO", "PATH_VECTOR", "PATH_BULK", "PATH_STAGED", "MAX_RANKS",
    "a2av_route", "a2av_route_backward", "a2av_expert_matmul", "a2av_expert_matmul_backward",
    "a2av_expert_matmul_workspace_bytes", "a2av_combine_weighted", "a2av_combine_weighted_backward",
    "A2avRoute", "A2avExpert", "F32", "BF16", "F16", "MAX_TOPK", "MAX_ROUTE_GROUPS",
]

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_BAD_SPLITS, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
ERR_BAD_INDEX = -6
MAX_DISPATCH_KEYS = 1024
PATH_AUTO, PATH_VECTOR, PATH_BULK, PATH_STAGED = 0, 1, 2, 3
MAX_RANKS = 32
MAX_EXCHANGES = 4
COMBINE_WORKSPACE_BYTES = 256 + 16 * 32 * 32
F32, BF16, F16 = 0, 1, 2
MAX_TOPK, MAX_ROUTE_GROUPS = 32, 32
_SCORES = {"softmax": 0, "sigmoid": 1}
_ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}

_lib = None


class A2avExchange(ctypes.Structure):
    """``a2av_exchange_t``: one exchange of an ``a2av_run_multi`` call."""
    _fields_ = [("in_ptrs", ctypes.POINTER(ctypes.c_void_p)),
                ("in_splits_dev", ctypes.c_void_p),
                ("out_ptrs", ctypes.POINTER(ctypes.c_void_p)),
                ("out_splits_offsets_dev", ctypes.c_void_p),
                ("row_bytes", ctypes.c_int64)]


class A2avRoute(ctypes.Structure):
    """``a2av_route_t``: how ``a2av_route`` chooses."""
    _fields_ = [(n, ctypes.c_int) for n in ("experts", "topk", "dtype", "score", "groups",
                                            "top_groups", "group_top", "renormalise")]
    _fields_.append(("scale", ctypes.c_float))


class A2avExpert(ctypes.Structure):
    """``a2av_expert_t``: the shape of ``a2av_expert_matmul``."""
    _fields_ = [("experts_per_peer", ctypes.c_int), ("in_features", ctypes.c_int64),
                ("out_features", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("gated", ctypes.c_int)]


class A2avError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {a2av_error_string(code)} ({code})")
        self.code = code


def load():
    """The loaded ``liba2av.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY):
        raise ImportError(
            f"{LIBRARY} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (nvcc, sm_103a)")
    lib = ctypes.CDLL(LIBRARY)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    pp = ctypes.POINTER(ctypes.c_void_p)
    lib.a2av_create.argtypes = [ci, i64, i64, pp]
    lib.a2av_run.argtypes = [vp, pp, vp, pp, vp, i64, vp]
    lib.a2av_combine.argtypes = [vp, pp, vp, pp, vp, i64, vp]
    lib.a2av_status.argtypes = [vp, vp, ctypes.POINTER(ci)]
    lib.a2av_destroy.argtypes = [vp]
    lib.a2av_set_path.argtypes = [vp, ci]
    lib.a2av_set_grid.argtypes = [vp, ci]
    lib.a2av_last_launch.argtypes = [vp, ctypes.POINTER(ci), ctypes.POINTER(ci),
                                     ctypes.POINTER(ci)]
    lib.a2av_run_noalloc.argtypes = [ci, i64, i64, pp, vp, pp, vp, i64, vp, ctypes.POINTER(ci)]
    lib.a2av_last_dispatch.argtypes = [vp, ctypes.POINTER(ci), ctypes.POINTER(ci),
                                       ctypes.POINTER(ctypes.c_char_p)]
    i64p = ctypes.POINTER(i64)
    lib.a2av_dispatch_workspace_bytes.argtypes = [ci, ci, i64]
    lib.a2av_dispatch_workspace_bytes.restype = i64
    lib.a2av_dispatch.argtypes = [vp, ci, pp, i64p, pp, pp, i64p, pp, vp, pp, vp, i64, vp, i64, vp]
    lib.a2av_dispatch.restype = ci
    lib.a2av_run_multi.argtypes = [vp, ci, ctypes.POINTER(A2avExchange), vp]
    lib.a2av_combine_items.argtypes = [vp, ci, pp, vp, pp, pp, i64p, pp, i64, vp, i64, vp]
    lib.a2av_combine_items.restype = ci
    lib.a2av_error_string.argtypes = [ci]
    lib.a2av_error_string.restype = ctypes.c_char_p
    lib.a2av_version.argtypes = []
    route_p, expert_p = ctypes.POINTER(A2avRoute), ctypes.POINTER(A2avExpert)
    # (the pointer arrays of these calls go as addresses)
    lib.a2av_route.argtypes = [vp, route_p, vp, i64p, vp, vp, vp, vp, vp]
    lib.a2av_route_backward.argtypes = [vp, route_p, vp, i64p, vp, vp, vp, vp]
    lib.a2av_expert_matmul.argtypes = [vp, expert_p, vp, i64p, vp, vp, vp, vp, vp, vp, vp]
    lib.a2av_expert_matmul_backward.argtypes = [vp, expert_p, vp, i64p, vp, vp, vp, vp, vp, vp, vp,
                                                vp, i64, vp]
    lib.a2av_expert_matmul_workspace_bytes.argtypes = [ci, expert_p, i64]
    lib.a2av_expert_matmul_workspace_bytes.restype = i64
    lib.a2av_combine_weighted.argtypes = [vp, ci, ci, i64, ci, vp, i64p, vp, vp, vp, vp, i64p, vp, vp,
                                          vp]
    lib.a2av_combine_weighted_backward.argtypes = [vp, ci, ci, i64, ci, vp, i64p, vp, vp, vp, vp,
                                                   i64p, vp, vp, vp, vp]
    for f in ("a2av_create", "a2av_run", "a2av_combine", "a2av_status", "a2av_destroy", "a2av_set_path",
              "a2av_set_grid", "a2av_last_launch", "a2av_version", "a2av_run_noalloc",
              "a2av_run_multi", "a2av_route", "a2av_route_backward", "a2av_expert_matmul",
              "a2av_expert_matmul_backward", "a2av_combine_weighted",
              "a2av_combine_weighted_backward"):
        getattr(lib, f).restype = ci
    _lib = lib
    return lib


# ------------------------------------------------ the C ABI, name for name --
def a2av_version() -> int:
    return load().a2av_version()


def a2av_error_string(code: int) -> str:
    return load().a2av_error_string(int(code)).decode()


def a2av_create(world_size: int, in_capacity_rows: int = 0, out_capacity_rows: int = 0):
    """Returns (status, handle); handle is None unless status is OK."""
    h = ctypes.c_void_p()
    rc = load().a2av_create(int(world_size), int(in_capacity_rows), int(out_capacity_rows),
                            ctypes.byref(h))
    return rc, (h if rc == OK else None)


def _ptr_array(ptrs):
    arr = (ctypes.c_void_p * max(len(ptrs), 1))()
    for k, p in enumerate(ptrs):
        arr[k] = int(p) if p else None
    return arr


def a2av_run(handle, in_ptrs, in_splits_dev: int, out_ptrs, out_splits_offsets_dev: int,
             row_bytes: int, stream: int = 0) -> int:
    """Raw entry point: integer device addresses, integer cudaStream_t."""
    return load().a2av_run(handle, _ptr_array(in_ptrs), ctypes.c_void_p(int(in_splits_dev) or None),
                           _ptr_array(out_ptrs),
                           ctypes.c_void_p(int(out_splits_offsets_dev) or None), int(row_bytes),
                           ctypes.c_void_p(int(stream) or None))


def a2av_combine(handle, in_ptrs, dispatch_splits_offsets_dev: int, out_ptrs,
                 out_splits_offsets_dev: int, row_bytes: int, stream: int = 0) -> int:
    """Raw reverse exchange: integer device addresses, integer cudaStream_t."""
    return load().a2av_combine(handle, _ptr_array(in_ptrs),
                               ctypes.c_void_p(int(dispatch_splits_offsets_dev) or None),
                               _ptr_array(out_ptrs),
                               ctypes.c_void_p(int(out_splits_offsets_dev) or None),
                               int(row_bytes), ctypes.c_void_p(int(stream) or None))


def a2av_run_multi(handle, exchanges, stream: int = 0) -> int:
    """``exchanges``: a sequence of (in_ptrs, in_splits_dev, out_ptrs,
    out_splits_offsets_dev, row_bytes), each as for ``a2av_run``."""
    arr = (A2avExchange * max(len(exchanges), 1))()
    keep = []
    for k, (ins, sp, outs, so, rb) in enumerate(exchanges):
        ia, oa = _ptr_array(ins), _ptr_array(outs)
        keep += [ia, oa]
        arr[k] = A2avExchange(ctypes.cast(ia, ctypes.POINTER(ctypes.c_void_p)), int(sp) or None,
                              ctypes.cast(oa, ctypes.POINTER(ctypes.c_void_p)), int(so) or None,
                              int(rb))
    return load().a2av_run_multi(handle, len(exchanges), arr if exchanges else None,
                                 ctypes.c_void_p(int(stream) or None))


def a2av_combine_items(handle, keys_per_peer: int, peer_ptrs, in_splits_dev: int, key_ptrs,
                       sorted_pos_ptrs, items_per_rank, item_out_ptrs, row_bytes: int,
                       workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    """Raw fused combine: integer device addresses, host lists of counts."""
    return load().a2av_combine_items(
        handle, int(keys_per_peer), _ptr_array(peer_ptrs),
        ctypes.c_void_p(int(in_splits_dev) or None), _ptr_array(key_ptrs),
        _ptr_array(sorted_pos_ptrs), _i64_array(items_per_rank), _ptr_array(item_out_ptrs),
        int(row_bytes), ctypes.c_void_p(int(workspace) or None), int(workspace_bytes),
        ctypes.c_void_p(int(stream) or None))


def a2av_status(handle, stream: int = 0):
    """Returns (status, device_status)."""
    v = ctypes.c_int(0)
    rc = load().a2av_status(handle, ctypes.c_void_p(int(stream) or None), ctypes.byref(v))
    return rc, v.value


def a2av_destroy(handle) -> int:
    return load().a2av_destroy(handle)


def a2av_set_path(handle, path: int) -> int:
    return load().a2av_set_path(handle, int(path))


def a2av_set_grid(handle, ctas_per_sm: int) -> int:
    return load().a2av_set_grid(handle, int(ctas_per_sm))


def a2av_last_launch(handle):
    """Returns (status, path, grid, block) of the handle's last run."""
    p, g, b = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    rc = load().a2av_last_launch(handle, ctypes.byref(p), ctypes.byref(g), ctypes.byref(b))
    return rc, p.value, g.value, b.value


def a2av_last_dispatch(handle):
    """Returns (status, kernels, memsets, copy_kernel) of the handle's last
    a2av_dispatch or a2av_combine_items."""
    k, m, name = ctypes.c_int(), ctypes.c_int(), ctypes.c_char_p()
    rc = load().a2av_last_dispatch(handle, ctypes.byref(k), ctypes.byref(m), ctypes.byref(name))
    return rc, k.value, m.value, (name.value or b"").decode()


def a2av_run_noalloc(world_size: int, in_capacity_rows: int, out_capacity_rows: int, in_ptrs,
                     in_splits_dev: int, out_ptrs, out_splits_offsets_dev: int, row_bytes: int,
                     stream: int = 0, wait: bool = True):
    """The allocation-free entry point (no handle; see include/a2av.h).

    Returns (status, device_status); with ``wait`` False the call is
    asynchronous and device_status is None."""
    v = ctypes.c_int(0)
    rc = load().a2av_run_noalloc(int(world_size), int(in_capacity_rows), int(out_capacity_rows),
                                 _ptr_array(in_ptrs), ctypes.c_void_p(int(in_splits_dev) or None),
                                 _ptr_array(out_ptrs),
                                 ctypes.c_void_p(int(out_splits_offsets_dev) or None),
                                 int(row_bytes), ctypes.c_void_p(int(stream) or None),
                                 ctypes.byref(v) if wait else None)
    return rc, (v.value if wait else None)


def a2av_dispatch_workspace_bytes(world_size: int, keys_per_peer: int,
                                  max_items_per_rank: int) -> int:
    return load().a2av_dispatch_workspace_bytes(int(world_size), int(keys_per_peer),
                                                int(max_items_per_rank))


def _i64_array(values):
    return (ctypes.c_int64 * max(len(values), 1))(*[int(v) for v in values])


def a2av_dispatch(handle, keys_per_peer: int, rows_ptrs, rows_per_rank, src_row_ptrs, key_ptrs,
                  items_per_rank, out_ptrs, out_splits_offsets_dev: int, sorted_pos_ptrs,
                  in_splits_dev: int, row_bytes: int, workspace: int, workspace_bytes: int,
                  stream: int = 0) -> int:
    """Raw fused dispatch: integer device addresses, host lists of counts."""
    return load().a2av_dispatch(
        handle, int(keys_per_peer), _ptr_array(rows_ptrs), _i64_array(rows_per_rank),
        _ptr_array(src_row_ptrs), _ptr_array(key_ptrs), _i64_array(items_per_rank),
        _ptr_array(out_ptrs), ctypes.c_void_p(int(out_splits_offsets_dev) or None),
        _ptr_array(sorted_pos_ptrs), ctypes.c_void_p(int(in_splits_dev) or None),
        int(row_bytes), ctypes.c_void_p(int(workspace) or None), int(workspace_bytes),
        ctypes.c_void_p(int(stream) or None))


def _address(p):
    return ctypes.c_void_p(int(p) if p else None)


def _optional_ptrs(ptrs):
    return None if ptrs is None else _ptr_array(ptrs)


def a2av_route(handle, route: A2avRoute, logits_ptrs, tokens_per_rank, bias: int, key_ptrs,
               weight_ptrs, counts: int, stream: int = 0) -> int:
    """Raw routing (include/a2av_moe.h): integer device addresses, host lists of counts."""
    return load().a2av_route(handle, ctypes.byref(route), _ptr_array(logits_ptrs),
                             _i64_array(tokens_per_rank), _address(bias), _ptr_array(key_ptrs),
                             _ptr_array(weight_ptrs), _address(counts), _address(stream))


def a2av_route_backward(handle, route: A2avRoute, logits_ptrs, tokens_per_rank, key_ptrs,
                        d_weight_ptrs, d_logits_ptrs, stream: int = 0) -> int:
    """Raw gradient of the routing weights."""
    return load().a2av_route_backward(handle, ctypes.byref(route), _ptr_array(logits_ptrs),
                                      _i64_array(tokens_per_rank), _ptr_array(key_ptrs),
                                      _ptr_array(d_weight_ptrs), _ptr_array(d_logits_ptrs),
                                      _address(stream))


def a2av_expert_matmul(handle, shape: A2avExpert, rows_ptrs, rows_per_peer, counts: int,
                       weight_ptrs, bias_ptrs, residual_ptrs, out_ptrs, pre_ptrs,
                       stream: int = 0) -> int:
    """Raw experts' product: integer device addresses, lists (or None) per peer."""
    return load().a2av_expert_matmul(
        handle, ctypes.byref(shape), _ptr_array(rows_ptrs), _i64_array(rows_per_peer),
        _address(counts), _ptr_array(weight_ptrs), _optional_ptrs(bias_ptrs),
        _optional_ptrs(residual_ptrs), _ptr_array(out_ptrs), _optional_ptrs(pre_ptrs),
        _address(stream))


def a2av_expert_matmul_workspace_bytes(world_size: int, shape: A2avExpert, total_rows: int) -> int:
    return load().a2av_expert_matmul_workspace_bytes(int(world_size), ctypes.byref(shape),
                                                     int(total_rows))


def a2av_expert_matmul_backward(handle, shape: A2avExpert, rows_ptrs, rows_per_peer, counts: int,
                                weight_ptrs, pre_ptrs, d_out_ptrs, d_rows_ptrs, d_weight_ptrs,
                                d_bias_ptrs, workspace: int, workspace_bytes: int,
                                stream: int = 0) -> int:
    """Raw gradients of the experts' product."""
    return load().a2av_expert_matmul_backward(
        handle, ctypes.byref(shape), _ptr_array(rows_ptrs), _i64_array(rows_per_peer),
        _address(counts), _ptr_array(weight_ptrs), _optional_ptrs(pre_ptrs),
        _ptr_array(d_out_ptrs), _optional_ptrs(d_rows_ptrs), _optional_ptrs(d_weight_ptrs),
        _optional_ptrs(d_bias_ptrs), _address(workspace), int(workspace_bytes), _address(stream))


def a2av_combine_weighted(handle, keys_per_peer: int, topk: int, hidden: int, dtype: int,
                          peer_ptrs, rows_per_peer, in_splits_dev: int, key_ptrs, sorted_pos_ptrs,
                          weight_ptrs, tokens_per_rank, residual_ptrs, out_ptrs,
                          stream: int = 0) -> int:
    """Raw weighted combine: integer device addresses, lists (or None) per rank."""
    return load().a2av_combine_weighted(
        handle, int(keys_per_peer), int(topk), int(hidden), int(dtype), _ptr_array(peer_ptrs),
        _i64_array(rows_per_peer), _address(in_splits_dev), _ptr_array(key_ptrs), _ptr_array(sorted_pos_ptrs),
        _optional_ptrs(weight_ptrs), _i64_array(tokens_per_rank), _optional_ptrs(residual_ptrs),
        _ptr_array(out_ptrs), _address(stream))


def a2av_combine_weighted_backward(handle, keys_per_peer: int, topk: int, hidden: int, dtype: int,
                                   peer_ptrs, rows_per_peer, in_splits_dev: int, key_ptrs,
                                   sorted_pos_ptrs, weight_ptrs, tokens_per_rank, d_out_ptrs, d_peer_ptrs,
                                   d_weight_ptrs, stream: int = 0) -> int:
    """Raw gradients of the weighted combine."""
    return load().a2av_combine_weighted_backward(
        handle, int(keys_per_peer), int(topk), int(hidden), int(dtype), _optional_ptrs(peer_ptrs),
        _i64_array(rows_per_peer), _address(in_splits_dev), _ptr_array(key_ptrs), _ptr_array(sorted_pos_ptrs),
        _optional_ptrs(weight_ptrs), _i64_array(tokens_per_rank), _ptr_array(d_out_ptrs),
        _optional_ptrs(d_peer_ptrs), _optional_ptrs(d_weight_ptrs), _address(stream))


# --------------------------------------------------------- torch-facing --
class _PlainMarshal:
    """``_marshal`` (csrc/marshal.cpp) without the compiled module."""

    @staticmethod
    def pointers(address, count, *lists):
        for tensors, dtype, shapes in lists:
            if tensors is None:
                continue
            try:
                if len(tensors) != count or not all(
                        t.is_cuda and t.dtype == dtype and t.is_contiguous() for t in tensors) or (
                        shapes is not None and [t.shape for t in tensors] != shapes):
                    return False
            except AttributeError:  # None among them
                return False
            for r, t in enumerate(tensors):
                ctypes.c_void_p.from_address(address + 8 * r).value = t.data_ptr()
            address += 8 * count
        return True

    @staticmethod
    def rows(tensors):
        try:
            shapes = [t.shape for t in tensors]
        except AttributeError:
            return None
        if not shapes or any(len(s) != 2 or s[1] != shapes[0][-1] for s in shapes):
            return None
        return [s[0] for s in shapes], shapes[0][1]

    @staticmethod
    def sizes(tensors):
        try:
            return [t.numel() for t in tensors]
        except AttributeError:
            return None

    @staticmethod
    def route(*args):
        return None  # (the method goes through its arguments itself)

    route_backward = expert_matmul = expert_matmul_backward = route
    combine_weighted = combine_weighted_backward = route


def _load_marshal():
    """The compiled module, where there is one that was built for this torch."""
    import torch
    try:
        from . import _marshal
    except ImportError:
        return _PlainMarshal
    return _marshal if _marshal.torch_version == torch.__version__ else _PlainMarshal


class _Kept(threading.local):
    """The default workspaces of an object's calls, one for each call and stream
    in each thread, so that calls that may be in flight together share none."""

    def __init__(self):
        self.buffers = {}


class BoundCall:
    """One library call whose arguments were marshalled once (``A2av.bind_run``,
    ``bind_run_multi``, ``bind_dispatch``).  Calling it enqueues the same
    launch again -- on the stream given at bind time, or on ``stream`` -- with
    the same buffers: the tensors must stay alive and keep their storage, while
    the device data they hold (splits, keys, rows) may change between calls.
    It skips the per-call Python checks and pointer gathering, which cost more
    host time than a small exchange takes on the device.  Bound without a
    workspace, it uses that of the stream's other calls: bind it with one of its
    own if a graph that captures it is to be replayed beside them."""

    def __init__(self, engine, fn, what, args, stream_index, keep, workspace=None):
        # workspace: of a call that was given none, its place in args, its name and its size
        self._engine, self._fn, self._what = engine, fn, what
        self._args, self._si, self._keep, self._ws = tuple(args), stream_index, keep, workspace

    def __call__(self, stream=None):
        args = self._args
        if stream is not None:
            args = list(args)
            queue = ctypes.c_void_p(A2av._stream(stream) or None)
            if self._ws is not None and queue.value != args[self._si].value:
                # (another stream than the workspace's: the one of that stream)
                i, name, need = self._ws
                held = self._engine._default_workspace(name, need, stream)
                args[i], args[i + 1] = ctypes.c_void_p(held.data_ptr()), held.numel()
            args[self._si] = queue
        rc = self._fn(*args)
        if rc != OK:
            raise A2avError(rc, self._what)


class A2av:
    """One handle over ``world_size`` ranks; tensors in, tensors out.

    ``run(inputs, in_splits, outputs, out_splits_offsets, row_bytes)`` takes
    W CUDA tensors (any dtype, contiguous; ``None`` or empty for a rank
    without a buffer), the int64 [W, W] split matrix on the device, W output
    tensors and the int64 [W, 2, W] out_splits_offsets tensor, and enqueues
    the exchange on ``stream`` (default: torch's current stream).  Device
    detected errors are read with ``status()``.
    """

    def __init__(self, world_size: int, in_capacity_rows: int = 0, out_capacity_rows: int = 0,
                 path: int = PATH_AUTO, ctas_per_sm: int = 0):
        rc, h = a2av_create(world_size, in_capacity_rows, out_capacity_rows)
        if rc != OK:
            raise A2avError(rc, "a2av_create")
        self.handle, self.world_size, self._path = h, int(world_size), int(path)
        import torch
        self._device = torch.cuda.current_device()
        self._marshal = _load_marshal()
        self._address = getattr(h, "value", h)
        self._entries = {what: ctypes.cast(getattr(load(), "a2av_" + what), ctypes.c_void_p).value
                         for what in ("route", "route_backward", "expert_matmul",
                                      "expert_matmul_backward", "expert_matmul_workspace_bytes",
                                      "combine_weighted", "combine_weighted_backward")}
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._codes = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
        self._int32, self._int64, self._float = torch.int32, torch.int64, torch.float32
        self._counts = ctypes.c_int64 * self.world_size
        self._kept = _Kept()
        self._capture_status = ctypes.CDLL("libcuda.so.1").cuStreamIsCapturing
        self._capture_status.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int)]
        self._room = [ctypes.c_void_p * max(1, self.world_size * n) for n in range(9)]
        if path != PATH_AUTO:
            self._check(a2av_set_path(h, path), "a2av_set_path")
        if ctas_per_sm:
            self._check(a2av_set_grid(h, ctas_per_sm), "a2av_set_grid")

    @staticmethod
    def _check(rc, what):
        if rc != OK:
            raise A2avError(rc, what)

    @staticmethod
    def _stream(stream):
        import torch
        if stream is None:
            stream = torch.cuda.current_stream()
        return int(getattr(stream, "cuda_stream", stream))

    def _queue(self, stream):
        """The cudaStream_t to enqueue on: ``stream``, or torch's current one."""
        return _address(self._number(stream))

    def _number(self, stream):
        """``stream``, or torch's current one, as a number."""
        if stream is not None or self._raw_stream is None:
            return self._stream(stream)
        return self._raw_stream(self._device)

    def _on(self, stream):
        """``stream`` as torch's current one: what is allocated then is of its order."""
        import torch
        if not isinstance(stream, torch.cuda.Stream):
            queue = self._stream(stream)
            stream = torch.cuda.ExternalStream(queue) if queue else torch.cuda.default_stream()
        return torch.cuda.stream(stream)

    def _capturing(self, stream, queue):
        """Whether calls on ``stream``, whose number is ``queue``, go into a graph.
        (The driver tells for any stream, but not in a thread that has made no CUDA
        call yet; torch does for its current one.)"""
        status = ctypes.c_int(0)
        if self._capture_status(queue, ctypes.byref(status)) == 0:
            return status.value != 0
        import torch
        with self._on(torch.cuda.current_stream() if stream is None else stream):
            return torch.cuda.is_current_stream_capturing()

    def _held(self, what, stream):
        """The workspace kept for this call on ``stream``, or None."""
        queue = self._number(stream)
        return None if self._capturing(stream, queue) else self._kept.buffers.get((what, queue))

    def _default_workspace(self, what, need, stream):
        """The default workspace of a call on ``stream``: kept for the calls that
        follow on it, which take their turns.  The allocator hands out one that was
        too small in that stream's order only.  A call that is being captured takes
        one from the graph's own memory, which lives as long as the graph does and
        which no other call is given."""
        held = self._held(what, stream)
        if held is not None and held.numel() >= need:
            return held
        import torch
        queue = self._number(stream)
        with self._on(torch.cuda.current_stream() if stream is None else stream):
            held = torch.empty(need, dtype=torch.uint8, device="cuda")
        if not self._capturing(stream, queue):
            self._kept.buffers[what, queue] = held
        return held

    @staticmethod
    def _scratch(workspace):
        """Refuses a workspace whose numel() is not the memory behind its data_ptr()."""
        import torch
        if (not isinstance(workspace, torch.Tensor) or not workspace.is_cuda
                or not workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous CUDA tensor")

    def _buffers(self, tensors, what):
        """Pointer array for W buffers; True when one lives in pinned host memory."""
        W = self.world_size
        if len(tensors) != W:
            raise ValueError(f"{what}: expected {W} buffers, got {len(tensors)}")
        arr = (ctypes.c_void_p * W)()
        host = False
        for k, t in enumerate(tensors):
            if t is None or t.numel() == 0:
                continue
            if not t.is_contiguous():
                raise ValueError(f"{what}: buffers must be contiguous")
            if t.is_cuda:
                arr[k] = t.data_ptr()
            elif t.is_pinned():
                arr[k] = t.data_ptr()
                host = True
            else:
                raise ValueError(f"{what}: buffers must be CUDA tensors or pinned host tensors")
        return arr, host

    @staticmethod
    def _matrix(t, shape, name):
        import torch
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.int64 or not t.is_cuda
                or tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA int64 tensor of shape {shape}")
        return ctypes.c_void_p(t.data_ptr())

    def _launch_args(self, inputs, splits, outputs, out_splits_offsets, row_bytes, stream,
                     split_shape):
        """The C call's arguments (stream last) and whether a buffer is host memory."""
        W = self.world_size
        sp = self._matrix(splits, split_shape, "splits")
        so = self._matrix(out_splits_offsets, (W, 2, W), "out_splits_offsets")
        ins, host_in = self._buffers(inputs, "inputs")
        outs, host_out = self._buffers(outputs, "outputs")
        st = ctypes.c_void_p(self._stream(stream) or None)
        return [self.handle, ins, sp, outs, so, int(row_bytes), st], host_in or host_out

    def _launch(self, fn, what, inputs, splits, outputs, out_splits_offsets, row_bytes, stream,
                split_shape):
        # (buffers in pinned host memory are routed to the vector engine by
        # the library itself)
        args, _ = self._launch_args(inputs, splits, outputs, out_splits_offsets, row_bytes,
                                    stream, split_shape)
        self._check(fn(*args), what)

    def bind_run(self, inputs, in_splits, outputs, out_splits_offsets, row_bytes: int,
                 stream=None) -> BoundCall:
        """``run`` marshalled once: returns a BoundCall that re-enqueues the
        exchange on these buffers."""
        W = self.world_size
        args, _ = self._launch_args(inputs, in_splits, outputs, out_splits_offsets, row_bytes,
                                    stream, (W, W))
        keep = (inputs, in_splits, outputs, out_splits_offsets)
        return BoundCall(self, load().a2av_run, "a2av_run", args, len(args) - 1, keep)

    def run(self, inputs, in_splits, outputs, out_splits_offsets, row_bytes: int, stream=None):
        W = self.world_size
        self._launch(load().a2av_run, "a2av_run", inputs, in_splits, outputs, out_splits_offsets,
                     row_bytes, stream, (W, W))

    def run_multi(self, exchanges, stream=None):
        """Several exchanges over the same ranks in one launch (see
        include/a2av.h, a2av_run_multi).  ``exchanges``: a sequence of
        (inputs, in_splits, outputs, out_splits_offsets, row_bytes), each as
        for ``run``."""
        args, _, _ = self._multi_args(exchanges, stream)
        self._check(load().a2av_run_multi(*args), "a2av_run_multi")

    def _multi_args(self, exchanges, stream):
        W = self.world_size
        if not 1 <= len(exchanges) <= MAX_EXCHANGES:
            raise ValueError(f"run_multi takes 1..{MAX_EXCHANGES} exchanges")
        arr = (A2avExchange * len(exchanges))()
        keep, host = [arr], False
        for k, (inputs, splits, outputs, so, rb) in enumerate(exchanges):
            sp = self._matrix(splits, (W, W), "splits")
            sop = self._matrix(so, (W, 2, W), "out_splits_offsets")
            ins, h_in = self._buffers(inputs, "inputs")
            outs, h_out = self._buffers(outputs, "outputs")
            host = host or h_in or h_out
            keep += [ins, outs]
            arr[k] = A2avExchange(ctypes.cast(ins, ctypes.POINTER(ctypes.c_void_p)), sp,
                                  ctypes.cast(outs, ctypes.POINTER(ctypes.c_void_p)), sop,
                                  int(rb))
        st = ctypes.c_void_p(self._stream(stream) or None)
        return [self.handle, len(exchanges), arr, st], host, keep

    def bind_run_multi(self, exchanges, stream=None) -> BoundCall:
        """``run_multi`` marshalled once."""
        args, _, keep = self._multi_args(exchanges, stream)
        return BoundCall(self, load().a2av_run_multi, "a2av_run_multi", args, 3,
                         keep + [exchanges])

    def combine(self, inputs, dispatch_splits_offsets, outputs, out_splits_offsets,
                row_bytes: int, stream=None):
        """The reverse exchange: send every received chunk back to its source
        rank; ``dispatch_splits_offsets`` is the [W, 2, W] tensor a previous
        ``run`` wrote."""
        W = self.world_size
        self._launch(load().a2av_combine, "a2av_combine", inputs, dispatch_splits_offsets,
                     outputs, out_splits_offsets, row_bytes, stream, (W, 2, W))

    def dispatch(self, rows, src_rows, keys, keys_per_peer: int, outputs, out_splits_offsets,
                 sorted_pos, row_bytes: int, in_splits=None, workspace=None, stream=None,
                 _bind=False):
        """Fused dispatch: group each rank's items by key on the device and
        exchange their rows (see include/a2av.h, a2av_dispatch).

        ``rows[r]``: rank r's source rows (uint8 CUDA tensor, a multiple of
        ``row_bytes``); ``src_rows[r]`` / ``keys[r]``: int32 CUDA tensors, one
        entry per item; ``sorted_pos[r]``: int64 CUDA tensor receiving each
        item's position in key order; ``in_splits``: optional int64 [W, W]
        receiving the split matrix.  ``workspace``: scratch that no other call in
        flight has (sized by the largest item count); by default the object keeps
        a buffer for each stream in each thread, and a call under capture takes
        its own from the graph's memory."""
        import torch
        W = self.world_size
        for name, ts, dt in (("src_rows", src_rows, torch.int32), ("keys", keys, torch.int32),
                             ("sorted_pos", sorted_pos, torch.int64)):
            if len(ts) != W:
                raise ValueError(f"{name}: expected {W} tensors")
            for t in ts:
                if t is not None and t.numel() and (t.dtype != dt or not t.is_cuda
                                                    or not t.is_contiguous()):
                    raise ValueError(f"{name} must be contiguous CUDA {dt} tensors")
        if not (isinstance(out_splits_offsets, torch.Tensor) and out_splits_offsets.is_cuda
                and out_splits_offsets.dtype == torch.int64
                and tuple(out_splits_offsets.shape) == (W, 2, W)
                and out_splits_offsets.is_contiguous()):
            raise ValueError(f"out_splits_offsets must be a contiguous CUDA int64 [{W}, 2, {W}]")
        if in_splits is not None and (in_splits.dtype != torch.int64 or not in_splits.is_cuda
                                      or tuple(in_splits.shape) != (W, W)):
            raise ValueError(f"in_splits must be a CUDA int64 [{W}, {W}] tensor")
        items = [0 if t is None else t.numel() for t in keys]
        if any((0 if s is None else s.numel()) != m for s, m in zip(src_rows, items)):
            raise ValueError("src_rows and keys must have one entry per item")
        if any((0 if t is None else t.numel()) != m for t, m in zip(sorted_pos, items)):
            raise ValueError("sorted_pos must have one entry per item")
        need = a2av_dispatch_workspace_bytes(W, keys_per_peer, max(items))
        if need < 0:
            raise A2avError(ERR_UNSUPPORTED, "a2av_dispatch_workspace_bytes")
        own = None
        if workspace is not None:
            self._scratch(workspace)
        else:
            own = (12, "dispatch", need)
            workspace = self._default_workspace("dispatch", need, stream)
        n_rows = [0 if t is None else t.numel() // int(row_bytes) for t in rows]
        ptr = lambda ts: [0 if t is None or t.numel() == 0 else t.data_ptr() for t in ts]
        rows_arr, host_rows = self._buffers(rows, "rows")
        outs_arr, host_outs = self._buffers(outputs, "outputs")
        if host_rows or host_outs:
            raise ValueError("a2av_dispatch takes device buffers only")
        args = [self.handle, int(keys_per_peer), _ptr_array(list(rows_arr)), _i64_array(n_rows),
                _ptr_array(ptr(src_rows)), _ptr_array(ptr(keys)), _i64_array(items),
                _ptr_array(list(outs_arr)), ctypes.c_void_p(out_splits_offsets.data_ptr()),
                _ptr_array(ptr(sorted_pos)),
                ctypes.c_void_p(None if in_splits is None else in_splits.data_ptr()),
                int(row_bytes), ctypes.c_void_p(workspace.data_ptr()), int(workspace.numel()),
                self._queue(stream)]
        if _bind:
            keep = (rows, src_rows, keys, outputs, out_splits_offsets, sorted_pos, in_splits,
                    workspace)
            return BoundCall(self, load().a2av_dispatch, "a2av_dispatch", args, 14, keep, own)
        self._check(load().a2av_dispatch(*args), "a2av_dispatch")

    def bind_dispatch(self, rows, src_rows, keys, keys_per_peer: int, outputs,
                      out_splits_offsets, sorted_pos, row_bytes: int, in_splits=None,
                      workspace=None, stream=None) -> BoundCall:
        """``dispatch`` marshalled once: the item counts are fixed at bind time
        (the keys and source rows themselves may change between calls)."""
        return self.dispatch(rows, src_rows, keys, keys_per_peer, outputs, out_splits_offsets,
                             sorted_pos, row_bytes, in_splits, workspace, stream, _bind=True)

    def bind_combine_items(self, peers, in_splits, keys, sorted_pos, keys_per_peer: int,
                           item_out, row_bytes: int, workspace=None, stream=None) -> BoundCall:
        """``combine_items`` marshalled once (see BoundCall)."""
        return self.combine_items(peers, in_splits, keys, sorted_pos, keys_per_peer, item_out,
                                  row_bytes, workspace, stream, _bind=True)

    def combine_items(self, peers, in_splits, keys, sorted_pos, keys_per_peer: int, item_out,
                      row_bytes: int, workspace=None, stream=None, _bind=False):
        """The fused combine (see include/a2av.h, a2av_combine_items): every
        item's row from the peers' dispatch-layout buffers back to row i of
        ``item_out[r]``.  ``in_splits``, ``keys`` and ``sorted_pos`` as a
        dispatch took or wrote them.  ``workspace`` as in ``dispatch``."""
        import torch
        W = self.world_size
        sp = self._matrix(in_splits, (W, W), "in_splits")
        for name, ts, dt in (("keys", keys, torch.int32), ("sorted_pos", sorted_pos, torch.int64)):
            if len(ts) != W:
                raise ValueError(f"{name}: expected {W} tensors")
            for t in ts:
                if t is not None and t.numel() and (t.dtype != dt or not t.is_cuda
                                                    or not t.is_contiguous()):
                    raise ValueError(f"{name} must be contiguous CUDA {dt} tensors")
        items = [0 if t is None else t.numel() for t in keys]
        if any((0 if t is None else t.numel()) != m for t, m in zip(sorted_pos, items)):
            raise ValueError("sorted_pos must have one entry per item")
        if any((0 if t is None else t.numel()) < m * int(row_bytes)
               for t, m in zip(item_out, items)):
            raise ValueError("item_out[r] must hold one row per item of rank r")
        own = None
        if workspace is not None:
            self._scratch(workspace)
        else:
            own = (9, "combine_items", COMBINE_WORKSPACE_BYTES)
            workspace = self._default_workspace("combine_items", COMBINE_WORKSPACE_BYTES, stream)
        peer_arr, host_p = self._buffers(peers, "peers")
        out_arr, host_o = self._buffers(item_out, "item_out")
        if host_p or host_o:
            raise ValueError("a2av_combine_items takes device buffers only")
        ptr = lambda ts: [0 if t is None or t.numel() == 0 else t.data_ptr() for t in ts]
        args = [self.handle, int(keys_per_peer), _ptr_array(list(peer_arr)), sp,
                _ptr_array(ptr(keys)), _ptr_array(ptr(sorted_pos)), _i64_array(items),
                _ptr_array(list(out_arr)), int(row_bytes), ctypes.c_void_p(workspace.data_ptr()),
                int(workspace.numel()), self._queue(stream)]
        if _bind:
            keep = (peers, in_splits, keys, sorted_pos, item_out, workspace)
            return BoundCall(self, load().a2av_combine_items, "a2av_combine_items", args, 11, keep, own)
        self._check(load().a2av_combine_items(*args), "a2av_combine_items")

    # ------------------------------------------- the MoE layer's operators --
    def _dtype(self, tensors, name, allowed):
        """The element type that a list's tensors share, and its code."""
        for t in tensors:
            if t is not None:
                code = self._codes.get(t.dtype)
                if code not in allowed:
                    raise ValueError(f"{name}: {t.dtype} is not supported")
                return t.dtype, code
        raise ValueError(f"{name}: every tensor is missing")

    def _lists(self, *lists):
        """The pointer arrays of lists of W contiguous CUDA tensors, each
        (tensors, dtype, shapes, name): the expected shapes, or None for any.
        A list may be None, and so may a tensor without elements.  Returns the
        addresses (None for None) and what has to live as long as they do."""
        W = self.world_size
        arr = self._room[len(lists)]()
        base = ctypes.addressof(arr)
        if self._marshal.pointers(base, W, *[x[:3] for x in lists]):
            at = base
            out = []
            for x in lists:
                if x[0] is None:
                    out.append(None)
                else:
                    out.append(at)
                    at += 8 * W
            return out, arr
        arrays = [None if x[0] is None else self._list(*x) for x in lists]
        return [None if a is None else ctypes.addressof(a) for a in arrays], arrays

    def _list(self, tensors, dtype, shapes, name):
        """One of these arrays, tensor by tensor: says what is wrong with it."""
        W = self.world_size
        if len(tensors) != W:
            raise ValueError(f"{name}: expected {W} tensors, got {len(tensors)}")
        arr = (ctypes.c_void_p * W)()
        for r, t in enumerate(tensors):
            if t is None:
                if shapes is not None and 0 not in shapes[r]:
                    raise ValueError(f"{name}[{r}] is missing")
                continue
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous CUDA tensors")
            if shapes is not None and t.shape != shapes[r]:
                raise ValueError(f"{name}[{r}] must have shape {tuple(shapes[r])}, "
                                 f"not {tuple(t.shape)}")
            if t.dtype != dtype:
                raise ValueError(f"{name} must be {dtype} tensors, not {t.dtype}")
            arr[r] = t.data_ptr()
        return arr

    def _whole(self, what, stream, *args):
        """The call made by the compiled module in one go.  False when it has
        found something to look at: nothing has been enqueued then."""
        if self.handle is None:
            return False
        rc = getattr(self._marshal, what)(self._entries[what], self._address, self._number(stream),
                                          self.world_size, *args)
        if rc is None:
            return False
        if rc != OK:
            raise A2avError(rc, "a2av_" + what)
        return True

    def _call(self, what, args, keep, bind):
        fn = getattr(load(), what)
        if bind:
            return BoundCall(self, fn, what, args, len(args) - 1, keep)
        rc = fn(*args)
        if rc != OK:
            raise A2avError(rc, what)

    def _tokens(self, tensors, name):
        """Rows and the common second dimension of W [rows, n] tensors."""
        if len(tensors) != self.world_size:
            raise ValueError(f"{name}: expected {self.world_size} tensors, got {len(tensors)}")
        found = self._marshal.rows(tensors)
        if found is not None:
            return found
        shapes = [(0, None) if t is None else t.shape for t in tensors]
        widths = {s[-1] for s in shapes if s[-1:] != (None,)}
        if len(widths) != 1 or any(len(s) != 2 for s in shapes):
            raise ValueError(f"{name} must be 2-D tensors of one width")
        return [s[0] for s in shapes], widths.pop()

    def _route_args(self, logits, keys, weights, weights_name, topk, score, groups, top_groups,
                    group_top, renormalise, scale, d_logits=None):
        if score not in _SCORES:
            raise ValueError(f"score must be one of {sorted(_SCORES)}")
        rows, E = self._tokens(logits, "logits")
        dtype, code = self._dtype(logits, "logits", (F32, BF16, F16))
        topk = int(topk)
        if not 1 <= topk <= E:
            raise ValueError(f"topk must be in 1..{E}")
        route = A2avRoute(E, topk, code, _SCORES[score], int(groups), int(top_groups),
                          int(group_top), 1 if renormalise else 0, scale)
        shapes = [(n, topk) for n in rows]
        arrays, keep = self._lists(
            (logits, dtype, None, "logits"), (keys, self._int32, shapes, "keys"),
            (weights, self._float, shapes, weights_name),
            (d_logits, dtype, [(n, E) for n in rows] if d_logits is not None else None, "d_logits"))
        return route, arrays, self._counts(*rows), E, keep

    def route(self, logits, keys, weights, topk: int, counts=None, bias=None,
              score: str = "softmax", groups: int = 1, top_groups: int = 1, group_top: int = 1,
              renormalise: bool = True, scale: float = 1.0, stream=None, _bind=False):
        """Routing to experts (see include/a2av_moe.h, a2av_route).

        ``logits[r]``: rank r's [T, E] CUDA tensor (float32, bfloat16 or
        float16).  Written: ``keys[r]`` int32 [T, topk], the keys of a
        dispatch; ``weights[r]`` float32 [T, topk]; ``counts`` (optional)
        int64 [W, E], rank r's items for each expert.  ``bias``: optional
        float32 [E], added to the scores for the choice alone."""
        if not _bind and self._whole("route", stream, logits, keys, weights, topk, counts, bias,
                                     _SCORES.get(score), groups, top_groups, group_top, renormalise,
                                     scale):
            return
        cfg, (x, k, w, _), n, E, arrays = self._route_args(
            logits, keys, weights, "weights", topk, score, groups, top_groups, group_top,
            renormalise, scale)
        if bias is not None and (bias.dtype != self._float or not bias.is_cuda
                                 or bias.shape != (E,) or not bias.is_contiguous()):
            raise ValueError(f"bias must be a contiguous CUDA float32 [{E}] tensor")
        if counts is not None:
            self._matrix(counts, (self.world_size, E), "counts")
        args = [self.handle, ctypes.byref(cfg), x, n, None if bias is None else bias.data_ptr(), k, w,
                None if counts is None else counts.data_ptr(), self._queue(stream)]
        return self._call("a2av_route", args, (logits, keys, weights, counts, bias, arrays), _bind)

    def bind_route(self, logits, keys, weights, topk: int, **options) -> BoundCall:
        """``route`` marshalled once (see BoundCall)."""
        return self.route(logits, keys, weights, topk, **options, _bind=True)

    def route_backward(self, logits, keys, d_weights, d_logits, topk: int, score: str = "softmax",
                       renormalise: bool = True, scale: float = 1.0, stream=None):
        """The gradient of ``route``'s weights: ``d_logits[r]`` [T, E], of the
        logits' type, from ``d_weights[r]`` float32 [T, topk] and the keys that
        ``route`` wrote (see include/a2av_moe.h, a2av_route_backward)."""
        if d_logits is None:
            raise ValueError("d_logits is missing")
        if self._whole("route_backward", stream, logits, keys, d_weights, d_logits, topk,
                       _SCORES.get(score), renormalise, scale):
            return
        cfg, (x, k, w, d), n, E, arrays = self._route_args(
            logits, keys, d_weights, "d_weights", topk, score, 1, 1, 1, renormalise, scale, d_logits)
        self._call("a2av_route_backward",
                   [self.handle, ctypes.byref(cfg), x, n, k, w, d, self._queue(stream)], None, False)

    def _expert_args(self, rows, counts, weights, out, out_name, activation, gated):
        """The shape, the common arguments and what the others are checked by."""
        if activation not in _ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}")
        W = self.world_size
        n, D = self._tokens(rows, "rows")
        n_out, N = self._tokens(out, out_name)
        if n_out != n:
            raise ValueError(f"rows and {out_name} must have the same number of rows")
        if len(weights) != W or any(w is None or w.dim() != 3 for w in weights):
            raise ValueError(f"weights must be {W} tensors [experts, features, {D}]")
        K, Z = weights[0].shape[0], 2 * N if gated else N
        dtype, code = self._dtype(weights, "weights", (F16, BF16))
        self._matrix(counts, (W, W * K), "counts")
        shape = A2avExpert(K, D, N, code, _ACTIVATIONS[activation], int(bool(gated)))
        return shape, n, K, Z, dtype

    def expert_matmul(self, rows, counts, weights, outputs, activation: str = "none",
                      gated: bool = False, bias=None, residual=None, pre=None, stream=None,
                      _bind=False):
        """One product per expert (see include/a2av_moe.h, a2av_expert_matmul).

        ``rows[p]``: peer p's [rows, D] bfloat16 or float16 tensor in the
        dispatch's order; ``counts`` int64 [W, W * K] as ``route`` writes it;
        ``weights[p]`` [K, Z, D] with Z = N, or 2 N when ``gated``; written:
        ``outputs[p]`` [rows, N] and, when given, ``pre[p]`` [rows, Z].
        ``bias[p]`` [K, Z] and ``residual[p]`` [rows, N] are optional."""
        if not _bind and self._whole("expert_matmul", stream, rows, counts, weights, outputs,
                                     _ACTIVATIONS.get(activation), gated, bias, residual, pre):
            return
        shape, n, K, Z, dtype = self._expert_args(rows, counts, weights, outputs, "outputs",
                                                  activation, gated)
        D, N, W = shape.in_features, shape.out_features, self.world_size
        by_row = [(m, N) for m in n]
        (x, w, b, r, y, z), arrays = self._lists(
            (rows, dtype, None, "rows"), (weights, dtype, [(K, Z, D)] * W, "weights"),
            (bias, dtype, [(K, Z)] * W, "bias"), (residual, dtype, by_row, "residual"),
            (outputs, dtype, by_row, "outputs"), (pre, dtype, [(m, Z) for m in n], "pre"))
        args = [self.handle, ctypes.byref(shape), x, self._counts(*n), counts.data_ptr(), w, b, r, y,
                z, self._queue(stream)]
        keep = (rows, counts, weights, outputs, bias, residual, pre, arrays)
        return self._call("a2av_expert_matmul", args, keep, _bind)

    def bind_expert_matmul(self, rows, counts, weights, outputs, **options) -> BoundCall:
        """``expert_matmul`` marshalled once (see BoundCall): new counts and rows
        are allowed within the buffers' row counts."""
        return self.expert_matmul(rows, counts, weights, outputs, **options, _bind=True)

    def expert_matmul_backward(self, rows, counts, weights, d_outputs, d_rows=None, d_weights=None,
                               d_bias=None, pre=None, activation: str = "none",
                               gated: bool = False, workspace=None, stream=None):
        """The gradients of ``expert_matmul`` (see include/a2av_moe.h,
        a2av_expert_matmul_backward): any of ``d_rows``, ``d_weights`` and
        ``d_bias``, of the shapes of ``rows``, ``weights`` and the bias.
        ``pre`` is what the forward call wrote, needed with an activation or a
        gate.  ``workspace``: scratch that no other call in flight has; by default
        the object keeps a buffer for each stream in each thread, and a call under
        capture takes its own from the graph's memory."""
        kept = workspace if workspace is not None else self._held("expert_matmul_backward", stream)
        if self._whole("expert_matmul_backward", stream, rows, counts, weights, d_outputs, d_rows,
                       d_weights, d_bias, pre, _ACTIVATIONS.get(activation), gated, kept,
                       self._entries["expert_matmul_workspace_bytes"]):
            return
        shape, n, K, Z, dtype = self._expert_args(rows, counts, weights, d_outputs, "d_outputs",
                                                  activation, gated)
        D, N, W = shape.in_features, shape.out_features, self.world_size
        need = a2av_expert_matmul_workspace_bytes(W, shape, sum(n))
        if need < 0:
            raise A2avError(ERR_UNSUPPORTED, "a2av_expert_matmul_workspace_bytes")
        activated = activation != "none" or bool(gated)
        if activated and pre is None:
            raise ValueError("an activation's gradient needs pre")
        if workspace is not None:
            self._scratch(workspace)
        elif need:
            workspace = self._default_workspace("expert_matmul_backward", need, stream)
        each, by_row = [(K, Z, D)] * W, [(m, D) for m in n]
        (x, w, z, dy, dx, dw, db), arrays = self._lists(
            (rows, dtype, by_row, "rows"), (weights, dtype, each, "weights"),
            (pre if activated else None, dtype, [(m, Z) for m in n], "pre"),
            (d_outputs, dtype, [(m, N) for m in n], "d_outputs"), (d_rows, dtype, by_row, "d_rows"),
            (d_weights, dtype, each, "d_weights"), (d_bias, dtype, [(K, Z)] * W, "d_bias"))
        args = [self.handle, ctypes.byref(shape), x, self._counts(*n), counts.data_ptr(), w, z, dy, dx,
                dw, db, workspace.data_ptr() if need else None,
                workspace.numel() * workspace.element_size() if need else 0,
                self._queue(stream)]
        self._call("a2av_expert_matmul_backward", args, None, False)

    def _weighted_args(self, in_splits, keys, sorted_pos, keys_per_peer, token_rows, name, peers,
                       by_choice):
        """What both directions of the weighted combine share: K, k, H, the type
        and its code, the rows of the ranks and of the peers' buffers (lists of
        which are in ``peers``, as (tensors or None, name)).  k is the number of a
        token's items; without any token, the width that keys or the lists
        ``by_choice`` (weights) have."""
        self._matrix(in_splits, (self.world_size, self.world_size), "in_splits")
        n, H = self._tokens(token_rows, name)
        dtype, code = self._dtype(token_rows, name, (F32, BF16, F16))
        sizes = [self._marshal.sizes(ts) or [0 if t is None else t.numel() for t in ts]
                 for ts in (keys, sorted_pos)]
        k = next((m // T for m, T in zip(sizes[0], n) if T), None)
        if k is None:
            k = next((ts[0].shape[1] for ts in (keys, *by_choice)
                      if ts is not None and ts[0] is not None and ts[0].dim() == 2), 1)
        k = k or 1
        items = [T * k for T in n]
        for m, what in zip(sizes, ("keys", "sorted_pos")):
            if m != items:
                raise ValueError(f"{what} must have one entry per item of each rank")
        held = None
        for ts, what in peers:
            if ts is None:
                continue
            if len(ts) != self.world_size:
                raise ValueError(f"{what}: expected {self.world_size} tensors, got {len(ts)}")
            found = self._marshal.rows(ts)
            if found is None:  # None among them, or of other shapes
                if any(t is not None and (t.dim() != 2 or t.shape[1] != H) for t in ts):
                    raise ValueError(f"{what} must be [rows, {H}] tensors")
                found = [0 if t is None else t.shape[0] for t in ts], H
            if found[1] != H:
                raise ValueError(f"{what} must be [rows, {H}] tensors")
            if held is not None and found[0] != held:
                raise ValueError("peers and d_peers must have the same number of rows")
            held = found[0]
        return int(keys_per_peer), k, H, dtype, code, n, held

    def combine_weighted(self, peers, in_splits, keys, sorted_pos, keys_per_peer: int, weights,
                         outputs, residual=None, stream=None, _bind=False):
        """The weighted return path (see include/a2av_moe.h, a2av_combine_weighted).

        ``peers[p]``: peer p's rows, [rows, H] in the dispatch's layout;
        ``in_splits``, ``keys`` and ``sorted_pos`` as the dispatch took or
        wrote them (topk items a token); ``weights[r]`` float32 [T, topk], or
        None for 1; ``outputs[r]`` and the optional ``residual[r]`` [T, H]."""
        if not _bind and self._whole("combine_weighted", stream, peers, in_splits, keys, sorted_pos,
                                     keys_per_peer, weights, outputs, residual):
            return
        K, k, H, dtype, code, n, held = self._weighted_args(
            in_splits, keys, sorted_pos, keys_per_peer, outputs, "outputs", ((peers, "peers"),),
            (weights,))
        shapes = [(m, H) for m in n]
        (x, ka, pa, w, r, y), arrays = self._lists(
            (peers, dtype, None, "peers"), (keys, self._int32, None, "keys"),
            (sorted_pos, self._int64, None, "sorted_pos"),
            (weights, self._float, [(m, k) for m in n], "weights"),
            (residual, dtype, shapes, "residual"), (outputs, dtype, shapes, "outputs"))
        args = [self.handle, K, k, H, code, x, self._counts(*held), in_splits.data_ptr(), ka, pa, w,
                self._counts(*n), r, y, self._queue(stream)]
        keep = (peers, in_splits, keys, sorted_pos, weights, outputs, residual, arrays)
        return self._call("a2av_combine_weighted", args, keep, _bind)

    def bind_combine_weighted(self, peers, in_splits, keys, sorted_pos, keys_per_peer: int,
                              weights, outputs, **options) -> BoundCall:
        """``combine_weighted`` marshalled once (see BoundCall)."""
        return self.combine_weighted(peers, in_splits, keys, sorted_pos, keys_per_peer, weights,
                                     outputs, **options, _bind=True)

    def combine_weighted_backward(self, peers, in_splits, keys, sorted_pos, keys_per_peer: int,
                                  weights, d_outputs, d_peers=None, d_weights=None, stream=None):
        """The gradients of ``combine_weighted`` (see include/a2av_moe.h,
        a2av_combine_weighted_backward): ``d_peers[p]`` in the peers' layout,
        ``d_weights[r]`` float32 [T, topk]; either may be None (``peers`` too,
        without ``d_weights``)."""
        if (d_peers is None and d_weights is None) or (d_weights is not None and peers is None):
            raise ValueError("d_peers, or d_weights with peers, must be given")
        if self._whole("combine_weighted_backward", stream, peers, in_splits, keys, sorted_pos,
                       keys_per_peer, weights, d_outputs, d_peers, d_weights):
            return
        K, k, H, dtype, code, n, held = self._weighted_args(
            in_splits, keys, sorted_pos, keys_per_peer, d_outputs, "d_outputs",
            ((peers, "peers"), (d_peers, "d_peers")), (weights, d_weights))
        shapes = [(m, k) for m in n]
        (x, ka, pa, w, dy, dx, dw), arrays = self._lists(
            (peers, dtype, None, "peers"), (keys, self._int32, None, "keys"),
            (sorted_pos, self._int64, None, "sorted_pos"), (weights, self._float, shapes, "weights"),
            (d_outputs, dtype, [(m, H) for m in n], "d_outputs"), (d_peers, dtype, None, "d_peers"),
            (d_weights, self._float, shapes, "d_weights"))
        args = [self.handle, K, k, H, code, x, self._counts(*held), in_splits.data_ptr(), ka, pa, w,
                self._counts(*n), dy, dx, dw, self._queue(stream)]
        self._call("a2av_combine_weighted_backward", args, None, False)

    def status(self, stream=None) -> int:
        rc, v = a2av_status(self.handle, self._stream(stream))
        self._check(rc, "a2av_status")
        return v

    def last_launch(self):
        rc, p, g, b = a2av_last_launch(self.handle)
        self._check(rc, "a2av_last_launch")
        return {"path": p, "grid": g, "block": b}

    def last_dispatch(self):
        """What the last ``dispatch`` or ``combine_items`` enqueued."""
        rc, k, m, name = a2av_last_dispatch(self.handle)
        self._check(rc, "a2av_last_dispatch")
        return {"kernels": k, "memsets": m, "copy_kernel": name}

    def close(self):
        if self.handle is not None:
            a2av_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

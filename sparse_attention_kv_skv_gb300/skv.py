"""Python binding of libskv.so (include/skv.h): argument marshalling only.

Every function has the name of the C entry point it calls and passes plain
integers (device or host addresses, sizes, CUDA stream handles) through
ctypes.  No step of the path runs in Python, and there is no fallback: if the
library is missing, importing this module raises.

``Context`` is a convenience wrapper that takes torch tensors (it reads their
``data_ptr()`` and torch's current CUDA stream) and raises ``SkvError`` for
non-OK statuses.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libskv.so")

SKV_OK = 0
SKV_ERR_INVALID_ARG = 1
SKV_ERR_OOM = 2
SKV_ERR_BAD_REQUEST = 3
SKV_ERR_NO_FREE_REQUEST = 4
SKV_ERR_CONTEXT_FULL = 5
SKV_ERR_CUDA = 6

SKV_DEVERR_BAD_REQUEST = 1
SKV_DEVERR_BAD_INDEX = 2
SKV_DEVERR_DUPLICATE = 4
SKV_DEVERR_CONTEXT_FULL = 8
SKV_DEVERR_TIMEOUT = 16

SKV_Q4_ROW_BYTES = 336


class skv_config(ctypes.Structure):
    _fields_ = [
        ("max_requests", ctypes.c_int32),
        ("num_layers", ctypes.c_int32),
        ("max_context", ctypes.c_int64),
        ("row_bytes", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("hot_slots", ctypes.c_int32),
        ("max_batch", ctypes.c_int32),
        ("device", ctypes.c_int32),
    ]


class skv_index(ctypes.Structure):
    _fields_ = [
        ("keys", ctypes.c_void_p),
        ("request_stride", ctypes.c_int64),
        ("layer_stride", ctypes.c_int64),
        ("key_stride", ctypes.c_int64),
        ("heads", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("block", ctypes.c_int32),
        ("first", ctypes.c_int32),
        ("last", ctypes.c_int32),
        ("relu", ctypes.c_int32),
    ]


class skv_prefix(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_void_p),
        ("layer_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("n", ctypes.c_int64),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_attention_kv_skv_gb300.build` "
                          "(the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
    P = ctypes.POINTER
    sigs = {
        "skv_create": [P(skv_config), P(vp)],
        "skv_destroy": [vp],
        "skv_publish": [vp, vp, i64, P(i32), vp],
        "skv_write_back": [vp, vp, i32, vp, vp],
        "skv_extend": [vp, i32, vp, i64, vp],
        "skv_assemble": [vp, vp, i32, vp, vp, vp, vp, vp],
        "skv_assemble_host": [vp, vp, i32, vp, vp, vp, vp, vp],
        "skv_assemble_noalloc": [vp, vp, i32, vp, vp, vp, vp, vp],
        "skv_assemble_layer": [vp, vp, i32, i32, vp, vp, vp, vp, vp],
        "skv_prefetch": [vp, vp, i32, i32, vp, vp, vp, vp],
        "skv_prefetch_recent": [vp, vp, i32, i32, i32, vp, vp, vp],
        "skv_release": [vp, i32, vp],
        "skv_get_device_error": [vp, P(i32), vp],
        "skv_hot_buffer": [vp, P(vp), P(i64)],
        "skv_pool_rows": [vp, P(vp)],
        "skv_export_state": [vp, i32, vp, vp, vp, vp, vp, vp, vp],
        "skv_export_hot": [vp, i32, vp, vp],
        "skv_get_clock": [vp, P(ctypes.c_uint32), vp],
        "skv_get_stats": [vp, P(ctypes.c_uint64), P(ctypes.c_uint64), P(ctypes.c_uint64), vp],
        "skv_set_gather_events": [vp, vp, vp],
        "skv_set_attend_sms": [vp, i32],
        "skv_selftest_mma": [vp, vp, vp, i32, i32, i32, vp],
        "skv_attend": [vp, vp, i32, i32, vp, vp, vp, vp, ctypes.c_float, vp],
        "skv_selftest_attend_timeout": [vp, vp, i32, vp, vp, vp, vp],
        "skv_attend_q4": [vp, vp, i32, i32, vp, vp, vp, vp, ctypes.c_float, vp],
        "skv_pack_rows": [vp, vp, i64, i64, vp, vp, vp],
        "skv_unpack_rows": [vp, vp, i64, vp, vp],
        "skv_select_workspace": [vp, P(skv_index), i32, i32, P(i64)],
        "skv_select": [vp, P(skv_index), vp, i32, i32, vp, vp, vp, vp, i64, vp],
        "skv_selftest_select_timeout": [vp, P(skv_index), vp, i32, vp, vp, vp, vp, i64, vp],
        "skv_attend_prefix_workspace": [vp, P(skv_prefix), i32, i32, i32, P(i64)],
        "skv_attend_prefix": [vp, P(skv_prefix), i32, i32, i32, vp, vp, vp, ctypes.c_float, vp, i64, vp],
        "skv_join": [vp, i32, vp, vp, i64, vp, vp, vp],
        "skv_weigh_prefix_workspace": [vp, P(skv_prefix), i32, i32, i32, P(i64)],
        "skv_weigh_prefix": [vp, P(skv_prefix), i32, i32, i32, vp, vp, vp, i64, vp, i64, ctypes.c_float, ctypes.c_float, vp, i64, vp],
        "skv_evict_prefix_workspace": [vp, P(skv_prefix), i32, P(i64)],
        "skv_evict_prefix": [vp, P(skv_prefix), i32, vp, i64, i32, i32, i32, vp, vp, vp, vp, i64, vp],
        "skv_selftest_prefix_timeout": [vp, P(skv_prefix), i32, i32, vp, vp, vp, vp, i64, vp, i64, vp],
        "skv_pool_placement": [vp, P(i32), P(i32), P(ctypes.c_float)],
        "skv_host_node_for_pci": [ctypes.c_char_p, ctypes.c_char_p, P(i32)],
    }
    for name, args in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = st
    lib.skv_last_cuda_error.argtypes = []
    lib.skv_last_cuda_error.restype = ctypes.c_char_p
    lib.skv_status_string.argtypes = [st]
    lib.skv_status_string.restype = ctypes.c_char_p
    return lib


lib = _load()

# The C entry points under their own names (raw: they return the status).
skv_create = lib.skv_create
skv_destroy = lib.skv_destroy
skv_publish = lib.skv_publish
skv_write_back = lib.skv_write_back
skv_extend = lib.skv_extend
skv_assemble = lib.skv_assemble
skv_assemble_host = lib.skv_assemble_host
skv_assemble_noalloc = lib.skv_assemble_noalloc
skv_assemble_layer = lib.skv_assemble_layer
skv_prefetch = lib.skv_prefetch
skv_prefetch_recent = lib.skv_prefetch_recent
skv_release = lib.skv_release
skv_get_device_error = lib.skv_get_device_error
skv_hot_buffer = lib.skv_hot_buffer
skv_pool_rows = lib.skv_pool_rows
skv_export_state = lib.skv_export_state
skv_export_hot = lib.skv_export_hot
skv_get_clock = lib.skv_get_clock
skv_get_stats = lib.skv_get_stats
skv_set_gather_events = lib.skv_set_gather_events
skv_set_attend_sms = lib.skv_set_attend_sms
skv_selftest_mma = lib.skv_selftest_mma
skv_attend = lib.skv_attend
skv_attend_q4 = lib.skv_attend_q4
skv_select = lib.skv_select
skv_select_workspace = lib.skv_select_workspace
skv_pack_rows = lib.skv_pack_rows
skv_unpack_rows = lib.skv_unpack_rows
skv_selftest_attend_timeout = lib.skv_selftest_attend_timeout
skv_selftest_select_timeout = lib.skv_selftest_select_timeout
skv_attend_prefix_workspace = lib.skv_attend_prefix_workspace
skv_attend_prefix = lib.skv_attend_prefix
skv_join = lib.skv_join
skv_weigh_prefix_workspace = lib.skv_weigh_prefix_workspace
skv_weigh_prefix = lib.skv_weigh_prefix
skv_evict_prefix_workspace = lib.skv_evict_prefix_workspace
skv_evict_prefix = lib.skv_evict_prefix
skv_selftest_prefix_timeout = lib.skv_selftest_prefix_timeout
skv_pool_placement = lib.skv_pool_placement
skv_host_node_for_pci = lib.skv_host_node_for_pci
skv_last_cuda_error = lib.skv_last_cuda_error
skv_status_string = lib.skv_status_string


def host_node_for_pci(pci_bus_id: str, sysfs_root: str | None = None) -> int:
    """The host NUMA node nearest a PCI device (see skv_host_node_for_pci)."""
    n = ctypes.c_int32()
    check(skv_host_node_for_pci(sysfs_root.encode() if sysfs_root else None, pci_bus_id.encode(), ctypes.byref(n)),
          "skv_host_node_for_pci")
    return n.value


class SkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = f"{what}: {skv_status_string(status).decode()}"
        if status == SKV_ERR_CUDA:
            msg += f" ({skv_last_cuda_error().decode()})"
        super().__init__(msg)
        self.status = status


def check(status: int, what: str) -> None:
    if status != SKV_OK:
        raise SkvError(status, what)


def _raw_stream(device: int) -> int:
    """torch.cuda.current_stream(device).cuda_stream, in 0.1 instead of 4 us (replaced by torch's own at the first call)."""
    global _raw_stream
    import torch
    torch.cuda.init()
    _raw_stream = torch._C._cuda_getCurrentRawStream
    return _raw_stream(device)


def _stream_handle(stream, device: int) -> int:
    """A stream argument of a context on `device`: None -> torch's current stream of
    that device; an int -> as is; a torch.cuda.Stream -> its handle."""
    if stream is None:
        return _raw_stream(device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data  # numpy


_dtypes = {}  # torch's, by the names used here (filled at the first use: this module does not import torch)


def _is_type(t, dtype: str) -> bool:
    if not _dtypes:
        import torch
        _dtypes.update(bf16=torch.bfloat16, fp32=torch.float32, int32=torch.int32)
    return t.dtype is _dtypes[dtype]


def _need(t, dtype: str | None, nbytes: int, device: int, what: str, pinned: bool = False) -> None:
    """t is contiguous, of the type and size, and on the context's device (or, if allowed, in pinned host memory).
    An address given as an int is taken as it is."""
    if isinstance(t, int):
        return
    if dtype is not None and t.dtype is not _dtypes.get(dtype) and not _is_type(t, dtype):
        raise ValueError(f"{what} must be {dtype}, not {t.dtype}")
    if t.nbytes < nbytes or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous and hold {nbytes} bytes")
    if t.get_device() != device:
        _elsewhere(t, device, what, pinned)


def _elsewhere(t, device: int, what: str, pinned: bool = False) -> None:
    """Of a tensor that is not on the context's device."""
    if not (pinned and not t.is_cuda and t.is_pinned()):
        raise ValueError(f"{what} must be on the context's device (cuda:{device})" + (" or in pinned host memory" if pinned else ""))


@dataclasses.dataclass
class Config:
    max_requests: int
    num_layers: int
    max_context: int
    topk: int
    hot_slots: int
    max_batch: int
    row_bytes: int = 1152
    device: int = 0

    def c(self) -> skv_config:
        return skv_config(self.max_requests, self.num_layers, self.max_context, self.row_bytes, self.topk,
                          self.hot_slots, self.max_batch, self.device)


class Index:
    """The index keys a Top-k is selected by: keys [R][L][n][dim] bf16 on the
    device (any strides with adjacent dims; n >= ceil(max_context / block)), one
    key for `block` tokens (see skv_index)."""

    def __init__(self, keys, block: int = 1, first: int = 0, last: int = 0, relu: bool = True):
        self.keys, self.block = keys, block
        self.first, self.last, self.relu = first, last, int(bool(relu))

    def __setattr__(self, name, value):
        if name == "keys" and (value.dim() != 4 or value.stride(3) != 1 or not _is_type(value, "bf16")):
            raise ValueError("Index: keys must be [requests][layers][keys][dim] bf16 with adjacent values")
        object.__setattr__(self, name, value)
        # the C descriptions of what the index is now, by heads: calls of several threads may be under way
        object.__setattr__(self, "_c", {})

    def c(self, heads: int = 1):
        s = self._c.get(heads)
        if s is None:
            k = self.keys
            s = self._c[heads] = skv_index(k.data_ptr(), 2 * k.stride(0), 2 * k.stride(1), 2 * k.stride(2), heads, k.shape[3],
                                           self.block, self.first, self.last, self.relu)
        return ctypes.byref(s)

    def fits(self, cfg: Config) -> bool:
        n = self.keys.shape
        return n[0] >= cfg.max_requests and n[1] >= cfg.num_layers and n[2] * self.block >= cfg.max_context


class Prefix:
    """The rows of a text that a whole batch starts with: rows [L][n][576] bf16 on
    the device (any strides with adjacent values; see skv_prefix)."""

    def __init__(self, rows):
        self.rows = rows

    def __setattr__(self, name, value):
        if name == "rows":
            layers, n, dim = value.shape if value.dim() == 3 else (0, 0, 0)
            if dim != 576 or value.stride(2) != 1 or not _is_type(value, "bf16"):
                raise ValueError("Prefix: rows must be [layers][tokens][576] bf16 with adjacent values")
            # described once: a call of few tokens takes less time on the GPU than such look-ups take here
            c = skv_prefix(value.data_ptr(), 2 * value.stride(0), 2 * value.stride(1), n)
            object.__setattr__(self, "_made", (ctypes.byref(c), layers, n, value.get_device()))
        object.__setattr__(self, name, value)

    def c(self):
        return self._made[0]

    @property
    def n(self) -> int:
        return self._made[2]


_pointers = [ctypes.c_void_p * (2 * i) for i in range(9)]  # a join's parts: their outs, then their lses


class PrefixCalls:
    """The calls of a Context around a prefix that a whole batch shares."""

    def _prefix(self, prefix: Prefix, q, layer: int, B: int | None, what: str):
        """What a call's description starts with: (the prefix, B, units, heads, tokens, the context's device)."""
        c, layers, n, dev = prefix._made
        if layers < self.cfg.num_layers:
            raise ValueError(f"{what}: the prefix has fewer layers than the context")
        if dev != self.cfg.device:
            _elsewhere(prefix.rows, self.cfg.device, f"{what}: the prefix")
        layers = 1 if layer >= 0 else self.cfg.num_layers
        if q is None:
            return c, 0, layers, 0, n, self.cfg.device
        shape = q.shape
        if len(shape) != 3 or shape[2] != 576:
            raise ValueError(f"{what}: q must be [units][heads][576]")
        if B is None:
            B, rest = divmod(shape[0], layers)
            if rest:
                raise ValueError(f"{what}: q must hold a unit of every layer for each entry of the batch")
        return c, B, B * layers, shape[1], n, self.cfg.device

    def _weights(self, t, n: int, dev: int, what: str) -> int:
        """The row stride of weights [L][n] fp32 with adjacent values."""
        shape = t.shape
        if len(shape) != 2 or shape[0] < self.cfg.num_layers or shape[1] < n or not _is_type(t, "fp32"):
            raise ValueError(f"{what} must be [layers][tokens] fp32")
        step = t.stride()
        if shape[1] > 1 and step[1] != 1:
            raise ValueError(f"{what} must have adjacent values")
        if t.get_device() != dev:
            _elsewhere(t, dev, what)
        return step[0]

    def attend_prefix_workspace(self, prefix: Prefix, B: int, heads: int = 128, layer: int = -1) -> int:
        """Bytes of workspace an attend_prefix() of B entries needs."""
        n = ctypes.c_int64()
        check(skv_attend_prefix_workspace(self.h, prefix.c(), B, heads, layer, ctypes.byref(n)), "skv_attend_prefix_workspace")
        return n.value

    def attend_prefix(self, prefix: Prefix, q, out, lse, workspace, layer: int = -1, sm_scale: float | None = None,
                      B: int | None = None, stream=None) -> None:
        """MLA attention of a batch over a prefix that all of it shares (see skv_attend_prefix):
        q [units][heads][576] bf16 -> out [units][heads][512] bf16, lse [units][heads] (or None).
        workspace: attend_prefix_workspace() bytes."""
        c, B, units, heads, _, dev = self._prefix(prefix, q, layer, B, "attend_prefix")
        rows = units * heads
        _need(q, "bf16", rows * 1152, dev, "attend_prefix: q")
        _need(out, "bf16", rows * 1024, dev, "attend_prefix: out")
        if lse is not None:
            _need(lse, "fp32", rows * 4, dev, "attend_prefix: lse")
        _need(workspace, None, 0, dev, "attend_prefix: workspace")
        status = skv_attend_prefix(self.h, c, B, heads, layer, q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
                                   1.0 / 24.0 if sm_scale is None else sm_scale, workspace.data_ptr(), workspace.nbytes,
                                   _raw_stream(dev) if stream is None else _stream_handle(stream, dev))
        if status:
            check(status, "skv_attend_prefix")

    def join(self, outs, lses, out, lse=None, stream=None) -> None:
        """Join attention results over disjoint sets of tokens (see skv_join): outs, up to 8 of
        [...][512] bf16, and lses [...] fp32 -> out, lse, which may take a part's place."""
        parts, dev, size = len(outs), self.cfg.device, out.numel()
        if len(lses) != parts or not 1 <= parts <= 8:
            raise ValueError("join: 1 to 8 parts, each with its lse")
        if out.shape[-1] != 512:
            raise ValueError("join: out must be [...][512]")
        rows = size // 512
        for o, e in zip(outs, lses):
            if o.numel() != size or e.numel() != rows:
                raise ValueError("join: the parts and the result differ in size")
            _need(o, "bf16", rows * 1024, dev, "join: outs")
            _need(e, "fp32", rows * 4, dev, "join: lses")
        _need(out, "bf16", rows * 1024, dev, "join: out")
        if lse is not None:
            _need(lse, "fp32", rows * 4, dev, "join: lse")
        both = _pointers[parts](*[o.data_ptr() for o in outs], *[e.data_ptr() for e in lses])
        status = skv_join(self.h, parts, both, ctypes.byref(both, 8 * parts), rows,
                          out.data_ptr(), None if lse is None else lse.data_ptr(),
                          _raw_stream(dev) if stream is None else _stream_handle(stream, dev))
        if status:
            check(status, "skv_join")

    def weigh_prefix_workspace(self, prefix: Prefix, B: int, heads: int = 128, layer: int = -1) -> int:
        """Bytes of workspace a weigh_prefix() of B entries needs."""
        n = ctypes.c_int64()
        check(skv_weigh_prefix_workspace(self.h, prefix.c(), B, heads, layer, ctypes.byref(n)), "skv_weigh_prefix_workspace")
        return n.value

    def weigh_prefix(self, prefix: Prefix, q, lse, weights, out, workspace, layer: int = -1, sm_scale: float | None = None,
                     gain: float = 1.0, B: int | None = None, stream=None) -> None:
        """out = weights (or 0 for None) + gain times the attention weight that each of the prefix's
        tokens receives from the batch (see skv_weigh_prefix): q [units][heads][576] bf16, lse
        [units][heads], weights and out [L][n] fp32 (may be the same)."""
        c, B, units, heads, n, dev = self._prefix(prefix, q, layer, B, "weigh_prefix")
        rows = units * heads
        _need(q, "bf16", rows * 1152, dev, "weigh_prefix: q")
        _need(lse, "fp32", rows * 4, dev, "weigh_prefix: lse")
        w_stride = 0 if weights is None else self._weights(weights, n, dev, "weigh_prefix: weights")
        o_stride = self._weights(out, n, dev, "weigh_prefix: out")
        _need(workspace, None, 0, dev, "weigh_prefix: workspace")
        status = skv_weigh_prefix(self.h, c, B, heads, layer, q.data_ptr(), lse.data_ptr(), None if weights is None else weights.data_ptr(),
                                  w_stride, out.data_ptr(), o_stride, 1.0 / 24.0 if sm_scale is None else sm_scale, gain,
                                  workspace.data_ptr(), workspace.nbytes,
                                  _raw_stream(dev) if stream is None else _stream_handle(stream, dev))
        if status:
            check(status, "skv_weigh_prefix")

    def evict_prefix_workspace(self, prefix: Prefix, layer: int = -1) -> int:
        """Bytes of workspace an evict_prefix() needs."""
        n = ctypes.c_int64()
        check(skv_evict_prefix_workspace(self.h, prefix.c(), layer, ctypes.byref(n)), "skv_evict_prefix_workspace")
        return n.value

    def evict_prefix(self, prefix: Prefix, weights, kept, rows, kept_weights, workspace, first: int = 0, last: int = 0,
                     layer: int = -1, stream=None) -> None:
        """Keep a prefix's heaviest tokens (see skv_evict_prefix): weights [L][n] fp32 -> kept
        [layers of the call][keep] int32, ascending, their rows [..][keep][576] bf16 and weights [..][keep] (either may be
        None).  Prefix(rows) takes the old one's place."""
        c, _, layers, _, n, dev = self._prefix(prefix, None, layer, None, "evict_prefix")
        keep = kept.shape[-1]
        stride = self._weights(weights, n, dev, "evict_prefix: weights")
        _need(kept, "int32", 4 * layers * keep, dev, "evict_prefix: kept")
        if rows is not None:
            _need(rows, "bf16", 1152 * layers * keep, dev, "evict_prefix: rows")
        if kept_weights is not None:
            _need(kept_weights, "fp32", 4 * layers * keep, dev, "evict_prefix: kept_weights")
        _need(workspace, None, 0, dev, "evict_prefix: workspace")
        status = skv_evict_prefix(self.h, c, layer, weights.data_ptr(), stride, keep, first, last, kept.data_ptr(),
                                  None if rows is None else rows.data_ptr(), None if kept_weights is None else kept_weights.data_ptr(),
                                  workspace.data_ptr(), workspace.nbytes,
                                  _raw_stream(dev) if stream is None else _stream_handle(stream, dev))
        if status:
            check(status, "skv_evict_prefix")

    def selftest_prefix_timeout(self, prefix: Prefix, q, lse, out, weights, workspace, B: int | None = None, stream=None) -> None:
        """attend_prefix() (out given) or weigh_prefix() with its loads withheld (see skv_selftest_prefix_timeout)."""
        c, B, _, heads, _, dev = self._prefix(prefix, q, -1, B, "selftest_prefix_timeout")
        check(skv_selftest_prefix_timeout(self.h, c, B, heads, _ptr(q), _ptr(lse), _ptr(out), _ptr(weights),
                                          0 if weights is None else weights.stride(0), _ptr(workspace), workspace.nbytes,
                                          _stream_handle(stream, dev)), "skv_selftest_prefix_timeout")


class Context(PrefixCalls):
    """One library context (pool, hot buffer, maps) on one GPU."""

    def __init__(self, cfg: Config):
        self.cfg = cfg
        h = ctypes.c_void_p()
        c = cfg.c()
        check(skv_create(ctypes.byref(c), ctypes.byref(h)), "skv_create")
        self.h = h.value

    def close(self):
        if getattr(self, "h", None):
            check(skv_destroy(self.h), "skv_destroy")
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # lifecycle -------------------------------------------------------------
    def publish(self, T: int, rows=None, stream=None) -> int:
        r = ctypes.c_int32()
        check(skv_publish(self.h, _ptr(rows), T, ctypes.byref(r), _stream_handle(stream, self.cfg.device)), "skv_publish")
        return r.value

    def release(self, req: int, stream=None) -> None:
        check(skv_release(self.h, req, _stream_handle(stream, self.cfg.device)), "skv_release")

    def write_back(self, req_ids, rows, n: int | None = None, stream=None) -> None:
        n = req_ids.numel() if n is None else n
        check(skv_write_back(self.h, _ptr(req_ids), n, _ptr(rows), _stream_handle(stream, self.cfg.device)), "skv_write_back")

    def extend(self, req: int, rows, n: int, stream=None) -> None:
        """Append n tokens' rows [L][n][row_bytes] to request req."""
        check(skv_extend(self.h, req, _ptr(rows), n, _stream_handle(stream, self.cfg.device)), "skv_extend")

    def assemble(self, req_ids, topk, slots, hits, misses, B: int | None = None, stream=None) -> None:
        B = req_ids.numel() if B is None else B
        check(skv_assemble(self.h, _ptr(req_ids), B, _ptr(topk), _ptr(slots), _ptr(hits), _ptr(misses),
                           _stream_handle(stream, self.cfg.device)), "skv_assemble")

    def assemble_layer(self, layer: int, req_ids, topk, slots, hits, misses, B: int | None = None,
                       stream=None) -> None:
        """One layer's assemble: topk / slots are [B][k], hits / misses [B]."""
        B = req_ids.numel() if B is None else B
        check(skv_assemble_layer(self.h, _ptr(req_ids), B, layer, _ptr(topk), _ptr(slots), _ptr(hits),
                                 _ptr(misses), _stream_handle(stream, self.cfg.device)), "skv_assemble_layer")

    def prefetch(self, req_ids, cand, layer: int = -1, hits=None, misses=None, B: int | None = None,
                 stream=None) -> None:
        """Assemble of the candidate tokens without a slot tensor: cand is [B][L][k]
        (layer -1) or [B][k]; hits / misses ([B][L] or [B]) are optional."""
        B = req_ids.numel() if B is None else B
        check(skv_prefetch(self.h, _ptr(req_ids), B, layer, _ptr(cand), _ptr(hits), _ptr(misses),
                           _stream_handle(stream, self.cfg.device)), "skv_prefetch")

    def prefetch_recent(self, req_ids, n: int, layer: int = -1, hits=None, misses=None, B: int | None = None,
                        stream=None) -> None:
        """Prefetch of each request's n newest tokens (every layer, or one)."""
        B = req_ids.numel() if B is None else B
        check(skv_prefetch_recent(self.h, _ptr(req_ids), B, layer, n, _ptr(hits), _ptr(misses),
                                  _stream_handle(stream, self.cfg.device)), "skv_prefetch_recent")

    def assemble_noalloc(self, req_ids, topk, slots, hits, misses, B: int | None = None, stream=None) -> None:
        """skv_assemble with the gather work list in the library's static
        device array (allocates nothing; see include/skv.h)."""
        B = req_ids.numel() if B is None else B
        check(skv_assemble_noalloc(self.h, _ptr(req_ids), B, _ptr(topk), _ptr(slots), _ptr(hits), _ptr(misses),
                                   _stream_handle(stream, self.cfg.device)), "skv_assemble_noalloc")

    def assemble_host(self, req_ids, topk, slots, hits, misses, B: int | None = None, stream=None) -> None:
        B = len(req_ids) if B is None else B
        check(skv_assemble_host(self.h, _ptr(req_ids), B, _ptr(topk), _ptr(slots), _ptr(hits), _ptr(misses),
                                _stream_handle(stream, self.cfg.device)), "skv_assemble_host")

    def attend(self, req_ids, q, slots, out, lse=None, layer: int = -1, sm_scale: float | None = None,
               B: int | None = None, stream=None) -> None:
        """Sparse MLA attention over assembled slots (see skv_attend):
        q [units][128][576] bf16 -> out [units][128][512] bf16, lse [units][128]."""
        B = req_ids.numel() if B is None else B
        scale = (1.0 / 576 ** 0.5) if sm_scale is None else sm_scale
        check(skv_attend(self.h, _ptr(req_ids), B, layer, _ptr(q), _ptr(slots), _ptr(out), _ptr(lse), scale,
                         _stream_handle(stream, self.cfg.device)), "skv_attend")

    def attend_q4(self, req_ids, q, slots, out, lse=None, layer: int = -1, sm_scale: float | None = None,
                  B: int | None = None, stream=None) -> None:
        """attend() over a hot buffer of packed rows (row_bytes == SKV_Q4_ROW_BYTES; see skv_attend_q4)."""
        B = req_ids.numel() if B is None else B
        scale = (1.0 / 576 ** 0.5) if sm_scale is None else sm_scale
        units = B if layer >= 0 else B * self.cfg.num_layers
        dev = self.cfg.device
        _need(req_ids, "int32", 4 * B, dev, "attend_q4: req_ids")
        _need(q, "bf16", units * 128 * 1152, dev, "attend_q4: q")
        _need(slots, "int32", 4 * units * self.cfg.topk, dev, "attend_q4: slots")
        _need(out, "bf16", units * 128 * 1024, dev, "attend_q4: out")
        if lse is not None:
            _need(lse, "fp32", units * 512, dev, "attend_q4: lse")
        check(skv_attend_q4(self.h, _ptr(req_ids), B, layer, _ptr(q), _ptr(slots), _ptr(out), _ptr(lse), scale,
                            _stream_handle(stream, self.cfg.device)), "skv_attend_q4")

    def select_workspace(self, index: Index, B: int, layer: int = -1) -> int:
        """Bytes of workspace a select() of B entries needs."""
        n = ctypes.c_int64()
        check(skv_select_workspace(self.h, index.c(), B, layer, ctypes.byref(n)), "skv_select_workspace")
        return n.value

    def select(self, index: Index, req_ids, q, w, topk, workspace, layer: int = -1, B: int | None = None,
               stream=None) -> None:
        """Select each unit's Top-k tokens by index scores (see skv_select):
        q [units][heads][dim] bf16, w [units][heads] fp32 -> topk [units][k]
        int32, ascending, -1 behind the last.  workspace: select_workspace() bytes."""
        B = req_ids.numel() if B is None else B
        heads, dim = q.shape[-2:]
        units = B if layer >= 0 else B * self.cfg.num_layers
        if not index.fits(self.cfg):
            raise ValueError("select: the index has fewer requests, layers or keys than the context")
        if dim != index.keys.shape[3]:
            raise ValueError("select: q and the index keys differ in width")
        dev = self.cfg.device
        if index.keys.get_device() != dev:
            _elsewhere(index.keys, dev, "select: the index")
        _need(req_ids, "int32", 4 * B, dev, "select: req_ids")
        _need(q, "bf16", 2 * units * heads * dim, dev, "select: q")
        _need(w, "fp32", 4 * units * heads, dev, "select: w")
        _need(topk, "int32", 4 * units * self.cfg.topk, dev, "select: topk")
        _need(workspace, None, 0, dev, "select: workspace")
        check(skv_select(self.h, index.c(heads), _ptr(req_ids), B, layer, _ptr(q), _ptr(w), _ptr(topk), _ptr(workspace),
                         workspace.nbytes, _stream_handle(stream, self.cfg.device)), "skv_select")

    def pack_rows(self, rows, packed, values=None, stream=None) -> None:
        """bf16 rows [n][576] (rows may lie apart: rows.stride(0)) -> packed rows
        [n][336] bytes and, if given, the bf16 values they stand for [n][576]."""
        shape, step = rows.shape, rows.stride()
        if len(shape) != 2 or shape[1] != 576 or step[1] != 1 or (rows.dtype is not _dtypes.get("bf16") and not _is_type(rows, "bf16")):
            raise ValueError("pack_rows: rows must be [n][576] bf16 with adjacent values")
        n, dev = shape[0], self.cfg.device
        if rows.get_device() != dev:
            _elsewhere(rows, dev, "pack_rows: rows", True)
        _need(packed, None, 336 * n, dev, "pack_rows: packed", True)
        if values is not None:
            _need(values, "bf16", 1152 * n, dev, "pack_rows: values", True)
        status = skv_pack_rows(self.h, rows.data_ptr(), 2 * step[0] if n > 1 else 1152, n, packed.data_ptr(),
                               0 if values is None else values.data_ptr(),
                               _raw_stream(dev) if stream is None else _stream_handle(stream, dev))
        if status:
            check(status, "skv_pack_rows")

    def unpack_rows(self, packed, values, stream=None) -> None:
        """Packed rows [n][336] bytes -> the bf16 values they stand for [n][576]."""
        n, rest = divmod(packed.nbytes, 336)
        if rest or not packed.is_contiguous():
            raise ValueError("unpack_rows: packed must be contiguous and hold whole rows of 336 bytes")
        dev = self.cfg.device
        if packed.get_device() != dev:
            _elsewhere(packed, dev, "unpack_rows: packed", True)
        _need(values, "bf16", 1152 * n, dev, "unpack_rows: values", True)
        status = skv_unpack_rows(self.h, packed.data_ptr(), n, values.data_ptr(),
                                 _raw_stream(dev) if stream is None else _stream_handle(stream, dev))
        if status:
            check(status, "skv_unpack_rows")

    def selftest_attend_timeout(self, req_ids, q, slots, out, B: int | None = None, stream=None) -> None:
        """The attention kernel with its key loads withheld: its waits run out
        and it reports SKV_DEVERR_TIMEOUT (see skv_selftest_attend_timeout)."""
        B = req_ids.numel() if B is None else B
        check(skv_selftest_attend_timeout(self.h, _ptr(req_ids), B, _ptr(q), _ptr(slots), _ptr(out),
                                          _stream_handle(stream, self.cfg.device)), "skv_selftest_attend_timeout")

    def selftest_select_timeout(self, index: Index, req_ids, q, w, topk, workspace, B: int | None = None, stream=None) -> None:
        """select() with its loads withheld (see skv_selftest_select_timeout)."""
        B = req_ids.numel() if B is None else B
        check(skv_selftest_select_timeout(self.h, index.c(q.shape[-2]), _ptr(req_ids), B, _ptr(q), _ptr(w), _ptr(topk),
                                          _ptr(workspace), workspace.nbytes, _stream_handle(stream, self.cfg.device)),
              "skv_selftest_select_timeout")

    # inspection ------------------------------------------------------------
    def get_device_error(self, stream=None) -> int:
        bits = ctypes.c_int32()
        check(skv_get_device_error(self.h, ctypes.byref(bits), _stream_handle(stream, self.cfg.device)), "skv_get_device_error")
        return bits.value

    def hot_buffer(self):
        base, stride = ctypes.c_void_p(), ctypes.c_int64()
        check(skv_hot_buffer(self.h, ctypes.byref(base), ctypes.byref(stride)), "skv_hot_buffer")
        return base.value, stride.value

    def pool_rows(self) -> int:
        base = ctypes.c_void_p()
        check(skv_pool_rows(self.h, ctypes.byref(base)), "skv_pool_rows")
        return base.value

    def export_state(self, req: int, tok2slot: bool = True, stream=None):
        import numpy as np
        L, S, T = self.cfg.num_layers, self.cfg.hot_slots, self.cfg.max_context
        s2t = np.empty((L, S), np.int32)
        ts = np.empty((L, S), np.uint32)
        lru = np.empty((L, S), np.int32)
        t2s = np.empty((L, T), np.int32) if tok2slot else None
        ln = np.zeros(1, np.int64)
        act = np.zeros(1, np.int32)
        check(skv_export_state(self.h, req, _ptr(s2t), _ptr(ts), _ptr(t2s), _ptr(lru), _ptr(ln), _ptr(act),
                               _stream_handle(stream, self.cfg.device)), "skv_export_state")
        return {"slot2tok": s2t, "ts": ts, "lru": lru, "tok2slot": t2s, "len": int(ln[0]), "active": int(act[0])}

    def export_hot(self, req: int, stream=None):
        import numpy as np
        out = np.empty((self.cfg.num_layers, self.cfg.hot_slots, self.cfg.row_bytes), np.uint8)
        check(skv_export_hot(self.h, req, _ptr(out), _stream_handle(stream, self.cfg.device)), "skv_export_hot")
        return out

    def clock(self, stream=None) -> int:
        c = ctypes.c_uint32()
        check(skv_get_clock(self.h, ctypes.byref(c), _stream_handle(stream, self.cfg.device)), "skv_get_clock")
        return c.value

    def stats(self, stream=None):
        a, b, c = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
        check(skv_get_stats(self.h, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c), _stream_handle(stream, self.cfg.device)),
              "skv_get_stats")
        return {"calls": a.value, "hits": b.value, "misses": c.value}

    def pool_placement(self):
        """(wanted node, node holding most sampled pool pages, share there); -1 = none / not reported."""
        a, b, f = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_float()
        check(skv_pool_placement(self.h, ctypes.byref(a), ctypes.byref(b), ctypes.byref(f)), "skv_pool_placement")
        return a.value, b.value, f.value

    def set_attend_sms(self, sms: int = 0) -> None:
        """At most `sms` SMs for later attend() calls (0: all; see skv_set_attend_sms)."""
        check(skv_set_attend_sms(self.h, sms), "skv_set_attend_sms")

    def set_gather_events(self, before=None, after=None) -> None:
        check(skv_set_gather_events(self.h, before.cuda_event if before is not None else None,
                                    after.cuda_event if after is not None else None), "skv_set_gather_events")

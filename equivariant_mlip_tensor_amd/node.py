"""ctypes binding of libtpconv.so's node operators (include/tpconv_node.h).

What a mixture-of-experts potential runs on its atoms around the convolution:
species embedding, routing to experts, the experts' equivariant maps, and
dropout on irreps rows.  As in ``tpconv``, torch supplies device memory and
the stream and every step runs in the library's HIP kernels.

    x = torch.zeros(n, dim, device="cuda")
    tpconv_embedding_forward(types, table, out=x[:, :64])     # the scalar columns
    config = RouteConfig(n_experts=16, top_k=2)
    experts, gates = tpconv_route_forward(config, logits)
    plan   = tpconv_experts_plan("64x0e+64x1o", "64x0e+64x1o", 16, 2, "f32")
    layout = tpconv_experts_layout(plan, experts)
    y      = tpconv_experts_forward(plan, x, weights, experts, gates, layout)
    x      = tpconv_dropout_forward("64x0e+64x1o", 0.1, seed, step, y, residual=x)

Each forward has its backward; the layouts are those of the header.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .tpconv import F32, F64, _check, _lib, _on_launch_stream
from .tpconv import _need as _explain

NODE_EXPORTS = ("tpconv_embedding_forward", "tpconv_embedding_workspace_bytes", "tpconv_embedding_backward",
                "tpconv_route_forward", "tpconv_route_backward", "tpconv_experts_plan", "tpconv_experts_query",
                "tpconv_experts_maps", "tpconv_experts_destroy", "tpconv_experts_layout_bytes",
                "tpconv_experts_layout", "tpconv_experts_forward", "tpconv_experts_workspace_bytes",
                "tpconv_experts_backward", "tpconv_dropout_forward", "tpconv_dropout_backward")

MAX_EXPERTS, MAX_TOP_K, MAX_EXPERT_MUL = 256, 8, 256
_SCORES = {"softmax": 0, "sigmoid": 1}
_CODE = {torch.float32: F32, torch.float64: F64}
_DTYPE = {F32: torch.float32, F64: torch.float64}


class _RouteConfig(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("score", ctypes.c_int32), ("renormalise", ctypes.c_int32),
                ("scale", ctypes.c_double)]


class ExpertsInfo(ctypes.Structure):
    _fields_ = [("dim_in", ctypes.c_int64), ("dim_out", ctypes.c_int64), ("weight_numel", ctypes.c_int64),
                ("n_maps", ctypes.c_int64), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _declare():
    vp, i64, i32, sz, f64, u64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_double,
                                  ctypes.c_uint64)
    text = ctypes.c_char_p
    sig = {
        "tpconv_embedding_forward": (i32, [i32, i64, i64, i64, vp, vp, f64, vp, i64, vp]),
        "tpconv_embedding_workspace_bytes": (sz, [i32, i64, i64, i64]),
        "tpconv_embedding_backward": (i32, [i32, i64, i64, i64, vp, vp, i64, f64, vp, vp, sz, vp]),
        "tpconv_route_forward": (i32, [i32, i64, vp, vp, vp, vp, vp, vp]),
        "tpconv_route_backward": (i32, [i32, i64, vp, vp, vp, vp, vp, vp]),
        "tpconv_experts_plan": (i32, [text, text, i32, i32, i32, ctypes.POINTER(vp)]),
        "tpconv_experts_query": (i32, [vp, ctypes.POINTER(ExpertsInfo)]),
        "tpconv_experts_maps": (i32, [vp, vp]),
        "tpconv_experts_destroy": (None, [vp]),
        "tpconv_experts_layout_bytes": (sz, [vp, i64]),
        "tpconv_experts_layout": (i32, [vp, i64, vp, vp, sz, vp, vp]),
        "tpconv_experts_forward": (i32, [vp, i64, vp, vp, vp, vp, vp, vp, vp]),
        "tpconv_experts_workspace_bytes": (sz, [vp, i64]),
        "tpconv_experts_backward": (i32, [vp, i64] + [vp] * 10 + [sz, vp]),
        "tpconv_dropout_forward": (i32, [text, i32, i64, i64, f64, u64, u64, vp, vp, vp, vp]),
        "tpconv_dropout_backward": (i32, [text, i32, i64, i64, f64, u64, u64, vp, vp, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(_lib, name)
        f.restype = res
        f.argtypes = args


_declare()


# These calls are short enough for their checks to show: the common case of
# each is a few attribute reads, and pointers go to ctypes as integers.
def _need(t, shape, dtype, name):
    if t is None or t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _explain(t, shape, dtype, name)
    return t


def _need_bytes(t, name):
    """A device buffer of any dtype; its size and alignment are the library's to check."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous cuda tensor, got {tuple(t.shape)} on {t.device}, "
                         f"strides={t.stride()}")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream_handle(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _code(t: torch.Tensor, name: str) -> int:
    code = _CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: float32 or float64 expected, got {t.dtype}")
    return code


def _rows_view(t, n: int, dim: int, dtype, name: str) -> int:
    """Row stride (elements) of a device tensor [n, dim] with unit column stride."""
    if not t.is_cuda or t.dtype != dtype or tuple(t.shape) != (n, dim) or (n > 0 and dim > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected {dtype} cuda tensor of shape {(n, dim)} with unit column stride, "
                         f"got {t.dtype} {tuple(t.shape)} (cuda={t.is_cuda}, strides={t.stride()})")
    stride = t.stride(0)
    if n <= 1:
        return max(stride, dim)
    if stride < dim:
        raise ValueError(f"{name}: rows overlap (row stride {stride} below {dim})")
    return stride


# ------------------------------------------------------------------ embedding
def tpconv_embedding_workspace_bytes(dtype, n_rows: int, n_types: int, dim: int) -> int:
    return int(_lib.tpconv_embedding_workspace_bytes(_CODE.get(dtype, dtype), int(n_rows), int(n_types), int(dim)))


@_on_launch_stream
def tpconv_embedding_forward(types, table, scale: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """out[i] = scale * table[types[i]] (zeros for a type outside the table).  types: int32 [n], table:
    [n_types, dim]; out: [n, dim], may be a view of wider rows (x[:, :dim])."""
    if table.dim() != 2:
        raise ValueError("table must be 2-D")
    n, (n_types, dim), dt = types.numel(), table.shape, table.dtype
    code = _code(table, "table")
    _need(types, (n,), torch.int32, "types")
    _need(table, (n_types, dim), dt, "table")
    if out is None:
        out = table.new_empty((n, dim))
    stride = _rows_view(out, n, dim, dt, "out")
    _check(_lib.tpconv_embedding_forward(code, n, n_types, dim, _ptr(types), _ptr(table), float(scale), _ptr(out),
                                         stride, _stream_handle(stream)))
    return out


@_on_launch_stream
def tpconv_embedding_backward(types, grad_out, n_types: int, scale: float = 1.0, grad_table=None, workspace=None,
                              stream=None) -> torch.Tensor:
    """grad_table [n_types, dim] of <grad_out, tpconv_embedding_forward(types, table, scale)>.  grad_out:
    [n, dim], may be a view of wider rows."""
    if grad_out.dim() != 2:
        raise ValueError("grad_out must be 2-D")
    n, dim, dt = types.numel(), grad_out.shape[1], grad_out.dtype
    code = _code(grad_out, "grad_out")
    _need(types, (n,), torch.int32, "types")
    stride = _rows_view(grad_out, n, dim, dt, "grad_out")
    if grad_table is None:
        grad_table = grad_out.new_empty((n_types, dim))
    _need(grad_table, (n_types, dim), dt, "grad_table")
    if workspace is None:
        need = int(_lib.tpconv_embedding_workspace_bytes(code, n, n_types, dim))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=grad_out.device)
    _need_bytes(workspace, "workspace")
    _check(_lib.tpconv_embedding_backward(code, n, n_types, dim, _ptr(types), _ptr(grad_out), stride, float(scale),
                                          _ptr(grad_table), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream_handle(stream)))
    return grad_table


# -------------------------------------------------------------------- routing
class RouteConfig:
    """Routing of rows to experts: top_k of n_experts by softmax or sigmoid scores, optionally inside the top_groups
    best of n_groups groups; gates are scale * score, or renormalised over the chosen to sum to scale."""

    def __init__(self, n_experts: int, top_k: int, score: str = "softmax", n_groups: int = 1, top_groups: int = None,
                 renormalise: bool = True, scale: float = 1.0):
        if score not in _SCORES:
            raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
        self.n_experts, self.top_k = int(n_experts), int(top_k)
        self.n_groups = int(n_groups)
        self.top_groups = self.n_groups if top_groups is None else int(top_groups)
        self.score, self.renormalise, self.scale = score, bool(renormalise), float(scale)
        self.struct = _RouteConfig(self.n_experts, self.top_k, self.n_groups, self.top_groups, _SCORES[score],
                                   int(self.renormalise), self.scale)
        self._ref = ctypes.byref(self.struct)


@_on_launch_stream
def tpconv_route_forward(config: RouteConfig, logits, bias=None, experts=None, gates=None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(experts int32 [n, top_k], gates [n, top_k]) for logits [n, n_experts]; bias [n_experts] moves the selection
    only.  Masked experts have logit or bias -inf; places without an expert get -1 and gate 0."""
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    n, dt, dev = logits.shape[0], logits.dtype, logits.device
    code = _code(logits, "logits")
    _need(logits, (n, config.n_experts), dt, "logits")
    if bias is not None:
        _need(bias, (config.n_experts,), dt, "bias")
    shape = (n, config.top_k)
    if experts is None:
        experts = torch.empty(shape, dtype=torch.int32, device=dev)
    if gates is None:
        gates = logits.new_empty(shape)
    _need(experts, shape, torch.int32, "experts")
    _need(gates, shape, dt, "gates")
    _check(_lib.tpconv_route_forward(code, n, config._ref, _ptr(logits), _ptr(bias), _ptr(experts), _ptr(gates),
                                     _stream_handle(stream)))
    return experts, gates


@_on_launch_stream
def tpconv_route_backward(config: RouteConfig, logits, experts, grad_gates, grad_logits=None,
                          stream=None) -> torch.Tensor:
    """grad_logits [n, n_experts] of <grad_gates, gates> for the forward's experts."""
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    n, dt = logits.shape[0], logits.dtype
    code = _code(logits, "logits")
    _need(logits, (n, config.n_experts), dt, "logits")
    _need(experts, (n, config.top_k), torch.int32, "experts")
    _need(grad_gates, (n, config.top_k), dt, "grad_gates")
    if grad_logits is None:
        grad_logits = torch.empty_like(logits)
    _need(grad_logits, (n, config.n_experts), dt, "grad_logits")
    _check(_lib.tpconv_route_backward(code, n, config._ref, _ptr(logits), _ptr(experts), _ptr(grad_gates),
                                      _ptr(grad_logits), _stream_handle(stream)))
    return grad_logits


# -------------------------------------------------------------------- experts
class ExpertsPlan:
    """Owns a tpconv_experts_t; sizes as attributes."""

    def __init__(self, handle: ctypes.c_void_p):
        self.handle = handle
        info = ExpertsInfo()
        _check(_lib.tpconv_experts_query(handle, ctypes.byref(info)))
        self.info = info
        for f, _ in ExpertsInfo._fields_:
            setattr(self, f, getattr(info, f))
        self.torch_dtype = _DTYPE[info.dtype]

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.tpconv_experts_destroy(h)


class ExpertsLayout:
    """The order of one routing's rows and entries, in the device tensor it lives in."""

    def __init__(self, plan: ExpertsPlan, n_rows: int, buffer: torch.Tensor):
        self.plan, self.n_rows, self.buffer = plan, n_rows, buffer


def tpconv_experts_plan(irreps_in: str, irreps_out: str, n_experts: int, top_k: int, dtype="f32") -> ExpertsPlan:
    dt = {"f32": F32, "f64": F64, torch.float32: F32, torch.float64: F64, F32: F32, F64: F64}.get(dtype, dtype)
    h = ctypes.c_void_p()
    _check(_lib.tpconv_experts_plan(irreps_in.encode(), irreps_out.encode(), int(n_experts), int(top_k), int(dt),
                                    ctypes.byref(h)))
    return ExpertsPlan(h)


def tpconv_experts_query(plan: ExpertsPlan) -> ExpertsInfo:
    info = ExpertsInfo()
    _check(_lib.tpconv_experts_query(plan.handle, ctypes.byref(info)))
    return info


def tpconv_experts_maps(plan: ExpertsPlan):
    """List of (segment of irreps_in, segment of irreps_out, l, weight offset)."""
    buf = (ctypes.c_int64 * (4 * plan.n_maps))()
    _check(_lib.tpconv_experts_maps(plan.handle, buf))
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(plan.n_maps)]


def tpconv_experts_destroy(plan: ExpertsPlan) -> None:
    plan.__del__()


def tpconv_experts_layout_bytes(plan: ExpertsPlan, n_rows: int) -> int:
    return int(_lib.tpconv_experts_layout_bytes(plan.handle, int(n_rows)))


def tpconv_experts_workspace_bytes(plan: ExpertsPlan, n_rows: int) -> int:
    return int(_lib.tpconv_experts_workspace_bytes(plan.handle, int(n_rows)))


@_on_launch_stream
def tpconv_experts_layout(plan: ExpertsPlan, experts, load=None, buffer=None, stream=None) -> ExpertsLayout:
    """The layout of one routing (experts int32 [n, top_k]); load: int32 [n_experts], gets each expert's entries."""
    n = experts.shape[0]
    _need(experts, (n, plan.top_k), torch.int32, "experts")
    if load is not None:
        _need(load, (plan.n_experts,), torch.int32, "load")
    if buffer is None:
        need = int(_lib.tpconv_experts_layout_bytes(plan.handle, n))
        buffer = torch.empty(max(need, 256), dtype=torch.uint8, device=experts.device)
    _need_bytes(buffer, "buffer")
    _check(_lib.tpconv_experts_layout(plan.handle, n, _ptr(experts), _ptr(buffer),
                                      buffer.numel() * buffer.element_size(), _ptr(load), _stream_handle(stream)))
    return ExpertsLayout(plan, n, buffer)


def _layout_of(plan, n: int, layout):
    if layout is None:
        return None
    if layout.plan is not plan or layout.n_rows != n:
        raise ValueError("layout belongs to another plan or another number of rows")
    return _ptr(layout.buffer)


@_on_launch_stream
def tpconv_experts_forward(plan: ExpertsPlan, x, weights, experts, gates, layout: Optional[ExpertsLayout] = None,
                           out=None, stream=None) -> torch.Tensor:
    """out [n, dim_out] = sum over a row's experts of gate * expert's map of x [n, dim_in].  weights:
    [n_experts, weight_numel]; layout: of these experts, or None (rows as they come, the same result)."""
    n, dt, k = x.shape[0], plan.torch_dtype, plan.top_k
    _need(x, (n, plan.dim_in), dt, "x")
    _need(weights, (plan.n_experts, plan.weight_numel), dt, "weights")
    _need(experts, (n, k), torch.int32, "experts")
    _need(gates, (n, k), dt, "gates")
    if out is None:
        out = x.new_empty((n, plan.dim_out))
    _need(out, (n, plan.dim_out), dt, "out")
    _check(_lib.tpconv_experts_forward(plan.handle, n, _ptr(x), _ptr(weights), _ptr(experts), _ptr(gates),
                                       _layout_of(plan, n, layout), _ptr(out), _stream_handle(stream)))
    return out


@_on_launch_stream
def tpconv_experts_backward(plan: ExpertsPlan, x, weights, experts, gates, grad_out,
                            layout: Optional[ExpertsLayout] = None, grad_x=None, grad_weights=None, grad_gates=None,
                            need=(True, True, True), workspace=None,
                            stream=None) -> Tuple[Optional[torch.Tensor], ...]:
    """(grad_x, grad_weights, grad_gates) of <grad_out, tpconv_experts_forward(...)>; an output is None when `need`
    turns it off.  grad_weights needs the layout."""
    n, dt, k = x.shape[0], plan.torch_dtype, plan.top_k
    _need(x, (n, plan.dim_in), dt, "x")
    _need(weights, (plan.n_experts, plan.weight_numel), dt, "weights")
    _need(experts, (n, k), torch.int32, "experts")
    _need(gates, (n, k), dt, "gates")
    _need(grad_out, (n, plan.dim_out), dt, "grad_out")
    dev = x.device
    if need[0] and grad_x is None:
        grad_x = torch.empty((n, plan.dim_in), dtype=dt, device=dev)
    if need[1] and grad_weights is None:
        grad_weights = torch.empty((plan.n_experts, plan.weight_numel), dtype=dt, device=dev)
    if need[2] and grad_gates is None:
        grad_gates = torch.empty((n, k), dtype=dt, device=dev)
    for t, shp, nm in ((grad_x, (n, plan.dim_in), "grad_x"),
                       (grad_weights, (plan.n_experts, plan.weight_numel), "grad_weights"),
                       (grad_gates, (n, k), "grad_gates")):
        if t is not None:
            _need(t, shp, dt, nm)
    if workspace is None and (grad_weights is not None or grad_gates is not None):
        bytes_ = int(_lib.tpconv_experts_workspace_bytes(plan.handle, n))
        workspace = torch.empty(max(bytes_, 256), dtype=torch.uint8, device=dev)
    held = 0 if workspace is None else _need_bytes(workspace, "workspace").numel() * workspace.element_size()
    _check(_lib.tpconv_experts_backward(plan.handle, n, _ptr(x), _ptr(weights), _ptr(experts), _ptr(gates),
                                        _layout_of(plan, n, layout), _ptr(grad_out), _ptr(grad_x),
                                        _ptr(grad_weights), _ptr(grad_gates), _ptr(workspace), held,
                                        _stream_handle(stream)))
    return grad_x, grad_weights, grad_gates


# -------------------------------------------------------------------- dropout
@_on_launch_stream
def tpconv_dropout_forward(irreps: str, p: float, seed: int, offset: int, x, residual=None, out=None,
                           stream=None) -> torch.Tensor:
    """residual + keep * x / (1 - p) on irreps rows, one draw per channel; the mask depends on seed, offset and a
    channel's place alone.  out may be x or residual itself."""
    code = _code(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    _need(x, x.shape, x.dtype, "x")
    if residual is not None:
        _need(residual, x.shape, x.dtype, "residual")
    if out is None:
        out = torch.empty_like(x)
    _need(out, x.shape, x.dtype, "out")
    _check(_lib.tpconv_dropout_forward(irreps.encode(), code, x.shape[0], x.shape[1], float(p), int(seed), int(offset),
                                       _ptr(x), _ptr(residual), _ptr(out), _stream_handle(stream)))
    return out


@_on_launch_stream
def tpconv_dropout_backward(irreps: str, p: float, seed: int, offset: int, grad_out, grad_x=None,
                            stream=None) -> torch.Tensor:
    """keep * grad_out / (1 - p) with the forward's seed and offset (the residual's gradient is grad_out)."""
    code = _code(grad_out, "grad_out")
    if grad_out.dim() != 2:
        raise ValueError("grad_out must be 2-D")
    _need(grad_out, grad_out.shape, grad_out.dtype, "grad_out")
    if grad_x is None:
        grad_x = torch.empty_like(grad_out)
    _need(grad_x, grad_out.shape, grad_out.dtype, "grad_x")
    _check(_lib.tpconv_dropout_backward(irreps.encode(), code, grad_out.shape[0], grad_out.shape[1], float(p), int(seed),
                                        int(offset), _ptr(grad_out), _ptr(grad_x), _stream_handle(stream)))
    return grad_x

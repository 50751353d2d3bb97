"""ctypes binding of libtpconv.so's node operators (include/tpconv_node.h).

What a mixture-of-experts potential, or one with a feed-forward block, runs on
its atoms around the convolution: species embedding, routing to experts, the
experts' equivariant maps, dropout on irreps rows, their norm with the
residual's sum, rows in 8 bits, gated feed-forward products and linear maps.  As in ``tpconv``, torch supplies device memory and
the stream and every step runs in the library's HIP kernels.

    x = torch.zeros(n, dim, device="cuda")
    tpconv_embedding_forward(types, table, out=x[:, :64])     # the scalar columns
    config = RouteConfig(n_experts=16, top_k=2)
    experts, gates = tpconv_route_forward(config, logits)
    plan   = tpconv_experts_plan("64x0e+64x1o", "64x0e+64x1o", 16, 2, "f32")
    layout = tpconv_experts_layout(plan, experts)
    y      = tpconv_experts_forward(plan, x, weights, experts, gates, layout)
    x      = tpconv_dropout_forward("64x0e+64x1o", 0.1, seed, step, y, residual=x)

    norm   = tpconv_norm_plan("64x0e+64x1o")
    gated  = tpconv_gated_plan("64x0e+64x1o", "128x0e+128x1o")
    linear = tpconv_linear_plan("128x0e+128x1o", "64x0e+64x1o")
    y, h, kept = tpconv_norm_forward(norm, x, residual, gamma, need=(True, True, True))
    t      = tpconv_gated_forward(gated, y, weights, gate_weights, gate_bias)
    x      = tpconv_linear_forward(linear, t, weights2, bias, residual=h)
    ...                                       # y is freed; its rows in 8 bits, kept, serve the gradient
    g_y, g_weights, g_gate_weights, g_bias = tpconv_gated_backward(gated, kept, weights, gate_weights, gate_bias, g_t)

Each forward has its backward; the layouts are those of the header.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from .tpconv import F32, F64, _check, _lib, _on_launch_stream
from .tpconv import _need as _explain

NODE_EXPORTS = ("tpconv_embedding_forward", "tpconv_embedding_workspace_bytes", "tpconv_embedding_backward",
                "tpconv_route_forward", "tpconv_route_backward", "tpconv_experts_plan", "tpconv_experts_query",
                "tpconv_experts_maps", "tpconv_experts_destroy", "tpconv_experts_layout_bytes",
                "tpconv_experts_layout", "tpconv_experts_forward", "tpconv_experts_workspace_bytes",
                "tpconv_experts_backward", "tpconv_dropout_forward", "tpconv_dropout_backward",
                "tpconv_norm_plan", "tpconv_norm_query", "tpconv_norm_destroy", "tpconv_norm_forward",
                "tpconv_norm_workspace_bytes", "tpconv_norm_backward", "tpconv_pack8", "tpconv_unpack8",
                "tpconv_gated_plan", "tpconv_linear_plan", "tpconv_dense_query", "tpconv_dense_maps",
                "tpconv_dense_destroy", "tpconv_gated_forward", "tpconv_linear_forward",
                "tpconv_dense_workspace_bytes", "tpconv_gated_backward", "tpconv_linear_backward")

MAX_EXPERTS, MAX_TOP_K, MAX_EXPERT_MUL = 256, 8, 256
MAX_NORM_DIM, MAX_DENSE_MUL = 8192, 1024
_SCOPES = {"segment": 0, "row": 1}
_ACTIVATIONS = {"identity": 0, "silu": 1, "sigmoid": 2, "tanh": 3, "gelu": 4}
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


class NormInfo(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int64), ("channels", ctypes.c_int64), ("n_segments", ctypes.c_int32),
                ("scope", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("eps", ctypes.c_double)]


class DenseInfo(ctypes.Structure):
    _fields_ = [("dim_in", ctypes.c_int64), ("dim_out", ctypes.c_int64), ("weight_numel", ctypes.c_int64),
                ("n_maps", ctypes.c_int64), ("n_gates", ctypes.c_int64), ("n_scalars", ctypes.c_int64),
                ("n_bias", ctypes.c_int64), ("n_segments_in", ctypes.c_int32), ("dtype", ctypes.c_int32)]


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
        "tpconv_norm_plan": (i32, [text, i32, f64, i32, ctypes.POINTER(vp)]),
        "tpconv_norm_query": (i32, [vp, ctypes.POINTER(NormInfo)]),
        "tpconv_norm_destroy": (None, [vp]),
        "tpconv_norm_forward": (i32, [vp, i64] + [vp] * 8),
        "tpconv_norm_workspace_bytes": (sz, [vp, i64]),
        "tpconv_norm_backward": (i32, [vp, i64] + [vp] * 7 + [sz, vp]),
        "tpconv_pack8": (i32, [text, i64, i64, vp, vp, vp, vp]),
        "tpconv_unpack8": (i32, [text, i64, i64, vp, vp, vp, vp]),
        "tpconv_gated_plan": (i32, [text, text, i32, i32, i32, ctypes.POINTER(vp)]),
        "tpconv_linear_plan": (i32, [text, text, i32, i32, ctypes.POINTER(vp)]),
        "tpconv_dense_query": (i32, [vp, ctypes.POINTER(DenseInfo)]),
        "tpconv_dense_maps": (i32, [vp, vp]),
        "tpconv_dense_destroy": (None, [vp]),
        "tpconv_gated_forward": (i32, [vp, i64] + [vp] * 6),
        "tpconv_linear_forward": (i32, [vp, i64] + [vp] * 6),
        "tpconv_dense_workspace_bytes": (sz, [vp, i64]),
        "tpconv_gated_backward": (i32, [vp, i64] + [vp] * 12 + [sz, vp]),
        "tpconv_linear_backward": (i32, [vp, i64] + [vp] * 10 + [sz, vp]),
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


# ----------------------------------------------------------------------- norm
def _dtype_code(dtype):
    return {"f32": F32, "f64": F64, torch.float32: F32, torch.float64: F64, F32: F32, F64: F64}.get(dtype, dtype)


# The calls below launch on the current device, where all of their tensors have to be.
def _here(t, shape, dtype, name):
    if t is None or t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _explain(t, shape, dtype, name)
    at = torch._C._cuda_getDevice()
    if t.get_device() != at:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{at}")
    return t


def _scratch(need: int, workspace, device):
    """The workspace given, or one made for the call where it needs one, and its bytes."""
    if workspace is None:
        if need == 0:
            return None, 0
        return torch.empty(need, dtype=torch.uint8, device=device), need
    _need_bytes(workspace, "workspace")
    if workspace.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"workspace is on cuda:{workspace.get_device()}, not on the current device")
    return workspace, workspace.numel() * workspace.element_size()


class PackedRows:
    """fp32 irreps rows in 8 bits: codes uint8 [n, dim] (e4m3) and scales float32 [n, segments]."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.codes, self.scales = codes, scales


def _packed_here(packed: PackedRows, n: int, dim: int, n_segments: int):
    _here(packed.codes, (n, dim), torch.uint8, "codes")
    _here(packed.scales, (n, n_segments), torch.float32, "scales")
    return packed


class NormPlan:
    """Owns a tpconv_norm_t; sizes as attributes."""

    def __init__(self, handle: ctypes.c_void_p):
        self.handle = handle
        info = tpconv_norm_query(self)
        self.info = info
        for f, _ in NormInfo._fields_:
            setattr(self, f, getattr(info, f))
        self.torch_dtype = _DTYPE[info.dtype]

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.tpconv_norm_destroy(h)


def tpconv_norm_plan(irreps: str, scope: str = "segment", eps: float = 1e-6, dtype="f32") -> NormPlan:
    """Root-mean-square norm of irreps rows; scope: what is normalised together, each "segment" by itself or the whole
    "row" (its segments counted alike)."""
    if scope not in _SCOPES:
        raise ValueError(f"scope must be 'segment' or 'row', got {scope!r}")
    h = ctypes.c_void_p()
    _check(_lib.tpconv_norm_plan(irreps.encode(), _SCOPES[scope], float(eps), int(_dtype_code(dtype)),
                                 ctypes.byref(h)))
    return NormPlan(h)


def tpconv_norm_query(plan: NormPlan) -> NormInfo:
    info = NormInfo()
    _check(_lib.tpconv_norm_query(plan.handle, ctypes.byref(info)))
    return info


def tpconv_norm_destroy(plan: NormPlan) -> None:
    plan.__del__()


def tpconv_norm_workspace_bytes(plan: NormPlan, n_rows: int) -> int:
    return int(_lib.tpconv_norm_workspace_bytes(plan.handle, int(n_rows)))


@_on_launch_stream
def tpconv_norm_forward(plan: NormPlan, x, residual=None, gamma=None, out=None, sum=None, packed=None,
                        need=(True, True, False), stream=None):
    """(out, sum, packed): the norm of h = x + residual times gamma [channels], h itself (x, where there is no
    residual and no `sum` to write it to), and the norm in 8 bits; an output is None when `need` turns it off.  sum may
    be x or residual itself, or out may."""
    n, dt = x.shape[0], plan.torch_dtype
    shape = (n, plan.dim)
    _here(x, shape, dt, "x")
    if residual is not None:
        _here(residual, shape, dt, "residual")
    if gamma is not None:
        _here(gamma, (plan.channels,), dt, "gamma")
    if out is not None:
        _here(out, shape, dt, "out")
    elif need[0]:
        out = torch.empty_like(x)
    if sum is not None:
        _here(sum, shape, dt, "sum")
    elif need[1] and residual is not None:
        sum = torch.empty_like(x)
    if packed is not None:
        _packed_here(packed, n, plan.dim, plan.n_segments)
    elif need[2]:
        packed = PackedRows(x.new_empty(shape, dtype=torch.uint8),
                            x.new_empty((n, plan.n_segments), dtype=torch.float32))
    if out is not None or sum is not None or packed is not None:
        _check(_lib.tpconv_norm_forward(plan.handle, n, _ptr(x), _ptr(residual), _ptr(gamma), _ptr(sum), _ptr(out),
                                        None if packed is None else packed.codes.data_ptr(),
                                        None if packed is None else packed.scales.data_ptr(),
                                        _stream_handle(stream)))
    return out, x if sum is None and need[1] else sum, packed


@_on_launch_stream
def tpconv_norm_backward(plan: NormPlan, h, gamma, grad_out, grad_sum=None, grad_x=None, grad_gamma=None,
                         need=(True, True), workspace=None,
                         stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(grad_x, grad_gamma) of <grad_out, out> + <grad_sum, sum> for the forward's sum h; grad_x is x's and the
    residual's alike.  An output is None when `need` turns it off.  grad_x may be h, grad_out or grad_sum itself."""
    n, dt = h.shape[0], plan.torch_dtype
    shape = (n, plan.dim)
    _here(h, shape, dt, "h")
    _here(grad_out, shape, dt, "grad_out")
    if gamma is not None:
        _here(gamma, (plan.channels,), dt, "gamma")
    if grad_sum is not None:
        _here(grad_sum, shape, dt, "grad_sum")
    if grad_x is not None:
        _here(grad_x, shape, dt, "grad_x")
    elif need[0]:
        grad_x = torch.empty_like(h)
    if grad_gamma is not None:
        _here(grad_gamma, (plan.channels,), dt, "grad_gamma")
    elif need[1]:
        grad_gamma = h.new_empty(plan.channels)
    held = 0
    if grad_gamma is not None:
        workspace, held = _scratch(int(_lib.tpconv_norm_workspace_bytes(plan.handle, n)), workspace, h.device)
    _check(_lib.tpconv_norm_backward(plan.handle, n, _ptr(h), _ptr(gamma), _ptr(grad_out), _ptr(grad_sum),
                                     _ptr(grad_x), _ptr(grad_gamma), _ptr(workspace), held, _stream_handle(stream)))
    return grad_x, grad_gamma


@functools.lru_cache(maxsize=256)
def _text_and_segments(irreps: str):
    return irreps.encode(), irreps.count("+") + 1


@_on_launch_stream
def tpconv_pack8(irreps: str, x, packed: Optional[PackedRows] = None, stream=None) -> PackedRows:
    """fp32 irreps rows [n, dim] in 8 bits, with a scale for each row and segment."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    _here(x, x.shape, torch.float32, "x")
    text, n_segments = _text_and_segments(irreps)
    n, dim = x.shape
    if packed is None:
        packed = PackedRows(x.new_empty((n, dim), dtype=torch.uint8), x.new_empty((n, n_segments)))
    else:
        _packed_here(packed, n, dim, n_segments)
    _check(_lib.tpconv_pack8(text, n, dim, x.data_ptr(), packed.codes.data_ptr(), packed.scales.data_ptr(),
                             _stream_handle(stream)))
    return packed


@_on_launch_stream
def tpconv_unpack8(irreps: str, packed: PackedRows, out=None, stream=None) -> torch.Tensor:
    """The rows that `packed` stands for [n, dim]: code times scale."""
    if packed.codes.dim() != 2:
        raise ValueError("codes must be 2-D")
    n, dim = packed.codes.shape
    text, n_segments = _text_and_segments(irreps)
    _packed_here(packed, n, dim, n_segments)
    if out is None:
        out = packed.scales.new_empty((n, dim))
    else:
        _here(out, (n, dim), torch.float32, "out")
    _check(_lib.tpconv_unpack8(text, n, dim, packed.codes.data_ptr(), packed.scales.data_ptr(), out.data_ptr(),
                               _stream_handle(stream)))
    return out


# ----------------------------------------------------------- gated and linear
class DensePlan:
    """Owns a tpconv_dense_t (a gated or a linear map's plan); sizes as attributes."""

    def __init__(self, handle: ctypes.c_void_p):
        self.handle = handle
        info = tpconv_dense_query(self)
        self.info = info
        for f, _ in DenseInfo._fields_:
            setattr(self, f, getattr(info, f))
        self.torch_dtype = _DTYPE[info.dtype]

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.tpconv_dense_destroy(h)


def _activation(name, what):
    if name not in _ACTIVATIONS:
        raise ValueError(f"{what} must be one of {', '.join(_ACTIVATIONS)}; got {name!r}")
    return _ACTIVATIONS[name]


def tpconv_gated_plan(irreps_in: str, irreps_out: str, scalar_act: str = "silu", gate_act: str = "sigmoid",
                      dtype="f32") -> DensePlan:
    """Gated feed-forward product; scalar_act acts on the gates of irreps_out's even scalars, gate_act on the other
    channels' gates."""
    h = ctypes.c_void_p()
    _check(_lib.tpconv_gated_plan(irreps_in.encode(), irreps_out.encode(), _activation(scalar_act, "scalar_act"),
                                  _activation(gate_act, "gate_act"), int(_dtype_code(dtype)), ctypes.byref(h)))
    return DensePlan(h)


def tpconv_linear_plan(irreps_in: str, irreps_out: str, act: str = "identity", dtype="f32") -> DensePlan:
    """Equivariant linear map; act acts on irreps_out's even scalars."""
    h = ctypes.c_void_p()
    _check(_lib.tpconv_linear_plan(irreps_in.encode(), irreps_out.encode(), _activation(act, "act"),
                                   int(_dtype_code(dtype)), ctypes.byref(h)))
    return DensePlan(h)


def tpconv_dense_query(plan: DensePlan) -> DenseInfo:
    info = DenseInfo()
    _check(_lib.tpconv_dense_query(plan.handle, ctypes.byref(info)))
    return info


def tpconv_dense_maps(plan: DensePlan):
    """List of (segment of irreps_in, segment of irreps_out, l, weight offset)."""
    buf = (ctypes.c_int64 * (4 * plan.n_maps))()
    _check(_lib.tpconv_dense_maps(plan.handle, buf))
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(plan.n_maps)]


def tpconv_dense_destroy(plan: DensePlan) -> None:
    plan.__del__()


def tpconv_dense_workspace_bytes(plan: DensePlan, n_rows: int) -> int:
    return int(_lib.tpconv_dense_workspace_bytes(plan.handle, int(n_rows)))


@_on_launch_stream
def tpconv_gated_forward(plan: DensePlan, x, weights, gate_weights, gate_bias=None, out=None,
                         stream=None) -> torch.Tensor:
    """out [n, dim_out]: the maps' products of x [n, dim_in], each channel times the activation of its gate, a
    product of x's even scalars.  weights [weight_numel], gate_weights [n_scalars, n_gates], gate_bias [n_gates]."""
    n, dt = x.shape[0], plan.torch_dtype
    _here(x, (n, plan.dim_in), dt, "x")
    _here(weights, (plan.weight_numel,), dt, "weights")
    _here(gate_weights, (plan.n_scalars, plan.n_gates), dt, "gate_weights")
    if gate_bias is not None:
        _here(gate_bias, (plan.n_gates,), dt, "gate_bias")
    if out is None:
        out = x.new_empty((n, plan.dim_out))
    else:
        _here(out, (n, plan.dim_out), dt, "out")
    _check(_lib.tpconv_gated_forward(plan.handle, n, _ptr(x), _ptr(weights), _ptr(gate_weights), _ptr(gate_bias),
                                     _ptr(out), _stream_handle(stream)))
    return out


@_on_launch_stream
def tpconv_linear_forward(plan: DensePlan, x, weights, bias=None, residual=None, out=None,
                          stream=None) -> torch.Tensor:
    """out [n, dim_out] = residual + the maps' products of x [n, dim_in], with bias [n_bias] and the activation on the
    even scalars.  weights [weight_numel]; out may be residual itself."""
    n, dt = x.shape[0], plan.torch_dtype
    _here(x, (n, plan.dim_in), dt, "x")
    _here(weights, (plan.weight_numel,), dt, "weights")
    if bias is not None:
        _here(bias, (plan.n_bias,), dt, "bias")
    if residual is not None:
        _here(residual, (n, plan.dim_out), dt, "residual")
    if out is None:
        out = x.new_empty((n, plan.dim_out))
    else:
        _here(out, (n, plan.dim_out), dt, "out")
    _check(_lib.tpconv_linear_forward(plan.handle, n, _ptr(x), _ptr(weights), _ptr(bias), _ptr(residual), _ptr(out),
                                      _stream_handle(stream)))
    return out


def _input(plan: DensePlan, x, n: int):
    """Pointers to x, its codes and its scales, of rows or of PackedRows."""
    if isinstance(x, PackedRows):
        _packed_here(x, n, plan.dim_in, plan.n_segments_in)
        return None, x.codes.data_ptr(), x.scales.data_ptr()
    _here(x, (n, plan.dim_in), plan.torch_dtype, "x")
    return x.data_ptr(), None, None


@_on_launch_stream
def tpconv_gated_backward(plan: DensePlan, x, weights, gate_weights, gate_bias, grad_out, grad_x=None,
                          grad_weights=None, grad_gate_weights=None, grad_gate_bias=None, need=(True, True, True, None),
                          workspace=None, stream=None) -> Tuple[Optional[torch.Tensor], ...]:
    """(grad_x, grad_weights, grad_gate_weights[, grad_gate_bias]) of <grad_out, tpconv_gated_forward(...)>.  x: the
    forward's rows, or PackedRows of them (the gradients at the restored rows).  An output is None when `need` turns it
    off; the bias's is there where gate_bias is, or where `need` asks for it."""
    n, dt, dev = grad_out.shape[0], plan.torch_dtype, grad_out.device
    _here(grad_out, (n, plan.dim_out), dt, "grad_out")
    rows, codes, scales = _input(plan, x, n)
    _here(weights, (plan.weight_numel,), dt, "weights")
    _here(gate_weights, (plan.n_scalars, plan.n_gates), dt, "gate_weights")
    if gate_bias is not None:
        _here(gate_bias, (plan.n_gates,), dt, "gate_bias")
    with_bias = gate_bias is not None if need[3] is None else need[3]
    if need[0] and grad_x is None:
        grad_x = torch.empty((n, plan.dim_in), dtype=dt, device=dev)
    if need[1] and grad_weights is None:
        grad_weights = torch.empty_like(weights)
    if need[2] and grad_gate_weights is None:
        grad_gate_weights = torch.empty_like(gate_weights)
    if with_bias and grad_gate_bias is None:
        grad_gate_bias = torch.empty(plan.n_gates, dtype=dt, device=dev)
    for t, shp, nm in ((grad_x, (n, plan.dim_in), "grad_x"), (grad_weights, (plan.weight_numel,), "grad_weights"),
                       (grad_gate_weights, (plan.n_scalars, plan.n_gates), "grad_gate_weights"),
                       (grad_gate_bias, (plan.n_gates,), "grad_gate_bias")):
        if t is not None:
            _here(t, shp, dt, nm)
    workspace, held = _scratch(int(_lib.tpconv_dense_workspace_bytes(plan.handle, n)), workspace, dev)
    _check(_lib.tpconv_gated_backward(plan.handle, n, rows, codes, scales, _ptr(weights), _ptr(gate_weights),
                                      _ptr(gate_bias), _ptr(grad_out), _ptr(grad_x), _ptr(grad_weights),
                                      _ptr(grad_gate_weights), _ptr(grad_gate_bias), _ptr(workspace), held,
                                      _stream_handle(stream)))
    got = (grad_x, grad_weights, grad_gate_weights)
    return got + (grad_gate_bias,) if with_bias or grad_gate_bias is not None else got


@_on_launch_stream
def tpconv_linear_backward(plan: DensePlan, x, weights, bias, grad_out, grad_x=None, grad_weights=None, grad_bias=None,
                           need=(True, True, None), workspace=None, stream=None) -> Tuple[Optional[torch.Tensor], ...]:
    """(grad_x, grad_weights[, grad_bias]) of <grad_out, tpconv_linear_forward(...)> (the residual's is grad_out).  x:
    the forward's rows, or PackedRows of them; with the identity as activation grad_x alone may be asked for without
    x (None).  An output is None when `need` turns it off; the bias's is there where bias is, or where `need` asks for
    it."""
    n, dt, dev = grad_out.shape[0], plan.torch_dtype, grad_out.device
    _here(grad_out, (n, plan.dim_out), dt, "grad_out")
    rows, codes, scales = (None, None, None) if x is None else _input(plan, x, n)
    _here(weights, (plan.weight_numel,), dt, "weights")
    if bias is not None:
        _here(bias, (plan.n_bias,), dt, "bias")
    with_bias = bias is not None if need[2] is None else need[2]
    if need[0] and grad_x is None:
        grad_x = torch.empty((n, plan.dim_in), dtype=dt, device=dev)
    if need[1] and grad_weights is None:
        grad_weights = torch.empty_like(weights)
    if with_bias and grad_bias is None:
        grad_bias = torch.empty(plan.n_bias, dtype=dt, device=dev)
    for t, shp, nm in ((grad_x, (n, plan.dim_in), "grad_x"), (grad_weights, (plan.weight_numel,), "grad_weights"),
                       (grad_bias, (plan.n_bias,), "grad_bias")):
        if t is not None:
            _here(t, shp, dt, nm)
    workspace, held = _scratch(int(_lib.tpconv_dense_workspace_bytes(plan.handle, n)), workspace, dev)
    _check(_lib.tpconv_linear_backward(plan.handle, n, rows, codes, scales, _ptr(weights), _ptr(bias), _ptr(grad_out),
                                       _ptr(grad_x), _ptr(grad_weights), _ptr(grad_bias), _ptr(workspace), held,
                                       _stream_handle(stream)))
    got = (grad_x, grad_weights)
    return got + (grad_bias,) if with_bias or grad_bias is not None else got

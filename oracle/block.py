"""Plain fp64 definitions of a feed-forward block's operators on irreps rows:
the root-mean-square norm with the residual's sum, rows in 8 bits, the gated
product, and the linear map with bias, activation and residual.

numpy only, segment by segment, straight from the formulas; shares no code with
the GPU path.  Rows are [n, width]; a segment's columns are [mul][2l+1].  With
`size` the same sums run over absolute values (an activation's factor by its
bound of growth), which is what rounding errors are measured against.
"""

from __future__ import annotations

import math

import numpy as np

from .node import segments

TOP = 448.0      # largest value of an e4m3 code


def channels(irreps: str):
    """First channel of each segment, and their number."""
    out, at = [], 0
    for mul, _, _, _ in segments(irreps)[0]:
        out.append(at)
        at += mul
    return out, at


def part(x, seg):
    """A segment's columns as [n, mul, 2l+1]."""
    mul, l, _, at = seg
    return x[:, at:at + mul * (2 * l + 1)].reshape(len(x), mul, 2 * l + 1)


# ----------------------------------------------------------------------- norm
def factors(irreps, scope, eps, h):
    """r for each row and segment [n, segments]."""
    ms = np.stack([(part(h, s) ** 2).mean((1, 2)) for s in segments(irreps)[0]], 1)
    if scope == "row":
        ms = np.repeat(ms.mean(1, keepdims=True), ms.shape[1], 1)
    return 1.0 / np.sqrt(ms + eps)


def norm_forward(irreps, scope, eps, x, residual=None, gamma=None):
    """(y, h)."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    r = factors(irreps, scope, eps, h)
    first, C = channels(irreps)
    gamma = np.ones(C) if gamma is None else np.asarray(gamma, np.float64)
    y = np.empty_like(h)
    for i, s in enumerate(segments(irreps)[0]):
        part(y, s)[...] = gamma[first[i]:first[i] + s[0]][None, :, None] * part(h, s) * r[:, i][:, None, None]
    return y, h


def norm_backward(irreps, scope, eps, h, gamma, grad_out, grad_sum=None, size=False):
    """(grad_x, grad_gamma); size: of absolute values, with the difference taken as a sum."""
    h, g = np.asarray(h, np.float64), np.asarray(grad_out, np.float64)
    segs = segments(irreps)[0]
    r = factors(irreps, scope, eps, h)
    if size:
        h, g = np.abs(h), np.abs(g)
    first, C = channels(irreps)
    gamma = np.ones(C) if gamma is None else np.asarray(gamma, np.float64)
    w = [(np.abs(gamma) if size else gamma)[f:f + s[0]][None, :, None] for f, s in zip(first, segs)]
    dots = np.stack([(part(g, s) * v * part(h, s)).sum((1, 2)) for s, v in zip(segs, w)], 1)
    columns = np.array([s[0] * (2 * s[1] + 1) for s in segs], np.float64)
    if scope == "row":
        dots = np.repeat(dots.sum(1, keepdims=True), len(segs), 1)
        columns = columns * len(segs)
    grad, g_gamma = np.empty_like(h), np.empty(C)
    for i, s in enumerate(segs):
        rr = r[:, i][:, None, None]
        pull = part(h, s) * rr * (dots[:, i] * r[:, i] / columns[i])[:, None, None]
        part(grad, s)[...] = rr * (part(g, s) * w[i] + (pull if size else -pull))
        g_gamma[first[i]:first[i] + s[0]] = (part(g, s) * part(h, s) * rr).sum((0, 2))
    if grad_sum is not None:
        grad = grad + (np.abs(grad_sum) if size else np.asarray(grad_sum, np.float64))
    return grad, g_gamma


# --------------------------------------------------------------------- 8 bits
def e4m3_values():
    """The value of each of the 256 codes (OCP e4m3: 1-4-3 bits, bias 7, no infinities, NaN where all bits are set)."""
    out = np.empty(256)
    for code in range(256):
        sign, power, frac = -1.0 if code >> 7 else 1.0, (code >> 3) & 15, code & 7
        if power == 15 and frac == 7:
            out[code] = np.nan
        elif power == 0:
            out[code] = sign * frac * 2.0 ** -9
        else:
            out[code] = sign * (1 + frac / 8) * 2.0 ** (power - 7)
    return out


def e4m3_codes(v):
    """The code next to each of v (|v| <= 464), ties to the even code; zeros keep their sign."""
    v = np.asarray(v, np.float64)
    values = e4m3_values()[:127]
    at = np.searchsorted(values, np.abs(v))
    hi = np.minimum(at, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = values[hi] - np.abs(v), np.abs(v) - values[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(v), 127, code)
    return (code + 128 * np.signbit(v)).astype(np.uint8)


def pack8(irreps, x):
    """(codes uint8 [n, width], scales float32 [n, segments]) of fp32 rows; the scale, its inverse and the product
    that is rounded are fp32 numbers."""
    f = np.float32
    x = np.asarray(x, f)
    codes, scales = np.empty(x.shape, np.uint8), np.empty((len(x), len(segments(irreps)[0])), f)
    with np.errstate(all="ignore"):
        for i, (mul, l, _, at) in enumerate(segments(irreps)[0]):
            cols = slice(at, at + mul * (2 * l + 1))
            scale = np.abs(x[:, cols]).max(1) * f(1.0 / TOP)            # max keeps NaN
            scale = np.where(scale < np.finfo(f).tiny, np.finfo(f).tiny, scale).astype(f)
            codes[:, cols] = e4m3_codes((x[:, cols] * (f(1.0) / scale)[:, None]).astype(np.float64))
            scales[:, i] = scale
    return codes, scales


def unpack8(irreps, codes, scales):
    """fp32 rows."""
    out = np.empty(codes.shape, np.float32)
    with np.errstate(all="ignore"):
        for i, (mul, l, _, at) in enumerate(segments(irreps)[0]):
            cols = slice(at, at + mul * (2 * l + 1))
            out[:, cols] = e4m3_values().astype(np.float32)[codes[:, cols]] * scales[:, i][:, None]
    return out


# ---------------------------------------------------------------- activations
def activation(kind, z):
    """(value, slope)."""
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        if kind == "identity":
            return z, np.ones_like(z)
        if kind == "tanh":
            return np.tanh(z), 4.0 / (np.exp(z) + np.exp(-z)) ** 2
        if kind == "gelu":
            below = np.array([0.5 * math.erfc(-v / math.sqrt(2.0)) for v in z.reshape(-1)]).reshape(z.shape)
            return z * below, below + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        s, t = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
        return (s, s * t) if kind == "sigmoid" else (z * s, s + z * s * t)


# ----------------------------------------------------------- gated and linear
def maps(irreps_in, irreps_out):
    """[(segment of irreps_in, segment of irreps_out, first weight)] and the number of weights."""
    out, at = [], 0
    for s in segments(irreps_in)[0]:
        for t in segments(irreps_out)[0]:
            if (s[1], s[2]) == (t[1], t[2]):
                out.append((s, t, at))
                at += s[0] * t[0]
    return out, at


def even_scalars(irreps):
    """The segment 0e, or None."""
    return next((s for s in segments(irreps)[0] if (s[1], s[2]) == (0, "e")), None)


def matrix(weights, s, t, at):
    return np.asarray(weights, np.float64)[at:at + s[0] * t[0]].reshape(s[0], t[0])


def product(x, s, M):
    """sum_u M[u][v] x[i][u][m]."""
    return np.swapaxes(np.swapaxes(part(x, s), 1, 2) @ M, 1, 2)


def gates(irreps_in, irreps_out, x, gate_weights, gate_bias):
    """z of each row and channel of irreps_out."""
    s = even_scalars(irreps_in)
    z = part(x, s)[:, :, 0] @ np.asarray(gate_weights, np.float64)
    return z if gate_bias is None else z + np.asarray(gate_bias, np.float64)


def kinds(irreps_out, scalar_act, gate_act):
    """The activation of each segment of irreps_out."""
    return {(l, p): scalar_act if (l, p) == (0, "e") else gate_act for _, l, p, _ in segments(irreps_out)[0]}


def gated_forward(irreps_in, irreps_out, scalar_act, gate_act, x, weights, gate_weights, gate_bias=None):
    x = np.asarray(x, np.float64)
    out = np.zeros((len(x), segments(irreps_out)[1]))
    z = gates(irreps_in, irreps_out, x, gate_weights, gate_bias)
    first = dict(zip([s[3] for s in segments(irreps_out)[0]], channels(irreps_out)[0]))
    kind = kinds(irreps_out, scalar_act, gate_act)
    for s, t, at in maps(irreps_in, irreps_out)[0]:
        a = activation(kind[t[1], t[2]], z[:, first[t[3]]:first[t[3]] + t[0]])[0]
        part(out, t)[...] = a[:, :, None] * product(x, s, matrix(weights, s, t, at))
    return out


def gated_backward(irreps_in, irreps_out, scalar_act, gate_act, x, weights, gate_weights, gate_bias, grad_out):
    """(grad_x, grad_weights, grad_gate_weights, grad_gate_bias)."""
    x, G = np.asarray(x, np.float64), np.asarray(grad_out, np.float64)
    Wg = np.asarray(gate_weights, np.float64)
    z = gates(irreps_in, irreps_out, x, Wg, gate_bias)
    first = dict(zip([s[3] for s in segments(irreps_out)[0]], channels(irreps_out)[0]))
    kind = kinds(irreps_out, scalar_act, gate_act)
    gx, gW, dz = np.zeros_like(x), np.zeros(len(weights)), np.zeros_like(z)
    for s, t, at in maps(irreps_in, irreps_out)[0]:
        M, c = matrix(weights, s, t, at), slice(first[t[3]], first[t[3]] + t[0])
        a, slope = activation(kind[t[1], t[2]], z[:, c])
        g = part(G, t)
        du = a[:, :, None] * g
        dz[:, c] = slope * (g * product(x, s, M)).sum(2)
        part(gx, s)[...] = np.swapaxes(np.swapaxes(du, 1, 2) @ M.T, 1, 2)
        gW[at:at + M.size] = np.tensordot(part(x, s), du, ((0, 2), (0, 2))).reshape(-1)
    s = even_scalars(irreps_in)
    part(gx, s)[:, :, 0] += dz @ Wg.T
    return gx, gW, part(x, s)[:, :, 0].T @ dz, dz.sum(0)


def linear_forward(irreps_in, irreps_out, act, x, weights, bias=None, residual=None):
    x = np.asarray(x, np.float64)
    out = np.zeros((len(x), segments(irreps_out)[1]))
    for s, t, at in maps(irreps_in, irreps_out)[0]:
        y = product(x, s, matrix(weights, s, t, at))
        if (t[1], t[2]) == (0, "e"):
            y = activation(act, y if bias is None else y + np.asarray(bias, np.float64)[None, :, None])[0]
        part(out, t)[...] = y
    return out if residual is None else out + np.asarray(residual, np.float64)


def linear_backward(irreps_in, irreps_out, act, x, weights, bias, grad_out):
    """(grad_x, grad_weights, grad_bias)."""
    x, G = np.asarray(x, np.float64), np.asarray(grad_out, np.float64)
    gx, gW, gb = np.zeros_like(x), np.zeros(len(weights)), np.zeros(0)
    for s, t, at in maps(irreps_in, irreps_out)[0]:
        M, g = matrix(weights, s, t, at), part(G, t)
        if (t[1], t[2]) == (0, "e"):
            z = product(x, s, M)
            g = g * activation(act, z if bias is None else z + np.asarray(bias, np.float64)[None, :, None])[1]
            gb = g.sum((0, 2))
        part(gx, s)[...] = np.swapaxes(np.swapaxes(g, 1, 2) @ M.T, 1, 2)
        gW[at:at + M.size] = np.tensordot(part(x, s), g, ((0, 2), (0, 2))).reshape(-1)
    return gx, gW, gb


# -------------------------------------------------- sizes for rounding errors
# Bounds of an activation's growth and of its slope's: |a(z + d) - a(z)| <= GROWTH |d|, |a'(z + d) - a'(z)| <= BEND |d|
# (silu: 1.0999, 0.5; sigmoid: 1/4, 0.0963; tanh: 1, 0.7699; gelu: 1.1290, 0.7979).
GROWTH = {"identity": 1.0, "silu": 1.1, "sigmoid": 0.25, "tanh": 1.0, "gelu": 1.13}
BEND = {"identity": 0.0, "silu": 0.5, "sigmoid": 0.1, "tanh": 0.77, "gelu": 0.8}

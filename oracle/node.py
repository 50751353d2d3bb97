"""Plain fp64 definitions of the node operators: species embedding, routing to
experts, the experts' equivariant maps, dropout on irreps rows.

numpy only, one row or one expert at a time, straight from the formulas;
shares no code with the GPU path.  The functions that end in _many are the same
for many rows at a time, in array operations.
"""

from __future__ import annotations

import re

import numpy as np


def segments(irreps: str):
    """[(mul, l, parity, first column)] and the width of a row."""
    out, at = [], 0
    for term in irreps.split("+"):
        m = re.fullmatch(r"\s*(?:(\d+)\s*x\s*)?(\d+)\s*([eo])\s*", term)
        if m is None:
            raise ValueError(f"bad irreps term {term!r}")
        mul, l = int(m.group(1) or 1), int(m.group(2))
        out.append((mul, l, m.group(3), at))
        at += mul * (2 * l + 1)
    return out, at


# ------------------------------------------------------------------ embedding
def embedding_forward(types, table, scale=1.0):
    table = np.asarray(table, np.float64)
    out = np.zeros((len(types), table.shape[1]))
    for i, t in enumerate(types):
        if 0 <= t < len(table):
            out[i] = scale * table[t]
    return out


def embedding_backward(types, grad, n_types, scale=1.0):
    grad = np.asarray(grad, np.float64)
    out = np.zeros((n_types, grad.shape[1]))
    for i, t in enumerate(types):
        if 0 <= t < n_types:
            out[t] += scale * grad[i]
    return out


# -------------------------------------------------------------------- routing
def scores(z, kind):
    """Scores of one row of logits; 0 for a masked (-inf) one."""
    live = ~np.isneginf(z)
    s = np.zeros(len(z))
    if not live.any():
        return s
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            e = np.exp(-np.abs(z[live]))
            s[live] = np.where(z[live] >= 0, 1.0, e) / (1.0 + e)
        else:
            e = np.exp(z[live] - np.max(z[live]))
            s[live] = e / e.sum()
    return s


def keys(z, bias, kind):
    """Selection keys: scores plus bias, -inf for a masked expert (logit or bias -inf), NaN where the score is."""
    s, b = scores(z, kind), np.zeros(len(z)) if bias is None else np.asarray(bias, np.float64)
    masked = np.isneginf(z) | np.isneginf(b)
    return np.where(masked, -np.inf, s + np.where(masked, 0.0, b))


def group_keys(key, n_groups, low=np.finfo(np.float64).min / 2):
    """The sum of a group's two largest unmasked keys; `low` for NaN and for what is below it."""
    out = []
    for g in np.split(key, n_groups):
        live = g[~np.isneginf(g)]
        best = np.sort(np.where(live >= low, live, low))[::-1][:2]
        out.append(best.sum() if len(best) else -np.inf)
    return np.array(out)


def choose(z, bias, cfg, low=np.finfo(np.float64).min / 2):
    """Chosen experts of one row, in order (fewer than top_k when the rest is masked): by descending key, equal keys
    by descending logit, then by index; NaN keys after all others, by index."""
    key = keys(z, bias, cfg["score"])
    if cfg["n_groups"] > 1:
        order = np.argsort(-group_keys(key, cfg["n_groups"], low), kind="stable")[:cfg["top_groups"]]
        inside = np.repeat(np.isin(np.arange(cfg["n_groups"]), order), len(z) // cfg["n_groups"])
        key = np.where(inside, key, -np.inf)
    live = [e for e in range(len(z)) if not np.isneginf(key[e])]
    live.sort(key=lambda e: (1, 0.0, 0.0, e) if np.isnan(key[e]) else (0, -key[e], -z[e], e))
    return live[:cfg["top_k"]]


def log_scores(z, kind):
    """log s up to a constant of the row."""
    return np.minimum(z, 0.0) - np.log1p(np.exp(-np.abs(z))) if kind == "sigmoid" else z


def gates_of(z, picked, cfg):
    if not picked:
        return np.zeros(0)
    if cfg["renormalise"]:
        if cfg["score"] == "softmax" and np.isnan(scores(z, "softmax")).any():
            return np.full(len(picked), np.nan)                # NaN or +inf among the logits
        l = log_scores(z[picked], cfg["score"])
        w = np.exp(l - l.max())
        return cfg["scale"] * w / w.sum()
    return cfg["scale"] * scores(z, cfg["score"])[picked]


def route_forward(logits, bias, cfg):
    z = np.asarray(logits, np.float64)
    low = float(np.finfo(np.asarray(logits).dtype).min) / 2
    experts = np.full((len(z), cfg["top_k"]), -1, np.int32)
    gates = np.zeros((len(z), cfg["top_k"]))
    for i in range(len(z)):
        picked = choose(z[i], bias, cfg, low)
        experts[i, :len(picked)] = picked
        gates[i, :len(picked)] = gates_of(z[i], picked, cfg)
    return experts, gates


def route_backward(logits, experts, grad_gates, cfg):
    """grad_logits through the full Jacobian of the chosen scores; renormalised gates are functions of the chosen logits
    alone, and a masked expert's gradient is 0."""
    z, g = np.asarray(logits, np.float64), np.asarray(grad_gates, np.float64)
    out = np.zeros_like(z)
    for i in range(len(z)):
        at = [a for a in range(cfg["top_k"]) if 0 <= experts[i, a] < z.shape[1]]
        e = [int(experts[i, a]) for a in at]
        if not e:
            continue
        # renormalised over the chosen: as if they were the row
        w = gates_of(z[i, e], list(range(len(e))), cfg) if cfg["renormalise"] else None
        s = scores(z[i], cfg["score"])
        live = ~np.isneginf(z[i])
        ga = g[i, at]
        if cfg["renormalise"]:
            d = w * (ga - np.dot(ga, w) / cfg["scale"]) if cfg["scale"] else 0.0 * w
            if cfg["score"] == "sigmoid":
                d = d * (1.0 - s[e])
            np.add.at(out[i], e, d)
        elif cfg["score"] == "sigmoid":
            np.add.at(out[i], e, cfg["scale"] * ga * s[e] * (1.0 - s[e]))
        else:
            np.add.at(out[i], e, cfg["scale"] * ga * s[e])
            out[i, live] -= cfg["scale"] * s[live] * np.dot(ga, s[e])
    return out


def route_many(logits, bias, cfg):
    """route_forward of numbers and masks (no NaN), and the smallest distance between keys that a row's choice hangs
    on (inf where nothing is near)."""
    z = np.asarray(logits, np.float64)
    n, X = z.shape
    with np.errstate(all="ignore"):
        if cfg["score"] == "sigmoid":
            e = np.exp(-np.abs(z))
            s = np.where(z >= 0, 1.0, e) / (1.0 + e)
        else:
            e = np.where(np.isneginf(z), 0.0, np.exp(z - np.maximum(z.max(1, keepdims=True), -1e300)))
            s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    b = np.zeros(X) if bias is None else np.asarray(bias, np.float64)
    key = np.where(np.isneginf(z) | np.isneginf(b), -np.inf, s + np.where(np.isneginf(b), 0.0, b))
    gap = np.full(n, np.inf)
    if cfg["n_groups"] > 1:
        by = key.reshape(n, cfg["n_groups"], -1)
        two = -np.sort(-by, axis=2)[:, :, :2]
        best = np.where(np.isneginf(two[:, :, 0]), -np.inf, np.where(np.isneginf(two), 0.0, two).sum(2))
        order = np.argsort(-best, axis=1, kind="stable")
        inside = np.zeros(best.shape, bool)
        np.put_along_axis(inside, order[:, :cfg["top_groups"]], True, 1)
        if cfg["top_groups"] < cfg["n_groups"]:
            ranked = np.take_along_axis(best, order, 1)[:, cfg["top_groups"] - 1:cfg["top_groups"] + 1]
            gap = np.where(np.isneginf(ranked[:, 1]), np.inf, ranked[:, 0] - np.maximum(ranked[:, 1], -1e300))
        key = np.where(inside[:, :, None], by, -np.inf).reshape(n, X)
    at = np.argsort(-z, axis=1, kind="stable")
    at = np.take_along_axis(at, np.argsort(-np.take_along_axis(key, at, 1), axis=1, kind="stable"), 1)
    ranked = np.take_along_axis(key, at, 1)[:, :cfg["top_k"] + 1]
    apart = np.where(np.isneginf(ranked[:, 1:]), np.inf, ranked[:, :-1] - np.maximum(ranked[:, 1:], -1e300))
    gap = np.minimum(gap, apart.min(1, initial=np.inf))
    at = at[:, :cfg["top_k"]]
    has = ~np.isneginf(np.take_along_axis(key, at, 1))
    return np.where(has, at, -1).astype(np.int32), gates_many(z, at, has, s, cfg), gap


def gates_many(z, at, has, s, cfg):
    picked = np.take_along_axis(z, at, 1)
    if not cfg["renormalise"]:
        return cfg["scale"] * np.where(has, np.take_along_axis(s, at, 1), 0.0)
    with np.errstate(all="ignore"):
        l = np.where(has, log_scores(picked, cfg["score"]), -np.inf)
        w = np.where(has, np.exp(l - np.maximum(l.max(1, keepdims=True), -1e300)), 0.0)
    return cfg["scale"] * w / np.maximum(w.sum(1, keepdims=True), 1e-300)


def route_backward_many(logits, experts, gates, grad_gates, cfg):
    """route_backward for route_many's experts and gates."""
    z, g = np.asarray(logits, np.float64), np.where(experts < 0, 0.0, np.asarray(grad_gates, np.float64))
    at, c = np.maximum(experts, 0), cfg["scale"]
    with np.errstate(all="ignore"):
        rest = 1.0 / (1.0 + np.exp(np.take_along_axis(z, at, 1))) if cfg["score"] == "sigmoid" else 1.0   # 1 - s
        inner = (g * gates).sum(1, keepdims=True)
        d = np.where(experts < 0, 0.0, gates * (g - inner / c if cfg["renormalise"] else g) * rest)
    out = np.zeros_like(z)
    np.add.at(out, (np.arange(len(z))[:, None], at), d)
    if not cfg["renormalise"] and cfg["score"] == "softmax":
        e = np.where(np.isneginf(z), 0.0, np.exp(z - np.maximum(z.max(1, keepdims=True), -1e300)))
        out -= e / np.maximum(e.sum(1, keepdims=True), 1e-300) * inner
    return out


# -------------------------------------------------------------------- experts
def expert_maps(irreps_in, irreps_out):
    """[(mul_in, col_in, mul_out, col_out, 2l+1, weight offset)] and an expert's weights."""
    out, at = [], 0
    for mi, li, pi, ci in segments(irreps_in)[0]:
        for mo, lo, po, co in segments(irreps_out)[0]:
            if (li, pi) == (lo, po):
                out.append((mi, ci, mo, co, 2 * li + 1, at))
                at += mi * mo
    return out, at


def experts_forward(irreps_in, irreps_out, x, weights, experts, gates):
    x, weights, gates = (np.asarray(a, np.float64) for a in (x, weights, gates))
    out = np.zeros((len(x), segments(irreps_out)[1]))
    for i in range(len(x)):
        for a, e in enumerate(experts[i]):
            if not 0 <= e < len(weights):
                continue
            for mi, ci, mo, co, d, at in expert_maps(irreps_in, irreps_out)[0]:
                M = weights[e, at:at + mi * mo].reshape(mi, mo)
                out[i, co:co + mo * d] += gates[i, a] * (M.T @ x[i, ci:ci + mi * d].reshape(mi, d)).reshape(-1)
    return out


def experts_backward(irreps_in, irreps_out, x, weights, experts, gates, G):
    x, weights, gates, G = (np.asarray(a, np.float64) for a in (x, weights, gates, G))
    gx, gw, gg = np.zeros_like(x), np.zeros_like(weights), np.zeros_like(gates)
    for i in range(len(x)):
        for a, e in enumerate(experts[i]):
            if not 0 <= e < len(weights):
                continue
            for mi, ci, mo, co, d, at in expert_maps(irreps_in, irreps_out)[0]:
                M = weights[e, at:at + mi * mo].reshape(mi, mo)
                xs, Gs = x[i, ci:ci + mi * d].reshape(mi, d), G[i, co:co + mo * d].reshape(mo, d)
                gx[i, ci:ci + mi * d] += gates[i, a] * (M @ Gs).reshape(-1)
                gw[e, at:at + mi * mo] += gates[i, a] * (xs @ Gs.T).reshape(-1)
                gg[i, a] += np.sum(xs * (M @ Gs))
    return gx, gw, gg


def experts_many(irreps_in, irreps_out, x, weights, experts, gates, G):
    """experts_forward and experts_backward: (out, grad_x, grad_weights, grad_gates)."""
    x, weights, gates, G = (np.asarray(a, np.float64) for a in (x, weights, gates, G))
    out = np.zeros((len(x), segments(irreps_out)[1]))
    gx, gw, gg = np.zeros_like(x), np.zeros_like(weights), np.zeros_like(gates)
    for e in range(len(weights)):
        for a in range(experts.shape[1]):
            rows = np.nonzero(experts[:, a] == e)[0]          # each row once
            if not len(rows):
                continue
            w = gates[rows, a][:, None, None]
            for mi, ci, mo, co, d, at in expert_maps(irreps_in, irreps_out)[0]:
                M = weights[e, at:at + mi * mo].reshape(mi, mo)
                xs, Gs = x[rows, ci:ci + mi * d].reshape(-1, mi, d), G[rows, co:co + mo * d].reshape(-1, mo, d)
                out[rows, co:co + mo * d] += (w * (M.T @ xs)).reshape(len(rows), -1)
                back = M @ Gs
                gx[rows, ci:ci + mi * d] += (w * back).reshape(len(rows), -1)
                gw[e, at:at + mi * mo] += np.tensordot(w * xs, Gs, ((0, 2), (0, 2))).reshape(-1)
                gg[rows, a] += (xs * back).sum((1, 2))
    return out, gx, gw, gg


# -------------------------------------------------------------------- dropout
def philox4x32(counter, key, rounds=10):
    """Philox4x32 of four counter words and two key words (Python integers)."""
    c, k, low = list(counter), list(key), 0xFFFFFFFF
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def dropout_keep(irreps, n_rows, p, seed, offset):
    """Keep mask [n_rows, dim]: one draw for each channel of a row."""
    segs, dim = segments(irreps)
    channels = sum(s[0] for s in segs)
    low = 0xFFFFFFFF
    words = []
    for block in range((n_rows * channels + 3) // 4):
        words += philox4x32((block & low, block >> 32, offset & low, offset >> 32), (seed & low, seed >> 32))
    keep = np.array(words[:n_rows * channels], np.int64).reshape(n_rows, channels) >= int(np.floor(p * 2.0 ** 32))
    out = np.zeros((n_rows, dim), bool)
    c = 0
    for mul, l, _, at in segs:
        for u in range(mul):
            out[:, at + u * (2 * l + 1):at + (u + 1) * (2 * l + 1)] = keep[:, c:c + 1]
            c += 1
    return out


def dropout_keep_many(irreps, n_rows, p, seed, offset):
    """dropout_keep, all blocks of the generator at a time."""
    segs, dim = segments(irreps)
    channels = sum(m for m, _, _, _ in segs)
    low, half, block = np.uint64(0xFFFFFFFF), np.uint64(32), np.arange((n_rows * channels + 3) // 4, dtype=np.uint64)
    c = [block & low, block >> half, np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, 1).reshape(-1)[:n_rows * channels].reshape(n_rows, channels)
    of = np.concatenate([np.repeat(np.arange(m), 2 * l + 1) + sum(s[0] for s in segs[:i])
                         for i, (m, l, _, _) in enumerate(segs)])
    return (words >= np.uint64(int(np.floor(p * 2.0 ** 32))))[:, of]


def dropout_forward(irreps, p, seed, offset, x, residual=None):
    x = np.asarray(x, np.float64)
    out = np.where(dropout_keep(irreps, len(x), p, seed, offset), x / (1.0 - p), 0.0)
    return out if residual is None else out + np.asarray(residual, np.float64)

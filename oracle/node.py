"""Plain fp64 definitions of the node operators: species embedding, routing to
experts, the experts' equivariant maps, dropout on irreps rows.

numpy only, one row or one expert at a time, straight from the formulas;
shares no code with the GPU path.
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
    """grad_logits through the full Jacobian of the chosen scores."""
    z, g = np.asarray(logits, np.float64), np.asarray(grad_gates, np.float64)
    out = np.zeros_like(z)
    for i in range(len(z)):
        at = [a for a in range(cfg["top_k"]) if 0 <= experts[i, a] < z.shape[1]]
        e = [int(experts[i, a]) for a in at]
        if not e:
            continue
        w = gates_of(z[i], e, cfg)
        s = scores(z[i], cfg["score"])
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
            out[i] -= cfg["scale"] * s * np.dot(ga, s[e])
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


def dropout_forward(irreps, p, seed, offset, x, residual=None):
    x = np.asarray(x, np.float64)
    out = np.where(dropout_keep(irreps, len(x), p, seed, offset), x / (1.0 - p), 0.0)
    return out if residual is None else out + np.asarray(residual, np.float64)

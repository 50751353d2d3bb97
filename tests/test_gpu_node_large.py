"""GPU parity of the node operators at sizes where a block or a row of lanes
takes more than one turn: rows past one grid, groups past what LDS holds, rows
wider than a table in LDS.

Bounds are those of test_gpu_node.py, which derives them: at most
(n + c + 4) eps A for a sum of n terms with absolute values A and c factors,
and for gates (X + 2 |argument| + 32) eps.
"""

import sys

import numpy as np
import pytest

from oracle import node as on
from test_gpu_node import EPS, NP, config, dev, node, within  # noqa: F401  (node is a fixture)

pytestmark = pytest.mark.gpu


def log(msg):
    print(msg, file=sys.stderr, flush=True)


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("n,types,dim,stride", [(1200001, 119, 3, 3), (1100003, 5, 1, 2), (300001, 2000, 5, 7)])
def test_embedding(node, dt, n, types, dim, stride):  # noqa: F811
    """Rows past the forward's grid; more blocks of the gradient than one block of the join has threads."""
    log(f"[node] large embedding {dt} n={n} types={types} dim={dim}")
    rng = np.random.default_rng([n, types])
    t = rng.integers(-1, types + 1, n).astype(np.int32)
    table, wide = rng.standard_normal((types, dim)).astype(NP[dt]), rng.standard_normal((n, stride)).astype(NP[dt])
    out = dev(wide)
    node.tpconv_embedding_forward(dev(t), dev(table), 1.7, out=out[:, :dim])
    live = (t >= 0) & (t < types)
    want = wide.astype(np.float64)
    want[:, :dim] = np.where(live[:, None], 1.7 * table[np.where(live, t, 0)].astype(np.float64), 0.0)
    within(out, want, 3 * EPS[dt] * np.abs(want), "out")
    got = node.tpconv_embedding_backward(dev(t), dev(wide)[:, :dim], types, 1.7)
    count = np.bincount(t[live], minlength=types)[:, None]
    sums, sizes = ([np.bincount(t[live], weights=f(wide[live, c].astype(np.float64)), minlength=types)
                    for c in range(dim)] for f in (lambda v: v, np.abs))
    within(got, 1.7 * np.stack(sums, 1), (count + 6) * EPS[dt] * 1.7 * np.stack(sizes, 1), "grad_table")


def test_embedding_gradient_of_more_types_than_one_launch_has_blocks(node):  # noqa: F811
    """4.2 million types whose sums come from 293 blocks: a type for each block would pass 2^32 threads."""
    rng = np.random.default_rng(3)
    n, types = 300001, 4200000
    t = rng.integers(0, types, n).astype(np.int32)
    t[:3] = 0, types - 1, -1
    grad = rng.standard_normal((n, 2))
    got = node.tpconv_embedding_backward(dev(t), dev(grad), types).cpu().numpy()
    live = t >= 0
    count = np.bincount(t[live], minlength=types)
    for c in range(2):
        want, size = (np.bincount(t[live], weights=v[live, c], minlength=types) for v in (grad, np.abs(grad)))
        assert (np.abs(got[:, c] - want) <= (count + 6) * EPS["f64"] * size).all()


# -------------------------------------------------------------------- routing
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("score,renorm,n,X,G,T,k,biased", [
    ("softmax", False, 140001, 8, 1, 1, 2, False), ("sigmoid", True, 140001, 8, 4, 2, 3, True),
    ("softmax", True, 140001, 16, 1, 1, 3, False), ("sigmoid", True, 70007, 128, 8, 4, 6, True),
    ("softmax", False, 70007, 128, 1, 1, 8, False), ("sigmoid", False, 66001, 200, 1, 1, 5, True),
    ("softmax", True, 70007, 64, 8, 3, 4, False)])
def test_routing(node, dt, score, renorm, n, X, G, T, k, biased):  # noqa: F811
    """Each row of lanes takes a second row, its logits and experts on their way ahead."""
    log(f"[node] large routing {dt} {score} renorm={renorm} n={n} X={X} groups={G}/{T} k={k}")
    rng = np.random.default_rng([n, X, G, k])
    cfg, ocfg = config(node, n_experts=X, top_k=k, score=score, renormalise=renorm, n_groups=G, top_groups=T, scale=2.5)
    bias = (0.2 * rng.standard_normal(X)).astype(NP[dt]) if biased else None

    def draw(m):
        z = (1.5 * rng.standard_normal((m, X))).astype(NP[dt])
        z[rng.random((m, X)) < 0.05] = -np.inf
        z[rng.random(m) < 0.01] = -np.inf
        return z

    z = draw(n)
    want_e, want_g, gap = on.route_many(z, bias, ocfg)
    for _ in range(60):                                         # choices that hang on rounding are drawn again
        near = np.nonzero(gap < 1e-5)[0]
        if not len(near):
            break
        z[near] = draw(len(near))
        want_e[near], want_g[near], gap[near] = on.route_many(z[near], bias, ocfg)
    assert gap.min() >= 1e-5
    experts, gates = node.tpconv_route_forward(cfg, dev(z), None if bias is None else dev(bias))
    assert np.array_equal(experts.cpu().numpy(), want_e)
    tol = (X + 2 * 2 * np.abs(np.where(np.isneginf(z), 0.0, z)).max() + 32) * EPS[dt]
    within(gates, want_g, tol * np.abs(want_g), "gates")
    g = rng.standard_normal((n, k)).astype(NP[dt])
    got = node.tpconv_route_backward(cfg, dev(z), experts, dev(np.where(want_e < 0, np.nan, g).astype(NP[dt])))
    # each entry is a gate times (its gradient, less the gates' mean gradient)
    size = np.abs(want_g) * np.abs(g) * (want_e >= 0)
    total = size.sum(1, keepdims=True)
    mag = np.zeros((n, X))
    np.add.at(mag, (np.arange(n)[:, None], np.maximum(want_e, 0)), size + np.abs(want_g) * total / 2.5)
    if not renorm and score == "softmax":
        mag += np.where(np.isneginf(z), 0.0, np.exp(z - z.max(1, keepdims=True).clip(-1e30))) * total
    within(got, on.route_backward_many(z, want_e, want_g, g, ocfg), 3 * (tol + (k + 6) * EPS[dt]) * mag, "grad_logits")


# -------------------------------------------------------------------- experts
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("n,irr_in,irr_out,X,k", [
    (140001, "2x0e+1x1o", "1x1o+1x0e", 20, 8), (300001, "1x0e", "2x0e", 5, 1), (150001, "1x1o", "1x1o", 256, 2)])
def test_experts(node, dt, n, irr_in, irr_out, X, k):  # noqa: F811
    """The layout's groups have more entries than LDS holds and more rows than a thread keeps; all of its 64 groups."""
    import torch
    log(f"[node] large experts {dt} n={n} {irr_in} experts={X} k={k}")
    rng = np.random.default_rng([n, X])
    share = (np.arange(X + 1) + 1.0) ** -0.7
    experts = rng.choice(np.arange(-1, X), size=(n, k), p=share / share.sum()).astype(np.int32)   # doubles among them
    plan = node.tpconv_experts_plan(irr_in, irr_out, X, k, dt)
    x, G = (rng.standard_normal((n, d)).astype(NP[dt]) for d in (plan.dim_in, plan.dim_out))
    w, gates = rng.standard_normal((X, plan.weight_numel)).astype(NP[dt]), rng.random((n, k)).astype(NP[dt])
    args = [dev(a) for a in (x, w, experts, gates)]
    load = torch.zeros(X, dtype=torch.int32, device="cuda")
    layout = node.tpconv_experts_layout(plan, args[2], load=load)
    count = np.bincount(experts[experts >= 0], minlength=X)
    assert np.array_equal(load.cpu().numpy(), count)
    out = node.tpconv_experts_forward(plan, *args, layout)
    assert torch.equal(out, node.tpconv_experts_forward(plan, *args))
    got = (out, *node.tpconv_experts_backward(plan, *args, dev(G), layout))
    want = on.experts_many(irr_in, irr_out, x, w, experts, gates, G)
    size = on.experts_many(irr_in, irr_out, np.abs(x), np.abs(w), experts, gates, np.abs(G))
    maps, _ = on.expert_maps(irr_in, irr_out)
    mul_in, mul_out, d = (max(m[i] for m in maps) for i in (0, 2, 4))
    terms = (mul_in + k + 6, mul_out + k + 6, count.max() * d + 8, mul_in * d + mul_out + len(maps) + 8)
    for a, b, s, c, what in zip(got, want, size, terms, ("out", "grad_x", "grad_weights", "grad_gates")):
        within(a, b, c * EPS[dt] * s, what)
    again = node.tpconv_experts_backward(plan, *args, dev(G), node.tpconv_experts_layout(plan, args[2]))
    assert all(torch.equal(a, b) for a, b in zip(got[1:], again))


def test_experts_of_more_rows_than_one_launch_has_tiles(node):  # noqa: F811
    """2^30 rows of two channels: a block for each tile and map would pass 2^32 threads, for the rows and for the
    weights' gradient.  All values are small whole numbers and every sum stays below 2^24, so results are exact."""
    import torch
    n, irr = (1 << 30) + 48, "1x0e+1x0o"
    plan = node.tpconv_experts_plan(irr, irr, 2, 1)
    w = torch.tensor([[3.0, -2.0], [5.0, 7.0]], device="cuda")
    x, G = torch.empty((n, 2), device="cuda"), torch.empty((n, 2), device="cuda")
    e, gates = torch.empty((n, 1), dtype=torch.int32, device="cuda"), torch.empty((n, 1), device="cuda")
    step = 48 << 20

    def part(i0):
        """Rows i0.. of x, G, experts and gates, and what comes of them."""
        i = torch.arange(i0, min(n, i0 + step), device="cuda", dtype=torch.int32)
        a = torch.stack([1 + i % 3, 2 - i % 2], 1).float()
        b = torch.stack([1 - i % 4 // 2 * 2 + (i % 65536 == 5), i % 3 - 1], 1).float()   # a few above a sum of 0
        ex = ((i // 12) % 3 - 1).int()[:, None]                 # none, 0, 1
        gate = (1 + (i // 36) % 2).float()[:, None]
        we = torch.where(ex >= 0, w[ex[:, 0].clamp(min=0).long()], 0.0)
        live = torch.where(ex >= 0, gate, 0.0)
        return (a, b, ex, gate), (live * we * a, live * we * b, (we * a * b).sum(1, keepdim=True)), live * a * b

    sums = torch.zeros((2, 2), dtype=torch.float64, device="cuda")
    for i0 in range(0, n, step):
        (a, b, ex, gate), _, terms = part(i0)
        for to, value in ((x, a), (G, b), (e, ex), (gates, gate)):
            to[i0:i0 + step] = value
        for q in range(2):
            sums[q] += (terms * (ex == q)).double().sum(0)
    layout = node.tpconv_experts_layout(plan, e)
    out = node.tpconv_experts_forward(plan, x, w, e, gates, layout)
    gx, gw, gg = node.tpconv_experts_backward(plan, x, w, e, gates, G, layout)
    for i0 in range(0, n, step):
        want = part(i0)[1]
        for got, value, what in zip((out, gx, gg), want, ("out", "grad_x", "grad_gates")):
            assert torch.equal(got[i0:i0 + step], value), (what, i0)
    assert torch.equal(gw, sums.float()) and float(sums.abs().max()) < 2 ** 24
    del x, G, e, gates, layout, out, gx, gw, gg
    torch.cuda.empty_cache()


# -------------------------------------------------------------------- dropout
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("n,irreps,p", [
    (3001, "5x0e+5x1o", 0.3), (30011, "5x0e+5x1o", 0.3),          # tiles of several rows, 10 channels in a row
    (30011, "13x0e+1x1o", 0.5), (9001, "3x0e+1x2e", 0.25),        # 16 columns; 8 columns, 4 channels
    (30001, "32x0e+32x1o+31x2e", 0.1),                            # odd width: single elements, blocks of several tiles
    (3001, "1500x0e+900x1o", 0.4),                                # more pieces than are loaded ahead
    (101, "5461x1o+1x0e", 0.4), (41, "5461x1o+2x0e", 0.4),        # the widest row of the table, and one column more
    (37, "3001x0e+4500x1o+1x2e", 0.5)])
def test_dropout(node, dt, n, irreps, p):  # noqa: F811
    import torch
    log(f"[node] large dropout {dt} n={n} {irreps} p={p}")
    rng = np.random.default_rng([n, int(1000 * p)])
    dim = on.segments(irreps)[1]
    x, res = (rng.standard_normal((n, dim)).astype(NP[dt]) for _ in range(2))
    seed, offset = 0xFEDCBA9876543210, (1 << 40) + 7
    keep = on.dropout_keep_many(irreps, n, p, seed, offset)
    scaled = np.where(keep, x.astype(np.float64) / (1 - p), 0.0)
    holes = np.where(keep, x, np.nan).astype(NP[dt])
    for r in (None, res):
        base = 0.0 if r is None else r.astype(np.float64)
        rd = None if r is None else dev(r)
        got = node.tpconv_dropout_forward(irreps, p, seed, offset, dev(holes), rd)
        within(got, scaled + base, 4 * EPS[dt] * (np.abs(scaled) + np.abs(base)), "out")
        a = dev(holes)
        assert torch.equal(got, node.tpconv_dropout_forward(irreps, p, seed, offset, a, rd, out=a))
        # rows that no 16-byte piece starts at: the same, element by element
        odd = torch.empty(n * dim + 1, dtype=a.dtype, device="cuda")[1:].view(n, dim)
        odd.copy_(dev(holes))
        assert torch.equal(got, node.tpconv_dropout_forward(irreps, p, seed, offset, odd, rd))
    back = node.tpconv_dropout_backward(irreps, p, seed, offset, dev(holes))
    within(back, scaled, 4 * EPS[dt] * np.abs(scaled), "grad_x")

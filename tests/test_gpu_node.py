"""GPU parity of the node operators against the fp64 oracle (oracle/node.py),
through the Python binding.

Bounds.  Every output is a sum of products, so its error is bounded entry by
entry: with eps the unit roundoff of the data type (2^-24, 2^-53) and A the
same sum over absolute values, n terms and c factors give at most
(n + c + 4) eps A (each product and each addition rounds once; the order of
the sum does not matter).  A comes from the oracle on absolute values.  Gates
pass through exp and log1p (a few units in the last place) of an argument
that was itself rounded: relative error (X + 2 |argument| + 32) eps for X
experts.  The chosen experts are compared exactly, on logits whose keys are
further apart than that or tie exactly.
"""

import itertools
import sys

import numpy as np
import pytest

import workloads
from oracle import node as on

pytestmark = pytest.mark.gpu
NP = {"f32": np.float32, "f64": np.float64}
EPS = {"f32": 2.0 ** -24, "f64": 2.0 ** -53}


def log(msg):
    print(msg, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def node():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    from equivariant_mlip_tensor_amd import node
    return node


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def within(got, want, bound, what):
    got, want = np.asarray(got.cpu() if hasattr(got, "cpu") else got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - want))), np.argwhere(bad)[:3].tolist())


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("n,types,dim,stride,shift", [
    (0, 3, 4, 4, 0), (1, 1, 1, 1, 0), (16, 5, 4, 16, 0), (63, 2, 3, 7, 1), (64, 9, 64, 64, 0), (65, 97, 20, 33, 3),
    (1023, 1, 8, 8, 0), (1025, 4, 64, 256, 64), (3000, 119, 130, 131, 1), (5000, 7000, 12, 12, 0),
    (20011, 3, 64, 64, 0), (4096, 1100, 5, 9, 4)])
def test_embedding(node, dt, n, types, dim, stride, shift):
    import torch
    log(f"[node] embedding {dt} n={n} types={types} dim={dim} stride={stride} shift={shift}")
    rng = np.random.default_rng([n, types, dim])
    share = (np.arange(types) + 1.0) ** -1.2
    t = rng.choice(types, size=n, p=share / share.sum()).astype(np.int32)
    t[rng.random(n) < 0.05] = -1
    if n > 40:
        t[7], t[31] = types, 2 ** 31 - 1                      # outside the table
    table, wide = rng.standard_normal((types, dim)).astype(NP[dt]), rng.standard_normal((n, stride + shift)).astype(NP[dt])
    scale = 1.7
    out = dev(wide.copy())
    node.tpconv_embedding_forward(dev(t), dev(table), scale, out=out[:, shift:shift + dim])
    want = wide.astype(np.float64)                            # the other columns stay
    want[:, shift:shift + dim] = on.embedding_forward(t, table, scale)
    within(out, want, 3 * EPS[dt] * np.abs(want), "out")
    grad = dev(wide)[:, shift:shift + dim]
    nan = torch.full((types, dim), float("nan"), dtype=grad.dtype, device="cuda")
    got = node.tpconv_embedding_backward(dev(t), grad, types, scale, grad_table=nan)
    g = wide[:, shift:shift + dim]
    count = np.bincount(t[(t >= 0) & (t < types)], minlength=types)[:, None]
    within(got, on.embedding_backward(t, g, types, scale),
           (count + 6) * EPS[dt] * on.embedding_backward(t, np.abs(g), types, scale), "grad_table")
    again = node.tpconv_embedding_backward(dev(t), grad, types, scale)
    assert torch.equal(got, again)


def test_embedding_sorted_reversed_and_uniform_types(node):
    """Orders that put every run at a block's edge or none."""
    rng = np.random.default_rng(1)
    n, types, dim = 6000, 37, 32
    grad = rng.standard_normal((n, dim))
    for t in (np.arange(n) * types // n, (np.arange(n) * types // n)[::-1], np.arange(n) % types, np.full(n, 36)):
        t = t.astype(np.int32)
        got = node.tpconv_embedding_backward(dev(t), dev(grad), types)
        bound = (n + 6) * EPS["f64"] * on.embedding_backward(t, np.abs(grad), types)
        within(got, on.embedding_backward(t, grad, types), bound, "grad_table")


@pytest.mark.parametrize("types", [1, 40, 511, 512, 700])
def test_embedding_gradient_of_many_rows(node, types):
    """The longest blocks, with as many types as are sorted by counting and more."""
    rng = np.random.default_rng(types)
    n, dim = 140001, 3
    t = rng.integers(-1, types + 1, n).astype(np.int32)
    grad = rng.standard_normal((n, dim)).astype(np.float32)
    got = node.tpconv_embedding_backward(dev(t), dev(grad), types)
    count = np.bincount(t[(t >= 0) & (t < types)], minlength=types)[:, None]
    bound = (count + 6) * EPS["f32"] * on.embedding_backward(t, np.abs(grad), types)
    within(got, on.embedding_backward(t, grad, types), bound, "grad_table")


# -------------------------------------------------------------------- routing
def config(node, **kw):
    return node.RouteConfig(**kw), dict(score=kw.get("score", "softmax"), renormalise=kw.get("renormalise", True),
                                        n_groups=kw.get("n_groups", 1), top_groups=kw.get("top_groups", 1),
                                        top_k=kw["top_k"], scale=kw.get("scale", 1.0))


def separated(rng, n, X, bias, cfg, dt, masked):
    """Logits whose choices do not hang on rounding: rows with a gap below 1e-4 among the candidates are redrawn."""
    z = np.zeros((n, X), NP[dt])
    for i in range(n):
        while True:
            row = (1.5 * rng.standard_normal(X)).astype(NP[dt])
            row[rng.random(X) < masked] = -np.inf
            key = on.keys(row.astype(np.float64), bias, cfg["score"])
            gaps = [1.0]
            if cfg["n_groups"] > 1:
                gk = np.sort(on.group_keys(key, cfg["n_groups"]))[::-1]
                gk = gk[~np.isneginf(gk)]
                if cfg["top_groups"] < len(gk):
                    gaps.append(gk[cfg["top_groups"] - 1] - gk[cfg["top_groups"]])
                order = np.argsort(-on.group_keys(key, cfg["n_groups"]), kind="stable")[:cfg["top_groups"]]
                key = np.where(np.repeat(np.isin(np.arange(cfg["n_groups"]), order), X // cfg["n_groups"]), key, -np.inf)
            k = np.sort(key[~np.isneginf(key)])[::-1][:cfg["top_k"] + 1]
            gaps += list(k[:-1] - k[1:])
            if min(gaps) > (1e-5 if X > 100 else 1e-4):
                z[i] = row
                break
    return z


def gate_bound(z, cfg, dt):
    live = np.where(np.isneginf(z), 0.0, np.abs(z.astype(np.float64)))
    return (z.shape[1] + 2 * 2 * live.max(initial=0.0) + 32) * EPS[dt]


ROUTES = [(1, 1, 1, 1, 1), (5, 2, 1, 1, 2), (64, 8, 1, 1, 2), (33, 16, 4, 2, 3), (130, 7, 1, 1, 4), (40, 64, 8, 3, 6),
          (65, 96, 6, 6, 8), (30, 256, 8, 4, 8), (21, 100, 50, 9, 8), (257, 33, 1, 1, 8), (9, 64, 64, 5, 5)]


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("score,renorm", list(itertools.product(("softmax", "sigmoid"), (True, False))))
@pytest.mark.parametrize("n,X,G,T,k", ROUTES)
def test_routing(node, dt, score, renorm, n, X, G, T, k):
    import torch
    log(f"[node] routing {dt} {score} renorm={renorm} n={n} X={X} groups={G}/{T} k={k}")
    rng = np.random.default_rng([n, X, G, k])
    cfg, ocfg = config(node, n_experts=X, top_k=k, score=score, renormalise=renorm, n_groups=G, top_groups=T, scale=2.5)
    bias = (0.2 * rng.standard_normal(X)).astype(NP[dt]) if (X + k) % 2 else None
    z = separated(rng, n, X, bias, ocfg, dt, 0.05)
    if n > 4:
        z[3] = -np.inf                                         # a padding row
        z[4, 1:] = -np.inf                                     # one expert left
    experts, gates = node.tpconv_route_forward(cfg, dev(z), None if bias is None else dev(bias))
    want_e, want_g = on.route_forward(z, bias, ocfg)
    assert np.array_equal(experts.cpu().numpy(), want_e)
    tol = gate_bound(z, ocfg, dt)
    within(gates, want_g, tol * np.abs(want_g), "gates")
    g = rng.standard_normal((n, k)).astype(NP[dt])
    g_nan = np.where(want_e < 0, np.nan, g).astype(NP[dt])     # nothing may be read where no expert was chosen
    got = node.tpconv_route_backward(cfg, dev(z), experts, dev(g_nan))
    ref = on.route_backward(z, want_e, g, ocfg)
    # each entry is a gate times (its gradient, less the gates' mean gradient)
    size = np.abs(want_g) * np.abs(g)
    total = size.sum(1, keepdims=True)
    mag = np.zeros((n, X))
    for i in range(n):
        for a, e in enumerate(want_e[i]):
            if e >= 0:
                mag[i, e] += size[i, a] + abs(want_g[i, a]) * total[i, 0] / 2.5
        if not renorm and score == "softmax":
            mag[i] += on.scores(z[i].astype(np.float64), score) * total[i, 0]
    within(got, ref, 3 * (tol + (k + 6) * EPS[dt]) * mag, "grad_logits")
    assert torch.equal(got, node.tpconv_route_backward(cfg, dev(z), experts, dev(g_nan)))


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_routing_ties_go_to_the_lowest_index(node, dt, score):
    rng = np.random.default_rng(8)
    for X, G, T, k in ((8, 1, 1, 3), (64, 1, 1, 8), (200, 1, 1, 8), (24, 6, 3, 5), (128, 8, 4, 8)):
        cfg, ocfg = config(node, n_experts=X, top_k=k, score=score, n_groups=G, top_groups=T)
        z = rng.integers(-2, 3, (70, X)).astype(NP[dt])
        z[rng.random(z.shape) < 0.3] = -np.inf
        z[0] = 0
        if score == "softmax":
            z[1] = np.finfo(NP[dt]).min                        # the type's lowest value is a number, not a mask
        experts, gates = node.tpconv_route_forward(cfg, dev(z))
        want_e, want_g = on.route_forward(z, None, ocfg)
        assert np.array_equal(experts.cpu().numpy(), want_e), (X, G)
        within(gates, want_g, 400 * EPS[dt] * np.abs(want_g), "gates")


@pytest.mark.parametrize("dt", ["f32", "f64"])
def test_routing_extremes(node, dt):
    """Scores that all underflow still give gates that sum to scale; the lowest value and the mask side by side; NaN."""
    import torch
    big = 5000.0
    z = np.full((4, 6), -big, NP[dt])
    z[0, 4] = -big + 1
    z[1] = [big, -big, 0, big, -np.inf, 1]
    z[2] = [np.finfo(NP[dt]).min, -np.inf, -np.inf, -np.inf, -np.inf, -np.inf]
    z[3] = [0, np.nan, 1, 2, -np.inf, 3]
    for score in ("softmax", "sigmoid"):
        cfg, ocfg = config(node, n_experts=6, top_k=2, score=score, scale=3.0)
        experts, gates = node.tpconv_route_forward(cfg, dev(z))
        want_e, want_g = on.route_forward(z[:3], None, ocfg)
        if score == "softmax":
            assert np.array_equal(experts.cpu().numpy()[:3], want_e)
        assert abs(float(gates[0].sum()) - 3.0) < 1e-5 and abs(float(gates[1].sum()) - 3.0) < 1e-5
        # log of a score of exp(-5000) is known to 5000 eps
        within(gates[2], want_g[2], 32 * EPS[dt] * 3.0, "one expert left")
        if score == "softmax":
            within(gates[:2], want_g[:2], 4 * big * EPS[dt] * 3.0, "gates")
            assert torch.isnan(gates[3]).all()                  # a NaN makes its row's softmax NaN
        else:
            assert experts[3].tolist() == [5, 3] and torch.isfinite(gates[3]).all()
    # backward of an index outside the experts, and of one that stands twice
    cfg, ocfg = config(node, n_experts=6, top_k=3)
    zz = np.random.default_rng(0).standard_normal((2, 6)).astype(NP[dt])
    e = np.array([[2, 9, -5], [4, 4, 1]], np.int32)
    g = np.array([[1.0, np.nan, np.nan], [0.5, -1.5, 2.0]], NP[dt])
    got = node.tpconv_route_backward(cfg, dev(zz), dev(e), dev(g))
    within(got, on.route_backward(zz, np.where(e > 5, -1, e), np.nan_to_num(g), ocfg), 400 * EPS[dt], "grad_logits")


def test_routing_gradient_against_differences(node):
    rng = np.random.default_rng(11)
    for score, renorm in itertools.product(("softmax", "sigmoid"), (True, False)):
        cfg, ocfg = config(node, n_experts=12, top_k=3, score=score, renormalise=renorm, scale=1.5)
        z = separated(rng, 8, 12, None, ocfg, "f64", 0.0)
        g, step = rng.standard_normal((8, 3)), 1e-5
        experts, _ = node.tpconv_route_forward(cfg, dev(z))
        grad = node.tpconv_route_backward(cfg, dev(z), experts, dev(g)).cpu().numpy()
        d = rng.standard_normal(z.shape)
        lo, hi = (node.tpconv_route_forward(cfg, dev(z + s * step * d)) for s in (-1, 1))
        assert (lo[0] == experts).all() and (hi[0] == experts).all()     # gaps of 1e-4 outlast the step
        num = float(((hi[1] - lo[1]) * dev(g)).sum()) / (2 * step)
        # third derivatives are O(1), 24 terms: h^2 * 24 / 6 plus eps / h
        assert abs(num - float((grad * d).sum())) < 1e-7


# -------------------------------------------------------------------- experts
SAME = "8x0e+8x1o"
EXPERTS = [
    # n, irreps_in, irreps_out, experts, top_k
    (0, SAME, SAME, 4, 2), (1, "1x0e", "1x0e", 1, 1), (1, "32x0e+32x1o+32x2e+32x3o", "32x0e+32x1o+32x2e+32x3o", 8, 2),
    (3, "4x0e+4x1o", "4x0e+4x1o", 4, 2), (17, "5x0e+3x1o+7x2e", "6x2e+2x0e+9x1o", 3, 3),
    (64, "16x0e+16x1o+16x2e", "16x0e+16x1o+16x2e", 16, 2), (65, "17x1o+33x0e", "31x0e+15x1o", 5, 1),
    (129, "64x0e+64x1o+64x2e+64x3o", "64x0e+64x1o+64x2e+64x3o", 6, 2), (200, "3x4e+2x3o+1x0e", "5x4e+4x0e+2x1e", 64, 4),
    (300, "8x0e+8x1o+4x1e", "8x1e+8x0e+2x0o+4x1o", 256, 8), (70, "200x0e+65x1o", "130x0e+256x1o", 4, 2),
    (40, "256x4e", "256x4e", 3, 2), (2500, "8x0e+4x2e", "12x0e+8x2e", 7, 2), (37, "65x3o", "1x3o", 2, 2),
    (33, "1x3o", "100x3o", 9, 2)]


def routing_of(rng, n, X, k, nowhere=0.1):
    experts = np.stack([rng.permutation(X)[:k] if k <= X else rng.integers(0, X, k) for _ in range(n)]) \
        if n else np.zeros((0, k))
    experts = experts.astype(np.int32)
    experts[rng.random((n, k)) < nowhere] = -1
    return experts, rng.random((n, k))


def check_experts(node, dt, irr_in, irr_out, X, experts, gates, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    n, k = experts.shape
    plan = node.tpconv_experts_plan(irr_in, irr_out, X, k, dt)
    x, G = (rng.standard_normal((n, d)).astype(NP[dt]) for d in (plan.dim_in, plan.dim_out))
    w, gates = rng.standard_normal((X, plan.weight_numel)).astype(NP[dt]), gates.astype(NP[dt])
    gates_in = np.where((experts < 0) | (experts >= X), np.nan, gates).astype(NP[dt])   # may not be read
    args = [dev(a) for a in (x, w, experts, gates_in)]
    load = torch.full((X,), -7, dtype=torch.int32, device="cuda")
    layout = node.tpconv_experts_layout(plan, args[2], load=load)
    valid = experts[(experts >= 0) & (experts < X)]
    assert np.array_equal(load.cpu().numpy(), np.bincount(valid, minlength=X))
    out = node.tpconv_experts_forward(plan, *args, layout, out=torch.full((n, plan.dim_out), float("nan"),
                                                                          dtype=args[0].dtype, device="cuda"))
    maps, _ = on.expert_maps(irr_in, irr_out)
    mul_in, mul_out, d = (max(m[i] for m in maps) for i in (0, 2, 4))
    e, aw, ag, ax, aG = EPS[dt], np.abs(w), np.abs(gates), np.abs(x), np.abs(G)
    ref = on.experts_forward(irr_in, irr_out, x, w, experts, gates)
    within(out, ref, (mul_in + k + 6) * e * on.experts_forward(irr_in, irr_out, ax, aw, experts, ag), "out")
    assert torch.equal(out, node.tpconv_experts_forward(plan, *args))          # without the layout: bit by bit
    gx, gw, gg = node.tpconv_experts_backward(plan, *args, dev(G), layout)
    rx, rw, rg = on.experts_backward(irr_in, irr_out, x, w, experts, gates, G)
    bx, bw, bg = on.experts_backward(irr_in, irr_out, ax, aw, experts, ag, aG)
    count = np.bincount(valid, minlength=X).max(initial=0)
    within(gx, rx, (mul_out + k + 6) * e * bx, "grad_x")
    within(gw, rw, (count * d + 8) * e * bw, "grad_weights")
    within(gg, rg, (mul_in * d + mul_out + len(maps) + 8) * e * bg, "grad_gates")
    # each output alone, and again: the same bits
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        one = node.tpconv_experts_backward(plan, *args, dev(G), layout if need[1] else None, need=need)
        for a, b, on_ in zip(one, (gx, gw, gg), need):
            assert torch.equal(a, b) if on_ else a is None
    return out, gx, gw, gg


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: f"{c[0]}-{c[3]}-{c[4]}")
def test_experts(node, dt, case):
    log(f"[node] experts {dt} {case}")
    n, irr_in, irr_out, X, k = case
    experts, gates = routing_of(np.random.default_rng([n, X]), n, X, k)
    check_experts(node, dt, irr_in, irr_out, X, experts, gates)


@pytest.mark.parametrize("dt", ["f32", "f64"])
def test_experts_uneven_duplicate_and_invalid_entries(node, dt):
    rng = np.random.default_rng(9)
    n, X, irr = 150, 5, "6x0e+5x1o"
    one = np.full((n, 2), 3, np.int32)                     # one expert, twice in every row
    none = np.full((n, 2), -1, np.int32)
    mixed, _ = routing_of(rng, n, X, 2)
    mixed[::7, 0], mixed[::5, 1], mixed[10:20] = X, 2 ** 31 - 1, -2 ** 31
    mixed[40:60, 1] = mixed[40:60, 0]
    hot = np.where(rng.random((n, 2)) < 0.05, 1, 4).astype(np.int32)
    for experts in (one, none, mixed, hot):
        outs = check_experts(node, dt, irr, irr, X, experts, rng.random((n, 2)))
        if experts is none:
            assert all(float(o.abs().max()) == 0.0 for o in outs)


def test_experts_nan_stays_in_its_row(node):
    """A NaN row reaches its own outputs and the weights of its own experts, and nothing else."""
    import torch
    rng = np.random.default_rng(10)
    n, X, k, irr = 100, 6, 2, "9x0e+8x1o"
    experts, gates = routing_of(rng, n, X, k, 0.0)
    plan = node.tpconv_experts_plan(irr, irr, X, k, "f32")
    x, G = (rng.standard_normal((n, plan.dim_in)).astype(np.float32) for _ in range(2))
    w = rng.standard_normal((X, plan.weight_numel)).astype(np.float32)
    x[37] = np.nan
    x[60, 3] = np.inf
    a = [dev(v) for v in (x, w, experts, gates.astype(np.float32))]
    layout = node.tpconv_experts_layout(plan, a[2])
    out = node.tpconv_experts_forward(plan, *a, layout)
    gx, gw, gg = node.tpconv_experts_backward(plan, *a, dev(G), layout)
    rows = torch.isfinite(out).all(1).cpu().numpy()
    assert not rows[37] and not rows[60] and rows.sum() == n - 2
    assert torch.isfinite(gx).all()
    hit = sorted(set(experts[37]) | set(experts[60]))
    fine = torch.isfinite(gw).all(1).cpu().numpy()
    assert [e for e in range(X) if not fine[e]] == hit
    assert torch.isfinite(gg).all(1).cpu().numpy().sum() == n - 2


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("irr", ["9x0e+8x1o", "32x0e+20x2e", "64x3o+40x4e"])
def test_experts_infinities_of_other_experts_stay_out(node, dt, irr):
    """Weights that are infinite, NaN or overflow reach the rows of their expert alone."""
    import torch
    rng = np.random.default_rng(11)
    n, X, k = 100, 6, 2
    experts, gates = routing_of(rng, n, X, k, 0.1)
    gates[5] = 0.0
    experts[5] = [2, 3]                                    # gates of 0: nothing of them either
    plan = node.tpconv_experts_plan(irr, irr, X, k, dt)
    x, G = (rng.standard_normal((n, plan.dim_in)).astype(NP[dt]) for _ in range(2))
    w = rng.standard_normal((X, plan.weight_numel)).astype(NP[dt])
    big = np.sqrt(np.finfo(NP[dt]).max)
    x *= big / 64                                          # products with the third's weights overflow, others do not
    G *= big / 64
    bad = w.copy()
    bad[2, ::3], bad[2, 1::3], bad[3] = np.nan, np.inf, bad[3] * big * 64
    others = ~np.isin(experts, [2, 3]).any(1) | (gates == 0).all(1)
    assert 20 < others.sum() < 80
    x, e, g, G = dev(x), dev(experts), dev(gates.astype(NP[dt])), dev(G)
    layout = node.tpconv_experts_layout(plan, e)
    for lay in (layout, None):
        for need in ((True, False, True), (True, False, False)):
            clean, dirty = ((node.tpconv_experts_forward(plan, x, dev(v), e, g, lay),
                             *node.tpconv_experts_backward(plan, x, dev(v), e, g, G, lay, need=need))
                            for v in (w, bad))
            assert torch.equal(clean[0][others], dirty[0][others]) and torch.equal(clean[1][others], dirty[1][others])
            assert not torch.isfinite(dirty[0][~others]).any(1).all()
            if need[2]:
                rows = torch.from_numpy(~np.isin(experts, [2, 3])).cuda()
                assert torch.equal(clean[3][rows], dirty[3][rows])


def test_experts_gradient_against_differences(node):
    rng = np.random.default_rng(12)
    irr_in, irr_out, X, k, n = "5x0e+4x1o+2x2e", "3x0e+6x1o+2x2e", 4, 2, 50
    experts, gates = routing_of(rng, n, X, k)
    plan = node.tpconv_experts_plan(irr_in, irr_out, X, k, "f64")
    x, G = rng.standard_normal((n, plan.dim_in)), rng.standard_normal((n, plan.dim_out))
    w = rng.standard_normal((X, plan.weight_numel))
    e = dev(experts)
    layout = node.tpconv_experts_layout(plan, e)
    grads = node.tpconv_experts_backward(plan, dev(x), dev(w), e, dev(gates), dev(G), layout)
    base = dict(x=x, w=w, g=gates)
    for name, grad in zip("xwg", grads):
        d = rng.standard_normal(base[name].shape)

        def f(s):
            v = dict(base, **{name: base[name] + s * d})
            return float((node.tpconv_experts_forward(plan, dev(v["x"]), dev(v["w"]), e, dev(v["g"]), layout)
                          * dev(G)).sum())
        # linear in each argument: only the difference's own rounding is left (about 1e4 terms, step 1/2)
        assert abs(f(0.5) - f(-0.5) - float((grad.cpu().numpy() * d).sum())) < 1e-9


# -------------------------------------------------------------------- dropout
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("n,irreps,p", [
    (0, "4x0e", 0.5), (1, "1x0e", 0.5), (1, "3x1o", 0.3), (7, "3x0e+5x1o+2x2e", 0.5), (16, "4x0e+4x1o", 0.1),
    (33, "32x0e+32x1o+32x2e", 0.25), (50, "5x4e+1x0o+1x0o", 0.9), (129, "13x0e", 0.0), (64, "8x3o+8x0e", 0.999),
    (300, "1x1o", 0.5)])
def test_dropout(node, dt, n, irreps, p):
    import torch
    log(f"[node] dropout {dt} n={n} {irreps} p={p}")
    rng = np.random.default_rng([n, int(1000 * p)])
    dim = on.segments(irreps)[1]
    x, res = (rng.standard_normal((n, dim)).astype(NP[dt]) for _ in range(2))
    seed, offset = 0xFEDCBA9876543210, (1 << 40) + 7
    keep = on.dropout_keep(irreps, n, p, seed, offset)
    want = on.dropout_forward(irreps, p, seed, offset, x, res)
    scaled = np.where(keep, np.abs(x.astype(np.float64)) / (1 - p), 0.0)
    for r, ref in ((res, want), (None, want - res)):
        got = node.tpconv_dropout_forward(irreps, p, seed, offset, dev(x), None if r is None else dev(r))
        base = 0.0 if r is None else r.astype(np.float64)
        ref = np.where(keep, x.astype(np.float64) / (1 - p), 0.0) + base
        within(got, ref, 4 * EPS[dt] * (scaled + np.abs(base)), "out")
    back = node.tpconv_dropout_backward(irreps, p, seed, offset, dev(x))
    assert torch.equal(back, got)                              # the same operation
    assert np.array_equal(back.cpu().numpy() != 0, keep & (x != 0))
    # what is dropped is not read into the result; in place on x and on the residual
    holes = np.where(keep, x, np.nan).astype(NP[dt])
    first = node.tpconv_dropout_forward(irreps, p, seed, offset, dev(x), dev(res))
    a, b = dev(holes), dev(res)
    assert torch.equal(first, node.tpconv_dropout_forward(irreps, p, seed, offset, a, b, out=a))
    a = dev(holes)
    assert torch.equal(first, node.tpconv_dropout_forward(irreps, p, seed, offset, a, b, out=b))


def test_dropout_rate_and_independent_draws(node):
    import torch
    n, irreps = 4096, "64x0e"
    one = torch.ones((n, 64), device="cuda")
    for p in (0.1, 0.5):
        masks = [node.tpconv_dropout_forward(irreps, p, 7, step, one) != 0 for step in range(3)]
        total = n * 64
        for m in masks:      # within 5 standard deviations
            assert abs(float(m.float().mean()) - (1 - p)) < 5 * np.sqrt(p * (1 - p) / total)
        same = float((masks[0] == masks[1]).float().mean())
        chance = p * p + (1 - p) * (1 - p)
        assert abs(same - chance) < 5 * np.sqrt(chance * (1 - chance) / total)


# -------------------------------------------------------- streams and capture
def test_refused_tensors(node):
    import torch
    x = torch.zeros((4, 8), device="cuda")
    types = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        node.tpconv_embedding_forward(types.long(), x)
    with pytest.raises(ValueError):
        node.tpconv_embedding_forward(types, x.half())
    with pytest.raises(ValueError):
        node.tpconv_embedding_forward(types, x, out=torch.zeros((8, 4), device="cuda").t())
    with pytest.raises(ValueError):
        node.tpconv_embedding_forward(types, x, out=x[:1].expand(4, 8))
    cfg = node.RouteConfig(8, 2)
    with pytest.raises(ValueError):
        node.tpconv_route_forward(cfg, x[:, :7])
    with pytest.raises(ValueError):
        node.tpconv_route_forward(cfg, x.cpu())
    with pytest.raises(ValueError):
        node.tpconv_route_forward(cfg, x, bias=torch.zeros(8, dtype=torch.float64, device="cuda"))
    with pytest.raises(RuntimeError, match="TPCONV_E_INVALID_ARG"):
        node.tpconv_route_forward(node.RouteConfig(8, 2, n_groups=3), x)
    plan = node.tpconv_experts_plan("8x0e", "8x0e", 3, 2)
    e, g, w = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda"), \
        torch.zeros((3, 64), device="cuda")
    layout = node.tpconv_experts_layout(plan, e[:3].contiguous())
    with pytest.raises(ValueError):
        node.tpconv_experts_forward(plan, x, w, e, g, layout)              # of another number of rows
    with pytest.raises(ValueError):
        node.tpconv_experts_forward(plan, x, w[:2], e, g)
    with pytest.raises(RuntimeError):
        node.tpconv_experts_backward(plan, x, w, e, g, x)                  # grad_weights without a layout
    with pytest.raises(RuntimeError):
        node.tpconv_dropout_forward("7x0e", 0.5, 1, 1, x)
    with pytest.raises(ValueError):
        node.tpconv_dropout_forward("8x0e", 0.5, 1, 1, x.t())


def layer(node, t, stream=None):
    """Every operator once, forward and backward, on one small layer."""
    kw = {} if stream is None else dict(stream=stream)
    x = node.tpconv_embedding_forward(t["types"], t["table"], 0.5, out=t["x"][:, :16], **kw)
    experts, gates = node.tpconv_route_forward(t["cfg"], t["logits"], **kw)
    layout = node.tpconv_experts_layout(t["plan"], experts, **kw)
    y = node.tpconv_experts_forward(t["plan"], t["x"], t["w"], experts, gates, layout, **kw)
    out = node.tpconv_dropout_forward(t["irreps"], 0.2, 3, 4, y, t["x"], **kw)
    gy = node.tpconv_dropout_backward(t["irreps"], 0.2, 3, 4, t["G"], **kw)
    gx, gw, gg = node.tpconv_experts_backward(t["plan"], t["x"], t["w"], experts, gates, gy, layout, **kw)
    gz = node.tpconv_route_backward(t["cfg"], t["logits"], experts, gg, **kw)
    gt = node.tpconv_embedding_backward(t["types"], gx[:, :16], t["table"].shape[0], 0.5, **kw)
    return [x, experts, gates, out, gx, gw, gg, gz, gt]


def layer_inputs(node, n, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    irreps, X, k = "16x0e+16x1o+16x2e", 8, 2
    plan = node.tpconv_experts_plan(irreps, irreps, X, k)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(types=torch.randint(0, 9, (n,), generator=g, device="cuda").int(), table=r(9, 16),
                x=r(n, plan.dim_in), logits=r(n, X), cfg=node.RouteConfig(X, k), plan=plan, irreps=irreps,
                w=r(X, plan.weight_numel), G=r(n, plan.dim_out))


def test_other_stream(node):
    import torch
    t = layer_inputs(node, 3000)
    want = [a.clone() for a in layer(node, t)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = layer(node, t, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_graph_capture_and_replays(node):
    import torch
    t = layer_inputs(node, 2500)
    layer(node, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(node, t)
    for step in range(4):
        new = layer_inputs(node, 2500, seed=step + 1)
        for name in ("types", "table", "x", "logits", "w", "G"):
            t[name].copy_(new[name])
        graph.replay()
        torch.cuda.synchronize()
        have = [a.clone() for a in got]
        t["x"].copy_(new["x"])
        want = layer(node, t)                                   # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(have, want):
            assert torch.equal(a, b)

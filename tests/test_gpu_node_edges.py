"""GPU parity of the node operators where their kernels have an edge: many
experts in one tile, keys that are no numbers, saturated scores, sizes past
one grid, buffers that cannot be used.

Bounds are those of test_gpu_node.py, which derives them: at most
(n + c + 4) eps A for a sum of n terms with absolute values A and c factors.
"""

import sys

import numpy as np
import pytest

from oracle import node as on
from test_gpu_node import EPS, NP, check_experts, config, dev, node, separated, within  # noqa: F401  (node is a fixture)

pytestmark = pytest.mark.gpu


def log(msg):
    print(msg, file=sys.stderr, flush=True)


# -------------------------------------------------------------------- experts
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("irr", ["16x0e", "17x1o", "40x2e", "20x3o+16x0e", "64x4e"])
def test_experts_many_experts_in_a_tile(node, dt, irr):  # noqa: F811
    """A tile's experts follow one another through the same places in LDS: over a hundred of them, several times."""
    import torch
    log(f"[node] many experts in a tile {dt} {irr}")
    rng = np.random.default_rng(21)
    n, X, k = 48, 160, 8
    experts = np.stack([rng.permutation(X)[:k] for _ in range(n)]).astype(np.int32)
    experts[5] = 3                                              # one expert in all places of a row
    experts[11, ::2] = -1
    gates = rng.random((n, k))
    first = check_experts(node, dt, irr, irr, X, experts, gates)
    for _ in range(3):
        again = check_experts(node, dt, irr, irr, X, experts, gates)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# -------------------------------------------------------------------- routing
def same(got, want, tol, what):
    """Within tol of |want|; NaN exactly where the definition has NaN."""
    got = got.cpu().numpy().astype(np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), (what, got, want)
    assert (np.abs(got - want)[~nan] <= (tol * np.abs(want))[~nan]).all(), (what, got, want)


# twice the logits' size and 32 units for exp and log1p, X for the sums (as in test_gpu_node.py); logits below 8
def gate_tol(X, dt):
    return (X + 2 * 8 + 32) * EPS[dt]


def put_not_numbers(rng, z, per):
    """NaN, +inf and -inf in all constellations of a row and of a group of `per`."""
    X, nan, inf = z.shape[1], np.nan, np.inf
    z[0, X // 2] = nan                                          # one NaN
    z[1] = nan                                                  # all of a row
    z[2, :per] = nan                                            # all of a group
    z[3, 0] = inf
    z[4] = -inf                                                 # a padding row
    z[5, :-1], z[5, -1] = -inf, nan                             # NaN is all that is not masked
    z[6, ::2], z[6, 1::2] = nan, -inf
    z[7, rng.random(X) < 0.5] = nan
    z[8, :per], z[8, per - 1] = -inf, nan                       # a group with one NaN alone
    z[9, rng.random(X) < 0.3], z[9, 0] = -inf, nan


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("X,G,T,k", [(8, 1, 1, 3), (12, 4, 2, 3), (24, 6, 3, 5), (64, 8, 2, 4), (100, 50, 9, 8),
                                     (256, 64, 5, 8), (7, 7, 3, 3)])
def test_routing_of_not_numbers(node, dt, score, renorm, X, G, T, k):  # noqa: F811
    """NaN keys come after every number and before the masked experts, in groups as without, and their gates are
    NaN: a row of a router that has diverged is never taken for a padding row."""
    log(f"[node] routing of NaN {dt} {score} renorm={renorm} X={X} groups={G}/{T} k={k}")
    rng = np.random.default_rng([X, G])
    cfg, ocfg = config(node, n_experts=X, top_k=k, score=score, renormalise=renorm, n_groups=G, top_groups=T)
    for bias in (None, (0.1 * rng.standard_normal(X)).astype(NP[dt])):
        z = separated(rng, 40, X, bias, ocfg, dt, 0.05)
        put_not_numbers(rng, z, X // G)
        experts, gates = node.tpconv_route_forward(cfg, dev(z), None if bias is None else dev(bias))
        want_e, want_g = on.route_forward(z, bias, ocfg)
        assert np.array_equal(experts.cpu().numpy(), want_e)
        same(gates, want_g, gate_tol(X, dt), "gates")
        assert (want_e[1] >= 0).all() and np.isnan(want_g[1]).all()
        assert (want_e[5, 0], want_e[4, 0]) == (X - 1, -1)


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("X,G,T,k", [(8, 1, 1, 3), (12, 4, 2, 3), (24, 6, 3, 5), (64, 8, 2, 4), (256, 64, 5, 8)])
def test_routing_with_infinite_and_lowest_biases(node, dt, score, X, G, T, k):  # noqa: F811
    """A bias of -inf masks its expert; the type's lowest value puts it last, and its group behind the others'."""
    log(f"[node] routing biases {dt} {score} X={X} groups={G}/{T} k={k}")
    rng = np.random.default_rng([X, G, 1])
    cfg, ocfg = config(node, n_experts=X, top_k=k, score=score, n_groups=G, top_groups=T)
    per, low = X // G, np.finfo(NP[dt]).min
    masks = [np.zeros(X) for _ in range(6)]
    masks[0][: X - 2] = -np.inf                                 # fewer than top_k left
    masks[1][::2] = -np.inf
    masks[2][:per] = -np.inf                                    # a whole group
    masks[3][:] = -np.inf                                       # nothing left
    masks[4][:per], masks[4][-1] = low, low                     # a group put last, and one expert of another
    masks[5][0], masks[5][X // 2] = np.inf, -np.inf
    for bias in masks:
        bias = bias.astype(NP[dt])
        z = separated(rng, 20, X, np.where(bias == low, -np.inf, bias), ocfg, dt, 0.2)
        z[4] = np.nan
        experts, gates = node.tpconv_route_forward(cfg, dev(z), dev(bias))
        want_e, want_g = on.route_forward(z, bias, ocfg)
        assert np.array_equal(experts.cpu().numpy(), want_e), bias
        same(gates, want_g, gate_tol(X, dt), "gates")
        assert not np.isneginf(bias[want_e[want_e >= 0]]).any()


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("X,k", [(6, 2), (8, 4), (16, 3), (50, 8), (256, 8)])
def test_routing_of_saturated_scores_goes_by_the_logits(node, dt, score, X, k):  # noqa: F811
    """Scores that round to 1 or to 0 are told apart by their logits, with a bias of zeros as without one."""
    rng = np.random.default_rng([X, k])
    cfg, ocfg = config(node, n_experts=X, top_k=k, score=score, scale=3.0)
    z = np.zeros((40, X))
    z[0] = -5000.0
    z[0, X // 2] += 1.0                                         # all underflow as sigmoids
    z[1] = 60.0 + rng.permutation(X)                            # all 1 as sigmoids
    z[2] = -3000.0 - rng.permutation(X)
    z[3] = np.where(rng.random(X) < 0.5, 1.0, -1.0) * (1000.0 + rng.permutation(X))
    z[4] = np.where(np.arange(X) < X // 2, 70.0, 71.0)          # ties of logits as well: the lowest index
    z[5] = np.finfo(NP[dt]).min
    z[6], z[6, 1:] = np.finfo(NP[dt]).min, -4000.0 - rng.permutation(X - 1)
    z[7:] = 2000.0 * rng.integers(-2, 3, (33, X)) + rng.integers(0, 5, (33, X))
    z[8:, 0] = -np.inf
    z = z.astype(NP[dt])
    zero = np.zeros(X, NP[dt])
    want_e, want_g = on.route_forward(z, None, ocfg)
    for bias in (None, zero, -zero):
        experts, gates = node.tpconv_route_forward(cfg, dev(z), None if bias is None else dev(bias))
        assert np.array_equal(experts.cpu().numpy(), want_e)
        # gates are formed from differences of logits up to 8000, exact here, and their exponentials
        within(gates, want_g, (X + 64) * EPS[dt] * np.abs(want_g) + 1e-30, "gates")


def test_routing_in_groups_goes_by_the_logits_too(node):  # noqa: F811
    """Inside the chosen groups; groups whose keys tie go by their index."""
    cfg, ocfg = config(node, n_experts=12, top_k=4, score="sigmoid", n_groups=3, top_groups=2)
    z = np.array([[50, 51, 52, 53, -50, -51, -52, -53, 60, 61, 62, 63],
                  [-200, -201, -202, -203, 300, 301, 302, 303, 0, 0, 1, 1]], np.float32)
    zero = np.zeros(12, np.float32)
    for bias in (None, zero):
        experts, _ = node.tpconv_route_forward(cfg, dev(z), None if bias is None else dev(bias))
        assert np.array_equal(experts.cpu().numpy(), on.route_forward(z, bias, ocfg)[0])
        assert experts.cpu().numpy().tolist() == [[11, 10, 9, 8], [7, 6, 5, 4]]


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_of_a_row_does_not_depend_on_its_neighbours(node, dt, renorm):  # noqa: F811
    """Bit by bit: among rows whose sigmoids underflow, are NaN or are masked, as alone."""
    import torch
    rng = np.random.default_rng(5)
    for X, k in ((8, 2), (16, 3), (100, 6)):
        cfg = node.RouteConfig(X, k, score="sigmoid", renormalise=renorm)
        z = rng.standard_normal((64, X)).astype(NP[dt])
        other = z.copy()
        other[1::2] = -4000.0 + other[1::2]
        other[3::8] = np.nan
        other[5::8] = -np.inf
        g = rng.standard_normal((64, k)).astype(NP[dt])
        e, a = node.tpconv_route_forward(cfg, dev(z))
        e2, b = node.tpconv_route_forward(cfg, dev(other))
        assert torch.equal(e[::2], e2[::2]) and torch.equal(a[::2], b[::2])
        d, d2 = (node.tpconv_route_backward(cfg, dev(v), i, dev(g)) for v, i in ((z, e), (other, e2)))
        assert torch.equal(d[::2], d2[::2])


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("n,X,k", [(5000, 256, 1), (2341, 256, 7), (2100, 200, 8)])
def test_experts_in_groups_longer_than_two_rows_a_thread(node, dt, n, X, k):  # noqa: F811
    """Many experts make the layout's groups longer; two groups, the second short."""
    log(f"[node] long groups {dt} n={n} X={X} k={k}")
    rng = np.random.default_rng([n, X])
    experts = rng.integers(-1, X + 1, (n, k)).astype(np.int32)   # none, doubles and an index outside among them
    experts[: n // 8] = X - 1
    check_experts(node, dt, "3x0e+1x1o", "2x0e+2x1o", X, experts, rng.random((n, k)))


# ------------------------------------------------------------------- refusals
def test_buffers_that_are_not_on_the_device_are_refused(node):  # noqa: F811
    """Workspaces and layout buffers in host memory or with gaps, before anything is launched."""
    import torch
    x = torch.zeros((4, 8), device="cuda")
    types = torch.zeros(4, dtype=torch.int32, device="cuda")
    plan = node.tpconv_experts_plan("8x0e", "8x0e", 3, 2)
    e, g, w = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda"), \
        torch.zeros((3, 64), device="cuda")
    layout = node.tpconv_experts_layout(plan, e)
    wide = torch.zeros((1 << 16, 2), dtype=torch.uint8, device="cuda")[:, 0]
    for buffer in (torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(1 << 16, dtype=torch.uint8).pin_memory(), wide):
        with pytest.raises(ValueError):
            node.tpconv_embedding_backward(types, x, 3, workspace=buffer)
        with pytest.raises(ValueError):
            node.tpconv_experts_layout(plan, e, buffer=buffer)
        with pytest.raises(ValueError):
            node.tpconv_experts_backward(plan, x, w, e, g, x, layout, workspace=buffer)
        with pytest.raises(ValueError):
            node.tpconv_experts_backward(plan, x, w, e, g, x, need=(False, False, True), workspace=buffer)
    with pytest.raises(RuntimeError, match="TPCONV_E_WORKSPACE"):
        node.tpconv_experts_layout(plan, e, buffer=torch.zeros(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("dim", [3, 4, 64])
def test_embedding_of_padding_rows_is_zero_whatever_the_scale(node, dt, dim):  # noqa: F811
    import torch
    t = np.array([-1, 0, 7, 1, -1], np.int32)
    table = torch.ones((2, dim), dtype=getattr(torch, {"f32": "float32", "f64": "float64"}[dt]), device="cuda")
    for scale in (float("inf"), float("nan")):
        out = node.tpconv_embedding_forward(dev(t), table, scale).cpu().numpy()
        assert (out[[0, 2, 4]] == 0).all() and not np.isfinite(out[[1, 3]]).any()
        grad = node.tpconv_embedding_backward(dev(t), torch.ones((5, dim), dtype=table.dtype, device="cuda"), 3, scale)
        assert (grad[2] == 0).all() and not torch.isfinite(grad[:2]).any()


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("mul", [1, 5, 16, 17, 50, 65])
def test_experts_gate_gradients_that_are_infinite(node, dt, mul):  # noqa: F811
    """One product overflows, in the last channel: the gate's gradient is infinite with its sign, not NaN."""
    import torch
    rng = np.random.default_rng(mul)
    irr, n, k, X = f"{mul}x1o", 20, 2, 3
    plan = node.tpconv_experts_plan(irr, irr, X, k, dt)
    x, G = (rng.random((n, 3 * mul)) + 0.5 for _ in range(2))
    w = rng.random((X, mul, mul)) + 0.5
    G[:, -1], w[1, mul - 1, mul - 1] = 1e10, 0.5 * float(np.finfo(NP[dt]).max)   # of the last component alone
    experts = np.tile(np.array([0, 1], np.int32), (n, 1))
    experts[::3] = [2, 0]
    a = [dev(v.astype(NP[dt])) for v in (x, w.reshape(X, -1))] + [dev(experts)] + [dev(np.ones((n, k), NP[dt]))]
    layout = node.tpconv_experts_layout(plan, a[2])
    gg = node.tpconv_experts_backward(plan, *a, dev(G.astype(NP[dt])), layout, need=(False, False, True))[2]
    assert (torch.isposinf(gg).cpu().numpy() == (experts == 1)).all() and not torch.isnan(gg).any()


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("X,G,T,k", [(8, 1, 1, 3), (24, 6, 3, 5), (100, 50, 9, 8), (7, 7, 3, 3)])
def test_routing_gradient_of_not_numbers(node, dt, score, renorm, X, G, T, k):  # noqa: F811
    """NaN where the formula has one, for the same rows as the forward; the masked get 0."""
    rng = np.random.default_rng([X, G, 2])
    cfg, ocfg = config(node, n_experts=X, top_k=k, score=score, renormalise=renorm, n_groups=G, top_groups=T)
    z = separated(rng, 40, X, None, ocfg, dt, 0.05)
    put_not_numbers(rng, z, X // G)
    experts, _ = node.tpconv_route_forward(cfg, dev(z))
    e = experts.cpu().numpy()
    g = rng.standard_normal((40, k)).astype(NP[dt])
    g[11, 0] = np.nan
    got = node.tpconv_route_backward(cfg, dev(z), experts, dev(np.where(e < 0, 1.0, g).astype(NP[dt])))
    got = got.cpu().numpy().astype(np.float64)
    with np.errstate(all="ignore"):
        want = on.route_backward(z, e, g, ocfg)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert (got[np.isneginf(z)] == 0).all()
    # a gate (1 at most) times gradients of the row, and their rounding as in test_gpu_node.py
    size = 3 * (gate_tol(X, dt) + (k + 6) * EPS[dt]) * 2 * np.nansum(np.abs(np.where(e < 0, 0.0, g)), 1, keepdims=True)
    assert (np.abs(got - want) <= size)[~np.isnan(want)].all()


def test_experts_second_derivatives_from_the_same_calls(node):  # noqa: F811
    """The maps are linear in x, in the weights and in the gates, so the gradients of

        S = <grad_x, u> + <grad_weights, v> + <grad_gates, t>

    are sums of forwards and backwards with one argument replaced by its direction; here against differences."""
    import torch
    rng = np.random.default_rng(31)
    irr_in, irr_out, n, X, k = "5x0e+4x1o+3x2e", "3x0e+6x1o+2x2e", 40, 4, 2
    plan = node.tpconv_experts_plan(irr_in, irr_out, X, k, "f64")
    experts = rng.integers(-1, X, (n, k)).astype(np.int32)
    e = dev(experts)
    layout = node.tpconv_experts_layout(plan, e)
    shapes = dict(x=(n, plan.dim_in), w=(X, plan.weight_numel), g=(n, k), G=(n, plan.dim_out))
    a = {name: dev(rng.standard_normal(s)) for name, s in shapes.items()}
    u, v, t = (dev(rng.standard_normal(shapes[name])) for name in "xwg")

    def forward(x, w, g):
        return node.tpconv_experts_forward(plan, x, w, e, g, layout)

    def backward(x, w, g, G):
        return node.tpconv_experts_backward(plan, x, w, e, g, G, layout)

    def S(x, w, g, G):
        return sum(float((p * q).sum()) for p, q in zip(backward(x, w, g, G), (u, v, t)))

    x, w, g, G = a["x"], a["w"], a["g"], a["G"]
    at_u, at_v, at_t = backward(u, w, g, G), backward(x, v, g, G), backward(x, w, t, G)
    second = dict(G=forward(u, w, g) + forward(x, v, g) + forward(x, w, t), x=at_v[0] + at_t[0], w=at_u[1] + at_t[1],
                  g=at_u[2] + at_v[2])
    for name, grad in second.items():
        d = dev(rng.standard_normal(shapes[name]))
        lo, hi = (S(**dict(a, **{name: a[name] + s * d})) for s in (-0.5, 0.5))
        # linear in each argument: only the difference's own rounding is left (about 1e4 terms of size 10, step 1/2)
        assert abs(hi - lo - float((grad * d).sum())) < 1e-8, name


# -------------------------------------------------------------------- capture
@pytest.mark.parametrize("irr,X,k", [("64x4e", 3, 2), ("200x3o+5x0e", 200, 8)])
def test_experts_with_more_than_64_kib_of_lds_in_a_graph(node, irr, X, k):  # noqa: F811
    """Blocks above the default limit of LDS are set up outside the stream: calls can be captured all the same."""
    import torch
    n, g = 300, torch.Generator(device="cuda").manual_seed(3)
    plan = node.tpconv_experts_plan(irr, irr, X, k, "f64")

    def inputs():
        r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
        return [r(n, plan.dim_in), r(X, plan.weight_numel),
                torch.randint(-1, X, (n, k), generator=g, device="cuda").int(), r(n, k), r(n, plan.dim_out)]

    def call(x, w, e, gates, G):
        layout = node.tpconv_experts_layout(plan, e)
        return (node.tpconv_experts_forward(plan, x, w, e, gates, layout),
                *node.tpconv_experts_backward(plan, x, w, e, gates, G, layout))

    held = inputs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                              # the first call of these kernels
        got = call(*held)
    for _ in range(3):
        new = inputs()
        for a, b in zip(held, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        have = [a.clone() for a in got]
        for a, b in zip(have, call(*new)):
            assert torch.equal(a, b)

"""Pins of the node operators' fp64 definitions (oracle/node.py) against
mathematics they do not use: published generator outputs, central
differences, adjointness, one-hot and dense forms, rotations, brute force.

Differences: a central difference with step h of a smooth function of size
O(1) is off by its third derivative times h^2/6 plus eps/h; with h = 1e-5 both
are below 1e-9, so 1e-7 absolute holds with room for the functions' scale.
"""

import itertools

import numpy as np
import pytest

import workloads
from oracle import node as on
from oracle.irreps import parse_irreps
from oracle.so2 import wigner_D

H, TOL = 1e-5, 1e-7


def difference(f, x, direction):
    return (f(x + H * direction) - f(x - H * direction)) / (2 * H)


# ------------------------------------------------------------------ generator
@pytest.mark.parametrize("counter,key,words", [
    # the generator's published known answers (ten rounds)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, words):
    assert tuple(on.philox4x32(counter, key)) == words


def test_dropout_mask_is_shared_by_a_channel_and_kept_at_the_rate():
    irreps = "3x0e+5x1o+2x2e"
    keep = on.dropout_keep(irreps, 400, 0.3, 11, 5)
    for mul, l, _, at in on.segments(irreps)[0]:
        block = keep[:, at:at + mul * (2 * l + 1)].reshape(400, mul, 2 * l + 1)
        assert (block == block[:, :, :1]).all()
    # 4000 draws: the kept share is within 5 standard deviations of 0.7
    share = np.mean(on.dropout_keep("10x0e", 400, 0.3, 11, 5))
    assert abs(share - 0.7) < 5 * np.sqrt(0.3 * 0.7 / 4000)
    assert on.dropout_keep(irreps, 7, 0.0, 1, 2).all()
    assert (on.dropout_keep("4x0e", 8, 0.5, 1, 2) != on.dropout_keep("4x0e", 8, 0.5, 1, 3)).any()
    # a row's draws do not depend on how many rows follow
    assert (on.dropout_keep(irreps, 9, 0.5, 1, 2) == on.dropout_keep(irreps, 20, 0.5, 1, 2)[:9]).all()


def test_dropout_is_equivariant():
    rng = np.random.default_rng(3)
    irreps, n = "4x0e+3x1o+2x2e", 6
    x, res = rng.standard_normal((2, n, on.segments(irreps)[1]))
    R = workloads.random_rotation(rng)

    def rotate(a):
        out = np.empty_like(a)
        for mul, l, _, at in on.segments(irreps)[0]:
            blk = a[:, at:at + mul * (2 * l + 1)].reshape(n, mul, 2 * l + 1)
            out[:, at:at + mul * (2 * l + 1)] = (blk @ wigner_D(l, R)[l][0].T).reshape(n, -1)
        return out

    a = rotate(on.dropout_forward(irreps, 0.4, 5, 1, x, res))
    b = on.dropout_forward(irreps, 0.4, 5, 1, rotate(x), rotate(res))
    np.testing.assert_allclose(a, b, atol=1e-12)


# ------------------------------------------------------------------ embedding
def test_embedding_is_a_one_hot_product():
    rng = np.random.default_rng(0)
    types = np.array([2, 0, -1, 3, 2, 7, 0])
    table, grad = rng.standard_normal((4, 5)), rng.standard_normal((7, 5))
    hot = (types[:, None] == np.arange(4)).astype(float)
    np.testing.assert_allclose(on.embedding_forward(types, table, 1.5), 1.5 * hot @ table, atol=1e-15)
    np.testing.assert_allclose(on.embedding_backward(types, grad, 4, 1.5), 1.5 * hot.T @ grad, atol=1e-14)


# -------------------------------------------------------------------- routing
CONFIGS = [dict(score=s, renormalise=r, n_groups=g, top_groups=t, top_k=k, scale=c)
           for s, r, (g, t, k), c in itertools.product(("softmax", "sigmoid"), (True, False),
                                                       ((1, 1, 3), (4, 2, 4)), (1.0, 2.5))]


@pytest.mark.parametrize("cfg", CONFIGS, ids=str)
def test_route_gradient_against_differences(cfg):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((5, 12))
    z[1, 3] = z[2, :9] = -np.inf
    z[3] = -np.inf
    bias = 0.3 * rng.standard_normal(12)
    experts, gates = on.route_forward(z, bias, cfg)
    g = rng.standard_normal(gates.shape)
    grad = on.route_backward(z, experts, g, cfg)
    assert np.all(grad[np.isneginf(z)] == 0)
    for i in range(len(z)):
        picked = [int(e) for e in experts[i] if e >= 0]
        live = np.where(~np.isneginf(z[i]))[0]
        for e in live:
            d = np.zeros(12)
            d[e] = 1.0
            num = difference(lambda y: np.dot(g[i, :len(picked)], on.gates_of(y, picked, cfg)), z[i], d)
            assert abs(num - grad[i, e]) < TOL


def test_route_selection_brute_force_ties_and_masks():
    cfg = dict(score="sigmoid", renormalise=False, n_groups=3, top_groups=2, top_k=3, scale=1.0)
    rng = np.random.default_rng(2)
    for _ in range(200):
        z = np.round(rng.standard_normal(9), 1)                   # ties on purpose
        z[rng.random(9) < 0.25] = -np.inf
        key = on.keys(z, None, "sigmoid")
        got = on.choose(z, None, cfg)
        groups = []
        for g in range(3):
            live = sorted((k for k in key[3 * g:3 * g + 3] if k > -np.inf), reverse=True)
            groups.append(sum(live[:2]) if live else -np.inf)
        kept = sorted(range(3), key=lambda g: (-groups[g], g))[:2]
        want = sorted((e for e in range(9) if e // 3 in kept and key[e] > -np.inf), key=lambda e: (-key[e], e))[:3]
        assert got == want
    assert on.choose(np.full(9, -np.inf), None, cfg) == []


def test_route_nan_comes_after_numbers_and_before_masks():
    nan, inf = np.nan, np.inf
    cfg = dict(score="sigmoid", renormalise=True, n_groups=3, top_groups=2, top_k=4, scale=1.0)
    z = np.array([[nan, nan, 1.0, 2.0, nan, -inf],              # groups: NaN twice; two numbers; NaN alone
                  [nan, nan, nan, nan, nan, nan],
                  [-inf, -inf, nan, -inf, -inf, -inf],
                  [3.0, nan, -inf, -inf, 1.0, 2.0]])
    experts, gates = on.route_forward(z, None, cfg)
    assert experts.tolist() == [[3, 2, 4, -1], [0, 1, 2, 3], [2, -1, -1, -1], [0, 5, 4, 1]]
    assert np.isnan(gates[:, 0]).all() and (gates[2, 1:] == 0).all()
    # softmax: every score of such a row is NaN, and so are its gates, chosen from what is not masked
    experts, gates = on.route_forward(z, None, dict(cfg, score="softmax"))
    assert experts[3].tolist()[:2] == [0, 1] and np.isnan(gates[experts >= 0]).all()
    assert on.route_forward(np.array([[inf, 0.0, 1.0, 2.0]]), None, dict(cfg, n_groups=1, score="softmax",
                                                                         top_k=2))[0].tolist() == [[0, 1]]


def test_route_bias_of_minus_infinity_masks():
    """As if the expert's logit were -inf, but for the softmax's sum."""
    rng = np.random.default_rng(6)
    for score, groups in itertools.product(("softmax", "sigmoid"), (1, 3)):
        cfg = dict(score=score, renormalise=True, n_groups=groups, top_groups=min(2, groups), top_k=3, scale=1.0)
        z = rng.standard_normal((20, 9))
        bias = np.where(rng.random(9) < 0.4, -np.inf, 0.0)
        z[0, 0] = np.nan
        experts, gates = on.route_forward(z, bias, cfg)
        e, g = on.route_forward(np.where(np.isneginf(bias), -np.inf, z)[1:], None, cfg)
        assert (experts[1:] == e).all()
        np.testing.assert_allclose(gates[1:], g, rtol=1e-14)
        assert not np.isneginf(bias[experts[experts >= 0]]).any()


def test_route_of_saturated_scores_goes_by_the_logits():
    """In the order of the exact scores, which the logits have: in 64 bits sigmoids above 40 are 1."""
    rng = np.random.default_rng(7)
    cfg = dict(score="sigmoid", renormalise=True, n_groups=1, top_groups=1, top_k=4, scale=1.0)
    z = np.where(rng.random((30, 10)) < 0.5, 900.0, -900.0) + rng.integers(0, 6, (30, 10))
    for bias in (None, np.zeros(10)):
        experts, _ = on.route_forward(z, bias, cfg)
        assert (experts == np.argsort(-z, axis=1, kind="stable")[:, :4]).all()


def test_renormalised_gates_sum_to_scale_where_scores_underflow():
    for kind in ("softmax", "sigmoid"):
        cfg = dict(score=kind, renormalise=True, n_groups=1, top_groups=1, top_k=2, scale=3.0)
        z = np.full((1, 4), -5000.0)
        z[0, 2] += np.log(2.0)
        experts, gates = on.route_forward(z, None, cfg)
        np.testing.assert_allclose(gates.sum(), 3.0, rtol=1e-12)
        if kind == "softmax":
            np.testing.assert_allclose(gates[0], [2.0, 1.0], rtol=1e-12)


# -------------------------------------------------------------------- experts
IRREPS = [("3x0e+2x1o", "4x0e+3x1o"), ("2x1o+3x0e+2x2e", "1x2e+5x1e+2x1o"), ("4x0e", "6x0e")]


@pytest.mark.parametrize("irr_in,irr_out", IRREPS)
def test_experts_against_dense_matrices_and_differences(irr_in, irr_out):
    rng = np.random.default_rng(4)
    X, k, n = 3, 2, 5
    d_in, d_out, numel = on.segments(irr_in)[1], on.segments(irr_out)[1], on.expert_maps(irr_in, irr_out)[1]
    x, G = rng.standard_normal((n, d_in)), rng.standard_normal((n, d_out))
    w, gates = rng.standard_normal((X, numel)), rng.random((n, k))
    experts = np.array([[0, 2], [1, -1], [2, 2], [-1, -1], [1, 0]])
    out = on.experts_forward(irr_in, irr_out, x, w, experts, gates)
    # each expert as one dense matrix: its action on unit vectors
    one = np.ones((d_in, 1))
    dense = [on.experts_forward(irr_in, irr_out, np.eye(d_in), w, np.full((d_in, 1), e), one) for e in range(X)]
    want = np.stack([sum((gates[i, a] * x[i] @ dense[e] for a, e in enumerate(experts[i]) if e >= 0),
                         np.zeros(d_out)) for i in range(n)])
    np.testing.assert_allclose(out, want, atol=1e-13)
    gx, gw, gg = on.experts_backward(irr_in, irr_out, x, w, experts, gates, G)
    for name, arr, grad in (("x", x, gx), ("w", w, gw), ("gates", gates, gg)):
        d = rng.standard_normal(arr.shape)
        d /= np.linalg.norm(d)
        args = dict(x=x, w=w, gates=gates)

        def f(a):
            q = dict(args, **{name: a})
            return np.sum(G * on.experts_forward(irr_in, irr_out, q["x"], q["w"], experts, q["gates"]))
        assert abs(difference(f, arr, d) - np.sum(grad * d)) < TOL, name
    assert np.all(gg[experts < 0] == 0)


def test_experts_are_equivariant():
    rng = np.random.default_rng(5)
    irr_in, irr_out, n = "3x0e+2x1o+2x2e", "2x0e+3x1o+1x2e", 4
    x = rng.standard_normal((n, on.segments(irr_in)[1]))
    w = rng.standard_normal((2, on.expert_maps(irr_in, irr_out)[1]))
    experts, gates = np.array([[0, 1], [1, 0], [1, -1], [0, 0]]), rng.random((n, 2))
    R = workloads.random_rotation(rng)

    def rotate(a, irreps):
        out = np.empty_like(a)
        for mul, l, _, at in on.segments(irreps)[0]:
            blk = a[:, at:at + mul * (2 * l + 1)].reshape(n, mul, 2 * l + 1)
            out[:, at:at + mul * (2 * l + 1)] = (blk @ wigner_D(l, R)[l][0].T).reshape(n, -1)
        return out

    np.testing.assert_allclose(rotate(on.experts_forward(irr_in, irr_out, x, w, experts, gates), irr_out),
                               on.experts_forward(irr_in, irr_out, rotate(x, irr_in), w, experts, gates), atol=1e-12)


# ------------------------------------------------------- many rows at a time
@pytest.mark.parametrize("cfg", CONFIGS, ids=str)
def test_route_of_many_rows_is_that_of_each(cfg):
    rng = np.random.default_rng(13)
    z = 2.0 * rng.standard_normal((60, 12))
    z[:20] = np.round(z[:20])                                     # ties
    z[rng.random(z.shape) < 0.3] = -np.inf
    z[7], z[8] = -np.inf, 50.0 * z[8]
    for bias in (None, 0.2 * rng.standard_normal(12), np.where(rng.random(12) < 0.3, -np.inf, 0.1)):
        experts, gates = on.route_forward(z, bias, cfg)
        e, g, gap = on.route_many(z, bias, cfg)
        assert np.array_equal(e, experts)
        np.testing.assert_allclose(g, gates, rtol=1e-13, atol=0)
        grad = rng.standard_normal(gates.shape)
        np.testing.assert_allclose(on.route_backward_many(z, e, g, grad, cfg),
                                   on.route_backward(z, experts, grad, cfg), rtol=1e-11, atol=1e-15)
        # the gap: choices outlast a change of the keys by less than half of it
        for i in range(len(z)):
            key = on.keys(z[i], bias, cfg["score"])
            if cfg["n_groups"] == 1 and gap[i] < np.inf:
                k = np.sort(key[~np.isneginf(key)])[::-1][:cfg["top_k"] + 1]
                assert abs(gap[i] - (k[:-1] - k[1:]).min()) < 1e-15


def test_experts_and_dropout_of_many_rows_are_those_of_each():
    rng = np.random.default_rng(14)
    irr_in, irr_out, n, X, k = "3x0e+2x1o+1x2e", "2x1o+4x0e", 40, 5, 3
    x, G = rng.standard_normal((n, on.segments(irr_in)[1])), rng.standard_normal((n, on.segments(irr_out)[1]))
    w, gates = rng.standard_normal((X, on.expert_maps(irr_in, irr_out)[1])), rng.random((n, k))
    experts = rng.integers(-1, X + 1, (n, k))                     # none, doubles and an index outside among them
    want = (on.experts_forward(irr_in, irr_out, x, w, experts, gates),
            *on.experts_backward(irr_in, irr_out, x, w, experts, gates, G))
    for a, b in zip(on.experts_many(irr_in, irr_out, x, w, experts, gates, G), want):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-13)
    for irr in ("3x0e+2x1o+1x2e", "1x1o+1x1o+7x0e", "5x0e"):
        args = (irr, 33, 0.3, 0xFEDCBA9876543210, (1 << 40) + 7)
        assert (on.dropout_keep_many(*args) == on.dropout_keep(*args)).all()


def test_experts_of_many_rows_where_an_expert_has_none():
    rng = np.random.default_rng(15)
    x, G, w = rng.standard_normal((4, 5)), rng.standard_normal((4, 5)), rng.standard_normal((6, 5))
    for experts in (np.array([[0], [5], [-1], [5]]), np.full((4, 1), -1)):
        gates = rng.random((4, 1))
        want = (on.experts_forward("2x0e+1x1o", "2x0e+1x1o", x, w, experts, gates),
                *on.experts_backward("2x0e+1x1o", "2x0e+1x1o", x, w, experts, gates, G))
        for a, b in zip(on.experts_many("2x0e+1x1o", "2x0e+1x1o", x, w, experts, gates, G), want):
            np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-13)


def test_segments_agree_with_the_convolution_oracle():
    for text in ("32x0e+32x1o", "4x1o+2x0e + 3x2e"):
        assert on.segments(text)[1] == parse_irreps(text).dim

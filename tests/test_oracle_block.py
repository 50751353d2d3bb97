"""Pins of the fp64 definitions in oracle/block.py: closed forms, differences,
rotation equivariance, torch's 8-bit conversion."""

import math

import numpy as np
import pytest

from oracle import block as ob
from oracle.node import segments
from oracle.so2 import wigner_D

IRREPS = "3x0e+2x1o+4x2e+1x3o+2x0o"


def rows(rng, irreps, n):
    return rng.standard_normal((n, segments(irreps)[1]))


def difference(f, v, h=1e-6):
    """Central differences of the scalar f at the array v."""
    out = np.zeros_like(v)
    for i in np.ndindex(*v.shape):
        keep = v[i]
        v[i] = keep + h
        up = f(v)
        v[i] = keep - h
        out[i] = (up - f(v)) / (2 * h)
        v[i] = keep
    return out


def rotated(irreps, R, x):
    out = np.empty_like(x)
    for s in segments(irreps)[0]:
        ob.part(out, s)[...] = ob.part(x, s) @ wigner_D(s[1], R)[s[1]][0].T
    return out


def rotation(rng):
    q, _ = np.linalg.qr(rng.standard_normal((3, 3)))
    return q * np.sign(np.linalg.det(q))


@pytest.mark.parametrize("scope", ["segment", "row"])
def test_norm(scope):
    rng = np.random.default_rng(1)
    x, res, G, H = (rows(rng, IRREPS, 3) for _ in range(4))
    gamma = rng.standard_normal(ob.channels(IRREPS)[1])
    y, h = ob.norm_forward(IRREPS, scope, 1e-3, x, res, gamma)
    assert np.array_equal(h, x + res)
    # one segment of one row by hand; the row's factor from the plain mean of its segments' means
    ms = [np.mean(h[0, s[3]:s[3] + s[0] * (2 * s[1] + 1)] ** 2) for s in segments(IRREPS)[0]]
    by = ms[1] if scope == "segment" else np.mean(ms)
    assert np.allclose(y[0, 3:9], h[0, 3:9] / np.sqrt(by + 1e-3) * np.repeat(gamma[3:5], 3), rtol=1e-14)

    def loss(v, w):
        y, h = ob.norm_forward(IRREPS, scope, 1e-3, v, res, w)
        return (y * G).sum() + (h * H).sum()
    gx, gg = ob.norm_backward(IRREPS, scope, 1e-3, h, gamma, G, H)
    assert np.allclose(gx, difference(lambda v: loss(v, gamma), x.copy()), atol=1e-8)
    assert np.allclose(gg, difference(lambda w: loss(x, w), gamma.copy()), atol=1e-8)
    R = rotation(rng)
    turned = ob.norm_forward(IRREPS, scope, 1e-3, rotated(IRREPS, R, x), rotated(IRREPS, R, res), gamma)[0]
    assert np.allclose(turned, rotated(IRREPS, R, y), atol=1e-12)


def test_norm_of_scalars_is_the_plain_one():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 10))
    want = x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6)
    for scope in ("segment", "row"):
        assert np.allclose(ob.norm_forward("10x0e", scope, 1e-6, x)[0], want, rtol=1e-15)


def test_e4m3_codes_are_torchs():
    import torch
    rng = np.random.default_rng(3)
    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ob.e4m3_values(), values, equal_nan=True)
    v = np.concatenate([rng.uniform(-448, 448, 4000), 2.0 ** rng.uniform(-12, 8.8, 4000), values[:127],
                        (values[:126] + values[1:127]) / 2, [0.0, -0.0, 448.0001]]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ob.e4m3_codes(v), want)


def test_pack8_restores():
    rng = np.random.default_rng(4)
    x = (rows(rng, IRREPS, 40) * np.exp(8 * rng.standard_normal((40, 1)))).astype(np.float32)
    x[5] = 0
    codes, scales = ob.pack8(IRREPS, x)
    back = ob.unpack8(IRREPS, codes, scales)
    for s in segments(IRREPS)[0]:
        a, b = ob.part(x, s).reshape(40, -1), ob.part(back, s).reshape(40, -1)
        assert (np.abs(a - b) <= np.abs(a).max(1, keepdims=True) / 28 * 1.00001).all()
    assert not back[5].any()
    # restored rows get the same codes (their scales may round to a neighbour: 448 s times the fp32 number 1/448)
    live = np.arange(40) != 5
    assert np.array_equal(ob.pack8(IRREPS, back)[0][live], codes[live])


@pytest.mark.parametrize("act", sorted(ob.GROWTH))
def test_activations(act):
    from scipy.stats import norm as gauss
    z = np.linspace(-30, 30, 6001)
    value, slope = ob.activation(act, z)
    plain = {"identity": lambda v: v, "tanh": np.tanh, "sigmoid": lambda v: 0.5 * (1 + np.tanh(v / 2)),
             "silu": lambda v: 0.5 * v * (1 + np.tanh(v / 2)), "gelu": lambda v: v * gauss.cdf(v)}[act]
    assert np.allclose(value, plain(z), atol=1e-14, rtol=1e-13)
    h = 1e-5
    assert np.allclose(slope, (plain(z + h) - plain(z - h)) / (2 * h), atol=1e-9)
    assert (np.abs(slope) <= ob.GROWTH[act]).all()
    assert (np.abs(np.diff(slope)) <= ob.BEND[act] * np.diff(z) + 1e-15).all()
    far = ob.activation(act, np.array([-1e4, 1e4]))
    assert np.isfinite(far).all()


@pytest.mark.parametrize("act,gate", [("silu", "sigmoid"), ("gelu", "tanh"), ("sigmoid", "silu"),
                                      ("identity", "identity")])
def test_gated(act, gate):
    rng = np.random.default_rng(5)
    irr_in, irr_out = "2x1o+3x0e+2x2e+1x0o", "2x0o+3x1o+4x0e"
    x, G = rows(rng, irr_in, 3), rows(rng, irr_out, 3)
    W = rng.standard_normal(ob.maps(irr_in, irr_out)[1])
    Wg, b = rng.standard_normal((3, 9)), rng.standard_normal(9)
    out = ob.gated_forward(irr_in, irr_out, act, gate, x, W, Wg, b)
    # an entry by hand: 1o's second channel, third component; its gate is channel 2 + 1
    z = sum(x[1, 6 + u] * Wg[u, 3] for u in range(3)) + b[3]
    M = W[:6].reshape(2, 3)
    want = ob.activation(gate, z)[0] * sum(x[1, 3 * u + 2] * M[u, 1] for u in range(2))
    assert np.isclose(out[1, 2 + 3 * 1 + 2], want, rtol=1e-13)

    def loss(x=x, W=W, Wg=Wg, b=b):
        return (ob.gated_forward(irr_in, irr_out, act, gate, x, W, Wg, b) * G).sum()
    got = ob.gated_backward(irr_in, irr_out, act, gate, x, W, Wg, b, G)
    for name, v, g in zip(("x", "W", "Wg", "b"), (x, W, Wg, b), got):
        assert np.allclose(g, difference(lambda t: loss(**{name: t}), v.copy()), atol=2e-8), name
    R = rotation(rng)
    turned = ob.gated_forward(irr_in, irr_out, act, gate, rotated(irr_in, R, x), W, Wg, b)
    assert np.allclose(turned, rotated(irr_out, R, out), atol=1e-12)


@pytest.mark.parametrize("act", sorted(ob.GROWTH))
def test_linear(act):
    rng = np.random.default_rng(6)
    irr_in, irr_out = "2x1o+3x0e+2x2e+2x0o", "2x0o+3x1o+4x0e"
    x, G, res = rows(rng, irr_in, 3), rows(rng, irr_out, 3), rows(rng, irr_out, 3)
    W, b = rng.standard_normal(ob.maps(irr_in, irr_out)[1]), rng.standard_normal(4)
    out = ob.linear_forward(irr_in, irr_out, act, x, W, b, res)
    M = W[6:18].reshape(3, 4)
    want = res[2, 11 + 3] + ob.activation(act, sum(x[2, 6 + u] * M[u, 3] for u in range(3)) + b[3])[0]
    assert np.isclose(out[2, 11 + 3], want, rtol=1e-13)

    def loss(x=x, W=W, b=b):
        return (ob.linear_forward(irr_in, irr_out, act, x, W, b, res) * G).sum()
    got = ob.linear_backward(irr_in, irr_out, act, x, W, b, G)
    for name, v, g in zip(("x", "W", "b"), (x, W, b), got):
        assert np.allclose(g, difference(lambda t: loss(**{name: t}), v.copy()), atol=2e-8), name
    assert not got[0][:, 9:19].any()                              # 2e has no partner
    R = rotation(rng)
    turned = ob.linear_forward(irr_in, irr_out, act, rotated(irr_in, R, x), W, b, rotated(irr_out, R, res))
    assert np.allclose(turned, rotated(irr_out, R, out), atol=1e-12)


def test_slope_of_tanh_far_out():
    """1/cosh^2, down to where it is no longer a normal number."""
    z = np.array([-354, -320.5, -300, -17, 0, 3, 299, 310, 354, 400, 1e6])
    value, slope = ob.activation("tanh", z)
    want = np.array([0.0 if abs(v) > 355 else 1 / math.cosh(v) ** 2 for v in z])
    assert np.array_equal(value, np.tanh(z)) and np.allclose(slope, want, rtol=1e-13, atol=0)

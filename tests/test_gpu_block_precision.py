"""The feed-forward block's operators where the general bounds of
test_gpu_block.py are too wide to tell, against the fp64 oracle, and calls that
the binding does not make.  eps is the unit roundoff of the data type (2^-24,
2^-53)."""

import ctypes

import numpy as np
import pytest

from oracle import block as ob
from oracle.node import segments
from test_gpu_block import TOL, block_inputs, check_gated, features, host, log, shifted
from test_gpu_node import EPS, NP, dev, node, within  # noqa: F401  (node is a fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- linear map, C callers
@pytest.mark.parametrize("dt,irr_in,irr_out,place", [
    ("f32", "4x0e+4x1o", "4x0e+4x1o", dev), ("f32", "32x0e+8x1o+4x2e", "32x0e+16x1o+4x2e", dev),
    ("f32", "64x0e+36x1o+4x3o", "60x0e+64x1o+8x3o", dev), ("f32", "64x0e+36x1o+4x3o", "60x0e+64x1o+8x3o", shifted),
    ("f32", "65x0e+33x4e", "70x4e+130x0e", dev), ("f64", "4x0e+4x1o", "4x0e+4x1o", dev)])
def test_linear_parameters_without_weights(node, dt, irr_in, irr_out, place):  # noqa: F811
    """With the identity, the parameters' gradients read no weights, and a C caller may give none."""
    import torch
    plan = node.tpconv_linear_plan(irr_in, irr_out, dtype=dt)
    for n in (1, 65, 3001):
        log(f"[block] linear without weights {dt} {irr_in} -> {irr_out} n={n} {place.__name__}")
        x, G, W = block_inputs(np.random.default_rng(n), dt, irr_in, irr_out, n)
        xd, Gd, Wd = place(x), place(G), dev(W)
        _, want_W, want_b = node.tpconv_linear_backward(plan, xd, Wd, None, Gd, need=(False, True, True))
        inputs = [(xd.data_ptr(), None, None)]
        if dt == "f32":
            kept = node.tpconv_pack8(irr_in, xd)
            inputs.append((None, kept.codes.data_ptr(), kept.scales.data_ptr()))
        held = node.tpconv_dense_workspace_bytes(plan, n)
        ws = torch.empty(max(held, 1), dtype=torch.uint8, device="cuda")
        for i, rows in enumerate(inputs):
            if i == 1:
                _, want_W, want_b = node.tpconv_linear_backward(plan, kept, Wd, None, Gd, need=(False, True, True))
            gW, gb = torch.full_like(want_W, 7.0), torch.full_like(want_b, 7.0)
            assert node._lib.tpconv_linear_backward(
                plan.handle, n, *rows, None, None, Gd.data_ptr(), None, gW.data_ptr(), gb.data_ptr(), ws.data_ptr(),
                held, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
            assert torch.equal(gW, want_W) and torch.equal(gb, want_b)


# ---------------------------------------------------------------- activations
def arguments(dt, act, slope, mul):
    """[n, mul] arguments over the range in which the result is a number in full precision: it reaches far down one
    side (both sides for a slope), to where that is subnormal or 0.  fp64: not beyond the exponential's range."""
    low = 102.0 if dt == "f32" else 700.0
    if slope and dt == "f32":
        low = 86.0                     # the gradient passes the matrix cores: normal numbers alone
    if act == "tanh":
        low /= 2
    return np.concatenate([np.linspace(-low, low, 16384 - 512), np.linspace(-2, 2, 512)]).reshape(-1, mul).astype(NP[dt])


def activation_bounds(dt, act, z):
    """Bounds of sigmoid, silu and their and tanh's slopes relative to their own size.  With e = e^-|z|, its hardware
    exponential and the factor with it are within 4 eps (a unit is up to 2), 1 + e within 3, its reciprocal within 5; so
    one sigmoid is within 5 and the other, times e, within 10; products and sums round once each.  What is formed of
    subnormal numbers is off by half of the least one for each product, once times z.  tanh's slope: 4 s t at 2 z."""
    e, least = EPS[dt], 2.0 ** (-149 if dt == "f32" else -1074)
    value, slope = ob.activation(act, z)
    s, t = ob.activation("sigmoid", z)[0], ob.activation("sigmoid", -z)[0]
    of_value = {"sigmoid": 10 * e * s, "silu": 11 * e * np.abs(value)}.get(act)
    of_slope = {"sigmoid": 16 * e * slope, "tanh": 16 * e * slope,
                "silu": 10 * e * s + 18 * e * np.abs(z) * s * t + e * np.abs(slope)}[act]
    tiny = 3 * least * (1 + np.abs(z))
    return value, slope, None if of_value is None else TOL[dt] * of_value + tiny, TOL[dt] * of_slope + tiny


@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("act", ["sigmoid", "silu", "tanh"])
def test_activations_relative_to_their_size(node, dt, act):  # noqa: F811
    """Where an activation or its slope saturates at 0, its small values are right too: linear maps with W = 1 (in the
    one-pass gradients and the other way), and gates."""
    for mul in (1, 4):
        irr = f"{mul}x0e"
        log(f"[block] {act} {dt} relative to its size, {mul} channels")
        W = dev(np.eye(mul, dtype=NP[dt]).reshape(-1))
        linear = node.tpconv_linear_plan(irr, irr, act, dt)
        z = arguments(dt, act, False, mul)
        value, _, bound, _ = activation_bounds(dt, act, z.astype(np.float64))
        if bound is not None:
            within(node.tpconv_linear_forward(linear, dev(z), W), value, bound, "value")
        z = arguments(dt, act, True, mul)
        _, slope, _, bound = activation_bounds(dt, act, z.astype(np.float64))
        got = node.tpconv_linear_backward(linear, dev(z), W, None, dev(np.ones_like(z)), need=(True, False, False))[0]
        within(got, slope, bound, "slope")
        # gates of 0e: channels 0 .. mul are the arguments, the next is 1 and every product's row
        wide = f"{2 * mul}x0e"
        gated = node.tpconv_gated_plan(wide, irr, scalar_act=act, dtype=dt)
        M, Wg = np.zeros((2 * mul, mul), NP[dt]), np.zeros((2 * mul, mul), NP[dt])
        M[mul] = 1
        Wg[:mul] = np.eye(mul)
        one = np.ones_like(z)
        got = node.tpconv_gated_backward(gated, dev(np.concatenate([z, one], 1)), dev(M.reshape(-1)), dev(Wg), None,
                                         dev(one), need=(True, False, False, False))[0]
        within(host(got)[:, :mul], slope, bound, "gate's slope")
        z = arguments(dt, act, False, mul)
        value, _, bound, _ = activation_bounds(dt, act, z.astype(np.float64))
        if bound is not None:
            x = dev(np.concatenate([z, np.ones_like(z)], 1))
            within(node.tpconv_gated_forward(gated, x, dev(M.reshape(-1)), dev(Wg)), value, bound, "gate's value")


# ----------------------------------------------------------------------- norm
@pytest.mark.parametrize("scope", ["segment", "row"])
@pytest.mark.parametrize("irreps", ["1x0e", "2x0e", "1x0e+6x0e+3x1o", "1x1o+4x0e", "64x0e+64x1o+64x2e+64x3o", "1000x1o+1x0e",
                                    "8192x0e"])
def test_norm_gradient_is_rounded_once(node, irreps, scope):  # noqa: F811
    """fp32 grad_x is formed in 64 bits and rounded once, so it is within eps of itself however much of its two terms
    cancels (in a segment of one column all but what eps leaves), and (8 width + 256) 2^-53 of these: a sum over
    `width` columns is off by width 2^-53 of its absolute values, r by half that of the mean square, and each enters up
    to three times, in the oracle as in the kernel."""
    e, width = EPS["f32"], segments(irreps)[1]
    for n, scale in ((1, 1.0), (37, 1.0), (37, 1e18), (37, 1e-3), (700, 1.0)):
        for more in (False, True):
            log(f"[block] norm gradient {irreps} {scope} n={n} scale {scale} {more}")
            rng = np.random.default_rng([n, width, more])
            h, G, H = ((s * features(rng, irreps, n, "f32")).astype(np.float32) for s in (scale, 1, 1e-3))
            gamma = rng.standard_normal(ob.channels(irreps)[1]).astype(np.float32)
            plan = node.tpconv_norm_plan(irreps, scope=scope, eps=1e-6)
            args = (h, gamma, G, H if more else None)
            gx = node.tpconv_norm_backward(plan, *(None if a is None else dev(a) for a in args), need=(True, False))[0]
            want = ob.norm_backward(irreps, scope, 1e-6, *args)[0]
            size = ob.norm_backward(irreps, scope, 1e-6, *args, size=True)[0]
            within(gx, want, e * np.abs(want) + (8 * width + 256) * 2.0 ** -53 * size + 2.0 ** -149, "grad_x")


def rounded_to_fp32(y, apart):
    """y in fp32, and where that is certain of a y that is off by `apart` of itself: not next to the middle of two fp32
    numbers, and a number in full precision."""
    down, up = (np.abs(y) * (1 + s * apart) for s in (-1, 1))
    sure = (down.astype(np.float32) == up.astype(np.float32)) & (np.abs(y) > 2.0 ** -120)
    return y.astype(np.float32), sure | (y == 0)


@pytest.mark.parametrize("scope", ["segment", "row"])
@pytest.mark.parametrize("irreps", ["1x0e", "3x0e+1x1o+2x2e", "32x0e+32x1o+32x2e+32x3o", "64x0e+64x1o+64x2e+64x3o",
                                    "1000x1o+1x0e"])
def test_norm_is_rounded_once(node, irreps, scope):  # noqa: F811
    """The fp32 norm is that of 64 bits, rounded once, and its codes are those of the definition: bit by bit, but for
    what lies within (4 width + 64) 2^-53 of the middle of two fp32 numbers, and the segments that hold such a value
    (at the widest, up to 4.5e-5 of the values and 13 % of the segments of 3000 columns)."""
    width = segments(irreps)[1]
    plan = node.tpconv_norm_plan(irreps, scope=scope, eps=1e-6)
    for n in (1, 333, 4096):
        log(f"[block] norm rounded once {irreps} {scope} n={n}")
        rng = np.random.default_rng([n, width])
        x, res = features(rng, irreps, n, "f32"), features(rng, irreps, n, "f32")
        gamma = (1 + 0.3 * rng.standard_normal(plan.channels)).astype(np.float32)
        y, h, p = node.tpconv_norm_forward(plan, dev(x), dev(res), dev(gamma), need=(True, True, True))
        want, sure = rounded_to_fp32(ob.norm_forward(irreps, scope, 1e-6, host(h), None, gamma)[0],
                                     (4 * width + 64) * 2.0 ** -53)
        assert sure.mean() > 0.999
        assert np.array_equal(y.cpu().numpy()[sure], want[sure])
        codes, scales = ob.pack8(irreps, want)
        for i, s in enumerate(segments(irreps)[0]):
            cols = slice(s[3], s[3] + s[0] * (2 * s[1] + 1))
            rows = sure[:, cols].all(1)
            assert rows.mean() > 0.8 or n == 1
            assert np.array_equal(p.scales.cpu().numpy()[rows, i], scales[rows, i])
            assert np.array_equal(p.codes.cpu().numpy()[rows, cols], codes[rows, cols])


# ---------------------------------------------------- few channels, many gates
@pytest.mark.parametrize("dt", ["f32", "f64"])
@pytest.mark.parametrize("irr_in,irr_out", [
    ("16x0e+16x1o+16x2e+16x3o", "16x0e+64x1o+64x2e+64x3o"), ("8x0e+8x1o", "64x1o+8x0e"), ("1x0e+16x1o", "300x1o"),
    ("32x0e+16x1o", "16x1o+500x0e")])
def test_many_gates(node, dt, irr_in, irr_out):  # noqa: F811
    """The even scalars' gradient, a product over many more gates than it has channels."""
    for n in (1, 65, 333):
        log(f"[block] many gates {dt} {irr_in} -> {irr_out} n={n}")
        check_gated(node, dt, irr_in, irr_out, n)

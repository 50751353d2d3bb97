"""Host-side checks of the feed-forward block's C entry points (CPU only: no
kernel is launched): plans, workspace sizes, and every refusal."""

import ctypes
import os

import pytest

from oracle import block as ob
from oracle.node import segments

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "equivariant_mlip_tensor_amd", "libtpconv.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libtpconv.so not built")

OK, INVALID, IRREPS, UNSUPPORTED, NO_PATHS, WORKSPACE = 0, 1, 2, 3, 4, 5
PTR = ctypes.c_void_p(256)          # never read: every call here returns before a launch
ODD = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def node():
    from equivariant_mlip_tensor_amd import node
    return node


def test_norm_plan(node):
    plan = node.tpconv_norm_plan("4x0e+3x1o+2x1o", scope="row", eps=1e-5, dtype="f64")
    assert (plan.dim, plan.channels, plan.n_segments, plan.scope, plan.dtype, plan.eps) == (19, 9, 3, 1, 1, 1e-5)
    assert node.tpconv_norm_workspace_bytes(plan, 1000) >= 8 * 19
    assert node.tpconv_norm_workspace_bytes(plan, -1) == 0 and node.tpconv_norm_workspace_bytes(plan, 1 << 31) == 0
    with pytest.raises(ValueError):
        node.tpconv_norm_plan("4x0e", scope="column")


@pytest.mark.parametrize("irreps,scope,eps,dt,status", [
    ("4x0z", 0, 1e-6, 0, IRREPS), ("", 0, 1e-6, 0, IRREPS), ("4x5e", 0, 1e-6, 0, UNSUPPORTED),
    ("+".join(["1x0e"] * 33), 0, 1e-6, 0, UNSUPPORTED), ("8193x0e", 0, 1e-6, 0, UNSUPPORTED),
    ("2000x2e", 0, 1e-6, 0, UNSUPPORTED), ("16777216x4e", 0, 1e-6, 0, UNSUPPORTED), ("4x0e", 2, 1e-6, 0, INVALID),
    ("4x0e", -1, 1e-6, 0, INVALID), ("4x0e", 0, 0.0, 0, INVALID), ("4x0e", 0, -1.0, 0, INVALID), ("4x0e", 0, 1e-40, 0, INVALID),
    ("4x0e", 0, float("inf"), 0, INVALID), ("4x0e", 0, float("nan"), 0, INVALID), ("4x0e", 0, 1e-6, 2, INVALID)])
def test_norm_plan_errors(node, irreps, scope, eps, dt, status):
    h = ctypes.c_void_p()
    assert node._lib.tpconv_norm_plan(irreps.encode(), scope, eps, dt, ctypes.byref(h)) == status
    assert not h.value and node._lib.tpconv_last_error()


def test_norm_refusals(node):
    lib, h = node._lib, ctypes.c_void_p()
    assert lib.tpconv_norm_plan(None, 0, 1e-6, 0, ctypes.byref(h)) == INVALID
    assert lib.tpconv_norm_plan(b"4x0e", 0, 1e-6, 0, None) == INVALID
    assert lib.tpconv_norm_query(None, ctypes.byref(node.NormInfo())) == INVALID
    assert lib.tpconv_norm_workspace_bytes(None, 4) == 0
    lib.tpconv_norm_destroy(None)
    p32, p64 = node.tpconv_norm_plan("4x0e+2x1o"), node.tpconv_norm_plan("4x0e+2x1o", dtype="f64")

    def fwd(plan=p32.handle, n=4, x=PTR, res=PTR, gamma=PTR, s=PTR, out=PTR, codes=None, scales=None):
        return lib.tpconv_norm_forward(plan, n, x, res, gamma, s, out, codes, scales, None)
    for kw in (dict(plan=None), dict(n=-1), dict(n=1 << 31), dict(x=None), dict(s=None, out=None),
               dict(codes=PTR), dict(scales=PTR), dict(plan=p64.handle, codes=PTR, scales=PTR)):
        assert fwd(**kw) == INVALID, kw
    assert fwd(n=0, x=None, s=None, out=None) == OK

    def bwd(plan=p32.handle, n=4, rows=PTR, g=PTR, gx=PTR, gg=PTR, ws=PTR, held=1 << 40):
        return lib.tpconv_norm_backward(plan, n, rows, None, g, None, gx, gg, ws, held, None)
    for kw in (dict(plan=None), dict(n=-1), dict(n=1 << 31), dict(rows=None), dict(g=None)):
        assert bwd(**kw) == INVALID, kw
    assert lib.tpconv_norm_workspace_bytes(p32.handle, 4) == 0                    # a block's rows need none
    assert bwd(n=4000, ws=None) == WORKSPACE and bwd(n=4000, ws=ODD) == WORKSPACE
    assert bwd(n=4000, held=lib.tpconv_norm_workspace_bytes(p32.handle, 4000) - 1) == WORKSPACE
    assert bwd(gx=None, gg=None) == OK and bwd(n=0, gg=None, rows=None, g=None) == OK


def test_pack8_refusals(node):
    lib = node._lib

    def calls(irr=b"4x0e+2x1o", n=4, dim=10, a=PTR, b=PTR, c=PTR):
        return lib.tpconv_pack8(irr, n, dim, a, b, c, None), lib.tpconv_unpack8(irr, n, dim, a, b, c, None)
    for kw in (dict(irr=None), dict(n=-1), dict(n=1 << 31), dict(dim=9), dict(dim=11), dict(a=None), dict(b=None),
               dict(c=None)):
        assert calls(**kw) == (INVALID, INVALID), kw
    assert calls(irr=b"4x0z") == (IRREPS, IRREPS)
    assert calls(irr=b"2x5e", dim=22) == (UNSUPPORTED, UNSUPPORTED)
    assert calls(irr=b"8200x0e", dim=8200) == (UNSUPPORTED, UNSUPPORTED)
    assert calls(n=0, a=None, b=None, c=None) == (OK, OK)


@pytest.mark.parametrize("irr_in,irr_out", [
    ("4x0e+4x1o", "4x0e+4x1o"), ("3x1o+5x0e+2x2e", "7x2e+4x1o"), ("1024x0e", "1x0e"), ("2x0e+1x4e", "2x4e + 3x0e")])
def test_dense_plans(node, irr_in, irr_out):
    maps, numel = ob.maps(irr_in, irr_out)
    C = ob.channels(irr_out)[1]
    for plan in (node.tpconv_gated_plan(irr_in, irr_out, dtype="f64"), node.tpconv_linear_plan(irr_in, irr_out)):
        assert (plan.dim_in, plan.dim_out) == (segments(irr_in)[1], segments(irr_out)[1])
        assert plan.weight_numel == numel and plan.n_maps == len(maps)
        assert plan.n_segments_in == irr_in.count("+") + 1
        assert [(m[2], m[3]) for m in node.tpconv_dense_maps(plan)] == [(s[1], at) for s, _, at in maps]
        assert node.tpconv_dense_workspace_bytes(plan, -1) == 0
        assert node.tpconv_dense_workspace_bytes(plan, 1 << 31) == 0
    gated, linear = node.tpconv_gated_plan(irr_in, irr_out), node.tpconv_linear_plan(irr_in, irr_out)
    assert (gated.n_gates, gated.n_scalars, gated.n_bias) == (C, ob.even_scalars(irr_in)[0], C)
    even = ob.even_scalars(irr_out)
    assert (linear.n_gates, linear.n_scalars, linear.n_bias) == (0, 0, even[0] if even else 0)


@pytest.mark.parametrize("irr_in,irr_out,act,gate,dt,status", [
    ("4x1q", "4x1o", 1, 2, 0, IRREPS), ("4x0e", "", 1, 2, 0, IRREPS), ("4x0e+4x5e", "4x5e", 1, 2, 0, UNSUPPORTED),
    ("1025x0e", "1x0e", 1, 2, 0, UNSUPPORTED), ("4x0e+2x0e", "4x0e", 1, 2, 0, UNSUPPORTED),
    ("4x0e+4x1o", "4x1e", 1, 2, 0, NO_PATHS), ("4x0e", "4x0e+1x1o", 1, 2, 0, NO_PATHS),
    ("4x0e", "4x0e", 5, 2, 0, INVALID), ("4x0e", "4x0e", -1, 2, 0, INVALID), ("4x0e", "4x0e", 1, 2, 7, INVALID)])
def test_dense_plan_errors(node, irr_in, irr_out, act, gate, dt, status):
    lib = node._lib
    for call in (lambda h: lib.tpconv_gated_plan(irr_in.encode(), irr_out.encode(), act, gate, dt, h),
                 lambda h: lib.tpconv_linear_plan(irr_in.encode(), irr_out.encode(), act, dt, h)):
        h = ctypes.c_void_p()
        assert call(ctypes.byref(h)) == status
        assert not h.value and lib.tpconv_last_error()


def test_gated_needs_even_scalars_and_a_known_gate(node):
    lib, h = node._lib, ctypes.c_void_p()
    assert lib.tpconv_gated_plan(b"4x1o+2x0o", b"4x1o", 1, 2, 0, ctypes.byref(h)) == NO_PATHS
    assert lib.tpconv_gated_plan(b"4x0e", b"4x0e", 1, 9, 0, ctypes.byref(h)) == INVALID
    assert lib.tpconv_linear_plan(b"4x1o+2x0o", b"4x1o", 1, 0, ctypes.byref(h)) == OK
    lib.tpconv_dense_destroy(h)
    for kw in (dict(scalar_act="relu"), dict(gate_act="relu")):
        with pytest.raises(ValueError):
            node.tpconv_gated_plan("4x0e", "4x0e", **kw)
    with pytest.raises(ValueError):
        node.tpconv_linear_plan("4x0e", "4x0e", act="relu")


def test_dense_refusals(node):
    lib, big = node._lib, 1 << 40
    gated, linear = node.tpconv_gated_plan("4x0e+2x1o", "4x0e+2x1o"), node.tpconv_linear_plan("4x0e", "4x0e", act="silu")
    plain, g64 = node.tpconv_linear_plan("4x0e", "4x0e"), node.tpconv_gated_plan("4x0e", "4x0e", dtype="f64")
    assert lib.tpconv_dense_query(None, ctypes.byref(node.DenseInfo())) == INVALID
    assert lib.tpconv_dense_maps(None, None) == INVALID and lib.tpconv_dense_workspace_bytes(None, 4) == 0
    lib.tpconv_dense_destroy(None)

    def gf(plan=gated.handle, n=4, x=PTR, w=PTR, wg=PTR, b=PTR, out=PTR):
        return lib.tpconv_gated_forward(plan, n, x, w, wg, b, out, None)

    def lf(plan=linear.handle, n=4, x=PTR, w=PTR, b=PTR, r=PTR, out=PTR):
        return lib.tpconv_linear_forward(plan, n, x, w, b, r, out, None)
    for f in (gf, lf):
        for kw in (dict(plan=None), dict(n=-1), dict(n=1 << 31), dict(x=None), dict(w=None), dict(out=None)):
            assert f(**kw) == INVALID, (f, kw)
        assert f(n=0, x=None, w=None, out=None) == OK
    assert gf(wg=None) == INVALID
    assert gf(plan=linear.handle) == INVALID and lf(plan=gated.handle) == INVALID      # the other kind's plan

    def gb(plan=gated.handle, n=4, x=PTR, c=None, s=None, w=PTR, wg=PTR, G=PTR, outs=(PTR,) * 4, ws=PTR, held=big):
        return lib.tpconv_gated_backward(plan, n, x, c, s, w, wg, None, G, *outs, ws, held, None)

    def lb(plan=linear.handle, n=4, x=PTR, c=None, s=None, w=PTR, G=PTR, outs=(PTR,) * 3, ws=PTR, held=big):
        return lib.tpconv_linear_backward(plan, n, x, c, s, w, None, G, *outs, ws, held, None)
    for f in (gb, lb):
        for kw in (dict(plan=None), dict(n=-1), dict(n=1 << 31), dict(x=None), dict(w=None), dict(G=None),
                   dict(c=PTR), dict(s=PTR), dict(c=PTR, s=PTR), dict(x=None, c=PTR), dict(x=None, s=PTR)):
            assert f(**kw) == INVALID, (f, kw)
        assert f(ws=None) == WORKSPACE and f(ws=ODD) == WORKSPACE
    assert gb(wg=None) == INVALID and gb(plan=linear.handle) == INVALID and lb(plan=gated.handle) == INVALID
    assert gb(plan=g64.handle, x=None, c=PTR, s=PTR) == INVALID                        # 8 bits of fp32 rows alone
    assert gb(held=lib.tpconv_dense_workspace_bytes(gated.handle, 4) - 1) == WORKSPACE
    assert lb(held=lib.tpconv_dense_workspace_bytes(linear.handle, 4) - 1) == WORKSPACE
    assert gb(outs=(None,) * 4) == OK and lb(outs=(None,) * 3) == OK
    # with the identity, grad_x alone needs neither x nor a workspace, the parameters' gradients need x
    assert lb(plan=plain.handle, n=4, x=None, outs=(None, PTR, None)) == INVALID
    assert lb(plan=plain.handle, n=4, x=None, outs=(None, None, PTR)) == INVALID
    assert lb(plan=plain.handle, n=4, x=None, w=None, outs=(PTR, None, None)) == INVALID


def test_sizes_past_every_grid(node):
    """Plans with the most maps and channels, and the most rows: sizes in 64 bits, found at once."""
    import time
    wide = "+".join(f"1024x{l}{p}" for l in range(5) for p in "eo")
    for dt, size in (("f32", 4), ("f64", 8)):
        gated, linear = node.tpconv_gated_plan(wide, wide, dtype=dt), node.tpconv_linear_plan(wide, wide, "silu", dtype=dt)
        assert gated.weight_numel == linear.weight_numel == 10 << 20 and gated.n_gates == 10240
        for n in ((1 << 31) - 1, 1 << 20, 1):
            begin = time.perf_counter()
            held = node.tpconv_dense_workspace_bytes(gated, n)
            assert held >= size * n * (gated.dim_out + gated.n_gates)
            assert node.tpconv_dense_workspace_bytes(linear, n) >= size * n * linear.n_bias
            assert time.perf_counter() - begin < 0.05
        norm = node.tpconv_norm_plan("8192x0e", dtype=dt)
        assert 0 < node.tpconv_norm_workspace_bytes(norm, (1 << 31) - 1) < 1 << 28


def test_dense_workspace_is_bounded(node):
    """The rows and gates of grad_out, and parts of the parameters' gradients: some 20 MB or the parameters."""
    for dt, size in (("f32", 4), ("f64", 8)):
        for irr_in, irr_out in (("64x0e+64x1o+64x2e+64x3o",) * 2, ("1x0e", "1x0e"), ("1024x0e", "1024x0e"),
                                ("1024x0e+1024x4e", "1024x0e+1024x4e"), ("16x0e+16x4e", "200x0e+200x4e")):
            gated = node.tpconv_gated_plan(irr_in, irr_out, dtype=dt)
            linear = node.tpconv_linear_plan(irr_in, irr_out, act="silu", dtype=dt)
            for n in (0, 1, 17, 2048, 28000, 214648, 1000003):
                params = gated.weight_numel + (gated.n_scalars + 1) * gated.n_gates
                parts = max(64 << 20, 5 * size * params)
                rows = size * n * (gated.dim_out + gated.n_gates)
                assert node.tpconv_dense_workspace_bytes(gated, n) <= rows + parts, (dt, irr_in, n)
                assert node.tpconv_dense_workspace_bytes(linear, n) <= size * n * linear.n_bias + parts

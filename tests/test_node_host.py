"""Host-side checks of the node operators' C entry points (CPU only: no kernel
is launched): the header's exports, the experts' plan, and every refusal."""

import ctypes
import os
import re

import pytest

from oracle import node as on

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "equivariant_mlip_tensor_amd", "libtpconv.so")
HEADER = os.path.join(ROOT, "include", "tpconv_node.h")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libtpconv.so not built")

OK, INVALID, IRREPS, UNSUPPORTED, NO_PATHS, WORKSPACE = 0, 1, 2, 3, 4, 5
PTR = ctypes.c_void_p(256)          # never read: every call here returns before a launch


@pytest.fixture(scope="module")
def node():
    from equivariant_mlip_tensor_amd import node
    return node


def test_exports_every_declared_symbol(node):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(tpconv_[a-z0-9_]+)\s*\(", text)))
    assert sorted(node.NODE_EXPORTS) == declared
    lib = ctypes.CDLL(LIB)
    for name in declared:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("irr_in,irr_out", [
    ("4x0e+4x1o", "4x0e+4x1o"), ("3x1o+5x0e+2x2e", "7x2e+1x1e+4x1o"), ("256x0e", "1x0e"), ("1x4e", "2x4e + 3x0o")])
def test_plan_matches_oracle(node, irr_in, irr_out):
    plan = node.tpconv_experts_plan(irr_in, irr_out, 5, 2, "f64")
    maps, numel = on.expert_maps(irr_in, irr_out)
    assert (plan.dim_in, plan.dim_out) == (on.segments(irr_in)[1], on.segments(irr_out)[1])
    assert plan.weight_numel == numel and plan.n_maps == len(maps)
    assert [(m[2], m[3]) for m in node.tpconv_experts_maps(plan)] == [((m[4] - 1) // 2, m[5]) for m in maps]
    assert (plan.n_experts, plan.top_k, plan.dtype) == (5, 2, 1)
    assert node.tpconv_experts_layout_bytes(plan, -1) == 0
    assert node.tpconv_experts_layout_bytes(plan, 1 << 31) == 0
    assert node.tpconv_experts_workspace_bytes(plan, -1) == 0


@pytest.mark.parametrize("irr_in,irr_out,X,k,dt,status", [
    ("4x1q", "4x1o", 2, 1, 0, IRREPS), ("4x1o", "", 2, 1, 0, IRREPS), ("0x1o", "1x1o", 2, 1, 0, IRREPS),
    ("4x5e", "4x5e", 2, 1, 0, UNSUPPORTED), ("257x0e", "1x0e", 2, 1, 0, UNSUPPORTED),
    ("4x1o+2x1o", "4x1o", 2, 1, 0, UNSUPPORTED), ("4x1o", "4x1e", 2, 1, 0, NO_PATHS),
    ("4x1o", "4x1o", 0, 1, 0, INVALID), ("4x1o", "4x1o", 2, 0, 0, INVALID), ("4x1o", "4x1o", 257, 1, 0, UNSUPPORTED),
    ("4x1o", "4x1o", 16, 9, 0, UNSUPPORTED), ("4x1o", "4x1o", 2, 1, 5, INVALID)])
def test_plan_errors(node, irr_in, irr_out, X, k, dt, status):
    h = ctypes.c_void_p()
    assert node._lib.tpconv_experts_plan(irr_in.encode(), irr_out.encode(), X, k, dt, ctypes.byref(h)) == status
    assert not h.value and node._lib.tpconv_last_error()


def test_null_handles(node):
    lib, h, info = node._lib, ctypes.c_void_p(), node.ExpertsInfo()
    assert lib.tpconv_experts_plan(None, b"1x0e", 2, 1, 0, ctypes.byref(h)) == INVALID
    assert lib.tpconv_experts_plan(b"1x0e", None, 2, 1, 0, ctypes.byref(h)) == INVALID
    assert lib.tpconv_experts_plan(b"1x0e", b"1x0e", 2, 1, 0, None) == INVALID
    assert lib.tpconv_experts_query(None, ctypes.byref(info)) == INVALID
    assert lib.tpconv_experts_maps(None, None) == INVALID
    assert lib.tpconv_experts_layout_bytes(None, 4) == 0 and lib.tpconv_experts_workspace_bytes(None, 4) == 0
    assert lib.tpconv_experts_layout(None, 0, None, None, 0, None, None) == INVALID
    assert lib.tpconv_experts_forward(None, 0, *([None] * 7)) == INVALID
    assert lib.tpconv_experts_backward(None, 0, *([None] * 10), 0, None) == INVALID
    lib.tpconv_experts_destroy(None)


def test_experts_refusals(node):
    lib, plan = node._lib, node.tpconv_experts_plan("4x0e", "4x0e", 3, 2, "f32")
    h = plan.handle
    assert lib.tpconv_experts_forward(h, -1, *([PTR] * 6), None) == INVALID
    assert lib.tpconv_experts_forward(h, 1 << 30, *([PTR] * 6), None) == INVALID       # rows * top_k = 2^31
    for missing in (0, 1, 2, 3, 5):                                                    # layout (4) may be NULL
        args = [PTR] * 6
        args[missing] = None
        assert lib.tpconv_experts_forward(h, 4, *args, None) == INVALID, missing
    assert lib.tpconv_experts_forward(h, 4, PTR, PTR, PTR, PTR, ctypes.c_void_p(264), PTR, None) == INVALID
    assert lib.tpconv_experts_forward(h, 0, *([None] * 6), None) == OK
    big = 1 << 40
    need = lib.tpconv_experts_layout_bytes(h, 4)
    assert lib.tpconv_experts_layout(h, 4, None, PTR, big, None, None) == INVALID
    assert lib.tpconv_experts_layout(h, 4, PTR, ctypes.c_void_p(264), big, None, None) == WORKSPACE
    assert lib.tpconv_experts_layout(h, 4, PTR, PTR, need - 1, None, None) == WORKSPACE
    assert lib.tpconv_experts_layout(h, 4, PTR, None, big, None, None) == WORKSPACE

    def backward(x=PTR, w=PTR, e=PTR, g=PTR, lay=PTR, G=PTR, gx=PTR, gw=PTR, gg=PTR, ws=PTR, held=big):
        return lib.tpconv_experts_backward(h, 4, x, w, e, g, lay, G, gx, gw, gg, ws, held, None)
    assert backward(gx=None, gw=None, gg=None) == OK
    for kw in (dict(e=None), dict(g=None), dict(G=None), dict(w=None), dict(x=None), dict(lay=None),
               dict(lay=ctypes.c_void_p(264))):
        assert backward(**kw) == INVALID, kw
    assert backward(ws=None) == WORKSPACE
    assert backward(held=lib.tpconv_experts_workspace_bytes(h, 4) - 1) == WORKSPACE
    assert backward(ws=ctypes.c_void_p(264)) == WORKSPACE


def test_embedding_refusals(node):
    lib = node._lib

    def fwd(dt=0, n=4, v=3, d=2, types=PTR, table=PTR, out=PTR, stride=2):
        return lib.tpconv_embedding_forward(dt, n, v, d, types, table, 1.0, out, stride, None)

    def bwd(dt=0, n=4, v=3, d=2, types=PTR, grad=PTR, stride=2, gt=PTR, ws=PTR, held=1 << 40):
        return lib.tpconv_embedding_backward(dt, n, v, d, types, grad, stride, 1.0, gt, ws, held, None)
    for f in (fwd, bwd):
        for kw in (dict(dt=2), dict(n=-1), dict(v=-1), dict(n=1 << 31), dict(v=1 << 31), dict(d=0), dict(stride=1),
                   dict(types=None)):
            assert f(**kw) == INVALID, (f, kw)
    assert fwd(table=None) == INVALID and fwd(out=None) == INVALID
    assert bwd(grad=None) == INVALID and bwd(gt=None) == INVALID
    assert bwd(ws=ctypes.c_void_p(264)) == WORKSPACE
    need = lib.tpconv_embedding_workspace_bytes(0, 4000, 3, 2)
    assert bwd(n=4000, held=need - 1) == WORKSPACE and bwd(n=4000, ws=None) == WORKSPACE
    assert fwd(n=0, types=None, out=None) == OK and bwd(v=0, gt=None) == OK
    for bad in ((2, 4, 3, 2), (0, -1, 3, 2), (0, 4, -1, 2), (0, 4, 3, 0)):
        assert lib.tpconv_embedding_workspace_bytes(*bad) == 0


def test_routing_refusals(node):
    lib = node._lib

    def calls(dt=0, n=4, a=PTR, b=PTR, c=PTR, d=PTR, cfg=True, **kw):
        v = dict(n_experts=8, top_k=2, n_groups=1, top_groups=1, score=0, renormalise=1, scale=1.0)
        v.update(kw)
        s = ctypes.byref(node._RouteConfig(*v.values())) if cfg else None
        return (lib.tpconv_route_forward(dt, n, s, a, None, b, c, None),
                lib.tpconv_route_backward(dt, n, s, a, b, c, d, None))
    for kw in (dict(cfg=False), dict(dt=3), dict(n=-1), dict(n=1 << 31), dict(n_experts=0), dict(top_k=0),
               dict(n_groups=0), dict(top_groups=0), dict(n_groups=3), dict(top_groups=2),
               dict(top_k=3, n_groups=8, top_groups=2), dict(score=2), dict(renormalise=2),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(a=None), dict(b=None), dict(c=None),
               dict(n_experts=4, top_k=5)):
        assert calls(**kw) == (INVALID, INVALID), kw
    assert calls(d=None)[1] == INVALID
    for kw in (dict(n_experts=512), dict(n_experts=16, top_k=9), dict(n_experts=128, n_groups=128, top_groups=4)):
        assert calls(**kw) == (UNSUPPORTED, UNSUPPORTED), kw
    assert calls(n=0, a=None, b=None, c=None, d=None) == (OK, OK)
    with pytest.raises(ValueError):
        node.RouteConfig(8, 2, score="tanh")


def test_dropout_refusals(node):
    lib = node._lib

    def calls(irr=b"4x0e+2x1o", dt=0, n=4, dim=10, p=0.5, x=PTR, out=PTR):
        return (lib.tpconv_dropout_forward(irr, dt, n, dim, p, 1, 2, x, None, out, None),
                lib.tpconv_dropout_backward(irr, dt, n, dim, p, 1, 2, x, out, None))
    for kw in (dict(irr=None), dict(dt=2), dict(n=-1), dict(n=1 << 31), dict(dim=9), dict(p=1.0), dict(p=-0.1),
               dict(p=float("nan")), dict(x=None), dict(out=None)):
        assert calls(**kw) == (INVALID, INVALID), kw
    assert calls(irr=b"4x0z") == (IRREPS, IRREPS)
    assert calls(irr=b"4x5e", dim=44) == (UNSUPPORTED, UNSUPPORTED)
    assert calls(irr=b"+".join([b"1x0e"] * 33), dim=33) == (UNSUPPORTED, UNSUPPORTED)
    assert calls(irr=b"16777216x0e", dim=1 << 24) == (UNSUPPORTED, UNSUPPORTED)
    assert calls(n=0, x=None, out=None) == (OK, OK)


def test_row_counts_whose_entries_pass_64_bits(node):
    """Rows times top_k is compared, not formed: 2^61 rows of 8 entries would wrap to none."""
    lib = node._lib
    for k in (1, 2, 7, 8):
        plan = node.tpconv_experts_plan("4x0e", "4x0e", 16, k, "f32")
        h = plan.handle
        most = ((1 << 31) - 1) // k
        assert lib.tpconv_experts_layout_bytes(h, most) > 0 and lib.tpconv_experts_workspace_bytes(h, most) > 0
        for n in (most + 1, 1 << 31, 1 << 61, (1 << 61) + 1, min((1 << 64) // k + 1, (1 << 63) - 1), (1 << 63) - 1):
            assert lib.tpconv_experts_layout_bytes(h, n) == 0, (k, n)
            assert lib.tpconv_experts_workspace_bytes(h, n) == 0, (k, n)
            for status in (lib.tpconv_experts_forward(h, n, *([None] * 7)),
                           lib.tpconv_experts_layout(h, n, None, None, 0, None, None),
                           lib.tpconv_experts_backward(h, n, *([None] * 10), 0, None)):
                assert status == INVALID and b"rows times top_k" in lib.tpconv_last_error(), (k, n)


def test_workspace_is_bounded_by_the_entries(node):
    """The parts of the weights' gradient: a few for each hundred entries, however many the experts are."""
    lib = node._lib
    for dt, size in (("f32", 4), ("f64", 8)):
        for irr in ("16x0e", "64x0e+64x1o+64x2e+64x3o", "256x4e"):
            for X, k in ((1, 1), (16, 2), (64, 4), (200, 7), (256, 1), (256, 2), (256, 8)):
                plan = node.tpconv_experts_plan(irr, irr, X, k, dt)
                for n in (1, 100, 2048, 2049, 4096, 28000, 32768, 131072, 1000003):
                    entries = n * k
                    parts = entries // (32 if entries * plan.n_maps > 131072 else 8) + X + 1
                    shares = sum((m // 16 + 1) for m in [int(t.split("x")[0]) for t in irr.split("+")]) * entries
                    bound = size * (parts * plan.weight_numel + shares) + 4096
                    assert lib.tpconv_experts_workspace_bytes(plan.handle, n) <= bound, (dt, irr, X, k, n)
    plan = node.tpconv_experts_plan("64x0e+64x1o+64x2e+64x3o", "64x0e+64x1o+64x2e+64x3o", 256, 8, "f32")
    assert lib.tpconv_experts_workspace_bytes(plan.handle, 32768) < 0.45e9     # x is 0.13 GB

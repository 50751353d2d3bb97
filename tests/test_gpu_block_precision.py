"""The feed-forward block's operators where the general bounds of
test_gpu_block.py are too wide to tell, and calls that the binding does not make."""

import ctypes

import numpy as np
import pytest

from test_gpu_block import block_inputs, log, shifted
from test_gpu_node import dev, node  # noqa: F401  (node is a fixture)

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

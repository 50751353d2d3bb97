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
from test_gpu_node import EPS, NP, check_experts, config, dev, node, within  # noqa: F401  (node is a fixture)

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

"""The mixture-of-experts layer of examples/moe_layer.py: its whole gradient
against differences, and a few steps of training.

fp64 on the 16-atom workload; the difference of the total along a direction,
step h = 1e-5, is off by its third derivative times h^2 / 6 plus eps / h times
the total's size: 1e-7 relative to the direction's and gradient's lengths holds
with room.  The step is too short to change a chosen expert (checked).
"""

import os
import sys

import pytest

import workloads

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import moe_layer
    finally:
        sys.path.pop(0)
    return moe_layer


def test_gradients_against_differences(example):
    import torch
    layer = example.MoELayer(workloads.WORKLOADS["tiny"], n_types=3, n_experts=4, top_k=2, p_drop=0.3)
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(like):
        d = torch.randn(like.shape, generator=g, device="cuda", dtype=like.dtype)
        return d / d.norm()

    cot = torch.randn(layer.n, generator=g, device="cuda", dtype=torch.float64)

    def total(params, vec=None):
        out = layer.forward(7, params=params, vec=vec)
        return float((cot * layer.energy(out)).sum()), layer.saved[7]

    _, chosen = total(layer.params)
    grad, g_pos = layer.backward(cot)
    h = 1e-5
    for name in ("table", "router", "weights", "readout"):
        d = normal(layer.params[name])
        sides = [total(dict(layer.params, **{name: layer.params[name] + s * h * d})) for s in (-1, 1)]
        assert all(torch.equal(c, chosen) for _, c in sides)
        num, got = (sides[1][0] - sides[0][0]) / (2 * h), float((grad[name] * d).sum())
        assert abs(num - got) < 1e-7 * (1 + float(grad[name].norm())), (name, num, got)
    # moving the atoms moves the edge vectors: vec = pos[src] - pos[dst]
    w = workloads.make_graph(layer.w)
    src, dst = (torch.from_numpy(w[k]).long().cuda() for k in ("src", "dst"))
    d = normal(torch.zeros((layer.n, 3), dtype=torch.float64, device="cuda"))
    sides = [total(layer.params, vec=layer.vec + s * h * (d[src] - d[dst])) for s in (-1, 1)]
    assert all(torch.equal(c, chosen) for _, c in sides)
    num, got = (sides[1][0] - sides[0][0]) / (2 * h), float((g_pos * d).sum())
    assert abs(got) > 1e-3 and abs(num - got) < 1e-7 * (1 + float(g_pos.norm())), ("positions", num, got)


def test_a_few_steps_of_training(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["moe_layer.py", "--workload", "c1k", "--steps", "11"])
    example.main()
    lines = [l for l in capsys.readouterr().out.splitlines() if l.startswith("step")]
    miss = [float(l.split("miss")[1].split()[0]) for l in lines]
    assert len(miss) == 3 and miss[-1] < miss[0]

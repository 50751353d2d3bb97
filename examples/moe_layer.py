"""One mixture-of-experts layer of an interatomic potential, trained for a few steps.

    python examples/moe_layer.py [--workload c1k] [--experts 8] [--top-k 2] [--steps 20]

Species embedding -> Clebsch-Gordan convolution (harmonics inside its kernels)
-> routing by the atoms' scalars -> the experts' equivariant maps -> dropout
onto the residual -> a second convolution -> a linear readout of the scalars:
energies, and forces from the gradient with respect to the positions.  Every
step but the two small dense products (router, readout) is a call of the
library; torch holds the tensors.  Inputs are synthetic (workloads/), the target a random
energy per atom.
"""

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import workloads  # noqa: E402
from equivariant_mlip_tensor_amd import node  # noqa: E402
from equivariant_mlip_tensor_amd import tpconv as tp  # noqa: E402


class MoELayer:
    """The layer's plans, parameters, forward and backward on one graph."""

    def __init__(self, w: workloads.Workload, n_types=4, n_experts=8, top_k=2, p_drop=0.1, seed=0):
        self.w, self.p_drop, self.seed = w, p_drop, seed
        self.plan = tp.tpconv_plan(w.irreps_in, w.sh_lmax, w.irreps_out, w.dtype)
        self.experts_plan = node.tpconv_experts_plan(w.irreps_out, w.irreps_out, n_experts, top_k, w.dtype)
        self.config = node.RouteConfig(n_experts, top_k)
        d = workloads.make_inputs(w, self.plan.n_paths, self.plan.weight_numel)
        dt, dev = self.plan.torch_dtype, "cuda"
        self.n, self.mul = d["n_nodes"], self.plan.mul          # the scalars are the first `mul` columns
        self.graph = tp.tpconv_graph_create(self.n, *(torch.from_numpy(d[k]).to(dev) for k in ("src", "dst")))
        self.vec = torch.from_numpy(d["vec"].astype(w.np_dtype)).to(dev)
        self.W = torch.from_numpy(np.ascontiguousarray(d["W"])).to(dev)     # the edges' path weights: inputs here
        g = torch.Generator(device=dev).manual_seed(seed)
        self.types = torch.randint(0, n_types, (self.n,), generator=g, device=dev).int()
        U, X = self.mul, n_experts

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=dev, dtype=dt)

        self.params = dict(table=normal(n_types, U), router=normal(U, X) / U ** 0.5,
                           weights=normal(X, self.experts_plan.weight_numel) / U ** 0.5,
                           readout=normal(U) / (U * self.n) ** 0.5)
        self.load = torch.zeros(X, dtype=torch.int32, device=dev)           # entries of each expert, this step

    def forward(self, step: int, params=None, vec=None):
        """The features after the second convolution [n, dim]; what the backward needs is kept in self.saved."""
        p, U = params or self.params, self.mul
        vec = self.vec if vec is None else vec
        x = torch.zeros((self.n, self.plan.dim_in), dtype=self.plan.torch_dtype, device="cuda")
        node.tpconv_embedding_forward(self.types, p["table"], out=x[:, :U])
        y = tp.tpconv_forward_vec(self.plan, self.graph, x, vec, self.W)
        scalars = y[:, :U].contiguous()
        logits = scalars @ p["router"]
        experts, gates = node.tpconv_route_forward(self.config, logits)
        layout = node.tpconv_experts_layout(self.experts_plan, experts, load=self.load)
        z = node.tpconv_experts_forward(self.experts_plan, y, p["weights"], experts, gates, layout)
        mixed = node.tpconv_dropout_forward(self.w.irreps_out, self.p_drop, self.seed, step, z, residual=y)
        out = tp.tpconv_forward_vec(self.plan, self.graph, mixed, vec, self.W)
        self.saved = (step, p, vec, x, y, scalars, logits, experts, gates, layout, mixed, out)
        return out

    def energy(self, out):
        """Energies of the atoms (the total is their sum)."""
        return out[:, :self.mul] @ self.saved[1]["readout"]

    def backward(self, grad_energy):
        """Gradients of sum(grad_energy * energy): the parameters', and the positions' [n, 3]."""
        step, p, vec, x, y, scalars, logits, experts, gates, layout, mixed, out = self.saved
        U = self.mul
        grad = dict(readout=grad_energy @ out[:, :U])
        g_out = torch.zeros_like(out)
        g_out[:, :U] = grad_energy[:, None] * p["readout"]
        g_mixed, g_vec2, _ = tp.tpconv_backward_vec(self.plan, self.graph, mixed, vec, self.W, g_out,
                                                    need=(True, True, False))
        g_z = node.tpconv_dropout_backward(self.w.irreps_out, self.p_drop, self.seed, step, g_mixed)
        g_y, grad["weights"], g_gates = node.tpconv_experts_backward(self.experts_plan, y, p["weights"], experts,
                                                                     gates, g_z, layout)
        g_y += g_mixed                                                      # the residual
        g_logits = node.tpconv_route_backward(self.config, logits, experts, g_gates)
        grad["router"] = scalars.t() @ g_logits
        g_y[:, :U] += g_logits @ p["router"].t()
        g_x, g_vec, _ = tp.tpconv_backward_vec(self.plan, self.graph, x, vec, self.W, g_y, need=(True, True, False))
        g_pos = tp.tpconv_positions_backward(self.plan, self.graph, g_vec + g_vec2)
        grad["table"] = node.tpconv_embedding_backward(self.types, g_x[:, :U], p["table"].shape[0])
        return grad, g_pos


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--workload", default="c1k", choices=sorted(workloads.WORKLOADS))
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.02)
    args = ap.parse_args()
    layer = MoELayer(workloads.WORKLOADS[args.workload], n_experts=args.experts, top_k=args.top_k)
    target = torch.randn(layer.n, device="cuda", dtype=layer.plan.torch_dtype,
                         generator=torch.Generator(device="cuda").manual_seed(1))
    begin = time.perf_counter()
    for step in range(args.steps):
        miss = layer.energy(layer.forward(step)) - target
        grad, g_pos = layer.backward(2.0 * miss / layer.n)
        with torch.no_grad():
            for name, g in grad.items():                                    # steps of a length of their own
                p = layer.params[name]
                p -= args.lr * p.norm() * g / g.norm().clamp(min=1e-30)
        if step % 5 == 0 or step == args.steps - 1:
            print(f"step {step:3d}  mean squared miss {float((miss ** 2).mean()):.4f}  "
                  f"largest force {float(g_pos.abs().max()):.3e}  atoms per expert {layer.load.tolist()}", flush=True)
    torch.cuda.synchronize()
    print(f"{layer.n} atoms, {layer.graph.n_edges} edges: {(time.perf_counter() - begin) / args.steps * 1e3:.2f} ms "
          "per step (first step's start-up included)")


if __name__ == "__main__":
    main()

"""A residual stream through layers whose expert products run block-scaled on the tensor cores.

    python examples/scaled_layers.py [--tokens T] [--layers L]

Each layer: moe_add_rmsnorm adds the previous layer's output to the residual stream and normalises it (bf16 for the
router; this example's projection-free stream has no other use of the norm), moe_scaled_forward routes the tokens and
runs the experts on NVFP4 activations and weights.  The same stream through moe_forward (16-bit activations, the same
NVFP4 weights) gives the size of what the 4-bit activations cost.  Synthetic weights and tokens.
"""
import argparse
import dataclasses
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantised_moe_expert_gb300 as qm  # noqa: E402
from quantised_moe_expert_gb300 import synth  # noqa: E402


def run(shape: synth.LayerShape, tokens: int, layers: int, seed: int = 0):
    """Relative difference, layer by layer, of the residual streams of the two ways."""
    hosts = [synth.make_weights(shape, seed + i) for i in range(layers)]
    plain = [qm.DeviceLayer(h) for h in hosts]
    T, H = tokens, shape.hidden
    x0 = torch.from_numpy(synth.make_x(shape, T, seed).view(np.int16)).cuda()
    # the factor of h, from the tokens the layer will see after its norm
    normed = torch.empty_like(x0)
    qm.moe_add_rmsnorm(x0, None, None, 0.0, 1e-6, T, H, None, normed, 0, None)
    scaled = [qm.ScaledLayer.from_nvfp4(h, qm.calibrate_h_scale(p, normed, margin=2.0)) for h, p in zip(hosts, plain)]
    ws, ws_s = qm.workspace(plain[0].cfg, T), qm.scaled_workspace(scaled[0].cfg, qm.MOE_SCALED_NVFP4, T)
    weight = torch.full((H,), 0x3F80, dtype=torch.int16, device="cuda")           # 1.0

    def stream(layer_call):
        s, y, x, states = x0.clone(), None, torch.empty_like(x0), []
        for i in range(layers):
            qm.moe_add_rmsnorm(s, y, weight, 0.0, 1e-6, T, H, s, x, 0, None)
            y = torch.empty_like(x0)
            layer_call(i, x, y)
            states.append(s.view(torch.bfloat16).double() + y.view(torch.bfloat16).double())
        return states

    a = stream(lambda i, x, y: qm.moe_forward(plain[i].cfg, plain[i].w, x, T, None, None, y, None, None, None,
                                              qm.MOE_PATH_AUTO, ws))
    b = stream(lambda i, x, y: qm.moe_scaled_forward(scaled[i].cfg, scaled[i].w, x, T, None, None, y, None, None, None, ws_s))
    assert qm.moe_get_device_status(ws) == 0 and qm.moe_get_device_status(ws_s) == 0
    return [float((u - v).norm() / u.norm()) for u, v in zip(a, b)]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--layers", type=int, default=3)
    a = ap.parse_args()
    shape = dataclasses.replace(synth.QWEN_SHAPE_NVFP4, n_experts=32)
    for i, d in enumerate(run(shape, a.tokens, a.layers)):
        print(f"after layer {i}: residual stream with 4-bit activations {d:.3f} (relative) from 16-bit activations")


if __name__ == "__main__":
    main()

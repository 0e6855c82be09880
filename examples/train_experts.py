"""Train a small routed expert layer, then serve it in FP8.

A layer learns to reproduce a fixed random layer of the same sizes (the same
routing) with the operators of include/moe_train.h; its weights are then
quantised and run through moe_fp8_block_scale_forward.

    python examples/train_experts.py [--steps 60] [--state-bits 8]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_block_scale_gb300 import _lib as L                      # noqa: E402
from fp8_block_scale_gb300.training import ExpertLayer           # noqa: E402


def train(steps=60, state_bits=32, tokens=512, H=256, I=128, E=8, top_k=2, lr=2e-3, seed=0):
    """(losses, output of the trained layer, output of its FP8 form)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    teacher = ExpertLayer(tokens, H, I, E, top_k, generator=gen)
    layer = ExpertLayer(tokens, H, I, E, top_k, state_bits=state_bits, generator=gen)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, H, device="cuda", generator=gen).to(torch.bfloat16)
        logits = torch.randn(tokens, E, device="cuda", generator=gen)
        teacher.route(logits)
        want = teacher.forward(x).float()
        layer.route(logits)
        err = layer.forward(x).float() - want
        losses.append(err.square().mean())
        layer.backward((err * (2.0 / err.numel())).to(torch.bfloat16))
        layer.step(lr)
    if int(layer.status.item()):
        raise RuntimeError(f"device status {int(layer.status.item()):#x}")

    # the same tokens through the quantised layer
    w13, w13_scale, w2, w2_scale = layer.quantized()
    q = torch.empty(tokens, H, dtype=torch.uint8, device="cuda")
    q_scale = torch.empty(tokens, H // 128, device="cuda")
    L.moe_quantize_act_1x128(x, q, q_scale)
    out = torch.zeros(tokens, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(L.moe_forward_workspace_size(tokens, H, I, E, top_k, layer.block_m, layer.sorted_ids.numel()),
                     dtype=torch.uint8, device="cuda")
    L.moe_workspace_init(ws)
    L.moe_fp8_block_scale_forward(L.make_fwd_args(
        q, q_scale, w13, w13_scale, w2, w2_scale, layer.topk_weights, layer.sorted_ids, layer.expert_ids,
        layer.num_padded, out, ws, top_k, layer.block_m))
    trained = layer.forward(x)
    return [float(v) for v in losses], trained, out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, choices=(32, 8), default=32)
    a = ap.parse_args()
    losses, trained, served = train(a.steps, a.state_bits)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.5f}")
    d = (served.float() - trained.float()).norm() / trained.float().norm()
    print(f"FP8 output against the BF16 layer: relative difference {float(d):.4f}")


if __name__ == "__main__":
    main()

"""A training and serving step of one MoE layer with its MXFP4 and balance operators.

The router is trained on its balance and z losses (a few plain gradient steps on
its weights), the experts' weights are quantised once to MXFP4, and the layer
runs on them: per-expert counts even out, and the 4-bit layer's output is
compared with the bf16 layer's on the same routing.

    python examples/mxfp4_layer.py [--tokens 2048] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import combine_moe_route_04_gb300 as moe  # noqa: E402


def quantize_experts(w):
    """W [E, K, N] bf16 to the MXFP4 matrix [E * N, K] the products read."""
    E, K, N = w.shape
    codes, scales = moe.alloc_mxfp4(E * N, K)
    moe.moe_quantize_weights_mxfp4(w, E, K, N, codes, scales)
    return codes, scales


class Router:
    """A linear router trained on its balance (and z) loss alone."""

    def __init__(self, s, generator):
        self.s = moe.shape(*s)
        T, H, _, E, k = s
        self.weight = torch.randn((H, E), generator=generator, device="cuda") / H ** 0.5
        self.weight[:, : max(1, E // 8)] *= 2.0  # some experts are asked for more than others
        self.route_ws = moe.alloc_workspace(self.s)
        self.loss_ws = moe.alloc_balance_workspace(self.s)
        self.picks = moe.alloc_route_outputs(self.s)
        i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
        self.counts, self.num_tokens = torch.empty(E, **i32), torch.empty(1, **i32)
        self.mean_probs, self.losses = torch.empty(E, **f32), torch.empty(2, **f32)
        self.dlogits = torch.empty((T, E), **f32)

    def step(self, x, mask, grad, rate):
        """One step on the tokens with mask non-zero; returns (losses, counts) before it."""
        logits = x @ self.weight
        p = self.picks
        moe.moe_route(self.s, logits, p["topk_ids"], p["topk_w"], p["counts"], p["off_pad"], p["block_expert"],
                      p["num_blocks"], p["gather_idx"], p["scatter_idx"], self.route_ws)
        moe.moe_balance_loss(self.s, logits, p["topk_ids"], mask, self.counts, self.num_tokens, self.mean_probs,
                             self.losses, self.loss_ws)
        moe.moe_balance_loss_backward(self.s, logits, mask, self.counts, self.num_tokens, grad, self.dlogits)
        seen = self.losses.clone(), self.counts.clone()
        self.weight -= rate * (x.t() @ self.dlogits)
        return seen


def main(tokens=2048, steps=20, hidden=1024, inter=512, experts=32, top_k=4, seed=0):
    s = (tokens, hidden, inter, experts, top_k)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, hidden), generator=g, device="cuda")
    mask = torch.ones(tokens, dtype=torch.bool, device="cuda")
    mask[-tokens // 8:] = False  # padding at the end of the batch
    router = Router(s, g)
    grad = torch.tensor([1.0, 1e-3], device="cuda")
    history = [router.step(x, mask, grad, rate=2.0) for _ in range(steps)]
    for i in (0, steps - 1):
        losses, counts = history[i]
        print("step %3d  balance %.4f  z %.3f  busiest expert %d of %d picks"
              % (i, losses[0], losses[1], counts.max(), counts.sum()))

    def weights(K, N):
        return (torch.randn((experts, K, N), generator=g, device="cuda") / K ** 0.5).bfloat16()

    w_gate, w_up, w_down = weights(hidden, inter), weights(hidden, inter), weights(inter, hidden)
    quantized = [t for w in (w_gate, w_up, w_down) for t in quantize_experts(w)]
    xb, logits = x.bfloat16(), (x @ router.weight).contiguous()
    out4, out16 = torch.empty_like(xb), torch.empty_like(xb)
    ws4, ws16 = moe.alloc_mxfp4_workspace(s), moe.alloc_workspace(s)
    moe.moe_forward_mxfp4(s, logits, xb, *quantized, out4, ws4)
    moe.moe_forward(s, logits, xb, w_gate, w_up, w_down, out16, ws16)
    for ws in (ws4, ws16, router.route_ws, router.loss_ws):
        rc = moe.last_device_status(ws)
        if rc != 0:
            raise RuntimeError("device status %s" % moe.STATUS_NAMES.get(rc, rc))
    off = float((out4.float() - out16.float()).norm() / out16.float().norm())
    print("4-bit layer against the bf16 layer: relative difference %.3f" % off)
    return history, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    main(tokens=a.tokens, steps=a.steps)

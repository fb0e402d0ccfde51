"""Training one MoE layer with its backward pass and serving it in 8-bit integers.

The layer is wrapped as a torch function (the library's forward and backward
between plain torch operations), its experts and its router are trained for some
steps on a regression with the router's balance loss beside it, then the experts'
weights are quantised once and the layer runs on 8-bit integers.

    python examples/train_layer.py [--tokens 2048] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import combine_moe_route_04_gb300 as moe  # noqa: E402


class ExpertLayer(torch.autograd.Function):
    """out = layer(logits, x, w_gate, w_up, w_down); logits float32, the rest bf16.

    Every forward keeps a workspace (routing, gathered rows, h, Y) and g, u until its
    backward has run; the backward's scratch is its own.  There is no second
    derivative: a backward that is to be differentiated again (create_graph) is
    refused.  Every backward forms all five gradients, as the library's call does."""

    @staticmethod
    def forward(ctx, s, logits, x, w_gate, w_up, w_down):
        rows = moe.capacity(s)[1]
        ws = moe.alloc_workspace(s)
        g, u = (torch.empty((rows, s[2]), dtype=torch.bfloat16, device=x.device) for _ in range(2))
        out = torch.empty_like(x)
        moe.moe_forward_train(s, logits.contiguous(), x.contiguous(), w_gate, w_up, w_down, g, u, out, ws)
        ctx.s, ctx.ws = s, ws
        ctx.save_for_backward(w_gate, w_up, w_down, g, u)
        return out

    @staticmethod
    def backward(ctx, dout):
        if torch.is_grad_enabled():  # create_graph: these gradients would be taken for constants
            raise RuntimeError("ExpertLayer has no second derivative: its backward does not take create_graph")
        w_gate, w_up, w_down, g, u = ctx.saved_tensors
        s, dout = ctx.s, dout.contiguous()
        bws = moe.alloc_backward_workspace(s)
        dx, dlogits = torch.empty_like(dout), torch.empty((s[0], s[3]), dtype=torch.float32, device=dout.device)
        grads = [torch.empty_like(w) for w in (w_gate, w_up, w_down)]
        moe.moe_backward(s, w_gate, w_up, w_down, g, u, dout, dx, *grads, dlogits, ctx.ws, bws)
        return None, dlogits, dx, *grads


class Balance:
    """The router's balance loss and its gradient beside the layer's."""

    def __init__(self, s, device="cuda"):
        T, _, _, E, k = s
        self.s = s
        self.picks, self.route_ws = moe.alloc_route_outputs(s, device), moe.alloc_workspace(s, device)
        self.ws = moe.alloc_balance_workspace(s, device)
        self.counts, self.num = (torch.empty(n, dtype=torch.int32, device=device) for n in (E, 1))
        self.mean, self.losses = (torch.empty(n, device=device) for n in (E, 2))
        self.dlogits = torch.empty((T, E), device=device)

    def gradient(self, logits, weights):
        """d(weights[0] * balance + weights[1] * z) / dlogits at these logits."""
        p = self.picks
        moe.moe_route(self.s, logits, p["topk_ids"], p["topk_w"], p["counts"], p["off_pad"], p["block_expert"],
                      p["num_blocks"], p["gather_idx"], p["scatter_idx"], self.route_ws)
        moe.moe_balance_loss(self.s, logits, p["topk_ids"], None, self.counts, self.num, self.mean, self.losses,
                             self.ws)
        moe.moe_balance_loss_backward(self.s, logits, None, self.counts, self.num, weights, self.dlogits)
        return self.dlogits


def quantize_experts(w):
    """W [E, K, N] bf16 to the 8-bit matrix [E * N, K] that the products read."""
    E, K, N = w.shape
    codes, scales = moe.alloc_int8(E * N, K)
    moe.moe_quantize_weights_int8(w, E, K, N, codes, scales)
    return codes, scales


def main(tokens=2048, steps=20, hidden=512, inter=384, experts=16, top_k=4, rate=0.1, seed=0):
    s = (tokens, hidden, inter, experts, top_k)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x, target = normal(tokens, hidden).bfloat16(), normal(tokens, hidden)
    router = (normal(hidden, experts) / hidden ** 0.5).requires_grad_()
    weights = [(normal(experts, K, N) / K ** 0.5).bfloat16().requires_grad_()
               for K, N in ((hidden, inter), (hidden, inter), (inter, hidden))]
    balance, mix = Balance(s), torch.tensor([1e-2, 1e-3], device="cuda")
    history = []
    for step in range(steps):
        logits = x.float() @ router
        out = ExpertLayer.apply(s, logits, x, *weights)
        loss = ((out.float() - target) ** 2).sum() / tokens
        aux = balance.gradient(logits.detach(), mix)
        # both losses' gradients reach the router through the logits
        grads = torch.autograd.grad([loss, logits], [router, *weights], [None, aux])
        history.append((float(loss.detach()), [g.clone() for g in grads]))
        with torch.no_grad():
            router -= rate * grads[0]
            for w, g in zip(weights, grads[1:]):
                w.copy_(w.float() - rate * g.float())
        if step in (0, steps - 1):
            print("step %3d  loss %.2f  balance %.4f" % (step, history[-1][0], balance.losses[0]))

    with torch.no_grad():
        logits = (x.float() @ router).contiguous()
        w8 = [t for w in weights for t in quantize_experts(w.detach())]
        out8, out16 = torch.empty_like(x), torch.empty_like(x)
        ws8, ws16 = moe.alloc_int8_workspace(s), moe.alloc_workspace(s)
        moe.moe_forward_int8(s, logits, x, *w8, out8, ws8)
        moe.moe_forward(s, logits, x, *[w.detach() for w in weights], out16, ws16)
    for ws in (ws8, ws16, balance.ws, balance.route_ws):
        rc = moe.last_device_status(ws)
        if rc != 0:
            raise RuntimeError("device status %s" % moe.STATUS_NAMES.get(rc, rc))
    off = float((out8.float() - out16.float()).norm() / out16.float().norm())
    print("8-bit layer against the bf16 layer: relative difference %.4f" % off)
    return history, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    main(tokens=a.tokens, steps=a.steps)

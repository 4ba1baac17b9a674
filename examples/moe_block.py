"""A MoE block on a prompt, its next token, and a routed training step, on one set of packed weights.

    python examples/moe_block.py [--tokens 512] [--hidden 2880] [--inner 2880] [--experts 32] [--top-k 4] [--fmt mxfp4]

1. Prompt: the residual's addition and the RMS norm, the router, and the expert layer on all tokens
   (qmv_rms_norm, qmv_moe_router, qmv_moe_prefill_layer).
2. Decode: the next token through the same weights (qmv_moe_layer_combine). The two agree to the prompt
   path's quantization of the activations.
3. A training step's routing: a trainable map in the experts' place between the dispatch and the weighted
   return, its gradient, the router weights' and the input's (qmv_moe_sort, qmv_moe_dispatch,
   qmv_moe_return and their gradients; the MX experts' own input gradients are not among the calls),
   the balance loss, and the logits' gradient from both (qmv_moe_balance, qmv_moe_router_grad).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_moe_gb300 as qmv  # noqa: E402

DEV = "cuda:0"
EPS = 1e-5


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV)


def random_experts(fmt, experts, inner, hidden, seed):
    """(gate/up descriptor, packed weights, down descriptor, packed weights) of random codes and scales."""
    import numpy as np

    g = np.random.default_rng(seed)
    bits, (lo, hi) = {"mxfp4": (4, (112, 122)), "mxfp8": (8, (107, 117))}[fmt]

    def matrix(n, k):
        codes = g.integers(0, 256 if bits == 4 else 127, size=(experts, n, k * bits // 8), dtype=np.uint8)
        return codes, g.integers(lo, hi + 1, size=(experts, n, k // 32), dtype=np.uint8)

    gate_up, down = qmv.wdesc(fmt, inner, hidden, experts), qmv.wdesc(fmt, hidden, inner, experts)
    w_gate_up = qmv.qmv_pack_gate_up(gate_up, *matrix(inner, hidden), *matrix(inner, hidden))
    w_down = qmv.qmv_pack_weights(down, *matrix(hidden, inner))
    return gate_up, torch.from_numpy(w_gate_up).to(DEV), down, torch.from_numpy(w_down).to(DEV)


class Block:
    """Norm, router and experts of one layer; weights are packed once and serve prompt and decode."""

    def __init__(self, a, seed=0):
        self.hidden, self.inner, self.experts, self.top_k = a.hidden, a.inner, a.experts, a.top_k
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.gate_up, self.w_gate_up, self.down, self.w_down = random_experts(a.fmt, a.experts, a.inner, a.hidden, seed)
        self.gain = torch.ones(a.hidden, dtype=torch.bfloat16, device=DEV)
        self.router = (torch.randn(a.experts, a.hidden, generator=g, device=DEV) / a.hidden ** 0.5).bfloat16()

    def route(self, normed):
        """(expert ids, their weights, logits) of each token."""
        logits = normed @ self.router.T
        tokens = logits.shape[0]
        ids, weights = empty(tokens, self.top_k, dtype=torch.int32), empty(tokens, self.top_k, dtype=torch.float32)
        qmv.qmv_moe_router("bf16", logits, self.experts, None, tokens, self.experts, self.top_k, "softmax", True, 1.0, ids, weights)
        return ids, weights, logits

    def router_gradient(self, logits, ids, dweights, share):
        """(balance loss, gradient of the logits from the weights' and from share times that loss)."""
        tokens, experts, top_k = logits.shape[0], self.experts, self.top_k
        counts, means, loss = empty(experts + 1, dtype=torch.int32), empty(experts, dtype=torch.float32), empty(1, dtype=torch.float32)
        ws = empty(qmv.qmv_moe_balance_workspace_bytes(tokens, experts), dtype=torch.uint8)
        qmv.qmv_moe_balance("bf16", logits, experts, None, ids, tokens, experts, top_k, "softmax", counts, means, loss, ws)
        dlogits = torch.empty_like(logits)
        qmv.qmv_moe_router_grad("bf16", logits, experts, None, ids, dweights, counts, torch.full_like(loss, share), tokens, experts,
                                top_k, "softmax", True, 1.0, dlogits, experts)
        return loss, dlogits

    def norm(self, x, residual):
        """(normed, x + residual) of rows x."""
        rows = x.shape[0]
        normed, total = torch.empty_like(x), torch.empty_like(x)
        qmv.qmv_rms_norm("bf16", x, self.hidden, residual, self.hidden, self.gain, rows, self.hidden, EPS, total, "plain", normed)
        return normed, total

    def prompt(self, x, residual):
        normed, total = self.norm(x, residual)
        ids, weights, _ = self.route(normed)
        tokens = x.shape[0]
        ws = empty(qmv.qmv_moe_prefill_layer_workspace_bytes(self.gate_up, self.down, tokens, self.top_k), dtype=torch.uint8)
        y = empty(tokens, self.hidden)
        qmv.qmv_moe_prefill_layer(self.gate_up, self.w_gate_up, self.down, self.w_down, "bf16", normed, self.hidden, ids, weights,
                                  tokens, self.top_k, ws, y)
        return y, total

    def decode(self, x, residual):
        """Up to 16 tokens with bf16 activations."""
        normed, total = self.norm(x, residual)
        ids, weights, _ = self.route(normed)
        tokens = x.shape[0]
        ws = empty(qmv.qmv_moe_layer_combine_workspace_bytes(self.gate_up, self.down, tokens, self.top_k), dtype=torch.uint8)
        y = empty(tokens, self.hidden)
        qmv.qmv_moe_layer_combine(self.gate_up, self.w_gate_up, self.down, self.w_down, normed, ids, weights, tokens, self.top_k,
                                  ws, y)
        return y, total


class Routed(torch.autograd.Function):
    """Tokens to the experts' order."""

    @staticmethod
    def forward(ctx, x, row_of_slot, top_k):
        ctx.save_for_backward(row_of_slot)
        ctx.shape = (*x.shape, top_k)
        x = x.contiguous()
        xs = empty(x.shape[0] * top_k, x.shape[1], dtype=x.dtype)
        qmv.qmv_moe_dispatch(x.dtype, x, x.shape[1], x.shape[0], top_k, x.shape[1], row_of_slot, xs)
        return xs

    @staticmethod
    def backward(ctx, dxs):
        (row_of_slot,), (tokens, width, top_k) = ctx.saved_tensors, ctx.shape
        dx = empty(tokens, width, dtype=dxs.dtype)
        qmv.qmv_moe_dispatch_grad(dxs.dtype, dxs.contiguous(), tokens, top_k, width, row_of_slot, dx, width)
        return dx, None, None


class Returned(torch.autograd.Function):
    """The experts' rows back to their tokens, with the router's weights (fp32)."""

    @staticmethod
    def forward(ctx, ys, weights, row_of_slot):
        ys, weights = ys.contiguous(), weights.contiguous()
        ctx.save_for_backward(ys, weights, row_of_slot)
        tokens, top_k = weights.shape
        y = empty(tokens, ys.shape[1], dtype=ys.dtype)
        qmv.qmv_moe_return(ys.dtype, ys, weights, tokens, top_k, ys.shape[1], row_of_slot, y, ys.shape[1])
        return y

    @staticmethod
    def backward(ctx, dy):
        ys, weights, row_of_slot = ctx.saved_tensors
        tokens, top_k = weights.shape
        dys, dweights = torch.empty_like(ys), torch.empty_like(weights)
        qmv.qmv_moe_return_grad(ys.dtype, dy.contiguous(), ys.shape[1], ys, weights, tokens, top_k, ys.shape[1], row_of_slot, dys,
                                dweights)
        return dys, dweights, None


def training_step(block, x, target):
    """Loss and gradients of a scale per column on the experts' rows, of the router's weights, of x and of the logits (with a
    hundredth of the balance loss), and that loss."""
    tokens, experts, top_k = x.shape[0], block.experts, block.top_k
    ids, weights, logits = block.route(x)
    i32 = torch.int32
    offsets, row_of_slot, slot_of_row = empty(experts + 1, dtype=i32), empty(tokens * top_k, dtype=i32), empty(tokens * top_k, dtype=i32)
    qmv.qmv_moe_sort(ids, tokens, top_k, experts, offsets, row_of_slot, slot_of_row)
    x, weights = x.clone().requires_grad_(), weights.requires_grad_()
    scale = torch.ones(x.shape[1], dtype=torch.bfloat16, device=DEV, requires_grad=True)
    y = Returned.apply(Routed.apply(x, row_of_slot, top_k) * scale, weights, row_of_slot)
    loss = (y.float() - target.float()).square().mean()
    loss.backward()
    balance, dlogits = block.router_gradient(logits, ids, weights.grad, 0.01)
    return loss.detach(), scale.grad, weights.grad, x.grad, dlogits, balance


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 512), ("hidden", 2880), ("inner", 2880), ("experts", 32), ("top-k", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--fmt", choices=("mxfp4", "mxfp8"), default="mxfp4")
    a = ap.parse_args(argv)
    block = Block(a)
    g = torch.Generator(device=DEV).manual_seed(1)
    x, residual = (torch.randn(a.tokens, a.hidden, generator=g, device=DEV).bfloat16() for _ in range(2))
    y, total = block.prompt(x, residual)
    few = min(a.tokens, 4)
    y1, _ = block.decode(x[:few].contiguous(), residual[:few].contiguous())
    apart = ((y[:few].float() - y1.float()).norm() / y1.float().norm()).item()
    print(f"prompt: {a.tokens} tokens; the first {few} through the decode layer differ by {apart:.3f} (activations in {a.fmt})")
    loss, dscale, dweights, dx, dlogits, balance = training_step(block, total, y)
    print(f"training step: loss {loss.item():.4f}, |d scale| {dscale.float().norm().item():.4f}, "
          f"|d weights| {dweights.norm().item():.4f}, |dx| {dx.float().norm().item():.4f}, "
          f"balance loss {balance.item():.4f}, |d logits| {dlogits.float().norm().item():.4f}")
    status = qmv.qmv_device_status(clear=True)
    if status:
        raise SystemExit(f"device status {status}")
    return apart, loss.item(), (dscale, dweights, dx, dlogits)


if __name__ == "__main__":
    main()

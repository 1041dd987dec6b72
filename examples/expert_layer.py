"""A mixture-of-experts layer on the expert operators: a few training steps on
synthetic data, then single tokens through the trained layer, and the layer
inside a block with norms, served in 8 bits.

    python examples/expert_layer.py [--tokens N] [--width H] [--experts E] [--slots K] [--steps S]

Each token goes to its K best experts, each expert is a two-matrix network, and
the layer's output is the experts' outputs weighted by the router.  The block
around it norms what goes in, and on the way out norms the layer's output,
gates it, adds it to the scaled residual stream and norms that for the next
block.  The operators compute values and gradients; the Functions below tie
them to torch's autograd.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lsd_radix_sort_key_gb300 as rs  # noqa: E402


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, position, offsets):
        ctx.save_for_backward(position, offsets)
        return rs.expert_dispatch(x, position, offsets)

    @staticmethod
    def backward(ctx, grad):
        return rs.expert_dispatch_grad(grad.contiguous(), *ctx.saved_tensors), None, None


class Matmul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, offsets, activation):
        ctx.activation = activation
        if activation == "none":
            y, pre = rs.expert_matmul(x, w, offsets, bias=bias), None
        else:
            y, pre = rs.expert_matmul(x, w, offsets, bias=bias, activation=activation, return_pre=True)
        ctx.save_for_backward(x, w, offsets, pre)
        return y

    @staticmethod
    def backward(ctx, grad):
        x, w, offsets, pre = ctx.saved_tensors
        dx, dw, dbias = ctx.needs_input_grad[:3]  # the ones wanted
        grads = rs.expert_matmul_grad(grad.contiguous(), x, w, offsets, pre=pre, activation=ctx.activation, need_dx=dx,
                                      need_dw=dw, bias=dbias)
        return (*grads, None, None)


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, position, offsets):
        ctx.save_for_backward(y, weights, position, offsets)
        return rs.expert_combine(y, weights, position, offsets)

    @staticmethod
    def backward(ctx, grad):
        return (*rs.expert_combine_grad(grad.contiguous(), *ctx.saved_tensors), None, None)


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        ctx.save_for_backward(x, weight)
        return rs.expert_norm(x, weight)

    @staticmethod
    def backward(ctx, grad):
        return rs.expert_norm_grad(grad.contiguous(), *ctx.saved_tensors)[:2]


class NormOut(torch.autograd.Function):
    """The way out of a block and into the next: (y, h) of expert_norm."""

    @staticmethod
    def forward(ctx, x, block, weight, block_weight, gate, residual_scale):
        y, h = rs.expert_norm(x, weight, block=block, block_weight=block_weight, gate=gate, residual_scale=residual_scale)
        ctx.residual_scale = residual_scale
        ctx.save_for_backward(y, block, weight, block_weight, gate)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        y, block, weight, block_weight, gate = ctx.saved_tensors
        dx, dweight, dblock, dafter, dgate = rs.expert_norm_grad(
            dh.contiguous(), y, weight, dy=dy.contiguous(), block=block, block_weight=block_weight, gate=gate,
            residual_scale=ctx.residual_scale)
        return dx, dblock, dweight, dafter, dgate, None


class ExpertLayer(torch.nn.Module):
    def __init__(self, width, hidden, experts, slots, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.slots = slots

        def weights(*shape, scale):
            return torch.nn.Parameter((torch.randn(*shape, device=device) * scale).to(dtype))

        self.router = torch.nn.Parameter(torch.randn(width, experts, device=device) * width**-0.5)
        self.up, self.up_bias = weights(experts, hidden, width, scale=width**-0.5), weights(experts, hidden, scale=0.0)
        self.down = weights(experts, width, hidden, scale=hidden**-0.5)
        self.down_bias = weights(experts, width, scale=0.0)

    def route(self, x):
        """The tokens' experts [T, K] and their weights, summing to one."""
        logits, ids = (x.float() @ self.router).topk(self.slots, dim=1)
        return torch.softmax(logits, dim=1), ids

    def forward(self, x):
        weights, ids = self.route(x)
        _, position, offsets = rs.expert_sort(ids, self.router.shape[1])
        rows = Dispatch.apply(x, position, offsets)
        mid = Matmul.apply(rows, self.up, self.up_bias, offsets, "silu")
        out = Matmul.apply(mid, self.down, self.down_bias, offsets, "none")
        return Combine.apply(out, weights, position, offsets)


class ExpertBlock(torch.nn.Module):
    """An ExpertLayer with the norms around it: x -> (y, h), the residual stream
    and what the next block reads."""

    def __init__(self, width, hidden, experts, slots, dtype=torch.bfloat16, device="cuda", residual_scale=0.9):
        super().__init__()
        self.layer, self.residual_scale = ExpertLayer(width, hidden, experts, slots, dtype, device), residual_scale
        self.before, self.after, self.next = (torch.nn.Parameter(torch.ones(width, device=device)) for _ in range(3))
        self.gate = torch.nn.Parameter(torch.full((width,), 0.5, device=device))
        self.quantized = None

    def forward(self, x):
        out = self.layer(Norm.apply(x, self.before))
        return NormOut.apply(x, out, self.next, self.after, self.gate, self.residual_scale)

    @torch.no_grad()
    def quantize(self):
        """The experts' weights in 8 bits, once after training."""
        self.quantized = (*rs.expert_quantize_weights(self.layer.up), *rs.expert_quantize_weights(self.layer.down))
        return self

    @torch.no_grad()
    def serve(self, x):
        """forward() with 8-bit products: rows are quantised as they are dispatched,
        and the first product's result by the product itself."""
        up, up_scales, down, down_scales = self.quantized
        layer = self.layer
        h = rs.expert_norm(x, self.before)
        weights, ids = layer.route(h)
        _, position, offsets = rs.expert_sort(ids, layer.router.shape[1])
        rows, scales = rs.expert_dispatch_quantized(h, position, offsets)
        mid, scales = rs.expert_matmul_quantized(rows, scales, up, up_scales, offsets, bias=layer.up_bias,
                                                 activation="silu", dtype=x.dtype, quantize=True)
        out = rs.expert_matmul_quantized(mid, scales, down, down_scales, offsets, bias=layer.down_bias, dtype=x.dtype)
        out = rs.expert_combine(out, weights, position, offsets)
        return rs.expert_norm(x, self.next, block=out, block_weight=self.after, gate=self.gate,
                              residual_scale=self.residual_scale)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--slots", type=int, default=2)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = ExpertLayer(a.width, 2 * a.width, a.experts, a.slots)
    target = torch.randn(a.width, a.width, device="cuda") * a.width**-0.5
    optimizer = torch.optim.Adam(layer.parameters(), lr=2e-3)
    losses = []
    for _ in range(a.steps):
        x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
        loss = (layer(x).float() - torch.tanh(x.float() @ target)).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(float(loss.detach()))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps of {a.tokens} tokens")
    with torch.no_grad():  # the same tokens one at a time give the same rows, up to rounding
        x = torch.randn(8, a.width, device="cuda").bfloat16()
        whole = layer(x).float()
        single = torch.cat([layer(x[i:i + 1]) for i in range(8)]).float()
        print(f"single tokens against the batch: largest difference {float((whole - single).abs().max()):.2e}")
    block = ExpertBlock(a.width, 2 * a.width, a.experts, a.slots)
    block.layer = layer
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16().requires_grad_()
    y, h = block(x)
    (y.float().square().mean() + h.float().mean()).backward()
    served = block.quantize().serve(x.detach())[0].float()
    off = float((served - y.detach().float()).norm() / y.detach().float().norm())
    print(f"the block in 8 bits against 16: {off:.1e} of its output")
    return losses


if __name__ == "__main__":
    main()

"""A mixture-of-experts layer on the expert-parallel path: forward and one
training step.

    route -> dispatch -> moe_group -> expert_product (gated) -> expert_product (down)
          -> moe_ungroup -> combine

and back, through the same calls: the gradient of combine is a dispatch of the
output's gradient along the cached layout, the gradient of dispatch is a
combine.  The router's own product and the per-row scalings between the calls
are plain torch.  With ``checkpoints`` the pre-activations are kept in 8 bits and
the activations recomputed; ``decode`` takes a few tokens through norm, routing
and experts without dispatch.

    python examples/moe_layer.py            # a few steps on random data, loss printed
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_ep_layout_06_gb300 as ep  # noqa: E402


class MoeLayer:
    """W logical ranks of T tokens each; E experts of hidden size H and inner
    size F, top-k routing with renormalised softmax weights."""

    def __init__(self, W=2, E=8, k=2, T=128, H=256, F=192, dtype=torch.bfloat16, balance_coef=0.01, z_coef=0.001,
                 device="cuda", seed=0, checkpoints=False):
        g = torch.Generator(device=device).manual_seed(seed)

        def param(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).to(dtype)

        self.k, self.balance_coef, self.z_coef, self.checkpoints = k, balance_coef, z_coef, checkpoints
        self.router = param(E, H)
        self.gate_up = param(E, 2 * F, H)            # the experts of rank r are r * E/W ...
        self.down = param(E, H, F)
        self.down_bias = torch.zeros(E, H, dtype=dtype, device=device)
        self.norm = torch.ones(H, dtype=dtype, device=device)     # of decode
        self.op = ep.EpDispatchCombineOp(ep.EpDispatchCombineConfig(
            world_size=W, num_experts=E, topk=k, hidden=H, max_tokens_per_rank=T,
            max_grouped_rows_per_rank=W * T * k))

    def forward(self, x, num_tokens=None):
        """x: [W][T][H].  Returns the experts' output, same shape; rows past
        num_tokens are unspecified."""
        op = self.op
        logits = torch.matmul(x, self.router.T)
        weights, indices = ep.route(logits, self.k, num_tokens=num_tokens)
        loss, counts, _ = ep.balance_loss(logits, indices, balance_coef=self.balance_coef, z_coef=self.z_coef,
                                          num_tokens=num_tokens)
        ids = indices.clamp(min=0)                    # absent tokens carry -1; dispatch leaves them out
        op.dispatch(x, weights, None, ids, num_tokens=num_tokens)
        rows, _, count, offset = op.moe_group()
        h, pre = ep.expert_product(rows, self.gate_up, count, offset, activation="swiglu", save_pre=True)
        ep.expert_product(h, self.down, count, offset, bias=self.down_bias, out=op.moe_y)
        op.moe_ungroup()
        out, _ = op.combine()
        if self.checkpoints:                          # 8 bits in place of h and pre
            h, pre = None, ep.checkpoint(pre, count, offset)
        self.saved = (x, logits, ids, indices, counts, num_tokens, rows, h, pre, count, offset)
        return out, loss[0]

    def backward(self, grad_out, grad_loss):
        """Gradients of sum(out * grad_out) + grad_loss * balance: by x and by
        the parameters, in the order (x, router, gate_up, down, down_bias)."""
        op, k = self.op, self.k
        x, logits, ids, indices, counts, num_tokens, rows, h, pre, count, offset = self.saved
        rows, y, g_w = rows.clone(), op.moe_y.clone(), op.moe_w.clone()     # the replay reuses the segments
        # grad_out to every row that the token was sent to, weights 1
        op.dispatch_send_replay(grad_out, torch.ones_like(grad_out[..., :k], dtype=torch.float32), ids,
                                num_tokens=num_tokens)
        op.dispatch_recv()
        g_rows, _, _, _ = op.moe_group()
        W, gcap = g_w.shape
        used = torch.arange(gcap, device=x.device) < count.sum(1, keepdim=True)
        zero = torch.zeros((), dtype=x.dtype, device=x.device)
        g_rows, y = (torch.where(used[..., None], t, zero) for t in (g_rows, y))
        # out = sum of weight * y over a token's experts
        entry = op.moe_src.clone()                    # received row * k + choice
        token = torch.gather(op.src_pos, 1, torch.where(used, entry // k, 0).long())
        place = (token.long() * k + entry % k)[used]
        grad_weights = torch.zeros(ids.shape, dtype=torch.float32, device=x.device)
        grad_weights.view(-1)[place] = (g_rows.float() * y.float()).sum(-1)[used]
        g_y = (g_rows.float() * torch.where(used, g_w, 0.0)[..., None]).to(x.dtype)
        scales = None
        if self.checkpoints:
            pre, scales = pre
            h = ep.checkpoint_restore(pre, scales, count, offset, activation="swiglu", dtype=x.dtype)
        g_h, g_down, g_bias = ep.expert_product_backward(g_y, h, self.down, count, offset, bias_grad=True)
        g_x, g_gate_up, _ = ep.expert_product_backward(g_h, rows, self.gate_up, count, offset, pre=pre,
                                                       pre_scales=scales, activation="swiglu")
        op.moe_ungroup(g_x)
        grad_x, _ = op.combine()
        g_logits = ep.route_backward(grad_weights, logits, ids, num_tokens=num_tokens, grad_loss=grad_loss,
                                     counts=counts, balance_coef=self.balance_coef, z_coef=self.z_coef)
        here = (indices[..., :1] >= 0)
        grad_x = torch.where(here, grad_x, zero) + torch.matmul(g_logits, self.router)
        g_router = torch.matmul(g_logits.flatten(0, 1).T, torch.where(here, x, zero).flatten(0, 1))
        return grad_x, g_router, g_gate_up, g_down, g_bias

    def decode(self, x, residual):
        """x: what the block before adds to the residual stream, [T][H], a few
        tokens.  Returns (the layer's output, the residual stream): the next
        block's pair."""
        y, total = ep.rms_norm(x, self.norm, residual=residual)
        weights, indices = ep.route(torch.matmul(y, self.router.T), self.k)
        return ep.moe_few_tokens(y, weights, indices, self.gate_up, self.down, down_bias=self.down_bias), total


def main():
    torch.manual_seed(0)
    layer = MoeLayer()
    x = torch.randn(2, 128, 256, device="cuda").to(torch.bfloat16)
    goal = torch.randn(2, 128, 256, device="cuda") * 0.3
    one = torch.ones((), device="cuda")
    for step in range(20):
        out, balance = layer.forward(x)
        off = out.float() - goal
        grads = layer.backward((2.0 * off / off.shape[-1]).to(x.dtype), one)
        if step % 5 == 0:
            print(f"step {step}: squared error {off.square().sum(-1).mean().item():.4f}, balance {balance.item():.5f}")
        for p, g in zip((layer.router, layer.gate_up, layer.down, layer.down_bias), grads[1:]):
            p -= (0.05 * g.float()).to(p.dtype)
    assert layer.op.get_error() == (0, 0) and ep.moe_error() == 0


if __name__ == "__main__":
    main()

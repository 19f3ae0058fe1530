"""One pre-norm MoE block for training: forward, and the gradient of everything.

The residual stream h and the block's normalised input xn (the previous block's
last step, or moe_block_norm without a block output) go in; the next stream and
the next block's normalised input come out. Forward over T tokens:
  1. moe_route, moe_route_grouped: logits xn . gate, scores, top-k, statistics;
  2. moe_permute: capacity drops and the expert-major rows;
  3. moe_expert_gemm with W1 and GELU (the value before it kept), with W2;
  4. moe_block_norm: combine, norm, token gate, residual, the next block's norm.
Backward, from the gradients of the next stream, of the next normalised input
and of the balance loss:
  4. moe_block_norm_bwd; 3. moe_expert_gemm with the transposed weights (GELU's
  slope in its epilogue) and moe_expert_wgrad; 1. moe_route_grouped_bwd, and the
  router's own two products as those of a single expert; 2. moe_block_norm without
  norms adds up what reaches xn, from the router and from the token's rows.
Every step runs in the library's kernels on the current stream but for the sum of the
gate's bias' gradient and, accumulated, of the small weights' gradients; nothing
synchronises with the host, so both directions can be captured in a CUDA graph. A
small run of it all:
python -m top_routing_expert_gb300.block
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (BlockConfig, BlockWorkspace, MoeShape, RouteConfig, Workspace, _shape, moe_block_norm,
               moe_block_norm_bwd, moe_expert_gemm, moe_expert_wgrad, moe_permute, moe_route,
               moe_route_grouped, moe_route_grouped_bwd)


class BlockWeights:
    """Weights of a block, or (zeros) their gradients: W1 [E, H, h], W2 [E, h, H]
    and gate [H, E] (bf16; gradients fp32), post and pre [H] fp32 (the norm of
    the block's output, and the one that the next block begins with), gate_bias
    [E] fp32 or None."""

    def __init__(self, W1, W2, gate, post, pre, gate_bias=None):
        self.W1, self.W2, self.gate, self.post, self.pre = W1, W2, gate, post, pre
        self.gate_bias = gate_bias

    @classmethod
    def zeros_like(cls, w: "BlockWeights") -> "BlockWeights":
        z = lambda t: torch.zeros(t.shape, dtype=torch.float32, device=t.device)
        return cls(z(w.W1), z(w.W2), z(w.gate), z(w.post), z(w.pre),
                   None if w.gate_bias is None else z(w.gate_bias))


class TrainBlock:
    """Buffers of one block shape. backward() belongs to the last forward(), whose
    intermediate values are in the attributes until the next one; dev_status
    collects the MOE_DEV_* bits."""

    def __init__(self, shape, route: RouteConfig, block: BlockConfig, device="cuda"):
        s: MoeShape = _shape(shape)
        self.shape, self.route, self.block = s, route, block
        new = lambda *n, dt=torch.bfloat16: torch.empty(n, dtype=dt, device=device)
        rows, i32, f32 = s.T * s.top_k, torch.int32, torch.float32
        self.ws = Workspace(s, device=device)
        self.block_ws = BlockWorkspace(s.T, s.H, device=device)
        self.dev_status = torch.zeros(1, dtype=i32, device=device)
        self.logits = new(s.T, s.E, dt=f32)
        self.topk_idx, self.topk_w = new(s.T, s.top_k, dt=i32), new(s.T, s.top_k, dt=f32)
        self.routed_counts, self.P, self.aux = new(s.E, dt=i32), new(s.E, dt=f32), new(1, dt=f32)
        self.kept_counts, self.offsets = new(s.E, dt=i32), new(s.E + 1, dt=i32)
        self.dest_row, self.src_token = new(s.T, s.top_k, dt=i32), new(rows, dt=i32)
        self.x_perm, self.y_perm = new(rows, s.H), new(rows, s.H)
        self.u, self.act = new(rows, s.h), new(rows, s.h)
        # gradients of the intermediate values; the router's in a width the
        # products take, 0 in the columns past E
        self.g_y, self.g_x, self.g_u = new(rows, s.H), new(rows, s.H), new(rows, s.h)
        self.g_topk_w, self.g_logits = new(s.T, s.top_k, dt=f32), new(s.T, s.E, dt=f32)
        wide = (s.E + 63) // 64 * 64
        self.g_scores = torch.zeros(s.T, wide, dtype=torch.bfloat16, device=device)
        self.gate_wide = torch.zeros(s.H, wide, dtype=torch.bfloat16, device=device)
        self.g_gate_wide = new(1, s.H, wide, dt=f32)
        self.g_router = new(s.T, s.H)
        self.one_segment = torch.tensor([0, s.T], dtype=i32, device=device)
        self.add = BlockConfig.make(post_norm=False)
        # one call's gradients of the small weights, where they are accumulated
        self.g_post, self.g_pre, self.g_bias = new(s.H, dt=f32), new(s.H, dt=f32), new(s.E, dt=f32)
        self._kept = None

    def forward(self, h: torch.Tensor, xn: torch.Tensor, w: BlockWeights, out: torch.Tensor,
                xn_next: Optional[torch.Tensor] = None, token_gate: Optional[torch.Tensor] = None,
                select_bias: Optional[torch.Tensor] = None) -> torch.Tensor:
        """out, xn_next [T, H] (bf16) from the stream h and the normalised input
        xn [T, H]. token_gate [T] (fp32) multiplies the block's output, select_bias
        acts on the choice of experts alone. backward() reads xn, out, w and
        token_gate again: they have to be as they were."""
        s, ws, st = self.shape, self.ws, self.dev_status
        self._kept = (xn, w, out, token_gate)
        if s.T == 0:  # empty tensors have no address to pass
            for t in (self.routed_counts, self.P, self.aux, self.kept_counts, self.offsets):
                t.zero_()
            return out
        moe_route(s, xn, w.gate, w.gate_bias, self.topk_idx, self.topk_w, logits_out=self.logits,
                  dev_status=st, ws=ws)
        moe_route_grouped(s, self.route, self.logits, select_bias, self.topk_idx, self.topk_w,
                          routed_counts=self.routed_counts, P=self.P, aux=self.aux,
                          dev_status=st, ws=ws)
        moe_permute(s, xn, self.topk_idx, self.kept_counts, self.offsets, self.dest_row,
                    self.src_token, self.x_perm, dev_status=st, ws=ws)
        moe_expert_gemm(self.x_perm, self.offsets, w.W1, self.act, epilogue="gelu", pre=self.u,
                        dev_status=st)
        moe_expert_gemm(self.act, self.offsets, w.W2, self.y_perm, dev_status=st)
        moe_block_norm(self.block, h, self.y_perm, out, xn=xn_next, dest_row=self.dest_row,
                       topk_w=self.topk_w, post_weight=w.post, gate=token_gate, pre_weight=w.pre)
        return out

    def backward(self, grad_out: Optional[torch.Tensor], grad_xn_next: Optional[torch.Tensor],
                 grad_h: torch.Tensor, grad_xn: torch.Tensor, grads: BlockWeights,
                 grad_token_gate: Optional[torch.Tensor] = None,
                 grad_aux: Optional[torch.Tensor] = None, accumulate=False) -> None:
        """grad_h, grad_xn [T, H] (bf16) and the weights' gradients (fp32) from those
        of out and xn_next [T, H] (bf16; either may be None) and of aux [1].
        accumulate: False, the weights' gradients are written; "all", each is added
        to what is there (every micro-batch but a step's first); True, those of W1
        and W2 alone are added and the others written, for a caller who adds up the
        small ones. Gradients of tokens are written in any case."""
        if accumulate not in (False, True, "all"):
            raise ValueError(f'accumulate must be False, True or "all", got {accumulate!r}')
        every = accumulate == "all"
        if self._kept is None:
            raise RuntimeError("backward() without a forward()")
        s, st = self.shape, self.dev_status
        xn, w, out, token_gate = self._kept
        if s.T == 0:
            small = [] if every else [grads.post, grads.pre, grads.gate, grads.gate_bias]
            for t in small + ([] if accumulate else [grads.W1, grads.W2]):
                if t is not None:
                    t.zero_()
            return
        g_post, g_pre, g_bias = ((self.g_post, self.g_pre, self.g_bias) if every else
                                 (grads.post, grads.pre, grads.gate_bias))
        if grad_xn_next is None:
            g_pre.zero_()
        moe_block_norm_bwd(self.block, out, self.y_perm, grad_out, grad_h, self.g_y,
                           grad_xn=grad_xn_next, dest_row=self.dest_row, topk_w=self.topk_w,
                           post_weight=w.post, gate=token_gate, pre_weight=w.pre,
                           grad_topk_w=self.g_topk_w, grad_post=g_post,
                           grad_gate=grad_token_gate,
                           grad_pre=g_pre if grad_xn_next is not None else None,
                           ws=self.block_ws)
        moe_expert_gemm(self.g_y, self.offsets, w.W2, self.g_u, transposed=True,
                        epilogue="gelu_grad", pre=self.u, dev_status=st)
        moe_expert_wgrad(self.act, self.g_y, self.offsets, grads.W2, accumulate=accumulate,
                         dev_status=st)
        moe_expert_gemm(self.g_u, self.offsets, w.W1, self.g_x, transposed=True, dev_status=st)
        moe_expert_wgrad(self.x_perm, self.g_u, self.offsets, grads.W1, accumulate=accumulate,
                         dev_status=st)
        moe_route_grouped_bwd(s, self.route, self.logits, self.topk_idx, self.g_topk_w,
                              self.g_logits, grad_aux=grad_aux,
                              routed_counts=self.routed_counts if grad_aux is not None else None)
        if w.gate_bias is not None:
            torch.sum(self.g_logits, 0, out=g_bias)
        # the router is a product with a single expert, logits = xn . gate, and its
        # gradient enters the two products in bf16, which they take: off by 2^-8 of each
        # value at most, as every gradient that goes from step to step is
        self.g_scores[:, :s.E].copy_(self.g_logits)
        self.gate_wide[:, :s.E].copy_(w.gate)
        moe_expert_gemm(self.g_scores, self.one_segment, self.gate_wide[None], self.g_router,
                        transposed=True, dev_status=st)
        # what reaches xn, g_router + sum_j g_x[dest_j], in fp32 and rounded once
        moe_block_norm(self.add, self.g_router, self.g_x, grad_xn, dest_row=self.dest_row)
        moe_expert_wgrad(xn, self.g_scores, self.one_segment, self.g_gate_wide, dev_status=st)
        g_gate = self.g_gate_wide[0, :, :s.E]
        if not every:
            grads.gate.copy_(g_gate)
            return
        grads.gate.add_(g_gate)
        grads.post.add_(g_post)
        grads.pre.add_(g_pre)
        if w.gate_bias is not None:
            grads.gate_bias.add_(g_bias)


def main() -> None:
    T, H, E, k, h = 2048, 512, 64, 6, 256
    g = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *n, std=1.0: (std * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)
    w = BlockWeights(draw(E, H, h, std=H ** -0.5), draw(E, h, H, std=h ** -0.5),
                     draw(H, E, std=H ** -0.5), torch.ones(H, device="cuda"),
                     torch.ones(H, device="cuda"))
    config = RouteConfig.make("sigmoid", n_groups=8, topk_groups=3, group_top=2, scale=2.5)
    block = TrainBlock(MoeShape.make(T, H, E, k, h, 1.25), config, BlockConfig.make())
    x, xn = draw(T, H), draw(T, H)
    moe_block_norm(block.block, x, None, None, xn=xn)        # the first block's norm
    out, xn_next, grad_h, grad_xn = (torch.empty_like(x) for _ in range(4))
    block.forward(x, xn, w, out, xn_next)
    grads = BlockWeights.zeros_like(w)
    block.backward(draw(T, H), draw(T, H), grad_h, grad_xn, grads,
                   grad_aux=torch.full((1,), 0.01, device="cuda"))
    torch.cuda.synchronize()
    norms = ", ".join(f"{n} {getattr(grads, n).norm().item():.2f}" for n in ("W1", "W2", "gate", "post", "pre"))
    print(f"tokens {T}, experts {E}: aux {block.aux.item():.4f}, kept rows "
          f"{block.offsets[E].item()} of {T * k}, |out| {out.float().norm().item():.2f}, gradients "
          f"{norms}, status {block.dev_status.item()}")


if __name__ == "__main__":
    main()

"""An MoE layer with grouped routing and 4-bit (MX4) experts.

One forward over T tokens:
  1. moe_route: the router GEMM, for its logits (x . gate + gate_bias);
  2. moe_route_grouped: softmax or sigmoid scores, selection bias, groups,
     top-k, weights, balance statistics;
  3. moe_permute: capacity drops and the expert-major rows;
  4. moe_quantize_rows_mx4 of the kept rows, moe_expert_gemm_mx4 with W1 and
     GELU, the same again with W2;
  5. moe_combine with the routing weights.
The router's gradient (moe_route_grouped_bwd) is formed from what the forward
kept. Every step runs in the library's kernels on the current stream; nothing
synchronises with the host, so forward and router_grad can be captured in a
CUDA graph. A small run of it all:  python -m top_routing_expert_gb300.mx4
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (MoeShape, Mx4Weights, RouteConfig, Workspace, _shape, moe_combine,
               moe_expert_gemm_mx4, moe_permute, moe_quantize_rows_mx4, moe_route,
               moe_route_grouped, moe_route_grouped_bwd)


class Mx4Layer:
    """Buffers and 4-bit weights of one layer shape. After forward() the
    routing (logits, topk_idx, topk_w, routed_counts, P, aux), the dispatch
    (offsets, dest_row) and the intermediate rows are in the attributes of
    those names until the next one; dev_status collects the MOE_DEV_* bits."""

    def __init__(self, shape, config: RouteConfig, W1: torch.Tensor, W2: torch.Tensor):
        s: MoeShape = _shape(shape)
        if tuple(W1.shape) != (s.E, s.H, s.h) or tuple(W2.shape) != (s.E, s.h, s.H):
            raise ValueError(f"W1 must be [E, H, h] and W2 [E, h, H] of the shape "
                             f"(E={s.E}, H={s.H}, h={s.h})")
        self.shape, self.config = s, config
        self.weights = Mx4Weights(W1, W2)
        dev = W1.device
        new = lambda *n, dt=torch.float32: torch.empty(n, dtype=dt, device=dev)
        rows = s.T * s.top_k
        i32, u8, bf16 = torch.int32, torch.uint8, torch.bfloat16
        self.ws = Workspace(s, device=dev)
        self.dev_status = torch.zeros(1, dtype=i32, device=dev)
        self.logits = new(s.T, s.E)
        self.topk_idx, self.topk_w = new(s.T, s.top_k, dt=i32), new(s.T, s.top_k)
        self.routed_counts, self.P, self.aux = new(s.E, dt=i32), new(s.E), new(1)
        self.kept_counts, self.offsets = new(s.E, dt=i32), new(s.E + 1, dt=i32)
        self.dest_row, self.src_token = new(s.T, s.top_k, dt=i32), new(rows, dt=i32)
        self.x_perm, self.act, self.y_perm = (new(rows, n, dt=bf16) for n in (s.H, s.h, s.H))
        packed = lambda n: (new(rows, n // 2, dt=u8), new((n + 127) // 128, rows, 4, dt=u8))
        self.x_q, self.x_scale = packed(s.H)
        self.act_q, self.act_scale = packed(s.h)

    def forward(self, x: torch.Tensor, gate: torch.Tensor, y: torch.Tensor,
                gate_bias: Optional[torch.Tensor] = None,
                select_bias: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y [T, H] = the layer of x [T, H] (bf16). gate_bias is part of the
        logits, select_bias acts on the choice of experts alone."""
        s, ws, st = self.shape, self.ws, self.dev_status
        if s.T == 0:  # empty tensors have no address to pass
            for t in (self.routed_counts, self.P, self.aux, self.kept_counts, self.offsets):
                t.zero_()
            return y
        moe_route(s, x, gate, gate_bias, self.topk_idx, self.topk_w, logits_out=self.logits,
                  dev_status=st, ws=ws)
        moe_route_grouped(s, self.config, self.logits, select_bias, self.topk_idx, self.topk_w,
                          routed_counts=self.routed_counts, P=self.P, aux=self.aux,
                          dev_status=st, ws=ws)
        moe_permute(s, x, self.topk_idx, self.kept_counts, self.offsets, self.dest_row,
                    self.src_token, self.x_perm, dev_status=st, ws=ws)
        w, kept = self.weights, self.offsets[s.E:]
        moe_quantize_rows_mx4(self.x_perm, self.x_q, self.x_scale, n_rows=kept)
        moe_expert_gemm_mx4(self.x_q, self.x_scale, self.offsets, w.W1q, w.w1_scale, self.act,
                            gelu=True, dev_status=st)
        moe_quantize_rows_mx4(self.act, self.act_q, self.act_scale, n_rows=kept)
        moe_expert_gemm_mx4(self.act_q, self.act_scale, self.offsets, w.W2q, w.w2_scale,
                            self.y_perm, dev_status=st)
        moe_combine(s, self.y_perm, self.dest_row, self.topk_w, y)
        return y

    def router_grad(self, grad_topk_w: torch.Tensor, grad_logits: torch.Tensor,
                    grad_aux: Optional[torch.Tensor] = None) -> torch.Tensor:
        """grad_logits [T, E] from the gradients of topk_w [T, k] and of aux
        [1], for the routing of the last forward()."""
        if self.shape.T == 0:
            return grad_logits
        moe_route_grouped_bwd(self.shape, self.config, self.logits, self.topk_idx, grad_topk_w,
                              grad_logits, grad_aux=grad_aux,
                              routed_counts=self.routed_counts if grad_aux is not None else None)
        return grad_logits


def main() -> None:
    T, H, E, k, h = 2048, 512, 64, 6, 256
    g = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *n, std=1.0: (std * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)
    x, gate = draw(T, H), draw(H, E, std=H ** -0.5)
    W1, W2 = draw(E, H, h, std=H ** -0.5), draw(E, h, H, std=h ** -0.5)
    config = RouteConfig.make("sigmoid", n_groups=8, topk_groups=3, group_top=2, scale=2.5)
    layer = Mx4Layer(MoeShape.make(T, H, E, k, h, 1.25), config, W1, W2)
    y = torch.empty_like(x)
    layer.forward(x, gate, y, select_bias=0.01 * torch.randn(E, generator=g, device="cuda"))
    grad = layer.router_grad(torch.ones_like(layer.topk_w), torch.empty_like(layer.logits),
                             grad_aux=torch.full((1,), 0.01, device="cuda"))
    torch.cuda.synchronize()
    print(f"tokens {T}, experts {E}: aux {layer.aux.item():.4f}, "
          f"kept rows {layer.offsets[E].item()} of {T * k}, |y| {y.float().norm().item():.2f}, "
          f"|grad logits| {grad.norm().item():.3e}, status {layer.dev_status.item()}")


if __name__ == "__main__":
    main()

"""One MoE block trained for a few steps, every hot operator a call of this library:

    y = layer_norm(x);  logits = y Wg^T;  ids, w, counts, balance = moe_gate(logits)
    D = the experts' grouped FP8 GEMM over the routed, quantised rows;  out = x + combine(D, w)
    loss = mean (out - target)^2 / 2 + balance

and the gradient of all of it: combine, the grouped data and weight gradients with e5m2 dY, gate, layer norm; then the
global norm of the gradients, clipping, and a plain SGD step.  The router's matrix product (a few experts wide)
and the transposes for the weight gradient are torch's.

    python examples/moe_block_training.py [--steps 10] [--tokens 2048] [--hidden 1024] [--experts 8] [--topk 2]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_block_gb300 as g  # noqa: E402


class MoEBlock:
    """The parameters (fp32 masters) and one step's forward and backward pass."""

    def __init__(self, hidden: int, experts: int, topk: int, seed: int = 0, loss_coef: float = 0.01):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.topk, self.loss_coef = topk, loss_coef
        self.weight = torch.ones(hidden, device="cuda")
        self.bias = torch.zeros(hidden, device="cuda")
        self.router = torch.randn((experts, hidden), generator=gen, device="cuda") / hidden ** 0.5
        self.experts = torch.randn((experts, hidden, hidden), generator=gen, device="cuda") / hidden ** 0.5
        # the gradients stay in these buffers, so they are listed once
        self.d_experts = torch.empty(self.experts.shape, dtype=torch.bfloat16, device="cuda")
        self.d_router, self.d_weight, self.d_bias = (torch.empty_like(t) for t in (self.router, self.weight, self.bias))
        self.grads = g.GradList([self.d_experts, self.d_router, self.d_weight, self.d_bias])

    def forward(self, x, token_mask=None):
        """x f32 [T, hidden] -> (out f32 [T, hidden], the balance loss f32 [1], what backward needs)."""
        E = self.experts.shape[0]
        y, mean, rstd = g.layer_norm(x, self.weight, self.bias, out_dtype=torch.bfloat16)
        logits = y.float() @ self.router.t()
        ids, w, counts, balance = g.moe_gate(logits, self.topk, loss_coef=self.loss_coef, token_mask=token_mask)
        q, s, offsets, row_token, entry_row = g.route_gather_quantize_1x128(y, ids, E)
        qw, sw = g.quantize_128x128(self.experts.bfloat16())
        D = torch.empty((q.shape[0], self.experts.shape[1]), dtype=torch.bfloat16, device=x.device)
        g.fp8_grouped_gemm_contiguous(q, s, qw, sw, D, offsets)
        out = g.moe_combine(D, entry_row, w, residual=x)
        return out, balance, (x, y, mean, rstd, logits, ids, w, counts, offsets, row_token, entry_row, D, token_mask)

    def backward(self, dout, saved):
        """dout f32 [T, hidden], and 1 for the balance loss -> dx f32; the parameters' gradients in their buffers."""
        x, y, mean, rstd, logits, ids, w, counts, offsets, row_token, entry_row, D, token_mask = saved
        dD, dw = g.moe_combine_backward(dout, D, entry_row, row_token, w)
        # the data gradient dD W and, over each expert's rows, the weight gradient dD^T X
        qd, sd = g.quantize_1x128_e5m2(dD)
        qt, st = g.quantize_128x128(self.experts.transpose(1, 2).contiguous().bfloat16())
        dX = torch.empty((dD.shape[0], y.shape[1]), dtype=torch.bfloat16, device=x.device)
        g.fp8_grouped_gemm_contiguous_dgrad(qd, sd, qt, st, dX, offsets)
        X = y[row_token.clamp(min=0).long()] * (row_token >= 0)[:, None]
        qdt, sdt = g.quantize_1x128_e5m2(dD.t().contiguous())
        qxt, sxt = g.quantize_1x128(X.t().contiguous())
        g.fp8_grouped_gemm_wgrad(qdt, sdt, qxt, sxt, self.d_experts, offsets)
        # the gradient of the gather is the combine without weights; of the choice, the gate's
        dlogits = g.moe_gate_backward(logits, ids, counts, dw, torch.ones(1, device=x.device), loss_coef=self.loss_coef,
                                      token_mask=token_mask)
        dy = g.moe_combine(dX, entry_row, residual=dlogits @ self.router)
        torch.matmul(dlogits.t(), y.float(), out=self.d_router)
        dx = torch.empty_like(x)
        g.fp8g_layer_norm_backward(dy, x, self.weight, mean, rstd, dx, self.d_weight, self.d_bias)
        return dx.add_(dout)

    def update(self, rate: float, max_norm: float) -> torch.Tensor:
        norm = g.clip_grad_norm(self.grads, max_norm)
        for p, d in zip((self.experts, self.router, self.weight, self.bias), self.grads.grads):
            p.add_(d.float(), alpha=-rate)
        return norm


def train(steps: int, tokens: int, hidden: int, experts: int, topk: int, rate: float = 20.0, max_norm: float = 1.0,
          seed: int = 0, verbose: bool = False):
    """-> [(loss, balance loss, gradient norm)] of the steps, on one fixed batch of synthetic tokens."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((tokens, hidden), generator=gen, device="cuda")
    target = x + 0.5 * torch.tanh(x.roll(1, 1))
    block = MoEBlock(hidden, experts, topk, seed)
    log = []
    for step in range(steps):
        out, balance, saved = block.forward(x)
        diff = out - target
        loss = diff.square().mean() / 2
        block.backward(diff / diff.numel(), saved)
        norm = block.update(rate, max_norm)
        log.append((float(loss), float(balance), float(norm)))
        if verbose:
            print("step %2d  loss %.5f  balance %.5f  gradient norm %.5f" % (step, *log[-1]))
    status = g.fp8g_get_status()
    if status:
        raise g.Fp8GemmError(status, "training step")
    return log


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 10), ("tokens", 2048), ("hidden", 1024), ("experts", 8), ("topk", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    train(a.steps, a.tokens, a.hidden, a.experts, a.topk, verbose=True)

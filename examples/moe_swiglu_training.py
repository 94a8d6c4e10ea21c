"""A MoE block with gated experts trained for a few steps, every hot operator a call of this library:

    y = rms_norm(x) w;  logits = y Wr^T;  ids, p = moe_route(logits, bias)       (sigmoid scores, groups, balance bias)
    gu = the experts' first grouped FP8 GEMM over the routed, quantised rows;  a = swiglu(gu), quantised
    f = combine(the second grouped GEMM of a, p)
    h = x + scale gate (rms_norm(f) post);  z = rms_norm(h) w_next               (the next block's input)
    loss = mean (z - target)^2 / 2

and the gradient of all of it, with e5m2 gradients through the grouped GEMMs; then the gradients' global norm and one
AdamW step that clips by it, on bf16 experts with fp32 masters and 8-bit states, and the balance bias' own step.  The
router's matrix product (a few experts wide) and the transposes for the weight gradients are torch's.

    python examples/moe_swiglu_training.py [--steps 10] [--tokens 2048] [--hidden 1024] [--inner 512] [--experts 16] [--topk 4]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_block_gb300 as g  # noqa: E402

BF16 = torch.bfloat16


class GatedMoEBlock:
    """The parameters and one step's forward and backward pass."""

    def __init__(self, hidden: int, inner: int, experts: int, topk: int, groups: int = 4, topk_groups: int = 2,
                 seed: int = 0, state_bits: int = 8):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
        self.route = dict(score="sigmoid", renormalize=True, scale=1.0)
        self.groups, self.topk_groups, self.topk, self.scale = groups, topk_groups, topk, 0.5
        self.bias = torch.zeros(experts, device="cuda")  # moved by the counts, not by a gradient
        self.weight, self.post, self.next_weight = (torch.ones(hidden, device="cuda") for _ in range(3))
        self.gate = torch.full((hidden,), 0.5, device="cuda")
        self.router = rand(experts, hidden) / hidden ** 0.5
        self.w_in = (rand(experts, 2 * inner, hidden) / hidden ** 0.5).to(BF16)
        self.w_out = (rand(experts, hidden, inner) / inner ** 0.5).to(BF16)
        self.params = [self.w_in, self.w_out, self.router, self.weight, self.post, self.gate, self.next_weight]
        # the gradients stay in these buffers, so everything is listed once
        self.grads = [torch.empty_like(p) for p in self.params]
        (self.d_in, self.d_out, self.d_router, self.d_weight, self.d_post, self.d_gate, self.d_next) = self.grads
        self.list = g.GradList(self.grads)
        self.opt = g.AdamWList(self.params, self.grads, masters=True, state_bits=state_bits,
                               weight_decay=[0.1, 0.1, 0.0, 0.0, 0.0, 0.0, 0.0])

    def forward(self, x, token_mask=None):
        """x f32 [T, hidden] -> (z bf16 [T, hidden], what backward needs)."""
        E = self.router.shape[0]
        _, y, rstd, _ = g.residual_rms_norm(x, None, self.weight, out_dtype=BF16)
        logits = y.float() @ self.router.t()
        ids, p, counts = g.moe_route(logits, self.topk, bias=self.bias, groups=self.groups, topk_groups=self.topk_groups,
                                     token_mask=token_mask, **self.route)
        q, s, offsets, row_token, entry_row = g.route_gather_quantize_1x128(y, ids, E)
        M = q.shape[0]
        gu = torch.zeros((M, self.w_in.shape[1]), dtype=BF16, device=x.device)  # rows of no expert stay zero
        g.fp8_grouped_gemm_contiguous(q, s, *g.quantize_128x128(self.w_in), gu, offsets)
        qa, sa, _ = g.swiglu_quantize_1x128(gu, ld_sa=M)
        D = torch.empty((M, self.w_out.shape[1]), dtype=BF16, device=x.device)
        g.fp8_grouped_gemm_contiguous(qa, sa, *g.quantize_128x128(self.w_out), D, offsets)
        f = g.moe_combine(D, entry_row, p)
        h, z, rstd_h, rstd_f = g.residual_rms_norm(x, f, self.next_weight, gate=self.gate, scale=self.scale,
                                                   post_norm=True, post_weight=self.post)
        return z, (x, y, rstd, logits, ids, p, counts, offsets, row_token, entry_row, gu, D, f, h, rstd_h, rstd_f, token_mask)

    def backward(self, dz, saved):
        """dz bf16 [T, hidden] -> dx f32; the parameters' gradients in their buffers."""
        (x, y, rstd, logits, ids, p, counts, offsets, row_token, entry_row, gu, D, f, h, rstd_h, rstd_f, mask) = saved
        dx, df = torch.empty_like(x), torch.empty_like(f)
        g.fp8g_residual_rms_norm_backward(dz, None, h, f, rstd_h, rstd_f, self.next_weight, dx, df, self.d_next, self.d_gate,
                                          self.d_post, gate=self.gate, scale=self.scale, post_norm=True,
                                          post_weight=self.post)
        dD, dp = g.moe_combine_backward(df, D, entry_row, row_token, p)
        # the second product's data gradient, the activation's, and over each expert's rows the weight gradient
        da = self._data_gradient(dD, self.w_out, offsets)
        dgu, a = g.swiglu_backward(da, gu)
        self._weight_gradient(dD, a, self.d_out, offsets)
        dX = self._data_gradient(dgu, self.w_in, offsets)
        X = y[row_token.clamp(min=0).long()] * (row_token >= 0)[:, None]
        self._weight_gradient(dgu, X, self.d_in, offsets)
        dlogits = g.moe_route_backward(logits, ids, dp, token_mask=mask, **self.route)
        dy = g.moe_combine(dX, entry_row, residual=dlogits @ self.router)  # the gradient of the gather
        torch.matmul(dlogits.t(), y.float(), out=self.d_router)
        g.fp8g_residual_rms_norm_backward(dy, dx, x, None, rstd, None, self.weight, dx, dweight=self.d_weight)
        return dx

    def _data_gradient(self, d, weight, offsets):
        """d [M, N] times each expert's weight [N, K] -> [M, K]."""
        out = torch.empty((d.shape[0], weight.shape[2]), dtype=BF16, device=d.device)
        g.fp8_grouped_gemm_contiguous_dgrad(*g.quantize_1x128_e5m2(d), *g.quantize_128x128(weight.transpose(1, 2).contiguous()),
                                            out, offsets)
        return out

    def _weight_gradient(self, d, rows, out, offsets):
        """Over each expert's rows: d^T rows."""
        g.fp8_grouped_gemm_wgrad(*g.quantize_1x128_e5m2(d.t().contiguous()), *g.quantize_1x128(rows.t().contiguous()), out,
                                 offsets)

    def update(self, rate: float, max_norm: float, counts, balance: float = 1e-3) -> torch.Tensor:
        norm = g.grad_norm(self.list)
        g.adamw_step(self.opt, rate, beta2=0.95, norm=norm, max_norm=max_norm)
        load = counts.float()
        self.bias.add_(torch.sign(load.mean() - load), alpha=balance)
        return norm


def train(steps: int, tokens: int, hidden: int, inner: int, experts: int, topk: int, rate: float = 3e-3,
          max_norm: float = 1.0, seed: int = 0, verbose: bool = False):
    """-> [(loss, gradient norm)] of the steps, on one fixed batch of synthetic tokens."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((tokens, hidden), generator=gen, device="cuda")
    target = torch.tanh(x.roll(1, 1))
    block = GatedMoEBlock(hidden, inner, experts, topk, seed=seed)
    log = []
    for step in range(steps):
        z, saved = block.forward(x)
        diff = z.float() - target
        block.backward((diff / diff.numel()).to(BF16), saved)
        norm = block.update(rate, max_norm, saved[6])
        log.append((float(diff.square().mean() / 2), float(norm)))
        if verbose:
            print("step %2d  loss %.5f  gradient norm %.5f" % (step, *log[-1]))
    status = g.fp8g_get_status()
    if status:
        raise g.Fp8GemmError(status, "training step")
    return log


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 10), ("tokens", 2048), ("hidden", 1024), ("inner", 512), ("experts", 16), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    train(a.steps, a.tokens, a.hidden, a.inner, a.experts, a.topk, verbose=True)

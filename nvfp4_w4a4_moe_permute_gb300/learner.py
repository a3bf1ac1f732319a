"""One policy-update step of a learner whose expert MLP runs its forward in
NVFP4 and its backward in BF16 (the split of the learner paths that the miniTE
report summary measures, section "Respect the timing boundaries").

The model is one MoE layer with a residual and an output head:

    y      = x + MoE(x)                         NVFP4 W4A4 (MoEMLP's entry points)
    logits = y head^T                           BF16 product, one expert
    loss   = -mean(advantage * logprob(token)) - entropy_bonus * mean(entropy)

and a step is forward, loss, BF16 backward, the gradients' norm and clipping factor,
AdamW on FP32 master weights, and the requantization of the new weights:

    python -m nvfp4_w4a4_moe_permute_gb300.learner --steps 8

Every product, softmax, movement of rows, optimizer step and quantization runs in the
library's kernels; torch provides memory and the residual sum.
"""
from __future__ import annotations

import argparse

import torch

from . import minite as M


class PolicyLearner:
    """Weights, their NVFP4 copies, the optimizer and the buffers of one shape
    (T tokens, hidden H, expert intermediate I, E experts, top-k, V tokens)."""

    def __init__(self, T, H, I, E, k, V, lr=1e-3, entropy_bonus=0.0, temperature=1.0,
                 state_bits=8, weight_decay=0.0, seed=0, device="cuda"):
        self.T, self.H, self.I, self.E, self.k, self.V = T, H, I, E, k, V
        self.entropy_bonus, self.temperature = entropy_bonus, temperature
        d = torch.device(device)
        g = torch.Generator(device=d).manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=g, device=d) * shape[-1] ** -0.5

        # FP32 master weights and the BF16 copies that every kernel reads
        self.master = [weight(E, 2 * I, H), weight(E, H, I), weight(V, H)]
        self.wgu, self.wd, self.head = [w.to(torch.bfloat16) for w in self.master]
        self.optimizer = M.AdamW(self.master, copies=[self.wgu, self.wd, self.head], lr=lr,
                                 betas=(0.9, 0.95), weight_decay=weight_decay, state_bits=state_bits)
        self.grads = [torch.zeros_like(w) for w in self.master]
        self.mlp = M.MoEMLP(T, H, I, E, k, d)
        rows = T * k
        bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        self.h = torch.empty((rows, I), dtype=bf, device=d)
        self.dgu = torch.empty((rows, 2 * I), dtype=bf, device=d)
        # the SwiGLU backward's NVFP4 outputs, which the BF16 backward does not use
        self.dgu_q = (torch.empty((rows, I), dtype=u8, device=d),
                      torch.empty(M.sf_bytes(rows + 128 * E, 2 * I), dtype=u8, device=d),
                      torch.empty(rows, dtype=f32, device=d))
        self.logits = torch.empty((T, V), dtype=bf, device=d)
        self.dx_rows = torch.empty((rows, H), dtype=bf, device=d)
        self.in_order = torch.empty((rows, H), dtype=bf, device=d)   # dy, then x, in expert order
        self.all_rows = torch.tensor([0, T], dtype=torch.int32, device=d)
        self.status = self.mlp.status
        self.requantize()

    def requantize(self):
        """The forward's NVFP4 copies of the expert weights, one scale an expert."""
        self.wgu_q = M.quantize(self.wgu, per_group=True)
        self.wd_q = M.quantize(self.wd, per_group=True)

    def forward(self, x, topk_ids, topk_w, tokens, alternatives=0):
        """x [T, H] bf16, topk_ids int32 and topk_w fp32 [T, k], tokens int32 [T]
        (negative: no loss); returns token_logprobs' result."""
        mlp, st = self.mlp, self.status
        mlp.permute_quant(x, topk_ids, topk_w)
        M.minite_grouped_gemm_nvfp4(mlp.a_codes, mlp.a_sf, mlp.a_g, self.wgu_q["codes"],
                                    self.wgu_q["sf"], self.wgu_q["g"], mlp.offsets, mlp.sf_offsets,
                                    mlp.gate_up, st)
        M.minite_swiglu_weighted_quant_keep_h(mlp.gate_up, mlp.perm_w, self.E, mlp.offsets,
                                              mlp.sf_offsets, mlp.h_codes, mlp.h_sf, mlp.h_g, self.h,
                                              st)
        M.minite_grouped_gemm_nvfp4(mlp.h_codes, mlp.h_sf, mlp.h_g, self.wd_q["codes"],
                                    self.wd_q["sf"], self.wd_q["g"], mlp.offsets, mlp.sf_offsets,
                                    mlp.down, st)
        M.minite_moe_combine(mlp.down, mlp.dest_row, mlp.y, st)
        self.y = x + mlp.y
        M.grouped_gemm_bf16(self.y, self.head.view(1, self.V, self.H), self.all_rows, out=self.logits,
                            status=st)
        return M.token_logprobs(self.logits, tokens, self.temperature, alternatives, status=st)

    def backward(self, x, tokens, out, grad_logprob, grad_entropy, accumulate=False):
        """Gradients of the weights into ``grads`` (added with ``accumulate``:
        one more micro-batch); returns the gradient of x. The logits' buffer
        becomes their gradient."""
        mlp, st = self.mlp, self.status
        d = M.token_logprobs_backward(self.logits, tokens, out, grad_logprob, grad_entropy,
                                      self.temperature, out=self.logits, status=st)
        gwgu, gwd, ghead = self.grads
        M.grouped_wgrad_bf16(d, self.y, self.all_rows, out=ghead.view(1, self.V, self.H),
                             accumulate=accumulate, status=st)
        dy = M.grouped_gemm_bf16(d, self.head.view(1, self.V, self.H), self.all_rows, w_as_stored=True,
                                 status=st)
        dd = M.spread_rows(dy, mlp.dest_row, self.in_order, status=st)   # the combine's backward
        M.grouped_wgrad_bf16(dd, self.h, mlp.offsets, out=gwd, accumulate=accumulate, status=st)
        dh = M.grouped_gemm_bf16(dd, self.wd, mlp.offsets, w_as_stored=True, status=st)
        M.minite_swiglu_backward_quant_keep(mlp.gate_up, dh, mlp.perm_w, self.E, mlp.offsets,
                                            mlp.sf_offsets, *self.dgu_q, self.dgu, st)
        x_rows = M.spread_rows(x, mlp.dest_row, self.in_order, status=st)
        M.grouped_wgrad_bf16(self.dgu, x_rows, mlp.offsets, out=gwgu, accumulate=accumulate, status=st)
        M.grouped_gemm_bf16(self.dgu, self.wgu, mlp.offsets, w_as_stored=True, out=self.dx_rows, status=st)
        dx = torch.empty_like(x)
        M.minite_moe_combine(self.dx_rows, mlp.dest_row, dx, st)
        return dx + dy

    def step(self, x, topk_ids, topk_w, tokens, advantages, grad_scale=None, max_grad_norm=None):
        """Forward, backward, optimizer step and requantization; returns the
        forward's result. ``advantages`` fp32 [T]. With ``max_grad_norm`` the
        gradients' global norm is clipped to it (its value, a device scalar, is
        ``grad_norm`` of the result), in place of a ``grad_scale``."""
        if grad_scale is not None and max_grad_norm is not None:
            raise M.MiniteError("PolicyLearner.step: either grad_scale or max_grad_norm")
        out = self.forward(x, topk_ids, topk_w, tokens)
        n = self.T
        self.backward(x, tokens, out, advantages * (-1.0 / n),
                      torch.full_like(advantages, -self.entropy_bonus / n) if self.entropy_bonus else None)
        if max_grad_norm is not None:
            r = M.grad_norm(self.grads, max_grad_norm)
            grad_scale, out["grad_norm"] = r["scale"], r["norm"]
        self.optimizer.step(self.grads, grad_scale=grad_scale)
        self.requantize()
        return out


def synthetic_batch(T, H, E, k, V, seed=0, device="cuda"):
    """Inputs of a step: hidden states, top-k softmax routing of normal logits,
    sampled tokens and advantages."""
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=device).to(torch.bfloat16)
    score = torch.softmax(torch.randn(T, E, generator=g, device=device), 1)
    w, ids = torch.sort(score, dim=1, descending=True, stable=True)
    w, ids = w[:, :k].contiguous(), ids[:, :k].to(torch.int32).contiguous()
    tokens = torch.randint(0, V, (T,), generator=g, device=device, dtype=torch.int32)
    return x, ids, w / w.sum(1, keepdim=True), tokens, torch.rand(T, generator=g, device=device)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inter", 768), ("experts", 128),
                        ("topk", 8), ("vocab", 32768), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--max-grad-norm", type=float, default=None)
    a = ap.parse_args()
    learner = PolicyLearner(a.tokens, a.hidden, a.inter, a.experts, a.topk, a.vocab)
    x, ids, w, tokens, adv = synthetic_batch(a.tokens, a.hidden, a.experts, a.topk, a.vocab)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for i in range(a.steps):
        begin.record()
        out = learner.step(x, ids, w, tokens, adv, max_grad_norm=a.max_grad_norm)
        end.record()
        end.synchronize()
        print(f"step {i}: mean advantage * logprob {(adv * out['logprob']).mean().item():.4f}, "
              f"entropy {out['entropy'].mean().item():.3f}, {begin.elapsed_time(end):.2f} ms, "
              f"device status {int(learner.status.item())}"
              + (f", gradient norm {out['grad_norm'].item():.4f}" if "grad_norm" in out else ""))


if __name__ == "__main__":
    main()

"""The feed-forward half of a block around a mixture-of-experts MLP, with norms
before and after it: trained in bf16, its products optionally in fp8 with a
scale per block of 128, and served in fp8.

For residual rows r (sorted by expert), router gates and expert counts:
  n   = N(r; w_in)                      norm_residual_fwd
  h   = silu(g) u,  [g | u] = n W1^T    ragged_gemm_fprop_swiglu    (fp8: fp8_gemm_fprop, swiglu_fwd)
  y   = h W2^T                          ragged_gemm_fprop           (fp8: fp8_gemm_fprop)
  r'  = r + c gate N(y; w_post)         norm_residual_fwd, and with it
  n'  = N(r'; w_out)                    the next half's input
backward from dr' and dn':
  dy, dr, dgate, dw_post, dw_out        norm_residual_bwd
  [dg | du], h again                    ragged_gemm_dgrad_swiglu    (fp8: fp8_gemm_dgrad, swiglu_bwd)
  dn, dW1, dW2                          ragged_gemm_dgrad, _wgrad   (fp8: fp8_gemm_dgrad; dW stays in bf16)
  dr, dw_in                             norm_residual_bwd

Run: python examples/feed_forward_block.py   (needs a GB300)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_grouped_group_gb300 as mxq  # noqa: E402

BF16 = torch.bfloat16


class Block:
    """E gated experts of width H -> F -> H between two norms; bf16 weights."""

    def __init__(self, E, H, F, scale=0.5, seed=0, fp8=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
        one = lambda: (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16)  # noqa: E731
        self.w1, self.w2 = r(E, 2 * F, H, std=H ** -0.5), r(E, H, F, std=F ** -0.5)
        self.w_in, self.w_post, self.w_out = one(), one(), one()
        self.scale, self.fp8 = scale, fp8

    def forward(self, r, gate, m_splits):
        _, n, st_in = mxq.norm_residual_fwd(r, pre_weight=self.w_in, res_out=False)
        if self.fp8:
            w1, w2 = mxq.fp8_quantize_weight(self.w1), mxq.fp8_quantize_weight(self.w2)
            y1 = mxq.fp8_gemm_fprop(*mxq.fp8_quantize_rows(n), *w1, m_splits)
            h = mxq.swiglu_fwd(y1)
            y = mxq.fp8_gemm_fprop(*mxq.fp8_quantize_rows(h), *w2, m_splits)
        else:
            w1 = w2 = None
            h, y1 = mxq.ragged_gemm_fprop_swiglu(n, self.w1, m_splits, y_out=True)
            y = mxq.ragged_gemm_fprop(h, self.w2, m_splits)
        r2, n2, st_out = mxq.norm_residual_fwd(y, r, post_weight=self.w_post, pre_weight=self.w_out, gate=gate,
                                               scale=self.scale)
        return r2, n2, (r, gate, n, st_in, y1, y, r2, st_out, w1, w2)

    def backward(self, dr2, dn2, saved, m_splits):
        """The gradients of r, gate and the weights, by name."""
        r, gate, n, st_in, y1, y, r2, st_out, w1, w2 = saved
        out = mxq.norm_residual_bwd(dr2, dn2, y, r2, st_out, self.w_post, self.w_out, gate, self.scale)
        dy = out["dx"]
        if self.fp8:
            dy1 = mxq.swiglu_bwd(mxq.fp8_gemm_dgrad(*mxq.fp8_quantize_rows(dy), *w2, m_splits), y1)
            h = mxq.swiglu_fwd(y1)
            dn = mxq.fp8_gemm_dgrad(*mxq.fp8_quantize_rows(dy1), *w1, m_splits)
        else:
            dy1, h = mxq.ragged_gemm_dgrad_swiglu(dy, self.w2, y1, m_splits, h_out=True)
            dn = mxq.ragged_gemm_dgrad(dy1, self.w1, m_splits)
        grads = {"w2": mxq.ragged_gemm_wgrad(dy, h, m_splits), "w1": mxq.ragged_gemm_wgrad(dy1, n, m_splits),
                 "w_post": out["dpost_weight"], "w_out": out["dpre_weight"], "gate": out["dgate"]}
        first = mxq.norm_residual_bwd(out["dresidual"], dn, None, r, st_in, pre_weight=self.w_in, dx_out=False)
        grads["r"], grads["w_in"] = first["dresidual"], first["dpre_weight"]
        return grads

    def serve(self, weights, r, gate, m_splits):
        """A few tokens through codes and scales of W1 and W2, r updated in place; the next half's input."""
        (w1, s1), (w2, s2) = weights
        _, n, _ = mxq.norm_residual_fwd(r, pre_weight=self.w_in, res_out=False, stats_out=False)
        y1 = mxq.fp8_gemm_fprop(*mxq.fp8_quantize_rows(n), w1, s1, m_splits)
        y = mxq.fp8_gemm_fprop(*mxq.fp8_quantize_rows(mxq.swiglu_fwd(y1)), w2, s2, m_splits)
        return mxq.norm_residual_fwd(y, r, post_weight=self.w_post, pre_weight=self.w_out, gate=gate, scale=self.scale,
                                     stats_out=False, out=(r, None, None))[1]


def main(E=4, H=512, F=256, M=1536, steps=5, lr=0.02):
    g = torch.Generator(device="cuda").manual_seed(7)
    r = torch.randn(M, H, generator=g, device="cuda").to(BF16)
    gate = torch.rand(M, generator=g, device="cuda")
    target = torch.tanh(r.float().roll(1, dims=1)).to(BF16)
    counts = torch.bincount(torch.randint(0, E * E, (M,), generator=g, device="cuda") // E % E, minlength=E)
    losses = {}
    for fp8 in (False, True):
        block, losses[fp8] = Block(E, H, F, fp8=fp8), []
        for _ in range(steps):
            r2, n2, saved = block.forward(r, gate, counts)
            diff = n2.float() - target.float()
            losses[fp8].append((diff * diff).mean().item())
            grads = block.backward(torch.zeros_like(r2), (diff * (2.0 / M)).to(BF16), saved, counts)
            for name in ("w1", "w2", "w_in", "w_post", "w_out"):
                w = getattr(block, name)
                w.copy_(w.float() - lr * grads[name])
        print("%s: loss %.4f -> %.4f" % ("fp8 " if fp8 else "bf16", losses[fp8][0], losses[fp8][-1]))
    few = torch.tensor([3, 0, 1, 4], dtype=torch.int64, device="cuda")
    tokens, weights = r[:8].clone(), (mxq.fp8_quantize_weight(block.w1), mxq.fp8_quantize_weight(block.w2))
    n2 = block.serve(weights, tokens, gate[:8].contiguous(), few)
    print("served 8 tokens in fp8, next input %s" % (tuple(n2.shape),))
    return losses, n2


if __name__ == "__main__":
    main()

"""A small mixture-of-experts MLP in bf16, trained for a few steps and then
served in int8, on the ragged operators of the library.

Training (all expert counts as a router gives them, no padding):
  y1 = X W1^T + b1           ragged_gemm_fprop
  h  = D(silu(g) u)          swiglu_dropout_fwd        [g | u] = y1
  y  = h W2^T                ragged_gemm_fprop
  o  = X + D(y)              dropout with the residual
backward, with every mask made again from {seed, offset}:
  dy = D(do)                 dropout
  dh, dW2                    ragged_gemm_dgrad, ragged_gemm_wgrad (fp32)
  dy1                        swiglu_dropout_bwd
  dX, dW1                    ragged_gemm_dgrad, ragged_gemm_wgrad
Serving: weights quantized once per output channel, tokens per row
  (int8_quantize_rows, int8_gemm_fprop), a step of a few tokens at a time.

Run: python examples/ragged_expert_mlp.py   (needs a GB300)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_grouped_group_gb300 as mxq  # noqa: E402

BF16 = torch.bfloat16


class ExpertMLP:
    """E experts of width H -> F (SwiGLU) -> H with dropout p, fp32 master weights."""

    def __init__(self, E, H, F, p, seed=0, lr=0.05):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
        self.w1, self.w2 = r(E, 2 * F, H, std=H ** -0.5), r(E, H, F, std=F ** -0.5)
        self.E, self.H, self.F, self.p, self.lr = E, H, F, p, lr
        # one {seed, offset} per dropout site; the offset is advanced on the device after each step
        self.rng = [torch.tensor([seed + 1 + i, 0], dtype=torch.int64, device="cuda") for i in range(2)]
        self.dw1, self.dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)

    def forward(self, x, m_splits, train):
        p = self.p if train else 0.0
        w1, w2 = self.w1.to(BF16), self.w2.to(BF16)
        y1 = mxq.ragged_gemm_fprop(x, w1, m_splits)
        h = mxq.swiglu_dropout_fwd(y1, self.rng[0], p)
        y = mxq.ragged_gemm_fprop(h, w2, m_splits)
        return mxq.dropout(y, self.rng[1], p, residual=x), (x, w1, w2, y1, h)

    def backward(self, do, saved, m_splits):
        x, w1, w2, y1, h = saved
        dy = mxq.dropout(do, self.rng[1], self.p)
        dh = mxq.ragged_gemm_dgrad(dy, w2, m_splits)
        mxq.ragged_gemm_wgrad(dy, h, m_splits, out=self.dw2)
        dy1 = mxq.swiglu_dropout_bwd(dh, y1, self.rng[0], self.p)
        mxq.ragged_gemm_wgrad(dy1, x, m_splits, out=self.dw1)
        return do + mxq.ragged_gemm_dgrad(dy1, w1, m_splits)

    def step(self, x, target, m_splits):
        out, saved = self.forward(x, m_splits, train=True)
        diff = out.float() - target.float()
        self.backward((diff * (2.0 / diff.numel())).to(BF16), saved, m_splits)
        for w, dw in ((self.w1, self.dw1), (self.w2, self.dw2)):
            w.add_(dw, alpha=-self.lr * diff.numel() / diff.shape[0])
        for r in self.rng:
            r[1] += 1
        return (diff * diff).mean()

    def quantized(self):
        """int8 codes and one scale per output channel of both weights."""
        def q(w):
            E, N, K = w.shape
            codes, scale = mxq.int8_quantize_rows(w.to(BF16).view(E * N, K))
            return codes.view(E, N, K), scale.view(E, N)
        return q(self.w1), q(self.w2)


def serve(weights, x, m_splits, rng):
    """One int8 step of the layer for a few tokens."""
    (w1, s1), (w2, s2) = weights
    y1 = mxq.int8_gemm_fprop(*mxq.int8_quantize_rows(x), w1, s1, m_splits)
    h = mxq.swiglu_dropout_fwd(y1, rng, 0.0)
    y = mxq.int8_gemm_fprop(*mxq.int8_quantize_rows(h), w2, s2, m_splits)
    return mxq.dropout(y, rng, 0.0, residual=x)


def main(E=4, H=512, F=256, M=1536, steps=30, p=0.1):
    mlp = ExpertMLP(E, H, F, p)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(M, H, generator=g, device="cuda").to(BF16)
    target = (x.float() + torch.tanh(x.float().roll(1, dims=1))).to(BF16)
    counts = torch.bincount(torch.randint(0, E * E, (M,), generator=g, device="cuda") // E % E, minlength=E)
    losses = [mlp.step(x, target, counts).item() for _ in range(steps)]
    print("loss %.4f -> %.4f over %d steps, rows per expert %s" % (losses[0], losses[-1], steps, counts.tolist()))

    weights = mlp.quantized()
    few = torch.tensor([3, 0, 1, 4], dtype=torch.int64, device="cuda")
    tokens = x[:8].contiguous()
    ref, _ = mlp.forward(tokens, few, train=False)
    out = serve(weights, tokens, few, mlp.rng[0])
    err = ((out.float() - ref.float()).norm() / (ref.float() - tokens.float()).norm()).item()
    print("int8 serving of 8 tokens: %.4f of the layer's update off (relative 2-norm)" % err)
    return losses, err


if __name__ == "__main__":
    main()

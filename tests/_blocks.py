"""Plain 64-bit definitions of the block-scaled fp8 products and of a block's
norms, and the tolerances that the GPU tests state their results in."""
import torch

U = 2.0 ** -24  # fp32's unit roundoff
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value
E4M3 = torch.float8_e4m3fn


def codes(v, top):
    """e4m3 codes under the block maxima `top` (broadcast) by the calls' own fp32 steps, and the fp32 scales."""
    top = top.clamp(min=2.0 ** -100)
    most = torch.full_like(top, 448.0)  # tensor by tensor: IEEE divisions
    q = (v * (most / top)).clamp(-448.0, 448.0).to(E4M3)
    scale = top / most
    bad = ~torch.isfinite(top)
    return torch.where(bad, torch.zeros_like(v), q.float()).to(E4M3), torch.where(bad, torch.full_like(scale, float("nan")), scale)


def quantize_rows(x):
    x = x.float()
    q = torch.empty(x.shape, dtype=E4M3, device=x.device)
    scale = []
    for c in range(0, x.shape[1], 128):
        v = x[:, c:c + 128]
        top = v.abs().amax(dim=1, keepdim=True)
        top = torch.where(v.isfinite().all(dim=1, keepdim=True), top, torch.full_like(top, float("inf")))
        q[:, c:c + 128], s = codes(v, top)
        scale.append(s[:, 0])
    return q, torch.stack(scale)


def quantize_weight(w):
    E, N, K = w.shape
    w = w.float()
    q = torch.empty(w.shape, dtype=E4M3, device=w.device)
    scale = torch.empty((E, -(-N // 128), -(-K // 128)), device=w.device)
    for e in range(E):
        for i in range(scale.shape[1]):
            for j in range(scale.shape[2]):
                at = (e, slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                v = w[at]
                top = v.abs().max() if v.isfinite().all() else v.new_tensor(float("inf"))
                q[at], scale[e, i, j] = codes(v, top.reshape(1, 1))
    return q, scale


def row_values(q, scale):
    return q.double() * scale.double().t().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def weight_values(q, scale):
    s = scale.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    return q.double() * s[:, :q.shape[1], :q.shape[2]]


def fp8_tolerance(red, dtype):
    """Relative to the sum of the products' magnitudes. A block's 128 products are added 32 at a time, each step losing
    at most two units in the last place of the accumulator (alignment, then the addition): 4 x 2^-22, 5 with the first.
    The product of the scales is rounded once, each block's fused multiply-add and the bias once."""
    return 5 * 2.0 ** -22 + (-(-red // 128) + 3) * U + (HALF[dtype] if dtype == torch.bfloat16 else 0.0)


# ---------------------------------------------------------------- norms
def norm_fwd(x, r, post, pre, gate, scale, eps):
    """(r', n, stats) of 64-bit tensors; differentiable."""
    one = torch.ones(x.shape[0], dtype=x.dtype, device=x.device)
    s1 = torch.rsqrt((x * x).mean(dim=1) + eps) if post is not None else one
    v = x * s1[:, None] * (post if post is not None else 1.0)
    if gate is not None:
        v = v * gate[:, None]
    r2 = scale * v if r is None else r + scale * v
    s2 = torch.rsqrt((r2 * r2).mean(dim=1) + eps) if pre is not None else one
    return r2, r2 * s2[:, None] * pre if pre is not None else None, torch.stack([s1, s2])


def norm_bwd(dres, dn, x, res, stats, post, pre, gate, scale):
    """The gradients by the formulas, from the saved r' and statistics, and the same sums of their terms' magnitudes."""
    out, mag = {}, {}
    M, F = (dn if dn is not None else dres).shape
    like = dn if dn is not None else dres
    D = dres if dres is not None else torch.zeros_like(like)
    D_mag = D.abs()
    if pre is not None:
        rh = res * stats[1][:, None]
        t = dn * pre
        D = D + stats[1][:, None] * (t - rh * (t * rh).mean(dim=1, keepdim=True))
        D_mag = D_mag + stats[1][:, None] * (t.abs() + rh.abs() * (t * rh).abs().mean(dim=1, keepdim=True))
        out["dpre_weight"], mag["dpre_weight"] = (dn * rh).sum(dim=0), (dn * rh).abs().sum(dim=0)
    out["dresidual"], mag["dresidual"] = D, D_mag
    a = scale * (gate if gate is not None else torch.ones(M, dtype=like.dtype, device=like.device))[:, None]
    xh = x * stats[0][:, None] if x is not None else None
    w = post if post is not None else torch.ones(F, dtype=like.dtype, device=like.device)
    if gate is not None:
        out["dgate"] = scale * (D * w * xh).sum(dim=1)
        mag["dgate"] = abs(scale) * (D_mag * (w * xh).abs()).sum(dim=1)
    if post is None:
        out["dx"], mag["dx"] = a * D, (a * D_mag).abs()
        return out, mag
    out["dpost_weight"], mag["dpost_weight"] = (a * D * xh).sum(dim=0), ((a * xh).abs() * D_mag).sum(dim=0)
    s1 = stats[0][:, None]
    out["dx"] = a * s1 * (D * w - xh * (D * w * xh).mean(dim=1, keepdim=True))
    mag["dx"] = (a * s1).abs() * (D_mag * w.abs() + xh.abs() * (D_mag * (w * xh).abs()).mean(dim=1, keepdim=True))
    return out, mag

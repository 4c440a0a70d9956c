"""Cases and plain forms of the gated feed-forward products, the block-scaled fp8 products and the norms of a block.

E experts own consecutive rows of a token-major tensor (expert e the rows
off_e .. off_e + m_e, any m_e >= 0, none a multiple of anything).

  swiglu_fprop  [g | u] = X[m, :] . W1[e(m)]^T + b1[e(m)],  h = silu(g) u; on request [g | u] as well
  swiglu_dgrad  dh = dY[m, :] . W2[e(m)] and the gradient [dg | du] of the saved [g | u]:
                dg = dh u s (1 + g (1 - s)), du = dh g s, s = 1 / (1 + exp(-g)); on request h again
  fp8_fprop     x and W in e4m3 with fp32 scales, one for 128 values of a token's row and one for 128 x 128 of W:
                Y[m, n] = sum over blocks j of 128 columns: xs[j, m] ws[e, n / 128, j] (Xq[m, j] . Wq[e, n, j]) + b[e, n]
  fp8_dgrad     dX = dY . W on the same codes of W, dY quantized by rows
  norm          r' = r + c gate[m] N(x; w_post), n = N(r'; w_pre), N(v; w) = v w / sqrt(mean(v^2) + eps)
  norm_grad     the gradients of x, r, w_post, w_pre and gate from those of r' and n

A block's scale is max(|v|, 2^-100) / 448, and the code of v the e4m3 value nearest to v (448 / max): even codes on ties.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # FC1 with its activation in one decoding step of 8 sequences, top-2: 16 rows over 8 experts, bound by reading W1
        {"name": "swiglu_decode_16", "op": "swiglu_fprop", "E": 8, "M": 16, "K": 2048, "F": 2048, "alpha": 100.0,
         "bias": True, "pad": 0, "keep": False},
        # the same layer in training (16k routed rows, the default benchmark's), [g | u] kept for the backward pass
        {"name": "swiglu_16k", "op": "swiglu_fprop", "E": 8, "M": 16384, "K": 2048, "F": 2048, "alpha": 100.0,
         "bias": False, "pad": 0, "keep": True},
        # FC2's input gradient through the activation with odd widths and a slice of a wider dY, 48 uneven experts
        {"name": "swiglu_dgrad_odd", "op": "swiglu_dgrad", "E": 48, "M": 10007, "N": 1416, "F": 2056, "alpha": 1.0,
         "pad": 64, "keep": False},
        # the largest workload of the repository: 128 experts, 128k rows, skewed routing; h made again for FC2's dW
        {"name": "swiglu_dgrad_128k_skew", "op": "swiglu_dgrad", "E": 128, "M": 131072, "N": 7168, "F": 1024, "alpha": 0.5,
         "pad": 0, "keep": True},
        # serving a checkpoint in block-scaled fp8, one step of 8 sequences, top-2
        {"name": "fp8_decode_16", "op": "fp8_fprop", "E": 8, "M": 16, "K": 2048, "N": 4096, "alpha": 100.0, "bias": True,
         "pad": 0, "out": "bf16", "quantize_w": False},
        # the largest workload as a training step runs it: the weights have changed since the last one
        {"name": "fp8_128k_skew", "op": "fp8_fprop", "E": 128, "M": 131072, "K": 7168, "N": 2048, "alpha": 0.5,
         "bias": False, "pad": 0, "out": "bf16", "quantize_w": True},
        # an input gradient whose widths are no multiples of the blocks
        {"name": "fp8_dgrad_odd", "op": "fp8_dgrad", "E": 48, "M": 10007, "K": 1424, "N": 2064, "alpha": 1.0, "pad": 0,
         "out": "f32"},
        # the input gradient of the default benchmark layer
        {"name": "fp8_dgrad_16k", "op": "fp8_dgrad", "E": 8, "M": 16384, "K": 2048, "N": 4096, "alpha": 100.0, "pad": 0,
         "out": "bf16"},
        # 8 sequences' hidden rows between two blocks of a decoding step, bound by the launch
        {"name": "norm_decode_8", "op": "norm", "M": 8, "F": 2048, "dtype": "bf16", "post": True, "pre": True,
         "gate": True, "c": 1.0},
        # the same between two blocks in training, an odd number of rows
        {"name": "norm_40k", "op": "norm", "M": 40961, "F": 2048, "dtype": "bf16", "post": True, "pre": True, "gate": True,
         "c": 0.5},
        # the largest hidden width of the repository's workloads, few rows: weight gradients over a short axis
        {"name": "norm_grad_1023x7168", "op": "norm_grad", "M": 1023, "F": 7168, "dtype": "f32", "post": True, "pre": True,
         "gate": False, "c": 1.0},
        # 84k rows, as the 64-expert workload routes
        {"name": "norm_grad_84k", "op": "norm_grad", "M": 83968, "F": 1024, "dtype": "bf16", "post": True, "pre": True,
         "gate": True, "c": 0.5},
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["swiglu_fprop", "swiglu_dgrad", "fp8_fprop", "fp8_dgrad", "norm", "norm_grad"])
    while op.startswith("norm"):
        c = {"op": op, "M": _log_int(rng, 1, 131072), "F": _log_int(rng, 64, 16384, 8), "dtype": rng.choice(["bf16", "f32"]),
             "post": rng.random() < 0.7, "pre": True, "gate": rng.random() < 0.5, "c": rng.choice([1.0, 0.5, 0.125])}
        if c["M"] * c["F"] <= 1.2e8:
            return c
    while True:
        swiglu, fprop = op.startswith("swiglu"), op.endswith("fprop")
        c = {"op": op, "E": _log_int(rng, 1, 128), "M": _log_int(rng, 1, 65536), "alpha": rng.choice([0.3, 1.0, 100.0]),
             "pad": rng.choice([0, 0, 64])}
        if swiglu:
            c["K" if fprop else "N"] = _log_int(rng, 128, 7168, 8)
            c["F"] = _log_int(rng, 64, 4096, 8)
            c["keep"] = rng.random() < 0.5
            mac = (c["K"] * 2 if fprop else c["N"]) * c["F"]
        else:
            c["K"], c["N"] = _log_int(rng, 128, 7168, 16), _log_int(rng, 128, 7168, 16)
            c["out"] = rng.choice(["bf16", "bf16", "f32"])
            mac = c["K"] * c["N"]
        if fprop:
            c["bias"] = rng.random() < 0.5
            if not swiglu:
                c["quantize_w"] = rng.random() < 0.3
        if 2.0 * c["M"] * mac <= 1.5e12 and c["E"] * mac <= 6e8:
            return c


def _counts(case, seed):
    """Rows per expert: a draw of M rows over experts whose shares are Dirichlet (alpha small: skewed, some empty)."""
    r = np.random.default_rng(seed)
    share = r.dirichlet(np.full(case["E"], case["alpha"]))
    return [int(v) for v in r.multinomial(case["M"], share / share.sum())]


def _rows(gen, rows, cols, pad=0, std=1.0):
    """(rows, cols) bf16 normal values, of row stride cols + pad."""
    t = torch.empty((rows, cols + pad), dtype=BF16, device="cuda").normal_(0.0, std, generator=gen)
    return t[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm", "norm_grad"):
        M, F, dt = case["M"], case["F"], BF16 if case["dtype"] == "bf16" else F32
        normal = lambda std, *shape: torch.empty(shape, dtype=F32, device="cuda").normal_(0.0, std, generator=gen)
        s["x"] = normal(0.7, M, F).to(dt)
        s["r"] = normal(3.0, M, F).to(dt)
        s["w_post"] = (1.0 + normal(0.2, F)).to(dt) if case["post"] else None
        s["w_pre"] = (1.0 + normal(0.2, F)).to(dt) if case["pre"] else None
        s["gate"] = torch.sigmoid(normal(1.0, M)) if case["gate"] else None
        if op == "norm_grad":  # what the forward pass left: r' and the inverse root mean squares
            r2, _, stats = _norm_plain(s)
            s.update(r_out=r2, stats=stats, d_r=normal(0.02, M, F).to(dt), d_n=normal(0.02, M, F).to(dt))
            del s["r"]
        return s
    E, M = case["E"], case["M"]
    s["counts"] = _counts(case, seed)  # the plain form's loop bounds; the kernels read the device's copy
    s["m_splits"] = torch.tensor(s["counts"], dtype=torch.int64, device="cuda")
    if op == "swiglu_fprop":
        s["x"] = _rows(gen, M, case["K"], case["pad"])
        s["w"] = _rows(gen, E * 2 * case["F"], case["K"], 0, 0.02).view(E, 2 * case["F"], case["K"])
        s["bias"] = _rows(gen, E, 2 * case["F"], 0, 0.02) if case["bias"] else None
    elif op == "swiglu_dgrad":
        s["dy"] = _rows(gen, M, case["N"], case["pad"], 2.0 ** -8)
        s["w"] = _rows(gen, E * case["N"], case["F"], 0, 0.02).view(E, case["N"], case["F"])
        s["y"] = _rows(gen, M, 2 * case["F"])
    else:
        N, K = case["N"], case["K"]
        if op == "fp8_fprop":
            s["x"] = _rows(gen, M, K, case["pad"])
            s["bias"] = _rows(gen, E, N, 0, 0.02) if case["bias"] else None
        else:
            s["dy"] = _rows(gen, M, N, case["pad"], 2.0 ** -8)
        w = _rows(gen, E * N, K, 0, 0.02).view(E, N, K)
        if op == "fp8_fprop" and case["quantize_w"]:
            s["w"] = w
        else:  # the checkpoint's codes and scales
            s["wq"], s["ws"] = _quantize_w_plain(w)
    return s


# ---------------------------------------------------------------- plain forms
def _spans(counts):
    """(expert, its rows) of the experts that have any."""
    ends = np.cumsum(counts)
    return [(e, slice(int(b - m), int(b))) for e, (m, b) in enumerate(zip(counts, ends)) if m]


def _out(s):
    return BF16 if s["out"] == "bf16" else F32


def _codes(v, top):
    """e4m3 codes of v under the block maxima `top`, which broadcast over it, and the scales."""
    top = top.clamp(min=2.0 ** -100)
    most = torch.full_like(top, 448.0)  # tensor by tensor: a division each (a scalar's is done by its reciprocal)
    return (v * (most / top)).clamp(-448.0, 448.0).to(E4M3), top / most


def _blocks(v):
    """The last dimension in blocks of 128, the last one filled up with zeros."""
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % 128)).unflatten(-1, (-1, 128))


def _quantize_x_plain(x):
    """Codes (M, K) and scales (K / 128, M)."""
    v = _blocks(x.float())
    q, scale = _codes(v, v.abs().amax(dim=2, keepdim=True))
    return q.flatten(1)[:, :x.shape[1]].contiguous(), scale.squeeze(2).t().contiguous()


def _quantize_w_plain(w):
    """Codes (E, N, K) and scales (E, N / 128, K / 128)."""
    E, N, K = w.shape
    q = torch.empty(w.shape, dtype=E4M3, device=w.device)
    scale = torch.empty((E, -(-N // 128), -(-K // 128)), dtype=F32, device=w.device)
    for e in range(E):  # an expert at a time: the intermediate values are twice the weights' size
        v = torch.nn.functional.pad(_blocks(w[e].float()), (0, 0, 0, 0, 0, -N % 128)).unflatten(0, (-1, 128))
        c, sc = _codes(v, v.abs().amax(dim=(1, 3), keepdim=True))
        q[e] = c.flatten(0, 1).flatten(1)[:N, :K]
        scale[e] = sc.squeeze(3).squeeze(1)
    return q, scale


def _x_values(q, scale):
    """What the codes of rows stand for."""
    return q.float() * scale.t().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _w_values(q, scale):
    """What the codes of one expert's weight stand for."""
    return q.float() * scale.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def _swiglu_fprop_plain(s):
    F = s["F"]
    h = torch.empty((s["M"], F), dtype=BF16, device="cuda")
    y = torch.empty((s["M"], 2 * F), dtype=BF16, device="cuda") if s["keep"] else None
    for e, r in _spans(s["counts"]):
        v = s["x"][r].float() @ s["w"][e].float().t()
        if s["bias"] is not None:
            v = v + s["bias"][e].float()
        h[r] = v[:, :F] * torch.sigmoid(v[:, :F]) * v[:, F:]
        if y is not None:
            y[r] = v
    return (h, y) if s["keep"] else h


def _swiglu_dgrad_plain(s):
    F = s["F"]
    d1 = torch.empty((s["M"], 2 * F), dtype=BF16, device="cuda")
    h = torch.empty((s["M"], F), dtype=BF16, device="cuda") if s["keep"] else None
    for e, r in _spans(s["counts"]):
        dh = s["dy"][r].float() @ s["w"][e].float()
        g, u = s["y"][r].float().chunk(2, dim=1)
        sg = torch.sigmoid(g)
        d1[r, :F] = dh * u * sg * (1 + g * (1 - sg))
        d1[r, F:] = dh * g * sg
        if h is not None:
            h[r] = g * sg * u
    return (d1, h) if s["keep"] else d1


def _fp8_fprop_plain(s):
    q, xs = _quantize_x_plain(s["x"])
    wq, ws = _quantize_w_plain(s["w"]) if s["quantize_w"] else (s["wq"], s["ws"])
    x = _x_values(q, xs)
    y = torch.empty((s["M"], s["N"]), dtype=_out(s), device="cuda")
    for e, r in _spans(s["counts"]):
        v = x[r] @ _w_values(wq[e], ws[e]).t()
        y[r] = v if s["bias"] is None else v + s["bias"][e].float()
    out = {"xq": q, "xs": xs, "y": y}
    return {**out, "wq": wq, "ws": ws} if s["quantize_w"] else out


def _fp8_dgrad_plain(s):
    q, ds = _quantize_x_plain(s["dy"])
    d = _x_values(q, ds)
    dx = torch.empty((s["M"], s["K"]), dtype=_out(s), device="cuda")
    for e, r in _spans(s["counts"]):
        dx[r] = d[r] @ _w_values(s["wq"][e], s["ws"][e])
    return {"dyq": q, "dys": ds, "dx": dx}


def _rstd(v):
    return 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _norm_plain(s):
    """r', n and the inverse root mean squares (2, M) of x (1 without its norm) and r'."""
    x, dt = s["x"].float(), s["x"].dtype
    post = _rstd(x) if s["post"] else torch.ones((x.shape[0], 1), dtype=F32, device=x.device)
    v = x * post * s["w_post"].float() if s["post"] else x
    if s["gate"] is not None:
        v = v * s["gate"][:, None]
    r = s["r"].float() + s["c"] * v
    pre = _rstd(r)
    return r.to(dt), (r * pre * s["w_pre"].float()).to(dt), torch.cat([post, pre], dim=1).t().contiguous()


def _norm_grad_plain(s):
    dt = s["x"].dtype
    post, pre = s["stats"][0][:, None], s["stats"][1][:, None]
    r_hat = s["r_out"].float() * pre
    d_n = s["d_n"].float()
    d_w_pre = (d_n * r_hat).sum(dim=0)
    t = d_n * s["w_pre"].float()
    d_r = s["d_r"].float() + pre * (t - r_hat * (t * r_hat).mean(dim=1, keepdim=True))
    d_v = s["c"] * d_r
    x_hat = s["x"].float() * post
    v = x_hat * s["w_post"].float() if s["post"] else x_hat
    d_gate = (d_v * v).sum(dim=1) if s["gate"] is not None else None
    if s["gate"] is not None:
        d_v = d_v * s["gate"][:, None]
    out = {"d_r": d_r.to(dt), "d_w_pre": d_w_pre}
    if s["post"]:
        out["d_w_post"] = (d_v * x_hat).sum(dim=0)
        t = d_v * s["w_post"].float()
        d_v = post * (t - x_hat * (t * x_hat).mean(dim=1, keepdim=True))
    out["d_x"] = d_v.to(dt)
    if d_gate is not None:
        out["d_gate"] = d_gate
    return out


_PLAIN = {"swiglu_fprop": _swiglu_fprop_plain, "swiglu_dgrad": _swiglu_dgrad_plain, "fp8_fprop": _fp8_fprop_plain,
          "fp8_dgrad": _fp8_dgrad_plain, "norm": _norm_plain, "norm_grad": _norm_grad_plain}


def _run_own(s):
    import moe_expert_grouped_group_gb300 as mxq

    op = s["op"]
    if op == "swiglu_fprop":
        return mxq.ragged_gemm_fprop_swiglu(s["x"], s["w"], s["m_splits"], bias=s["bias"], y_out=s["keep"])
    if op == "swiglu_dgrad":
        return mxq.ragged_gemm_dgrad_swiglu(s["dy"], s["w"], s["y"], s["m_splits"], h_out=s["keep"])
    if op == "fp8_fprop":
        q, xs = mxq.fp8_quantize_rows(s["x"])
        wq, ws = mxq.fp8_quantize_weight(s["w"]) if s["quantize_w"] else (s["wq"], s["ws"])
        y = mxq.fp8_gemm_fprop(q, xs, wq, ws, s["m_splits"], bias=s["bias"], out_dtype=_out(s))
        out = {"xq": q.view(E4M3), "xs": xs, "y": y}
        return {**out, "wq": wq.view(E4M3), "ws": ws} if s["quantize_w"] else out
    if op == "fp8_dgrad":
        q, ds = mxq.fp8_quantize_rows(s["dy"])
        dx = mxq.fp8_gemm_dgrad(q, ds, s["wq"], s["ws"], s["m_splits"], out_dtype=_out(s))
        return {"dyq": q.view(E4M3), "dys": ds, "dx": dx}
    if op == "norm":
        return mxq.norm_residual_fwd(s["x"], s["r"], post_weight=s["w_post"], pre_weight=s["w_pre"], gate=s["gate"],
                                     scale=s["c"], eps=EPS)
    g = mxq.norm_residual_bwd(s["d_r"], s["d_n"], s["x"], s["r_out"], s["stats"], post_weight=s["w_post"],
                              pre_weight=s["w_pre"], gate=s["gate"], scale=s["c"])
    names = {"dresidual": "d_r", "dpre_weight": "d_w_pre", "dpost_weight": "d_w_post", "dx": "d_x", "dgate": "d_gate"}
    return {names[k]: v for k, v in g.items()}


def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------- work and 64-bit values
def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, size = case["M"] * case["F"], 2 if case["dtype"] == "bf16" else 4
        weights = (case["post"] + case["pre"]) * case["F"]
        if op == "norm":  # x, r in; r', n out
            moved, flops = 4 * size * n + size * weights + (8 + 4 * case["gate"]) * case["M"], 10 * n
        else:  # dr', dn, r' in, x too where its norm or a gate needs it; dr, dx out
            moved = ((6 if case["post"] or case["gate"] else 5) * size * n + (size + 4) * weights
                     + (8 + 8 * case["gate"]) * case["M"])
            flops = 20 * n
        return {"bytes": int(moved), "flops": flops}
    E, M = case["E"], case["M"]
    # experts that get rows, from the draw's expectation under equal shares: the others' weights need not be read
    used = E * (1.0 - (1.0 - 1.0 / E) ** M)
    if op == "swiglu_fprop":
        F, K = case["F"], case["K"]
        moved = 2 * M * K + 2 * int(used) * 2 * F * K + 2 * M * F * (3 if case["keep"] else 1)
        return {"bytes": int(moved + 8 * E + (4 * E * F if case["bias"] else 0)), "flops": 4 * M * F * K}
    if op == "swiglu_dgrad":
        F, N = case["F"], case["N"]
        return {"bytes": int(2 * M * N + 2 * int(used) * N * F + 8 * M * F + (2 * M * F if case["keep"] else 0) + 8 * E),
                "flops": 2 * M * F * N}
    N, K, out = case["N"], case["K"], 2 if case["out"] == "bf16" else 4
    red, width = (K, N) if op == "fp8_fprop" else (N, K)
    moved = 2 * M * red + M * red + 4 * M * -(-red // 128) + out * M * width + 8 * E
    if case.get("quantize_w"):
        moved += 3 * E * N * K + 4 * E * -(-N // 128) * -(-K // 128)
    else:
        moved += int(used) * N * K + 4 * int(used) * -(-N // 128) * -(-K // 128)
    return {"bytes": int(moved + (2 * E * N if case.get("bias") else 0)), "flops": 2 * M * N * K}


def _codes64(v, top):
    """The codes of the 32-bit definition as 64-bit values, and the scales in 64 bits."""
    top = torch.maximum(top, torch.full_like(top, 2.0 ** -100))
    inv = torch.div(torch.full_like(top, 448.0), top)
    return torch.clamp(v * inv, -448, 448).to(E4M3).double(), top.double() / 448.0


def _row_values64(x):
    """(scales (K / 128, M), the values that the codes stand for)."""
    scales, values = [], []
    for c in range(0, x.shape[1], 128):
        v = x[:, c:c + 128].float()
        q, sc = _codes64(v, v.abs().max(dim=1, keepdim=True)[0])
        scales.append(sc[:, 0])
        values.append(q * sc)
    return torch.stack(scales), torch.cat(values, dim=1)


def _weight_values64(s, e):
    """(scales, values) of expert e's weight, from its codes or from the weight itself."""
    w = s["w"][e].float() if "w" in s else s["wq"][e].double()
    N, K = w.shape
    values = torch.empty((N, K), dtype=torch.float64, device=w.device)
    scales = torch.empty((-(-N // 128), -(-K // 128)), dtype=torch.float64, device=w.device)
    for i in range(scales.shape[0]):
        band = w[128 * i:128 * i + 128]
        for j in range(scales.shape[1]):
            block = band[:, 128 * j:128 * j + 128]
            if "w" in s:
                q, sc = _codes64(block, block.abs().max())
            else:
                q, sc = block, s["ws"][e, i, j].double()
            scales[i, j] = sc
            values[128 * i:128 * i + 128, 128 * j:128 * j + 128] = q * sc
    return scales, values


def exact(case, seed):
    op = case["op"]
    if op not in ("norm", "norm_grad") and work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    if op == "norm":
        x = s["x"].double()
        post = torch.rsqrt(torch.mean(x ** 2, dim=1) + EPS) if s["post"] else torch.ones_like(x[:, 0])
        factor = case["c"] * post if s["gate"] is None else case["c"] * post * s["gate"].double()
        r = s["r"].double() + torch.einsum("mf,m->mf", x, factor) * (s["w_post"].double() if s["post"] else 1.0)
        pre = torch.rsqrt(torch.mean(r ** 2, dim=1) + EPS)
        return r, torch.einsum("mf,m,f->mf", r, pre, s["w_pre"].double()), torch.stack([post, pre])
    if op == "norm_grad":
        F = case["F"]
        post, pre = s["stats"].double()
        x, r, d_n = s["x"].double(), s["r_out"].double(), s["d_n"].double()
        w2 = s["w_pre"].double()
        dot = torch.einsum("mf,mf,f->m", d_n, r, w2)
        D = s["d_r"].double() + pre[:, None] * d_n * w2 - (pre ** 3 * dot / F)[:, None] * r
        out = {"d_r": D, "d_w_pre": torch.einsum("mf,mf,m->f", d_n, r, pre)}
        gate = torch.ones_like(pre) if s["gate"] is None else s["gate"].double()
        a = case["c"] * gate
        if s["post"]:
            w1 = s["w_post"].double()
            out["d_w_post"] = torch.einsum("mf,mf,m->f", D, x, a * post)
            dot = torch.einsum("mf,mf,f->m", D, x, w1)
            out["d_x"] = (a * post)[:, None] * D * w1 - (a * post ** 3 * dot / F)[:, None] * x
            d_gate = case["c"] * post * dot
        else:
            out["d_x"] = a[:, None] * D
            d_gate = case["c"] * torch.einsum("mf,mf->m", D, x)
        if s["gate"] is not None:
            out["d_gate"] = d_gate
        return out
    off, parts, more, scales = 0, [], [], []
    if op.startswith("fp8"):
        row_scales, rows = _row_values64(s["x"] if op == "fp8_fprop" else s["dy"])
    for e, m in enumerate(s["counts"]):
        r = slice(off, off + m)
        off += m
        if op.startswith("fp8"):
            if m or "w" in s:
                sc, w = _weight_values64(s, e)
                scales.append(sc)
            if m:
                v = torch.einsum("mk,nk->mn" if op == "fp8_fprop" else "mn,nk->mk", rows[r], w)
                parts.append(v if s.get("bias") is None else v + s["bias"][e].double())
            continue
        if m == 0:
            continue
        if op == "swiglu_fprop":
            v = torch.einsum("mk,nk->mn", s["x"][r].double(), s["w"][e].double())
            v = v if s["bias"] is None else v + s["bias"][e].double()
            g, u = v[:, :case["F"]], v[:, case["F"]:]
            parts.append(g / (1.0 + torch.exp(-g)) * u)
            more.append(v)
        else:
            d = torch.einsum("mn,nf->mf", s["dy"][r].double(), s["w"][e].double())
            g, u = s["y"][r].double()[:, :case["F"]], s["y"][r].double()[:, case["F"]:]
            sig = 1.0 / (1.0 + torch.exp(-g))
            parts.append(torch.cat([d * u * (sig + g * sig * (1.0 - sig)), d * g * sig], dim=1))
            more.append(g * sig * u)
    y = torch.cat(parts)
    if op == "fp8_fprop":
        out = {"xq": None, "xs": row_scales, "y": y}
        return {**out, "wq": None, "ws": torch.stack(scales)} if "w" in s else out
    if op == "fp8_dgrad":
        return {"dyq": None, "dys": row_scales, "dx": y}
    return (y, torch.cat(more)) if s["keep"] else y

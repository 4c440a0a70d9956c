"""Cases and plain forms of the bf16, int8 and dropout operators of an MoE expert layer.

What is computed, for E experts that own consecutive rows of a token-major
tensor (expert e the rows off_e .. off_e + m_e, any m_e >= 0, none a multiple
of anything):

  fprop          Y[m, :]  = X[m, :] . W[e(m)]^T + b[e(m)]
  dgrad          dX[m, :] = dY[m, :] . W[e(m)]
  wgrad          dW[e]    = dY_e^T . X_e
  int8           each token row is quantized to int8 with a scale of its own, then
                 Y[m, n]  = xs[m] ws[e, n] sum_k xq[m, k] wq[e, n, k] + b[e, n]
  swiglu_dropout h = D(silu(g) u), [g | u] the rows of FC1's output
  swiglu_dropout_grad   its gradient [dg | du] from dh, the mask made again
  dropout        y = residual + D(x)

D keeps element i with probability 1 - t / 65536, t = round(65536 p), and
scales what it keeps by 65536 / (65536 - t). Element i is dropped when the
(i mod 8)-th 16-bit word, low half first, of Philox 4x32-10 (Salmon, Moraes,
Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) at the
counter (i div 8, offset) under the key `seed` is below t.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


def listed():
    return [
        # one decoding step of 8 sequences, top-2: 16 rows over 8 experts, bound by reading the weights
        {"name": "fprop_decode_16", "op": "fprop", "E": 8, "M": 16, "K": 2048, "N": 4096, "alpha": 100.0, "bias": True,
         "pad": 0, "out": "bf16"},
        # the expert layer of the default benchmark (16k routed rows) with the counts as the router gives them
        {"name": "fprop_16k", "op": "fprop", "E": 8, "M": 16384, "K": 2048, "N": 4096, "alpha": 100.0, "bias": True,
         "pad": 0, "out": "bf16"},
        # the largest workload of the repository: 128 experts, 128k rows, skewed routing
        {"name": "fprop_128k_skew", "op": "fprop", "E": 128, "M": 131072, "K": 7168, "N": 2048, "alpha": 0.5,
         "bias": False, "pad": 0, "out": "bf16"},
        # a gradient with odd widths and a row stride wider than the row (a slice of a packed activation)
        {"name": "dgrad_odd", "op": "dgrad", "E": 48, "M": 10007, "K": 1416, "N": 2056, "alpha": 1.0, "bias": False,
         "pad": 64, "out": "bf16"},
        # weight gradients of the default benchmark layer in fp32, as a main gradient keeps them
        {"name": "wgrad_16k", "op": "wgrad", "E": 8, "M": 16384, "K": 2048, "N": 4096, "alpha": 100.0, "bias": False,
         "pad": 0, "out": "f32"},
        # many experts of uneven size, some with a handful of rows or none: FC2 of the 32-expert workload
        {"name": "wgrad_skew", "op": "wgrad", "E": 32, "M": 30011, "K": 1536, "N": 4096, "alpha": 0.3, "bias": False,
         "pad": 0, "out": "bf16"},
        # serving a quantized expert layer, one step of 8 sequences, top-2
        {"name": "int8_decode_16", "op": "int8", "E": 8, "M": 16, "K": 2048, "N": 4096, "alpha": 100.0, "bias": True,
         "pad": 0, "out": "bf16"},
        # a prompt batch through the same layer
        {"name": "int8_16k", "op": "int8", "E": 8, "M": 16384, "K": 2048, "N": 4096, "alpha": 100.0, "bias": True,
         "pad": 0, "out": "bf16"},
        # the smallest workload's activation: 512 rows, bound by the launch
        {"name": "swiglu_dropout_512", "op": "swiglu_dropout", "M": 512, "F": 512, "p": 0.4},
        # the activation between FC1 and FC2 of the 32-expert workload
        {"name": "swiglu_dropout_64k", "op": "swiglu_dropout", "M": 65536, "F": 1536, "p": 0.4},
        # its gradient on the 64-expert workload's rows
        {"name": "swiglu_dropout_grad_84k", "op": "swiglu_dropout_grad", "M": 83968, "F": 1024, "p": 0.1},
        # the layer's output onto the residual stream, an odd number of rows
        {"name": "dropout_residual_40k", "op": "dropout", "M": 40961, "F": 2048, "p": 0.1, "dtype": "bf16",
         "residual": True},
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["fprop", "dgrad", "wgrad", "int8", "swiglu_dropout", "swiglu_dropout_grad", "dropout"])
    if op in ("fprop", "dgrad", "wgrad", "int8"):
        while True:
            c = {"op": op, "E": _log_int(rng, 1, 128), "M": _log_int(rng, 1, 65536),
                 "K": _log_int(rng, 128, 7168, 16 if op == "int8" else 8), "N": _log_int(rng, 128, 7168, 8),
                 "alpha": rng.choice([0.3, 1.0, 100.0]), "bias": op in ("fprop", "int8") and rng.random() < 0.5,
                 "pad": rng.choice([0, 0, 64]) if op != "int8" else 0, "out": rng.choice(["bf16", "bf16", "f32"])}
            if 3072 in (c["K"], c["N"], c["M"]):
                continue
            if 2.0 * c["M"] * c["N"] * c["K"] <= 1.5e12 and c["E"] * c["N"] * c["K"] <= 6e8:
                return c
    while True:
        c = {"op": op, "M": _log_int(rng, 1, 131072), "F": _log_int(rng, 64, 7168, 8), "p": round(rng.uniform(0.05, 0.6), 3)}
        if 3072 in (c["M"], c["F"]) or c["M"] * c["F"] > 1.2e8:
            continue
        if op == "dropout":
            c["dtype"], c["residual"] = rng.choice(["bf16", "f32"]), rng.random() < 0.5
        return c


def _counts(case, seed):
    """Rows per expert: a draw of M rows over experts whose shares are Dirichlet (alpha small: skewed, some empty)."""
    r = np.random.default_rng(seed)
    share = r.dirichlet(np.full(case["E"], case["alpha"]))
    return [int(v) for v in r.multinomial(case["M"], share / share.sum())]


def _rows(gen, rows, cols, pad, std=1.0):
    """(rows, cols) bf16 normal values, of row stride cols + pad."""
    t = torch.empty((rows, cols + pad), dtype=BF16, device="cuda").normal_(0.0, std, generator=gen)
    return t[:, :cols]


def _quantize_rows_plain(x):
    """Symmetric int8 with one scale per row: s = max(|x|, 2^-100) / 127, q = rint(x (127 / max))."""
    x = x.float()
    top = x.abs().amax(dim=1, keepdim=True).clamp(min=2.0 ** -100)
    most = torch.full_like(top, 127.0)  # tensor by tensor: a division each (a scalar's is done by its reciprocal)
    q = torch.round(x * (most / top)).clamp(-127.0, 127.0)
    return q.to(torch.int8), (top / most).squeeze(1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("fprop", "dgrad", "wgrad", "int8"):
        E, M, N, K = case["E"], case["M"], case["N"], case["K"]
        s["counts"] = _counts(case, seed)  # the plain form's loop bounds; the kernels read the device's copy
        s["m_splits"] = torch.tensor(s["counts"], dtype=torch.int64, device="cuda")
        if op != "dgrad":
            s["x"] = _rows(gen, M, K, case["pad"])
        if op in ("dgrad", "wgrad"):
            s["dy"] = _rows(gen, M, N, case["pad"])
        if op != "wgrad":
            s["w"] = _rows(gen, E * N, K, 0, 0.02).view(E, N, K)
        s["bias"] = _rows(gen, E, N, 0, 0.02) if case["bias"] else None
        if op == "int8":  # the checkpoint's weights: int8 codes and a scale per output channel
            q, ws = _quantize_rows_plain(s.pop("w").view(E * N, K))
            s["wq"], s["ws"] = q.view(E, N, K), ws.view(E, N)
        return s
    M, F = case["M"], case["F"]
    # {seed, offset} of the generator, on the device so that a captured graph can be replayed with new ones
    s["rng"] = torch.tensor([seed * 7919 + 12345678901, (seed * 104729) % (1 << 40)], dtype=torch.int64, device="cuda")
    if op == "dropout":
        dt = BF16 if case["dtype"] == "bf16" else F32
        s["x"] = torch.empty((M, F), dtype=dt, device="cuda").normal_(generator=gen)
        s["residual"] = torch.empty((M, F), dtype=dt, device="cuda").normal_(generator=gen) if case["residual"] else None
        return s
    s["y"] = torch.empty((M, 2 * F), dtype=BF16, device="cuda").normal_(generator=gen)
    if op == "swiglu_dropout_grad":
        s["dh"] = torch.empty((M, F), dtype=BF16, device="cuda").normal_(generator=gen)
    return s


# ---------------------------------------------------------------- plain forms
def _spans(counts):
    """(expert, its rows) of the experts that have any."""
    ends = np.cumsum(counts)
    return [(e, slice(int(b - m), int(b))) for e, (m, b) in enumerate(zip(counts, ends)) if m]


def _out(s):
    return BF16 if s["out"] == "bf16" else F32


def _fprop_plain(s):
    y = torch.empty((s["M"], s["N"]), dtype=_out(s), device="cuda")
    for e, r in _spans(s["counts"]):
        v = s["x"][r].float() @ s["w"][e].float().t()
        y[r] = v if s["bias"] is None else v + s["bias"][e].float()
    return y


def _dgrad_plain(s):
    dx = torch.empty((s["M"], s["K"]), dtype=_out(s), device="cuda")
    for e, r in _spans(s["counts"]):
        dx[r] = s["dy"][r].float() @ s["w"][e].float()
    return dx


def _wgrad_plain(s):
    dw = torch.zeros((s["E"], s["N"], s["K"]), dtype=_out(s), device="cuda")
    for e, r in _spans(s["counts"]):
        dw[e] = s["dy"][r].float().t() @ s["x"][r].float()
    return dw


def _int8_plain(s):
    q, xs = _quantize_rows_plain(s["x"])
    y = torch.empty((s["M"], s["N"]), dtype=_out(s), device="cuda")
    for e, r in _spans(s["counts"]):
        v = (q[r].float() @ s["wq"][e].float().t()) * xs[r, None] * s["ws"][e]
        y[r] = v if s["bias"] is None else v + s["bias"][e].float()
    return {"q": q, "scale": xs, "y": y}


def _philox_plain(rng, n):
    """The 16-bit words of the first ceil(n / 8) counters, n of them, as int64 (32-bit values in 64-bit lanes)."""
    low = 0xFFFFFFFF
    c = torch.arange((n + 7) // 8, dtype=torch.int64, device=rng.device)
    x0, x1 = c & low, c >> 32
    x2, x3 = (rng[1] & low).expand_as(c), ((rng[1] >> 32) & low).expand_as(c)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57  # 64-bit products, kept modulo 2^64
        x0, x1, x2, x3 = ((b >> 32) & low) ^ x1 ^ k0, b & low, ((a >> 32) & low) ^ x3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([x0 & 0xFFFF, x0 >> 16, x1 & 0xFFFF, x1 >> 16, x2 & 0xFFFF, x2 >> 16, x3 & 0xFFFF, x3 >> 16], dim=1)
    return words.view(-1)[:n]


def _drop_plain(v, rng, p):
    t = round(p * 65536)
    keep = _philox_plain(rng, v.numel()).view(v.shape) >= t
    return torch.where(keep, v * (65536.0 / (65536 - t)), torch.zeros_like(v))


def _swiglu_dropout_plain(s):
    g, u = s["y"].float().chunk(2, dim=1)
    return _drop_plain(g * torch.sigmoid(g) * u, s["rng"], s["p"]).to(BF16)


def _swiglu_dropout_grad_plain(s):
    g, u = s["y"].float().chunk(2, dim=1)
    d = _drop_plain(s["dh"].float(), s["rng"], s["p"])
    sg = torch.sigmoid(g)
    return torch.cat([d * u * sg * (1 + g * (1 - sg)), d * g * sg], dim=1).to(BF16)


def _dropout_plain(s):
    v = _drop_plain(s["x"].float(), s["rng"], s["p"])
    return (v if s["residual"] is None else v + s["residual"].float()).to(s["x"].dtype)


_PLAIN = {"fprop": _fprop_plain, "dgrad": _dgrad_plain, "wgrad": _wgrad_plain, "int8": _int8_plain,
          "swiglu_dropout": _swiglu_dropout_plain, "swiglu_dropout_grad": _swiglu_dropout_grad_plain,
          "dropout": _dropout_plain}


def _run_own(s):
    import moe_expert_grouped_group_gb300 as mxq

    op = s["op"]
    if op == "fprop":
        return mxq.ragged_gemm_fprop(s["x"], s["w"], s["m_splits"], bias=s["bias"], out_dtype=_out(s))
    if op == "dgrad":
        return mxq.ragged_gemm_dgrad(s["dy"], s["w"], s["m_splits"], out_dtype=_out(s))
    if op == "wgrad":
        return mxq.ragged_gemm_wgrad(s["dy"], s["x"], s["m_splits"], out_dtype=_out(s))
    if op == "int8":
        q, xs = mxq.int8_quantize_rows(s["x"])
        y = mxq.int8_gemm_fprop(q, xs, s["wq"], s["ws"], s["m_splits"], bias=s["bias"], out_dtype=_out(s))
        return {"q": q, "scale": xs, "y": y}
    if op == "swiglu_dropout":
        return mxq.swiglu_dropout_fwd(s["y"], s["rng"], s["p"])
    if op == "swiglu_dropout_grad":
        return mxq.swiglu_dropout_bwd(s["dh"], s["y"], s["rng"], s["p"])
    return mxq.dropout(s["x"], s["rng"], s["p"], residual=s["residual"])


def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------- work and 64-bit values
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("fprop", "dgrad", "wgrad", "int8"):
        E, M, N, K = case["E"], case["M"], case["N"], case["K"]
        # experts that get rows, from the draw's expectation under equal shares: the others' weights need not be read
        used = E * (1.0 - (1.0 - 1.0 / E) ** M)
        flops, out = 2 * M * N * K, size[case["out"]]
        if op == "wgrad":
            moved = 2 * M * (N + K) + out * E * N * K
        elif op == "int8":
            moved = 2 * M * K + M * K + 4 * M + int(used) * (N * K + 4 * N) + out * M * N
        else:
            moved = 2 * M * (K if op == "fprop" else N) + 2 * int(used) * N * K + out * M * (N if op == "fprop" else K)
        return {"bytes": int(moved + 8 * E + (2 * E * N if case["bias"] else 0)), "flops": flops}
    n = case["M"] * case["F"]
    if op == "swiglu_dropout":
        return {"bytes": 6 * n, "flops": 10 * n}
    if op == "swiglu_dropout_grad":
        return {"bytes": 10 * n, "flops": 20 * n}
    return {"bytes": (3 if case["residual"] else 2) * size[case["dtype"]] * n, "flops": 3 * n}


def _keep64(state, n):
    """Which of n elements D keeps, by the generator's definition on unsigned 64-bit host integers."""
    seed, offset = (int(v) for v in state["rng"].cpu())
    m32 = np.uint64(0xFFFFFFFF)
    block = np.arange((n + 7) // 8, dtype=np.uint64)
    ctr = [block & m32, block >> np.uint64(32), np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p0, p1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(p1 >> np.uint64(32)) ^ ctr[1] ^ np.uint64(key[0]), p1 & m32,
               (p0 >> np.uint64(32)) ^ ctr[3] ^ np.uint64(key[1]), p0 & m32]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(ctr, axis=1).astype("<u4").view("<u2").reshape(-1)[:n]
    return torch.from_numpy(words.astype(np.int32) >= round(state["p"] * 65536)).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("fprop", "dgrad", "wgrad", "int8"):
        if 2.0 * case["M"] * case["N"] * case["K"] > 5e12:
            return None
        off, parts = 0, []
        for e, m in enumerate(s["counts"]):
            if m == 0 and op != "wgrad":
                continue
            rows = slice(off, off + m)
            off += m
            if op == "fprop":
                v = torch.einsum("mk,nk->mn", s["x"][rows].double(), s["w"][e].double())
            elif op == "dgrad":
                v = torch.einsum("mn,nk->mk", s["dy"][rows].double(), s["w"][e].double())
            elif op == "wgrad":
                v = torch.einsum("mn,mk->nk", s["dy"][rows].double(), s["x"][rows].double())
            else:
                # the codes are whole numbers with no 64-bit value of their own: those of the 32-bit definition
                x = s["x"][rows].float()
                top = torch.clamp(x.abs().max(dim=1)[0], min=2.0 ** -100)
                q = torch.clamp(torch.round(x * torch.div(torch.full_like(top, 127.0), top)[:, None]), -127, 127)
                v = torch.einsum("mk,nk->mn", q.double(), s["wq"][e].double())
                v = v * (top.double()[:, None] / 127.0) * s["ws"][e].double()[None, :]
            if op in ("fprop", "int8") and s["bias"] is not None:
                v = v + s["bias"][e].double()
            parts.append(v)
        if op == "wgrad":
            return torch.stack(parts)
        y = torch.cat(parts)
        if op == "int8":
            top = torch.clamp(s["x"].double().abs().max(dim=1)[0], min=2.0 ** -100)
            return {"q": None, "scale": top / 127.0, "y": y}
        return y
    n = case["M"] * case["F"]
    if n > 5e7:  # the host generator would take too long
        return None
    keep = _keep64(s, n).view(case["M"], case["F"])
    scale = 65536.0 / (65536 - round(case["p"] * 65536))
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    if op == "dropout":
        v = torch.where(keep, s["x"].double() * scale, zero)
        return v if s["residual"] is None else v + s["residual"].double()
    g, u = s["y"].double()[:, :case["F"]], s["y"].double()[:, case["F"]:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    if op == "swiglu_dropout":
        return torch.where(keep, g * sig * u * scale, zero)
    d = torch.where(keep, s["dh"].double() * scale, zero)
    return torch.cat([d * u * (sig + g * sig * (1.0 - sig)), d * g * sig], dim=1)

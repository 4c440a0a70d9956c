"""Plain 64-bit definitions of the ragged products and of counter-based
dropout, and the tolerances the GPU tests state their results in."""
import numpy as np
import torch


def spans(counts):
    off = 0
    for e, m in enumerate(counts):
        yield e, slice(off, off + m)
        off += m


def fprop64(x, w, counts, bias=None):
    """(result, sum of |products|) in fp64, whatever the inputs' type."""
    M, N = x.shape[0], w.shape[1]
    y = torch.zeros((M, N), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    for e, r in spans(counts):
        a, b = x[r].double(), w[e].double()
        y[r], mag[r] = a @ b.t(), a.abs() @ b.abs().t()
        if bias is not None:
            y[r] += bias[e].double()
            mag[r] += bias[e].double().abs()
    return y, mag


def dgrad64(dy, w, counts):
    return fprop64(dy, w.transpose(1, 2), counts)


def wgrad64(dy, x, counts):
    dw, mag = [], []
    for _, r in spans(counts):
        a, b = dy[r].double(), x[r].double()
        dw.append(a.t() @ b)
        mag.append(a.abs().t() @ b.abs())
    return torch.stack(dw), torch.stack(mag)


# Products of bf16 (or of whole numbers held in f16) are exact in fp32. The
# tensor core adds them 16 at a time to an fp32 accumulator; each such step may
# lose up to one unit in the last place of the largest magnitude involved,
# 2^-23, twice (alignment of the products, then the accumulator), and no
# magnitude exceeds the sum of the products' magnitudes. So a sum over `red`
# terms is within (red / 16 + 1) 2^-22 of it, plus one fp32 rounding each for a
# bias and two scales (4 x 2^-24), plus bf16's unit roundoff 2^-8 when it is
# rounded to bf16.
def sum_tolerance(red, bf16):
    return (red / 16 + 2) * 2.0 ** -22 + 4 * 2.0 ** -24 + (2.0 ** -8 if bf16 else 0.0)


def assert_products(got, ref, mag, red, what=""):
    got = got.double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), what
    err = (got - ref).abs()
    bound = sum_tolerance(red, True if what == "bf16" else False) * mag
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert worst <= 0, (what, worst, (err / mag.clamp(min=1e-300)).max().item())


def philox_words(seed, offset, n):
    """The first n 16-bit words of Philox 4x32-10 at counters (0, offset), (1, offset), ... under `seed`."""
    u = np.uint64
    m32 = u(0xFFFFFFFF)
    block = np.arange((n + 7) // 8, dtype=np.uint64)
    c = [block & m32, block >> u(32), np.full_like(block, offset & 0xFFFFFFFF),
         np.full_like(block, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k[0]), b & m32, (a >> u(32)) ^ c[3] ^ u(k[1]), a & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=1).astype("<u4").view("<u2").reshape(-1)[:n]


def keep_mask(seed, offset, p, shape):
    n = int(np.prod(shape))
    t = int(np.rint(p * 65536))
    return torch.from_numpy((philox_words(seed, offset, n).astype(np.int64) >= t).reshape(shape))


def keep_scale(p):
    t = int(np.rint(p * 65536))
    return 0.0 if t == 65536 else 65536.0 / (65536 - t)


def swiglu64(y):
    g, u = y.double().chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


def swiglu_grad64(dh, y):
    g, u = y.double().chunk(2, dim=1)
    s = torch.sigmoid(g)
    d = dh.double()
    return torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], dim=1)

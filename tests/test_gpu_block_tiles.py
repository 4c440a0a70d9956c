"""fp8 and gated products where every CTA computes several full-width tiles, one after another: staging boxes, factor
groups, accumulators and the rows' exchange are used again, and every row of the results is compared."""
import pytest
import torch

from ._blocks import fp8_tolerance, row_values, weight_values
from ._ragged import dgrad64, fprop64
from .test_gpu_fp8 import make, mxq, splits  # noqa: F401 (mxq is a fixture)
from .test_gpu_ragged_swiglu import APPROX, HALF, check, dgrad_reference, fprop_reference, normal

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

PAIRS = [3000, 0, 1777, 5001]                               # 195 tiles of 256 features and more, for 76 pairs of SMs
ONE_SM = [60 + (37 * e) % 69 for e in range(64)]            # 320 tiles for 152 SMs
FEW = [(5 * e) % 17 for e in range(64)]                     # tiles of up to 32 rows


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts", [PAIRS, ONE_SM, FEW], ids=["pairs", "one_sm", "few"])
def test_fp8(mxq, counts, dtype):  # noqa: F811
    """Sums of 12 blocks forward and 9 backward: whole and broken groups of factors, three to a tile."""
    N, K = 1040, 1424
    x, xs, w, ws = make(7, counts, N, K, False)
    bias = normal(3, len(counts), N, std=100.0)
    ms = splits(counts)
    y = mxq.fp8_gemm_fprop(x, xs, w, ws, ms, bias=bias, out_dtype=dtype)
    ref, mag = fprop64(row_values(x, xs), weight_values(w, ws), counts, bias)
    assert ((y.double() - ref).abs() <= fp8_tolerance(K, dtype) * mag).all(), ((y.double() - ref).abs() / mag).max()
    assert torch.equal(y, mxq.fp8_gemm_fprop(x, xs, w, ws, ms, bias=bias, out_dtype=dtype))
    d, ds, w, ws = make(8, counts, N, K, True)
    dx = mxq.fp8_gemm_dgrad(d, ds, w, ws, ms, out_dtype=dtype)
    ref, mag = dgrad64(row_values(d, ds), weight_values(w, ws), counts)
    assert ((dx.double() - ref).abs() <= fp8_tolerance(N, dtype) * mag).all(), ((dx.double() - ref).abs() / mag).max()
    assert torch.equal(dx, mxq.fp8_gemm_dgrad(d, ds, w, ws, ms, out_dtype=dtype))


@pytest.mark.parametrize("counts", [PAIRS, FEW], ids=["pairs", "few"])
def test_gated(mxq, counts):  # noqa: F811
    F, K = 1032, 1416
    M, E, ms = sum(counts), len(counts), splits(counts)
    x, w, b = normal(1, M, K + 24)[:, :K], normal(2, E, 2 * F, K, std=1.5 * K ** -0.5), normal(3, E, 2 * F)
    h, eh, y, ey = fprop_reference(x, w, counts, b)
    got, got_y = mxq.ragged_gemm_fprop_swiglu(x, w, ms, bias=b, y_out=True)
    check(got, h, eh, "h")
    check(got_y, y, ey, "y")
    again = mxq.ragged_gemm_fprop_swiglu(x, w, ms, bias=b, y_out=True)
    assert torch.equal(got, again[0]) and torch.equal(got_y, again[1])
    del h, eh, y, ey
    w2 = normal(4, E, K, F, std=K ** -0.5)
    d, ed, h = dgrad_reference(x, w2, got_y, counts)
    got_d, got_h = mxq.ragged_gemm_dgrad_swiglu(x, w2, got_y, ms, h_out=True)
    check(got_d, d, ed, "dy1")
    check(got_h, h, APPROX * h.abs(), "h again")
    again = mxq.ragged_gemm_dgrad_swiglu(x, w2, got_y, ms, h_out=True)
    assert torch.equal(got_d, again[0]) and torch.equal(got_h, again[1])


# one tile a pair, and 108 tiles for 76 pairs
@pytest.mark.parametrize("counts,F", [([300, 3], 72), ([1500, 0, 499], 1416)])
def test_gated_long_sums(mxq, counts, F):  # noqa: F811
    """Sums of more than 2^15 terms of one sign on pairs of SMs: pieces of 8192 terms (2^-23 of the sum per 16 at most,
    twice), joined in fp32."""
    K, M, E = (1 << 15) + 264, sum(counts), len(counts)
    x, w = normal(1, M, K).abs_(), normal(2, E, 2 * F, K, std=2.0 ** -15).abs_()
    h, _, y, _ = fprop_reference(x, w, counts, None)
    got, got_y = mxq.ragged_gemm_fprop_swiglu(x, w, splits(counts), y_out=True)
    rel = (8192 / 16 + 8) * 2.0 ** -22
    assert ((got_y.double() - y).abs() <= (HALF + rel) * y).all()
    check(got, h, 2.2 * rel * h.abs() * (1 + y[:, :F]), "h")
    del w, h, y
    w2, y1 = normal(4, E, K, F, std=2.0 ** -15).abs_(), normal(5, M, 2 * F)
    d, _, _ = dgrad_reference(x, w2, y1, counts)
    got = mxq.ragged_gemm_dgrad_swiglu(x, w2, y1, splits(counts))
    check(got, d, (rel + APPROX) * dgrad_size(x, w2, y1, counts), "dy1")


def dgrad_size(dy, w, y, counts):
    """|dh| times the magnitudes of the terms of SwiGLU's derivatives."""
    dh = dgrad64(dy, w, counts)[1]
    g, u = y.double().chunk(2, dim=1)
    s = torch.sigmoid(g)
    return torch.cat([dh * (u * s).abs() * (1 + g.abs()), dh * (g * s).abs()], dim=1)

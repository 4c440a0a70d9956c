"""fp8 products whose two scales are far apart: their products at both ends of what the calls allow, and beyond it."""
import pytest
import torch

from ._blocks import E4M3, fp8_tolerance, row_values, weight_values
from ._ragged import dgrad64, fprop64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# An absolute error beside the relative one, where values are below 2^-126: half a step of the type (2^-134, 2^-150) for
# the last rounding, half a step of fp32 for each block's addition; and as the calls say, half a step of fp32 for the product
# of the two scales, which the block's sum of products multiplies.
SUBNORMAL = {BF16: 2.0 ** -134, F32: 2.0 ** -150}
# few rows with split sums and without, tiles of one SM, pairs
COUNTS = [[4], [7, 0, 9], [5, 0, 32, 1], [100, 0, 60], [300, 0, 129]]


@pytest.fixture(scope="module")
def mxq():
    import moe_expert_grouped_group_gb300 as m

    return m


def make(seed, counts, N, K, dgrad):
    """Blocks of the weight along the sum have scales near 2^-32 and near 2^58 in turn, the latter with the smallest codes.
    Rows in turn: ordinary scales; codes 0, and then the smallest codes, under scales whose product with the large ones is
    2^125 to 2^127.9; codes in the first kind of blocks only, under scales whose product is 2^-146 to 2^-123."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, E, red = sum(counts), len(counts), N if dgrad else K
    blocks = -(-red // 128)
    spread = lambda lo, hi, *shape: torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g).exp2()  # noqa: E731
    codes = lambda *shape: torch.empty(shape, device="cuda").normal_(generator=g).mul_(100).clamp_(-448, 448)  # noqa: E731
    smallest = lambda v: torch.where(v < 0, -2.0 ** -9, 2.0 ** -9)  # noqa: E731
    w, x = codes(E, N, K), codes(M, red)
    odd = torch.arange(red, device="cuda") // 128 % 2 == 1
    w = torch.where(odd[None, :, None] if dgrad else odd[None, None, :], smallest(w), w).to(E4M3)
    big = torch.arange(blocks, device="cuda") % 2 == 1
    big = big[None, :, None] if dgrad else big[None, None, :]
    shape = (E, -(-N // 128), -(-K // 128))
    ws = torch.where(big, spread(58, 60, *shape), spread(-36, -28, *shape))
    kind = torch.arange(M, device="cuda") % 4
    x[kind == 2] = smallest(x[kind == 2])
    x[kind == 1] = 0.0
    x[(kind == 3)[:, None] & odd[None, :]] = 0.0
    xs = spread(-4, 4, blocks, M)
    for k, lo, hi in ((1, 67, 67.9), (2, 67, 67.9), (3, -110, -95)):
        xs[:, kind == k] = spread(lo, hi, blocks, int((kind == k).sum()))
    return x.to(E4M3), xs, w, ws, kind


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
def test_both_ends(mxq, counts, dgrad, dtype):
    N, K = (656, 400) if dgrad else (272, 656)
    x, xs, w, ws, kind = make(sum(counts), counts, N, K, dgrad)
    y = (mxq.fp8_gemm_dgrad if dgrad else mxq.fp8_gemm_fprop)(x, xs, w, ws, torch.tensor(counts, device="cuda"), out_dtype=dtype)
    of = dgrad64 if dgrad else fprop64
    ref, mag = of(row_values(x, xs), weight_values(w, ws), counts)
    sums = of(x.float(), w.float(), counts)[1]
    err = fp8_tolerance(N if dgrad else K, dtype) * mag + SUBNORMAL[dtype] + (xs.shape[0] + sums) * SUBNORMAL[F32]
    assert ref.isfinite().all() and (y[kind == 1] == 0).all()
    assert ((y.double() - ref).abs() <= err).all(), [((y.double() - ref).abs() / err)[kind == k].max().item() for k in range(4)]


@pytest.mark.parametrize("counts", COUNTS[1:])
def test_beyond(mxq, counts):
    """Infinite and NaN scales, and those whose product is beyond fp32's range, leave other rows and channels alone."""
    N, K = 272, 656
    x, xs, w, ws, _ = make(1, counts, N, K, False)
    xs, ws = torch.ones_like(xs), torch.ones_like(ws)
    ms = torch.tensor(counts, device="cuda")
    clean = mxq.fp8_gemm_fprop(x, xs, w, ws, ms)
    xs[0, 1], xs[2, 2], xs[1, 3], ws[0, 1, 1] = float("inf"), float("nan"), 2.0 ** 100, 2.0 ** 40
    y = mxq.fp8_gemm_fprop(x, xs, w, ws, ms)
    assert not y[1:3].isfinite().any() and not y[3, 128:256].isfinite().any()
    same = torch.ones(sum(counts), N, dtype=torch.bool, device="cuda")
    same[1:3], same[3, :], same[:counts[0], 128:256] = False, False, False
    assert torch.equal(y[same], clean[same])
    y = mxq.fp8_gemm_fprop(x, xs, w, torch.ones_like(ws), ms)
    assert y[3].isfinite().all() and torch.equal(y[4:], clean[4:])

"""Each kernel that a ragged product may take (a pair of SMs; one SM, its sum whole or split over 2, 4 or 8; dot
products): that values stay where they belong, wrong counts write nothing, and fp32 results are as exact as fp32."""
import pytest
import torch

from tests._gpu import dev_i64, lib, require_gpu
from tests._ragged import assert_products, spans, wgrad64
from tests.test_gpu_ragged import rand

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# rows per expert that reach the dot products, the one-SM tiles and the pairs' tiles; the third expert is the bad one
GROUPS = {"dot": [1, 2, 3, 1, 0], "few": [7, 5, 30, 1, 9], "pair": [37, 5, 300, 1, 90]}


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3.0e38])
@pytest.mark.parametrize("group", GROUPS)
def test_values_stay_in_their_expert(mxq, group, value):
    counts, N, K = GROUPS[group], 136, 80
    M, ms = sum(counts), dev_i64(counts)
    x, dy, w = rand(1, M, K), rand(2, M, N), rand(3, 5, N, K)
    bad = slice(sum(counts[:2]), sum(counts[:3]))
    xb, dyb, wb = x.clone(), dy.clone(), w.clone()
    xb[bad], dyb[bad], wb[2] = value, value, value
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for dt in (BF16, F32):
        assert torch.equal(mxq.ragged_gemm_fprop(xb, wb, ms, out_dtype=dt)[keep],
                           mxq.ragged_gemm_fprop(x, w, ms, out_dtype=dt)[keep])
        assert torch.equal(mxq.ragged_gemm_dgrad(dyb, wb, ms, out_dtype=dt)[keep],
                           mxq.ragged_gemm_dgrad(dy, w, ms, out_dtype=dt)[keep])
        others = torch.tensor([0, 1, 3, 4], device="cuda")
        assert torch.equal(mxq.ragged_gemm_wgrad(dyb, xb, ms, out_dtype=dt)[others],
                           mxq.ragged_gemm_wgrad(dy, x, ms, out_dtype=dt)[others])
    if value != value:
        assert torch.isnan(mxq.ragged_gemm_fprop(xb, wb, ms)[bad]).all()
        assert torch.isnan(mxq.ragged_gemm_dgrad(dyb, wb, ms)[bad]).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("group", GROUPS)
def test_int8_rows_and_channels_stay_alone(mxq, group, value):
    """A row without a scale, and a channel whose weights have none."""
    counts, N, K = GROUPS[group], 136, 80
    M, ms = sum(counts), dev_i64(counts)
    x, w = rand(1, M, K), rand(3, 5, N, K)

    def run(x, w, dt):
        wq, ws = mxq.int8_quantize_rows(w.view(5 * N, K))
        return mxq.int8_gemm_fprop(*mxq.int8_quantize_rows(x), wq.view(5, N, K), ws.view(5, N), ms, out_dtype=dt)

    xb, wb = x.clone(), w.clone()
    row, channel = sum(counts[:2]), 37
    xb[row, 11], wb[2, channel, 5] = value, value
    third = slice(sum(counts[:2]), sum(counts[:3]))
    for dt in (BF16, F32):
        got, clean = run(xb, wb, dt), run(x, w, dt)
        nan = torch.zeros_like(clean, dtype=torch.bool)
        nan[row], nan[third, channel] = True, True
        assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], clean[~nan])


# M rows that are right for none of these: too few, too many, one negative, one that alone passes M
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("change,bits", [((0, 0, -1, 0, 0), 4), ((0, 1, 0, 0, 0), 4), ((-1000, 1000, 0, 0, 0), 6),
                                         ((0, 0, 0, 0, 1 << 40), 4)], ids=str)
def test_wrong_counts(mxq, group, change, bits):
    counts, N, K = GROUPS[group], 136, 80
    M, ms = sum(counts), dev_i64([c + d for c, d in zip(counts, change)])
    x, dy, w = rand(1, M, K), rand(2, M, N), rand(3, 5, N, K)
    xq, xs = mxq.int8_quantize_rows(x)
    wq, ws = mxq.int8_quantize_rows(w.view(5 * N, K))
    wq, ws = wq.view(5, N, K), ws.view(5, N)
    for dt in (BF16, F32):
        for call, shape in ((lambda s, o: mxq.ragged_gemm_fprop(x, w, ms, status=s, out=o), (M, N)),
                            (lambda s, o: mxq.ragged_gemm_dgrad(dy, w, ms, status=s, out=o), (M, K)),
                            (lambda s, o: mxq.ragged_gemm_wgrad(dy, x, ms, status=s, out=o), (5, N, K)),
                            (lambda s, o: mxq.int8_gemm_fprop(xq, xs, wq, ws, ms, status=s, out=o), (M, N))):
            s, out = mxq.new_status(), torch.full(shape, 7.0, dtype=dt, device="cuda")
            call(s, out)
            assert mxq.status_read(s) == bits and bool((out == 7).all())


# The tensor core's truncations are at most 32 in an accumulator (512 terms), each under 2^-23 of what it holds:
# for terms of random sign some 2^-21 of the sum in the 2-norm, whatever the number of accumulators. The bound
# leaves a factor of two; one accumulator of 4096 terms (256 truncations) would pass it.
@pytest.mark.parametrize("counts,wide", [([1], 136), ([3], 520), ([20], 1280), ([20], 2560), ([20], 5120), ([20], 10240),
                                         ([300], 520), ([70, 0, 200], 136)],
                         ids=["dot1", "dot3", "split8", "split4", "split2", "whole", "pair", "pairs"])
@pytest.mark.parametrize("depth", [4096, 7168])
def test_fp32_results_are_as_exact_as_fp32(mxq, counts, wide, depth):
    M, E, ms = sum(counts), len(counts), dev_i64(counts)
    t, w = rand(1, M, depth), rand(2, E, wide, depth)
    ref = torch.zeros((M, wide), dtype=torch.float64, device="cuda")
    for e, r in spans(counts):
        ref[r] = t[r].double() @ w[e].double().t()
    for got in (mxq.ragged_gemm_fprop(t, w, ms, out_dtype=F32),
                mxq.ragged_gemm_dgrad(t, w.transpose(1, 2).contiguous(), ms, out_dtype=F32)):
        assert ((got.double() - ref).norm() / ref.norm()).item() < 2.0 ** -20


def test_each_experts_gradient_by_its_own_length(mxq):
    counts, N, K = [1, 2049, 0, 7, 513, 16], 136, 264
    M = sum(counts)
    dy, x = rand(1, M, N), rand(2, M, K)
    ref, mag = wgrad64(dy, x, counts)
    dw = mxq.ragged_gemm_wgrad(dy, x, dev_i64(counts))
    half = mxq.ragged_gemm_wgrad(dy, x, dev_i64(counts), out_dtype=BF16)
    for e, m in enumerate(counts):
        assert_products(dw[e], ref[e], mag[e], min(m, 512), "f32")
        assert_products(half[e], ref[e], mag[e], m, "bf16")

"""Sums of the int8 product past 2^24, where an fp32 accumulator that truncates would lose bits: codes of one
sign, each kernel shape (dot products, one SM, a pair of SMs) and depth."""
import pytest
import torch

from tests._gpu import dev_i64, lib, require_gpu
from tests._ragged import spans
from tests.test_gpu_ragged import rand

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
WHOLE = (1 << 17) - 16  # the deepest sum that 32-bit integers hold whatever the codes
# rows: single tokens, a few rows an expert, many
SHAPES = {"dot": [1, 0, 3], "few": [17, 0, 30], "pair": [130, 0, 257, 1]}


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


def inputs(counts, N, K, lo, hi, seed=3):
    M, E = sum(counts), len(counts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = lambda *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g, device="cuda") + 0.01  # noqa: E731
    return code(M, K), u(M), code(E, N, K), u(E, N), rand(4, E, N, std=100.0)


def sums64(xq, wq, counts):
    return torch.cat([xq[r].double() @ wq[e].double().t() for e, r in spans(counts)])  # whole numbers below 2^53


def steps32(xq, xs, wq, ws, bias, counts):
    """The definition: the sum rounded to fp32 once, then one fp32 rounding for each scale and the bias."""
    s = sums64(xq, wq, counts).float()
    return torch.cat([s[r] * xs[r, None] * ws[e] + bias[e].float() for e, r in spans(counts)])


@pytest.mark.parametrize("lo,hi", [(100, 128), (-128, -99), (-128, 128)])
@pytest.mark.parametrize("N,K", [(136, 1024), (136, 1040), (264, 2048), (72, 7168), (136, 33792), (8, WHOLE)])
@pytest.mark.parametrize("shape", SHAPES)
def test_fp32_results_are_the_definitions_bits(mxq, shape, N, K, lo, hi):
    counts = SHAPES[shape]
    xq, xs, wq, ws, bias = inputs(counts, N, K, lo, hi)
    y = mxq.int8_gemm_fprop(xq, xs, wq, ws, dev_i64(counts), bias=bias, out_dtype=F32)
    assert torch.equal(y, steps32(xq, xs, wq, ws, bias, counts))


@pytest.mark.parametrize("K", [1024, 1040, 2048, 7168, 32768, 32784, WHOLE])
@pytest.mark.parametrize("shape", SHAPES)
def test_bf16_results(mxq, shape, K):
    counts, N = SHAPES[shape], 40
    xq, xs, wq, ws, bias = inputs(counts, N, K, 100, 128)
    y = mxq.int8_gemm_fprop(xq, xs, wq, ws, dev_i64(counts), bias=bias)
    want = steps32(xq, xs, wq, ws, bias, counts)
    if shape == "dot" or K <= 1024 or K > 32768:
        assert torch.equal(y, want.to(BF16))
    else:  # one truncation of 2^-23 per 16 of K, the three fp32 steps, the rounding to bf16's 8 bits
        mag = torch.cat([sums64(xq, wq, counts)[r] * xs[r, None].double() * ws[e].double() + bias[e].double().abs()
                         for e, r in spans(counts)])
        assert torch.all((y.double() - want.double()).abs() <= (K / 16 * 2.0 ** -23 + 2.0 ** -8) * mag)


@pytest.mark.parametrize("shape", SHAPES)
def test_sums_beyond_32_bits(mxq, shape):
    """Every code -128: pieces of 1024 are 2^24, exact, and are added in fp32 with one rounding each at most."""
    counts, N, K = SHAPES[shape], 24, (1 << 18) + 48
    xq, _, wq, _, _ = inputs(counts, N, K, -128, -127)
    one, ones = torch.ones(sum(counts), device="cuda"), torch.ones((len(counts), N), device="cuda")
    y = mxq.int8_gemm_fprop(xq, one, wq, ones, dev_i64(counts), out_dtype=F32)
    assert torch.all((y.double() - K * 16384.0).abs() <= (K / 1024 + 1) * 2.0 ** -24 * K * 16384.0)


def test_a_token_alone_and_in_a_batch(mxq):
    xq, xs, wq, ws, bias = inputs([300], 264, 4096, 90, 128)
    batch = mxq.int8_gemm_fprop(xq, xs, wq, ws, dev_i64([300]), bias=bias, out_dtype=F32)
    for m in (1, 20):
        alone = mxq.int8_gemm_fprop(xq[:m], xs[:m], wq, ws, dev_i64([m]), bias=bias, out_dtype=F32)
        assert torch.equal(alone, batch[:m])


@pytest.mark.parametrize("dt", [F32, BF16], ids=str)
@pytest.mark.parametrize("K,calls", [(2048, 400), (7168, 300)])
def test_stages_are_read_before_they_are_filled_again(mxq, dt, K, calls):
    """Whole tiles whose stores go on while the next tile's stages are loaded, again and again."""
    counts, N = [2049, 700], 1024
    xq, xs, wq, ws, _ = inputs(counts, N, K, -128, 128)
    ms, wrong = dev_i64(counts), torch.zeros((), dtype=torch.int64, device="cuda")
    zero = torch.zeros((2, N), dtype=BF16, device="cuda")
    want = steps32(xq, xs, wq, ws, zero, counts).to(dt)
    y = torch.empty_like(want)
    for _ in range(calls):
        y.fill_(float("nan"))
        mxq.int8_gemm_fprop(xq, xs, wq, ws, ms, out=y)
        wrong += (y != want).sum()
    assert wrong.item() == 0

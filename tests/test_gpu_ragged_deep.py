"""bf16 results of sums so long that a truncating fp32 accumulator would lose more than the rounding to bf16 does:
terms of one sign, 2^15 to 2^24 of them."""
import pytest
import torch

from tests._gpu import dev_i64, lib, require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# The rounding to bf16 (2^-8 of the value: 8 bits), and 2^-12 of the sum for what was lost before it: that is up to 2^15
# terms in one accumulator (2^-23 per 16), or the pieces of a longer sum and their additions.
REL = 2.0 ** -8 + 2.0 ** -12


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


def positive(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(*shape, generator=g, device="cuda").add_(0.5).to(BF16)


def dot64(a, b):
    """a^T b in fp64, a million rows at a time."""
    out = torch.zeros((a.shape[1], b.shape[1]), dtype=torch.float64, device="cuda")
    for i in range(0, a.shape[0], 1 << 20):
        out += a[i:i + (1 << 20)].double().t() @ b[i:i + (1 << 20)].double()
    return out


@pytest.mark.parametrize("accumulate", [False, True], ids=["new", "added"])
@pytest.mark.parametrize("counts,N,K", [([1 << 24], 8, 8), ([1 << 22, 0, 40, 32768, 32769], 24, 40),
                                        ([(1 << 19) + 77, 5, 1 << 16], 264, 520)], ids=str)
def test_wgrad(mxq, counts, N, K, accumulate):
    M, E = sum(counts), len(counts)
    dy, x, ms = positive(1, M, N), positive(2, M, K), dev_i64(counts)
    prior = positive(3, E, N, K) * 4096
    out = mxq.ragged_gemm_wgrad(dy, x, ms, accumulate=accumulate, out=prior.clone())
    off = 0
    for e, m in enumerate(counts):
        want = dot64(dy[off:off + m], x[off:off + m])
        off += m
        if accumulate:
            want += prior[e].double()
        assert torch.all((out[e].double() - want).abs() <= REL * want), (e, m)
    if accumulate:
        assert all(torch.equal(out[e], prior[e]) for e, m in enumerate(counts) if m == 0)


@pytest.mark.parametrize("counts", [[70], [40, 0, 300], [20]], ids=str)
@pytest.mark.parametrize("depth", [32768, 32776, 1 << 18, 1 << 20])
def test_fprop_and_dgrad(mxq, counts, depth):
    M, E, ms = sum(counts), len(counts), dev_i64(counts)
    t, w, bias = positive(1, M, depth), positive(2, E, 8, depth), positive(3, E, 8) * 1024
    y = mxq.ragged_gemm_fprop(t, w, ms, bias=bias)
    dx = mxq.ragged_gemm_dgrad(t, w.transpose(1, 2).contiguous(), ms)
    off = 0
    for e, m in enumerate(counts):
        want = dot64(t[off:off + m].t(), w[e].t())
        assert torch.all((dx[off:off + m].double() - want).abs() <= REL * want)
        want += bias[e].double()
        assert torch.all((y[off:off + m].double() - want).abs() <= REL * want)
        off += m

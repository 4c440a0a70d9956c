"""The ragged operators together, on split sums, past 32-bit offsets, on a
busy stream, and as the example runs them."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests._gpu import dev_i64, lib, require_gpu
from tests._ragged import assert_products, dgrad64, fprop64, philox_words, wgrad64
from tests.test_gpu_ragged import rand

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


# one-SM tiles whose sum is split over 2, 4 and 8 CTAs (deep sums, few tiles), a last stage that is not whole,
# several tiles to a cluster, one token and as many as a tile holds
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [16], [17, 0, 5], [32], [31, 33]])
@pytest.mark.parametrize("N,K", [(136, 2048), (264, 4104), (2056, 1032), (4096, 520), (72, 7168)])
def test_split_sums(mxq, counts, N, K):
    M, E, ms = sum(counts), len(counts), dev_i64(counts)
    x, dy, w, bias = rand(1, M, K), rand(2, M, N), rand(3, E, N, K), rand(4, E, N)
    for dt, tag in ((BF16, "bf16"), (F32, "f32")):
        y = mxq.ragged_gemm_fprop(x, w, ms, bias=bias, out_dtype=dt)
        assert_products(y, *fprop64(x, w, counts, bias), K, tag)
        assert torch.equal(y, mxq.ragged_gemm_fprop(x, w, ms, bias=bias, out_dtype=dt))
        assert_products(mxq.ragged_gemm_dgrad(dy, w, ms, out_dtype=dt), *dgrad64(dy, w, counts), N, tag)


def test_fp32_sums_are_as_exact_as_fp32(mxq):
    """fp32 results over a long sum: no further from the exact ones than an fp32 matrix product that adds
    term by term may be (random signs: about sqrt(terms) roundings; the bound allows 2^-20 in the 2-norm)."""
    x, dy, ms = rand(1, 4096, 264), rand(2, 4096, 136), dev_i64([4096])
    dw = mxq.ragged_gemm_wgrad(dy, x, ms)
    ref = dy.double().t() @ x.double()
    assert ((dw[0].double() - ref).norm() / ref.norm()).item() < 2.0 ** -20


# dW matrices that end inside a tile, a pair's second half and a 32 x 32 piece, every matrix beside another's
@pytest.mark.parametrize("N,K", [(8, 8), (24, 40), (40, 136), (264, 264), (520, 1000), (1000, 520)])
@pytest.mark.parametrize("dt,tag", [(BF16, "bf16"), (F32, "f32")])
def test_wgrad_writes_its_matrices_only(mxq, N, K, dt, tag):
    counts, pad = [3, 0, 70, 1, 200], 4096
    E, M = len(counts), sum(counts)
    dy, x = rand(1, M, N), rand(2, M, K)
    whole = torch.full((2 * pad + E * N * K,), 7.0, device="cuda", dtype=dt)
    out = whole[pad:-pad].view(E, N, K)
    out.fill_(float("nan"))
    mxq.ragged_gemm_wgrad(dy, x, dev_i64(counts), out=out)
    assert bool((whole[:pad] == 7.0).all()) and bool((whole[-pad:] == 7.0).all())
    assert not bool(out[1].any())
    assert_products(out, *wgrad64(dy, x, counts), max(counts), tag)


# adding to dW: fp32 is exactly one fp32 addition of the call's sums, at subnormals, infinities and NaN too; bf16 is
# rounded once, from the fp32 sum with the old value; an empty expert's matrix and everything beside stay as they were
@pytest.mark.parametrize("N,K", [(8, 8), (40, 136), (264, 264), (1000, 520)])
@pytest.mark.parametrize("counts", [[3, 0, 70, 1, 200], [0, 1500, 1]])
def test_wgrad_adds_once(mxq, N, K, counts):
    E, M, pad, ms = len(counts), sum(counts), 4096, dev_i64(counts)
    dy, x = rand(1, M, N), rand(2, M, K)
    dy[:, 1], dy[:, 2] = 2.0 ** -126, 0.0  # sums about the smallest normal number; sums of 0
    prior = rand(5, E, N, K).float() * 3
    prior[:, 1] = 2.0 ** -127
    prior[:, 3], prior[:, 4], prior[:, 5] = float("nan"), float("inf"), -0.0
    dw = mxq.ragged_gemm_wgrad(dy, x, ms)
    whole = torch.full((2 * pad + E * N * K,), 7.0, device="cuda")
    out = whole[pad:-pad].view(E, N, K)
    out.copy_(prior)
    mxq.ragged_gemm_wgrad(dy, x, ms, out=out, accumulate=True)
    full = [e for e in range(E) if counts[e]]
    want = prior.clone()
    want[full] = (prior.cpu()[full] + dw.cpu()[full]).cuda()
    assert torch.equal(out.nan_to_num(1e30), want.nan_to_num(1e30)) and torch.equal(out.isnan(), want.isnan())
    assert bool((whole[:pad] == 7.0).all()) and bool((whole[-pad:] == 7.0).all())
    whole = torch.full((2 * pad + E * N * K,), 7.0, device="cuda", dtype=BF16)
    out = whole[pad:-pad].view(E, N, K)
    out.copy_(prior)
    ref, mag = wgrad64(dy, x, counts)
    old = out.double()
    mxq.ragged_gemm_wgrad(dy, x, ms, out=out, accumulate=True)
    finite = old[0, :, 0].isfinite()  # rows 3 and 4 hold the NaN and the infinities
    finite[1] = False  # subnormal in bf16: no relative bound
    assert_products(out[:, finite], ref[:, finite] + old[:, finite], mag[:, finite] + old[:, finite].abs(), max(counts), "bf16")
    assert bool(out[:, 3].isnan().all()) and bool((out[:, 4] == float("inf")).all())
    assert bool((whole[:pad] == 7.0).all()) and bool((whole[-pad:] == 7.0).all())


def test_offsets_past_32_bits(mxq):
    M, N, K = 70000, 32768, 8  # 2.3e9 outputs
    x, w, counts = rand(1, M, K), rand(3, 2, N, K), [40001, 29999]
    y = mxq.ragged_gemm_fprop(x, w, dev_i64(counts))
    rows = torch.tensor([0, 40000, 40001, 65535, 65536, 65537, M - 1], device="cuda")
    for r in rows.tolist():
        ref, mag = fprop64(x[r:r + 1], w[int(r >= counts[0])][None], [1])
        assert_products(y[r:r + 1], ref, mag, K, "bf16")
    del y
    dy = rand(2, 24, N)  # dW of 2.6e9 entries, its last expert's beyond 2^32 bytes
    xk = rand(4, 24, 40000)
    dw = mxq.ragged_gemm_wgrad(dy, xk, dev_i64([20, 4]), out_dtype=BF16)
    for e, r in ((0, slice(0, 20)), (1, slice(20, 24))):
        for n in (0, 17000, N - 1):
            a, b = dy[r, n:n + 1].double(), xk[r].double()
            assert_products(dw[e, n:n + 1], a.t() @ b, a.abs().t() @ b.abs(), 20, "bf16")


def test_dropout_past_32_bits(mxq):
    n = (1 << 32) + 1003
    x = torch.ones(n, dtype=BF16, device="cuda")
    out = mxq.dropout(x, torch.tensor([9, 10], device="cuda"), 0.5, out=x)
    for at in (0, (1 << 31) - 8, (1 << 32) - 8, (1 << 32), n - 16 - n % 8):
        block = at // 8
        want = words_at(block, 9, 10)
        got = (out[block * 8:block * 8 + 8] != 0).cpu().numpy()
        assert np.array_equal(got, want >= 32768), at
    tail = (out[n - n % 8:] != 0).cpu().numpy()
    assert np.array_equal(tail, words_at(n // 8, 9, 10)[:n % 8] >= 32768)


def words_at(block, seed, offset):
    """The eight words of one counter, which may be past 32 bits."""
    c = [block & 0xFFFFFFFF, block >> 32, offset & 0xFFFFFFFF, offset >> 32]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.array([h for v in c for h in (v & 0xFFFF, v >> 16)])


def test_words_at_is_the_vector_definition():
    assert np.array_equal(words_at(3, 77, 1 << 35), philox_words(77, 1 << 35, 32)[24:])


def test_back_to_back_calls_see_each_others_results(mxq):
    """Calls may begin while the one before ends: a chain on one stream, repeated, with inputs that the
    stream itself writes just before, gives what separate, synchronized calls give."""
    counts, H, F = [70, 0, 3, 55], 136, 64
    M, ms = sum(counts), dev_i64(counts)
    w1, w2 = rand(1, 4, 2 * F, H, std=0.1), rand(2, 4, H, F, std=0.1)
    rng = torch.tensor([1, 0], device="cuda")

    def chain(x, sync):
        done = torch.cuda.synchronize if sync else lambda: None
        for i in range(4):
            rng[1] = i
            done()
            y1 = mxq.ragged_gemm_fprop(x, w1, ms)
            done()
            h = mxq.swiglu_dropout_fwd(y1, rng, 0.3)
            done()
            q, s = mxq.int8_quantize_rows(h)
            done()
            y = mxq.ragged_gemm_fprop(h, w2, ms)
            done()
            x = mxq.dropout(y, rng, 0.3, residual=x)
            done()
        return x, q, s

    x = rand(3, M, H)
    want = chain(x, True)
    for _ in range(20):
        got = chain(x, False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_example_trains_and_serves(mxq):
    spec = importlib.util.spec_from_file_location("ragged_expert_mlp", os.path.join(ROOT, "examples", "ragged_expert_mlp.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, err = ex.main()
    assert losses[-1] < 0.8 * losses[0] and all(np.isfinite(losses))
    assert err < 0.05

"""int8 row quantizer and ragged int8 products against their definitions."""
import pytest
import torch

from tests._gpu import dev_i64, lib, require_gpu
from tests._ragged import assert_products, fprop64, spans
from tests.test_gpu_ragged import GROUPS, rand

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


def quantize32(x):
    """The definition's fp32 steps, on the host."""
    x = x.float().cpu()
    top = x.abs().amax(dim=1, keepdim=True).clamp(min=2.0 ** -100)
    most = torch.full_like(top, 127.0)  # torch divides a scalar by a tensor through its reciprocal
    q = torch.round(x * (most / top)).clamp(-127, 127)
    bad = ~torch.isfinite(x).all(dim=1)
    q[bad] = 0
    return q.to(torch.int8), torch.where(bad, torch.full_like(top[:, 0], float("nan")), (top / most)[:, 0])


@pytest.mark.parametrize("M,K,pad", [(1, 16, 0), (3, 48, 8), (5, 2048, 0), (7, 2064, 64), (300, 512, 0), (2, 20000, 0),
                                     (1300, 80, 0)])
def test_quantizer(mxq, M, K, pad):
    x = rand(1, M, K, pad=pad)
    q, s = mxq.int8_quantize_rows(x)
    qr, sr = quantize32(x)
    assert torch.equal(q.cpu(), qr) and torch.equal(s.cpu(), sr)


def test_quantizer_edges(mxq):
    x = torch.zeros((8, 32), device="cuda")
    x[1, 5] = 1e-38                                   # below 2^-100: codes 0 by the floor on the maximum
    x[2, :] = torch.linspace(-127, 127, 32, device="cuda").round() * 0.5  # ties and exact halves
    x[3, 0], x[3, 1] = 3.3e38, -1.0
    x[4, 7] = float("inf")
    x[5, 31] = float("nan")
    x[6, :] = -2.0
    x[7, 0], x[7, 1:] = 127.0, torch.arange(1, 32, device="cuda") - 16.5  # ties to even
    x = x.to(BF16)
    q, s = mxq.int8_quantize_rows(x)
    qr, sr = quantize32(x)
    assert torch.equal(q.cpu(), qr)
    assert torch.equal(torch.isnan(s.cpu()), torch.isnan(sr)) and torch.isnan(sr).sum() == 2
    ok = ~torch.isnan(sr)
    assert torch.equal(s.cpu()[ok], sr[ok])
    assert torch.all(q[0] == 0) and torch.all(q[1] == 0)


@pytest.mark.parametrize("N,K", [(8, 16), (136, 80), (264, 1008), (520, 272), (1024, 2048)])
@pytest.mark.parametrize("group", GROUPS)
def test_products(mxq, group, N, K):
    counts = GROUPS[group]
    M, E = sum(counts), len(counts)
    g = torch.Generator(device="cuda").manual_seed(3)
    code = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    xq, wq = code(M, K), code(E, N, K)
    xs = torch.rand(M, generator=g, device="cuda") + 0.01
    ws = torch.rand(E, N, generator=g, device="cuda") + 0.01
    bias, ms = rand(4, E, N, std=100.0), dev_i64(counts)
    ref, mag = fprop64(xq, wq, counts)
    for e, r in spans(counts):
        f = xs[r, None].double() * ws[e].double()
        ref[r] *= f
        mag[r] *= f
    for dt, tag in ((BF16, "bf16"), (F32, "f32")):
        assert_products(mxq.int8_gemm_fprop(xq, xs, wq, ws, ms, out_dtype=dt), ref, mag, K, tag)
    rb, mb = ref.clone(), mag.clone()
    for e, r in spans(counts):
        rb[r] += bias[e].double()
        mb[r] += bias[e].double().abs()
    assert_products(mxq.int8_gemm_fprop(xq, xs, wq, ws, ms, bias=bias, out_dtype=F32), rb, mb, K, "f32")


def test_sums_are_exact_where_fp32_holds_them(mxq):
    """Every partial sum below 2^24: the product is the whole number itself."""
    counts, N, K = [5, 0, 70], 136, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    xq = torch.randint(-128, 128, (75, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-128, 128, (3, N, K), generator=g, device="cuda", dtype=torch.int8)
    xq[0], wq[0, 0] = -128, -128
    one, ones = torch.ones(75, device="cuda"), torch.ones((3, N), device="cuda")
    y = mxq.int8_gemm_fprop(xq, one, wq, ones, dev_i64(counts), out_dtype=F32)
    assert torch.equal(y.double(), fprop64(xq, wq, counts)[0])
    assert y[0, 0] == 256 * 128 * 128


def test_an_infinite_row_stays_one_row(mxq):
    x, w, ms = rand(1, 40, 64), rand(2, 2, 72, 64), dev_i64([17, 23])
    wq, ws = mxq.int8_quantize_rows(w.view(144, 64))
    run = lambda x: mxq.int8_gemm_fprop(*mxq.int8_quantize_rows(x), wq.view(2, 72, 64), ws.view(2, 72), ms)  # noqa: E731
    clean = run(x)
    x[16, 3] = float("inf")
    y = run(x)
    rest = torch.arange(40, device="cuda") != 16
    assert torch.isnan(y[16]).all() and torch.equal(y[rest], clean[rest])


def test_single_token_and_graph_replay(mxq):
    x, w = rand(1, 1, 2048), rand(2, 4, 264, 2048, std=0.02)
    wq, ws = mxq.int8_quantize_rows(w.view(-1, 2048))
    wq, ws, ms = wq.view(4, 264, 2048), ws.view(4, 264), dev_i64([0, 1, 0, 0])
    q, xs = torch.empty((1, 2048), dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    y = torch.empty((1, 264), dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.int8_quantize_rows(x, out=(q, xs))
        mxq.int8_gemm_fprop(q, xs, wq, ws, ms, out=y)
    for e in (1, 3, 0):
        ms.zero_()
        ms[e] = 1
        x.mul_(1.5)
        graph.replay()
        qr, sr = quantize32(x)
        assert torch.equal(q.cpu(), qr)
        ref, mag = fprop64(q, wq[e:e + 1], [1])
        f = xs.double()[:, None] * ws[e].double()
        assert_products(y, ref * f, mag * f, 2048, "bf16")


def test_wrong_counts_and_refusals(mxq):
    xq = torch.zeros((32, 64), dtype=torch.int8, device="cuda")
    wq = torch.zeros((2, 72, 64), dtype=torch.int8, device="cuda")
    xs, ws, ms = torch.ones(32, device="cuda"), torch.ones((2, 72), device="cuda"), dev_i64([16, 16])
    out = torch.full((32, 72), 7.0, dtype=BF16, device="cuda")
    for counts, bits in (([16, 15], 4), ([-16, 48], 6)):
        s = mxq.new_status()
        mxq.int8_gemm_fprop(xq, xs, wq, ws, dev_i64(counts), status=s, out=out)
        assert mxq.status_read(s) == bits and torch.all(out == 7)
    assert mxq.int8_gemm_fprop(xq[:0], xs[:0], wq, ws, dev_i64([0, 0])).shape == (0, 72)
    assert mxq.int8_quantize_rows(rand(1, 0, 64))[0].shape == (0, 64)
    for call in (
        lambda: mxq.int8_quantize_rows(rand(1, 4, 64).float()),
        lambda: mxq.int8_quantize_rows(rand(1, 4, 72)),                       # K % 16
        lambda: mxq.int8_quantize_rows(rand(1, 4, 64, pad=4)),                # stride % 8
        lambda: mxq.int8_quantize_rows(rand(1, 4, 64), out=(xq[:3], xs)),     # codes too small
        lambda: mxq.int8_gemm_fprop(xq.view(torch.uint8), xs, wq, ws, ms),
        lambda: mxq.int8_gemm_fprop(xq, xs.double(), wq, ws, ms),
        lambda: mxq.int8_gemm_fprop(xq, xs[:31], wq, ws, ms),
        lambda: mxq.int8_gemm_fprop(xq, xs, wq, ws[:1], ms),
        lambda: mxq.int8_gemm_fprop(xq[:, :48], xs, wq, ws, ms),
        lambda: mxq.int8_gemm_fprop(xq, xs, wq, ws, torch.tensor([16, 16])),
        lambda: mxq.int8_gemm_fprop(xq[:, :40].contiguous(), xs, wq[:, :, :40].contiguous(), ws, ms),
    ):
        with pytest.raises(mxq.MXQError):
            call()


# single tokens and a handful of rows an expert: dot products on the integer units; 9 rows in one of four
# experts are two slices of it; 17 and 40 rows an expert go to the tensor cores
@pytest.mark.parametrize("counts", [[1], [2], [3], [4], [0, 8], [9, 0, 0, 0], [1, 2, 3, 4, 5, 6], [0, 0, 0, 16, 0],
                                    [17], [40, 3]])
@pytest.mark.parametrize("N,K", [(8, 16), (24, 528), (136, 1008), (1000, 2048), (40, 7168)])
def test_few_rows(mxq, counts, N, K):
    M, E, ms = sum(counts), len(counts), dev_i64(counts)
    g = torch.Generator(device="cuda").manual_seed(5)
    code = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    xq, wq, bias = code(M, K), code(E, N, K), rand(4, E, N, std=100.0)
    xs, ws = torch.rand(M, generator=g, device="cuda") + 0.01, torch.rand(E, N, generator=g, device="cuda") + 0.01
    ref, mag = fprop64(xq, wq, counts)
    for e, r in spans(counts):
        f = xs[r, None].double() * ws[e].double()
        ref[r], mag[r] = ref[r] * f + bias[e].double(), mag[r] * f + bias[e].double().abs()
    for dt, tag in ((BF16, "bf16"), (F32, "f32")):
        y = mxq.int8_gemm_fprop(xq, xs, wq, ws, ms, bias=bias, out_dtype=dt)
        assert_products(y, ref, mag, K, tag)
        assert torch.equal(y, mxq.int8_gemm_fprop(xq, xs, wq, ws, ms, bias=bias, out_dtype=dt))


def test_the_largest_sums_of_the_integer_path(mxq):
    """K just below 2^17 with every code -128: the sum 2^31 - 2^18 still fits."""
    K = (1 << 17) - 16
    xq = torch.full((1, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((1, 8, K), -128, dtype=torch.int8, device="cuda")
    one, ones = torch.ones(1, device="cuda"), torch.ones((1, 8), device="cuda")
    y = mxq.int8_gemm_fprop(xq, one, wq, ones, dev_i64([1]), out_dtype=F32)
    assert torch.all(y == float(K * 16384))
    K = 1 << 17  # the tensor cores' fp32 sums
    xq, wq = xq.new_full((1, K), -128), wq.new_full((1, 8, K), -128)
    y = mxq.int8_gemm_fprop(xq, one, wq, ones, dev_i64([1]), out_dtype=F32)
    assert torch.all((y - K * 16384.0).abs() <= K / 16 * 2.0 ** -22 * K * 16384.0)

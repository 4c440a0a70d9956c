"""fp8 products with a scale per block, and their quantizers, against their 64-bit definitions."""
import pytest
import torch

from ._blocks import E4M3, fp8_tolerance, quantize_rows, quantize_weight, row_values, weight_values
from ._ragged import dgrad64, fprop64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mxq():
    import moe_expert_grouped_group_gb300 as m

    return m


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0, std, generator=g).to(BF16)


def splits(counts):
    return torch.tensor(counts, dtype=torch.int64, device="cuda")


def same_codes(got, want):
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def same_scales(got, want):
    assert got.shape == want.shape and torch.equal(got.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("M,K,pad", [(1, 16, 0), (1, 128, 0), (3, 144, 8), (31, 2048, 0), (33, 1424, 64), (257, 400, 16),
                                     (1000, 7168, 0)])
def test_quantize_rows(mxq, M, K, pad):
    x = normal(M + K, M, K + pad)
    x[:, ::7] *= 50.0  # magnitudes that differ from block to block
    x[M // 2, :128] = 0.0
    x = x[:, :K]
    q, s = mxq.fp8_quantize_rows(x)
    want_q, want_s = quantize_rows(x)
    same_codes(q, want_q)
    same_scales(s, want_s)


@pytest.mark.parametrize("E,N,K", [(1, 8, 16), (3, 72, 144), (2, 128, 128), (2, 264, 400), (5, 1000, 1424)])
def test_quantize_weight(mxq, E, N, K):
    w = normal(E + N + K, E, N, K, std=0.02)
    w[0, :8] *= 1000.0
    q, s = mxq.fp8_quantize_weight(w)
    want_q, want_s = quantize_weight(w)
    same_codes(q, want_q)
    same_scales(s, want_s)


def test_quantize_extremes(mxq):
    """Zeros of both signs, subnormals, the largest and the smallest values, infinities, NaN, and their neighbours."""
    x = torch.zeros(8, 256, dtype=BF16, device="cuda")
    x[0, 5] = -0.0
    x[1, 3], x[1, 200] = 3e38, 1e-38
    x[2, 0], x[2, 1] = 2.0 ** -133, 2.0 ** -126
    x[3, 130] = float("inf")
    x[4, 127] = float("nan")
    x[5, 0], x[5, 1:100] = -448.0, 0.0009765625
    x[6, 255] = float("-inf")
    x[:, 64] += 1e-3
    want_q, want_s = quantize_rows(x)
    q, s = mxq.fp8_quantize_rows(x)
    same_codes(q, want_q)
    assert torch.equal(s.isnan(), want_s.isnan()) and torch.equal(s.nan_to_num(), want_s.nan_to_num())
    assert s.isnan().nonzero().tolist() == [[0, 4], [1, 3], [1, 6]]
    w = x.view(1, 8, 256)
    want_q, want_s = quantize_weight(w)
    q, s = mxq.fp8_quantize_weight(w)
    same_codes(q, want_q)
    assert s.isnan().all() and want_s.isnan().all()


def make(seed, counts, N, K, dgrad):
    """Codes and scales of both operands, with scales of their own: not powers of two, far apart."""
    M, red = sum(counts), N if dgrad else K
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(M, red, device="cuda").normal_(generator=g).mul_(100).clamp_(-448, 448).to(E4M3)
    w = torch.empty(len(counts), N, K, device="cuda").normal_(generator=g).mul_(100).clamp_(-448, 448).to(E4M3)
    xs = torch.empty(-(-red // 128), M, device="cuda").uniform_(-8, 8, generator=g).exp2()
    ws = torch.empty(len(counts), -(-N // 128), -(-K // 128), device="cuda").uniform_(-8, 8, generator=g).exp2()
    return x, xs, w, ws


SHAPES = [
    # counts, N, K: one token, few rows (split sums, one or several waves), pairs, ragged ends, experts without rows
    ([1], 8, 16),
    ([1], 2048, 4096),
    ([0, 5, 0, 32, 1], 272, 400),
    ([16], 4096, 2048),
    ([2] * 8, 528, 1040),
    ([33, 0, 31], 144, 144),
    ([300], 256, 128),
    ([129, 0, 257, 64, 1], 400, 528),
    ([511, 130], 1040, 656),
    ([255, 256, 1000], 2064, 1424),
    # tiles of one SM: whole and ragged ones, several of an expert, experts without rows, last blocks of both kinds of width
    ([128], 256, 128),
    ([33], 24, 16),
    ([100, 0, 60], 144, 144),
    ([17] * 8, 272, 1040),
    ([127, 128, 129], 656, 272),
    ([1, 300, 0, 40], 2064, 1424),
    ([129], 144, 272),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_fprop(mxq, counts, N, K, dtype):
    x, xs, w, ws = make(N + K, counts, N, K, False)
    bias = normal(3, len(counts), N, std=100.0)
    y = mxq.fp8_gemm_fprop(x.view(torch.uint8), xs, w.view(torch.uint8), ws, splits(counts), bias=bias, out_dtype=dtype)
    ref, mag = fprop64(row_values(x, xs), weight_values(w, ws), counts, bias)
    assert ((y.double() - ref).abs() <= fp8_tolerance(K, dtype) * mag).all(), ((y.double() - ref).abs() / mag).max()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,N,K", [(c, -(-n // 16) * 16, k) for c, n, k in SHAPES])
def test_dgrad(mxq, counts, N, K, dtype):
    d, ds, w, ws = make(N + K, counts, N, K, True)
    dx = mxq.fp8_gemm_dgrad(d, ds, w, ws, splits(counts), out_dtype=dtype)
    ref, mag = dgrad64(row_values(d, ds), weight_values(w, ws), counts)
    assert ((dx.double() - ref).abs() <= fp8_tolerance(N, dtype) * mag).all(), ((dx.double() - ref).abs() / mag).max()


@pytest.mark.parametrize("counts", [[7, 0, 9], [200, 0, 300]])
def test_non_finite_rows(mxq, counts):
    """A row that holds NaN or infinities gives NaN in its own results and nowhere else; likewise a weight's channels."""
    M, N, K = sum(counts), 272, 400
    x, w = normal(1, M, K), normal(2, len(counts), N, K, std=0.02)
    x[2, 399], x[5, 0] = float("nan"), float("inf")
    w[2, 130, 17] = float("-inf")
    q, xs = mxq.fp8_quantize_rows(x)
    wq, ws = mxq.fp8_quantize_weight(w)
    y = mxq.fp8_gemm_fprop(q, xs, wq, ws, splits(counts))
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[2], bad[5] = True, True
    bad[counts[0]:, 128:256] = True
    assert torch.equal(y.isnan(), bad) and y[~bad].isfinite().all()


@pytest.mark.parametrize("counts", [[7, 0, 9], [200, 0, 300]])
def test_wrong_counts_write_nothing(mxq, counts):
    x, xs, w, ws = make(1, counts, 272, 400, False)
    for wrong, bit in (([counts[0] + 1, 0, counts[2]], 4), ([counts[0], -1, counts[2] + 1], 2)):
        status = mxq.new_status()
        out = torch.full((sum(counts), 272), 7.0, dtype=BF16, device="cuda")
        mxq.fp8_gemm_fprop(x, xs, w, ws, splits(wrong), status=status, out=out)
        assert mxq.status_read(status) & bit and (out == 7.0).all()


def test_many_experts(mxq):
    """As many experts as a call takes, most without rows: few rows on average, and tiles of one SM and of a pair."""
    E, N, K = 1024, 24, 144
    for per, some in ((1, 7), (40, 331), (140, 331)):
        counts = [0] * E
        for e in range(0, E, some):
            counts[e] = E * per // len(range(0, E, some))
        x, xs, w, ws = make(E, counts, N, K, False)
        y = mxq.fp8_gemm_fprop(x, xs, w, ws, splits(counts))
        ref, mag = fprop64(row_values(x, xs), weight_values(w, ws), counts)
        assert ((y.double() - ref).abs() <= fp8_tolerance(K, BF16) * mag).all()
    with pytest.raises(mxq.MXQError):
        mxq.fp8_gemm_fprop(x[:0], xs[:, :0].contiguous(), w.repeat(2, 1, 1), ws.repeat(2, 1, 1), splits(counts + counts))


def test_offsets_beyond_32_bits(mxq):
    """Rows, results and weights of more than 2^31 elements: the last ones."""
    M = (1 << 18) + 3
    ms = splits([M - 5, 5])
    x = normal(1, 16, 8208).repeat(-(-M // 16), 1)[:M]
    w = normal(2, 2, 16, 8208, std=0.02)
    q, s = mxq.fp8_quantize_rows(x)
    tail_q, tail_s = quantize_rows(x[-16:])
    same_codes(q[-16:], tail_q)
    same_scales(s[:, -16:].contiguous(), tail_s)
    wq, ws = mxq.fp8_quantize_weight(w)
    y = mxq.fp8_gemm_fprop(q, s, wq, ws, ms)
    ref, mag = fprop64(row_values(tail_q, tail_s), weight_values(wq.view(E4M3), ws), [11, 5])
    assert ((y[-16:].double() - ref).abs() <= fp8_tolerance(8208, BF16) * mag).all()
    del x, q, s, y
    d = normal(3, 16, 16).repeat(-(-M // 16), 1)[:M].contiguous()  # dX (M, 8208)
    q, s = mxq.fp8_quantize_rows(d)
    for dtype in (BF16, F32):
        dx = mxq.fp8_gemm_dgrad(q, s, wq, ws, ms, out_dtype=dtype)
        ref, mag = dgrad64(row_values(q[-16:].view(E4M3), s[:, -16:]), weight_values(wq.view(E4M3), ws), [11, 5])
        assert ((dx[-16:].double() - ref).abs() <= fp8_tolerance(16, dtype) * mag).all()
        del dx
    w = normal(4, 3, 1, 1, std=0.02).expand(3, 32768, 32768).contiguous()
    w[2, -128:, -128:] = normal(5, 128, 128)
    wq, ws = mxq.fp8_quantize_weight(w)
    tail_q, tail_s = quantize_weight(w[2:, -128:, -128:])
    same_codes(wq[2:, -128:, -128:].contiguous(), tail_q)
    same_scales(ws[2:, -1:, -1:].contiguous(), tail_s)
    xq, xs = mxq.fp8_quantize_rows(normal(6, 3, 32768))
    y = mxq.fp8_gemm_fprop(xq, xs, wq, ws, splits([1, 1, 1]))
    v = row_values(xq.view(E4M3), xs)[2]
    values = weight_values(wq[2:, -128:].view(E4M3), ws[2:, -1:])[0]
    assert ((y[2, -128:].double() - values @ v).abs() <= fp8_tolerance(32768, BF16) * (values.abs() @ v.abs())).all()


def test_no_rows(mxq):
    ms = splits([0, 0])
    w, ws = mxq.fp8_quantize_weight(normal(1, 2, 32, 48))
    q, xs = mxq.fp8_quantize_rows(torch.empty(0, 48, dtype=BF16, device="cuda"))
    assert q.shape == (0, 48) and xs.shape == (1, 0)
    assert mxq.fp8_gemm_fprop(q, xs, w, ws, ms).shape == (0, 32)


def test_refusals(mxq):
    counts, N, K = [3, 4], 32, 272  # three blocks: a dimension of one would not count in a shape
    x, xs, w, ws = make(1, counts, N, K, False)
    ms = splits(counts)
    for args in ((x, xs.t().contiguous(), w, ws, ms), (x, xs, w, ws[:1], ms), (x, xs, w.transpose(1, 2), ws, ms),
                 (x, xs, w, ws, splits([7])), (x, xs.double(), w, ws, ms), (x.float(), xs, w, ws, ms),
                 (x, xs, w, ws, ms.cpu())):
        with pytest.raises(mxq.MXQError):
            mxq.fp8_gemm_fprop(*args)
    with pytest.raises(mxq.MXQError):
        mxq.fp8_gemm_fprop(x, xs, w, ws, ms, out_dtype=torch.float16)
    with pytest.raises(mxq.MXQError):  # dgrad's rows need widths of whole 16 bytes
        mxq.fp8_gemm_dgrad(torch.zeros(7, 24, dtype=torch.uint8, device="cuda"), torch.ones(1, 7, device="cuda"),
                           torch.zeros(2, 24, 48, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, 1, device="cuda"), ms)
    for bad in (normal(1, 4, 24), normal(1, 4, 32).t(), normal(1, 4, 32).float()):
        with pytest.raises(mxq.MXQError):
            mxq.fp8_quantize_rows(bad)
    for bad in (normal(1, 4, 32), normal(1, 2, 4, 32), normal(1, 2, 32, 8)):
        with pytest.raises(mxq.MXQError):
            mxq.fp8_quantize_weight(bad)

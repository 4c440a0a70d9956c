"""Gated products on bf16 with any expert counts: FC1 with its activation, FC2's dgrad through it."""
import pytest
import torch

from ._ragged import dgrad64, fprop64, sum_tolerance

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HALF = 2.0 ** -8  # half a bf16 step, relative to the value
APPROX = 2.0 ** -19  # the sigmoid's hardware approximations (near 2^-22 each) and the fp32 steps behind them


@pytest.fixture(scope="module")
def mxq():
    import moe_expert_grouped_group_gb300 as m

    return m


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0, std, generator=g).to(BF16)


def splits(counts):
    return torch.tensor(counts, dtype=torch.int64, device="cuda")


def check(got, ref, err, what):
    assert got.shape == ref.shape
    off, bound = (got.double() - ref).abs(), err + HALF * (ref.abs() + err)
    assert (off <= bound).all(), (what, (off / bound.clamp(min=1e-300)).max().item())


# counts, F, K (or N): one token, few rows (sums split over clusters, one and several waves), pairs, experts without rows,
# widths that end inside a chunk of eight lanes, a tile and a stage
SHAPES = [
    ([1], 8, 8),
    ([1], 2048, 4096),
    ([0, 5, 0, 32, 1], 264, 392),
    ([16], 2048, 2048),
    ([2] * 8, 520, 1032),
    ([1] * 16, 136, 72),
    ([33, 0, 31], 72, 136),
    ([300], 128, 64),
    ([129, 0, 257, 64, 1], 392, 520),
    ([511, 130], 1032, 648),
    ([255, 256, 1000], 1416, 2056),
]


def fprop_reference(x, w, counts, bias):
    """h and [g | u] in 64 bits with the errors that the fp32 sums allow them."""
    F = w.shape[1] // 2
    y, mag = fprop64(x, w, counts, bias)
    ey = sum_tolerance(x.shape[1], False) * mag
    (g, u), (eg, eu) = y.split(F, dim=1), ey.split(F, dim=1)
    silu = g * torch.sigmoid(g)
    h = silu * u  # |silu'| < 1.1
    return h, 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + APPROX * h.abs(), y, ey


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("counts,F,K", SHAPES)
def test_fprop(mxq, counts, F, K, bias):
    M, E = sum(counts), len(counts)
    x, w = normal(M + K, M, K + 24)[:, :K], normal(F, E, 2 * F, K, std=1.5 * K ** -0.5)
    b = normal(3, E, 2 * F) if bias else None
    h, eh, y, ey = fprop_reference(x, w, counts, b)
    got = mxq.ragged_gemm_fprop_swiglu(x, w, splits(counts), bias=b)
    check(got, h, eh, "h")
    got2, got_y = mxq.ragged_gemm_fprop_swiglu(x, w, splits(counts), bias=b, y_out=True)
    assert torch.equal(got, got2)
    check(got_y, y, ey, "y")


def dgrad_reference(dy, w, y, counts):
    """[dg | du] and h in 64 bits with the errors that the fp32 sums allow them."""
    dh, mag = dgrad64(dy, w, counts)
    e = sum_tolerance(dy.shape[1], False) * mag
    g, u = y.double().chunk(2, dim=1)
    s = torch.sigmoid(g)
    d = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=1)
    size = torch.cat([(u * s).abs() * (1 + g.abs()), (g * s).abs()], dim=1)
    return d, (torch.cat([e, e], dim=1) + APPROX * torch.cat([dh, dh], dim=1).abs()) * size, g * s * u


@pytest.mark.parametrize("counts,F,N", SHAPES)
def test_dgrad(mxq, counts, F, N):
    M, E = sum(counts), len(counts)
    dy, w, y = normal(M + N, M, N + 24)[:, :N], normal(F, E, N, F, std=N ** -0.5), normal(5, M, 2 * F, std=2.0)
    d, ed, h = dgrad_reference(dy, w, y, counts)
    got = mxq.ragged_gemm_dgrad_swiglu(dy, w, y, splits(counts))
    check(got, d, ed, "dy1")
    got2, got_h = mxq.ragged_gemm_dgrad_swiglu(dy, w, y, splits(counts), h_out=True)
    assert torch.equal(got, got2)
    check(got_h, h, APPROX * h.abs(), "h")


@pytest.mark.parametrize("counts", [[40, 3]])
def test_long_sums(mxq, counts):
    """Sums of more than 2^15 terms of one sign, which one accumulator would truncate."""
    F, K = 72, (1 << 15) + 264
    x, w = normal(1, sum(counts), K).abs(), normal(2, 2, 2 * F, K, std=2.0 ** -15).abs()
    h, _, y, _ = fprop_reference(x, w, counts, None)
    got, got_y = mxq.ragged_gemm_fprop_swiglu(x, w, splits(counts), y_out=True)
    # pieces of 8192 terms (2^-23 of the sum per 16 at most, twice), then bf16
    rel = (8192 / 16 + 8) * 2.0 ** -22
    assert ((got_y.double() - y).abs() <= (HALF + rel) * y).all()
    check(got, h, 2.2 * rel * h.abs() * (1 + y[:, :F]), "h")
    w2 = normal(4, 2, K, F, std=2.0 ** -15).abs()
    y1 = normal(5, sum(counts), 2 * F)
    d, ed, _ = dgrad_reference(x, w2, y1, counts)
    check(mxq.ragged_gemm_dgrad_swiglu(x, w2, y1, splits(counts)), d, ed, "dy1")


@pytest.mark.parametrize("counts", [[7, 0, 9], [200, 0, 300]])
def test_non_finite_rows(mxq, counts):
    """NaN and infinities stay in their rows; sums that overflow give what the formulas give."""
    M, F, K = sum(counts), 136, 200
    x, w = normal(1, M, K), normal(2, 3, 2 * F, K, std=0.02)
    clean, clean_y = mxq.ragged_gemm_fprop_swiglu(x, w, splits(counts), y_out=True)
    x[2, 199], x[5, 0] = float("nan"), float("inf")
    h, y = mxq.ragged_gemm_fprop_swiglu(x, w, splits(counts), y_out=True)
    keep = [m for m in range(M) if m not in (2, 5)]
    assert torch.equal(h[keep], clean[keep]) and torch.equal(y[keep], clean_y[keep])
    assert h[2].isnan().all() and not y[5].isfinite().any()
    w2, dy = normal(3, 3, K, F, std=0.02), normal(4, M, K)
    clean = mxq.ragged_gemm_dgrad_swiglu(dy, w2, clean_y, splits(counts))
    dy[counts[0], 3] = float("nan")
    d = mxq.ragged_gemm_dgrad_swiglu(dy, w2, clean_y, splits(counts))
    keep = [m for m in range(M) if m != counts[0]]
    assert torch.equal(d[keep], clean[keep]) and d[counts[0]].isnan().all()


@pytest.mark.parametrize("counts", [[7, 0, 9], [200, 0, 300]])
def test_wrong_counts_write_nothing(mxq, counts):
    M, F, K = sum(counts), 136, 200
    x, w, w2, y = normal(1, M, K), normal(2, 3, 2 * F, K), normal(3, 3, K, F), normal(4, M, 2 * F)
    for wrong, bit in (([counts[0] + 1, 0, counts[2]], 4), ([counts[0], -1, counts[2] + 1], 2)):
        status = mxq.new_status()
        h, d = torch.full((M, F), 7.0, dtype=BF16, device="cuda"), torch.full((M, 2 * F), 7.0, dtype=BF16, device="cuda")
        mxq.ragged_gemm_fprop_swiglu(x, w, splits(wrong), status=status, out=h)
        mxq.ragged_gemm_dgrad_swiglu(x, w2, y, splits(wrong), status=status, out=d)
        assert mxq.status_read(status) & bit and (h == 7.0).all() and (d == 7.0).all()


def test_many_experts(mxq):
    E, F, K = 1024, 24, 72
    w, w2 = normal(1, E, 2 * F, K, std=0.1), normal(2, E, K, F, std=0.1)
    for per, some in ((1, 7), (40, 331)):
        counts = [0] * E
        for e in range(0, E, some):
            counts[e] = E * per // len(range(0, E, some))
        M = sum(counts)
        x, y = normal(3, M, K), normal(4, M, 2 * F)
        h, eh, _, _ = fprop_reference(x, w, counts, None)
        check(mxq.ragged_gemm_fprop_swiglu(x, w, splits(counts)), h, eh, "h")
        d, ed, _ = dgrad_reference(x, w2, y, counts)
        check(mxq.ragged_gemm_dgrad_swiglu(x, w2, y, splits(counts)), d, ed, "dy1")


def test_offsets_beyond_32_bits(mxq):
    """[g | u] and its gradient of more than 2^31 elements: the last rows."""
    M, F, K = (1 << 18) + 3, 4104, 16
    x = normal(1, 16, K).repeat(-(-M // 16), 1)[:M].contiguous()
    w = normal(2, 2, 2 * F, K, std=0.3)
    h, y = mxq.ragged_gemm_fprop_swiglu(x, w, splits([M - 5, 5]), y_out=True)
    ref, eh, ry, ey = fprop_reference(x[-16:], w, [11, 5], None)
    check(h[-16:], ref, eh, "h")
    check(y[-16:], ry, ey, "y")
    w2 = normal(3, 2, K, F, std=0.3)
    d, h2 = mxq.ragged_gemm_dgrad_swiglu(x, w2, y, splits([M - 5, 5]), h_out=True)
    ref, ed, rh = dgrad_reference(x[-16:], w2, y[-16:], [11, 5])
    check(d[-16:], ref, ed, "dy1")
    check(h2[-16:], rh, APPROX * rh.abs(), "h")


def test_no_rows(mxq):
    ms = splits([0, 0])
    x, y = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, 48, dtype=BF16, device="cuda")
    assert mxq.ragged_gemm_fprop_swiglu(x, normal(1, 2, 48, 64), ms).shape == (0, 24)
    assert mxq.ragged_gemm_dgrad_swiglu(x, normal(1, 2, 64, 24), y, ms).shape == (0, 48)


def test_mlp_gradients(mxq):
    """A gated MLP's gradients against those of its 64-bit definition: the error of each is within what the bf16
    roundings of h, [g | u] and [dg | du] on the way allow, 2^-8 each of the terms' magnitudes."""
    counts, K, F = [70, 0, 33, 1], 200, 136
    M, E = sum(counts), len(counts)
    x, w1, w2 = normal(1, M, K), normal(2, E, 2 * F, K, std=K ** -0.5), normal(3, E, K, F, std=F ** -0.5)
    dy, ms = normal(4, M, K), splits(counts)
    h, y1 = mxq.ragged_gemm_fprop_swiglu(x, w1, ms, y_out=True)
    d1, h2 = mxq.ragged_gemm_dgrad_swiglu(dy, w2, y1, ms, h_out=True)
    got = {"x": mxq.ragged_gemm_dgrad(d1, w1, ms, out_dtype=torch.float32), "w1": mxq.ragged_gemm_wgrad(d1, x, ms),
           "w2": mxq.ragged_gemm_wgrad(dy, h2, ms)}
    leaves = [t.double().requires_grad_() for t in (x, w1, w2)]
    off, loss = 0, 0.0
    for e, m in enumerate(counts):
        r = slice(off, off + m)
        g, u = (leaves[0][r] @ leaves[1][e].t()).chunk(2, dim=1)
        loss = loss + ((g * torch.sigmoid(g) * u) @ leaves[2][e].t() * dy[r].double()).sum()
        off += m
    loss.backward()
    # terms' magnitudes: products of |d1| with |w1| or |x|, of |dy| with |h|; g and u enter d1 twice each, with slopes of
    # |g| + 2 at most
    d_mag = (d1.double().abs() + (dgrad64(dy, w2, counts)[0].repeat(1, 2)).abs() * (y1.double().abs() + 2)) * 8
    mags = {"x": dgrad64(d_mag, w1, counts)[1],
            "w1": torch.stack([d_mag[a:a + m].t() @ x[a:a + m].double().abs() for a, m in zip((0, 70, 70, 103), counts)]),
            "w2": torch.stack([dy[a:a + m].double().abs().t() @ (h.double().abs() + y1.double()[:, :F].abs() + y1.double()[:, F:].abs())[a:a + m]
                               for a, m in zip((0, 70, 70, 103), counts)])}
    for k, leaf in zip(("x", "w1", "w2"), leaves):
        assert ((got[k].double() - leaf.grad).abs() <= 2.0 ** -8 * mags[k] + 1e-12).all(), k


def test_graph(mxq):
    """Captured and replayed on new values and counts: the bits of the calls themselves."""
    F, K = 264, 392
    w, w2 = normal(1, 4, 2 * F, K, std=0.05), normal(2, 4, K, F, std=0.05)
    x, dy, ms = normal(3, 300, K), normal(4, 300, K), splits([100, 50, 0, 150])

    def step():
        h, y = mxq.ragged_gemm_fprop_swiglu(x, w, ms, y_out=True)
        return (h, y) + mxq.ragged_gemm_dgrad_swiglu(dy, w2, y, ms, h_out=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed, counts in ((11, [0, 299, 1, 0]), (12, [75, 75, 75, 75])):
        x.copy_(normal(seed, 300, K))
        dy.copy_(normal(seed + 9, 300, K))
        ms.copy_(splits(counts))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_refusals(mxq):
    x, w, ms = normal(1, 5, 64), normal(2, 2, 48, 64), splits([2, 3])
    w2, y = normal(3, 2, 64, 24), normal(4, 5, 48)
    for args, kw in (((x, w[:, :47], ms), {}), ((x[:, :56], w, ms), {}), ((x.t(), w, ms), {}), ((x.float(), w, ms), {}),
                     ((x, w, splits([5])), {}), ((x, w, ms.cpu()), {}), ((x, w, ms), dict(bias=normal(1, 2, 24))),
                     ((x, w, ms), dict(out=torch.empty(5, 48, dtype=BF16, device="cuda"))),
                     ((normal(1, 5, 60), normal(2, 2, 48, 60), ms), {}), ((x, normal(2, 2, 24, 64), ms), {})):
        with pytest.raises(mxq.MXQError):
            mxq.ragged_gemm_fprop_swiglu(*args, **kw)
    for args in ((x, w2, y[:, :24].contiguous(), ms), (x, w2.transpose(1, 2), y, ms), (x, w2, y.float(), ms),
                 (x, w2, None, ms), (x, w2, y[:4], ms)):
        with pytest.raises(mxq.MXQError):
            mxq.ragged_gemm_dgrad_swiglu(*args)

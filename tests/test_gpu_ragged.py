"""Ragged bf16 grouped products (fprop, dgrad, wgrad) against fp64."""
import pytest
import torch

from tests._gpu import dev_i64, lib, require_gpu
from tests._ragged import assert_products, dgrad64, fprop64, wgrad64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


def rand(seed, *shape, pad=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(*shape[:-1], shape[-1] + pad, generator=g, device="cuda").mul_(std).to(BF16)
    return t[..., :shape[-1]]


# counts around the 16-row step, the 64-row box and the 256-row slice; empty and lone experts
GROUPS = {
    "one_token": [1],
    "one_of_many": [0, 0, 1, 0],
    "steps": [15, 16, 17, 0, 31, 33],
    "boxes": [63, 64, 65, 1, 127, 129],
    "slices": [255, 256, 257, 0, 513, 3],
    "long": [1, 2049, 0, 700],
    "first_and_last_empty": [0, 40, 0],
    "single_expert": [700],
}
# (N, K): one box; odd widths; edges past 128 and 256; deeper than the ring
WIDTHS = [(8, 8), (136, 72), (256, 512), (264, 1000), (520, 264), (1024, 136)]


@pytest.mark.parametrize("widths", WIDTHS, ids=str)
@pytest.mark.parametrize("group", GROUPS)
def test_products(mxq, group, widths):
    counts, (N, K) = GROUPS[group], widths
    M, E = sum(counts), len(counts)
    pad = 8 if N % 16 else 0
    x, dy, w = rand(1, M, K, pad=pad), rand(2, M, N, pad=pad), rand(3, E, N, K)
    bias, ms = rand(4, E, N), dev_i64(counts)
    for dt, tag in ((BF16, "bf16"), (F32, "f32")):
        assert_products(mxq.ragged_gemm_fprop(x, w, ms, out_dtype=dt), *fprop64(x, w, counts), K, tag)
        assert_products(mxq.ragged_gemm_fprop(x, w, ms, bias=bias, out_dtype=dt), *fprop64(x, w, counts, bias), K, tag)
        assert_products(mxq.ragged_gemm_dgrad(dy, w, ms, out_dtype=dt), *dgrad64(dy, w, counts), N, tag)
        ref, mag = wgrad64(dy, x, counts)
        assert_products(mxq.ragged_gemm_wgrad(dy, x, ms, out_dtype=dt), ref, mag, max(counts), tag)
        prior = rand(5, E, N, K).to(dt)
        got = mxq.ragged_gemm_wgrad(dy, x, ms, accumulate=True, out=prior.clone())
        assert_products(got, ref + prior.double(), mag + prior.double().abs(), max(counts), tag)
        empty = torch.tensor([m == 0 for m in counts], device="cuda")
        assert torch.equal(got[empty], prior[empty])  # an empty expert's dW is not touched


@pytest.mark.parametrize("E", [512, 1024])
def test_many_experts(mxq, E):
    counts = [(7 * e + 3) % 5 if e % 3 else 0 for e in range(E)]
    M, N, K = sum(counts), 136, 64
    x, dy, w, ms = rand(1, M, K), rand(2, M, N), rand(3, E, N, K), dev_i64(counts)
    assert_products(mxq.ragged_gemm_fprop(x, w, ms), *fprop64(x, w, counts), K, "bf16")
    assert_products(mxq.ragged_gemm_dgrad(dy, w, ms), *dgrad64(dy, w, counts), N, "bf16")
    assert_products(mxq.ragged_gemm_wgrad(dy, x, ms), *wgrad64(dy, x, counts), 5, "f32")


def test_no_rows_at_all(mxq):
    ms, w = dev_i64([0, 0]), rand(3, 2, 64, 72)
    x, dy = rand(1, 0, 72), rand(2, 0, 64)
    assert mxq.ragged_gemm_fprop(x, w, ms).shape == (0, 64)
    assert mxq.ragged_gemm_dgrad(dy, w, ms).shape == (0, 72)
    dw = mxq.ragged_gemm_wgrad(dy, x, ms, out=torch.full((2, 64, 72), 7.0, device="cuda"))
    assert torch.all(dw == 0)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3.0e38])
def test_values_stay_in_their_expert(mxq, value):
    """Rows of a neighbour share tiles, boxes and blocks with an expert, and never its results."""
    counts, N, K = [37, 5, 300, 1, 90], 136, 72
    M, ms = sum(counts), dev_i64([37, 5, 300, 1, 90])
    x, dy, w = rand(1, M, K), rand(2, M, N), rand(3, 5, N, K)
    bad = slice(42, 342)  # expert 2
    xb, dyb, wb = x.clone(), dy.clone(), w.clone()
    xb[bad], dyb[bad], wb[2] = value, value, value
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[bad] = False
    experts = torch.tensor([0, 1, 3, 4], device="cuda")
    assert torch.equal(mxq.ragged_gemm_fprop(xb, wb, ms)[keep], mxq.ragged_gemm_fprop(x, w, ms)[keep])
    assert torch.equal(mxq.ragged_gemm_dgrad(dyb, wb, ms)[keep], mxq.ragged_gemm_dgrad(dy, w, ms)[keep])
    assert torch.equal(mxq.ragged_gemm_wgrad(dyb, xb, ms)[experts], mxq.ragged_gemm_wgrad(dy, x, ms)[experts])
    if value != value:
        assert torch.isnan(mxq.ragged_gemm_fprop(xb, wb, ms)[bad]).all()


def test_same_bits_every_time(mxq):
    counts, N, K = [1000, 3, 0, 517], 520, 1000
    M, ms = sum(counts), dev_i64(counts)
    x, dy, w = rand(1, M, K), rand(2, M, N), rand(3, 4, N, K)
    calls = (lambda: mxq.ragged_gemm_fprop(x, w, ms), lambda: mxq.ragged_gemm_dgrad(dy, w, ms),
             lambda: mxq.ragged_gemm_wgrad(dy, x, ms))
    for call in calls:
        first = call()
        for _ in range(3):
            assert torch.equal(call(), first)


@pytest.mark.parametrize("counts,bits", [([10, 20], 4), ([-1, 33], 6), ([40, -8], 6), ([1 << 62, 1 << 62], 4),
                                         ([0, 0], 4)])
def test_wrong_counts_write_nothing_and_set_the_status(mxq, counts, bits):
    x, dy, w, ms = rand(1, 32, 64), rand(2, 32, 72), rand(3, 2, 72, 64), dev_i64(counts)
    outs = (torch.full((32, 72), 7.0, dtype=BF16, device="cuda"), torch.full((32, 64), 7.0, dtype=BF16, device="cuda"),
            torch.full((2, 72, 64), 7.0, device="cuda"))
    for call in (lambda s: mxq.ragged_gemm_fprop(x, w, ms, status=s, out=outs[0]),
                 lambda s: mxq.ragged_gemm_dgrad(dy, w, ms, status=s, out=outs[1]),
                 lambda s: mxq.ragged_gemm_wgrad(dy, x, ms, status=s, out=outs[2])):
        s = mxq.new_status()
        call(s)
        assert mxq.status_read(s) == bits
    assert all(torch.all(o == 7) for o in outs)


def test_another_stream_and_graph_replay_with_new_counts(mxq):
    M, N, K = 300, 136, 200
    x, dy, w = rand(1, M, K), rand(2, M, N), rand(3, 3, N, K)
    ms = dev_i64([100, 100, 100])
    y, dx = torch.empty((M, N), dtype=BF16, device="cuda"), torch.empty((M, K), dtype=BF16, device="cuda")
    dw = torch.empty((3, N, K), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.ragged_gemm_fprop(x, w, ms, out=y)
        mxq.ragged_gemm_dgrad(dy, w, ms, out=dx)
        mxq.ragged_gemm_wgrad(dy, x, ms, out=dw)
    side = torch.cuda.Stream()
    for counts in ([100, 100, 100], [0, 299, 1], [300, 0, 0]):
        with torch.cuda.stream(side):
            ms.copy_(torch.tensor(counts))
            graph.replay()
        side.synchronize()
        assert_products(y, *fprop64(x, w, counts), K, "bf16")
        assert_products(dx, *dgrad64(dy, w, counts), N, "bf16")
        assert_products(dw, *wgrad64(dy, x, counts), max(counts), "f32")


def test_gradients_by_differences(mxq):
    """<dY, Y(X + h V) - Y(X - h V)> / 2h = <dX, V>, and the same for W: fprop is linear in each."""
    counts, N, K = [70, 1, 0, 33], 72, 136
    M, ms, h = sum(counts), dev_i64(counts), 0.5
    x, dy, w = rand(1, M, K), rand(2, M, N), rand(3, 4, N, K)
    f = lambda x, w: (dy.double() * mxq.ragged_gemm_fprop(x, w, ms, out_dtype=F32).double()).sum().item()  # noqa: E731
    for grad, at, shape in ((mxq.ragged_gemm_dgrad(dy, w, ms, out_dtype=F32), lambda v: (x + v, w), x),
                            (mxq.ragged_gemm_wgrad(dy, x, ms), lambda v: (x, w + v), w)):
        v = rand(9, *shape.shape)
        (x1, w1), (x0, w0) = at(h * v), at(-h * v)
        num = (f(x1, w1) - f(x0, w0)) / (2 * h)
        # bf16 sums x + h v are rounded: use the steps that were taken
        step = ((x1.double() - x0.double()) if grad.shape == x.shape else (w1.double() - w0.double())) / (2 * h)
        ana = (grad.double() * step).sum().item()
        size = (grad.double() * step).abs().sum().item()
        assert abs(num - ana) <= 1e-5 * size


def test_refusals(mxq):
    x, w, dy, ms = rand(1, 32, 64), rand(3, 2, 72, 64), rand(2, 32, 72), dev_i64([16, 16])
    E = mxq.MXQError
    for call in (
        lambda: mxq.ragged_gemm_fprop(x.float(), w, ms),                       # types
        lambda: mxq.ragged_gemm_fprop(x, w.half(), ms),
        lambda: mxq.ragged_gemm_fprop(x, w, ms.int()),
        lambda: mxq.ragged_gemm_fprop(x, w, torch.tensor([16, 16])),           # host counts
        lambda: mxq.ragged_gemm_fprop(x, w, None),
        lambda: mxq.ragged_gemm_fprop(x, w, dev_i64([32])),                    # counts for another E
        lambda: mxq.ragged_gemm_fprop(x, w[:, :, :56], ms),                    # widths that do not match
        lambda: mxq.ragged_gemm_fprop(x, w.transpose(1, 2), ms),
        lambda: mxq.ragged_gemm_fprop(x.t(), w, ms),                           # rows not contiguous
        lambda: mxq.ragged_gemm_fprop(rand(1, 32, 60), rand(3, 2, 72, 60), ms),  # K % 8
        lambda: mxq.ragged_gemm_fprop(x, rand(3, 2, 68, 64), ms),              # N % 8
        lambda: mxq.ragged_gemm_fprop(rand(1, 32, 64, pad=4), w, ms),          # stride % 8
        lambda: mxq.ragged_gemm_fprop(rand(1, 32, 72)[:, 4:68], w, ms),        # address % 16
        lambda: mxq.ragged_gemm_fprop(x, w, ms, out=torch.empty((32, 64), dtype=BF16, device="cuda")),
        lambda: mxq.ragged_gemm_fprop(x, w, ms, out_dtype=torch.float16),
        lambda: mxq.ragged_gemm_fprop(x, w, ms, bias=rand(4, 2, 64)),
        lambda: mxq.ragged_gemm_dgrad(dy, w[:, :64], ms),
        lambda: mxq.ragged_gemm_wgrad(dy, x[:16], ms),
        lambda: mxq.ragged_gemm_wgrad(dy, x, ms, accumulate=True),
        lambda: mxq.ragged_gemm_wgrad(dy, x, ms, status=torch.zeros(1, device="cuda")),
    ):
        with pytest.raises(E):
            call()

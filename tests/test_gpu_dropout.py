"""Counter-based dropout, alone and inside SwiGLU, against its definition."""
import numpy as np
import pytest
import torch

from tests._gpu import assert_swiglu_close, host, lib, require_gpu, swiglu_bwd_slack, swiglu_fwd_slack
from tests._ragged import keep_mask, keep_scale, swiglu64, swiglu_grad64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


def rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def rand(seed, *shape, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def drop64(v, seed, offset, p):
    v = v.double().cpu()
    return torch.where(keep_mask(seed & (2**64 - 1), offset & (2**64 - 1), p, tuple(v.shape)), v * keep_scale(p),
                       torch.zeros((), dtype=torch.float64))


# fp32: the scale's rounding, the product's and the sum's; bf16: its unit roundoff besides
def tolerance(dtype):
    return 3 * 2.0 ** -24 + (2.0 ** -8 if dtype == BF16 else 0.0)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 63, 1000, 4099, 1 << 20])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(mxq, n, p, dtype):
    seed, offset = 0x123456789ABCDEF, (5 << 40) + n
    x, r = rand(1, n, dtype=dtype), rand(2, n, dtype=dtype)
    keep = keep_mask(seed, offset, p, (n,)).cuda()
    d = drop64(x, seed, offset, p).cuda()
    got = mxq.dropout(x, rng(seed, offset), p)
    assert torch.all(got[~keep] == 0)
    assert torch.all((got.double() - d).abs() <= tolerance(dtype) * d.abs())
    got = mxq.dropout(x, rng(seed, offset), p, residual=r)
    assert torch.equal(got[~keep], r[~keep])
    assert torch.all((got.double() - (d + r.double())).abs() <= tolerance(dtype) * (d.abs() + r.double().abs()))
    if p == 0:
        assert torch.equal(mxq.dropout(x, rng(seed, offset), p), x)


# several vectors a thread (beyond one for each of the device's threads), ends inside a block's vectors
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("n", [1 << 22, (1 << 22) + 8 * 700 + 3])
def test_large_dropout(mxq, n, dtype):
    x, r, p = rand(1, n, dtype=dtype), rand(2, n, dtype=dtype), 0.3
    d = drop64(x, 11, 13, p).cuda()
    got = mxq.dropout(x, rng(11, 13), p)
    assert torch.equal(got != 0, d != 0)
    assert torch.all((got.double() - d).abs() <= tolerance(dtype) * d.abs())
    want = mxq.dropout(x, rng(11, 13), p, residual=r)
    assert torch.all((want.double() - (d + r.double())).abs() <= tolerance(dtype) * (d.abs() + r.double().abs()))
    mxq.dropout(x, rng(11, 13), p, residual=r, out=r)
    assert torch.equal(r, want)
    mxq.dropout(x, rng(11, 13), p, out=x)
    assert torch.equal(x, got)


def test_negative_seed_and_offset_are_their_64_bits(mxq):
    x = torch.ones(5000, device="cuda")
    got = mxq.dropout(x, rng(-3, -7), 0.5)
    assert torch.equal(got.cpu() != 0, keep_mask(2**64 - 3, 2**64 - 7, 0.5, (5000,)))


def test_out_may_be_an_input(mxq):
    x, r, g = rand(1, 4099), rand(2, 4099), rng(3, 4)
    want = mxq.dropout(x, g, 0.3, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(mxq.dropout(a, g, 0.3, residual=r, out=a), want)
    assert torch.equal(mxq.dropout(x, g, 0.3, residual=b, out=b), want)


def test_dropped_elements_hide_what_they_held(mxq):
    for v in (float("nan"), float("inf")):
        x = torch.full((4096,), v, device="cuda")
        keep = keep_mask(1, 2, 0.5, (4096,)).cuda()
        y = mxq.dropout(x, rng(1, 2), 0.5)
        assert torch.all(y[~keep] == 0) and not torch.isfinite(y[keep]).any()
        y1 = torch.full((64, 128), v, device="cuda").to(BF16)
        keep = keep_mask(1, 2, 0.5, (64, 64)).cuda()
        assert torch.all(mxq.swiglu_dropout_fwd(y1, rng(1, 2), 0.5)[~keep] == 0)
        dy = mxq.swiglu_dropout_bwd(rand(3, 64, 64), y1, rng(1, 2), 0.5)
        assert torch.all(dy[:, :64][~keep] == 0) and torch.all(dy[:, 64:][~keep] == 0)


@pytest.mark.parametrize("M,F", [(1, 8), (3, 24), (17, 136), (512, 512), (33, 1416), (5, 20000)])
@pytest.mark.parametrize("p", [0.0, 0.4, 1.0])
def test_swiglu_dropout(mxq, M, F, p):
    seed, offset = 99, 1 << 33
    y, dh, g = rand(1, M, 2 * F), rand(2, M, F), rng(99, 1 << 33)
    y[0, :4] = torch.tensor([-90.0, -86.5, 90.0, 0.0], device="cuda")
    keep = keep_mask(seed, offset, p, (M, F))
    keep2 = torch.cat([keep, keep], dim=1)
    h, dy = mxq.swiglu_dropout_fwd(y, g, p), mxq.swiglu_dropout_bwd(dh, y, g, p)
    assert torch.all(h[~keep.cuda()] == 0) and torch.all(dy[~keep2.cuda()] == 0)
    s = keep_scale(p)
    ref = torch.where(keep, swiglu64(y.cpu()) * s, torch.zeros(()).double()).to(BF16)
    refd = torch.where(keep2, swiglu_grad64(dh.cpu(), y.cpu()) * s, torch.zeros(()).double()).to(BF16)
    # the scale is one more fp32 rounding: the tolerance of the unscaled activation, times the scale
    assert_swiglu_close(host(h), host(ref), max(s, 1.0) * swiglu_fwd_slack(host(y)), "h")
    assert_swiglu_close(host(dy), host(refd), max(s, 1.0) * swiglu_bwd_slack(host(dh), host(y)), "dy")
    if p == 0:
        assert torch.equal(h, mxq.swiglu_fwd(y)) and torch.equal(dy, mxq.swiglu_bwd(dh, y))


def test_mask_does_not_depend_on_the_shape_of_the_launch(mxq):
    big = mxq.dropout(torch.ones(3_000_017, device="cuda"), rng(11, 12), 0.25)
    for n in (1, 1000, 999_999):
        assert torch.equal(mxq.dropout(torch.ones(n, device="cuda"), rng(11, 12), 0.25), big[:n])
    ones = torch.full((300, 2048), 1.0, dtype=BF16, device="cuda")
    assert torch.equal(mxq.swiglu_dropout_fwd(ones, rng(11, 12), 0.25).reshape(-1) != 0, big[:300 * 1024] != 0)


def test_graph_replay_with_a_new_offset(mxq):
    x, g, out = torch.ones(10000, device="cuda"), rng(5, 0), torch.empty(10000, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.dropout(x, g, 0.5, out=out)
    for offset in (0, 1, 2):
        g[1] = offset
        graph.replay()
        assert np.array_equal(out.cpu().numpy() != 0, keep_mask(5, offset, 0.5, (10000,)).numpy())


def test_empty_and_refusals(mxq):
    g, y, dh = rng(1, 2), rand(1, 4, 32), rand(2, 4, 16)
    assert mxq.dropout(rand(1, 0), g, 0.5).numel() == 0
    assert mxq.swiglu_dropout_fwd(rand(1, 0, 32), g, 0.5).shape == (0, 16)
    assert mxq.swiglu_dropout_bwd(rand(1, 0, 16), rand(1, 0, 32), g, 0.5).shape == (0, 32)
    for call in (
        lambda: mxq.dropout(y, g, -0.01),
        lambda: mxq.dropout(y, g, 1.01),
        lambda: mxq.dropout(y, g, float("nan")),
        lambda: mxq.dropout(y, g.cpu(), 0.5),
        lambda: mxq.dropout(y, g.int(), 0.5),
        lambda: mxq.dropout(y, g[:1], 0.5),
        lambda: mxq.dropout(y.half(), g, 0.5),
        lambda: mxq.dropout(y, g, 0.5, residual=y.float()),
        lambda: mxq.dropout(y, g, 0.5, residual=y[:3]),
        lambda: mxq.dropout(y, g, 0.5, out=torch.empty(127, dtype=BF16, device="cuda")),
        lambda: mxq.dropout(y[:, 1:], g, 0.5),
        lambda: mxq.swiglu_dropout_fwd(y, g, 2.0),
        lambda: mxq.swiglu_dropout_fwd(rand(1, 4, 24), g, 0.5),               # F % 8
        lambda: mxq.swiglu_dropout_fwd(y.float(), g, 0.5),
        lambda: mxq.swiglu_dropout_bwd(dh[:3], y, g, 0.5),
        lambda: mxq.swiglu_dropout_bwd(dh, y, g, 0.5, out=dh),
    ):
        with pytest.raises(mxq.MXQError):
            call()

"""Operands of another shape with as many or more bytes: the ragged, int8 and dropout calls say so."""
import pytest
import torch

from tests._gpu import dev_i64, lib, require_gpu
from tests.test_gpu_ragged import rand

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
E, M, N, K = 2, 32, 72, 64


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


def test_swiglu_dropout(mxq):
    g, y, dh = torch.tensor([1, 2], device="cuda"), rand(1, 4, 32), rand(2, 4, 16)
    for call in (
        lambda: mxq.swiglu_dropout_fwd(rand(1, 4, 33), g, 0.5),                    # no halves
        lambda: mxq.swiglu_dropout_fwd(rand(1, 2, 4, 32), g, 0.5),
        lambda: mxq.swiglu_dropout_fwd(y, g, 0.5, out=rand(3, 16, 4)),
        lambda: mxq.swiglu_dropout_fwd(y, g, 0.5, out=rand(3, 4, 32)),
        lambda: mxq.swiglu_dropout_bwd(dh, rand(1, 4, 33), g, 0.5),
        lambda: mxq.swiglu_dropout_bwd(rand(2, 4, 32), y, g, 0.5),
        lambda: mxq.swiglu_dropout_bwd(rand(2, 16, 4), y, g, 0.5),
        lambda: mxq.swiglu_dropout_bwd(dh, y, g, 0.5, out=rand(3, 8, 16)),
    ):
        with pytest.raises(mxq.MXQError):
            call()
    assert torch.equal(mxq.swiglu_dropout_bwd(dh.view(-1), y, g, 0.5), mxq.swiglu_dropout_bwd(dh, y, g, 0.5))


def test_dropout(mxq):
    g, x = torch.tensor([1, 2], device="cuda"), rand(1, 4, 32)
    for call in (
        lambda: mxq.dropout(x, g, 0.5, residual=rand(2, 32, 4)),
        lambda: mxq.dropout(x, g, 0.5, residual=rand(2, 8, 32)),
        lambda: mxq.dropout(x, g, 0.5, residual=rand(2, 1, 32)),
        lambda: mxq.dropout(x, g, 0.5, out=rand(2, 32, 4)),
        lambda: mxq.dropout(x, g, 0.5, out=rand(2, 8, 32)),
    ):
        with pytest.raises(mxq.MXQError):
            call()
    out = torch.empty(128, dtype=BF16, device="cuda")
    assert mxq.dropout(x, g, 0.5, residual=x.view(-1), out=out) is out
    assert torch.equal(out.view(4, 32), mxq.dropout(x, g, 0.5, residual=x))


def test_bias_scales_and_codes(mxq):
    x, w, ms = rand(1, M, K), rand(3, E, N, K), dev_i64([16, 16])
    xq, xs = mxq.int8_quantize_rows(x)
    wq, ws = mxq.int8_quantize_rows(w.view(E * N, K))
    wq, bias = wq.view(E, N, K), rand(4, E, N)
    for call in (
        lambda: mxq.ragged_gemm_fprop(x, w, ms, bias=bias.t().contiguous()),
        lambda: mxq.ragged_gemm_fprop(x, w, ms, bias=rand(4, E + 1, N)),
        lambda: mxq.int8_gemm_fprop(xq, xs, wq, ws.view(E, N).t().contiguous(), ms),
        lambda: mxq.int8_gemm_fprop(xq, xs, wq, ws.view(E, N), ms, bias=bias.t().contiguous()),
        lambda: mxq.int8_gemm_fprop(xq, torch.ones(M + 1, device="cuda"), wq, ws.view(E, N), ms),
        lambda: mxq.int8_gemm_fprop(xq, xs.view(2, M // 2), wq, ws.view(E, N), ms),
        lambda: mxq.int8_quantize_rows(x, out=(torch.empty((K, M), dtype=torch.int8, device="cuda"), xs)),
        lambda: mxq.int8_quantize_rows(x, out=(xq, torch.empty(M + 1, device="cuda"))),
    ):
        with pytest.raises(mxq.MXQError):
            call()
    want = mxq.int8_gemm_fprop(xq, xs, wq, ws.view(E, N), ms, bias=bias)
    # a column of scales, and the flat scales and bias of all experts
    assert torch.equal(mxq.int8_gemm_fprop(xq, xs.view(M, 1), wq, ws, ms, bias=bias.view(-1)), want)


@pytest.mark.parametrize("counts", [[1, 2], [17, 14], [100, 29]], ids=str)
def test_scales_at_any_float(mxq, counts):
    """A slice of a batch: its scales begin at any float of the batch's."""
    m = sum(counts)
    x, w, ms = rand(1, m + 3, K), rand(3, E, N, K), dev_i64(counts)
    wq, ws = mxq.int8_quantize_rows(w.view(E * N, K))
    wq, ws = wq.view(E, N, K), ws.view(E, N)
    xq, xs = mxq.int8_quantize_rows(x)
    for at in (1, 2, 3):
        rows = slice(at, at + m)
        codes, scales = torch.empty_like(xq[rows]), torch.zeros(m + 6, device="cuda")
        mxq.int8_quantize_rows(x[rows], out=(codes, scales[at:at + m]))
        assert torch.equal(scales[at:at + m], xs[rows]) and not scales[:at].any() and not scales[at + m:].any()
        late = torch.zeros(E * N + 3, device="cuda")
        late[at:at + E * N] = ws.view(-1)
        for dt in (BF16, torch.float32):
            want = mxq.int8_gemm_fprop(xq[rows], xs[rows].clone(), wq, ws, ms, out_dtype=dt)
            got = mxq.int8_gemm_fprop(xq[rows], xs[rows], wq, late[at:at + E * N].view(E, N), ms, out_dtype=dt)
            assert torch.equal(got, want)

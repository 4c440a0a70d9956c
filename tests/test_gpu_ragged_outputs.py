"""Allocation of the outputs of the ragged, int8 and dropout calls."""
import pytest
import torch

from tests._gpu import dev_i64, lib, require_gpu
from tests.test_gpu_ragged import rand

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def mxq():
    require_gpu()
    return lib()


def outputs(mxq):
    x, w, ms, g = rand(1, 32, 64), rand(3, 2, 72, 64), dev_i64([16, 16]), torch.tensor([1, 2], device="cuda")
    q, s = mxq.int8_quantize_rows(x)
    return [mxq.ragged_gemm_fprop(x, w, ms), mxq.ragged_gemm_fprop(x, w, ms, out_dtype=F32),
            mxq.ragged_gemm_wgrad(rand(2, 32, 72), x, ms), q, s, mxq.swiglu_dropout_fwd(x, g, 0.5),
            mxq.dropout(rand(4, 2, 3, 5, 7), g, 0.5)]


def changed_signature(size, stride):
    raise AssertionError("called with arguments of its own")


def another_tensor(size, stride, dtype):
    return torch.empty_strided(size, stride, dtype=dtype)  # on the host


@pytest.mark.parametrize("other", [None, changed_signature, another_tensor])
def test_without_the_private_allocator(mxq, monkeypatch, other):
    want = outputs(mxq)
    monkeypatch.setattr(mxq.mxq, "_empty_strided", other)
    monkeypatch.setattr(mxq.mxq, "_fast_empty", None, raising=False)  # not tried yet
    got = outputs(mxq)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and a.stride() == b.stride() and a.dtype == b.dtype and a.device == b.device


def test_deterministic_mode_fills_what_is_not_written(mxq):
    x, w, s = rand(1, 32, 64), rand(3, 2, 72, 64), mxq.new_status()
    torch.use_deterministic_algorithms(True)
    try:
        y = mxq.ragged_gemm_fprop(x, w, dev_i64([16, 15]), status=s)  # wrong counts: nothing is written
    finally:
        torch.use_deterministic_algorithms(False)
    assert mxq.status_read(s) != 0 and torch.isnan(y).all()

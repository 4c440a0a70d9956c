"""The entry points of the ragged products and of dropout refuse bad arguments
on the host, before any pointer is used (CPU only)."""
import pytest
import torch

P = 1 << 20  # a 16-byte-aligned address that is never dereferenced
NULL, SHAPE, ARCH, FLAGS, ALIGN, VALUE = -1, -2, -4, -7, -8, -10
M, N, K, E = 100, 72, 64, 3


@pytest.fixture(scope="module")
def L():
    from moe_expert_grouped_group_gb300.build import build
    from moe_expert_grouped_group_gb300.mxq import load

    return load(build())


CALLS = {
    "mxq_ragged_gemm_fprop": (P, K, P, None, M, N, K, E, P, 0, P, None, None),
    "mxq_ragged_gemm_dgrad": (P, N, P, M, N, K, E, P, 0, P, None, None),
    "mxq_ragged_gemm_wgrad": (P, N, P, K, M, N, K, E, P, 0, P, None, None),
    "mxq_int8_quantize_rows": (P, K, M, K, P, P, None),
    "mxq_int8_gemm_fprop": (P, P, P, P, None, M, N, K, E, P, 0, P, None, None),
    "mxq_swiglu_dropout_fwd": (P, M, K, P, 0.5, P, None),
    "mxq_swiglu_dropout_bwd": (P, P, M, K, P, 0.5, P, None),
    "mxq_dropout": (P, None, M, P, 0.5, 0, P, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_missing_pointers(L, name):
    args = list(CALLS[name])
    assert args[0] == P
    args[0] = None
    assert getattr(L, name)(*args) == NULL


@pytest.mark.parametrize("name,at", [("mxq_ragged_gemm_fprop", 9), ("mxq_ragged_gemm_dgrad", 8),
                                     ("mxq_ragged_gemm_wgrad", 9), ("mxq_int8_gemm_fprop", 10), ("mxq_dropout", 5)])
def test_unknown_flags(L, name, at):
    args = list(CALLS[name])
    args[at] = 1 << 20
    assert getattr(L, name)(*args) == FLAGS


@pytest.mark.parametrize("name", CALLS)
def test_no_gb300_no_result(L, name):
    """On a host without a GB300 every call says so; nothing runs in its place."""
    if torch.cuda.is_available() and torch.cuda.get_device_capability(0) == (10, 3):
        pytest.skip("a GB300 is present: the GPU tests cover these calls")
    assert getattr(L, name)(*CALLS[name]) == ARCH


def test_error_text(L):
    assert L.mxq_error_string(VALUE).decode() == "a scalar argument is outside its range"

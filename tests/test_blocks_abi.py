"""The entry points of the gated products, the block-scaled fp8 products and a block's norms refuse bad arguments on the host, before any
pointer is used, and the definitions that the GPU tests compare with agree with differences (CPU only)."""
import pytest
import torch

from ._blocks import norm_bwd, norm_fwd

P = 1 << 20  # a 16-byte-aligned address that is never dereferenced
NULL, ARCH, FLAGS = -1, -4, -7
M, N, K, E, F = 100, 80, 64, 3, 256
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    from moe_expert_grouped_group_gb300.build import build
    from moe_expert_grouped_group_gb300.mxq import load

    return load(build())


CALLS = {
    "mxq_ragged_gemm_fprop_swiglu": (P, K, P, P, M, F, K, E, P, P, P, None, None),
    "mxq_ragged_gemm_dgrad_swiglu": (P, N, P, P, M, N, F, E, P, P, P, None, None),
    "mxq_fp8_quantize_rows": (P, K, M, K, P, P, None),
    "mxq_fp8_quantize_weight": (P, N, K, E, P, P, None),
    "mxq_fp8_gemm_fprop": (P, P, P, P, None, M, N, K, E, P, 0, P, None, None),
    "mxq_fp8_gemm_dgrad": (P, P, P, P, M, N, K, E, P, 0, P, None, None),
    "mxq_norm_residual_fwd": (P, P, P, P, P, M, F, 1.0, 1e-6, 0, P, P, P, None, None),
    "mxq_norm_residual_bwd": (P, P, P, P, P, P, P, P, M, F, 1.0, 0, P, P, P, P, P, None, P, BIG, None),
}
REQUIRED = {
    "mxq_ragged_gemm_fprop_swiglu": (0, 2, 8, 9),
    "mxq_ragged_gemm_dgrad_swiglu": (0, 2, 3, 8, 9),
    "mxq_fp8_quantize_rows": (0, 4, 5),
    "mxq_fp8_quantize_weight": (0, 4, 5),
    "mxq_fp8_gemm_fprop": (0, 1, 2, 3, 9, 11),
    "mxq_fp8_gemm_dgrad": (0, 1, 2, 3, 8, 10),
    # n_out and pre_weight go together; so do a weight's, the gate's and dn's gradients with what they belong to
    "mxq_norm_residual_fwd": (0, 3, 11),
    "mxq_norm_residual_bwd": (1, 2, 3, 4, 5, 6, 7, 14, 15, 16),
}


@pytest.mark.parametrize("name,at", [(n, i) for n, r in REQUIRED.items() for i in r])
def test_missing_pointers(L, name, at):
    args = list(CALLS[name])
    assert args[at] == P
    args[at] = None
    # without a GB300 the check of the device may come before that of m_splits
    assert getattr(L, name)(*args) in ((NULL, ARCH) if "gemm" in name and args[at - 1] == E else (NULL,))


@pytest.mark.parametrize("name,at", [("mxq_fp8_gemm_fprop", 10), ("mxq_fp8_gemm_dgrad", 9), ("mxq_norm_residual_fwd", 9),
                                     ("mxq_norm_residual_bwd", 11)])
def test_unknown_flags(L, name, at):
    args = list(CALLS[name])
    args[at] = 1 << 20
    assert getattr(L, name)(*args) == FLAGS


@pytest.mark.parametrize("name", CALLS)
def test_no_gb300_no_result(L, name):
    if torch.cuda.is_available() and torch.cuda.get_device_capability(0) == (10, 3):
        pytest.skip("a GB300 is present: the GPU tests cover these calls")
    assert getattr(L, name)(*CALLS[name]) == ARCH


def test_workspace(L):
    from moe_expert_grouped_group_gb300.mxq import OP_NORM_RESIDUAL_BWD

    size = lambda m, f: L.mxq_workspace_bytes(OP_NORM_RESIDUAL_BWD, m, 0, f, 0, 0)
    assert size(0, 8) == 2 * 8 * 4  # one empty block
    assert size(1, 2048) == 2 * 2048 * 4
    assert size(10, 0) == size(-1, 8) == size(10, 1 << 20) == 0
    for f in (8, 256, 2048, 16384):  # bounded in the number of rows
        assert size(1 << 27, f) == size(1 << 28, f) > 0


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_norm_gradients_are_the_definitions(post, pre, gated):
    """The formulas against automatic differentiation of the definition and against its differences."""
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    m, f, scale, eps = 5, 24, 0.5, 1e-3
    t = {"x": n(m, f), "r": n(m, f), "post": 1 + 0.3 * n(f) if post else None, "pre": 1 + 0.3 * n(f) if pre else None,
         "gate": n(m) if gated else None}
    dres, dn = n(m, f), n(m, f)

    def loss(v):
        r2, out, _ = norm_fwd(v["x"], v["r"], v["post"], v["pre"], v["gate"], scale, eps)
        return (r2 * dres).sum() + ((out * dn).sum() if pre else 0.0)

    leaves = {k: v.clone().requires_grad_() for k, v in t.items() if v is not None}
    loss({**t, **leaves}).backward()
    r2, _, stats = norm_fwd(t["x"], t["r"], t["post"], t["pre"], t["gate"], scale, eps)
    got, _ = norm_bwd(dres, dn if pre else None, t["x"], r2, stats, t["post"], t["pre"], t["gate"], scale)
    names = {"x": "dx", "r": "dresidual", "post": "dpost_weight", "pre": "dpre_weight", "gate": "dgate"}
    assert {names[k] for k in leaves} == set(got)
    for k, v in leaves.items():
        assert torch.allclose(got[names[k]], v.grad, rtol=1e-11, atol=1e-12), k
        d = n(*t[k].shape)
        h = 1e-5  # the difference's own error is of order h^2 and of the rounding over h
        diff = (loss({**t, k: t[k] + h * d}) - loss({**t, k: t[k] - h * d})) / (2 * h)
        assert abs(diff - (got[names[k]] * d).sum()) <= 1e-7 * (1 + (got[names[k]] * d).abs().sum())


def test_tensors_of_another_device(monkeypatch):
    from moe_expert_grouped_group_gb300 import mxq

    class On:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    monkeypatch.setattr(mxq, "_current_device", lambda: 1)
    monkeypatch.setattr(mxq, "_several_devices", lambda: True)
    mxq._here(On(1), "x", None, On(1), *mxq._outputs(None), *mxq._outputs((On(1), None)))
    for args in ((On(0),), (On(1), On(0)), (On(1), None, *mxq._outputs(On(0))), (On(1), *mxq._outputs((On(1), On(0))))):
        with pytest.raises(mxq.MXQError, match="on device 0, the current one is 1"):
            mxq._here(args[0], "x", *args[1:])

"""What the block's calls return where outputs are given: all that was asked for and nothing else."""
import pytest
import torch

from .test_gpu_norm import make, mxq  # noqa: F401 (mxq is a fixture)
from .test_gpu_ragged_swiglu import normal, splits

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def test_norm_gradients_returned(mxq):  # noqa: F811
    """A tensor given for a gradient that the call does not compute is neither written nor returned."""
    a = make(5, 40, 512, BF16)
    r, _, stats = mxq.norm_residual_fwd(**a)
    dres, dn = make(1, 40, 512, BF16)["x"], make(2, 40, 512, BF16)["x"]
    args = (dres, dn, a["x"], r, stats)
    want = mxq.norm_residual_bwd(*args, a["post_weight"], a["pre_weight"], a["gate"])
    given = {k: torch.full_like(v, 7.0) for k, v in want.items()}
    got = mxq.norm_residual_bwd(*args, a["post_weight"], a["pre_weight"], a["gate"], dx_out=False, out=given)
    assert set(got) == set(want) - {"dx"} and (given["dx"] == 7.0).all() and set(given) == set(want)
    assert all(got[k] is given[k] and torch.equal(got[k], want[k]) for k in got)
    given = {k: torch.full_like(v, 7.0) for k, v in want.items()}
    got = mxq.norm_residual_bwd(*args, None, a["pre_weight"], None, out=given)
    assert set(got) == {"dx", "dresidual", "dpre_weight"}
    assert all((given[k] == 7.0).all() for k in ("dpost_weight", "dgate"))
    given = {"dx": torch.full_like(want["dx"], 7.0), "dgate": None}  # the rest is made
    got = mxq.norm_residual_bwd(*args, a["post_weight"], a["pre_weight"], a["gate"], out=given)
    assert got["dx"] is given["dx"] and set(got) == set(want) and all(torch.equal(got[k], want[k]) for k in want)
    with pytest.raises(mxq.MXQError):  # a name that is no gradient's
        mxq.norm_residual_bwd(*args, a["post_weight"], a["pre_weight"], a["gate"], out={"dresidue": want["dx"]})


@pytest.mark.parametrize("counts", [[2, 3], [100, 200]])
def test_gated_pairs(mxq, counts):  # noqa: F811
    """None in a pair of outputs: that one is made."""
    M, F, K, ms = sum(counts), 72, 136, splits(counts)
    x, w, w2 = normal(1, M, K), normal(2, 2, 2 * F, K), normal(3, 2, K, F)
    h, y = mxq.ragged_gemm_fprop_swiglu(x, w, ms, y_out=True)
    d, h2 = mxq.ragged_gemm_dgrad_swiglu(x, w2, y, ms, h_out=True)
    for call, args, flag, want in ((mxq.ragged_gemm_fprop_swiglu, (x, w, ms), "y_out", (h, y)),
                                   (mxq.ragged_gemm_dgrad_swiglu, (x, w2, y, ms), "h_out", (d, h2))):
        for given in ((None, None), (torch.full_like(want[0], 7.0), None), (None, torch.full_like(want[1], 7.0)),
                      [torch.full_like(v, 7.0) for v in want]):
            got = call(*args, **{flag: True}, out=given)
            assert all(g is None or a is g for a, g in zip(got, given))
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        for given in (torch.empty_like(want[0]), (want[0],), want + want):
            with pytest.raises(mxq.MXQError):
                call(*args, **{flag: True}, out=given)

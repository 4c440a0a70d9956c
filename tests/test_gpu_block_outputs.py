"""What the block's calls return where outputs are given: all that was asked for and nothing else."""
import pytest
import torch

from .test_gpu_norm import make, mxq  # noqa: F401 (mxq is a fixture)

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

"""Norms and their gradients where every CTA, cluster or team of lanes walks several rows: its ring of stages goes round
more than twice, the sums' buffers are used again, and what is held from one row to the next is another row's."""
import pytest
import torch

from ._blocks import U, norm_bwd
from .test_gpu_norm import BF16, F32, check_fwd, close, dbl, make, mxq  # noqa: F401 (mxq is a fixture)

pytestmark = pytest.mark.gpu
# roundings of a row's sum: 8 in a thread, 5 of a warp, at most 2 + 5 over a row's 64 warps; a dozen for the rest
ROW = 32

# rows, columns: lanes of a warp (three widths), one CTA to a row (two to 32 warps), a cluster of eight
FORWARD = [(120001, 64), (60001, 120), (30001, 256), (130001, 512), (20001, 2056), (5000, 4096), (2001, 8192), (3001, 9000),
           (1501, 16384)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,F", FORWARD)
def test_forward(mxq, M, F, dtype):  # noqa: F811
    for form in (dict(), dict(gate=False), dict(post=False), dict(pre=False, residual=False)):
        a = make(M + F, M, F, dtype, **form)
        check_fwd(a, 0.5, 1e-5, *mxq.norm_residual_fwd(**a, scale=0.5, eps=1e-5))


# lanes of a warp, one CTA to a row, clusters of four and of eight
BACKWARD = [(60001, 64), (30001, 128), (20001, 256), (9001, 1000), (6001, 2048), (3001, 4096), (1023, 7168), (900, 8192),
            (600, 9000), (700, 16384)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,F", BACKWARD)
def test_backward(mxq, M, F, dtype):  # noqa: F811
    for form in (dict(), dict(gate=False), dict(post=False), dict(pre=False)):
        a = make(M + F, M, F, dtype, **form)
        res, _, stats = mxq.norm_residual_fwd(**a, scale=0.5)
        dres, dn = make(1, M, F, dtype)["x"], make(2, M, F, dtype)["x"] if a["pre_weight"] is not None else None
        args = (a["x"], res, stats, a["post_weight"], a["pre_weight"], a["gate"], 0.5)
        got = mxq.norm_residual_bwd(dres, dn, *args)
        ref, mag = norm_bwd(dbl(dres), dbl(dn), *[dbl(v) if torch.is_tensor(v) else v for v in args])
        assert set(ref) == set(got)
        # a weight's gradient: the rows of one walk after another (19 walks at least, clusters of eight on 152 SMs; 152
        # without clusters), eight warps' parts, then at most 912 partial rows, 32 at once
        walks = 19 if F > 4096 else 152
        rows = -(-M // walks) + 8 + 29 + 5
        for k in ref:
            close(got[k], ref[k], (2 * ROW + (rows if k.endswith("weight") else 0)) * U * mag[k], (k, form))


def test_long_axis_distinct_rows(mxq):  # noqa: F811
    """Rows past 2^31 elements that differ from each other, in values that every step keeps exact but for single units of
    fp32, which the rounding to bf16 takes off: a row in another's place shows."""
    M, F = (1 << 18) + 3, 8200
    c = 1.0 + (torch.arange(M, device="cuda") % 127) / 128.0  # 127 rows before one comes again: no walk's stride
    w = torch.full((F,), 2.0, dtype=BF16, device="cuda")
    x = torch.ones(M, F, dtype=BF16, device="cuda")
    r, n, stats = mxq.norm_residual_fwd(x, post_weight=w, pre_weight=w, gate=c)
    assert (r == (2.0 * c).to(BF16)[:, None]).all() and (n == 2.0).all()
    torch.testing.assert_close(stats, torch.stack([torch.ones_like(c), 0.5 / c]), rtol=1e-5, atol=0.0)
    del x
    # t = dn w is the same in a row, so what the norm adds to dres is 0
    dres = (3.0 - c).to(BF16)[:, None].expand(M, F).contiguous()
    g = mxq.norm_residual_bwd(dres, n, None, r, torch.stack([torch.ones_like(c), 0.5 / c]), pre_weight=w, dx_out=False)
    assert torch.equal(g["dresidual"], dres)
    torch.testing.assert_close(g["dpre_weight"], torch.full((F,), 2.0 * M, device="cuda"), rtol=1e-5, atol=0.0)


@pytest.mark.parametrize("F", [256, 2048, 9000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_squares_beyond_range(mxq, F, dtype):  # noqa: F811
    """A row whose squares' sum is beyond fp32's range counts as infinitely large, its norm as 0; the other rows keep their
    bits, and the gradients through such a row stay finite."""
    a = make(5, 9, F, dtype)
    clean = mxq.norm_residual_fwd(**a)
    a["x"][3], a["residual"][6, 1] = 2.0 ** 70, 2.0 ** 70
    got = r, n, stats = mxq.norm_residual_fwd(**a)
    keep = [0, 1, 2, 4, 5, 7, 8]
    assert all(torch.equal(c[keep], g[keep]) for c, g in zip(clean[:2], got))
    assert torch.equal(r[3], a["residual"][3]) and (n[6] == 0).all() and stats[0, 3] == 0 and stats[1, 6] == 0
    dres, dn = make(1, 9, F, dtype)["x"], make(2, 9, F, dtype)["x"]
    g = mxq.norm_residual_bwd(dres, dn, a["x"], r, stats, a["post_weight"], a["pre_weight"], a["gate"])
    assert all(v.isfinite().all() for v in g.values()) and (g["dx"][3] == 0).all()
    assert torch.equal(g["dresidual"][6], dres[6])


@pytest.mark.parametrize("M,F", [(20001, 256), (9001, 1000), (3001, 4096), (1023, 7168), (3001, 9000)])
def test_in_place_walks(mxq, M, F):  # noqa: F811
    """r' over the residual or x, n over x, dr over dr', while the rows behind are on their way: the bits of the calls with
    outputs of their own."""
    a = make(5, M, F, BF16)
    r, n, stats = mxq.norm_residual_fwd(**a)
    b = {k: v.clone() for k, v in a.items()}
    r2, n2, stats2 = mxq.norm_residual_fwd(**b, out=(b["residual"], b["x"], None))
    assert r2 is b["residual"] and n2 is b["x"]
    assert torch.equal(r, r2) and torch.equal(n, n2) and torch.equal(stats, stats2)
    x = a["x"].clone()
    r2, n2, _ = mxq.norm_residual_fwd(**{**a, "x": x}, out=(x, None, None))
    assert r2 is x and torch.equal(r, r2) and torch.equal(n, n2)
    dres, dn = make(1, M, F, BF16)["x"], make(2, M, F, BF16)["x"]
    args = (dn, a["x"], r, stats, a["post_weight"], a["pre_weight"], a["gate"])
    want = mxq.norm_residual_bwd(dres, *args)
    got = mxq.norm_residual_bwd(dres, *args, out={"dresidual": dres})
    assert got["dresidual"] is dres and all(torch.equal(want[k], got[k]) for k in want)

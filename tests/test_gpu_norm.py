"""Norms before and after a block, and their gradients, against their 64-bit definitions."""
import pytest
import torch

from ._blocks import HALF, U, norm_bwd, norm_fwd

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# fp32 roundings on the way to a result beside its rounding: a row's sum of squares passes through at most 32 additions
# in a thread (4 vectors of 8), 5 of a warp and 4 of a team, the statistics, weights and factors through a dozen more.
STEPS = 64


@pytest.fixture(scope="module")
def mxq():
    import moe_expert_grouped_group_gb300 as m

    return m


def make(seed, M, F, dtype, post=True, pre=True, gate=True, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda std, *shape: torch.empty(shape, device="cuda").normal_(0, std, generator=g)
    return dict(x=normal(0.7, M, F).to(dtype), residual=normal(3.0, M, F).to(dtype) if residual else None,
                post_weight=(1 + normal(0.3, F)).to(dtype) if post else None,
                pre_weight=(1 + normal(0.3, F)).to(dtype) if pre else None,
                gate=torch.sigmoid(normal(1.0, M)) if gate else None)


def dbl(t):
    return None if t is None else t.double()


def close(got, ref, err, what):
    """Within `err` of the definition, and half a step of the type on top."""
    assert got.shape == ref.shape, what
    off = (got.double() - ref).abs()
    bound = err + HALF[got.dtype] * (ref.abs() + err) * (1 if got.dtype == BF16 else 0)
    assert (off <= bound).all(), (what, (off / bound.clamp(min=1e-300)).max().item())


SHAPES = [(1, 8), (3, 64), (2, 248), (5, 256), (70, 264), (9, 1000), (7, 2048), (300, 2056), (4, 4096), (5, 4104), (1, 7168),
          (3, 8192), (2, 8200), (3, 16384)]
FORMS = [dict(), dict(gate=False), dict(post=False), dict(post=False, gate=False), dict(pre=False), dict(residual=False),
         dict(pre=False, post=False, gate=False)]


def check_fwd(a, scale, eps, r, n, stats):
    d = {k: dbl(v) for k, v in a.items()}
    ref_r, ref_n, ref_s = norm_fwd(d["x"], d["residual"], d["post_weight"], d["pre_weight"], d["gate"], scale, eps)
    part = (ref_r - (0 if d["residual"] is None else d["residual"])).abs()
    err = STEPS * U * (part + (0 if d["residual"] is None else d["residual"].abs()))
    if r is not None:
        close(r, ref_r, err, "r'")
    if n is not None:
        # an error e of r' enters n by itself and by the norm of its row, which it moves by at most |e| / |r'|
        rows = err.norm(dim=1, keepdim=True) / ref_r.norm(dim=1, keepdim=True)
        close(n, ref_n, err * (ref_s[1][:, None] * d["pre_weight"].abs()) + ref_n.abs() * (rows + STEPS * U), "n")
    if stats is not None:
        rel = torch.stack([torch.full_like(ref_s[0], STEPS * U), STEPS * U + err.norm(dim=1) / ref_r.norm(dim=1)])
        close(stats, ref_s, rel * ref_s, "stats")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,F", SHAPES)
def test_forward(mxq, M, F, dtype):
    a = make(M + F, M, F, dtype)
    check_fwd(a, 0.5, 1e-5, *mxq.norm_residual_fwd(**a, scale=0.5, eps=1e-5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", FORMS)
def test_forward_forms(mxq, form, dtype):
    for M, F in ((37, 320), (5, 6000)):
        a = make(M, M, F, dtype, **form)
        r, n, stats = mxq.norm_residual_fwd(**a)
        assert (n is None) == (a["pre_weight"] is None)
        check_fwd(a, 1.0, 1e-6, r, n, stats)
        if n is not None:  # r' and stats left out
            r2, n2, s2 = mxq.norm_residual_fwd(**a, res_out=False, stats_out=False)
            assert r2 is None and s2 is None and torch.equal(n, n2)


def check_bwd(a, dres, dn, res, stats, scale, g):
    d = {k: dbl(v) for k, v in a.items()}
    ref, mag = norm_bwd(dbl(dres), dbl(dn), d["x"], dbl(res), stats.double(), d["post_weight"], d["pre_weight"], d["gate"],
                        scale)
    assert set(ref) == set(g)
    M = a["x"].shape[0]
    for k in ref:
        # sums over rows: one addition a row at most, and as many again when partial sums are joined
        close(g[k], ref[k], (2 * STEPS + (2 * M if k.endswith("weight") else 0)) * U * mag[k], k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,F", SHAPES + [(2000, 96), (1500, 2048)])
def test_backward(mxq, M, F, dtype):
    a = make(M + F, M, F, dtype)
    res, _, stats = mxq.norm_residual_fwd(**a, scale=0.5)
    dres, dn = make(1, M, F, dtype)["x"], make(2, M, F, dtype)["x"]
    del a["residual"]
    g = mxq.norm_residual_bwd(dres, dn, a["x"], res, stats, a["post_weight"], a["pre_weight"], a["gate"], 0.5)
    a["residual"] = None
    check_bwd(a, dres, dn, res, stats, 0.5, g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", FORMS[:-1])
@pytest.mark.parametrize("with_dres", [True, False])
def test_backward_forms(mxq, form, with_dres, dtype):
    for M, F in ((37, 320), (5, 6000), (3, 9000)):
        a = make(M, M, F, dtype, **form)
        res, _, stats = mxq.norm_residual_fwd(**a)
        pre = a["pre_weight"] is not None
        if not with_dres and not pre:
            continue
        dres, dn = make(1, M, F, dtype)["x"] if with_dres else None, make(2, M, F, dtype)["x"] if pre else None
        g = mxq.norm_residual_bwd(dres, dn, a["x"], res, stats, a["post_weight"], a["pre_weight"], a["gate"])
        check_bwd(a, dres, dn, res, stats, 1.0, g)


def test_long_axis(mxq):
    """More rows than one walk of the grid, rows past 2^31 elements, and the last rows right."""
    M, F = (1 << 18) + 3, 8200
    x = torch.ones(M, F, dtype=BF16, device="cuda")
    x[-2:] = 3.0
    w = torch.full((F,), 2.0, dtype=BF16, device="cuda")
    r, n, _ = mxq.norm_residual_fwd(x, post_weight=w, pre_weight=w, stats_out=False)
    assert (r == 2.0).all() and (n == 2.0).all()
    del r
    g = mxq.norm_residual_bwd(None, n, None, x, torch.ones(2, M, device="cuda"), pre_weight=w)
    assert (g["dpre_weight"] == 2.0 * (M - 2) + 12.0).all()


def test_in_place(mxq):
    a = make(5, 33, 2048, BF16)
    r, n, stats = mxq.norm_residual_fwd(**a)
    b = {k: v.clone() for k, v in a.items()}
    r2, n2, _ = mxq.norm_residual_fwd(**b, out=(b["residual"], b["x"], None))
    assert r2 is b["residual"] and torch.equal(r, r2) and torch.equal(n, n2)
    dres, dn = make(1, 33, 2048, BF16)["x"], make(2, 33, 2048, BF16)["x"]
    args = (dn, a["x"], r, stats, a["post_weight"], a["pre_weight"], a["gate"])
    g = mxq.norm_residual_bwd(dres, *args)
    g2 = mxq.norm_residual_bwd(dres, *args, out={"dresidual": dres})
    assert g2["dresidual"] is dres and all(torch.equal(g[k], g2[k]) for k in g)


def test_non_finite_rows(mxq):
    a = make(5, 9, 512, BF16)
    clean = mxq.norm_residual_fwd(**a)
    a["x"][3, 7], a["residual"][5, 100], a["gate"][6] = float("nan"), float("inf"), float("nan")
    got = mxq.norm_residual_fwd(**a)
    keep = [0, 1, 2, 4, 7, 8]
    for c, g in zip(clean[:2], got[:2]):
        assert torch.equal(c[keep], g[keep])
    assert got[1][[3, 6]].isnan().all() and got[1][5, 100].isnan() and (got[1][5, :100] == 0).all()


@pytest.mark.parametrize("F", [64, 512, 4104, 9000])
def test_no_rows(mxq, F):
    a = make(5, 0, F, F32)
    r, n, stats = mxq.norm_residual_fwd(**a)
    assert r.shape == n.shape == (0, F) and stats.shape == (2, 0)
    g = mxq.norm_residual_bwd(r, n, a["x"], r, stats, a["post_weight"], a["pre_weight"], a["gate"])
    assert (g["dpost_weight"] == 0).all() and (g["dpre_weight"] == 0).all() and g["dgate"].shape == (0,)


def test_one_output(mxq):
    """dx or dresidual left out: the other's bits are the same; neither is refused."""
    a = make(5, 40, 512, BF16)
    r, n, stats = mxq.norm_residual_fwd(**a)
    dres, dn = make(1, 40, 512, BF16)["x"], make(2, 40, 512, BF16)["x"]
    args = (dres, dn, a["x"], r, stats, a["post_weight"], a["pre_weight"], a["gate"])
    g = mxq.norm_residual_bwd(*args)
    for left_out in ("dx", "dresidual"):
        h = mxq.norm_residual_bwd(*args, **{left_out + "_out": False})
        assert left_out not in h and set(h) | {left_out} == set(g) and all(torch.equal(h[k], g[k]) for k in h)
    with pytest.raises(mxq.MXQError):
        mxq.norm_residual_bwd(*args, dx_out=False, dresidual_out=False)


def test_graph_and_bits(mxq):
    """The same bits from call to call, and from a captured graph replayed on new values."""
    a = make(5, 700, 1024, BF16)
    dres, dn = make(1, 700, 1024, BF16)["x"], make(2, 700, 1024, BF16)["x"]

    def step():
        res, n, stats = mxq.norm_residual_fwd(**a)
        return n, mxq.norm_residual_bwd(dres, dn, a["x"], res, stats, a["post_weight"], a["pre_weight"], a["gate"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n, g = step()
    for seed in (11, 12):
        for k, v in make(seed, 700, 1024, BF16).items():
            a[k].copy_(v)
        graph.replay()
        n2, g2 = step()
        assert torch.equal(n, n2) and all(torch.equal(g[k], g2[k]) for k in g)


def test_refusals(mxq):
    a = make(5, 4, 64, BF16)
    for k, v in (("x", a["x"].t()), ("x", a["x"].half()), ("residual", a["residual"].float()), ("post_weight", a["x"][0][:8]),
                 ("gate", a["gate"].to(BF16)), ("gate", a["gate"][:2]), ("pre_weight", a["pre_weight"].cpu())):
        with pytest.raises(mxq.MXQError):
            mxq.norm_residual_fwd(**{**a, k: v})
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(scale=float("inf")), dict(eps=-1.0), dict(eps=1e-60)):
        with pytest.raises(mxq.MXQError):
            mxq.norm_residual_fwd(**a, **kw)
    with pytest.raises(mxq.MXQError):  # no output at all
        mxq.norm_residual_fwd(a["x"], res_out=False)
    with pytest.raises(mxq.MXQError):
        mxq.norm_residual_fwd(torch.zeros(2, 12, device="cuda"))
    with pytest.raises(mxq.MXQError):
        mxq.norm_residual_fwd(torch.zeros(2, 16392, device="cuda"))
    r, n, stats = mxq.norm_residual_fwd(**a)
    w = (a["post_weight"], a["pre_weight"], a["gate"])
    for args in ((None, None, a["x"], r, stats, *w), (r, None, a["x"], r, stats, *w), (r, n, None, r, stats, *w),
                 (r, n, a["x"], None, stats, *w), (r, n, a["x"], r, None, *w), (r, n, a["x"], r, stats[:1], *w),
                 (r, n.float(), a["x"], r, stats, *w)):
        with pytest.raises(mxq.MXQError):
            mxq.norm_residual_bwd(*args)
    with pytest.raises(mxq.MXQError):  # a workspace too small
        mxq.norm_residual_bwd(r, n, a["x"], r, stats, *w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))

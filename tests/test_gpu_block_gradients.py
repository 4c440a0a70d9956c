"""The feed-forward half's gradients in bounds tight enough to see a missing term: every product takes the codes that the
block itself quantized, so that what is left are bf16 roundings, in fp8 as in bf16."""
import pytest
import torch

from ._blocks import norm_bwd, norm_fwd, row_values, weight_values
from .test_gpu_feed_forward_block import BF16, example, mxq, reference  # noqa: F401 (mxq is a fixture)

pytestmark = pytest.mark.gpu
# At most ten bf16 roundings lie on the way to a result, each off by at most 2^-8 of a value and passed on by a factor of 2
# at most; they are of either sign, so that their squares add in the 2-norm.
BOUND = 10 ** 0.5 * 2 * 2.0 ** -8


def formulas(block, r, gate, counts, dr2, dn2, rows=None, weights=None, mean=True):
    """Results and gradients in 64 bits by the formulas. rows: what the codes of n, h, dy and [dg | du] stand for, weights:
    those of W1 and W2 (None: the values themselves). mean=False leaves the mean term out of the norms' gradients."""
    f = lambda t: t.double()  # noqa: E731
    w1, w2 = weights or (f(block.w1), f(block.w2))
    spans, off = [], 0
    for m in counts:
        spans.append(slice(off, off + m))
        off += m
    times = lambda v, w, t: torch.cat([v[s] @ (w[e].t() if t else w[e]) for e, s in enumerate(spans)])  # noqa: E731
    outer = lambda a, b: torch.stack([a[s].t() @ b[s] for s in spans])  # noqa: E731
    pick = lambda i, v: v if rows is None else rows[i]  # noqa: E731

    def bwd(dres, dn, x, res, stats, post, pre, gate_, c):
        g = norm_bwd(dres, dn, x, res, stats, post, pre, gate_, c)[0]
        if not mean:
            g["dresidual"] = (0 if dres is None else dres) + stats[1][:, None] * dn * pre
        return g

    n, st_in = norm_fwd(f(r), None, None, f(block.w_in), None, 1.0, 1e-6)[1:]
    y1 = times(pick(0, n), w1, True)
    g, u = y1.chunk(2, dim=1)
    s = torch.sigmoid(g)
    h = g * s * u
    y = times(pick(1, h), w2, True)
    r2, n2, st = norm_fwd(y, f(r), f(block.w_post), f(block.w_out), f(gate), block.scale, 1e-6)
    first = bwd(f(dr2), f(dn2), y, r2, st, f(block.w_post), f(block.w_out), f(gate), block.scale)
    dy = first["dx"]
    dh = times(pick(2, dy), w2, False)
    d1 = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=1)
    dn = times(pick(3, d1), w1, False)
    last = bwd(first["dresidual"], dn, None, f(r), torch.stack([torch.ones_like(st_in[0]), st_in[1]]), None, f(block.w_in), None, 1.0)
    return r2, n2, {"r": last["dresidual"], "gate": first["dgate"], "w1": outer(d1, n), "w2": outer(dy, h),
                    "w_in": last["dpre_weight"], "w_post": first["dpost_weight"], "w_out": first["dpre_weight"]}


def distance(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts", [[70, 0, 33, 153], [3, 0, 1, 4]])
def test_gradients(mxq, monkeypatch, counts, fp8):  # noqa: F811
    M, H, F = sum(counts), 256, 144
    module = example()
    block = module.Block(4, H, F, fp8=fp8)
    g = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    r, gate, dr2, dn2 = normal(M, H), torch.rand(M, generator=g, device="cuda"), normal(M, H), normal(M, H)
    ms = torch.tensor(counts, dtype=torch.int64, device="cuda")
    taken = {"fp8_quantize_rows": [], "fp8_quantize_weight": []}
    for name, list_ in taken.items():
        call = getattr(mxq, name)

        def record(t, call=call, list_=list_):
            list_.append(call(t))
            return list_[-1]

        monkeypatch.setattr(module.mxq, name, record)
    r2, n2, saved = block.forward(r, gate, ms)
    got = block.backward(dr2, dn2, saved, ms)
    codes = lambda q: q.view(torch.float8_e4m3fn)  # noqa: E731
    rows = [row_values(codes(q), s) for q, s in taken["fp8_quantize_rows"]] or None
    weights = [weight_values(codes(q), s) for q, s in taken["fp8_quantize_weight"]] or None
    assert (len(rows) == 4 and len(weights) == 2) if fp8 else rows is None
    want_r2, want_n2, want = formulas(block, r, gate, counts, dr2, dn2, rows, weights)
    assert set(got) == set(want)
    far = {k: d for k, d in [("r2", distance(r2, want_r2)), ("n2", distance(n2, want_n2))]
           + [(k, distance(got[k], want[k])) for k in want] if not d <= BOUND}
    assert not far, far
    without = formulas(block, r, gate, counts, dr2, dn2, rows, weights, mean=False)[2]
    assert distance(without["r"], want["r"]) > BOUND  # a term left out would show
    if not fp8:  # the formulas are what automatic differentiation gives
        auto = reference(block, r, gate, counts, dr2, dn2)[2]
        assert all(distance(want[k], auto[k]) < 1e-10 for k in want)

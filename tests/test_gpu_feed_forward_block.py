"""The block's operators together, as a model uses them: gradients of the whole half against its 64-bit definition,
captured and replayed, on two streams at once, and behind kernels that let them begin early."""
import importlib.util
import os
import re

import pytest
import torch

from ._blocks import norm_fwd
from .test_gpu_early_launch import CSRC, late, producer, same  # noqa: F401 (producer is a fixture)

BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("feed_forward_block", os.path.join(ROOT, "examples", "feed_forward_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def mxq():
    import moe_expert_grouped_group_gb300 as m

    return m


def test_norms_read_nothing_as_constant():
    """As tests/test_gpu_early_launch.py asks of the other kernels that may begin early."""
    with open(os.path.join(CSRC, "mxq_norm.cu"), encoding="utf-8") as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.search(r"__ldg|\.nc\b|\.nc\.|__restrict__", code)


@pytest.mark.gpu
def test_example_runs():
    losses, n2 = example().main(steps=2)
    assert n2.shape == (8, 512) and torch.isfinite(n2).all()
    assert all(len(v) == 2 for v in losses.values())


def reference(block, r, gate, counts, dr2, dn2):
    """The gradients in 64 bits, by automatic differentiation of the definition."""
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    t = {"r": leaf(r), "gate": leaf(gate), **{k: leaf(getattr(block, k)) for k in ("w1", "w2", "w_in", "w_post", "w_out")}}
    n = norm_fwd(t["r"], None, None, t["w_in"], None, 1.0, 1e-6)[1]
    parts, off = [], 0
    for e, m in enumerate(counts):
        g, u = (n[off:off + m] @ t["w1"][e].t()).chunk(2, dim=1)
        parts.append((g * torch.sigmoid(g) * u) @ t["w2"][e].t())
        off += m
    r2, n2, _ = norm_fwd(torch.cat(parts), t["r"], t["w_post"], t["w_out"], t["gate"], block.scale, 1e-6)
    ((r2 * dr2.double()).sum() + (n2 * dn2.double()).sum()).backward()
    return r2.detach(), n2.detach(), {k: v.grad for k, v in t.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts", [[70, 0, 33, 153], [3, 0, 1, 4]])
def test_gradients(mxq, counts, fp8):
    """Every result in the 2-norm. bf16: up to ten roundings lie on the way to a gradient, each off by at most 2^-8 of the
    value, and what follows one, norms and SwiGLU, passes it on by a factor of 2 at most. fp8: six quantizations at most,
    each off by at most 2^-4 of a value that is not tiny in its block; a product's sums mix errors of both signs, so that
    their squares add."""
    M, H, F = sum(counts), 256, 136 if not fp8 else 144
    block = example().Block(4, H, F, fp8=fp8)
    g = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    r, gate, dr2, dn2 = normal(M, H).to(BF16), torch.rand(M, generator=g, device="cuda"), normal(M, H).to(BF16), normal(M, H).to(BF16)
    ms = torch.tensor(counts, dtype=torch.int64, device="cuda")
    r2, n2, saved = block.forward(r, gate, ms)
    got = block.backward(dr2, dn2, saved, ms)
    want_r2, want_n2, want = reference(block, r, gate, counts, dr2, dn2)
    bound = 6 ** 0.5 * 2 * 2.0 ** -4 if fp8 else 10 * 2 * 2.0 ** -8
    assert set(got) == set(want)
    for k, a, b in [("r2", r2, want_r2), ("n2", n2, want_n2)] + [(k, got[k], want[k]) for k in want]:
        off = ((a.double() - b).norm() / b.norm()).item()
        assert off <= bound, (k, off)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_captured_and_concurrent(mxq, fp8):
    """One graph replayed on new values and counts, and two such blocks at once on streams of their own: the bits of the
    calls one after another."""
    E, H, F, M = 4, 512, 256, 300
    block = example().Block(E, H, F, fp8=fp8)
    g = torch.Generator(device="cuda").manual_seed(5)
    make = lambda: [torch.randn(M, H, generator=g, device="cuda").to(BF16), torch.rand(M, generator=g, device="cuda"),  # noqa: E731
                    torch.randn(M, H, generator=g, device="cuda").to(BF16), torch.randn(M, H, generator=g, device="cuda").to(BF16)]
    sets = [(make(), torch.tensor(c, dtype=torch.int64, device="cuda"))
            for c in ([100, 50, 0, 150], [0, 299, 1, 0], [2, 3, 290, 5])]

    def step(values, ms):
        r, gate, dr2, dn2 = values
        r2, n2, saved = block.forward(r, gate, ms)
        return {"r2": r2, "n2": n2, **block.backward(dr2, dn2, saved, ms)}

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    values, ms = [v.clone() for v in sets[0][0]], sets[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(values, ms)
    for (v, m), w in zip(sets, want):
        for a, b in zip(values, v):
            a.copy_(b)
        ms.copy_(m)
        graph.replay()
        assert all(torch.equal(out[k], w[k]) for k in w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for stream, s in zip(streams, sets):
            with torch.cuda.stream(stream):
                got.append(step(*s))
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert all(torch.equal(a[k], w[k]) for k in w)


# single rows, a few rows of an expert (its weights are asked for before the counts are known), tiles of one SM and of a pair
@pytest.mark.gpu
@pytest.mark.parametrize("counts,other", [([1, 2, 0], [0, 0, 3]), ([17, 0, 20], [5, 30, 2]), ([150, 3, 90], [1, 240, 2]),
                                          ([400, 3, 90], [1, 490, 2])], ids=str)
def test_early_launch_products(mxq, producer, counts, other):  # noqa: F811
    E, M, N, K = len(counts), sum(counts), 144, 528

    def inputs(seed, m):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
        code = lambda *s: torch.randn(*s, generator=g, device="cuda").mul(100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        u = lambda *s: torch.rand(*s, generator=g, device="cuda") + 0.01  # noqa: E731
        return (torch.tensor(m, device="cuda"), r(M, K), r(E, 2 * N, K), r(E, K, N), r(M, 2 * N), code(M, K), u(5, M),
                code(E, N, K), u(E, 2, 5), code(M, N), u(2, M), r(E, N))

    a, b = inputs(1, counts), inputs(2, other)
    calls = {
        "fprop": lambda ms, x, w1, w2, y, xq, xs, wq, ws, dq, ds, bias: mxq.ragged_gemm_fprop_swiglu(x, w1, ms, y_out=True),
        "dgrad": lambda ms, x, w1, w2, y, xq, xs, wq, ws, dq, ds, bias: mxq.ragged_gemm_dgrad_swiglu(x, w2, y, ms, h_out=True),
        "fp8": lambda ms, x, w1, w2, y, xq, xs, wq, ws, dq, ds, bias: mxq.fp8_gemm_fprop(xq, xs, wq, ws, ms, bias=bias),
        "fp8_32": lambda ms, x, w1, w2, y, xq, xs, wq, ws, dq, ds, bias: mxq.fp8_gemm_fprop(xq, xs, wq, ws, ms, out_dtype=F32),
        "fp8_dgrad": lambda ms, x, w1, w2, y, xq, xs, wq, ws, dq, ds, bias: mxq.fp8_gemm_dgrad(dq, ds, wq, ws, ms),
        "rows": lambda ms, x, w1, w2, y, xq, xs, wq, ws, dq, ds, bias: mxq.fp8_quantize_rows(x),
        "weight": lambda ms, x, w1, w2, y, xq, xs, wq, ws, dq, ds, bias: mxq.fp8_quantize_weight(w1),
        # the quantizer lets the product begin: codes, scales and all
        "chain": lambda ms, x, w1, w2, y, xq, xs, wq, ws, dq, ds, bias: mxq.fp8_gemm_fprop(*mxq.fp8_quantize_rows(x), wq, ws, ms),
    }
    for call in calls.values():
        want = call(*a)
        same(late(producer, a, b, call), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M,F", [(33, 128), (33, 512), (9, 4096), (5, 8200)])
def test_early_launch_norms(mxq, producer, M, F):  # noqa: F811
    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
        return r(M, F), r(M, F), r(F), r(F), torch.rand(M, generator=g, device="cuda"), torch.rand(2, M, generator=g, device="cuda") + 0.5

    a, b = inputs(1), inputs(2)
    fwd = lambda x, r, w1, w2, gate, st: mxq.norm_residual_fwd(x, r, w1, w2, gate, 0.5)  # noqa: E731
    bwd = lambda x, r, w1, w2, gate, st: tuple(mxq.norm_residual_bwd(x, r, x, r, st, w1, w2, gate, 0.5).values())  # noqa: E731
    for call in (fwd, bwd):
        want = call(*a)
        same(late(producer, a, b, call), want)

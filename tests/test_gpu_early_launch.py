"""The ragged products and dropout behind a kernel that lets them begin before
it has written what they read (programmatic dependent launch): counts, scales,
codes, tokens, weights and the generator's state arrive late and count all the
same."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from tests._gpu import lib, require_gpu

BF16, F32 = torch.bfloat16, torch.float32
HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "moe_expert_grouped_group_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.startswith(("mxq_ragged", "mxq_dropout"))))
def test_nothing_is_read_as_constant(name):
    """Non-coherent loads, and pointers that let the compiler make them, promise that nobody writes the data
    during the kernel's lifetime, which here begins beside the kernel that writes it."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.search(r"__ldg|\.nc\b|\.nc\.|__restrict__", code)


@pytest.fixture(scope="module")
def mxq():
    require_gpu()
    return lib()


@pytest.fixture(scope="module")
def producer(tmp_path_factory):
    require_gpu()
    from moe_expert_grouped_group_gb300.build import ARCH, nvcc

    so = str(tmp_path_factory.mktemp("early") / "early_producer.so")
    subprocess.run([nvcc(), *ARCH, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-o", so,
                    os.path.join(HERE, "early_producer.cu"), "-lcudart"], check=True, capture_output=True)
    f = ctypes.CDLL(so).early_producer_launch
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]
    f.restype = ctypes.c_int
    return f


def late(producer, tensors, stale, call):
    """call() on tensors that hold `stale` until a producer, launched just before, writes their values."""
    sizes = [(t.nbytes + 255) // 256 * 256 for t in tensors]
    src, dst = (torch.zeros(sum(sizes), dtype=torch.uint8, device="cuda") for _ in range(2))
    views = []
    for buf, values in ((src, tensors), (dst, stale)):
        at = 0
        for t, v, size in zip(tensors, values, sizes):
            part = buf[at:at + t.nbytes].view(t.dtype).view(t.shape)
            part.copy_(v)
            at += size
            if buf is dst:
                views.append(part)
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert producer(dst.data_ptr(), src.data_ptr(), src.numel(), 50000, stream) == 0
    got = call(*views)
    torch.cuda.synchronize()
    return got


def same(got, want):
    got, want = (v if isinstance(v, tuple) else (v,) for v in (got, want))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def values(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    code = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g, device="cuda") + 0.01  # noqa: E731
    return g, r, code, u


# single tokens and a few rows of many or of few experts, and tiles of a pair of SMs; the stale counts are as valid
@pytest.mark.parametrize("counts,other", [([1, 2, 0], [0, 0, 3]), ([17, 0, 20], [5, 30, 2]), ([150, 3, 90], [1, 240, 2])],
                         ids=str)
@pytest.mark.gpu
def test_products(mxq, producer, counts, other):
    E, M, N, K = len(counts), sum(counts), 136, 528
    new, old = values(1), values(2)

    def inputs(v, m):
        g, r, code, u = v
        return (torch.tensor(m, device="cuda"), r(M, K), r(M, N), r(E, N, K), r(E, N), code(M, K), code(E, N, K), u(M),
                u(E, N))

    a, b = inputs(new, counts), inputs(old, other)
    calls = {
        "fprop": lambda ms, x, dy, w, bias, xq, wq, xs, ws: mxq.ragged_gemm_fprop(x, w, ms, bias=bias),
        "fprop32": lambda ms, x, dy, w, bias, xq, wq, xs, ws: mxq.ragged_gemm_fprop(x, w, ms, bias=bias, out_dtype=F32),
        "dgrad": lambda ms, x, dy, w, bias, xq, wq, xs, ws: mxq.ragged_gemm_dgrad(dy, w, ms),
        "wgrad": lambda ms, x, dy, w, bias, xq, wq, xs, ws: mxq.ragged_gemm_wgrad(dy, x, ms),
        "wgrad16": lambda ms, x, dy, w, bias, xq, wq, xs, ws: mxq.ragged_gemm_wgrad(dy, x, ms, out_dtype=BF16),
        "int8": lambda ms, x, dy, w, bias, xq, wq, xs, ws: mxq.int8_gemm_fprop(xq, xs, wq, ws, ms, bias=bias),
        "int8_32": lambda ms, x, dy, w, bias, xq, wq, xs, ws: mxq.int8_gemm_fprop(xq, xs, wq, ws, ms, bias=bias,
                                                                                  out_dtype=F32),
        "quantize": lambda ms, x, dy, w, bias, xq, wq, xs, ws: mxq.int8_quantize_rows(x),
    }
    for call in calls.values():
        want = call(*a)
        same(late(producer, a, b, call), want)


@pytest.mark.gpu
def test_dropout(mxq, producer):
    def inputs(v, rng):
        g, r, code, u = v
        return torch.tensor(rng, device="cuda"), r(33, 512), r(33, 256), r(33, 512)

    a, b = inputs(values(1), [3, 4]), inputs(values(2), [3, 5])
    for call in (lambda rng, y, dh, res: mxq.dropout(y, rng, 0.4), lambda rng, y, dh, res: mxq.dropout(y, rng, 0.4, residual=res),
                 lambda rng, y, dh, res: mxq.swiglu_dropout_fwd(y, rng, 0.4),
                 lambda rng, y, dh, res: mxq.swiglu_dropout_bwd(dh, y, rng, 0.4)):
        want = call(*a)
        same(late(producer, a, b, call), want)


@pytest.mark.gpu
def test_block_quantizer(mxq, producer):
    """Rows longer than a warp holds."""
    a, b = ((values(s)[1](5, 4112),) for s in (1, 2))
    want = mxq.int8_quantize_rows(*a)
    same(late(producer, a, b, mxq.int8_quantize_rows), want)

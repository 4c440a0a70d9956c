"""The 64-bit definitions that the GPU tests compare with, against published
values and against differences (CPU only)."""
import numpy as np
import pytest
import torch

from tests._ragged import (dgrad64, fprop64, keep_mask, keep_scale, philox_words, swiglu64, swiglu_grad64, wgrad64)


def words32(seed, offset, n):
    return philox_words(seed, offset, 2 * n).view("<u4")


def test_philox_known_answers():
    """The published known answers of Philox 4x32-10 whose counter fits this use (block 0)."""
    assert [hex(v) for v in words32(0, 0, 4)] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]


def test_philox_words_are_uniform_and_independent_of_length():
    a, b = philox_words(77, 1 << 35, 200000), philox_words(77, 1 << 35, 1003)
    assert np.array_equal(a[:1003], b)
    hist = np.bincount(a >> 12, minlength=16)
    assert abs(hist - 12500).max() < 6 * np.sqrt(12500)
    assert not np.array_equal(philox_words(78, 1 << 35, 64), a[:64])
    assert not np.array_equal(philox_words(77, 0, 64), a[:64])


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_expectation_is_kept(p):
    keep = keep_mask(5, 9, p, (400, 500))
    n, k = keep.numel(), keep.sum().item()
    assert abs(k - n * (1 - p)) <= 6 * np.sqrt(n * max(p * (1 - p), 1e-5)) + n / 131072
    assert p == 1.0 or abs(keep_scale(p) * (65536 - round(p * 65536)) / 65536 - 1) < 1e-15


def test_product_gradients_by_differences():
    g = torch.Generator().manual_seed(0)
    counts, E, N, K = [3, 0, 5, 1], 4, 7, 6
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, dy = r(9, K), r(E, N, K), r(9, N)
    f = lambda x, w: (dy * fprop64(x, w, counts)[0]).sum()  # noqa: E731
    vx, vw, h = r(9, K), r(E, N, K), 0.5  # the form is linear in each: a wide step is exact
    dx = (f(x + h * vx, w) - f(x - h * vx, w)) / (2 * h)
    dw = (f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h)
    assert abs(dx - (dgrad64(dy, w, counts)[0] * vx).sum()) < 1e-12 * 1e3
    assert abs(dw - (wgrad64(dy, x, counts)[0] * vw).sum()) < 1e-12 * 1e3


def test_swiglu_dropout_gradient_by_differences():
    g = torch.Generator().manual_seed(1)
    y, dh, v = (torch.randn(5, n, generator=g, dtype=torch.float64) for n in (16, 8, 16))
    keep, s, h = keep_mask(3, 4, 0.4, (5, 8)), keep_scale(0.4), 1e-5
    f = lambda y: (dh * torch.where(keep, swiglu64(y) * s, torch.zeros(()).double())).sum()  # noqa: E731
    num = (f(y + h * v) - f(y - h * v)) / (2 * h)
    ana = (swiglu_grad64(torch.where(keep, dh * s, torch.zeros(()).double()), y) * v).sum()
    assert abs(num - ana) < 1e-8 * (1 + abs(ana))

"""Packed calls on inputs that are not all numbers."""
import numpy as np
import pytest
import torch

from tests.helpers import np64
from tests.test_gpu_packed import D, U, attn_ref, block, cu_of, randn

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ NaN and infinities in q and k

@pytest.mark.parametrize("H,Hkv,lens", [(4, 2, [100, 37, 260]), (32, 8, [900, 50, 700]), (3, 3, [300])])  # keys split; not; split
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("which,bad", [("q", float("nan")), ("q", float("inf")), ("k", float("nan")), ("k", float("inf")),
                                       ("k", -float("inf"))])
def test_attn_packed_nan_and_infinities(H, Hkv, lens, window, which, bad):
    """A query whose score of a visible key is NaN or +inf, or whose scores are all -inf, gets NaN, as
    the formula does; every other row what it gets from the numbers alone."""
    n = sum(lens)
    blk = block(H, Hkv, sliding_window=window)
    x = {"q": randn(1, n, H, D), "k": randn(2, n, Hkv, D), "v": randn(3, n, Hkv, D)}
    for row, head, channel in ((0, 0, 3), (70, Hkv - 1, 127), (n - 20, 0, 64)):
        x[which][row, head, channel] = bad
    out = blk.attn_packed(x["q"], x["k"], x["v"], cu_of(lens))
    assert blk.last_status() == 0
    at, seen = 0, 0
    with np.errstate(invalid="ignore"):
        for m in lens:
            sl = slice(at, at + m)
            ref, mag = attn_ref(*(np64(x[c][sl]) for c in "qkv"), window)
            got, nan = np64(out[sl]), np.isnan(ref)
            assert np.array_equal(np.isnan(got), nan)
            err = np.abs(got - ref)[~nan]
            # the two roundings to bf16 of p and the output, and 2e-4 for the scores (see test_gpu_packed)
            assert np.all(err <= ((U + 2e-4) * mag + U * np.abs(ref))[~nan])
            seen += nan.sum()
            at += m
    assert seen > 0  # the corner is there

"""The cap's tanh of the 8-bit cache's kernels, evaluated on the CPU from the
constants in their source: the polynomial near 0 and the form beyond it."""
import math
import os
import re

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "bit_attention_video_smooth_gb300", "csrc", "vca_cache.cuh")


@pytest.fixture(scope="module")
def constants():
    src = open(SRC).read()
    near = float(re.search(r"kTanhNear = ([0-9.]+)f;", src).group(1))
    t = [float(np.float32(re.search(rf"kT{i} = ([-+0-9.e]+)f", src).group(1))) for i in range(5)]
    return near, t


def _arguments(near):
    return np.linspace(near * 1e-4, near, 400001)


def test_the_polynomials_error(constants):
    """The stated error of the polynomial with its fp32 constants, evaluated exactly: 7.7e-8 relative."""
    near, t = constants
    u = _arguments(near)
    p = sum(c * u ** (2 * i + 1) for i, c in enumerate(t))
    off = np.abs(p / np.tanh(u * (math.log(2.0) / 2.0)) - 1.0).max()
    assert 7.6e-8 < off < 7.7e-8


def test_the_polynomials_error_in_fp32(constants):
    """With its own roundings (fused multiply-adds, as the kernels have them): 2^-22."""
    near, t = constants
    u = _arguments(near).astype(np.float32)
    w = u * u

    def fma(a, b, c):
        return (a.astype(np.float64) * b.astype(np.float64) + c).astype(np.float32)

    q = np.full_like(u, t[4])
    for c in t[3::-1]:
        q = fma(q, w, c)
    off = np.abs((u * q).astype(np.float64) / np.tanh(u.astype(np.float64) * (math.log(2.0) / 2.0)) - 1.0).max()
    assert off <= 2.0 ** -22


def test_the_form_beyond_the_border(constants):
    """1 - 2 / (1 + 2^u) from the border on, its power of two and quotient off by 2^-22 each: 2^-20 relative."""
    near, _ = constants
    u = np.linspace(near, 30.0, 400001)
    ref = np.tanh(u * (math.log(2.0) / 2.0))
    for a in (1 - 2.0 ** -22, 1 + 2.0 ** -22):
        for b in (1 - 2.0 ** -22, 1 + 2.0 ** -22):
            got = 1.0 - 2.0 * b / (1.0 + np.exp2(u) * a)
            assert (np.abs(got - ref) + 2.0 ** -24).max() <= 2.0 ** -20 * ref.min()

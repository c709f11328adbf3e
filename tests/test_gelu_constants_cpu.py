"""The polynomial behind bf16's gelu, with the constants that the kernels' source
has, against the normal distribution function in float64 (no GPU needed)."""
import os
import re

import numpy as np
import pytest
from scipy.special import erfcx

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_allreduce_reduction_02_amd", "csrc",
                      "cc_ffn_tile.h")
U = 2.0 ** -24


@pytest.fixture(scope="module")
def constants():
    """p of t = 1 / (1 + p x), and the coefficients from the highest power on, as float32."""
    text = open(SOURCE).read()
    at = text.index("float normal_cdf_bf16(")
    body = text[at:text.index("\n}", at)]
    p = re.search(r"fmaf\(([\d.]+)f, fabsf\(g\), 1\.0f\)", body).group(1)
    c = re.findall(r"float r = ([-\d.e]+)f;", body) + re.findall(r"fmaf\(r, t, ([-\d.e]+)f\)", body)
    assert len(c) == 9
    return np.float32(p), [np.float32(v) for v in c]


def test_the_fit(constants):
    """P alone, its constants rounded to float32: within two half steps over 0 .. 14.5."""
    p, c = constants
    x = np.linspace(0, 14.5, 1 << 20)
    t, r = 1 / (1 + np.float64(p) * x), np.zeros_like(x)
    for k in c:
        r = r * t + np.float64(k)
    assert np.abs(r / (0.5 * erfcx(x / np.sqrt(2))) - 1).max() < 2 * U


def test_the_whole_in_float32(constants):
    """The kernel's steps, each rounded to float32, the reciprocal and exp2 a step (2 U) high or low: what the comment
    says, (1.5 g^2 + 16) U of the value below 0 and 10 U of 1 above."""
    p, c = constants
    f, w = np.float32, np.float64
    g = -np.linspace(0, 13.0, 1 << 18).astype(f)
    for lean in (-2 * U, 0.0, 2 * U):
        t = (1 / w(f(w(p) * -w(g) + 1)) * (1 + lean)).astype(f)
        e = (np.exp2(w(f(w(f(w(g) * w(g))) * w(f(-0.72134752044448170))))) * (1 + lean)).astype(f)
        r = np.full_like(t, c[0])
        for k in c[1:]:
            r = (w(r) * w(t) + w(k)).astype(f)
        r = (w(r) * w(e)).astype(f)
        want = 0.5 * erfcx(-w(g) / np.sqrt(2)) * np.exp(-w(g) * w(g) / 2)
        assert (np.abs(r - want) <= (1.5 * w(g) ** 2 + 16) * U * want).all()
        assert (np.abs((1 - w(r)).astype(f) - (1 - want)) <= 10 * U).all()

"""The fitted polynomial of the GELU derivative: its error, and that the kernels hold its coefficients."""
import os
import re

import numpy as np
import pytest

import tiled_dense_gemm_bias_amd as gba
from tiled_dense_gemm_bias_amd import gelu_slope_fit as fit


def test_error_of_the_fp32_form():
    special = pytest.importorskip("scipy.special")
    z = np.concatenate([np.linspace(-12, 12, 400001), np.linspace(-60, 60, 2001)]).astype(np.float32)
    x = z.astype(np.float64)
    want = special.ndtr(x) + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi)
    assert np.abs(fit.slope(z) - want).max() < 4.2e-6


def test_fit_reproduces_the_coefficients():
    pytest.importorskip("scipy.special")
    c, e = fit.fit()
    assert e < 4.0e-6
    x = np.linspace(0, 6, 2001)
    here, kept = (np.polynomial.polynomial.polyval(x, v) for v in (c, fit.COEFFS))
    assert np.abs((here - kept) * np.exp(-x * x / 2)).max() < 2e-7


def test_kernels_hold_the_coefficients():
    src = open(os.path.join(os.path.dirname(gba.__file__), "csrc", "experts", "gx_common.hpp")).read()
    found = [float(v) for v in re.findall(r"(-?\d+\.\d{10,})f", src)]
    for v in fit.COEFFS:
        assert any(np.float32(v) == np.float32(f) for f in found), v


def test_limits():
    with np.errstate(over="ignore", invalid="ignore"):
        s = fit.slope(np.array([np.inf, -np.inf, np.nan, 1e30, -1e30, 0.0], np.float32))
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2]) and s[3] == 1 and s[4] == 0 and abs(s[5] - 0.5) < 5e-6

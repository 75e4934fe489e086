"""The packed attention's exp2 on the FMA pipe: its coefficients are the committed fit's of degree 4,
and an emulation of the kernel's float32 steps stays within the error that its comment states over the
weights it takes: up to 2^8, where the running maximum lags, and 2^7 of that more in f16."""
import importlib.util
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_video_diffusion_b200", "csrc")
SRC = open(os.path.join(CSRC, "dp_packed_tc.cu")).read()
C = [np.float32(re.search(rf"\bkC{i} = ([0-9.e+-]+)f", SRC).group(1)) for i in range(5)]
F32 = np.float32


def _fit():
    spec = importlib.util.spec_from_file_location("fit_exp2_poly", os.path.join(CSRC, "fit_exp2_poly.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod.float32_coeffs(4)


def _emulate(x):
    def fma(a, b, c):  # the float64 product of float32 values is exact
        return (a.astype(np.float64) * b + c).astype(F32)
    x = np.maximum(x.astype(F32), F32(-125.0))
    r = x + F32(12582912.0)
    f = fma(r - F32(12582912.0), -1.0, x)
    q = np.full_like(x, C[4])
    for c in C[3::-1]:
        q = fma(q, f.astype(np.float64), np.float64(c))
    return _add_exponent(q, r)


def _add_exponent(q, r):
    bits = (q.view(np.int32).astype(np.int64) + (r.view(np.int32).astype(np.int64) << 23)) & 0xFFFFFFFF
    return bits.astype(np.uint32).view(F32)


def test_coefficients_are_the_fit():
    c32, _, err32 = _fit()
    assert [float(v) for v in c32] == [float(v) for v in C]
    assert err32 <= 2.7e-6


def test_emulated_exp2_within_the_stated_error():
    """2.7e-6 and the roundings of the last two steps, 2^-24 each of at most sqrt(2) of the result,
    and of the four products before, which weigh less than one of them together."""
    x = np.concatenate([np.linspace(-125.0, 15.0, 2_000_001, dtype=F32), np.arange(-125, 16, dtype=F32),
                        np.arange(-125, 15, dtype=F32) + F32(0.5)])
    rel = np.abs(_emulate(x).astype(np.float64) / np.exp2(x.astype(np.float64)) - 1.0)
    assert float(rel.max()) <= 2.7e-6 + 3 * 2.0 ** -24 * np.sqrt(2.0)


def test_far_scores_and_nan():
    got = _emulate(np.array([-np.inf, -1e30, -126.0], dtype=F32))
    assert np.all(got <= 2.0 ** -124) and np.all(got >= 0)
    # the arithmetic's NaN, 0x7fffffff, comes out above kLost, which no row sum reaches:
    # 2^31 keys of at most 2^15
    nan = np.array([0x7FFFFFFF], dtype=np.uint32).view(F32)
    lost = float(re.search(r"kLost = ([0-9.e+]+)f", SRC).group(1))
    assert _add_exponent(nan, nan)[0] > lost > 2.0 ** 46

"""The weight call's exponential on the FMA pipe (add_exp2_poly2 in csrc/f32x2.cuh), emulated in float32
on the CPU against float64 2^x, with the coefficients read from the source: they are the committed fit
(kv_shared_b200/exp2_poly_fit.py) and the prefill kernels' own, and the stated relative error of 2.1e-7
holds over the whole range of exponents; beyond it the result is 0 or infinite, and a NaN stays one."""
import os
import re

import numpy as np
import test_exp2_poly as prefill                                 # puts the fit on the path
import exp2_poly_fit as fit  # noqa: E402

BOUND = 2.11e-7 + 2.0 ** -24          # the polynomial's, and the rounding of the sum


def _source():
    src = open(os.path.join(prefill.ROOT, "kv_shared_b200", "csrc", "f32x2.cuh")).read()
    body = src[src.index("exp2_poly2("):]
    return body[:body.index("\n}")]


def _coefficients():
    vals = [float(v) for v in re.findall(r"make_float2\(([-0-9.e]+)f, \1f\)", _source())]
    assert len(vals) == 6, vals
    return np.array(vals[::-1], dtype=np.float32)


def _clamp():
    (lo, hi), = set(re.findall(r"clamp_nan\(x\.[xy], ([-0-9.]+)f, ([0-9.]+)f\)", _source()))
    return np.float32(lo), np.float32(hi)


def _add_exp2(x, total=0.0):
    lo, hi = _clamp()
    x = np.minimum(np.maximum(np.asarray(x, np.float32), lo), hi)                # both keep a NaN
    magic = np.float32(12582912.0)
    t = x + magic
    j = t - magic
    p = fit.horner32(_coefficients(), x - j)
    s = (((t.view(np.uint32).astype(np.int64) << 23) + 0x3f800000) & 0xFFFFFFFF).astype(np.uint32).view(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        return (p.astype(np.float64) * s.astype(np.float64) + total).astype(np.float32)


def test_coefficients_are_the_committed_fit_and_the_prefill_kernels():
    assert np.array_equal(_coefficients(), prefill._kernel_coefficients())
    assert np.all(np.abs(_coefficients() / fit.lawson_fit().astype(np.float32) - 1.0) < 1e-6)


def test_relative_error_over_the_exponents():
    x = np.concatenate([np.linspace(-126.0, 127.49, 400001), np.arange(-126, 128), np.arange(-125, 127) + 0.5]).astype(np.float32)
    want = np.exp2(x.astype(np.float64))
    got = _add_exp2(x).astype(np.float64)
    # 2^-126.5 .. 2^-126 is below fp32's normal numbers: half of their spacing, 2^-150
    assert np.all(np.abs(got - want) <= BOUND * want + 2.0 ** -150)
    assert np.all(np.abs(_add_exp2(x[x < 20], 1.0) - (1 + want[x < 20])) <= BOUND * (1 + want[x < 20]))


def test_ends_of_the_range_and_nan():
    low = np.array([-126.51, -127, -128, -200, -1e30, -np.inf], np.float32)
    high = np.array([127.5, 128, 130, 255, 256, 384, 512, 1e30, np.inf], np.float32)
    assert np.array_equal(_add_exp2(low), np.zeros(len(low), np.float32))
    assert np.array_equal(_add_exp2(high), np.full(len(high), np.inf, np.float32))
    assert np.isnan(_add_exp2(np.array([np.nan], np.float32))).all()

"""The packed-prompt attention's FMA-pipe exponential (csrc/prompt.cu, exp2_pair), emulated in fp32 on the CPU: its
constants are the ones csrc/exp2_pair_fit.py derives, its relative error stays below 2.9e-6, and the ends of its range
behave: exactly 0 at and below -127, exactly 1 at 0, powers of two at integers."""
import importlib.util
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_microscaled_quantization_b200", "csrc")


def _fit():
    spec = importlib.util.spec_from_file_location("exp2_pair_fit", os.path.join(CSRC, "exp2_pair_fit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _constants():
    src = open(os.path.join(CSRC, "prompt.cu")).read()
    body = src[src.index("void exp2_pair("):]
    body = body[: body.index("v0 = __uint_as_float")]
    got = re.search(r'"f"\(1\.0f\), ((?:"f"\(0x1[^)]*\)(?:, )?)+)', body).group(1)
    return np.array([1.0] + [float.fromhex(h) for h in re.findall(r"(0x1\.[0-9a-f]+p[+-]\d+)f", got)], dtype=np.float32)


def _exp2(w):
    c = _constants()
    w = np.maximum(np.asarray(w, dtype=np.float32), np.float32(-127))
    magic = np.float32(12582912.0)
    t = (w + magic).astype(np.float32)
    f = (w - (t - magic)).astype(np.float32)
    p = np.full_like(f, c[-1])
    for k in c[-2::-1]:
        p = (p.astype(np.float64) * f + k).astype(np.float32)  # a fused multiply-add: one rounding
    with np.errstate(over="ignore"):
        bits = p.view(np.uint32) + (t.view(np.uint32) << np.uint32(23))
    return bits.view(np.float32)


def test_kernel_uses_the_derived_coefficients():
    assert np.allclose(_constants(), _fit().coefficients(), rtol=0, atol=2.0 ** -24)


def test_relative_error():
    w = np.random.default_rng(0).uniform(-125.5, 8, 400000).astype(np.float32)
    assert np.max(np.abs(_exp2(w).astype(np.float64) / 2.0 ** w.astype(np.float64) - 1)) < 2.95e-6


def test_ends_of_the_range():
    assert (_exp2(np.array([-127.0, -128.0, -1e30, -np.inf], dtype=np.float32)) == 0).all()
    w = np.arange(-126, 9, dtype=np.float32)
    np.testing.assert_array_equal(_exp2(w), 2.0 ** w.astype(np.float64))
    low = _exp2(np.linspace(-127, -126, 5001).astype(np.float32))
    assert (low >= 0).all() and low.max() <= 2.0 ** -126 * (1 + 3e-6)

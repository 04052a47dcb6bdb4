"""The polynomial of the epilogue's GELU against erfc in 64 bits (CPU): the
errors that the source states are those of the coefficients it holds."""
import os
import re

import numpy as np
import pytest

special = pytest.importorskip("scipy.special")

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "int4_weight_mixed_gb300", "csrc", "w4_epilogue.cuh")


def _source():
    text = open(SOURCE).read()
    body = text[text.index("float ep_gelu(float v)"):]
    body = body[:body.index("return")]
    coefs = [re.search(r"float p = (\S+)f;", body).group(1)] + re.findall(
        r"p = fmaf\(p, t, (\S+)f\);", body)
    comment = text[text.index("// GELU, v * (1 + erf"):text.index("float ep_gelu(float v)")]
    comment = " ".join(line.lstrip("/ ") for line in comment.splitlines())
    return np.array([float(c) for c in coefs]).astype(np.float32), comment


def test_the_polynomial_is_as_exact_as_stated():
    coefs, comment = _source()
    assert len(coefs) == 9
    stated = float(re.search(r"relative error (\S+) \* 2\^-24", comment).group(1))
    z = np.concatenate([np.linspace(0, 14, 400001), np.linspace(11, 12.5, 100001)])
    t = 1 / (1 + z / 2)
    p = np.polyval(coefs.astype(np.float64), t)
    worst = np.abs(p / (special.erfcx(z) / (2 * t)) - 1).max() * 2**24
    assert 0.9 * stated <= worst <= stated, worst


def test_gelu_in_fp32_is_within_its_bound():
    """Every step in fp32 (the exponential correctly rounded): within
    (2 v^2 + 12) 2^-24 of GELU wherever that is a normal number."""
    coefs, comment = _source()
    assert "(2 v^2 + 12) 2^-24" in comment
    f = np.float32
    v = np.concatenate([np.linspace(-13, 13, 400001), -np.logspace(-30, 1.1, 50001),
                        np.logspace(-30, 1.9, 50001)]).astype(f)
    a = np.abs(v)
    t = f(1) / (f(0.35355339) * a + f(1))
    p = np.full_like(v, coefs[0])
    for c in coefs[1:]:
        p = (p.astype(np.float64) * t + c).astype(f)  # one rounding, as fmaf
    e = np.exp2((v * v * f(-0.72134752)).astype(np.float64)).astype(f)
    got = np.maximum(v, f(0)) - a * t * p * e
    ref = v.astype(np.float64) * special.ndtr(v.astype(np.float64))
    ok = np.abs(ref) > 2.0**-120
    err = np.abs(got - ref)[ok] / np.abs(ref)[ok]
    bound = (2 * v[ok].astype(np.float64)**2 + 12) * 2.0**-24
    assert (err <= bound).all(), (err / bound).max()

"""The tanh approximations of capped scores, read out of the kernels' source: how far their
polynomials are from tanh, and with the rounding of their fp32 steps for some caps."""
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_cache_215_gb300", "csrc", "score.cuh")
f32 = np.float32


def numbers(text):
    return [float.fromhex(x) for x in re.findall(r"-?0x1\.[0-9a-f]+p-?\d+", text)]


def source(name):
    """The text of a function of the file."""
    text = open(SOURCE).read()
    at = text.index(name + "(")
    return text[at:text.index("\n}\n", at)]


def polynomials():
    """(name, coefficients of z, z^2, ... in x (1 + z (...)), range, bound, bound unrounded)."""
    chunk = re.findall(r"const float c\[\d\] = \{([^}]*)\}", source("cap_scores"))
    fine = re.findall(r"const float c\[\d\] = \{([^}]*)\}", source("cap_scores_fine"))
    assert len(chunk) == 3 and len(fine) == 1
    return [(f"chunk {i}", numbers(c), top, 2.0 ** -20.2, 2.0 ** -20.5)
            for i, (c, top) in enumerate(zip(chunk, (0.25, 0.5, 1.0)))] + \
        [("decode", numbers(fine[0]), 1.0, 2.0 ** -22.3, 2.0 ** -23.5)]


def fma(a, b, c):
    # (the product of two fp32 numbers is exact in fp64)
    return f32(a.astype(np.float64) * np.float64(b) + c)


@pytest.mark.parametrize("name,c,top,bound,unrounded", polynomials(), ids=lambda x: x if isinstance(x, str) else "")
def test_odd_polynomials(name, c, top, bound, unrounded):
    x = np.unique(np.concatenate([np.linspace(1e-4, top, 400001), np.exp(np.linspace(-12, np.log(top), 100001))])
                  .astype(f32))
    z = x.astype(np.float64) ** 2
    p = np.zeros_like(z)
    for k in reversed(c):
        p = (p + k) * z
    t = np.tanh(x.astype(np.float64))
    assert np.max(np.abs(x * (1 + p) - t) / t) <= unrounded
    for cap in (1.0, 30.0, 50.0, 43.28085, 72.13475):
        out, zz = f32(cap), x * x
        p = np.full_like(x, f32(c[-1]) * out)
        for k in reversed(c[:-1]):
            p = fma(p, zz, np.float64(f32(f32(k) * out)))
        y = x * fma(p, zz, np.float64(out))
        want = np.float64(out) * t
        assert np.max(np.abs(y.astype(np.float64) - want) / want) <= bound, cap


def test_tanh_score_below_its_break():
    c = numbers(source("tanh_score"))
    assert len(c) == 5 and "fabsf(x) < 0.6f" in source("tanh_score")
    x = np.linspace(1e-4, 0.6, 600001).astype(f32)
    z = x.astype(np.float64) ** 2
    p = np.zeros_like(z)
    for k in c:                                            # the highest first
        p = p * z + k
    t = np.tanh(x.astype(np.float64))
    assert np.max(np.abs(x + x * z * p - t) / t) <= 2.0 ** -27.6
    zz = x * x
    p = np.full_like(x, f32(c[0]))
    for k in c[1:]:
        p = fma(p, zz, np.float64(f32(k)))
    y = fma(x * zz, p, x.astype(np.float64))
    assert np.max(np.abs(y.astype(np.float64) - t) / t) <= 2.0 ** -23.6

"""The packed attention's polynomials (2^x and tanh on the FMA pipes): the coefficients and the
errors stated beside them are read from the source, and the kernel's fp32 steps replayed over
the whole range. A stated error holds and is not far above the largest one met."""
import os
import re

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "video_diffusion_transformer_wan_b200", "csrc", "packed_tc.cuh")
TEXT = open(SRC).read()


def _body(name):
    return re.search(name + r"\(unsigned long long \w+\) \{(.*?)\n\}", TEXT, re.S).group(1)


def _horner(name):
    """Coefficients of the chain of multiply-adds, the highest power first."""
    out = []
    for x in re.findall(r"[qp] = f2_fma\(([^;]*)\);", _body(name)):
        out += [float(v) for v in re.findall(r"f2_splat\(([-0-9.e]+)f\)", x)]
    return [np.float32(v) for v in out]


def _fma(a, b, c):
    return np.float32(np.float64(a) * np.float64(b) + np.float64(c))  # a product of two fp32 is exact in fp64


def _exp2(x):
    x = np.maximum(np.float32(x), np.float32(-125.0))
    t = np.float32(x + np.float32(12582912.0))
    f = _fma(t - np.float32(12582912.0), np.float32(-1.0), x)
    c = _horner("exp2_poly2")
    q = np.full_like(f, c[0])
    for k in c[1:]:
        q = _fma(q, f, k)
    return np.float64(q) * np.exp2(np.float64(t) - 12582912.0)


def _tanh(y):
    y = np.float32(y)
    z = np.float32(y * y)
    c = _horner("tanh_poly2")
    p = np.full_like(z, c[0])
    for k in c[1:]:
        p = _fma(p, z, k)
    return np.float64(np.float32(p * y))


def _stated(what, before):
    comment = re.sub(r"\n//", "", TEXT[:TEXT.index("unsigned long long " + before + "(")])
    return float(re.findall(what + r" (\d\.\de-\d+)", comment)[-1])


def _holds(worst, stated):
    assert worst <= stated <= 1.15 * worst, (worst, stated)


def test_exp2():
    assert len(_horner("exp2_poly2")) == 6
    x = np.concatenate([np.linspace(-0.5, 0.5, 400001), np.linspace(-125.0, 9.0, 1000003)]).astype(np.float32)
    _holds(np.max(np.abs(_exp2(x) / np.exp2(np.float64(x)) - 1)), _stated("fp32 steps:", "exp2_poly2"))
    assert np.all(_exp2(np.array([-1e30, -200.0], dtype=np.float32)) < 2.0 ** -124)  # clamped: all but nothing


def test_tanh():
    assert len(_horner("tanh_poly2")) == 5
    y = np.linspace(-0.5, 0.5, 1000002).astype(np.float32)
    t = np.tanh(np.float64(y))
    _holds(np.max(np.abs(_tanh(y) / t - 1)), _stated("relative error", "tanh_poly2"))
    _holds(np.max(np.abs(_tanh(y) - t)), _stated("absolute", "tanh_poly2"))


@pytest.mark.parametrize("name", ["exp2_poly2", "tanh_poly2"])
def test_coefficients_are_fp32(name):
    for m in re.findall(r"f2_splat\(([-0-9.e]+)f\)", _body(name)):
        assert float(np.float32(float(m))) == pytest.approx(float(m), rel=1e-8)

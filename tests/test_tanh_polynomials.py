"""The two polynomials behind capped scores, their coefficients read from the sources,
against tanh: the bounds stated beside them."""
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_15_gb300", "csrc")
NUMBER = r"-?\d+\.\d+(?:e-?\d+)?"


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_the_prompt_kernels_polynomial():
    text = source("attend_abi.cu").split("static const double c[5] = {", 1)[1].split("}", 1)[0]
    c = [float(x) for x in re.findall(NUMBER, text)]
    assert len(c) == 5
    y = np.linspace(1e-6, 0.6, 1_000_001)
    p = sum(ci * (y * y) ** i for i, ci in enumerate(c))
    assert np.abs(p - np.tanh(y) / y).max() <= 7.5e-8
    assert np.abs(y * p - np.tanh(y)).max() <= 3.9e-8


def test_the_series_near_zero():
    body = source("attend.cuh").split("float capped(", 1)[1].split("\n}", 1)[0]
    half, = [float(x) for x in re.findall(r"qk \* cap_in, y = x \* (" + NUMBER + ")f", body)]
    c = [float(x) for x in re.findall(r"(" + NUMBER + ")f", body.split("const float near", 1)[1].split("1.f)", 1)[0])]
    assert len(c) == 3 and abs(half - np.log(2) / 2) < 1e-8 and "fabsf(x) < 0.5f ? near : far" in body
    y = np.linspace(1e-6, 0.5 * half, 1_000_001)
    z = y * y
    near = y * (z * (z * (z * c[0] + c[1]) + c[2]) + 1)   # innermost first
    assert y[-1] < 0.174 and np.abs(near / np.tanh(y) - 1).max() <= 1.8e-8

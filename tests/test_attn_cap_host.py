"""The cap of attention scores, built for the host (tests/attn_cap_host.cpp), against 64 bits.

Errors in u = 2^-24 of the result t = tanh y, for |y| = a from 0.8 on: y has 2 roundings, the exponent 2 more, so e^2a is off by
8 a u and the exponential's own 4 u; the sum rounds once and the reciprocal is off by 2 u, so 2 / (1 + e^2a) = 1 - t by
((1 + t) / 2 (8 a + 4) + 3) u of itself; the difference and `top` round once each:
    (1 - t) / t ((1 + t) / 2 (8 a + 4) + 3) + 2 <= 7.9, the largest at a = 0.8.
Below it the polynomial and its evaluation have 2.3 (2^-22.8), y 2, `top` and the product with it 2: 6.3.  So 8 u, 2^-21.
The form without `exact` at any y: twice the reciprocal, 1 - t of either sign, off by that bracket, beside the difference's and
top's roundings: (1 - t) ((1 + t) / 2 (8 |y| + 4) + 3) + 2 |t| <= 9.4 u of the cap, the largest at y = -1: below 2^-20.
"""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "quantized_weight_mat_gb300", "csrc")
LOG2E = 1.4426950408889634
CAPS = [2.0 ** -60, 1e-9, 0.3, 1.0, 30.0, 50.0, 128.0, 1000.0, 1e6, 2.0 ** 60]


@pytest.fixture(scope="module")
def cap(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    so = str(tmp_path_factory.mktemp("caphost") / "attn_cap_host.so")
    subprocess.run(["g++", "-O2", "-ffp-contract=off", "-std=c++17", "-fPIC", "-shared", "-I", CSRC, "-o", so,
                    os.path.join(HERE, "attn_cap_host.cpp")], check=True)
    lib = ctypes.CDLL(so)

    def run(exact, cap, e, r, x):
        x, out = np.ascontiguousarray(x, np.float32), np.empty(len(x), np.float32)
        lib.cap_host(int(exact), ctypes.c_float(cap), e, r, len(x), x.ctypes.data_as(ctypes.c_void_p), out.ctypes.data_as(ctypes.c_void_p))
        return out
    return run


def scores(cap):
    """Scores times log2 e, of both signs: some 40000 up to 12 caps, and some down to 2^-40 caps."""
    y = np.concatenate([np.linspace(0, 2.0, 30001), np.linspace(2.0, 12.0, 8001), 2.0 ** np.linspace(-40, 0, 2001)])
    return (np.concatenate([y, -y]) * float(np.float32(cap)) * LOG2E).astype(np.float32)


def want(cap, x):
    top = float(np.float32(cap)) * LOG2E
    return top * np.tanh(x.astype(np.float64) / top)


@pytest.mark.parametrize("c", CAPS)
@pytest.mark.parametrize("e", [-1, 0, 1])
@pytest.mark.parametrize("r", [-1, 0, 1])
def test_relative_error(cap, c, e, r):
    x = scores(c)
    ref = want(c, x)
    err = np.abs(cap(True, c, e, r, x) - ref)
    assert (err <= 2.0 ** -21 * np.abs(ref)).all(), (err[ref != 0] / np.abs(ref[ref != 0])).max() * 2 ** 21


@pytest.mark.parametrize("c", [x for x in CAPS if x <= 256])
@pytest.mark.parametrize("e", [-1, 0, 1])
@pytest.mark.parametrize("r", [-1, 0, 1])
def test_error_in_caps(cap, c, e, r):
    x = scores(c)
    assert (np.abs(cap(False, c, e, r, x) - want(c, x)) <= 2.0 ** -20 * c * LOG2E).all()


@pytest.mark.parametrize("c", CAPS)
def test_it_is_odd(cap, c):
    x = scores(c)
    assert np.array_equal(cap(True, c, 0, 0, x), -cap(True, c, 0, 0, -x))


def test_ends(cap):
    x = np.array([np.inf, -np.inf, 3e38, -3e38, np.nan, 0.0], np.float32)
    top = np.float32(50 * LOG2E)
    for exact in (True, False):
        got = cap(exact, 50.0, 0, 0, x)
        assert np.array_equal(got[:4], [top, -top, top, -top]) and np.isnan(got[4]) and abs(got[5]) <= 1e-5

"""Rotary angles of far positions, against exact arithmetic: positions times frequencies as whole numbers,
reduced by 1 / (2 pi) to 256 bits."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import paged_kv_decode_gqa_b200 as pkv
from _gpu_helpers import dev, host
from _int8_reference import HALF

F16, F32, F64 = np.float16, np.float32, np.float64
D = 128
getcontext().prec = 90
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
BITS = 256
INV_TWO_PI = int(Decimal(2) ** BITS / TWO_PI)
# The angle's fp32 rounding (2^-26 of a turn) moves a sine by 0.71 x 2^-23.3 near pi / 4, the fp32 sine and cosine
# are within an ulp, 2^-24, a product is rounded once (2^-25) and their sum once: below 2^-22 of |x| + |y|.
ANGLE = 2.0 ** -22


def turns(pos, freq):
    """The fraction of a turn, in [-1/2, 1/2), of pos * freq (an int and a float32), to 2^-60 or better."""
    m, e = np.frexp(F64(freq))
    scaled = int(pos) * int(m * 2 ** 24) * INV_TWO_PI              # x 2^(e - 24 - BITS)
    one = 1 << (BITS + 24 - int(e))
    frac = scaled % one
    return float(Decimal(frac - one if 2 * frac >= one else frac) / Decimal(one))


def freqs():
    return (1e4 ** (-np.arange(64, dtype=F64) / 64)).astype(F32)


def positions(bits, count, seed):
    """Positions below 2^bits at which some pair's cosine and sine nearly cancel (as many for each of the fastest
    frequencies), and that pair's number."""
    rng = np.random.default_rng(seed)
    f, out = freqs(), []
    for j in (0, 1, 5, 11):
        found = 0
        while found < count:
            pos = int(rng.integers(1 << (bits - 1), 1 << bits)) * int(rng.choice([-1, 1]))
            if abs(abs(turns(pos, f[j])) - 0.125) < 2e-4:
                out.append((pos, j))
                found += 1
    return out


def test_the_exact_reduction_agrees_with_long_double_on_near_positions():
    f = freqs()
    for pos in (0, 1, 7, -3, 12345, 99999):
        for j in (0, 3, 40):
            a = np.longdouble(pos) * np.longdouble(f[j])
            t = turns(pos, f[j]) * 2 * np.pi
            assert abs(float(np.cos(a)) - np.cos(t)) < 1e-13 and abs(float(np.sin(a)) - np.sin(t)) < 1e-13


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [20, 31, 32, 40, 53])
def test_angles_keep_fp32_accuracy(bits):
    """x cos a - x sin a (or +, where the sine is negative) near pi / 4, where the f16 result is small and shows
    the angle's own error."""
    pkv.pkv_device_error()
    f, cases = freqs(), positions(bits, 6, bits)
    T = len(cases)
    q = np.zeros((T, 1, D), F16)
    want, size = np.zeros((T, 2)), np.zeros((T, 2))
    for t, (pos, j) in enumerate(cases):
        a = 2 * np.pi * turns(pos, f[j])
        x, y = 3.0, 3.0 * np.sign(np.cos(a) * np.sin(a))
        q[t, 0, j], q[t, 0, j + 64] = x, y
        want[t] = x * np.cos(a) - y * np.sin(a), y * np.cos(a) + x * np.sin(a)
        size[t] = abs(x) + abs(y)
    qd, k = dev(q), torch.zeros((T, 1, D), dtype=torch.float16, device="cuda")
    kc, vc = (torch.zeros((T // 16 + 1, 16, 1, D), dtype=torch.float16, device="cuda") for _ in range(2))
    out = torch.empty_like(qd)
    pkv.paged_kv_rope_cache_write(out, qd, k, k, kc, vc, dev(np.arange(T, dtype=np.int64)),
                                  dev(np.array([p for p, _ in cases], np.int64)), dev(f))
    got = host(out).astype(F64)
    for t, (pos, j) in enumerate(cases):
        err = np.abs(got[t, 0, [j, j + 64]] - want[t])
        assert (err <= HALF * np.abs(want[t]) + ANGLE * size[t] + 2.0 ** -25).all(), (pos, j, err)
    assert pkv.pkv_device_error() == 0

"""The rotation's reduction of angles (gdn_qk_norm_*, include/gdn_layer.h) against exact
arithmetic, without a GPU: what the kernel does in whole numbers, with its constants."""
import os
import random
import re
import struct
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "chunked_linear_recurrence_gated_gb300", "csrc", "gdn_qk_norm.cu")
ONE = 1 << 400
LOW = (1 << 64) - 1


def atan_of_inverse(n):
    term = total = ONE // n
    k, sign = 3, -1
    while term:
        term //= n * n
        total += sign * (term // k)
        k, sign = k + 2, -sign
    return total


PI = 4 * (4 * atan_of_inverse(5) - atan_of_inverse(239))  # Machin's formula, times ONE


def turns(f, pos):
    """pos f / (2 pi), exact to 2^-300."""
    return Fraction(f) * pos * Fraction(ONE, 2 * PI)


def kernel_constants():
    with open(SOURCE) as s:
        body = s.read().split("turn_step(double f) {")[1].split("return")[0]
    return [int(x, 16) for x in re.findall(r"0x([0-9A-Fa-f]{16})ull", body)]


def turn_step(f):
    c, rest = kernel_constants()
    u = struct.unpack("<Q", struct.pack("<d", f))[0]
    ex = u >> 52 & 0x7FF
    m = u & 0xFFFFFFFFFFFFF | (1 << 52 if ex else 0)
    product = m * c + (m * rest >> 64)
    r = product >> (1077 - max(ex, 1)) & LOW
    return -r & LOW if u >> 63 else r


def test_constants_are_the_digits_of_two_over_pi():
    digits = 2 * ONE * ONE // PI
    assert kernel_constants() == [digits >> 336, digits >> 272 & LOW]


def test_step_and_angle():
    r = random.Random(1)
    fs = [1.0, 1e4, 100.25, 1e-9, 5e-324, 2.0 ** 39, 2.0 ** 40 * (1 - 2.0 ** -53)]
    fs += [2.0 ** r.uniform(-60, 40) for _ in range(300)]
    for f in fs + [-f for f in fs]:
        step = turn_step(f)
        off = (Fraction(step) - turns(f, 1) * (1 << 64)) % (1 << 64)
        assert min(off, (1 << 64) - off) < 1, f
        for pos in (1, 2 ** 31 - 1, -2 ** 31, r.randrange(-2 ** 31, 2 ** 31)):
            kept = (step * pos & LOW) >> 32  # what the kernel rounds to fp32
            off = (Fraction(kept, 1 << 32) - turns(f, pos)) % 1
            assert min(off, 1 - off) < 2.0 ** -31, (f, pos)


@pytest.mark.parametrize("f", [0.0, -0.0])
def test_no_frequency(f):
    assert turn_step(f) == 0

"""The quantiser's division (fp4_quant.cuh) next to the boundaries that it decides, on the CPU.

x / d is computed as q = fl(x r), r = fl(1 / d), and one correction fl(q + fl(x - q d) r).  Restated in C with
correctly rounded operations, it has to lie on the same side of a boundary as the IEEE quotient fl(x / d)
(below, on, above), for every significand of the divisor, at the ends of the range of the matrix scale
(2^-100 to 2^117, block scales from 2^-9).  The limit below which the kernel scales x and g up, and by how
much, are read from its source.
"""
import ctypes
import os
import re
import subprocess

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_quantized_mx_b200",
                   "csrc", "fp4_quant.cuh")

C = r"""
#include <math.h>
#include <stdint.h>
#include <string.h>
static float bits(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
static uint32_t word(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
static int side(float y, float t) { return (y > t) - (y < t); }
/* decisions that differ, over the divisors bits(first), bits(first + step), .. (n of them), each times up */
int64_t differ(uint32_t first, uint32_t step, int64_t n, float up, const float* t, int nt) {
    int64_t bad = 0;
    for (int64_t i = 0; i < n; ++i) {
        const float d = bits(first + (uint32_t)i * step), ds = d * up, r = 1.0f / ds;
        for (int b = 0; b < nt; ++b) {
            const float at = t[b] * d;
            for (int o = -2; o <= 2; ++o) {
                const float x = bits(word(at) + (uint32_t)o), xs = x * up;
                if (!(x < INFINITY)) continue;
                const float q = xs * r;
                bad += side(fmaf(fmaf(-q, ds, xs), r, q), t[b]) != side(x / d, t[b]);
            }
        }
    }
    return bad;
}
"""
E2M1 = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
# between neighbours of E4M3: the subnormal ones, a normal binade (the others are powers of two times it), the last
E4M3 = tuple((2 * i + 1) * 2.0 ** -10 for i in range(8)) + tuple(1 + (2 * i + 1) / 16 for i in range(8)) + (432.0,)


@pytest.fixture(scope="module")
def differ(tmp_path_factory):
    d = tmp_path_factory.mktemp("division")
    (d / "div.c").write_text(C)
    subprocess.run(["gcc", "-O3", "-march=native", "-ffp-contract=off", "-fno-fast-math", "-shared", "-fPIC", "-o",
                    str(d / "div.so"), str(d / "div.c"), "-lm"], check=True)
    f = ctypes.CDLL(str(d / "div.so")).differ
    f.restype = ctypes.c_int64
    f.argtypes = [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_int64, ctypes.c_float, ctypes.POINTER(ctypes.c_float),
                  ctypes.c_int]

    def run(exponent, up, bounds, step=1):
        n = -(-(1 << 23) // step)
        return f((exponent + 127) << 23, step, n, up, (ctypes.c_float * len(bounds))(*bounds), len(bounds))
    return run


def constants():
    text = open(SRC).read()
    low, up = re.search(r"kSmallScale = 0x1p(-\d+)f, kSmallUp = 0x1p(\d+)f;", text).groups()
    return int(low), int(up)


def test_every_significand_at_the_smallest_scales(differ):
    """g in [2^-100, 2^-99) scaled up, and g from the limit on as it is; s = 2^-9, the smallest"""
    low, up = constants()
    assert differ(-109, 2.0 ** up, E2M1) == 0
    assert differ(low - 9, 1.0, E2M1) == 0


@pytest.mark.parametrize("below", range(1, 10))
def test_the_binades_between(differ, below):
    """the largest g that is still scaled up, and so on down; odd steps visit all kinds of significands"""
    low, up = constants()
    assert differ(low - 9 - below, 2.0 ** up, E2M1, 61) == 0


@pytest.mark.parametrize("exponent", [-80, 0, 100, 124, 125])
def test_larger_scales(differ, exponent):
    assert differ(exponent, 1.0, E2M1, 31) == 0


def test_block_scales(differ):
    """a / (6 g): 6 g in [2^-98, 2^-97) scaled up, in the binades around the limit, and up to the largest"""
    low, up = constants()
    assert differ(-98, 2.0 ** up, E4M3) == 0
    for exponent in (low + 2, low + 3, 0, 119):
        assert differ(exponent, 1.0, E4M3, 31) == 0


def test_small_scales_as_they_are_are_caught(differ):
    """the negative control: without scaling, x - q d needs bits below 2^-149"""
    assert differ(-109, 1.0, E2M1[:1]) > 0
    assert differ(-102, 1.0, E2M1[:1]) > 0

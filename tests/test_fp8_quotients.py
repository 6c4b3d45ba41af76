"""The two divisions that the e4m3 codes are made without, restated in C (FP32, fused multiply-adds) and compared with the
IEEE quotient:

  max|v| / 448    from the rounded reciprocal and one correction by its remainder, for every significand
  v / s           from one reciprocal of s and one correction.  Before its last rounding it is within 2^-46 of v / s, so it can
                  differ from the IEEE quotient only where v / s is within 2^-22 of an ulp of the middle of two FP32
                  numbers, and a code only where that middle lies beside a border between two codes, a number of five
                  significant bits.  With significands V, S in [2^23, 2^24) that takes an S within 4 of a multiple of 2^20:
                  every V is tried for those (within 16), and for every S the V beside each border.
"""
import ctypes as C
import subprocess

import pytest

SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <string.h>

static inline float scale_of(float a) {
    const float c = 1.0f / 448.0f, q = a * c;
    return __builtin_fmaf(__builtin_fmaf(-448.0f, q, a), c, q);
}
static inline uint32_t bits(float f) {
    uint32_t u;
    memcpy(&u, &f, 4);
    return u;
}
/* the kernel's steps: those of -v / s, and then the sign bit turned */
static inline float quotient(float v, float s, float y) {
    const float n = v * -y;
    const uint32_t u = bits(__builtin_fmaf(__builtin_fmaf(s, n, v), -y, n)) ^ 0x80000000u;
    float q;
    memcpy(&q, &u, 4);
    return q;
}

int64_t wrong_scales(int exponent) {
    int64_t bad = 0;
#pragma omp parallel for reduction(+ : bad)
    for (int32_t m = 1 << 23; m < 1 << 24; ++m) {
        const float a = ldexpf((float)m, exponent - 23);
        bad += scale_of(a) != a / 448.0f;
    }
    return bad;
}

/* every V for the S within `reach` of a multiple of 2^20 */
int64_t wrong_near_multiples(int reach) {
    int64_t bad = 0;
    for (int b = 8; b <= 16; ++b)
        for (int o = -reach; o <= reach; ++o) {
            const int32_t S = (b << 20) + o;
            if (S < 1 << 23 || S >= 1 << 24) continue;
            const float s = (float)S, y = 1.0f / s;
#pragma omp parallel for reduction(+ : bad)
            for (int32_t V = 1 << 23; V < 1 << 24; ++V) bad += quotient((float)V, s, y) != (float)V / s;
        }
    return bad;
}

/* every S, and the V beside S times each number of five significant bits */
int64_t wrong_beside_borders(void) {
    int64_t bad = 0;
#pragma omp parallel for reduction(+ : bad) schedule(dynamic, 4096)
    for (int32_t S = 1 << 23; S < 1 << 24; ++S) {
        const float s = (float)S, y = 1.0f / s;
        for (int B = 16; B < 32; ++B) {
            const int64_t p = (int64_t)S * B;             /* V = p / 16, of 24 or 25 bits */
            const int shift = p >= (int64_t)1 << 28 ? 5 : 4;
            const int32_t mid = (int32_t)((p + (1 << (shift - 1))) >> shift);
            for (int o = -3; o <= 3; ++o) {
                const float v = (float)(mid + o) * (float)(1 << (shift - 4));
                bad += quotient(v, s, y) != v / s;
            }
        }
    }
    return bad;
}

/* the same at the smallest scale that is not divided by, for the smallest values whose code is not 0, and zeros of
   either sign at both ends of the range */
int64_t wrong_at_the_ends(void) {
    int64_t bad = 0;
#pragma omp parallel for reduction(+ : bad)
    for (int32_t S = 1 << 23; S < 1 << 24; S += 5) {
        const float s = ldexpf((float)S, -103), y = 1.0f / s, t = ldexpf((float)S, 76), z = 1.0f / t;
        for (int e = 4; e <= 11; ++e)
            for (int B = 16; B < 32; ++B) {
                const float mid = ldexpf((float)((double)S * B / 16), -103 - e);
                for (int o = -2; o <= 2; ++o) {
                    const float v = o < 0 ? nextafterf(o < -1 ? nextafterf(mid, 0) : mid, 0)
                                          : o ? nextafterf(o > 1 ? nextafterf(mid, 1) : mid, 1) : mid;
                    bad += quotient(v, s, y) != v / s || bits(quotient(-v, s, y)) != bits(-v / s);
                }
            }
        bad += bits(quotient(-0.0f, s, y)) != 0x80000000u || bits(quotient(0.0f, s, y)) != 0;
        bad += bits(quotient(-0.0f, t, z)) != 0x80000000u || bits(quotient(0.0f, t, z)) != 0;
    }
    return bad;
}
"""


@pytest.fixture(scope="module")
def quotients(tmp_path_factory):
    at = tmp_path_factory.mktemp("quotients")
    (at / "q.c").write_text(SOURCE)
    subprocess.run(["gcc", "-O3", "-march=native", "-fopenmp", "-ffp-contract=off", "-fno-fast-math", "-std=gnu11", "-Wall",
                    "-shared", "-fPIC", "-o", str(at / "q.so"), str(at / "q.c"), "-lm"], check=True)
    lib = C.CDLL(str(at / "q.so"))
    for name in ("wrong_scales", "wrong_near_multiples", "wrong_beside_borders", "wrong_at_the_ends"):
        getattr(lib, name).restype = C.c_int64
    return lib


@pytest.mark.parametrize("exponent", [-100, 0, 127])  # values below 2^-100 and above 3e38 are divided
def test_every_scale(quotients, exponent):
    assert quotients.wrong_scales(exponent) == 0


def test_every_value_under_the_scales_near_a_multiple(quotients):
    assert quotients.wrong_near_multiples(16) == 0


def test_every_scale_beside_every_border(quotients):
    assert quotients.wrong_beside_borders() == 0


def test_the_ends_of_the_range_and_zeros(quotients):
    assert quotients.wrong_at_the_ends() == 0

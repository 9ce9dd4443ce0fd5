"""The norm divides without a division instruction: its scale max / Qmax by a
product with RN(1 / Qmax), its codes' quotient y / scale by one with 1 / scale after
a step of Newton's, each corrected by the exact remainder (Markstein's scheme).  The header
promises the correctly rounded quotients, so the scheme has to equal the IEEE
division wherever the kernel uses it: scales from 2^-80 up.

The same operations in C (gcc, no contraction, libm fmaf) against the IEEE
quotients: a prime stride through all maxima, and random pairs, also built to lie
next to a half step of either code."""
import os
import re
import subprocess
import tempfile

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_recurrent_state_decode_b200",
                   "csrc", "mixer", "qmixer_norm.cu")

C = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
static float u2f(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
static uint32_t f2u(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
static uint64_t s = 0x9e3779b97f4a7c15u;
static uint32_t rnd(void) { s ^= s << 13; s ^= s >> 7; s ^= s << 17; return (uint32_t)(s >> 32); }
static float divide(float y, float scale) {
    /* the hardware's reciprocal is within a unit of the rounded one: all three are tried */
    const float near = u2f(f2u(1.0f / scale) + rnd() % 3 - 1);
    const float inv = fmaf(fmaf(-scale, near, 1.0f), near, near), q = y * inv;
    return fmaf(fmaf(-scale, q, y), inv, q);
}
int main(void) {
    const float qmaxs[2] = {127.0f, 448.0f};
    long long bad = 0;
    for (int k = 0; k < 2; k++) {
        const float d = qmaxs[k], unit = 1.0f / d;
        for (uint64_t u = 0; u < 0x7f800000u; u += u < 0x01000000u || u > 0x7f000000u ? 1 : 37) {
            const float m = u2f((uint32_t)u), q = m * unit, got = fmaf(fmaf(-q, d, m), unit, q);
            if (!(got >= 0x1p-80f)) { bad += m / d >= 0x1.1p-80f; continue; }   /* divided by the instruction */
            bad += f2u(got) != f2u(m / d);
        }
    }
    printf("%lld\n", bad);
    bad = 0;
    for (int i = 0; i < 40000000; i++) {
        /* a scale from 2^-80 up whose maximum is finite, and a quotient up to 448 */
        const float scale = u2f((47u << 23) + rnd() % ((245u - 47u) << 23));
        float z = u2f((uint32_t)(127 + 9 - rnd() % 24) << 23 | (rnd() & 0x7fffff));
        if (z > 448.0f) z = 448.0f;
        if (i & 1) z = rintf(z) + 0.5f * (float)(rnd() & 1);                    /* next to a border */
        float y = z * scale;
        if (i & 2) y = u2f(f2u(y) + rnd() % 5 - 2);
        if (!(fabsf(y) >= 0x1p-126f) || !(y < INFINITY)) continue;
        const float q = y / scale;
        if (q < 0x1p-11f) continue;               /* no code of either type but zero */
        bad += f2u(divide(y, scale)) != f2u(q);
    }
    printf("%lld\n", bad);
    return 0;
}
"""


@pytest.fixture(scope="module")
def found():
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "c.c"), os.path.join(d, "c")
        with open(src, "w") as f:
            f.write(C)
        subprocess.run(["gcc", "-O2", "-std=c11", "-ffp-contract=off", "-mfma", src, "-o", exe, "-lm"], check=True)
        out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    return [int(v) for v in out]


def test_scales_are_the_rounded_quotients(found):
    assert found[0] == 0


def test_codes_are_of_the_rounded_quotient(found):
    assert found[1] == 0


def test_the_kernel_uses_this_scheme():
    code = open(SRC).read()
    assert re.search(r"fmaf\(fmaf\(-q, qmax, m\), unit, q\)", code)
    assert re.search(r"fma2\(fma2\(q, less, y\[i\]\), by, q\)", code)
    assert "odd = !(scale >= 0x1p-80f)" in code and "inv = fmaf(fmaf(-scale, near, 1.0f), near, near)" in code

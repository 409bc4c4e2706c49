"""The two-step quotient of the quantizing write (csrc/kv_cache.hip): x times the
correctly rounded inverse of s, and one step along the residual, against the
correctly rounded x / s.  In C on the CPU, with the same fused operations."""

import os
import subprocess
import tempfile

import pytest

SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>

static uint32_t state = 12345;
static uint32_t next(void) { return state = state * 1664525u + 1013904223u; }

int main(void)
{
    const int scales[4] = {0, -100, -20, 110}; /* the floor of a block's scale, ordinary ones, near the largest */
    long checked = 0, bad = 0;
    for (int k = 0; k < 4; ++k)
        for (int n = 0; n < 6000; ++n) {
            /* significands of s: the ends, powers of two beside them, then any */
            const uint32_t m = n < 23 ? 1u << n : n < 46 ? 0x7fffffu - (1u << (n - 23)) + 1 : n == 46 ? 0 : next() >> 9;
            const float s = ldexpf(1.0f + (float)m * 0x1p-23f, scales[k]), inverse = 1.0f / s;
            for (int e = -2; e <= 8; ++e)
                for (uint32_t x10 = 0; x10 < 1024; ++x10) { /* every 11-bit significand of x */
                    const float x = ldexpf(1.0f, e + scales[k]) * (1.0f + (float)x10 * 0x1p-10f);
                    const volatile float product = x * inverse; /* (rounded here) */
                    const float y = product, z = fmaf(fmaf(-y, s, x), inverse, y);
                    ++checked;
                    bad += z != x / s;
                }
        }
    printf("%ld %ld\n", checked, bad);
    return 0;
}
"""


def test_two_step_quotient_is_the_rounded_one():
    with tempfile.TemporaryDirectory() as tmp:
        source, program = os.path.join(tmp, "quotient.c"), os.path.join(tmp, "quotient")
        with open(source, "w") as f:
            f.write(SOURCE)
        built = subprocess.run(["gcc", "-O2", "-ffp-contract=off", source, "-o", program, "-lm"], capture_output=True, text=True)
        if built.returncode:
            pytest.skip("no C compiler: " + built.stderr[-200:])
        checked, bad = map(int, subprocess.run([program], capture_output=True, text=True, timeout=600, check=True).stdout.split())
    assert checked == 4 * 6000 * 11 * 1024 and bad == 0

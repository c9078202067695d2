"""The quotient of the fp32-scaled 8-bit rows (fp8.cuh's group_quotient: the product by
the rounded reciprocal, corrected by its exact error) against the binary32 division, at
the ties of E4M3, where one unit in the last place decides.  Compiled C: the arithmetic
is IEEE's, the same on the host and on the device."""
import ctypes
import os
import shutil
import subprocess

import pytest

SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <string.h>
static float from_bits(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
static uint32_t bits(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
float group_quotient(float x, float s, float inv) {
    const float q = x * inv, err = fmaf(q, fminf(s, 3.402823466e38f), -x);
    return fmaf(-err, inv, q);
}
/* Scales of every `step`-th significand, and of those within 256 of a multiple of 2^20,
 * where products with a tie's five bits come closest to a midpoint.  Numerators: the
 * nearest to scale times tie and five to each side.  Quotients that differ; `moved`
 * counts those of the product by the reciprocal that lie on another side of the tie. */
long differing(uint32_t step, long *moved) {
    long bad = 0;
    *moved = 0;
    for (uint32_t m = 0; m < 1u << 23; ++m) {
        const uint32_t low = (m + 256) & 0xfffffu;
        if (m % step != 0 && low > 512) continue;
        const float s = from_bits(0x3f800000u | m), inv = 1.0f / s;
        for (int tie = 1; tie < 32; tie += 2)
            for (int d = -5; d <= 5; ++d) {
                const float t = (float)tie, x = from_bits(bits(s * t) + (uint32_t)d);
                const float want = x / s, p = x * inv;
                bad += group_quotient(x, s, inv) != want;
                *moved += (want > t) - (want < t) != (p > t) - (p < t);
            }
    }
    return bad;
}
"""


def compiled(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, lib = str(tmp_path / "q.c"), str(tmp_path / "q.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    # no built-in fmaf: gcc for Arm folds -(q * s - x) into x - q * s, which is +0 and not
    # -0 where both are zero (the device's compiler keeps it: the norm's test has zeros)
    subprocess.run([cc, "-O2", "-ffp-contract=off", "-fno-builtin", "-shared", "-fPIC", src, "-o", lib, "-lm"],
                   check=True)
    return ctypes.CDLL(lib)


def test_the_corrected_product_is_the_quotient(tmp_path):
    lib = compiled(tmp_path)
    lib.differing.restype = ctypes.c_long
    moved = ctypes.c_long()
    assert lib.differing(101, ctypes.byref(moved)) == 0
    assert moved.value > 100000  # what the correction is for


def test_the_c_form_is_the_kernels():
    """The two lines of the C form are the kernel's."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "combine_expert_histogram_gb300", "csrc", "fp8.cuh")
    kernel = open(path).read()
    for line in SOURCE.split("float group_quotient")[1].splitlines()[1:3]:
        assert line.strip() in kernel


def test_zeros_and_infinite_scales(tmp_path):
    lib = compiled(tmp_path)
    q = lib.group_quotient
    q.restype, q.argtypes = ctypes.c_float, [ctypes.c_float] * 3
    inf = float("inf")
    text = lambda v: "nan" if v != v else repr(v)  # noqa: E731
    for x, s in ((0.0, 3.0), (-0.0, 3.0), (1.0, inf), (-1.0, inf), (-0.0, inf), (inf, inf),
                 (-inf, inf), (float("nan"), 2.0)):
        want = float("nan") if x != x or abs(x) == inf else x / s
        assert text(q(x, s, 0.0 if s == inf else 1 / s)) == text(want), (x, s)

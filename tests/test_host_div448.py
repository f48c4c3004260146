"""The block-128 casts divide a block's largest magnitude by 448 without a
divide instruction, as the NVFP4 scale divides by 6: q = fl(a z) with
z = fl(1/448), then fl(q + fl(a - 448 q) z).  a is at least 2^-100, so every
quotient is a normal fp32; the steps scale exactly with a by powers of two.
This runs every a of the binades at both ends of the range and of [1, 2) in C
with the host's correctly rounded fmaf against IEEE division."""
import shutil
import subprocess

import pytest

C_SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static unsigned long long run(uint32_t lo, uint32_t hi) {
    volatile float z = 1.0f / 448.0f;
    unsigned long long bad = 0;
    for (uint32_t u = lo; u < hi; ++u) {
        float a;
        memcpy(&a, &u, 4);
        float q = a * z;
        float r = fmaf(-q, 448.0f, a);
        float s = fmaf(r, z, q);
        volatile float ieee = a / 448.0f;
        if (s != ieee) ++bad;
    }
    return bad;
}

int main(void) {
    unsigned long long bad = 0;
    bad += run(27u << 23, 28u << 23);       /* [2^-100, 2^-99) */
    bad += run(127u << 23, 128u << 23);     /* [1, 2) */
    bad += run(254u << 23, 255u << 23);     /* the top binade */
    printf("%llu %a\n", bad, (double)(1.0f / 448.0f));
    return 0;
}
"""


def test_division_by_448_is_the_ieee_quotient(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "div448.c", tmp_path / "div448"
    src.write_text(C_SOURCE)
    subprocess.run([cc, "-O1", "-ffp-contract=off", "-fno-fast-math", "-o", str(exe), str(src),
                    "-lm"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True,
                         timeout=600).stdout.split()
    assert out[1] == "0x1.24924ap-9"          # z is the constant the kernels use
    assert int(out[0]) == 0

"""The quotient identities of the per-token INT8 quantiser and the fp8 cache store, checked on the CPU.

bf16 rows: s = RN(max|x| / 127) of a bf16 maximum takes one of 128 significands, x another 128; one correction of
RN(x * r), r = RN(1 / s), gives RN(x / s): checked for all of them at both relative exponents.
binary32 rows, and the arbitrary binary32 scale of the fp8 store: two corrections; checked on 2^26 random pairs of
significands, on scales next to powers of two, and on quotients next to the codes' rounding borders n + 1/2.
"""
import os
import shutil
import subprocess

import pytest

CHECK_C = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
static float from_bits(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
static uint32_t to_bits(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
static long total, bad;
static void check(float w, float s, int corrections)
{
    const float r = (float)(1.0 / (double)s), want = (float)((double)w / (double)s);
    float q = w * r;
    for (int i = 0; i < corrections; ++i) q = fmaf(fmaf(-q, s, w), r, q);
    ++total;
    bad += to_bits(q) != to_bits(want);
}
static uint64_t state = 88172645463325252ull;
static uint32_t rnd(void) { state ^= state << 13; state ^= state >> 7; state ^= state << 17; return (uint32_t)(state >> 32); }
int main(void)
{
    for (uint32_t a = 0; a < 128; ++a)
        for (uint32_t e = 0; e < 2; ++e) {
            const float s = (float)((double)from_bits(((127 + e) << 23) | (a << 16)) / 127.0);
            for (uint32_t x = 0; x < 128; ++x)
                for (uint32_t f = 0; f < 12; ++f) check(from_bits(((128 - f) << 23) | (x << 16)), s, 1);
        }
    printf("%ld %ld\n", total, bad);
    total = bad = 0;
    for (long i = 0; i < (1l << 26); ++i) {
        const uint32_t near = rnd() & 7;  /* one in four: a scale next to a power of two */
        const uint32_t m = near == 0 ? (rnd() & 15) : near == 1 ? 0x7fffffu - (rnd() & 15) : rnd() & 0x7fffffu;
        const float s = from_bits((127u << 23) | m);
        check(from_bits(((127u - (rnd() & 1)) << 23) | (rnd() & 0x7fffffu)), s, 2);
        const float n = (float)(rnd() % 128) + 0.5f;  /* quotients next to n + 1/2 */
        const float w = from_bits(to_bits(n * s) + (rnd() % 5) - 2);
        check(w, s, 2);
    }
    printf("%ld %ld\n", total, bad);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_corrected_quotients_are_correctly_rounded(tmp_path):
    src, exe = os.path.join(tmp_path, "q.c"), os.path.join(tmp_path, "q")
    open(src, "w").write(CHECK_C)
    subprocess.run(["gcc", "-O2", "-ffp-contract=off", "-o", exe, src, "-lm"], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    assert [tuple(map(int, line.split())) for line in lines if line] == [(128 * 2 * 128 * 12, 0), (1 << 27, 0)]

"""Logits as whole numbers, and ranges of them in bins (csrc/sample_keys.cuh), run on the host: a logit that a kernel's
f32 comparisons take into a range has its key in the range and so its bin in the histogram, and none of the range's
logits is left out.  The ranges end where a bin, or half of a range, may: at any key, that of -0 among them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
PROGRAM = r"""
#include <cmath>
#include <cstdio>
#include "sample_keys.cuh"
using namespace plm;

static int failed = 0;
#define CHECK(x) do { if (!(x)) { if (failed++ < 9) printf("line %d: %s\n", __LINE__, #x); } } while (0)

static unsigned state = 12345;
static unsigned next32() { state = state * 1664525u + 1013904223u; return state ^ state >> 15; }
static uint32_t any_key() {   // of a number, more often than not near 0
    const uint32_t lowest = LOWEST + 1, highest = 0xFF7FFFFFu;
    switch (next32() % 4) {
        case 0: return MINUS_ZERO + next32() % 9 - 4;
        case 1: return MINUS_ZERO + (next32() % (1u << 21)) - (1u << 20);
        default: return lowest + next32() % (highest - lowest);
    }
}

static void check(uint32_t lo, uint32_t end, uint32_t key) {
    const uint32_t hi = range_end(end);
    if (hi < lo) return;
    const KeyBins K(lo, hi);
    const float x = logit_of(key) + 0.0f, hi_x = logit_of(hi), lo_x = logit_of(lo);   // as a row's logits are read
    const uint32_t k = key_of(x);
    CHECK(k != MINUS_ZERO);
    const bool in = !(x > hi_x) && x >= lo_x;
    CHECK(in == (lo <= k && k <= hi));
    if (!in) return;
    const uint32_t b = (hi - k) >> K.shift;
    CHECK(b < (uint32_t)BINS && K.bin(k) == (int)b && K.first(b) >= k && K.last(b) <= k && K.last(b) >= lo && K.first(b) <= hi);
}

int main() {
    CHECK(key_of(-INFINITY) == LOWEST && key_of(-0.0f) == MINUS_ZERO && key_of(0.0f) == MINUS_ZERO + 1 && key_of(INFINITY) == 0xFF800000u);
    const uint32_t near[] = {MINUS_ZERO - 2, MINUS_ZERO - 1, MINUS_ZERO, MINUS_ZERO + 1, MINUS_ZERO + 2, MINUS_ZERO + 5000, MINUS_ZERO - 5000};
    for (uint32_t lo : near)
        for (uint32_t hi : near)
            for (uint32_t k : near) check(lo, hi, k);
    for (int i = 0; i < 2000000; ++i) {
        uint32_t a = any_key(), b = any_key();
        if (a > b) { const uint32_t c = a; a = b; b = c; }
        check(a, b, any_key());
        check(a, b, MINUS_ZERO);
        const KeyBins K(a, b);                             // where the next range may end: a bin's first, the middle
        const uint32_t k1 = K.first((int)(next32() % (((b - a) >> K.shift) + 1)));
        check(a, k1, MINUS_ZERO);
        check(a, a + (k1 - a) / 2, any_key());
    }
    for (int i = 0; i < 1000000; ++i) {
        const uint32_t k = any_key();
        CHECK(key_of(logit_of(k)) == k);
    }
    printf("%d failed\n", failed);
    return failed != 0;
}
"""


@pytest.mark.skipif(not os.path.exists(NVCC), reason="no nvcc")
def test_ranges_of_keys(tmp_path):
    source, program = str(tmp_path / "keys.cu"), str(tmp_path / "keys")
    with open(source, "w") as f:
        f.write(PROGRAM)
    subprocess.check_call([NVCC, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I",
                           os.path.join(ROOT, "quant_packed_gemv_gb300", "csrc"), source, "-o", program])
    done = subprocess.run([program], stdout=subprocess.PIPE, text=True)
    assert done.returncode == 0, done.stdout

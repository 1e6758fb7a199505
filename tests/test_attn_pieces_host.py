"""Where the pieces of an attention item lie (csrc/attn_tile.cuh), run on the host: the units of all items are cut
evenly over the CTAs, so CTA c holds units U c / ctas .. U (c + 1) / ctas - 1; a piece's slot is c + item where every
piece is kept, else 2 c + (1 if it begins the item).  And whatever first unit the workspace holds (a kernel whose wait
ran out may have left anything there), no place lies outside the slots."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "attn_tile.cuh"
using namespace plm;

static int failed = 0;
#define CHECK(x) do { if (!(x)) { if (failed++ < 9) printf("line %d: %s\n", __LINE__, #x); } } while (0)

static unsigned state = 12345;
static int below(int n) { state = state * 1664525u + 1013904223u; return (int)((state >> 8) % (unsigned)n); }

int main() {
    for (int trial = 0; trial < 400; ++trial) {
        TilePlan P = {};
        P.tile_rows = below(2) ? 256 : 128;
        P.ctas = 1 + below(MOST_CTAS);
        P.keep = below(2);
        const int items = 1 + below(300);
        std::vector<int> first(items), tiles(items), cta;
        int U = 0;
        for (int i = 0; i < items; ++i) {
            first[i] = U;
            tiles[i] = 1 + below(below(4) ? 6 : 400);
            U += tiles[i];
        }
        const int ctas = unit_ctas(P, U);
        for (int c = 0; c < ctas; ++c)
            while ((long long)cta.size() < (long long)U * (c + 1) / ctas) cta.push_back(c);
        const long long slots = P.keep ? P.ctas + items : 2LL * P.ctas;
        for (int i = 0; i < items; ++i) {
            const int row = below(P.tile_rows);
            const Pieces X = item_pieces(P, i, first[i], tiles[i], U, row);
            const int c0 = cta[first[i]], c1 = cta[first[i] + tiles[i] - 1];
            CHECK(X.n == c1 - c0 + 1);
            for (int p = 0; p < X.n; ++p)
                CHECK(X.at(p) == (P.keep ? (long long)c0 + p + i : 2LL * (c0 + p) + (p == 0)) * P.tile_rows + row);
            const int bad[] = {-1, -U, -0x7FFFFFFF - 1, -0x40000000, U, U + 1, 0x7F7F7F7F, 0x7FFFFFFF - tiles[i], -0x01010102};
            for (int u0 : bad) {
                const Pieces Y = item_pieces(P, i, u0, tiles[i], U, row);
                CHECK(Y.n <= ctas);
                for (int p = 0; p < Y.n; ++p) CHECK(Y.at(p) >= 0 && Y.at(p) < slots * P.tile_rows);
            }
        }
    }
    // many units, as far as they are allowed
    const int U = 0x7FFFFFFF, ctas = 152;
    for (int k = 0; k < 100000; ++k) {
        const int u = (int)(((long long)below(1 << 24) << 7) + below(128)) % U, c = unit_cta(u, U, ctas);
        CHECK((long long)U * c / ctas <= u && u < (long long)U * (c + 1) / ctas);
    }
    CHECK(unit_cta(U - 1, U, ctas) == ctas - 1 && unit_cta(0, U, ctas) == 0);
    printf("%d failed\n", failed);
    return failed != 0;
}
"""


@pytest.mark.skipif(not os.path.exists(NVCC), reason="no nvcc")
def test_places_of_pieces(tmp_path):
    source, program = str(tmp_path / "pieces.cu"), str(tmp_path / "pieces")
    with open(source, "w") as f:
        f.write(PROGRAM)
    subprocess.check_call([NVCC, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I",
                           os.path.join(ROOT, "quant_packed_gemv_gb300", "csrc"), source, "-o", program])
    done = subprocess.run([program], stdout=subprocess.PIPE, text=True)
    assert done.returncode == 0, done.stdout

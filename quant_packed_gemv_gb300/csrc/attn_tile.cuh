// How the tile kernel cuts its work, shared by the kernels that read its
// partial results.
//
// A UNIT is 128 keys for one row tile and key/value head.  An ITEM is a row
// tile of a job with all its keys: job one is the shared prefix, whose row
// tiles run over the rows of the whole batch; the others are the sequences'
// own keys.  The units of all items in order are cut evenly over the CTAs, so
// an item may be cut too; each piece leaves (m, l, O) in a slot.
#pragma once

#include "attn.cuh"

namespace plm {

constexpr int TK = 128;   // keys per unit

struct TilePlan {
    int tile_rows;         // rows per row tile (128 or 256)
    int ctas;
    int prefix_tiles;      // units per prefix item; 0: no prefix job
    int prefix_row_tiles;  // row tiles of the prefix job (per head)
    int own;               // own jobs in the tile kernel
    int own_row_tiles;     // row tiles of a sequence's rows (per head)
    // workspace
    int* units;            // [1] all units (own: known on the device only)
    int* item_unit;        // [own items] first unit of the item (own jobs)
    float* o;              // [slots][tile_rows][D], not divided by the sum
    float2* ml;            // [slots][tile_rows]: m (log2), l
};

// A sequence takes part in the shared prefix when each of its queries sees
// all of it.
__device__ __forceinline__ bool attn_shares(const AttnArgs& A, const TilePlan& P, int len) {
    return P.prefix_tiles > 0 && len - A.nq + 1 >= A.prefix;
}

// First own key of a sequence, and the end of the keys that row tile rt of it
// sees.
__device__ __forceinline__ int own_begin(const AttnArgs& A, const TilePlan& P, int len) {
    return attn_shares(A, P, len) ? A.prefix : 0;
}
__device__ __forceinline__ int own_end(const AttnArgs& A, const TilePlan& P, int len, int rt) {
    const long long last = min((long long)A.nq * A.group, (long long)(rt + 1) * P.tile_rows) - 1;
    return attn_seen(A, len, (int)(last / A.group));
}

// Units of (sequence, row tile) `pair` of the own jobs, for one head.
__device__ __forceinline__ int own_tiles(const AttnArgs& A, const TilePlan& P, int pair) {
    const int b = pair / P.own_row_tiles, rt = pair - b * P.own_row_tiles;
    const int len = attn_len(A, attn_row(A, b));
    return max(0, own_end(A, P, len, rt) - own_begin(A, P, len) + TK - 1) / TK;
}

// CTAs that get units: with fewer units than CTAs the others stay idle, so that
// no share between two others is empty.
__device__ __forceinline__ int unit_ctas(const TilePlan& P, int U) { return min(P.ctas, U); }

// The CTA (of ctas) that holds unit u of U.
__device__ __forceinline__ int unit_cta(int u, int U, int ctas) {
    int c = (int)((long long)u * ctas / U);
    while ((long long)U * (c + 1) / ctas <= u) ++c;
    return c;
}

// Slot of the piece of an item that CTA c holds.  With a prefix job every
// piece of every item is kept: items and CTAs both follow the units' order,
// so c + item is free.  Otherwise only cut items are: a CTA has at most one
// piece that does not begin its item and one cut piece that does.
__host__ __device__ __forceinline__ long long piece_slot(const TilePlan& P, int c, int item, bool begins) {
    return P.prefix_tiles > 0 ? (long long)c + item : 2LL * c + begins;
}

// One row's sums over partial results.
template <int PER> struct RowSum {
    float m = -INFINITY, l = 0.0f, o[PER] = {};
    __device__ __forceinline__ void add(float m2, float l2, const float (&o2)[PER]) {
        if (l2 == 0.0f) return;   // a piece without keys
        const float mn = fmaxf(m, m2);
        const float a = exp2f(m - mn), b = exp2f(m2 - mn);
        l = l * a + l2 * b;
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = o[i] * a + o2[i] * b;
        m = mn;
    }
};

// Units at most (the kernel counts them in an int).
long long tile_units(const AttnArgs& A, bool share, bool own);

// TilePlan of a problem; its workspace pointers are set from ws (may be null).
size_t tile_plan(const AttnArgs& A, int d, bool share, bool own, void* ws, TilePlan* P);

cudaError_t launch_attn_tile(const AttnArgs& A, const TilePlan& P, int type, int d, cudaStream_t stream);

// At most 16 query rows per sequence and key/value head; P: prefix results to
// add, or null.
cudaError_t launch_attn_rows(const AttnArgs& A, const TilePlan* P, int type, int d, cudaStream_t stream);

}  // namespace plm

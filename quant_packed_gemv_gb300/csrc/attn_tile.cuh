// How the tile kernel cuts its work, shared by the kernels that read its
// partial results.
//
// A UNIT is 128 keys for one row tile and key/value head.  An ITEM is a row
// tile with all its keys: of the shared prefix, whose row tiles run over the
// rows of the whole batch, or of a sequence's own keys (two launches, where a
// call has both).  The units of all items in order are cut evenly over the
// CTAs, so an item may be cut too; its pieces leave (m, l, O) in slots.
#pragma once

#include "attn.cuh"

namespace plm {

constexpr int TK = 128;   // keys per unit

struct TilePlan {
    int tile_rows;         // rows per row tile (128 or 256)
    int ctas;
    int prefix_tiles;      // units per prefix item; 0: no prefix job
    int prefix_row_tiles;  // row tiles of the prefix job (per head)
    int own_row_tiles;     // row tiles of a sequence's rows (per head)
    int job;               // what a launch does: 0 the prefix, 1 the own keys
    int keep;              // every piece is kept, to be added to others
    // workspace
    int* units;            // [1] all units (own: known on the device only)
    int* item_unit;        // [own items] first unit of the item (own, kept pieces)
    int4* cut;             // [ctas] the item that a CTA goes on with, if it does not begin with one
                           // (own, else): (sequence, row tile) or -1, head, first unit, units
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

// Slot of the piece of an item that CTA c holds.  Where every piece is kept:
// items and CTAs both follow the units' order, so c + item is free.  Otherwise
// only cut items are: a CTA has at most one piece that does not begin its item
// and one cut piece that does.
__host__ __device__ __forceinline__ long long piece_slot(const TilePlan& P, int c, int item, bool begins) {
    return P.keep ? (long long)c + item : 2LL * c + begins;
}

// The sums of N rows, by a warp: PER dims a lane.
template <int PER, int N = 1> struct RowSum {
    float m[N], l[N], o[N][PER];
    __device__ RowSum() {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            m[j] = -INFINITY;
            l[j] = 0.0f;
#pragma unroll
            for (int k = 0; k < PER; ++k) o[j][k] = 0.0f;
        }
    }

    // Adds the pieces of each row's item (item[j] < 0: none; first unit u0[j],
    // `tiles` of U units), row i[j] of its tile: a lane each for their weights,
    // then their dims, all in the order of the units.  The loads of the rows, and
    // of several pieces, are in flight together: each is a trip to L2.
    __device__ void pieces(const TilePlan& P, const int (&item)[N], const int (&u0)[N], int tiles, int U, const int (&i)[N],
                           int lane) {
        constexpr int AHEAD = N * PER <= 4 ? 8 : 4;
        const int ctas = unit_ctas(P, U);
        int c0[N], n[N], most = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            c0[j] = item[j] < 0 ? 0 : unit_cta(u0[j], U, ctas);
            n[j] = item[j] < 0 ? 0 : unit_cta(u0[j] + tiles - 1, U, ctas) - c0[j] + 1;
            most = max(most, n[j]);
        }
        for (int p0 = 0; p0 < most; p0 += 32) {
            long long at[N];
            float w[N];
            float2 ml[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const bool in = p0 + lane < n[j];
                at[j] = in ? piece_slot(P, c0[j] + p0 + lane, item[j], p0 + lane == 0) * P.tile_rows + i[j] : 0;
                ml[j] = in ? P.ml[at[j]] : make_float2(-INFINITY, 0.0f);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (ml[j].y == 0.0f) ml[j].x = -INFINITY;   // a piece without keys
                const float mn = fmaxf(m[j], warp_max(ml[j].x));
                const float old = m[j] == -INFINITY ? 0.0f : ex2(m[j] - mn);
                w[j] = ml[j].x == -INFINITY ? 0.0f : ex2(ml[j].x - mn);
                m[j] = mn;
                l[j] = l[j] * old + warp_sum(w[j] * ml[j].y);
#pragma unroll
                for (int k = 0; k < PER; ++k) o[j][k] *= old;
            }
            const int some = min(32, most - p0);
            for (int p = 0; p < some; p += AHEAD) {
                float v[N][AHEAD][PER];
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int q = 0; q < AHEAD; ++q) {
                        // past the row's pieces: its weight is 0, and any piece will do
                        const long long row = __shfl_sync(0xFFFFFFFFu, at[j], min(p + q, max(0, min(31, n[j] - p0 - 1))));
                        const float* src = P.o + row * (32 * PER) + PER * lane;
                        if constexpr (PER == 4) {
                            const float4 x = *reinterpret_cast<const float4*>(src);
                            v[j][q][0] = x.x; v[j][q][1] = x.y; v[j][q][2] = x.z; v[j][q][3] = x.w;
                        } else {
                            const float2 x = *reinterpret_cast<const float2*>(src);
                            v[j][q][0] = x.x; v[j][q][1] = x.y;
                        }
                    }
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int q = 0; q < AHEAD; ++q) {
                        const float f = p + q < 32 ? __shfl_sync(0xFFFFFFFFu, w[j], (p + q) & 31) : 0.0f;
                        if (f != 0.0f)
#pragma unroll
                            for (int k = 0; k < PER; ++k) o[j][k] = fmaf(f, v[j][q][k], o[j][k]);
                    }
            }
        }
    }

    // Row j to the output: o / l, or zeros and lse = -inf where there was no key.
    template <class E>
    __device__ void store(const AttnArgs& A, int j, long long tok, int qh, int lane) const {
        const float inv = l[j] == 0.0f ? 0.0f : 1.0f / l[j];
        const long long off = tok * A.o_ts + (long long)qh * A.o_hs + PER * lane;
        if constexpr (PER == 4) {
            attn_store4<E>(A, off, make_float4(o[j][0] * inv, o[j][1] * inv, o[j][2] * inv, o[j][3] * inv));
        } else if (A.o_f32) {
            *reinterpret_cast<float2*>(static_cast<float*>(A.o) + off) = make_float2(o[j][0] * inv, o[j][1] * inv);
        } else {
            *reinterpret_cast<uint32_t*>(static_cast<E*>(A.o) + off) = pack_pair<E>(o[j][0] * inv, o[j][1] * inv);
        }
        if (A.lse && lane == 0) A.lse[tok * A.heads + qh] = l[j] == 0.0f ? -INFINITY : (m[j] + log2f(l[j])) * 0.6931471805599453f;
    }
};

// Plan of a launch of the tile kernel: of the prefix (job 0), or of the own
// keys (job 1; share: the prefix is done apart).  Its workspace starts at ws
// (may be null); *bytes is its size, or SIZE_MAX if there are too many units.
TilePlan tile_plan(const AttnArgs& A, int d, int job, bool share, void* ws, size_t* bytes);

cudaError_t launch_attn_tile(const AttnArgs& A, const TilePlan& P, int type, int d, cudaStream_t stream);

// Adds the pieces of both launches for every row.
cudaError_t launch_attn_merge(const AttnArgs& A, const TilePlan& prefix, const TilePlan& own, int type, int d,
                              cudaStream_t stream);

// At most 32 query rows per sequence and key/value head; P: prefix results to
// add, or null.
cudaError_t launch_attn_rows(const AttnArgs& A, const TilePlan* P, int type, int d, cudaStream_t stream);

}  // namespace plm

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
    int tile_shift;        // its logarithm
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

// Sequence of a (sequence, row tile).
__device__ __forceinline__ int own_seq(const TilePlan& P, int pair) { return P.own_row_tiles == 1 ? pair : pair / P.own_row_tiles; }

// First own key of a sequence, and the end of the keys that row tile rt of it
// sees.
__device__ __forceinline__ int own_begin(const AttnArgs& A, const TilePlan& P, int len) {
    return attn_shares(A, P, len) ? A.prefix : 0;
}
__device__ __forceinline__ int own_end(const AttnArgs& A, const TilePlan& P, int len, int rt) {
    if (rt + 1 == P.own_row_tiles) return len;   // its last row is the last query's
    return attn_seen(A, len, (int)((((unsigned)(rt + 1) << P.tile_shift) - 1) / (unsigned)A.group));
}

// Units of (sequence, row tile) `pair` of the own jobs, for one head.
__device__ __forceinline__ int own_tiles(const AttnArgs& A, const TilePlan& P, int pair) {
    const int b = own_seq(P, pair), rt = pair - b * P.own_row_tiles;
    const int len = attn_len(A, attn_row(A, b));
    return max(0, own_end(A, P, len, rt) - own_begin(A, P, len) + TK - 1) / TK;
}

// The same of all a sequence's row tiles (by additions: the last row of tile rt is
// query ((rt + 1) tile_rows - 1) / group).
__device__ __forceinline__ int seq_tiles(const AttnArgs& A, const TilePlan& P, int len) {
    const int begin = own_begin(A, P, len), q = P.tile_rows / A.group, r = P.tile_rows - q * A.group;
    int sum = 0, t = -1, left = A.group - 1;   // t group + left: the last row so far (-1: none)
    for (int rt = 0; rt < P.own_row_tiles; ++rt) {
        t += q;
        left += r;
        if (left >= A.group) { left -= A.group; ++t; }
        const int end = rt + 1 == P.own_row_tiles ? len : attn_seen(A, len, t);
        sum += max(0, end - begin + TK - 1) / TK;
    }
    return sum;
}

// CTAs that get units: with fewer units than CTAs the others stay idle, so that
// no share between two others is empty.
__host__ __device__ __forceinline__ int unit_ctas(const TilePlan& P, int U) { return min(P.ctas, U); }

// The CTA (of ctas) that holds unit u of U: the last c with U c / ctas <= u,
// i.e. U c < (u + 1) ctas (an estimate, then exact steps: a 64-bit division is
// slow where a row's sums wait for it).  0 .. ctas - 1 whatever u is, so that a wrong
// unit never leads outside the slots.
__host__ __device__ __forceinline__ int unit_cta(int u, int U, int ctas) {
    const long long lim = ((long long)u + 1) * ctas;
    int c = (int)fmaxf(0.0f, fminf((float)(ctas - 1), (float)lim / (float)U));
    while (c > 0 && (long long)U * c >= lim) --c;
    while (c + 1 < ctas && (long long)U * (c + 1) < lim) ++c;
    return c;
}

// Slot of the piece of an item that CTA c holds.  Where every piece is kept:
// items and CTAs both follow the units' order, so c + item is free.  Otherwise
// only cut items are: a CTA has at most one piece that does not begin its item
// and one cut piece that does.
__host__ __device__ __forceinline__ long long piece_slot(const TilePlan& P, int c, int item, bool begins) {
    return P.keep ? (long long)c + item : 2LL * c + begins;
}

// Adding up.  The sums of a row are sum_p w_p O_p and sum_p w_p l_p with w_p =
// 2^(m_p - max m) over its parts p.  First all threads bring the rows' (m, l) into
// shared memory, then eight lanes a row turn them into weights, then the
// threads share the rows' dims, four each, and add the parts in order.  Every
// step has all its loads in flight at once: a row waits for three trips to L2,
// whatever its number of parts (a warp per row with the weights in lanes, or a
// thread per row, took 6 to 15 us where the parts were many).
// What costs time here otherwise is integer division, so each row's places are
// worked out once.
struct Pieces {
    long long first, next;   // row in P.ml and P.o of piece 0 (0 if there is none), of piece 1
    int step;                // rows from a piece to the next, after that
    int n;
    __host__ __device__ __forceinline__ long long at(int p) const { return p == 0 ? first : next + (long long)(p - 1) * step; }
};
// Of row i of an item (first unit u0, `tiles` of U units).
__host__ __device__ __forceinline__ Pieces item_pieces(const TilePlan& P, int item, int u0, int tiles, int U, int i) {
    const int ctas = unit_ctas(P, U), c0 = unit_cta(u0, U, ctas);
    Pieces X;
    X.n = unit_cta(u0 + tiles - 1, U, ctas) - c0 + 1;
    X.first = piece_slot(P, c0, item, true) * P.tile_rows + i;
    X.next = piece_slot(P, c0 + 1, item, false) * P.tile_rows + i;
    X.step = P.keep ? P.tile_rows : 2 * P.tile_rows;
    return X;
}

template <int ROWS, int MOST, int SETS> struct Sums {
    float2 ml[MOST][ROWS];      // (m, l) of the parts, then the weight in x
    float inv[ROWS];            // 1 / sum, 0 without keys
    Pieces pieces[SETS][ROWS];
    long long out[ROWS], lse[ROWS];   // places of the row in o and lse
    __device__ __forceinline__ void place(const AttnArgs& A, int k, long long tok, int qh) {
        out[k] = tok * A.o_ts + (long long)qh * A.o_hs;
        lse[k] = tok * A.heads + qh;
    }
};

// Brings (m, l) of the pieces' row into `ml`: every `step`-th piece.
template <int ROWS>
__device__ __forceinline__ void bring(const TilePlan& P, const Pieces& X, float2 (*ml)[ROWS], int k, int from, int step) {
    for (int p = from; p < X.n; p += step) ml[p][k] = P.ml[X.at(p)];
}

// Weights of row k from its n parts' (m, l), by eight neighbouring lanes (sub =
// 0 .. 7, which all take part); the first writes 1 / sum and the row's lse.
template <int ROWS, int MOST, int SETS>
__device__ __forceinline__ void weigh(const AttnArgs& A, Sums<ROWS, MOST, SETS>& S, int k, int n, bool in, int sub) {
    float m = -INFINITY, l = 0.0f;
    if (in)
        for (int p = sub; p < n; p += 8) {
            const float2 v = S.ml[p][k];
            if (v.y != 0.0f) m = fmaxf(m, v.x);   // l = 0: a part without keys
        }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (in)
        for (int p = sub; p < n; p += 8) {
            const float2 v = S.ml[p][k];
            const float w = v.y == 0.0f || v.x == -INFINITY ? 0.0f : ex2(v.x - m);
            if (v.y != 0.0f) l += w * v.y;
            S.ml[p][k].x = w;
        }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    if (in && sub == 0) {
        S.inv[k] = l == 0.0f ? 0.0f : 1.0f / l;
        if (A.lse) A.lse[S.lse[k]] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

// acc[i] += the dims d[i] .. d[i] + 3 of the pieces X[i], weighted (w: ROWS apart).
template <int D, int ROWS, int N>
__device__ __forceinline__ void add_pieces(const TilePlan& P, const Pieces* const (&X)[N], const float2* const (&w)[N],
                                           const int (&d)[N], float4 (&acc)[N]) {
    constexpr int AHEAD = 8;   // loads in flight of each
    int most = X[0]->n;
#pragma unroll
    for (int i = 1; i < N; ++i) most = max(most, X[i]->n);
#pragma unroll 1
    for (int p = 0; p < most; p += AHEAD) {
        float4 v[N][AHEAD];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)   // past the last piece: the last again, without weight
                v[i][q] = *reinterpret_cast<const float4*>(P.o + X[i]->at(max(0, min(p + q, X[i]->n - 1))) * D + d[i]);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const float f = p + q < X[i]->n ? w[i][(p + q) * ROWS].x : 0.0f;
                if (f != 0.0f) {   // O of a part without weight may hold anything
                    acc[i].x = fmaf(f, v[i][q].x, acc[i].x);
                    acc[i].y = fmaf(f, v[i][q].y, acc[i].y);
                    acc[i].z = fmaf(f, v[i][q].z, acc[i].z);
                    acc[i].w = fmaf(f, v[i][q].w, acc[i].w);
                }
            }
    }
}

constexpr int MOST_CTAS = 160;   // of the tile kernel: bounds a row's pieces

// Plan of a launch of the tile kernel: of the prefix (job 0), or of the own
// keys (job 1; share: the prefix is done apart).  Its workspace starts at ws
// (may be null); *bytes is its size, or SIZE_MAX if there are too many units.
TilePlan tile_plan(const AttnArgs& A, int d, int job, bool share, void* ws, size_t* bytes);

cudaError_t launch_attn_tile(const AttnArgs& A, const TilePlan& P, int type, int d, cudaStream_t stream);

// Adds the pieces of both launches for every row.
cudaError_t launch_attn_merge(const AttnArgs& A, const TilePlan& prefix, const TilePlan& own, int type, int d,
                              cudaStream_t stream);

// Few query rows per sequence and key/value head; P: prefix results to
// add, or null.
cudaError_t launch_attn_rows(const AttnArgs& A, const TilePlan* P, int type, int d, cudaStream_t stream);

cudaError_t launch_attn_rows8(const AttnArgs8& A, const TilePlan* P, int type, int d, cudaStream_t stream);

// CTAs of that kernel that the GPU takes well at once, for so many rows a sequence
// and head.
long long attn_rows_room(int d, int rows, bool kv8 = false);

}  // namespace plm

// Paged attention for few query rows per (sequence, key/value head), in chunks
// of up to 32: decode, and some drafted tokens (plm_attn_shared_prefix).
//
// Mathematics.  With R = tokens * group rows, each block of 16 keys is two
// small products: S^T = K Q^T (16 keys x 8 rows, sums over d) and O^T += V^T
// P^T (d x 8 rows, sums over 16 keys), P = 2^(S scale log2 e - m).  m is a
// running reference, not the exact maximum: it is raised (and O, l scaled)
// only when a score exceeds it by more than 2^8, so most blocks need one vote
// and no reduction; p stays below 2^8, far inside f16.
//
// Layout.  The keys are the M side of mma.sync m16n8k16, so 8 rows cost no
// padding, and the sums over d and over keys may run in any order.  Lane
// (g, t) = (lane / 4, lane % 4) therefore takes 16 bytes of K rows g and g + 8
// (dims 32 c + 8 t ..) and of V rows 2t, 2t + 1, 2t + 8, 2t + 9 (dims 64 c + 8 g
// ..) as they lie and uses them as fragments.  Rows of Q follow K's order of d;
// P^T needs one movmatrix per 8 x 8 block.  Up to 16 rows Q stays in registers;
// beyond, the warps share it in shared memory, so that O (32 registers per 8
// rows at D = 128) has room.
//
// 8-bit pages (plm_attn_kv8).  Codes become f16 pairs by two byte permutes and a
// subtraction, exactly, whatever the cache's type.  A block's power of two comes in
// after the first product, whose sums over 32 dims it scales in f32; so Q has to fit
// f16, and its rows are divided by powers of two, to 2^13 at most.  A key's values reach
// 2^120, so that a sum of 128 products would reach 2^140: the keys' codes are made 2^13
// times smaller, which costs nothing, and that comes back with the row's power of two.  The
// values' powers of two go into the codes before the second product, relative to the
// largest of the same 32 dims so far, and p is held 2^7 times as large, so that f16 keeps
// what is above 2^-32 of the row's largest.  The relative powers are exponents of f16 down
// to 2^-14 (two instructions a pair of keys), its smallest numbers down to 2^-24.  A warp
// that meets a block below that starts over, and then takes such blocks by products of their
// own, whose sums f32 holds down to 2^-126: no value is lost beside one that a row does not
// see or gives no share to (64 sequences of up to 4000 keys, 63 us: 67 with one key in 50
// 2^-16 of the others, 86 with 2^-30).  bf16 operands would be
// exact without any of this, but a code costs two instructions more in bf16, and
// instructions are what the 8-bit form is bound by: 64 sequences of up to 4000 keys took
// 72 us so, and take 63 with f16 operands, four CTAs an SM and the ring's place below.
//
// Bound: HBM (4 D bytes per key and head pair, ~2 operations per byte and row; 8-bit
// pages 2 D + D / 16, where issue comes first).  Each warp brings its blocks (8 KB of K
// and V at D = 128) into a ring of its own by cp.async, 16-byte chunks XORed so that the
// fragment loads are free of bank conflicts, rows beginning with the banks (rings 16 bytes
// off: 90 us instead of 82); keys past the end are filled with zeros and not read.  The warps
// of a CTA and the CTAs of a cluster take the blocks in turn and add their parts through
// shared memory, in a fixed order.  One GB300, 8 heads of 128, 4 query heads each, bf16, us
// for 16-bit pages and 8-bit ones: 64 sequences of up to 4000 keys 83 (6.4 TB/s) and 63
// (4.4), 256 of 2000 162 (6.5) and 109 (5.0), 4 of 1100 7.2 and 8.4, which is latency.  From 16
// rows on, 8-bit pages are the slower ones: 64 x 8 rows over up to 3000 keys 66 and 64, 16 rows 72
// and 75, 32 rows 124 and 142, 48 x 20 behind 8192 63 and 83.  With more than 8 rows an SM holds 8 warps
// (4 for 25 to 32 rows of 128), which issue the conversions.  Spills at the registers of those CTAs, bytes
// stored: 8-bit pages of 128 dims up to 8 rows 16, 25 to 32 rows 36 (16-bit pages 32).
#pragma once

#include <cstddef>
#include <type_traits>

#include "attn_tile.cuh"

namespace plm {

namespace {

constexpr int DW = 4;               // warps per CTA
constexpr int V_LEAST = 24;         // 2^-24 is the smallest number of f16
constexpr int F16_ONE = 15;         // the exponent of 1 in f16
constexpr float RAISE = 8.0f;       // log2 by which a score may exceed the reference
constexpr float LOG2E = 1.4426950408889634f;

template <class E> __device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                            uint32_t a3, uint32_t b0, uint32_t b1);
template <> __device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <> __device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                                    uint32_t a2, uint32_t a3, uint32_t b0,
                                                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four codes as two pairs of f16, 2^13 times smaller, exact: c as 2^-3 + (c + 128)
// 2^-13 less 2^-3 + 2^-6.
constexpr int CODES_DOWN = 13;
__device__ __forceinline__ void codes_down(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u, less = 0x30803080u;
    const uint32_t a = __byte_perm(u, 0x30303030u, 0x4140), b = __byte_perm(u, 0x30303030u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(less));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(less));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t words(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// Shared memory: Q fragments (NB > 2), then the warps' rings, in whose place
// the parts of the warps go at the end: references m and sums l of the rows,
// O [rows][D + 4] (padded against conflicts).
template <int D, int NB, bool KV8> struct RowsSmem {
    static constexpr int ROWS = 8 * NB, PITCH = D + 4;
    static constexpr int STAGES = KV8 && NB == 1 ? (D == 64 ? 6 : 3) : (KV8 ? 2 : 1) * (D == 64 ? 2 : 1) * (NB == 1 ? 2 : 3);
    static constexpr int STAGE = 16 * D * (KV8 ? 1 : 2);   // bytes of 16 keys' K, or V
    static constexpr int EXPS = KV8 ? 16 * (D / 32) : 0;   // of their exponents
    static constexpr int SLOT = 2 * (STAGE + EXPS);
    struct Parts {
        float m[DW][ROWS], l[DW][ROWS];
        float o[DW][ROWS][PITCH];
        Sums<ROWS, 8 * DW + MOST_CTAS, 1> sums;   // of the cluster's warps, then the prefix pieces
    };
    uint4 q[NB > 2 ? NB * (D / 32) * 32 : 1];
    union {
        alignas(128) uint8_t ring[DW][STAGES][SLOT];   // (a copied row begins with the banks)
        Parts part;
    };
    float q_size[KV8 ? ROWS : 1];   // powers of two that the rows of Q, and the codes, were divided by
};

// CTAs of 8 nb rows that an SM holds at once: registers bound the first, shared
// memory the others (228 KB, of which a CTA takes 1 KB for itself).
__host__ __device__ constexpr int rows_ctas(int d, int nb, bool kv8) { return nb == 1 ? (kv8 ? 4 : 3) : nb == 4 && d == 128 ? 1 : 2; }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// The first n bytes of 16, then zeros.
__device__ __forceinline__ void cp16_part(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// Where 16-byte chunk c of K row r, of V row r, lies in its part of the ring.
template <int D, bool KV8> __device__ __forceinline__ int k_chunk(int r, int c) {
    if (!KV8) return r * (2 * D) + ((c ^ ((r & 1) << 2)) << 4);
    return r * D + ((c ^ (D == 128 ? (r & 3) << 1 : r & 2)) << 4);
}
template <int D, bool KV8> __device__ __forceinline__ int v_chunk(int r, int c) {
    if (!KV8) return r * (2 * D) + ((c ^ (r & 6)) << 4);
    // (64 bytes a row: even rows would all begin in the same half of the banks)
    return D == 128 ? r * D + ((c ^ (r & 6)) << 4) : (r ^ ((r >> 1) & 1)) * D + ((c ^ ((r >> 1) & 2)) << 4);
}

// 8-bit pages: dims (D / 8) g .. of V rows 2t, 2t + 1, 2t + 8, 2t + 9, all in one block.
template <int D> __device__ __forceinline__ void bring_codes(const uint8_t* vs, int t, int g, uint32_t (&x)[4][D / 32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 2 * t + (i & 1) + 8 * (i >> 1);
        if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(vs + v_chunk<D, true>(r, g));
            x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(vs + v_chunk<D, true>(r, g >> 1) + 8 * (g & 1));
            x[i][0] = u.x; x[i][1] = u.y;
        }
    }
}

// 2^(e - of), e <= of; 0 for e = 0.
__device__ __forceinline__ float power_below(int e, int of) { return e ? __uint_as_float((uint32_t)max(e - of + 127, 0) << 23) : 0.0f; }
// Their values as operands: take(k, a0 .. a3) for dims 2 k, 2 k + 1 of the lane's.  f01, f89: the rows' powers of two in
// f16, 1 at most, 2^-V_LEAST at least or 0.
template <int D, class F> __device__ __forceinline__ void value_fragments(const uint32_t (&x)[4][D / 32], uint32_t f01, uint32_t f89, F take) {
    const uint32_t n01 = mul_pairs<__half>(f01, 0xE480E480u), n89 = mul_pairs<__half>(f89, 0xE480E480u);   // times -1152
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // c 2^.. as (1024 + (c + 128)) 2^.. less 1152 2^..: exact, one rounding that does nothing
            const uint32_t u0 = __byte_perm(x[0][w], x[1][w], i ? 0x7362 : 0x5140) ^ 0x80808080u;
            const uint32_t u8 = __byte_perm(x[2][w], x[3][w], i ? 0x7362 : 0x5140) ^ 0x80808080u;
            take(2 * w + i, fma_pairs(__byte_perm(u0, 0x64646464u, 0x4140), f01, n01), fma_pairs(__byte_perm(u0, 0x64646464u, 0x4342), f01, n01),
                 fma_pairs(__byte_perm(u8, 0x64646464u, 0x4140), f89, n89), fma_pairs(__byte_perm(u8, 0x64646464u, 0x4342), f89, n89));
        }
}

template <class E, int D, int NB, class Args>
__global__ void __launch_bounds__(DW * 32, rows_ctas(D, NB, std::is_same<Args, AttnArgs8>::value)) attn_rows_kernel(const __grid_constant__ Args A, const __grid_constant__ TilePlan P) {
    constexpr bool KV8 = std::is_same<Args, AttnArgs8>::value;
    using Element = typename std::conditional<KV8, int8_t, E>::type;   // of the pages
    using M = typename std::conditional<KV8, __half, E>::type;         // of the products
    using Sm = RowsSmem<D, NB, KV8>;
    constexpr int KC = D / 32, VC = D / 64;   // 16-byte chunks per lane of a K row, of a V row
    constexpr bool QS = NB > 2;
    extern __shared__ __align__(128) uint8_t rows_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(rows_raw);
    grid_launch_dependents();
    // after the tile kernel there is nothing to wait for yet: it starts this
    // kernel once the work before it has finished.  What that work wrote (lengths,
    // tables, q, pages) is then read from L2 (.cg): without a wait, a line that this
    // SM's L1 holds from before need not be fresh.  (48 x 5 tokens behind 8192: 78.5 us,
    // by L1 76.9; nothing shared, where L1 is safe, 200 x 2 tokens: 35 by L1, 37 so.)
    if (P.prefix_tiles == 0) grid_wait_prior();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int b = blockIdx.x / A.kv_heads, h = blockIdx.x - b * A.kv_heads;
    // rows r0 .. r0 + rows - 1 of the sequence and head (grid y: chunks of them)
    const int total = A.nq * A.group, chunk = (total + (int)gridDim.y - 1) / (int)gridDim.y;
    const int r0 = blockIdx.y * chunk, rows = min(chunk, total - r0);
    const int row = attn_row_of(A, A.seqs ? __ldcg(A.seqs + b) : b), len = row < 0 ? 0 : attn_cut(A, __ldcg(A.lens + row));
    const int* tab = A.table + (long long)max(row, 0) * A.table_stride;
    const long long head = (long long)h * A.kv_hs;
    const Element* kbase = static_cast<const Element*>(A.k) + head;
    const Element* vbase = static_cast<const Element*>(A.v) + head;
    const int mask = (1 << A.page_shift) - 1;

    const int all = attn_seen(A, len, small_row(A, r0));   // keys that every row sees

    const float sl2 = A.scale * LOG2E;
    const int streams = DW * gridDim.z, stream = blockIdx.z * DW + warp;
    const int blocks = (attn_seen(A, len, small_row(A, r0 + rows - 1)) + 15) >> 4;   // that the last row sees
    const bool shares = attn_shares(A, P, len);
    const int first = shares ? A.prefix >> 4 : 0;   // the prefix is a multiple of 16

    // Block i of this warp's turn into its ring; K and V rows are whole, 16 bytes
    // a lane
    constexpr int PER = 16 / (int)sizeof(Element), CH = D / PER;
    const int cc = lane % CH, cr = lane / CH;
    const uint32_t ring = smem_u32(&sm.ring[warp][0][0]);
    auto page_of = [&](int blk) -> int {
        if (blk >= blocks) return -1;
        const int* at = tab + ((blk << 4) >> A.page_shift);
        return P.prefix_tiles > 0 ? __ldcg(at) : __ldg(at);
    };
    auto fetch = [&](int blk, int page, int slot) {
        if (blk < blocks) {
            const int j = blk << 4;
            const bool there = page >= 0 && page < A.pages;
            const long long off = there ? (long long)page * A.page_stride + (long long)((j & mask) + cr) * A.kv_ts + PER * cc : 0;
            const uint32_t dst = ring + slot * Sm::SLOT;
#pragma unroll
            for (int r = 0; r < 16; r += 32 / CH) {
                const int row_ = r + cr;
                const bool in = there && j + row_ < len;
                const long long o_ = in ? off + (long long)r * A.kv_ts : 0;
                cp16(dst + k_chunk<D, KV8>(row_, cc), kbase + o_, in);
                cp16(dst + Sm::STAGE + v_chunk<D, KV8>(row_, cc), vbase + o_, in);
            }
            if constexpr (KV8) {   // the exponents: a few lanes; those past the end are zeros
                constexpr int EC = Sm::EXPS / 16;
                if (lane < 2 * EC) {
                    const int c = lane % EC;
                    const int n = there ? max(0, min(16, (len - j) * (D / 32) - 16 * c)) : 0;
                    const uint8_t* base = (lane < EC ? A.k_exps : A.v_exps) + (long long)h * A.exp_hs;
                    cp16_part(dst + 2 * Sm::STAGE + 16 * lane, n ? base + (long long)page * A.exp_page + (j & mask) * (D / 32) + 16 * c : base, n);
                }
            }
        }
        cp_commit();
    };

    // Q as the B operand: row 8 nb + g, dims 32 c + 8 t ..; zeros past the rows
    uint4 qf[QS ? 1 : NB][QS ? 1 : KC];
    auto q_part = [&](int nb, int c) {
        const int r = 8 * nb + g;
        if (r >= rows) return make_uint4(0, 0, 0, 0);
        const int tr = small_row(A, r0 + r);
        return __ldcg(reinterpret_cast<const uint4*>(static_cast<const E*>(A.q) + ((long long)b * A.nq + tr) * A.q_ts +
                                                     (long long)(h * A.group + r0 + r - tr * A.group) * A.q_hs + 8 * t + 32 * c));
    };
    if constexpr (KV8) {
        // as f16, a row divided by a power of two so that its largest value lies in 2^12 .. 2^13
        auto q_row = [&](int nb, uint4 (&f)[KC]) {
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                f[c] = q_part(nb, c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = pair_to_f32<E>(words(f[c], i));
                    top = max(top, max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu));
                }
            }
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int e = max(min((int)(top >> 23), 253), 14);   // 2^(e - 127 - 12) is taken out
            const float part = __uint_as_float((uint32_t)(254 - e) << 23) * 4096.0f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = pair_to_f32<E>(words(f[c], i));
                    h[i] = pack_pair<__half>(v.x * part, v.y * part);
                }
                f[c] = make_uint4(h[0], h[1], h[2], h[3]);
            }
            if (t == 0) sm.q_size[8 * nb + g] = __uint_as_float((uint32_t)(e - 12 + CODES_DOWN) << 23);   // (2^127 at most)
        };
        if constexpr (QS) {
            for (int nb = warp; nb < NB; nb += DW) {
                uint4 f[KC];
                q_row(nb, f);
#pragma unroll
                for (int c = 0; c < KC; ++c) sm.q[(nb * KC + c) * 32 + lane] = f[c];
            }
        } else {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) q_row(nb, qf[nb]);   // (each warp the same)
        }
        __syncthreads();
    } else if constexpr (QS) {
        for (int i = warp; i < NB * KC; i += DW) sm.q[i * 32 + lane] = q_part(i / KC, i % KC);
        __syncthreads();
    } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < KC; ++c) qf[nb][c] = q_part(nb, c);
    }
    float size[KV8 ? NB : 1][2];   // of rows 8 nb + 2t, + 1, with the scale
    if constexpr (KV8) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) size[nb][i] = sm.q_size[8 * nb + 2 * t + i] * sl2;
    }
    // p is 2^AHEAD times what the reference says, so that f16 holds smaller ones too
    constexpr float AHEAD = KV8 ? 7.0f : 0.0f;
    int v_size = 0;   // KV8: O is in steps of 2^(v_size - 127), the largest exponent of the lane's block so far
    uint32_t v_bias = (uint32_t)(-255 & 0xFFFF) * 0x00010001u;   // F16_ONE - v_size, twice (before the first block: no power at all)
    int seen[NB][2];   // keys that rows 8 nb + 2t, + 1 see
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rr = 8 * nb + 2 * t + i;
            seen[nb][i] = rr < rows ? attn_seen(A, len, small_row(A, r0 + rr)) : 0;
        }

    float m[NB][2], l[NB][2], o[NB][2 * VC * 2][4];   // o: D / 16 tiles of 16 dims x 8 rows
    // All blocks of this warp.  Without EXACT it gives up, and says so, where a block of values is
    // too small for f16 beside others: taken there and then, such blocks cost the loop 5 % where there are none
    auto all_blocks = [&](auto exact) -> bool {
        [[maybe_unused]] constexpr bool EXACT = decltype(exact)::value;
        int blk = first + stream, page = page_of(blk);
#pragma unroll
        for (int i = 0; i < Sm::STAGES - 1; ++i) {
            const int next = page_of(blk + (i + 1) * streams);
            fetch(blk + i * streams, page, i);
            page = next;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = -INFINITY;
            l[nb][0] = l[nb][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nb][i][j] = 0.0f;
        }
        for (int n = 0; blk < blocks; blk += streams, ++n) {
            const int j = blk << 4, ahead = blk + (Sm::STAGES - 1) * streams;
            const int next = page_of(ahead + streams);
            cp_wait<Sm::STAGES - 2>();
            __syncwarp();   // the block is there, and the slot of the one before has been read
            fetch(ahead, page, (n + Sm::STAGES - 1) % Sm::STAGES);
            page = next;
            const uint8_t* ks = &sm.ring[warp][n % Sm::STAGES][0];
            const uint8_t* vs = ks + Sm::STAGE;
            float s[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.0f;
            if constexpr (KV8) {
                // keys g and g + 8; a block of 32 dims has its own power of two
                uint32_t e[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t* at = vs + Sm::STAGE + (g + 8 * i) * (D / 32);
                    e[i] = D == 128 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
                }
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const uint8_t* at = ks + k_chunk<D, true>(g, 2 * c + (t >> 1)) + 8 * (t & 1);
                    const uint2 k0 = *reinterpret_cast<const uint2*>(at), k1 = *reinterpret_cast<const uint2*>(at + 8 * D);
                    uint32_t a[2][4];   // of two products: rows g, g + 8, then both again
                    codes_down(k0.x, a[0][0], a[0][2]);
                    codes_down(k1.x, a[0][1], a[0][3]);
                    codes_down(k0.y, a[1][0], a[1][2]);
                    codes_down(k1.y, a[1][1], a[1][3]);
                    const float f0 = __uint_as_float((e[0] >> (8 * c) & 0xFFu) << 23), f1 = __uint_as_float((e[1] >> (8 * c) & 0xFFu) << 23);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const uint4 qv = QS ? sm.q[(nb * KC + c) * 32 + lane] : qf[QS ? 0 : nb][QS ? 0 : c];
                        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma16816<M>(x, a[0][0], a[0][1], a[0][2], a[0][3], qv.x, qv.y);
                        mma16816<M>(x, a[1][0], a[1][1], a[1][2], a[1][3], qv.z, qv.w);
                        s[nb][0] = fmaf(x[0], f0, s[nb][0]);
                        s[nb][1] = fmaf(x[1], f0, s[nb][1]);
                        s[nb][2] = fmaf(x[2], f1, s[nb][2]);
                        s[nb][3] = fmaf(x[3], f1, s[nb][3]);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const int at = k_chunk<D, false>(g, 4 * c + t);
                    const uint4 k0 = *reinterpret_cast<const uint4*>(ks + at), k1 = *reinterpret_cast<const uint4*>(ks + at + 16 * D);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const uint4 qv = QS ? sm.q[(nb * KC + c) * 32 + lane] : qf[QS ? 0 : nb][QS ? 0 : c];
                        mma16816<E>(s[nb], k0.x, k1.x, k0.y, k1.y, qv.x, qv.y);
                        mma16816<E>(s[nb], k0.z, k1.z, k0.w, k1.w, qv.z, qv.w);
                    }
                }
            }
            const bool part = j + 16 > all;
            bool raise = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[nb][i] *= KV8 ? size[KV8 ? nb : 0][i & 1] : sl2;
                    if (part && j + g + 8 * (i >> 1) >= seen[nb][i & 1]) s[nb][i] = -INFINITY;
                    raise |= s[nb][i] > m[nb][i & 1] + RAISE;
                }
            if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = fmaxf(s[nb][i], s[nb][i + 2]);
#pragma unroll
                        for (int of = 4; of < 32; of <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, of));
                        const float mn = fmaxf(m[nb][i], x), keep = mn == -INFINITY ? 1.0f : ex2(m[nb][i] - mn);
                        m[nb][i] = mn;
                        l[nb][i] *= keep;
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            o[nb][k][i] *= keep;
                            o[nb][k][i + 2] *= keep;
                        }
                    }
            }
            uint32_t pb[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float base = m[nb][i & 1] == -INFINITY ? 0.0f : m[nb][i & 1] - AHEAD;   // a row without keys so far
                    p[i] = ex2(s[nb][i] - base);
                    l[nb][i & 1] += p[i];
                }
                // rounded to the cache's type (attn.cuh); l has the whole p
                pb[nb][0] = transpose8x8(pack_pair<M>(p[0], p[1]));
                pb[nb][1] = transpose8x8(pack_pair<M>(p[2], p[3]));
            }
            if constexpr (KV8) {
                constexpr int WORDS = D / 32;
                uint32_t v[4][WORDS], e[4];
                bring_codes<D>(vs, t, g, v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    e[i] = vs[Sm::STAGE + Sm::EXPS + (2 * t + (i & 1) + 8 * (i >> 1)) * (D / 32) + (D == 128 ? g >> 1 : g >> 2)];
                // f: the rows' powers of two in f16, 2^(e - v_size), as exponents of f16 where they are normal there
                const uint32_t e01 = __byte_perm(e[0], e[1], 0x5410), e89 = __byte_perm(e[2], e[3], 0x5410);
                const uint32_t x01 = __viaddmax_s16x2_relu(e01, v_bias, 0), x89 = __viaddmax_s16x2_relu(e89, v_bias, 0);
                uint32_t f01 = x01 << 10, f89 = x89 << 10;
                bool small = false;
                if (__any_sync(0xFFFFFFFFu, ((x01 | x89) & 0xFFF0FFF0u) | (((x01 - 0x00010001u) | (x89 - 0x00010001u)) & 0x80008000u))) {
                    // a larger block than before, one that is no exponent of f16, or zeros (rare)
                    int most = max(max(e[0], e[1]), max(e[2], e[3]));
                    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                    if (__any_sync(0xFFFFFFFFu, most > v_size)) {
                        const float keep = most > v_size ? ex2((float)(v_size - most)) : 1.0f;
                        v_size = max(most, v_size);
                        v_bias = (uint32_t)((F16_ONE - v_size) & 0xFFFF) * 0x00010001u;
                        f01 = __viaddmax_s16x2_relu(e01, v_bias, 0) << 10;
                        f89 = __viaddmax_s16x2_relu(e89, v_bias, 0) << 10;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[nb][k][i] *= keep;
                    }
                    int least = 255;
#pragma unroll
                    for (int i = 0; i < 4; ++i) least = min(least, e[i] ? (int)e[i] : 255);
                    if (__builtin_expect(__any_sync(0xFFFFFFFFu, least < v_size - F16_ONE + 1), 0)) {
                        small = __any_sync(0xFFFFFFFFu, least < v_size - V_LEAST);
                        if (!EXACT && small) return false;
                        f01 = pack_pair<__half>(power_below(e[0], v_size), power_below(e[1], v_size));
                        f89 = pack_pair<__half>(power_below(e[2], v_size), power_below(e[3], v_size));
                    }
                }
                value_fragments<D>(v, f01, f89, [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma16816<M>(o[nb][k], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
                });
                if (EXACT && small) {
                    // blocks too small for that: by themselves, relative to the largest of them, then of those still left
                    int left = v_size - V_LEAST;   // exponents below
#pragma unroll 1
                    for (;;) {
                        asm volatile("" ::: "memory");   // (the codes once more, from shared memory: kept in registers they cost every block)
                        uint32_t again[4][WORDS];
                        bring_codes<D>(vs, t, g, again);
                        int top = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = max(top, (int)e[i] < left ? (int)e[i] : 0);
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                        if (!__any_sync(0xFFFFFFFFu, top > 0)) break;
                        const float back = ex2((float)(top - v_size));
                        float f[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[i] = (int)e[i] < left ? power_below(e[i], top) : 0.0f;
                        value_fragments<D>(again, pack_pair<__half>(f[0], f[1]), pack_pair<__half>(f[2], f[3]), [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma16816<M>(y, a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[nb][k][i] = fmaf(y[i], back, o[nb][k][i]);
                            }
                        });
                        left = top - V_LEAST;
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                    uint4 vf[4];   // rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        vf[i] = *reinterpret_cast<const uint4*>(vs + v_chunk<D, false>(2 * t, 8 * c + g) + ((i & 1) + 8 * (i >> 1)) * (2 * D));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // dims 64 c + 8 g + 2 i, + 1
                        const uint32_t w0 = words(vf[0], i), w1 = words(vf[1], i), w2 = words(vf[2], i), w3 = words(vf[3], i);
                        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
                        const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma16816<E>(o[nb][4 * c + i], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
                    }
                }
            }
        }
        return true;
    };
    if (__builtin_expect(!all_blocks(std::false_type()) && KV8, 0)) {
        cp_wait<0>();
        __syncwarp();   // all that was brought has been read
        if constexpr (KV8) all_blocks(std::true_type());
    }
    cp_wait<0>();
    __syncthreads();   // the rings make room for the parts

    // this warp's part.  8-bit pages: with a power of two taken out of l and O that leaves l
    // between 1 and 2, so that O, in steps of the values again, is no larger than they are
    const float o_step = KV8 ? __uint_as_float((uint32_t)v_size << 23) : 1.0f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int of = 4; of < 32; of <<= 1) l[nb][i] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][i], of);
            float step = 1.0f;
            if constexpr (KV8) {
                const int e = l[nb][i] == 0.0f ? 127 : min((int)(__float_as_uint(l[nb][i]) >> 23), 253);
                const float part = __uint_as_float((uint32_t)(254 - e) << 23);
                m[nb][i] += (float)(e - 127) - AHEAD;
                l[nb][i] *= part;
                step = part * o_step;
            }
            if (g == 0) {
                sm.part.m[warp][8 * nb + 2 * t + i] = m[nb][i];
                sm.part.l[warp][8 * nb + 2 * t + i] = l[nb][i];
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                *reinterpret_cast<float2*>(&sm.part.o[warp][8 * nb + 2 * t + i][KV8 ? (D / 8) * g + 2 * k : 64 * (k >> 2) + 8 * g + 2 * (k & 3)]) =
                    make_float2(o[nb][k][i] * step, o[nb][k][i + 2] * step);
        }
    }
    const int cs = gridDim.z;   // the cluster: the CTAs of this pair
    // CTA z of it adds up rows z, z + cs, ..
    constexpr int ROWS2 = NB == 1 ? 8 : NB == 2 ? 16 : 32;   // rows, to a power of two
    const int mine = (rows - (int)blockIdx.z + cs - 1) / cs, parts = cs * DW;
    auto& sums = sm.part.sums;
    if ((int)threadIdx.x < mine) {
        const int k = threadIdx.x, r = r0 + blockIdx.z + k * cs, gr = b * total + r, t_ = small_row(A, r);
        sums.place(A, k, (long long)b * A.nq + t_, h * A.group + r - t_ * A.group);
        sums.pieces[0][k] = Pieces{0, 0, 0, 0};
        if (shares) {
            const int rt = gr >> P.tile_shift, item = h * P.prefix_row_tiles + rt;
            sums.pieces[0][k] = item_pieces(P, item, item * P.prefix_tiles, P.prefix_tiles,
                                            A.kv_heads * P.prefix_row_tiles * P.prefix_tiles, gr & (P.tile_rows - 1));
        }
    }
    if (cs > 1) cluster_barrier();
    else __syncthreads();
    if (P.prefix_tiles > 0) grid_wait_prior();   // the tile kernel's results
    {   // a thread per (row, every so manieth part)
        constexpr int SPAN = (DW * 32) / ROWS2;
        const int k = threadIdx.x % ROWS2, from = threadIdx.x / ROWS2;
        if (k < mine) {
            const int r = blockIdx.z + k * cs;
            bring(P, sums.pieces[0][k], sums.ml + parts, k, from, SPAN);
            for (int p = from; p < parts; p += SPAN)
                sums.ml[p][k] = make_float2(peer_f32(&sm.part.m[p % DW][r], p / DW), peer_f32(&sm.part.l[p % DW][r], p / DW));
        }
    }
    __syncthreads();
    for (int k0 = 0; k0 < mine; k0 += DW * 4) {
        const int k = min(k0 + (int)threadIdx.x / 8, mine - 1);
        weigh(A, sums, k, parts + sums.pieces[0][k].n, k0 + (int)threadIdx.x / 8 < mine, threadIdx.x & 7);
    }
    __syncthreads();
    constexpr int N = NB == 1 ? 1 : 2;   // 8 rows at most fill the threads once or twice
#pragma unroll 1
    for (int e0 = threadIdx.x; e0 < mine * (D / 4); e0 += N * DW * 32) {
        int k[N], d[N];
        float4 acc[N];
        const Pieces* X[N];
        const float2* w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = min(e0 + i * DW * 32, mine * (D / 4) - 1);
            k[i] = e / (D / 4);
            d[i] = 4 * (e % (D / 4));
            X[i] = &sums.pieces[0][k[i]];
            w[i] = &sums.ml[parts][k[i]];
            acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll 4
        for (int p = 0; p < parts; ++p)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float f = sums.ml[p][k[i]].x;
                const float4 v = peer_f32x4(&sm.part.o[p % DW][blockIdx.z + k[i] * cs][d[i]], p / DW);
                if (f != 0.0f) {
                    acc[i].x = fmaf(f, v.x, acc[i].x);
                    acc[i].y = fmaf(f, v.y, acc[i].y);
                    acc[i].z = fmaf(f, v.z, acc[i].z);
                    acc[i].w = fmaf(f, v.w, acc[i].w);
                }
            }
        if (shares) add_pieces<D, Sm::ROWS>(P, X, w, d, acc);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i * DW * 32 < mine * (D / 4)) {
                const float inv = sums.inv[k[i]];
                attn_store4<E>(A, sums.out[k[i]] + d[i], make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
            }
    }
    if (cs > 1) cluster_barrier();   // no CTA leaves while its part is read
}

template <class E, int D, int NB, class Args>
cudaError_t rows_launch(const Args& A, const TilePlan& P, int chunks, int cs, cudaStream_t stream) {
    const dim3 grid((unsigned)(A.batch * A.kv_heads), (unsigned)chunks, (unsigned)cs);
    using Sm = RowsSmem<D, NB, std::is_same<Args, AttnArgs8>::value>;
    constexpr int bytes = sizeof(Sm);
    static_assert(offsetof(Sm, ring) % 128 == 0 && Sm::SLOT % 16 == 0, "the rings' alignment");
    static_assert(rows_ctas(D, NB, std::is_same<Args, AttnArgs8>::value) * (bytes + 1024) <= 228 * 1024, "the CTAs of an SM");
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<E, D, NB, Args>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    if (cs == 1) return launch_kernel(attn_rows_kernel<E, D, NB, Args>, grid, dim3(DW * 32), bytes, stream, A, P);
    return launch_kernel_cluster(attn_rows_kernel<E, D, NB, Args>, grid, dim3(DW * 32), bytes, stream, (unsigned)cs, A, P);
}

template <class E, int D, class Args>
cudaError_t rows_nb(const Args& A, const TilePlan& P, int chunks, int cs, cudaStream_t stream) {
    const int rows = (A.nq * A.group + chunks - 1) / chunks;
    if (rows <= 8) return rows_launch<E, D, 1, Args>(A, P, chunks, cs, stream);
    if (rows <= 16) return rows_launch<E, D, 2, Args>(A, P, chunks, cs, stream);
    return rows <= 24 ? rows_launch<E, D, 3, Args>(A, P, chunks, cs, stream) : rows_launch<E, D, 4, Args>(A, P, chunks, cs, stream);
}

}  // namespace

// CTAs of a pair for a launch (attn_rows.cu).
int rows_cluster(const AttnArgs& A, int d, int chunks, int keys, bool kv8);

template <class Args>
cudaError_t rows_any(const Args& A, const TilePlan* plan, int type, int d, cudaStream_t stream) {
    const TilePlan P = plan ? *plan : TilePlan{};
    const int chunks = (A.nq * A.group + 31) / 32, cs = rows_cluster(A, d, chunks, plan ? A.cap - A.prefix : A.cap, std::is_same<Args, AttnArgs8>::value);
    if (type == PLM_F16) return d == 64 ? rows_nb<__half, 64>(A, P, chunks, cs, stream) : rows_nb<__half, 128>(A, P, chunks, cs, stream);
    return d == 64 ? rows_nb<__nv_bfloat16, 64>(A, P, chunks, cs, stream) : rows_nb<__nv_bfloat16, 128>(A, P, chunks, cs, stream);
}

}  // namespace plm

// Paged attention on the 5th-generation tensor cores (tcgen05): the shared
// prefix for all rows of a batch at once, and prompts.
//
// Mathematics.  A row tile is 128 query rows of one key/value head (of any
// sequences for the prefix; of one sequence otherwise).  Per unit of 128 keys
//   S = Q K^T (f32, tensor memory), P = 2^(scale log2 e S - m), O += P V,
// with a running reference m per row that is raised (O and l scaled) only
// when a score exceeds it by more than 2^8.  The sum l is of the unrounded p.
//
// Roles.  NT row tiles share the K and V tiles of a CTA (NT = 2 when there are
// that many rows: half the shared-memory traffic per product).  Per row tile a
// warpgroup, one thread per row (= TMEM lane): reads S, writes P over it, and
// at the end of a piece reads O.  One warp brings the pages' rows in by TMA (one
// box per page and 64 dims; pages out of range read as zeros), one issues the
// MMAs.  For NT = 2 the products of one tile run while the other tile's
// softmax does; for NT = 1 two S buffers do the same.
//   TMEM columns: S 0..255 (two buffers of 128), O 256.. (NT x D).
//   V is the MN-major operand as it lies in the page ([key][dim]); P is the
//   A operand in tensor memory.
//
// Work: equal shares of units per CTA (attn_tile.cuh), one CTA per SM.
// Bound: the tensor cores from ~270 rows per head on, HBM below.  Every wait
// is bounded; one that runs out records a fault and the kernel winds down.
// One GB300, bf16, 32 query heads on 8 of 128: 8 x 509 tokens behind 16384, 820 us
// (1.37 PFLOP/s with the join), 8192 tokens behind nothing 1000 us; 256 tokens' prefix of 32768, 115 us (1.2 PFLOP/s).
// The tensor pipe then waits for the starts and ends of pieces.
#include <cuda.h>

#include <cstring>

#include "attn_tile.cuh"

namespace plm {

namespace {

constexpr float RAISE = 8.0f, LOG2E = 1.4426950408889634f;
constexpr uint32_t TM_S = 0, TM_O = 256;   // TMEM columns

template <int D, int NT> struct TileSmem {
    static constexpr int HALF = 128 * 128;               // 128 rows x 64 values, 128-byte swizzle
    static constexpr int QTILE = (D / 64) * HALF, STAGE = (D / 64) * HALF;
    static constexpr int SLOTS = D == 64 ? 10 : NT == 2 ? 5 : 6;
    static constexpr int RING = NT * QTILE;
    static constexpr int BAR = RING + SLOTS * STAGE;
    // full, empty per slot; S ready, P ready, O done, Q ready, warps together per buffer
    static constexpr int NBAR = 2 * SLOTS + 10;
    static constexpr int TMEMP = BAR + 8 * NBAR;
    static constexpr int ALLOC = TMEMP + 16 + 1024;
    static_assert(ALLOC <= 227 * 1024, "shared memory");
};

// Low word of a shared-memory operand's descriptor: address and leading offset
// in units of 16 bytes.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) {
    return ((saddr >> 4) & 0x3FFF) | ((lead >> 4) << 16);
}
template <class E> struct KindOf;
template <> struct KindOf<__half> { static constexpr uint32_t AB = 0; };
template <> struct KindOf<__nv_bfloat16> { static constexpr uint32_t AB = (1u << 7) | (1u << 10); };
template <class E> __host__ __device__ constexpr uint32_t idesc(uint32_t n, bool b_mn) {
    return (1u << 4) | KindOf<E>::AB | (b_mn ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// The MMAs.  All lanes of the warp execute the code around them, so that the
// operands stay in uniform registers, and one lane (`lead`) issues: in a
// branch of one lane every operand is moved over, and an MMA took ~95 cycles
// to issue instead of the 64 it takes to run (prompts 456 -> 395 us).
// Operands in shared memory are given by the low words of their descriptors;
// the high word is the same for all.
#define PLM_DESC_HI "0x40004040"
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t lead) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "mov.b64 da, {%1, " PLM_DESC_HI "};\n\tmov.b64 db, {%2, " PLM_DESC_HI "};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(lead) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t lead) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "mov.b64 db, {%2, " PLM_DESC_HI "};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(lead) : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define PLM_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define PLM_R16(r, i) PLM_R4(r, i), PLM_R4(r, i + 4), PLM_R4(r, i + 8), PLM_R4(r, i + 12)
#define PLM_I4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
#define PLM_I16(r, i) PLM_I4(r, i), PLM_I4(r, i + 4), PLM_I4(r, i + 8), PLM_I4(r, i + 12)
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : PLM_R16(r, 0), PLM_R16(r, 16) : "r"(a));
}
// Eight columns, loaded at once; stored.
__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : PLM_R4(r, 0), PLM_R4(r, 4) : "r"(a) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(a), PLM_I4(r, 0), PLM_I4(r, 4) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 :: "r"(a), PLM_I16(r, 0), PLM_I16(r, 16) : "memory");
}
// Waits for the loads before it; names the registers of one so that nothing
// uses them earlier.
#define PLM_W4(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3])
#define PLM_W16(r, i) PLM_W4(r, i), PLM_W4(r, i + 4), PLM_W4(r, i + 8), PLM_W4(r, i + 12)
__device__ __forceinline__ void tmem_ld_wait(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : PLM_W16(r, 0), PLM_W16(r, 16) :: "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int token, int head, int page,
                                        uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 :: "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(token), "r"(head), "r"(page), "r"(smem_u32(bar))
                 : "memory");
}
// Two f32 in one 64-bit register.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A piece: consecutive units of one item.
struct Piece {
    bool begins, whole;
    int b, rt, h;       // sequence (own), row tile, head
    int key0, keys;     // first key of the piece; end of the keys to load (own: that its rows see)
    int tiles;
    int row;            // table row, or -1
    int item;
    int unit0;          // the item's first unit
};

// Walks the CTA's share of the units; every warp for itself, by all its lanes.
// (Outside the loops over units little is unrolled: a CTA runs that code once or
// twice, and most of its cost is to fetch it.)
struct Walk {
    int u, end;        // the next unit, the end of the share
    int prefix_row;    // prefix: table row that holds it
    int b, rt, T, h;   // own: sequence, row tile, its units per head, head
    int item_u0;       // own: first unit of the item

    // Returns the number of all units.  tables: page tables will be read.
    __device__ int start(const AttnArgs& A, const TilePlan& P, int lane, bool tables) {
        int U;
        if (P.job == 0) {
            U = A.kv_heads * P.prefix_row_tiles * P.prefix_tiles;
        } else {
            int sum = 0;
            for (int b = lane; b < A.batch; b += 32) sum += seq_tiles(A, P, attn_len(A, attn_row(A, b)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            U = sum * A.kv_heads;
        }
        const int ctas = unit_ctas(P, U);
        const bool mine = (int)blockIdx.x < ctas;
        u = mine ? (int)((long long)U * blockIdx.x / ctas) : U;
        end = mine ? (int)((long long)U * (blockIdx.x + 1) / ctas) : U;
        b = prefix_row = -1;
        rt = T = h = item_u0 = 0;
        if (P.job == 0 && tables)   // the first sequence that takes part
            for (int b0 = 0; b0 < A.batch && prefix_row < 0; b0 += 32) {
                const int b = b0 + lane, row = b < A.batch ? attn_row(A, b) : -1;
                const unsigned hit = __ballot_sync(0xFFFFFFFFu, row >= 0 && attn_shares(A, P, attn_len(A, row)));
                if (hit) prefix_row = __shfl_sync(0xFFFFFFFFu, row, __ffs(hit) - 1);
            }
        return U;
    }

    // The sequence, row tile, head and item of own unit u.
    __device__ void locate(const AttnArgs& A, const TilePlan& P, int lane) {
        int acc = 0;
        for (int b0 = 0; b0 < A.batch; b0 += 32) {
            const int n = b0 + lane < A.batch ? seq_tiles(A, P, attn_len(A, attn_row(A, b0 + lane))) : 0;
            int x = n * A.kv_heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, acc + x > u);
            if (hit) {
                const int w = __ffs(hit) - 1;
                b = b0 + w;
                int first = acc + __shfl_sync(0xFFFFFFFFu, x, w) - __shfl_sync(0xFFFFFFFFu, n, w) * A.kv_heads;
                for (rt = 0;; ++rt) {   // ends: u lies in one of the sequence's row tiles
                    T = own_tiles(A, P, b * P.own_row_tiles + rt);
                    if (u - first < T * A.kv_heads) break;
                    first += T * A.kv_heads;
                }
                h = (u - first) / T;
                item_u0 = first + h * T;
                return;
            }
            acc += __shfl_sync(0xFFFFFFFFu, x, 31);
        }
    }

    __device__ bool next(const AttnArgs& A, const TilePlan& P, int lane, Piece& S) {
        if (u >= end) return false;
        if (P.job == 0) {
            S.item = u / P.prefix_tiles;
            const int t0 = u - S.item * P.prefix_tiles;
            S.b = 0;
            S.h = S.item / P.prefix_row_tiles;
            S.rt = S.item - S.h * P.prefix_row_tiles;
            S.tiles = min(P.prefix_tiles - t0, end - u);
            S.unit0 = u - t0;
            S.begins = t0 == 0;
            S.whole = S.begins && S.tiles == P.prefix_tiles;
            S.key0 = t0 * TK;
            S.keys = A.prefix;
            S.row = prefix_row;
        } else {
            if (b < 0) locate(A, P, lane);
            else if (u == item_u0 + T) {   // the next item
                item_u0 = u;
                if (++h == A.kv_heads) {
                    h = 0;
                    do {   // u < end <= U: there is one
                        if (++rt == P.own_row_tiles) { rt = 0; ++b; }
                        T = own_tiles(A, P, b * P.own_row_tiles + rt);
                    } while (T == 0);
                }
            }
            const int t0 = u - item_u0;
            S.b = b;
            S.rt = rt;
            S.h = h;
            S.row = attn_row(A, S.b);
            const int len = attn_len(A, S.row);
            S.tiles = min(T - t0, end - u);
            S.unit0 = item_u0;
            S.begins = t0 == 0;
            S.whole = S.begins && S.tiles == T;
            S.key0 = own_begin(A, P, len) + t0 * TK;
            S.keys = own_end(A, P, len, S.rt);
            S.item = A.kv_heads * (b * P.own_row_tiles + rt) + h;
        }
        u += S.tiles;
        return true;
    }
};

// Row i of a piece's row tile: the token (row of q) and query head, or false.
__device__ __forceinline__ bool tile_row(const AttnArgs& A, const TilePlan& P, const Piece& S, int i, long long& tok,
                                         int& qh) {
    const unsigned r = ((unsigned)S.rt << P.tile_shift) + i;   // the rows fit 31 bits
    if (r >= (unsigned)(A.nq * A.group * (P.job == 0 ? A.batch : 1))) return false;
    const unsigned t = r / (unsigned)A.group;
    tok = (long long)S.b * A.nq + t;
    qh = S.h * A.group + (int)(r - t * A.group);
    return true;
}

// A bounded wait of a whole warp: all its lanes go on or none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
}

template <class E, int D, int NT>
__global__ void __launch_bounds__(NT * 128 + 64, 1)
attn_tile_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ TilePlan P,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, unsigned* fault) {
    using L = TileSmem<D, NT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BAR);
    uint64_t* empty = full + L::SLOTS;
    uint64_t* s_ready = empty + L::SLOTS;   // [2] per S buffer
    uint64_t* p_ready = s_ready + 2;        // [2] per S buffer, one arrival per warp
    uint64_t* o_done = p_ready + 2;         // [2] per row tile: a PV product has finished
    uint64_t* q_ready = o_done + 2;         // [2] per row tile
    uint64_t* together = q_ready + 2;       // [2] per row tile: its four warps
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::TMEMP);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int TMA_WARP = 4 * NT, MMA_WARP = 4 * NT + 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * L::SLOTS; ++i) mbar_init(&full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_ready[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&o_done[i], 1);
            mbar_init(&q_ready[i], 4);
            mbar_init(&together[i], 4);
        }
        fence_barrier_init();
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    // the kernels before this one have finished; only then may the next one
    // start, which reads what they wrote before it waits for this one
    grid_wait_prior();
    grid_launch_dependents();
    bool ok = true;
    Walk W;
    Piece S;
    if (warp == TMA_WARP) {
        const int U = W.start(A, P, lane, true);
        bool first = true;
        // ---------------------------------------------------- pages -> K, V
        const int bt = min(1 << A.page_shift, TK), per = TK / bt;   // tokens per box, boxes per 64 dims
        int n = 0;                                                  // tiles loaded: slot n % SLOTS
        const int part = lane / per, box = lane - part * per;
        const bool active = part < D / 64;
        // (goes on without loads once a wait has run out: the sums that follow find their
        // places by what is written here for each item)
        while (W.next(A, P, lane, S)) {
            const int* tab = A.table + (long long)max(S.row, 0) * A.table_stride;
            if (P.job == 1 && lane == 0) {
                if (P.keep) {
                    if (S.begins) P.item_unit[S.item] = S.unit0;
                } else if (first) {
                    P.cut[blockIdx.x] = make_int4(S.begins ? -1 : S.b * P.own_row_tiles + S.rt, S.h, S.unit0, W.T);
                }
            }
            first = false;
            // The first piece's Q comes before the ring is filled: 160 KB an SM are
            // 4 us of HBM, and Q, the code and the constants would queue behind them
            if (n == 0)
                for (int t = 0; ok && t < NT; ++t) ok = warp_wait(&q_ready[t], 0);
            for (int i = 0; ok && i < S.tiles; ++i) {
                const int j = S.key0 + i * TK + box * bt;
                int page = A.pages;   // out of range: the box is filled with zeros
                if (active && S.row >= 0 && j < S.keys) {
                    const int p = __ldg(tab + (j >> A.page_shift));
                    if (p >= 0 && p < A.pages) page = p;
                }
                const int token = j & ((1 << A.page_shift) - 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int slot = n % L::SLOTS;
                    if (n >= L::SLOTS) ok = warp_wait(&empty[slot], (n / L::SLOTS - 1) & 1);
                    if (!ok) break;
                    uint8_t* dst = sm + L::RING + slot * L::STAGE;
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], L::STAGE);
                    __syncwarp();
                    if (active)
                        tma_box(dst + part * L::HALF + box * bt * 128, kv ? &vmap : &kmap, 64 * part, token, S.h, page,
                                &full[slot]);
                }
            }
        }
        if (!ok)   // wind down: this CTA's copies have to land before it ends
            for (int i = max(0, n - L::SLOTS); i < n; ++i) mbar_wait(&full[i % L::SLOTS], (i / L::SLOTS) & 1);
        if (P.job == 1 && lane == 0) {
            if (blockIdx.x == 0) *P.units = U;
            if (first && !P.keep) P.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);   // no units
        }
    } else if (warp == MMA_WARP) {
        W.start(A, P, lane, false);
        // ------------------------------------------------------- the products
        constexpr uint32_t ID_S = idesc<E>(128, false), ID_O = idesc<E>(D, true);
        // the operands' descriptors; a place in shared memory adds bytes / 16
        const uint32_t qd = desc_lo(smem_u32(sm), 16), kd = desc_lo(smem_u32(sm + L::RING), 16),
                       vd = desc_lo(smem_u32(sm + L::RING), L::HALF);
        uint32_t leader;
        asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
        int n = 0;            // tiles taken from the ring
        int step = 0;         // units so far (all pieces)
        int pieces = 0;
        // S of row tile t (buffer sb) from the K tile in slot
        auto product_s = [&](int t, int sb, int slot) {
            const uint32_t a = qd + t * (L::QTILE / 16), b = kd + (uint32_t)slot * (L::STAGE / 16);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k >> 2) * L::HALF + (k & 3) * 32) / 16;
                mma_ss(tmem + TM_S + 128 * sb, a + off, b + off, ID_S, k > 0, leader);
            }
            if (leader) commit(&s_ready[sb]);
            __syncwarp();
        };
        auto product_o = [&](int t, int sb, int slot, bool first, bool last) {
            const uint32_t b = vd + (uint32_t)slot * (L::STAGE / 16);
            const uint32_t p = tmem + TM_S + 128 * sb, o = tmem + TM_O + D * t;
            mma_ts(o, p, b, ID_O, !first, leader);
#pragma unroll
            for (int k = 1; k < TK / 16; ++k) mma_ts(o, p + 8 * k, b + k * (2048 / 16), ID_O, 1, leader);
            if (leader && (NT == 1 || last)) commit(&o_done[t]);
            __syncwarp();
        };
        auto free_slot = [&](int slot) {
            if (leader) commit(&empty[slot]);
            __syncwarp();
        };
        while (ok && W.next(A, P, lane, S)) {
            // unit i of the piece: K is ring tile n0 + 2 i, V the next one
            const int n0 = n;
            n += 2 * S.tiles;
            auto wait_full = [&](int at) { return warp_wait(&full[at % L::SLOTS], (at / L::SLOTS) & 1); };
            for (int t = 0; ok && t < NT; ++t) ok = warp_wait(&q_ready[t], pieces & 1);
            if (ok) ok = wait_full(n0);
            if (!ok) break;
            tc_after();
#pragma unroll 1
            for (int t = 0; t < NT; ++t) product_s(t, NT == 2 ? t : step & 1, n0 % L::SLOTS);
            free_slot(n0 % L::SLOTS);
            for (int i = 0; ok && i < S.tiles; ++i, ++step) {
                const int vt = n0 + 2 * i + 1, kt = vt + 1;
                const bool more = i + 1 < S.tiles;
                if (NT == 1 && more) {   // the next S into the other buffer, before waiting for P
                    ok = wait_full(kt);
                    if (!ok) break;
                    tc_after();
                    product_s(0, (step + 1) & 1, kt % L::SLOTS);
                    free_slot(kt % L::SLOTS);
                }
                if (NT == 1) ok = wait_full(vt);
                if (!ok) break;
                const int left = S.keys - (S.key0 + i * TK);
#pragma unroll 1
                for (int t = 0; t < NT; ++t) {
                    const int sb = NT == 2 ? t : step & 1;
                    // P of this unit; for NT = 2 its arrivals also say that V and the next K have landed
                    ok = warp_wait(&p_ready[sb], NT == 2 ? step & 1 : (step >> 1) & 1);
                    if (!ok) break;
                    tc_after();
                    if (t == 0 && P.job == 1 && left < TK) {
                        // the pages' rows past the end may hold anything, and 0 * NaN is NaN
                        uint8_t* v = sm + L::RING + (vt % L::SLOTS) * L::STAGE;
                        for (int e = lane; e < (TK - left) * (D / 8); e += 32) {
                            const int r = left + e / (D / 8), c = e % (D / 8);
                            *reinterpret_cast<uint4*>(v + (c >> 3) * L::HALF + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                    product_o(t, sb, vt % L::SLOTS, i == 0, !more);
                    if (t == NT - 1) free_slot(vt % L::SLOTS);
                    if (NT == 2 && more) {
                        product_s(t, t, kt % L::SLOTS);
                        if (t == NT - 1) free_slot(kt % L::SLOTS);
                    }
                }
            }
            ++pieces;
        }
    } else {
        W.start(A, P, lane, false);
        // ------------------------------------- the softmax, a row per thread
        const int t = warp >> 2, i = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // a scale of 0 counts as 1e-30: every finite score then is as good as 0, and
        // -inf (a hidden key, a row's first maximum) stays -inf
        const float sl2 = fmaxf(fabsf(A.scale) * LOG2E, 1e-30f), raise_at = RAISE / sl2;
        int step = 0;   // units so far
        int pieces = 0;
        long long tok;
        int qh;
        // This warp's 32 rows of Q into the operand tile, whole rows at a time (a
        // row per thread instead costs 7 k cycles a piece, four times as much); a
        // negative scale turns its signs
        auto load_q = [&](const Piece& C) {
            const bool in = tile_row(A, P, C, t * 128 + i, tok, qh);
            const long long mine = in ? tok * A.q_ts + (long long)qh * A.q_hs : -1;
            const uint32_t sign = A.scale < 0.0f ? 0x80008000u : 0u;
            constexpr int CH = D / 8, AT = 32 / CH;   // 16-byte chunks of a row, rows at a time
            const int c = lane % CH;
            uint8_t* dst = sm + t * L::QTILE + (c >> 3) * L::HALF;
#pragma unroll 1
            for (int k0 = 0; k0 < 32 / AT; k0 += 8) {   // eight loads in flight
                uint4 v[8];
                bool have_row[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const long long off = __shfl_sync(0xFFFFFFFFu, mine, (k0 + k) * AT + lane / CH);
                    have_row[k] = off >= 0;
                    v[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const E*>(A.q) + (off >= 0 ? off : 0)) + c);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = (k0 + k) * AT + lane / CH;
                    uint4 u = have_row[k] ? v[k] : make_uint4(0, 0, 0, 0);
                    u.x ^= sign; u.y ^= sign; u.z ^= sign; u.w ^= sign;
                    *reinterpret_cast<uint4*>(dst + (32 * (warp & 3) + r) * 128 + (((c ^ r) & 7) << 4)) = u;
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready[t]);
        };
        bool have = W.next(A, P, lane, S);
        while (have && ok) {
            load_q(S);
            Piece next;   // worked out while the first S is on its way
            const bool more = W.next(A, P, lane, next);
            const bool in = tile_row(A, P, S, t * 128 + i, tok, qh);
            int seen = S.keys;   // keys that the row sees
            if (P.job == 1 && in) seen = attn_seen(A, attn_len(A, S.row), (int)(tok - (long long)S.b * A.nq));
            float m = -INFINITY, l = 0.0f;   // m in units of S
            for (int u = 0; ok && u < S.tiles; ++u, ++step) {
                const int sb = NT == 2 ? t : step & 1;
                if (NT == 2 && (warp & 3) == 0) {
                    // while S is on its way: V of this unit and the next K of the piece (a wait of
                    // the MMA warp leaves the tensor cores idle, one here does not)
                    const int vt = 2 * step + 1;
                    ok = warp_wait(&full[vt % L::SLOTS], (vt / L::SLOTS) & 1);
                    if (ok && u + 1 < S.tiles) ok = warp_wait(&full[(vt + 1) % L::SLOTS], ((vt + 1) / L::SLOTS) & 1);
                    if (!ok) break;
                }
                const uint32_t sa = tmem + lanes + TM_S + 128 * sb;
                ok = warp_wait(&s_ready[sb], NT == 2 ? step & 1 : (step >> 1) & 1);
                if (!ok) break;
                tc_after();
                const int left = seen - (S.key0 + u * TK);
                if (__any_sync(0xFFFFFFFFu, left < TK)) {
                    // keys that some row does not see: -inf in their place (rare)
#pragma unroll 1
                    for (int c = 0; c < TK; c += 8) {
                        uint32_t r[8];
                        tmem_ld8(sa + c, r);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (c + k >= left) r[k] = 0xFF800000u;
                        tmem_st8(sa + c, r);
                    }
                    tmem_st_wait();
                }
                // the row's S in halves of 64: the second is read twice, which
                // saves 64 registers
                float s[64];
                auto load_half = [&](int c0) {
                    uint32_t* r = reinterpret_cast<uint32_t*>(s);
                    tmem_ld32(sa + c0, r);
                    tmem_ld32(sa + c0 + 32, r + 32);
                    tmem_ld_wait(r);
                    tmem_ld_wait(r + 32);
                };
                float mx = -INFINITY, my = -INFINITY;
                auto half_max = [&] {
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        mx = max3(mx, s[c], s[c + 1]);
                        my = max3(my, s[c + 2], s[c + 3]);
                    }
                };
                load_half(64);
                half_max();
                load_half(0);
                half_max();
                mx = fmaxf(mx, my);
                const bool raise = mx > m + raise_at || m == -INFINITY;
                if (__any_sync(0xFFFFFFFFu, raise)) {
                    const float mn = raise ? fmaxf(m, mx) : m;
                    const float keep = mn == m ? 1.0f : ex2((m - mn) * sl2);
                    if (u > 0) {   // O holds the products of the units before
                        // (NT = 2: S of this unit was issued after them and is there)
                        if (NT == 1) ok = warp_wait(&o_done[t], (step - 1) & 1);
                        if (!ok) break;
                        tc_after();
                        const uint32_t oa = tmem + lanes + TM_O + D * t;
#pragma unroll 1
                        for (int c = 0; c < D; c += 8) {
                            uint32_t r[8];
                            tmem_ld8(oa + c, r);
#pragma unroll
                            for (int k = 0; k < 8; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * keep);
                            tmem_st8(oa + c, r);
                        }
                    }
                    l *= keep;
                    m = mn;
                }
                const float base = m == -INFINITY ? 0.0f : -m * sl2;
                const uint64_t sl22 = f2(sl2, sl2), base2 = f2(base, base);
                uint64_t la = f2(0.0f, 0.0f), lb = la;
#pragma unroll
                for (int c = 0; c < 128; c += 64) {   // P of a half lies where S has been read
                    if (c) load_half(c);
                    uint32_t pk[32];
#pragma unroll
                    for (int k = 0; k < 64; k += 4) {
                        float p0, p1, p2, p3;
                        f2_split(f2_fma(f2(s[k], s[k + 1]), sl22, base2), p0, p1);
                        f2_split(f2_fma(f2(s[k + 2], s[k + 3]), sl22, base2), p2, p3);
                        p0 = ex2(p0); p1 = ex2(p1); p2 = ex2(p2); p3 = ex2(p3);
                        la = f2_add(la, f2(p0, p1));
                        lb = f2_add(lb, f2(p2, p3));
                        pk[k / 2] = pack_pair<E>(p0, p1);   // rounded to the cache's type (attn.cuh); l has the whole p
                        pk[k / 2 + 1] = pack_pair<E>(p2, p3);
                    }
                    tmem_st32(sa + c / 2, pk);
                }
                float l0, l1;
                f2_split(f2_add(la, lb), l0, l1);
                l += l0 + l1;
                tmem_st_wait();
                // a wait tells two phases apart, no more: with two S buffers the
                // product before the last one may still be running here
                if (NT == 1 && step > 0) ok = warp_wait(&o_done[t], (step - 1) & 1);
                if (!ok) break;
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[sb]);
            }
            if (!ok) break;
            ok = warp_wait(&o_done[t], (NT == 1 ? step - 1 : pieces) & 1);
            ++pieces;
            if (!ok) break;
            tc_after();
            // O by way of the Q tile (its products are done), half of the dims at
            // a time: rows go out whole, 16-byte chunks XORed with the row against
            // bank conflicts
            const uint32_t oa = tmem + lanes + TM_O + D * t;
            const bool final = S.whole && !P.keep;
            const float f = !final ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;   // no key: zeros
            const float m2 = m * sl2;
            const long long slot_row = piece_slot(P, blockIdx.x, S.item, S.begins) * P.tile_rows + t * 128 + i;
            const long long mine = final ? (in ? tok * A.o_ts + (long long)qh * A.o_hs : -1) : slot_row * D;
            constexpr int CW = D / 2, CH = CW / 4, AT = 32 / CH;   // dims and chunks of a half, rows at a time
            const bool wide = !final || A.o_f32;
            uint8_t* out = final ? static_cast<uint8_t*>(A.o) : reinterpret_cast<uint8_t*>(P.o);
            // (a bounded wait, as every other: a barrier of the warps would hang if
            // one of them gave up)
            auto all_warps = [&](int nth) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&together[t]);
                return warp_wait(&together[t], nth);
            };
            ok = all_warps(0);   // they have seen the piece's last S
            if (!ok) break;
            float4* stage = reinterpret_cast<float4*>(sm + t * L::QTILE + (warp & 3) * (32 * CW * 4));
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
#pragma unroll 1
                for (int c = 0; c < CW; c += 16) {
                    uint32_t r[16];
                    tmem_ld8(oa + h * CW + c, r);
                    tmem_ld8(oa + h * CW + c + 8, r + 8);
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        stage[lane * CH + (((c + k) / 4) ^ (lane & (CH - 1)))] =
                            make_float4(__uint_as_float(r[k]) * f, __uint_as_float(r[k + 1]) * f,
                                        __uint_as_float(r[k + 2]) * f, __uint_as_float(r[k + 3]) * f);
                }
                __syncwarp();
                const int c = lane % CH;
#pragma unroll 1
                for (int k0 = 0; k0 < 32 / AT; k0 += 4) {
                    float4 v[4];
                    long long off[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = (k0 + k) * AT + lane / CH;
                        v[k] = stage[r * CH + (c ^ (r & (CH - 1)))];
                        off[k] = __shfl_sync(0xFFFFFFFFu, mine, r);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (off[k] >= 0) {
                            const long long at = off[k] + h * CW + 4 * c;
                            if (wide) *reinterpret_cast<float4*>(out + 4 * at) = v[k];
                            else *reinterpret_cast<uint2*>(out + 2 * at) = make_uint2(pack_pair<E>(v[k].x, v[k].y), pack_pair<E>(v[k].z, v[k].w));
                        }
                }
                __syncwarp();
            }
            if (!final) P.ml[slot_row] = make_float2(m2, l);
            else if (in && A.lse) A.lse[tok * A.heads + qh] = l == 0.0f ? -INFINITY : (m2 + log2f(l)) * 0.6931471805599453f;
            ok = all_warps(1);   // the tile is free
            if (!ok) break;
            have = more;
            S = next;
            // O has been read: the next piece's first product (after its P) may overwrite it
            tc_before();
        }
    }
    if (!ok && lane == 0) atomicOr(fault, 4u);
    tc_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
    }
}

constexpr int JR = 32;   // rows per block of 256 threads

// Adds up a block's rows, whose places and pieces (of plan P, then of W) are set.
template <class E, int D, int MOST, int SETS>
__device__ __forceinline__ void add_rows(const AttnArgs& A, Sums<JR, MOST, SETS>& sums, int rows, const TilePlan& P, const TilePlan& W) {
    __syncthreads();
    const int k0 = threadIdx.x % JR, from = threadIdx.x / JR;
    if (k0 < rows) {
        bring(P, sums.pieces[0][k0], sums.ml, k0, from, 256 / JR);
        if (SETS == 2) bring(W, sums.pieces[SETS - 1][k0], sums.ml + sums.pieces[0][k0].n, k0, from, 256 / JR);
    }
    __syncthreads();
    {   // eight lanes a row
        const int k = threadIdx.x / 8;
        const bool in = k < rows;
        weigh(A, sums, k, in ? sums.pieces[0][k].n + (SETS == 2 ? sums.pieces[SETS - 1][k].n : 0) : 0, in, threadIdx.x & 7);
    }
    __syncthreads();
#pragma unroll 1
    for (int e = threadIdx.x; e < rows * (D / 4); e += 256) {
        const int k = e / (D / 4), d = 4 * (e % (D / 4));
        float4 acc[1] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
        add_pieces<D, JR>(P, {&sums.pieces[0][k]}, {&sums.ml[0][k]}, {d}, acc);
        if (SETS == 2) add_pieces<D, JR>(W, {&sums.pieces[SETS - 1][k]}, {&sums.ml[sums.pieces[0][k].n][k]}, {d}, acc);
        const float inv = sums.inv[k];
        attn_store4<E>(A, sums.out[k] + d, make_float4(acc[0].x * inv, acc[0].y * inv, acc[0].z * inv, acc[0].w * inv));
    }
}

// The items that are cut between CTAs (own keys alone): block (c, y) adds up
// rows 32 y .. of the item that CTA c goes on with, if c - 1 began it.  The
// blocks from P.ctas on write the rows of sequences without keys.
template <class E, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ TilePlan P) {
    extern __shared__ __align__(16) uint8_t join_raw[];
    auto& sums = *reinterpret_cast<Sums<JR, MOST_CTAS, 1>*>(join_raw);
    grid_launch_dependents();
    grid_wait_prior();
    const bool cut_item = (int)blockIdx.x < P.ctas;
    const int U = *P.units;
    int4 cut = make_int4((int)blockIdx.x - P.ctas, 0, 0, 0);   // (sequence, row tile), head, first unit, units
    int heads = 1;
    if (cut_item) {
        cut = P.cut[blockIdx.x];
        if (cut.x < 0 || unit_cta(cut.z, U, unit_ctas(P, U)) != (int)blockIdx.x - 1) return;
    } else {
        if (own_tiles(A, P, cut.x) > 0) return;
        heads = A.kv_heads;
    }
    const int b = own_seq(P, cut.x), rt = cut.x - b * P.own_row_tiles, i0 = blockIdx.y * JR;
    const unsigned r0 = ((unsigned)rt << P.tile_shift) + i0, all = A.nq * A.group;
    const int rows = r0 < all ? (int)min((unsigned)JR, all - r0) : 0;
    for (int h = cut.y; h < cut.y + heads; ++h) {
        if ((int)threadIdx.x < rows) {
            const int k = threadIdx.x, t = (r0 + k) / (unsigned)A.group;
            sums.place(A, k, (long long)b * A.nq + t, h * A.group + (int)(r0 + k - t * A.group));
            sums.pieces[0][k] = Pieces{0, 0, 0, 0};
            if (cut_item) sums.pieces[0][k] = item_pieces(P, 0, cut.z, cut.w, U, i0 + k);
        }
        add_rows<E, D>(A, sums, rows, P, P);
        __syncthreads();
    }
}

// All rows: the pieces of their prefix item and of their own item.  A block
// adds up JR rows of a sequence and head.
template <class E, int D>
__global__ void __launch_bounds__(256) attn_merge_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ TilePlan P,
                                                         const __grid_constant__ TilePlan W) {
    extern __shared__ __align__(16) uint8_t merge_raw[];
    auto& sums = *reinterpret_cast<Sums<JR, 2 * MOST_CTAS, 2>*>(merge_raw);
    grid_launch_dependents();
    grid_wait_prior();
    const unsigned all = A.nq * A.group, chunks = (all + JR - 1) / JR;
    const unsigned bh = blockIdx.x / chunks, b = bh / A.kv_heads, r0 = (blockIdx.x - bh * chunks) * JR;
    const int h = bh - b * A.kv_heads, rows = (int)min((unsigned)JR, all - r0);
    if ((int)threadIdx.x < rows) {
        const int k = threadIdx.x;
        const unsigned r = r0 + k, t = r / (unsigned)A.group, gr = b * all + r;
        sums.place(A, k, (long long)b * A.nq + t, h * A.group + (int)(r - t * A.group));
        sums.pieces[0][k] = sums.pieces[1][k] = Pieces{0, 0, 0, 0};
        if (attn_shares(A, P, attn_len(A, attn_row(A, b)))) {
            const int item = h * P.prefix_row_tiles + (int)(gr >> P.tile_shift);
            sums.pieces[0][k] = item_pieces(P, item, item * P.prefix_tiles, P.prefix_tiles,
                                            A.kv_heads * P.prefix_row_tiles * P.prefix_tiles, gr & (P.tile_rows - 1));
        }
        const int pair = b * W.own_row_tiles + (int)(r >> W.tile_shift), tiles = own_tiles(A, W, pair), item = pair * A.kv_heads + h;
        if (tiles > 0) sums.pieces[1][k] = item_pieces(W, item, W.item_unit[item], tiles, *W.units, r & (W.tile_rows - 1));
    }
    add_rows<E, D>(A, sums, rows, P, W);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                               cudaSuccess && q == cudaDriverEntryPointSuccess;
        return found ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
    }();
    return fn;
}

// Pages as a tensor (dim, token, head, page); a box is 64 dims of the tokens
// of one page, at most 128.
bool page_map(CUtensorMap* map, const AttnArgs& A, const void* base, int type, int d) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t tokens = 1ull << A.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)d, tokens, (cuuint64_t)A.kv_heads, (cuuint64_t)A.pages};
    // an axis of length one may come with any stride
    const cuuint64_t strides[3] = {(cuuint64_t)A.kv_ts * 2, (cuuint64_t)(A.kv_heads > 1 ? A.kv_hs : A.kv_ts) * 2,
                                   (cuuint64_t)(A.pages > 1 ? A.page_stride : A.kv_ts) * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(tokens < TK ? tokens : TK), 1, 1}, one[4] = {1, 1, 1, 1};
    return enc(map, type == PLM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class E, int D, int NT>
cudaError_t tile_launch(const AttnArgs& A, const TilePlan& P, const CUtensorMap& km, const CUtensorMap& vm,
                        cudaStream_t stream) {
    unsigned* fault = fault_word();
    if (!fault) return cudaErrorInvalidDevicePointer;
    constexpr int bytes = TileSmem<D, NT>::ALLOC;
    cudaError_t e = cudaFuncSetAttribute(attn_tile_kernel<E, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    e = launch_kernel(attn_tile_kernel<E, D, NT>, dim3((unsigned)P.ctas), dim3(NT * 128 + 64), bytes, stream, A, P, km, vm, fault);
    if (e != cudaSuccess || P.job == 0 || P.keep) return e;
    constexpr int sums = sizeof(Sums<JR, MOST_CTAS, 1>);
    e = cudaFuncSetAttribute(attn_join_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sums);
    if (e != cudaSuccess) return e;
    return launch_kernel(attn_join_kernel<E, D>, dim3((unsigned)(P.ctas + A.batch * P.own_row_tiles), (unsigned)(P.tile_rows / JR)),
                         dim3(256), sums, stream, A, P);
}

template <class E, int D>
cudaError_t merge_launch(const AttnArgs& A, const TilePlan& P, const TilePlan& W, cudaStream_t stream) {
    const long long blocks = (long long)A.batch * A.kv_heads * (((long long)A.nq * A.group + JR - 1) / JR);
    constexpr int bytes = sizeof(Sums<JR, 2 * MOST_CTAS, 2>);
    const cudaError_t e = cudaFuncSetAttribute(attn_merge_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_kernel(attn_merge_kernel<E, D>, dim3((unsigned)blocks), dim3(256), bytes, stream, A, P, W);
}

template <class E>
cudaError_t tile_type(const AttnArgs& A, const TilePlan& P, const CUtensorMap& km, const CUtensorMap& vm, int d, cudaStream_t stream) {
    if (d == 64)
        return P.tile_rows == 256 ? tile_launch<E, 64, 2>(A, P, km, vm, stream) : tile_launch<E, 64, 1>(A, P, km, vm, stream);
    return P.tile_rows == 256 ? tile_launch<E, 128, 2>(A, P, km, vm, stream) : tile_launch<E, 128, 1>(A, P, km, vm, stream);
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace

// CTAs of the prefix launch.  With a multiple of the items, s each, no CTA holds
// pieces of two items; a piece costs its start and end (~3 units), and every eight
// pieces of an item a round of loads (~2 units) in the sums that follow.  One GB300,
// 61 streams behind 8176 (4 items of 64 units): 152 CTAs 23.9 us, 128 22.6, 64
// 18.1; 48 x 5 tokens behind 8192 (32 items of 64): 152 CTAs 88 us, 128 81.
static int prefix_ctas(long long items, long long tiles, int sms) {
    const long long units = items * tiles, all = units < sms ? units : sms, share = (units + all - 1) / all;
    long long best = all, cost = 4 * (share + 3) + 8 * ((tiles / share + 8) / 8);
    for (long long s = 1; s <= tiles && s * items <= sms; ++s) {
        const long long c = 4 * ((tiles + s - 1) / s) + 8 * ((s + 7) / 8);
        if (c < cost) {
            cost = c;
            best = s * items;
        }
    }
    return (int)best;
}

TilePlan tile_plan(const AttnArgs& A, int d, int job, bool share, void* ws, size_t* bytes) {
    const long long mine = (long long)A.nq * A.group, all = job == 0 ? mine * A.batch : mine;
    TilePlan T = {};
    T.job = job;
    T.keep = share;
    T.tile_rows = all > 128 ? 256 : 128;
    T.tile_shift = all > 128 ? 8 : 7;
    const long long row_tiles = (all + T.tile_rows - 1) / T.tile_rows;
    T.prefix_tiles = share ? (A.prefix + TK - 1) / TK : 0;
    const long long items = (long long)A.kv_heads * row_tiles * (job == 0 ? 1 : A.batch);
    const long long most = items * (job == 0 ? T.prefix_tiles : (A.cap + TK - 1) / TK);
    if (most > 0x7FFFFFFFLL) {
        *bytes = SIZE_MAX;
        return T;
    }
    (job == 0 ? T.prefix_row_tiles : T.own_row_tiles) = (int)row_tiles;
    const int sms = num_sms() < MOST_CTAS ? num_sms() : MOST_CTAS;
    T.ctas = (int)(most < sms ? (most < 1 ? 1 : most) : sms);
    if (job == 0) T.ctas = prefix_ctas(items, T.prefix_tiles, sms);
    const size_t slots = T.keep ? (size_t)(T.ctas + items) : 2 * (size_t)T.ctas;
    const size_t item_b = job == 1 && T.keep ? up256(4 * (size_t)items) : 0, cut_b = up256(sizeof(int4) * (size_t)T.ctas);
    const size_t ml_b = up256(slots * T.tile_rows * sizeof(float2));
    uint8_t* p = static_cast<uint8_t*>(ws);
    auto take = [&](size_t b) { uint8_t* r = p; p += ws ? b : 0; return r; };
    T.units = reinterpret_cast<int*>(take(256));
    T.item_unit = reinterpret_cast<int*>(take(item_b));
    T.cut = reinterpret_cast<int4*>(take(cut_b));
    T.ml = reinterpret_cast<float2*>(take(ml_b));
    T.o = reinterpret_cast<float*>(p);
    *bytes = 256 + item_b + cut_b + ml_b + up256(slots * T.tile_rows * (size_t)d * sizeof(float));
    return T;
}

cudaError_t launch_attn_merge(const AttnArgs& A, const TilePlan& prefix, const TilePlan& own, int type, int d,
                              cudaStream_t stream) {
    if (type == PLM_F16)
        return d == 64 ? merge_launch<__half, 64>(A, prefix, own, stream) : merge_launch<__half, 128>(A, prefix, own, stream);
    return d == 64 ? merge_launch<__nv_bfloat16, 64>(A, prefix, own, stream)
                   : merge_launch<__nv_bfloat16, 128>(A, prefix, own, stream);
}

cudaError_t launch_attn_tile(const AttnArgs& A, const TilePlan& P, int type, int d, cudaStream_t stream) {
    CUtensorMap km, vm;
    if (!page_map(&km, A, A.k, type, d) || !page_map(&vm, A, A.v, type, d)) return cudaErrorInvalidValue;
    return type == PLM_F16 ? tile_type<__half>(A, P, km, vm, d, stream) : tile_type<__nv_bfloat16>(A, P, km, vm, d, stream);
}

}  // namespace plm

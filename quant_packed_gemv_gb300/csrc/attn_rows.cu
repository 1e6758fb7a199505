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
// Bound: HBM (4 D bytes per key and head pair, ~2 operations per byte and
// row).  Each warp brings its blocks (8 KB of K and V at D = 128) into a ring of
// its own by cp.async, 16-byte chunks XORed so that the fragment loads are free
// of bank conflicts; keys past the end are filled with zeros and not read.  The
// warps of a CTA and the CTAs of a cluster take the blocks in turn and add
// their parts through shared memory, in a fixed order.  One GB300, 8 heads of 128
// in bf16: 64 sequences of up to 4000 keys, 95 us (5.5 TB/s); 256 of up to 2000,
// 176 us (6.0 TB/s), 182 with a cold L2; 4 of 1100, 9.3 us, which is latency.
#include "attn_tile.cuh"

namespace plm {

namespace {

constexpr int DW = 4;               // warps per CTA
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

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t words(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// Shared memory: Q fragments (NB > 2), then the warps' rings, in whose place
// the parts of the warps go at the end: references m and sums l of the rows,
// O [rows][D + 4] (padded against conflicts).
template <int D, int NB> struct RowsSmem {
    static constexpr int ROWS = 8 * NB, PITCH = D + 4;
    static constexpr int STAGES = (D == 64 ? 2 : 1) * (NB == 1 ? 2 : 3);
    static constexpr int STAGE = 16 * D * 2;   // bytes of 16 keys' K, or V
    struct Parts {
        float m[DW][ROWS], l[DW][ROWS];
        float o[DW][ROWS][PITCH];
        Sums<ROWS, 8 * DW + MOST_CTAS, 1> sums;   // of the cluster's warps, then the prefix pieces
    };
    uint4 q[NB > 2 ? NB * (D / 32) * 32 : 1];
    union {
        uint8_t ring[DW][STAGES][2][STAGE];
        Parts part;
    };
};

// CTAs of 8 nb rows that an SM holds at once: registers bound the first, shared
// memory the others (228 KB, of which a CTA takes 1 KB for itself).
__host__ __device__ constexpr int rows_ctas(int d, int nb) { return nb == 1 ? 3 : nb == 4 && d == 128 ? 1 : 2; }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

template <class E, int D, int NB>
__global__ void __launch_bounds__(DW * 32, rows_ctas(D, NB)) attn_rows_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ TilePlan P) {
    using Sm = RowsSmem<D, NB>;
    constexpr int KC = D / 32, VC = D / 64;   // 16-byte chunks per lane of a K row, of a V row
    constexpr bool QS = NB > 2;
    extern __shared__ __align__(16) uint8_t rows_raw[];
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
    const E* kbase = static_cast<const E*>(A.k) + head;
    const E* vbase = static_cast<const E*>(A.v) + head;
    const int mask = (1 << A.page_shift) - 1;

    const int all = attn_seen(A, len, small_row(A, r0));   // keys that every row sees

    const float sl2 = A.scale * LOG2E;
    const int streams = DW * gridDim.z, stream = blockIdx.z * DW + warp;
    const int blocks = (attn_seen(A, len, small_row(A, r0 + rows - 1)) + 15) >> 4;   // that the last row sees
    const bool shares = attn_shares(A, P, len);
    const int first = shares ? A.prefix >> 4 : 0;   // the prefix is a multiple of 16

    // Block i of this warp's turn into its ring; K and V rows are whole, 16 bytes
    // (8 dims) a lane, chunk c of row r at c ^ 4 (r % 2) for K, c ^ (r & 6) for V
    constexpr int CH = D / 8;
    const int cc = lane % CH, cr = lane / CH;
    const uint32_t ring = smem_u32(&sm.ring[warp][0][0][0]);
    auto page_of = [&](int blk) -> int {
        if (blk >= blocks) return -1;
        const int* at = tab + ((blk << 4) >> A.page_shift);
        return P.prefix_tiles > 0 ? __ldcg(at) : __ldg(at);
    };
    auto fetch = [&](int blk, int page, int slot) {
        if (blk < blocks) {
            const int j = blk << 4;
            const bool there = page >= 0 && page < A.pages;
            const long long off = there ? (long long)page * A.page_stride + (long long)((j & mask) + cr) * A.kv_ts + 8 * cc : 0;
            const uint32_t dst = ring + slot * (2 * Sm::STAGE);
#pragma unroll
            for (int r = 0; r < 16; r += 32 / CH) {
                const int row_ = r + cr;
                const bool in = there && j + row_ < len;
                const long long o_ = in ? off + (long long)r * A.kv_ts : 0;
                cp16(dst + row_ * (2 * D) + ((cc ^ ((row_ & 1) << 2)) << 4), kbase + o_, in);
                cp16(dst + Sm::STAGE + row_ * (2 * D) + ((cc ^ (row_ & 6)) << 4), vbase + o_, in);
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
    if constexpr (QS) {
        for (int i = warp; i < NB * KC; i += DW) sm.q[i * 32 + lane] = q_part(i / KC, i % KC);
        __syncthreads();
    } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < KC; ++c) qf[nb][c] = q_part(nb, c);
    }
    int seen[NB][2];   // keys that rows 8 nb + 2t, + 1 see
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rr = 8 * nb + 2 * t + i;
            seen[nb][i] = rr < rows ? attn_seen(A, len, small_row(A, r0 + rr)) : 0;
        }

    int blk = first + stream, page = page_of(blk);
#pragma unroll
    for (int i = 0; i < Sm::STAGES - 1; ++i) {
        const int next = page_of(blk + (i + 1) * streams);
        fetch(blk + i * streams, page, i);
        page = next;
    }

    float m[NB][2], l[NB][2], o[NB][2 * VC * 2][4];   // o: D / 16 tiles of 16 dims x 8 rows
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
        const uint8_t* ks = &sm.ring[warp][n % Sm::STAGES][0][0];
        const uint8_t* vs = ks + Sm::STAGE;
        float s[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int at = g * (2 * D) + (((4 * c + t) ^ ((g & 1) << 2)) << 4);
            const uint4 k0 = *reinterpret_cast<const uint4*>(ks + at), k1 = *reinterpret_cast<const uint4*>(ks + at + 16 * D);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint4 qv = QS ? sm.q[(nb * KC + c) * 32 + lane] : qf[QS ? 0 : nb][QS ? 0 : c];
                mma16816<E>(s[nb], k0.x, k1.x, k0.y, k1.y, qv.x, qv.y);
                mma16816<E>(s[nb], k0.z, k1.z, k0.w, k1.w, qv.z, qv.w);
            }
        }
        const bool part = j + 16 > all;
        bool raise = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[nb][i] *= sl2;
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
                const float base = m[nb][i & 1] == -INFINITY ? 0.0f : m[nb][i & 1];   // a row without keys so far
                p[i] = ex2(s[nb][i] - base);
                l[nb][i & 1] += p[i];
            }
            // rounded to the cache's type (attn.cuh); l has the whole p
            pb[nb][0] = transpose8x8(pack_pair<E>(p[0], p[1]));
            pb[nb][1] = transpose8x8(pack_pair<E>(p[2], p[3]));
        }
#pragma unroll
        for (int c = 0; c < VC; ++c) {
            const uint8_t* at = vs + 2 * t * (2 * D) + (((8 * c + g) ^ (2 * t)) << 4);
            uint4 vf[4];   // rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
            for (int i = 0; i < 4; ++i) vf[i] = *reinterpret_cast<const uint4*>(at + ((i & 1) + 8 * (i >> 1)) * (2 * D));
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
    cp_wait<0>();
    __syncthreads();   // the rings make room for the parts

    // this warp's part
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int of = 4; of < 32; of <<= 1) l[nb][i] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][i], of);
            if (g == 0) {
                sm.part.m[warp][8 * nb + 2 * t + i] = m[nb][i];
                sm.part.l[warp][8 * nb + 2 * t + i] = l[nb][i];
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                *reinterpret_cast<float2*>(&sm.part.o[warp][8 * nb + 2 * t + i][64 * (k >> 2) + 8 * g + 2 * (k & 3)]) =
                    make_float2(o[nb][k][i], o[nb][k][i + 2]);
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

template <class E, int D, int NB>
cudaError_t rows_launch(const AttnArgs& A, const TilePlan& P, int chunks, int cs, cudaStream_t stream) {
    const dim3 grid((unsigned)(A.batch * A.kv_heads), (unsigned)chunks, (unsigned)cs);
    constexpr int bytes = sizeof(RowsSmem<D, NB>);
    static_assert(rows_ctas(D, NB) * (bytes + 1024) <= 228 * 1024, "the CTAs of an SM");
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<E, D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    if (cs == 1) return launch_kernel(attn_rows_kernel<E, D, NB>, grid, dim3(DW * 32), bytes, stream, A, P);
    return launch_kernel_cluster(attn_rows_kernel<E, D, NB>, grid, dim3(DW * 32), bytes, stream, (unsigned)cs, A, P);
}

template <class E, int D>
cudaError_t rows_nb(const AttnArgs& A, const TilePlan& P, int chunks, int cs, cudaStream_t stream) {
    const int rows = (A.nq * A.group + chunks - 1) / chunks;
    if (rows <= 8) return rows_launch<E, D, 1>(A, P, chunks, cs, stream);
    if (rows <= 16) return rows_launch<E, D, 2>(A, P, chunks, cs, stream);
    return rows <= 24 ? rows_launch<E, D, 3>(A, P, chunks, cs, stream) : rows_launch<E, D, 4>(A, P, chunks, cs, stream);
}

// CTAs of a pair (at most 8: 32 warps): as many as the GPU holds at once (a second
// wave costs a whole start and end: 12 x 9 tokens behind 512, 30 us where one wave
// takes 17), while every warp still gets two blocks of 16 keys.  Long rows up to 16
// are cut into CTAs of 1024 keys and more whatever their number: the GPU hands them
// out as others end, so that sequences of unequal lengths even out (20 of up to
// 16000 keys, 8 heads of 128: 132 us in one wave, 115 so; 64 of up to 4000: 97 and
// 90; half the keys: 91; 4 tokens each, 3000: 85 and 78; 7 tokens: 73 and 75).
int rows_cluster(const AttnArgs& A, int d, int chunks, int keys) {
    const int rows = A.nq * A.group, cut = rows <= 16 ? 2048 : 0x7FFFFFFF;
    const long long pairs = (long long)A.batch * A.kv_heads * chunks, room = attn_rows_room(d, rows);
    int cs = 1;
    while (cs < 8 && keys > 2 * 16 * DW * cs && (pairs * cs * 2 <= room || keys / cs > cut)) cs *= 2;
    return cs;
}

}  // namespace

// Where an SM holds one CTA (25 to 32 rows of 128), a third more than fit at once
// still pays, as those of short sequences end early, and more does not.  Sequences x
// tokens, 4 query heads each on 8 heads, up to 3000 keys: 12 x 8 as 96 CTAs 50 us, as
// 192 39; 8 x 8 as 128 31, as 256 41; 18 x 8 as 144 50, as 288 57; 4 x 8 over 8000 as
// 128 41, as 256 70; 7 heads on 2, over 2000: 40 x 4 as 80 39, as 160 29; 60 x 4 as
// 120 40, as 240 46.
long long attn_rows_room(int d, int rows) {
    const int chunks = (rows + 31) / 32, ctas = rows_ctas(d, ((rows + chunks - 1) / chunks + 7) / 8), sms = num_sms();
    return ctas == 1 ? sms + sms / 3 : (long long)ctas * sms;
}

cudaError_t launch_attn_rows(const AttnArgs& A, const TilePlan* plan, int type, int d, cudaStream_t stream) {
    const TilePlan P = plan ? *plan : TilePlan{};
    const int chunks = (A.nq * A.group + 31) / 32, cs = rows_cluster(A, d, chunks, plan ? A.cap - A.prefix : A.cap);
    if (type == PLM_F16) return d == 64 ? rows_nb<__half, 64>(A, P, chunks, cs, stream) : rows_nb<__half, 128>(A, P, chunks, cs, stream);
    return d == 64 ? rows_nb<__nv_bfloat16, 64>(A, P, chunks, cs, stream) : rows_nb<__nv_bfloat16, 128>(A, P, chunks, cs, stream);
}

}  // namespace plm

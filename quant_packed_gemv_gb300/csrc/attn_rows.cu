// Paged attention for up to 32 query rows per (sequence, key/value head):
// decode, and a few drafted tokens (plm_attn_shared_prefix).
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
// (g, t) = (lane / 4, lane % 4) therefore loads 16 bytes of K rows g and
// g + 8 (dims 32 c + 8 t ..) and of V rows 2t, 2t + 1, 2t + 8, 2t + 9 (dims
// 64 c + 8 g ..) and uses them as fragments where they are: no shared memory.
// Rows of Q follow K's order of d; P^T needs one movmatrix per 8 x 8 block.
// Up to 16 rows Q stays in registers; beyond, the warps share it in shared
// memory, so that O (32 registers per 8 rows at D = 128) has room.
//
// Bound: HBM (4 D bytes per key and head pair, ~2 operations per byte and
// row).  A warp keeps the next 16 keys' K and this block's V in flight (8 KB
// at D = 128); the warps of a CTA and the CTAs of a cluster take the blocks
// in turn and add their parts through shared memory, in a fixed order.
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

// Shared memory: Q fragments (NB > 2), then the parts of a pair's warps: per
// warp the references m and sums l of its rows, then O [rows][D + 4] (padded
// against conflicts).
template <int D, int NB> struct RowsSmem {
    static constexpr int ROWS = 8 * NB, PITCH = D + 4;
    uint4 q[NB > 2 ? NB * (D / 32) * 32 : 1];
    float m[DW][ROWS], l[DW][ROWS];
    float o[DW][ROWS][PITCH];
};

template <class E, int D, int NB>
__global__ void __launch_bounds__(DW * 32, NB == 1 ? 3 : 2) attn_rows_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ TilePlan P) {
    using Sm = RowsSmem<D, NB>;
    constexpr int KC = D / 32, VC = D / 64;   // 16-byte chunks per lane of a K row, of a V row
    constexpr bool QS = NB > 2;
    extern __shared__ __align__(16) uint8_t rows_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(rows_raw);
    grid_launch_dependents();
    // after the tile kernel there is nothing to wait for yet: it starts this
    // kernel once the work before it has finished
    if (P.prefix_tiles == 0) grid_wait_prior();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int b = blockIdx.x / A.kv_heads, h = blockIdx.x - b * A.kv_heads;
    const int rows = A.nq * A.group;
    const int row = attn_row(A, b), len = attn_len(A, row);
    const int* tab = A.table + (long long)max(row, 0) * A.table_stride;
    const long long head = (long long)h * A.kv_hs;
    const E* kbase = static_cast<const E*>(A.k) + head + 8 * t;
    const E* vbase = static_cast<const E*>(A.v) + head + 8 * g;
    const int mask = (1 << A.page_shift) - 1;

    // Q as the B operand: row 8 nb + g, dims 32 c + 8 t ..; zeros past the rows
    uint4 qf[QS ? 1 : NB][QS ? 1 : KC];
    auto q_part = [&](int nb, int c) {
        const int r = 8 * nb + g;
        if (r >= rows) return make_uint4(0, 0, 0, 0);
        return *reinterpret_cast<const uint4*>(static_cast<const E*>(A.q) + ((long long)b * A.nq + r / A.group) * A.q_ts +
                                               (long long)(h * A.group + r % A.group) * A.q_hs + 8 * t + 32 * c);
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
            seen[nb][i] = rr < rows ? attn_seen(A, len, rr / A.group) : 0;
        }
    const int all = attn_seen(A, len, 0);   // keys that every row sees

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
    const float sl2 = A.scale * LOG2E;
    const int streams = DW * gridDim.z, stream = blockIdx.z * DW + warp;
    const int blocks = (len + 15) >> 4;
    const bool shares = attn_shares(A, P, len);
    const int first = shares ? A.prefix >> 4 : 0;   // the prefix is a multiple of 16

    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto page_of = [&](int blk) -> int { return blk < blocks ? __ldg(tab + ((blk << 4) >> A.page_shift)) : -1; };
    auto load_k = [&](int blk, int page, uint4 (&kf)[2][KC]) {
        const int j = blk << 4;
        const bool in = page >= 0 && page < A.pages;
        const E* p = kbase + (long long)page * A.page_stride + (long long)((j & mask) + g) * A.kv_ts;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < KC; ++c)
                kf[i][c] = in && j + g + 8 * i < len ? ldg_nc_v4(p + 8 * i * A.kv_ts + 32 * c) : zero;
    };

    int blk = first + stream, page = page_of(blk), page_n = page_of(blk + streams);
    uint4 kf[2][KC];
    if (blk < blocks) load_k(blk, page, kf);
    for (; blk < blocks; blk += streams) {
        const int j = blk << 4;
        uint4 vf[4][VC];   // rows 2t, 2t + 1, 2t + 8, 2t + 9
        {
            const bool in = page >= 0 && page < A.pages;
            const E* p = vbase + (long long)page * A.page_stride + (long long)((j & mask) + 2 * t) * A.kv_ts;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = (i & 1) + 8 * (i >> 1);
#pragma unroll
                for (int c = 0; c < VC; ++c)
                    vf[i][c] = in && j + 2 * t + k < len ? ldg_nc_v4(p + k * A.kv_ts + 64 * c) : zero;
            }
        }
        const int page_nn = page_of(blk + 2 * streams);
        float s[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.0f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 qv = QS ? sm.q[(nb * KC + c) * 32 + lane] : qf[QS ? 0 : nb][QS ? 0 : c];
                mma16816<E>(s[nb], kf[0][c].x, kf[1][c].x, kf[0][c].y, kf[1][c].y, qv.x, qv.y);
                mma16816<E>(s[nb], kf[0][c].z, kf[1][c].z, kf[0][c].w, kf[1][c].w, qv.z, qv.w);
            }
        }
        if (blk + streams < blocks) load_k(blk + streams, page_n, kf);
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
            pb[nb][0] = transpose8x8(pack_pair<E>(p[0], p[1]));
            pb[nb][1] = transpose8x8(pack_pair<E>(p[2], p[3]));
        }
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // dims 64 c + 8 g + 2 i, + 1
                const uint32_t w0 = words(vf[0][c], i), w1 = words(vf[1][c], i), w2 = words(vf[2][c], i),
                               w3 = words(vf[3][c], i);
                const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
                const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma16816<E>(o[nb][4 * c + i], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
            }
        page = page_n;
        page_n = page_nn;
    }

    // this warp's part
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int of = 4; of < 32; of <<= 1) l[nb][i] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][i], of);
            if (g == 0) {
                sm.m[warp][8 * nb + 2 * t + i] = m[nb][i];
                sm.l[warp][8 * nb + 2 * t + i] = l[nb][i];
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                *reinterpret_cast<float2*>(&sm.o[warp][8 * nb + 2 * t + i][64 * (k >> 2) + 8 * g + 2 * (k & 3)]) =
                    make_float2(o[nb][k][i], o[nb][k][i + 2]);
        }
    }
    const int cs = gridDim.z;   // the cluster: the CTAs of this pair
    if (cs > 1) cluster_barrier();
    else __syncthreads();
    if (P.prefix_tiles > 0) grid_wait_prior();   // the tile kernel's results
    // A warp adds up a row at a time, 4 (2 at D = 64) dims a lane: the parts of
    // the cluster's warps (at most 32, a lane each for their weights), then the
    // pieces of the row's prefix item, both in order.
    constexpr int PER = D / 32;
    for (int r = blockIdx.z + cs * warp; r < rows; r += cs * DW) {
        const bool part = lane < cs * DW;
        const int pz = lane / DW, pw = lane % DW;
        float pm = part ? peer_f32(&sm.m[pw][r], pz, cs) : -INFINITY;
        const float pl = part ? peer_f32(&sm.l[pw][r], pz, cs) : 0.0f;
        if (pl == 0.0f) pm = -INFINITY;   // no key
        RowSum<PER> R;
        R.m = warp_max(pm);
        const float wgt = pm == -INFINITY ? 0.0f : ex2(pm - R.m);
        R.l = warp_sum(wgt * pl);
        for (int p = 0; p < cs * DW; ++p) {
            const float f = __shfl_sync(0xFFFFFFFFu, wgt, p);
            float v[PER];
            peer_dims<PER>(&sm.o[p % DW][r][PER * lane], p / DW, cs, v);
            if (f != 0.0f)
#pragma unroll
                for (int i = 0; i < PER; ++i) R.o[i] = fmaf(f, v[i], R.o[i]);
        }
        if (shares) {
            const long long gr = (long long)b * rows + r, rt = gr / P.tile_rows;
            const int item = h * P.prefix_row_tiles + (int)rt, u0 = item * P.prefix_tiles;
            R.pieces(P, u0, P.prefix_tiles, A.kv_heads * P.prefix_row_tiles * P.prefix_tiles, item,
                     (int)(gr - rt * P.tile_rows), lane);
        }
        R.template store<E>(A, (long long)b * A.nq + r / A.group, h * A.group + r % A.group, lane);
    }
    if (cs > 1) cluster_barrier();   // no CTA leaves while its part is read
}

template <class E, int D, int NB>
cudaError_t rows_launch(const AttnArgs& A, const TilePlan& P, int cs, cudaStream_t stream) {
    const dim3 grid((unsigned)(A.batch * A.kv_heads), 1, (unsigned)cs);
    constexpr int bytes = sizeof(RowsSmem<D, NB>);
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<E, D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    if (cs == 1) return launch_kernel(attn_rows_kernel<E, D, NB>, grid, dim3(DW * 32), bytes, stream, A, P);
    return launch_kernel_cluster(attn_rows_kernel<E, D, NB>, grid, dim3(DW * 32), bytes, stream, (unsigned)cs, A, P);
}

template <class E, int D>
cudaError_t rows_nb(const AttnArgs& A, const TilePlan& P, int cs, cudaStream_t stream) {
    const int rows = A.nq * A.group;
    if (rows <= 8) return rows_launch<E, D, 1>(A, P, cs, stream);
    if (rows <= 16) return rows_launch<E, D, 2>(A, P, cs, stream);
    return rows <= 24 ? rows_launch<E, D, 3>(A, P, cs, stream) : rows_launch<E, D, 4>(A, P, cs, stream);
}

// CTAs of a pair (at most 8: 32 warps): while the pairs alone leave warps idle (12 fit an SM), and
// every warp still gets two blocks of 16 keys.
int rows_cluster(const AttnArgs& A, int keys) {
    const long long pairs = (long long)A.batch * A.kv_heads, room = 3LL * num_sms();
    int cs = 1;
    while (cs < 8 && pairs * cs * 2 <= room && keys > 2 * 16 * DW * cs) cs *= 2;
    return cs;
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& A, const TilePlan* plan, int type, int d, cudaStream_t stream) {
    const TilePlan P = plan ? *plan : TilePlan{};
    const int cs = rows_cluster(A, plan ? A.cap - A.prefix : A.cap);
    if (type == PLM_F16) return d == 64 ? rows_nb<__half, 64>(A, P, cs, stream) : rows_nb<__half, 128>(A, P, cs, stream);
    return d == 64 ? rows_nb<__nv_bfloat16, 64>(A, P, cs, stream) : rows_nb<__nv_bfloat16, 128>(A, P, cs, stream);
}

}  // namespace plm

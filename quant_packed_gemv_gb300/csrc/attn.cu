// Attention over a paged cache (plm_attn_shared_prefix).
//
// One warp per query row and head walks the keys 32 at a time: a lane's key
// gives its score (the query, f32, lies in shared memory), the running
// maximum and sum of the softmax are kept in f32, and the lanes then share
// the head's dimensions to add up p_j v_j.
#include "attn.cuh"

namespace plm {

namespace {

constexpr int AW = 4;   // warps per CTA

template <class E, int D>
__global__ void __launch_bounds__(AW * 32) attn_kernel(const __grid_constant__ AttnArgs A) {
    __shared__ __align__(16) float qs[AW][D];
    grid_launch_dependents();
    grid_wait_prior();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long item = (long long)blockIdx.x * AW + warp;
    if (item >= (long long)A.batch * A.nq * A.heads) return;
    const int h = (int)(item % A.heads);
    const long long tok = item / A.heads;
    const int b = (int)(tok / A.nq), t = (int)(tok - (long long)b * A.nq);
    const int row = attn_row(A, b);
    const int seen = min(attn_seen(A, attn_len(A, row), t), attn_len(A, row));
    const E* q = static_cast<const E*>(A.q) + tok * A.q_ts + h * A.q_hs;
    for (int i = lane; i < D; i += 32) qs[warp][i] = (float)q[i];
    __syncwarp();
    const int* tab = A.table + (long long)max(row, 0) * A.table_stride;
    const long long head = (long long)(h / A.group) * A.kv_hs;
    constexpr int PER = D / 32;
    float m = -INFINITY, l = 0.0f, acc[PER] = {};
    for (int j0 = 0; j0 < seen; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        long long off = -1;
        if (j < seen) {
            const int page = tab[j >> A.page_shift];
            if (page >= 0 && page < A.pages)
                off = page * A.page_stride + head + (j & ((1 << A.page_shift) - 1)) * A.kv_ts;
            s = 0.0f;
            if (off >= 0) {
                const uint4* kp = reinterpret_cast<const uint4*>(static_cast<const E*>(A.k) + off);
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 u = kp[c];
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = pair_to_f32<E>(w[i]);
                        s = fmaf(qs[warp][8 * c + 2 * i], f.x, s);
                        s = fmaf(qs[warp][8 * c + 2 * i + 1], f.y, s);
                    }
                }
            }
            s *= A.scale;
        }
        float mx = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.0f : mn;
        const float keep = expf(m - base), p = expf(s - base);
        l = l * keep + warp_sum(p);
        m = mn;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] *= keep;
        const int n = min(32, seen - j0);
        for (int k = 0; k < n; ++k) {
            const float pk = __shfl_sync(0xFFFFFFFFu, p, k);
            const long long ok = __shfl_sync(0xFFFFFFFFu, off, k);
            if (ok < 0) continue;
            const E* vp = static_cast<const E*>(A.v) + ok + PER * lane;
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] = fmaf(pk, (float)vp[i], acc[i]);
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // no key: o = 0, lse = -inf
    const long long oo = tok * A.o_ts + h * A.o_hs + PER * lane;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (A.o_f32) static_cast<float*>(A.o)[oo + i] = acc[i] * inv;
        else static_cast<E*>(A.o)[oo + i] = (E)(acc[i] * inv);
    }
    if (A.lse && lane == 0) A.lse[tok * A.heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <class E>
cudaError_t attn_type(const AttnArgs& A, int d, cudaStream_t stream) {
    const long long items = (long long)A.batch * A.nq * A.heads;
    const dim3 grid((unsigned)((items + AW - 1) / AW));
    return d == 64 ? launch_kernel(attn_kernel<E, 64>, grid, dim3(AW * 32), 0, stream, A)
                   : launch_kernel(attn_kernel<E, 128>, grid, dim3(AW * 32), 0, stream, A);
}

}  // namespace

size_t attn_workspace_bytes(long long, long long, long long, long long, long long, long long, long long) { return 0; }

cudaError_t launch_attn(const plm_attn_problem& p, void*, cudaStream_t stream) {
    AttnArgs A = {};
    A.q = p.q; A.o = p.o; A.lse = p.lse; A.k = p.k; A.v = p.v;
    A.table = p.table; A.lens = p.lens; A.seqs = p.seqs;
    A.batch = (int)p.batch; A.nq = (int)p.tokens; A.heads = (int)p.heads; A.kv_heads = (int)p.kv_heads;
    A.group = A.heads / A.kv_heads;
    A.q_ts = p.q_token_stride; A.q_hs = p.q_head_stride; A.o_ts = p.o_token_stride; A.o_hs = p.o_head_stride;
    A.page_stride = p.page_stride; A.kv_hs = p.kv_head_stride; A.kv_ts = p.kv_token_stride;
    A.table_stride = p.table_stride;
    while ((1LL << A.page_shift) < p.page_tokens) ++A.page_shift;
    A.pages = (int)p.pages; A.rows = (int)p.rows;
    A.prefix = (int)p.prefix_len;
    const long long room = p.table_stride * p.page_tokens;
    A.cap = (int)(p.max_len < room ? p.max_len : room);
    A.scale = p.scale;
    A.o_f32 = p.o_type == PLM_F32;
    if (A.nq * A.group <= 16) return launch_attn_rows(A, p.type, (int)p.head_dim, stream);
    return p.type == PLM_F16 ? attn_type<__half>(A, (int)p.head_dim, stream)
                             : attn_type<__nv_bfloat16>(A, (int)p.head_dim, stream);
}

}  // namespace plm

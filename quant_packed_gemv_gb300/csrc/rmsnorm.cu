// Residual sum, root-mean-square norm and the q8_K blocks of the result
// (plm_rmsnorm).
//
// Mathematics.  h = x + r (rounded to r's type); inv = 1 / sqrt(sum h^2 / k +
// eps); y = (h inv) w; per 256 values q8_K as plm_quantize_q8K makes it.
//
// Layout.  A row is cut into chunks of 256 values; a warp holds up to four of
// its row's chunks in registers from the first read to the last write, so
// each value passes memory once.  A lane holds values 4 lane .. + 3 of each
// half of a chunk: whole 512-byte lines per access.  Chunk sums go through
// shared memory and every warp adds them in the same order, which depends on k
// alone: a row's bits do not depend on m or on the launch.
//
// Bound: HBM (x, r and h once, 292 bytes of blocks per 256 values), ~25 instructions a value
// of a lane next to it.  One GB300: 8191 rows of 4096 in f32 with residual, sum and blocks
// 69 us, 6.4 TB/s; one row of 1024 2.2 us, which is the launch and two trips to memory.
// Rows that are no whole chunks take their values by four with a look at each place, and half
// of the lanes of a row of 128 hold nothing: 131056 such rows (a head each) 51 us, 2.6 TB/s.
#include "plm_device.cuh"
#include "plm_internal.h"
#include "values.cuh"

namespace plm {

namespace {

constexpr int NORM_WARPS = 16;    // of a row at most
constexpr int HELD = 4;           // chunks of a warp in registers at most

struct NormArgs {
    plm_rmsnorm_problem p;
    int warps;                    // per row
    bool x4, r4, s4, y4, w4;      // four values in one access
    bool whole;                   // all of them, and k whole chunks
};

// Four values as they lie in memory, and in f32: the loads of a warp's chunks are
// issued one after the other, with nothing between them that waits or branches.
template <int N> __device__ __forceinline__ void load_raw(const void* p, int type, const int (&at)[N], float4 (&v)[N]) {
    if (type == PLM_F32) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at[j]);
            v[j].x = __uint_as_float(u.x);
            v[j].y = __uint_as_float(u.y);
        }
    }
}
template <int N> __device__ __forceinline__ void as_f32(int type, float4 (&v)[N]) {
    if (type == PLM_F32) return;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint32_t a = __float_as_uint(v[j].x), b = __float_as_uint(v[j].y);
        if (type == PLM_F16) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
            v[j] = make_float4(x.x, x.y, y.x, y.y);
        } else {
            v[j] = make_float4(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
        }
    }
}

// (fused by hand: left to the compiler, the kernels round differently)
__device__ __forceinline__ float sum8(const float4& a, const float4& b) {
    const float s = fmaf(a.w, a.w, fmaf(a.z, a.z, fmaf(a.y, a.y, __fmul_rn(a.x, a.x))));
    const float t = fmaf(b.w, b.w, fmaf(b.z, b.z, fmaf(b.y, b.y, __fmul_rn(b.x, b.x))));
    return __fadd_rn(s, t);
}

// The q8_K blocks of a warp's N chunks v (values 4 lane .. and 128 + 4 lane ..), the
// first n of which are there: the arithmetic of q8K_quantize_warp, with the reductions
// as single instructions and the chunks side by side.
template <int N> __device__ __forceinline__ void put_q8K(uint8_t* const (&blk)[N], int n, const float (&v)[N][8], int lane) {
    uint32_t amax[N], idx[N];
    float mine[N], mx[N], d[N], iscale[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[j][i]));   // (of numbers: NaN has no size)
        amax[j] = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        idx[j] = 0x7FFFFFFFu;
        mine[j] = 0.0f;
#pragma unroll
        for (int i = 7; i >= 0; --i)
            if ((__float_as_uint(v[j][i]) & 0x7FFFFFFFu) == amax[j]) {
                idx[j] = 4 * lane + (i & 3) + (i < 4 ? 0 : 128);
                mine[j] = v[j][i];
            }
        idx[j] = __reduce_min_sync(0xFFFFFFFFu, idx[j]);   // the first occurrence
    }
#pragma unroll
    for (int j = 0; j < N; ++j) mx[j] = __shfl_sync(0xFFFFFFFFu, mine[j], (idx[j] & 127) >> 2);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        iscale[j] = __fdiv_rn(-128.0f, amax[j] ? mx[j] : 1.0f);   // (zeros and NaN: codes 0)
        d[j] = amax[j] ? __fdiv_rn(1.0f, iscale[j]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        int q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = min(127, __float2int_rn(__fmul_rn(iscale[j], v[j][i])));
        const uint32_t w0 = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
        const uint32_t w1 = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
        // sums of 16 codes: four lanes each, in both halves
        // both sums in one word, to 16 bits each (codes of the smallest values, whose scale is infinite, pass them)
        int both = (short)(q[0] + q[1] + q[2] + q[3]) + (q[4] + q[5] + q[6] + q[7]) * 65536;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) both += __shfl_xor_sync(0xFFFFFFFFu, both, o);
        const int next = __shfl_down_sync(0xFFFFFFFFu, both, 4);
        if (j >= n) continue;
        uint32_t* words = reinterpret_cast<uint32_t*>(blk[j]);
        words[1 + lane] = w0;
        words[33 + lane] = w1;
        if ((lane & 7) == 0) {   // sums 2h, 2h + 1 of each half
            const int s0 = (short)(both & 0xFFFF), s1 = (both - s0) >> 16, n0 = (short)(next & 0xFFFF), n1 = (next - n0) >> 16;
            words[65 + (lane >> 3)] = ((uint32_t)s0 & 0xFFFFu) | ((uint32_t)n0 << 16);
            words[69 + (lane >> 3)] = ((uint32_t)s1 & 0xFFFFu) | ((uint32_t)n1 << 16);
        }
        if (lane == 0) words[0] = __float_as_uint(d[j]);
    }
}

struct Row {
    const NormArgs& A;
    long long xo, ro, so, yo;   // the row's element offsets
    long long r;
    int lane;

    __device__ Row(const NormArgs& a, long long row, int ln)
        : A(a), xo(row * a.p.x_stride), ro(row * a.p.residual_stride), so(row * a.p.sum_stride), yo(row * a.p.y_stride), r(row), lane(ln) {}

    // Of four values from i on, how many there are (0 or less: none)
    __device__ __forceinline__ int left(int i) const { return (int)(A.p.k - i < 4 ? A.p.k - i : 4); }
    // h of a half chunk, from value i on
    __device__ __forceinline__ float4 h(int i) const {
        const int n = left(i);
        float4 v = load_four(A.p.x, A.p.x_type, xo + i, n, A.x4);
        if (A.p.residual) {
            const float4 b = load_four(A.p.residual, A.p.r_type, ro + i, n, A.r4);
            v.x = value_rounded(v.x + b.x, A.p.r_type);
            v.y = value_rounded(v.y + b.y, A.p.r_type);
            v.z = value_rounded(v.z + b.z, A.p.r_type);
            v.w = value_rounded(v.w + b.w, A.p.r_type);
        }
        return v;
    }
    __device__ __forceinline__ void keep(int i, const float4& v) const {
        if (A.p.sum) store_four(A.p.sum, A.p.r_type, so + i, left(i), A.s4, v);
    }
    __device__ __forceinline__ float4 w(int i) const {
        if (!A.p.weight) return make_float4(1.0f, 1.0f, 1.0f, 1.0f);
        return load_four(A.p.weight, A.p.w_type, i, left(i), A.w4);
    }
    // The outputs of chunks c, c + step, .., the first n of N; halves h and their weights w
    template <int N> __device__ __forceinline__ void put(long long c, int step, int n, const float4 (&h)[2 * N], const float4 (&w)[2 * N], float inv) const {
        float v[N][8];
        uint8_t* blk[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float4 a = h[2 * j], b = h[2 * j + 1], wa = w[2 * j], wb = w[2 * j + 1];
            v[j][0] = a.x * inv * wa.x; v[j][1] = a.y * inv * wa.y; v[j][2] = a.z * inv * wa.z; v[j][3] = a.w * inv * wa.w;
            v[j][4] = b.x * inv * wb.x; v[j][5] = b.y * inv * wb.y; v[j][6] = b.z * inv * wb.z; v[j][7] = b.w * inv * wb.w;
            blk[j] = static_cast<uint8_t*>(A.p.xq) + (r * (A.p.k / QK) + c + j * step) * Q8K_BYTES;
            if (A.p.y && j < n) {
                const int i = (int)((c + j * step) * QK) + 4 * lane;
                store_four(A.p.y, A.p.y_type, yo + i, left(i), A.y4, make_float4(v[j][0], v[j][1], v[j][2], v[j][3]));
                store_four(A.p.y, A.p.y_type, yo + i + 128, left(i + 128), A.y4, make_float4(v[j][4], v[j][5], v[j][6], v[j][7]));
            }
        }
        if (A.p.xq) put_q8K<N>(blk, n, v, lane);
    }
    __device__ __forceinline__ float inverse(float sum) const {
        return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, (float)A.p.k) + A.p.eps));
    }
};

// A row per A.warps warps, NCH chunks each.
template <int NCH>
__global__ void __launch_bounds__(NORM_WARPS * 32) rmsnorm_kernel(const __grid_constant__ NormArgs A) {
    __shared__ float sums[NORM_WARPS * HELD];   // of the rows' chunks
    grid_launch_dependents();
    grid_wait_prior();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = (int)(blockDim.x >> 5) / A.warps;
    const int mine = warp / A.warps, part = warp - mine * A.warps, chunks = (int)((A.p.k + QK - 1) / QK);
    const long long r = (long long)blockIdx.x * rows + mine;
    const bool in = r < A.p.m;
    const Row row(A, in ? r : 0, lane);
    float4 h[2 * NCH];   // the halves of the chunks
    float* own = sums + mine * A.warps * NCH;
    // (past the row's last chunk: the last again, not used)
    auto places = [&](int (&at)[2 * NCH]) {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            at[2 * j] = min(part + j * A.warps, chunks - 1) * QK + 4 * lane;
            at[2 * j + 1] = at[2 * j] + 128;
        }
    };
    if (in) {
        if (A.whole) {
            int at[2 * NCH];
            places(at);
            load_raw(static_cast<const uint8_t*>(A.p.x) + row.xo * type_bytes(A.p.x_type), A.p.x_type, at, h);
            if (A.p.residual) {
                float4 r4[2 * NCH];
                load_raw(static_cast<const uint8_t*>(A.p.residual) + row.ro * type_bytes(A.p.r_type), A.p.r_type, at, r4);
                as_f32(A.p.x_type, h);
                as_f32(A.p.r_type, r4);
#pragma unroll
                for (int j = 0; j < 2 * NCH; ++j)
                    h[j] = make_float4(h[j].x + r4[j].x, h[j].y + r4[j].y, h[j].z + r4[j].z, h[j].w + r4[j].w);
                if (A.p.r_type != PLM_F32)
#pragma unroll
                    for (int j = 0; j < 2 * NCH; ++j)
                        h[j] = make_float4(value_rounded(h[j].x, A.p.r_type), value_rounded(h[j].y, A.p.r_type), value_rounded(h[j].z, A.p.r_type),
                                           value_rounded(h[j].w, A.p.r_type));
            } else {
                as_f32(A.p.x_type, h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = part + j * A.warps, i = c * QK + 4 * lane;
                h[2 * j] = h[2 * j + 1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (c < chunks) {
                    h[2 * j] = row.h(i);
                    h[2 * j + 1] = row.h(i + 128);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = part + j * A.warps, i = c * QK + 4 * lane;
            const float s = warp_sum(sum8(h[2 * j], h[2 * j + 1]));
            if (lane == 0) own[c] = s;
            if (c < chunks) {
                row.keep(i, h[2 * j]);
                row.keep(i + 128, h[2 * j + 1]);
            }
        }
    }
    __syncthreads();
    if (!in) return;
    float s = lane < chunks ? own[lane] : 0.0f;
    if (lane + 32 < chunks) s += own[lane + 32];
    const float inv = row.inverse(warp_sum(s));
    float4 w[2 * NCH];
    if (A.p.weight && A.whole) {
        int at[2 * NCH];
        places(at);
        load_raw(A.p.weight, A.p.w_type, at, w);
        as_f32(A.p.w_type, w);
    } else {
#pragma unroll
        for (int j = 0; j < 2 * NCH; ++j) {
            const int i = (part + (j >> 1) * A.warps) * QK + 128 * (j & 1) + 4 * lane;
            w[j] = i < A.p.k ? row.w(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    }
    const int n = (chunks - part + A.warps - 1) / A.warps;
    row.put<NCH>(part, A.warps, n, h, w, inv);
}

// Rows too long for the registers: read twice.
__global__ void __launch_bounds__(NORM_WARPS * 32) rmsnorm_long_kernel(const __grid_constant__ NormArgs A) {
    __shared__ float sums[NORM_WARPS];
    grid_launch_dependents();
    grid_wait_prior();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Row row(A, blockIdx.x, lane);
    const long long chunks = (A.p.k + QK - 1) / QK;
    float s = 0.0f;
    for (long long c = warp; c < chunks; c += NORM_WARPS) {
        const int i = (int)(c * QK) + 4 * lane;
        const float4 a = row.h(i), b = i + 128 < A.p.k ? row.h(i + 128) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        s += warp_sum(sum8(a, b));
        row.keep(i, a);
        if (i + 128 < A.p.k) row.keep(i + 128, b);
    }
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NORM_WARPS; ++i) s += sums[i];
    const float inv = row.inverse(s);
    for (long long c = warp; c < chunks; c += NORM_WARPS) {
        const int i = (int)(c * QK) + 4 * lane;
        auto again = [&](int at) {   // the sum may have taken the place of what it is made of
            return A.p.sum ? load_four(A.p.sum, A.p.r_type, row.so + at, row.left(at), A.s4) : row.h(at);
        };
        const float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const bool two = i + 128 < A.p.k;
        const float4 a = again(i), b = two ? again(i + 128) : z;
        const float4 h[2] = {a, b}, w[2] = {row.w(i), two ? row.w(i + 128) : z};
        row.put<1>(c, 0, 1, h, w, inv);
    }
}

}  // namespace

cudaError_t launch_rmsnorm(const plm_rmsnorm_problem& p, cudaStream_t stream) {
    NormArgs A = {};
    A.p = p;
    const bool even = p.k % 4 == 0;
    auto four = [&](const void* q, long long stride, int type) { return even && four_aligned(q, p.m > 1 ? stride : 0, type); };
    A.x4 = four(p.x, p.x_stride, p.x_type);
    A.r4 = four(p.residual, p.residual_stride, p.r_type);
    A.s4 = four(p.sum, p.sum_stride, p.r_type);
    A.y4 = four(p.y, p.y_stride, p.y_type);
    A.w4 = four(p.weight, 0, p.w_type);
    A.whole = p.k % QK == 0 && A.x4 && (A.r4 || !p.residual) && (A.w4 || !p.weight);
    const long long chunks = (p.k + QK - 1) / QK;
    if (chunks > NORM_WARPS * HELD) {
        A.warps = NORM_WARPS;
        return launch_kernel(rmsnorm_long_kernel, dim3((unsigned)p.m), dim3(NORM_WARPS * 32), 0, stream, A);
    }
    // chunks a warp: few rows are spread over warps, many keep more loads of a warp in flight (8191 rows of 4096:
    // one chunk 78 us, two 69, four 78)
    int held = 1;
    while (held < HELD && (chunks > NORM_WARPS * held || (held < 2 && chunks > held && p.m * chunks >= 16LL * num_sms() * held))) held *= 2;
    A.warps = (int)((chunks + held - 1) / held);
    const int rows = A.warps >= 4 ? 1 : 8 / A.warps;   // of a CTA
    const dim3 grid((unsigned)((p.m + rows - 1) / rows)), block((unsigned)(32 * A.warps * rows));
    if (held == 1) return launch_kernel(rmsnorm_kernel<1>, grid, block, 0, stream, A);
    if (held == 2) return launch_kernel(rmsnorm_kernel<2>, grid, block, 0, stream, A);
    return launch_kernel(rmsnorm_kernel<4>, grid, block, 0, stream, A);
}

}  // namespace plm

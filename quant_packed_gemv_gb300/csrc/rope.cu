// Rotary positions (plm_rope): pairs (a, b) of every head turned by
// position * frequency, written as rows or into cache pages.
//
// Mathematics.  y = (a c - b s, b c + a s) with c + i s = scale e^(i angle),
// angle = 2 pi frac(p f).  f is a 64-bit fraction of a turn, so the low 64
// bits of the integer product p * f are the fraction, exactly; its top 32
// bits as a signed number are turns in [-1/2, 1/2), and sincospi of twice
// that needs no range reduction.
//
// Bound: HBM (each value read and written once, ~1 operation per byte).
// A CTA takes TB tokens: its threads first put the TB * R/2 (c, s) pairs into
// shared memory (one sincospi each, shared by all heads), then walk the
// tokens' head rows.  A unit is V pairs (or 2V values past the rotary part):
// V = 8 gives 16-byte accesses of 16-bit types; smaller V where the rotary
// size, a stride or a pointer is not a multiple of that.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/plm.h"
#include "plm_device.cuh"
#include "plm_internal.h"

namespace plm {

namespace {

constexpr int RT = 256;          // threads per CTA
constexpr int ROPE_CS = 1024;    // (c, s) pairs of a CTA's tokens at most

struct RopeArgs {
    plm_rope_tensor t[PLM_ROPE_MAX_TENSORS];
    int head0[PLM_ROPE_MAX_TENSORS + 1];   // first head of each tensor in the joint head index
    int count;
    const int32_t* positions;
    const unsigned long long* freqs;
    long long tokens;
    int d, r, tb, inverse;
    float scale;
};

template <int BYTES> struct Raw;
template <> struct Raw<2> { using T = unsigned short; };
template <> struct Raw<4> { using T = unsigned; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<16> { using T = uint4; };

// N values; accesses are W values wide, at most 16 bytes: p is aligned to that.
template <int W, class E, int N>
__device__ __forceinline__ void load_as(const E* p, float (&v)[N]) {
    constexpr int B = W * (int)sizeof(E) < 16 ? W * (int)sizeof(E) : 16;
    constexpr int PER = B / (int)sizeof(E);
    using R = typename Raw<B>::T;
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
        union { R r; E e[PER]; } u = {*reinterpret_cast<const R*>(p + i * PER)};
#pragma unroll
        for (int j = 0; j < PER; ++j) v[i * PER + j] = (float)u.e[j];
    }
}

template <int W, class E, int N>
__device__ __forceinline__ void store_as(E* p, const float (&v)[N]) {
    constexpr int B = W * (int)sizeof(E) < 16 ? W * (int)sizeof(E) : 16;
    constexpr int PER = B / (int)sizeof(E);
    using R = typename Raw<B>::T;
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
        union U { R r; E e[PER]; __device__ U() {} } u;
#pragma unroll
        for (int j = 0; j < PER; ++j) u.e[j] = (E)v[i * PER + j];
        *reinterpret_cast<R*>(p + i * PER) = u.r;
    }
}

template <int W, int N>
__device__ __forceinline__ void load_any(const void* base, long long off, int type, float (&v)[N]) {
    if (type == PLM_F32) load_as<W>(static_cast<const float*>(base) + off, v);
    else if (type == PLM_F16) load_as<W>(static_cast<const __half*>(base) + off, v);
    else load_as<W>(static_cast<const __nv_bfloat16*>(base) + off, v);
}
template <int W, int N>
__device__ __forceinline__ void store_any(void* base, long long off, int type, const float (&v)[N]) {
    if (type == PLM_F32) store_as<W>(static_cast<float*>(base) + off, v);
    else if (type == PLM_F16) store_as<W>(static_cast<__half*>(base) + off, v);
    else store_as<W>(static_cast<__nv_bfloat16*>(base) + off, v);
}

template <int V, bool HALF>
__global__ void __launch_bounds__(RT) rope_kernel(const __grid_constant__ RopeArgs A) {
    __shared__ __align__(16) float cs_c[ROPE_CS], cs_s[ROPE_CS];
    grid_launch_dependents();
    grid_wait_prior();
    const long long t0 = (long long)blockIdx.x * A.tb;
    const int nt = (int)min((long long)A.tb, A.tokens - t0);
    const int pairs = A.r >> 1;
    for (int i = threadIdx.x; i < nt * pairs; i += RT) {
        const int t = i / pairs;
        const unsigned long long turn =
            (unsigned long long)(long long)__ldg(A.positions + t0 + t) * __ldg(A.freqs + (i - t * pairs));
        float s, c;
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
        cs_c[i] = c * A.scale;
        cs_s[i] = A.inverse ? -s * A.scale : s * A.scale;
    }
    __syncthreads();
    const int upr = A.d / (2 * V);                    // units per head row
    const int heads = A.head0[A.count];
    const int units = nt * heads * upr;
    const int rot_units = pairs / V;
    for (int u = blockIdx.y * RT + threadIdx.x; u < units; u += RT * gridDim.y) {
        const int row = u / upr, un = u - row * upr;
        const int t = row / heads, hj = row - t * heads;
        int j = 0;
        while (hj >= A.head0[j + 1]) ++j;
        const plm_rope_tensor& T = A.t[j];
        const int h = hj - A.head0[j];
        const long long tok = t0 + t;
        const long long xo = tok * T.x_token_stride + h * T.x_head_stride;
        long long yo = h * T.y_head_stride;
        if (T.slots) {
            const long long slot = __ldg(T.slots + tok);
            if (slot < 0 || slot >= T.pages * T.page_tokens) continue;
            const long long page = slot / T.page_tokens;
            yo += page * T.page_stride + (slot - page * T.page_tokens) * T.y_token_stride;
        } else {
            yo += tok * T.y_token_stride;
        }
        if (un < rot_units && T.rotate) {
            float c[V], s[V], a[V], b[V];
            load_as<V>(cs_c + t * pairs + un * V, c);
            load_as<V>(cs_s + t * pairs + un * V, s);
            if (HALF) {
                load_any<V>(T.x, xo + un * V, T.x_type, a);
                load_any<V>(T.x, xo + pairs + un * V, T.x_type, b);
            } else {
                float v[2 * V];
                load_any<V>(T.x, xo + 2 * un * V, T.x_type, v);
#pragma unroll
                for (int i = 0; i < V; ++i) { a[i] = v[2 * i]; b[i] = v[2 * i + 1]; }
            }
            float p[V], q[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                p[i] = a[i] * c[i] - b[i] * s[i];
                q[i] = b[i] * c[i] + a[i] * s[i];
            }
            if (HALF) {
                store_any<V>(T.y, yo + un * V, T.y_type, p);
                store_any<V>(T.y, yo + pairs + un * V, T.y_type, q);
            } else {
                float v[2 * V];
#pragma unroll
                for (int i = 0; i < V; ++i) { v[2 * i] = p[i]; v[2 * i + 1] = q[i]; }
                store_any<V>(T.y, yo + 2 * un * V, T.y_type, v);
            }
        } else {
            float v[2 * V];
            load_any<V>(T.x, xo + 2 * un * V, T.x_type, v);
            store_any<V>(T.y, yo + 2 * un * V, T.y_type, v);
        }
    }
}

int type_bytes(int type) { return type == PLM_F32 ? 4 : 2; }

// Whether every access of V pairs is aligned to its size (at most 16 bytes).
bool rope_fits(const RopeArgs& A, int V) {
    if (A.d % (2 * V) || A.r % (2 * V)) return false;
    auto ok = [&](const void* p, int64_t s0, int64_t s1, int64_t s2, int type) {
        int64_t al = (int64_t)V * type_bytes(type);
        if (al > 16) al = 16;
        const int64_t el = al / type_bytes(type);
        return (uintptr_t)p % al == 0 && s0 % el == 0 && s1 % el == 0 && s2 % el == 0;
    };
    for (int j = 0; j < A.count; ++j) {
        const plm_rope_tensor& T = A.t[j];
        if (!ok(T.x, T.x_token_stride, T.x_head_stride, 0, T.x_type)) return false;
        if (!ok(T.y, T.y_token_stride, T.y_head_stride, T.slots ? T.page_stride : 0, T.y_type)) return false;
    }
    return true;
}

template <int V>
cudaError_t rope_launch(const RopeArgs& A, int layout, dim3 grid, cudaStream_t stream) {
    return layout == PLM_ROPE_HALF ? launch_kernel(rope_kernel<V, true>, grid, dim3(RT), 0, stream, A)
                                   : launch_kernel(rope_kernel<V, false>, grid, dim3(RT), 0, stream, A);
}

}  // namespace

cudaError_t launch_rope(const plm_rope_tensor* tensors, int count, const int32_t* positions, const uint64_t* freqs,
                        long long tokens, int head_dim, int rotary_dim, int layout, float scale, int inverse,
                        cudaStream_t stream) {
    RopeArgs A = {};
    A.count = count;
    for (int j = 0; j < count; ++j) {
        A.t[j] = tensors[j];
        A.head0[j + 1] = A.head0[j] + (int)tensors[j].heads;
    }
    A.positions = positions;
    A.freqs = reinterpret_cast<const unsigned long long*>(freqs);
    A.tokens = tokens;
    A.d = head_dim;
    A.r = rotary_dim;
    A.scale = scale;
    A.inverse = inverse;
    const int V = rope_fits(A, 8) ? 8 : rope_fits(A, 4) ? 4 : rope_fits(A, 2) ? 2 : 1;
    // Tokens per CTA: enough (c, s) pairs to occupy its threads, while every
    // SM still gets CTAs; few tokens are spread over CTAs by heads instead.
    const int sms = num_sms();
    int tb = 2 * RT / rotary_dim;
    if (tb > tokens / (2 * sms)) tb = (int)(tokens / (2 * sms));
    while (tb > 1 && (long long)tb * A.head0[count] * (head_dim / (2 * V)) > (1 << 20)) tb /= 2;   // int unit index
    if (tb < 1) tb = 1;
    A.tb = tb;
    const long long gx = (tokens + tb - 1) / tb;
    const long long units = (long long)tb * A.head0[count] * (head_dim / (2 * V));
    long long gy = (units + RT - 1) / RT;                 // CTAs that one unit per thread needs
    const long long room = 4LL * sms / gx;
    if (gy > room) gy = room;
    if (gy < 1) gy = 1;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    switch (V) {
        case 8: return rope_launch<8>(A, layout, grid, stream);
        case 4: return rope_launch<4>(A, layout, grid, stream);
        case 2: return rope_launch<2>(A, layout, grid, stream);
        default: return rope_launch<1>(A, layout, grid, stream);
    }
}

}  // namespace plm

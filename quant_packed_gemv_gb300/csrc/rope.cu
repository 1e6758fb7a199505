// Rotary positions (plm_rope): pairs (a, b) of every head turned by
// position * frequency, written as rows or into cache pages.
//
// Mathematics.  y = (a c - b s, b c + a s) with c + i s = scale e^(i angle),
// angle = 2 pi frac(p f).  f is a 64-bit fraction of a turn, so the low 64
// bits of the integer product p * f are the fraction, exactly; its top 32
// bits as a signed number are turns in [-1/2, 1/2), and sincospi of twice
// that needs no range reduction.
//
// Bound: HBM (each value read and written once, ~1 operation per byte); next is
// the issue of the address and conversion work around the two FMAs a pair.  A CTA
// takes TB tokens: its threads first put the TB * R/2 (c, s) pairs into shared
// memory (one sincospi each, shared by all heads) and work out where each token
// goes in the cache, then walk the head rows of one tensor after the other, in
// a loop made for its types.  A unit is V pairs (or 2V values past the rotary
// part): V = 8 gives 16-byte accesses of 16-bit types; smaller V where the rotary
// size, a stride or a pointer is not a multiple of that.  A thread steps from unit
// to unit by additions.  (With the types, the tensor and 64-bit divisions for the
// slots looked up per unit, the kernel ran at 70 % of the copy rate.)
// One GB300: 16381 tokens x 40 heads of 128, bf16: 55 us, 6.1 TB/s (91 % of a
// copy); 8191 x 48 heads, f32 to bf16 pages: 53.5 us, 5.6 TB/s; one token 2.9 us.
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
constexpr int ROPE_TB = 4;       // tokens of a CTA at most

struct RopeArgs {
    plm_rope_tensor t[PLM_ROPE_MAX_TENSORS];
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

// The head rows of one tensor, of types X to Y.
template <int V, bool HALF, class X, class Y>
__device__ __forceinline__ void rope_rows(const plm_rope_tensor& T, long long t0, int nt, int d, int pairs, const float* cs_c,
                                          const float* cs_s, const long long* place, int first, int step) {
    const int upr = d / (2 * V), rot_units = T.rotate ? pairs / V : 0;   // units per head row, turned ones
    const int heads = (int)T.heads;
    const X* const x = static_cast<const X*>(T.x) + t0 * T.x_token_stride;
    Y* const y = static_cast<Y*>(T.y);
    const long long xt = T.x_token_stride, xh = T.x_head_stride, yh = T.y_head_stride;
    const bool paged = T.slots != nullptr;
    int row = first / upr, un = first - row * upr, t = row / heads, h = row - t * heads;
    const int row_step = step / upr, un_step = step - row_step * upr, t_step = row_step / heads, h_step = row_step - t_step * heads;
    while (t < nt) {
        const long long base = place[t];
        if (!paged || base >= 0) {
            const X* const xp = x + t * xt + h * xh;
            Y* const yp = y + base + h * yh;
            if (un < rot_units) {
                float c[V], s[V], v[2 * V];
                if (HALF) {
                    load_as<V>(xp + un * V, *reinterpret_cast<float (*)[V]>(v));
                    load_as<V>(xp + pairs + un * V, *reinterpret_cast<float (*)[V]>(v + V));
                } else {
                    load_as<V>(xp + 2 * un * V, v);
                }
                load_as<V>(cs_c + t * pairs + un * V, c);
                load_as<V>(cs_s + t * pairs + un * V, s);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float& a = v[HALF ? i : 2 * i];
                    float& b = v[HALF ? V + i : 2 * i + 1];
                    const float p = a * c[i] - b * s[i], q = b * c[i] + a * s[i];
                    a = p;
                    b = q;
                }
                if (HALF) {
                    store_as<V>(yp + un * V, *reinterpret_cast<float (*)[V]>(v));
                    store_as<V>(yp + pairs + un * V, *reinterpret_cast<float (*)[V]>(v + V));
                } else {
                    store_as<V>(yp + 2 * un * V, v);
                }
            } else {
                float v[2 * V];
                load_as<V>(xp + 2 * un * V, v);
                store_as<V>(yp + 2 * un * V, v);
            }
        }
        un += un_step;
        int carry = 0;
        if (un >= upr) { un -= upr; carry = 1; }
        h += h_step + carry;
        t += t_step;
        while (h >= heads) { h -= heads; ++t; }
    }
}

// CTA (x, y): tokens x * TB .., tensors y, y + gridDim.y, ..
template <int V, bool HALF>
__global__ void __launch_bounds__(RT, 6) rope_kernel(const __grid_constant__ RopeArgs A) {
    __shared__ __align__(16) float cs_c[ROPE_CS], cs_s[ROPE_CS];
    __shared__ long long place[PLM_ROPE_MAX_TENSORS][ROPE_TB];   // a token's offset in y, -1: not written
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
    for (int i = threadIdx.x; i < nt * A.count; i += RT) {
        const int j = i / nt, t = i - j * nt;
        const plm_rope_tensor& T = A.t[j];
        long long yo = (t0 + t) * T.y_token_stride;
        if (T.slots) {
            const long long slot = __ldg(T.slots + t0 + t);
            yo = -1;
            if (slot >= 0 && slot < T.pages * T.page_tokens) {
                const long long page = slot / T.page_tokens;
                yo = page * T.page_stride + (slot - page * T.page_tokens) * T.y_token_stride;
            }
        }
        place[j][t] = yo;
    }
    __syncthreads();
#pragma unroll 1
    for (int j = blockIdx.y; j < A.count; j += gridDim.y) {
        const plm_rope_tensor& T = A.t[j];
        auto rows = [&](auto x, auto y) {
            rope_rows<V, HALF, decltype(x), decltype(y)>(T, t0, nt, A.d, pairs, cs_c, cs_s, place[j], threadIdx.x, RT);
        };
        auto from = [&](auto x) {
            if (T.y_type == PLM_F32) rows(x, float());
            else if (T.y_type == PLM_F16) rows(x, __half());
            else rows(x, __nv_bfloat16());
        };
        if (T.x_type == PLM_F32) from(float());
        else if (T.x_type == PLM_F16) from(__half());
        else from(__nv_bfloat16());
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
    for (int j = 0; j < count; ++j) A.t[j] = tensors[j];
    A.positions = positions;
    A.freqs = reinterpret_cast<const unsigned long long*>(freqs);
    A.tokens = tokens;
    A.d = head_dim;
    A.r = rotary_dim;
    A.scale = scale;
    A.inverse = inverse;
    const int V = rope_fits(A, 8) ? 8 : rope_fits(A, 4) ? 4 : rope_fits(A, 2) ? 2 : 1;
    // Tokens per CTA: enough (c, s) pairs to occupy its threads, while every
    // SM still gets CTAs; few tokens are spread over CTAs by tensors instead.
    const int sms = num_sms();
    // (Four tokens: 2 and 8 measured 66 and 56 us where 4 takes 55, on 16381 x 40
    // heads of 128 in bf16; 53 and 57 us on f32 into pages.)
    int tb = 2 * RT / rotary_dim < 4 ? 2 * RT / rotary_dim : ROPE_TB;
    if (tb > tokens / (2 * sms)) tb = (int)(tokens / (2 * sms));
    if (tb < 1) tb = 1;
    A.tb = tb;
    const long long gx = (tokens + tb - 1) / tb;
    const dim3 grid((unsigned)gx, gx < 2 * sms ? (unsigned)count : 1u);
    switch (V) {
        case 8: return rope_launch<8>(A, layout, grid, stream);
        case 4: return rope_launch<4>(A, layout, grid, stream);
        case 2: return rope_launch<2>(A, layout, grid, stream);
        default: return rope_launch<1>(A, layout, grid, stream);
    }
}

}  // namespace plm

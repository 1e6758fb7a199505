// A cache in 8 bits: rows turned by their positions and written as blocks of
// 32 codes with a power of two (plm_kv8_write), and read back (plm_kv8_read).
//
// Mathematics.  A block's power of two is 2^j, the smallest with amax 2^-j <
// 127.5: with amax = f 2^k, 1 <= f < 2, j = k - 6, or k - 5 where 64 f >= 127.5.
// Scaling by it is exact, so a code is one rounding, and the value code 2^j is
// exact in f32 and bf16.  The turning is plm_rope's (csrc/rope.cu).
//
// Layout.  Writing, eight lanes take a block, four values each: 16 bytes of f32
// in, 4 codes out, the block's maximum by three shuffles.  A lane of a turned
// row also loads the four values that its own are paired with (they are in L1).
// Reading, four lanes take a block, eight values each.
#include "plm_device.cuh"
#include "plm_internal.h"
#include "values.cuh"

namespace plm {

namespace {

constexpr int WT = 256;          // threads per CTA
constexpr int KV8_TB = 4;        // tokens of a CTA at most
constexpr float LARGEST = 0x1p120f;

struct Kv8Args {
    plm_kv8_tensor t[PLM_ROPE_MAX_TENSORS];
    bool four[PLM_ROPE_MAX_TENSORS];     // four values of a row in one access
    int count;
    const int32_t* positions;
    const unsigned long long* freqs;
    long long tokens;
    int d, r, tb, half, turned;          // turned: a tensor rotates
    float scale;
};

// Where a token's codes and exponents begin, -1: nowhere.
__device__ __forceinline__ longlong2 kv8_place(const plm_kv8_tensor& T, long long slot, int blocks) {
    if (slot < 0 || slot >= T.pages * T.page_tokens) return make_longlong2(-1, 0);
    const long long page = slot / T.page_tokens, at = slot - page * T.page_tokens;
    return make_longlong2(page * T.page_stride + at * T.token_stride, page * T.exp_page_stride + at * blocks);
}

__device__ __forceinline__ float cut(float v) {   // NaN: 0
    return v != v ? 0.0f : fminf(fmaxf(v, -LARGEST), LARGEST);
}

// Dim i of a row, turned.
__device__ __forceinline__ float turned_at(const Kv8Args& A, const plm_kv8_tensor& T, long long row, int i, const float* cs_c,
                                           const float* cs_s) {
    const float x = value_at(T.rows, T.type, row + i);
    if (i >= A.r) return x;
    const int h = A.r >> 1;
    const bool second = A.half ? i >= h : i & 1;
    const int p = A.half ? (second ? i - h : i) : i >> 1;
    const float z = value_at(T.rows, T.type, row + (A.half ? (second ? i - h : i + h) : i ^ 1));
    return second ? x * cs_c[p] + z * cs_s[p] : x * cs_c[p] - z * cs_s[p];
}

// CTA (x, y): tokens x * tb .., tensors y, y + gridDim.y, ..
__global__ void __launch_bounds__(WT) kv8_write_kernel(const __grid_constant__ Kv8Args A) {
    extern __shared__ __align__(16) float cs[];   // cos then sin of a token's pairs, per token
    __shared__ longlong2 place[PLM_ROPE_MAX_TENSORS][KV8_TB];
    grid_launch_dependents();
    grid_wait_prior();
    const long long t0 = (long long)blockIdx.x * A.tb;
    const int nt = (int)min((long long)A.tb, A.tokens - t0), blocks = A.d >> 5;
    const int pairs = A.turned ? A.r >> 1 : 0, pitch = (pairs + 3) & ~3;   // rows of the table stay 16-byte aligned
    float* const cs_c = cs;
    float* const cs_s = cs + nt * pitch;
    for (int i = threadIdx.x; i < nt * pairs; i += WT) {
        const int t = i / pairs, p = i - t * pairs;
        const unsigned long long turn = (unsigned long long)(long long)__ldg(A.positions + t0 + t) * __ldg(A.freqs + p);
        float s, c;
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
        cs_c[t * pitch + p] = c * A.scale;
        cs_s[t * pitch + p] = s * A.scale;
    }
    for (int i = threadIdx.x; i < nt * A.count; i += WT) {
        const int j = i / nt, t = i - j * nt;
        place[j][t] = kv8_place(A.t[j], __ldg(reinterpret_cast<const long long*>(A.t[j].slots) + t0 + t), blocks);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, sub = lane & 7;
#pragma unroll 1
    for (int j = blockIdx.y; j < A.count; j += gridDim.y) {
        const plm_kv8_tensor& T = A.t[j];
        const int units = nt * (int)T.heads * blocks, h = A.r >> 1;
        const bool four = A.four[j], turns = T.rotate != 0;
        // a turned block by whole accesses: every pair's two halves are multiples of four apart
        const bool plain = four && (A.half ? h % 4 == 0 : A.r % 4 == 0);
        for (int u0 = (threadIdx.x >> 5) * 4; u0 < units; u0 += WT / 8) {   // a warp's four blocks
            const int u = u0 + (lane >> 3);
            const bool in = u < units;
            const int row = in ? u / blocks : 0, b = in ? u - row * blocks : 0, t = row / (int)T.heads, head = row - t * (int)T.heads;
            const longlong2 at = place[j][t];
            const int i = 32 * b + 4 * sub;
            const long long from = (t0 + t) * T.row_token_stride + head * T.row_head_stride;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (in && at.x >= 0) {
                const float* c = cs_c + t * pitch;
                const float* s = cs_s + t * pitch;
                if (!turns || (plain && i >= A.r)) {
                    v = load_four(T.rows, T.type, from + i, 4, four);
                } else if (plain) {
                    v = load_four(T.rows, T.type, from + i, 4, true);
                    if (A.half) {
                        const bool second = i >= h;
                        const float4 z = load_four(T.rows, T.type, from + (second ? i - h : i + h), 4, true);
                        const int p = second ? i - h : i;
                        const float4 cc = *reinterpret_cast<const float4*>(c + p);
                        float4 ss = *reinterpret_cast<const float4*>(s + p);
                        if (!second) ss = make_float4(-ss.x, -ss.y, -ss.z, -ss.w);
                        v = make_float4(v.x * cc.x + z.x * ss.x, v.y * cc.y + z.y * ss.y, v.z * cc.z + z.z * ss.z, v.w * cc.w + z.w * ss.w);
                    } else {
                        const float2 cc = *reinterpret_cast<const float2*>(c + (i >> 1)), ss = *reinterpret_cast<const float2*>(s + (i >> 1));
                        v = make_float4(v.x * cc.x - v.y * ss.x, v.y * cc.x + v.x * ss.x, v.z * cc.y - v.w * ss.y, v.w * cc.y + v.z * ss.y);
                    }
                } else {
                    v = make_float4(turned_at(A, T, from, i, c, s), turned_at(A, T, from, i + 1, c, s), turned_at(A, T, from, i + 2, c, s),
                                    turned_at(A, T, from, i + 3, c, s));
                }
                v = make_float4(cut(v.x), cut(v.y), cut(v.z), cut(v.w));
            }
            uint32_t top = __float_as_uint(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            if (!in || at.x < 0) continue;
            // e = 127 + j, at least 27; zeros: 0
            int e = max((int)(top >> 23) - 6 + ((top & 0x7FFFFFu) >= 0x7F0000u ? 1 : 0), 27);
            if (top == 0) e = 0;
            const float back = e == 0 ? 0.0f : __uint_as_float((uint32_t)(254 - e) << 23);   // 2^-j
            const int q0 = __float2int_rn(v.x * back), q1 = __float2int_rn(v.y * back), q2 = __float2int_rn(v.z * back), q3 = __float2int_rn(v.w * back);
            *reinterpret_cast<uint32_t*>(T.codes + at.x + head * T.head_stride + i) =
                (uint32_t)(q0 & 0xFF) | (uint32_t)(q1 & 0xFF) << 8 | (uint32_t)(q2 & 0xFF) << 16 | (uint32_t)(q3 & 0xFF) << 24;
            if (sub == 0) T.exps[at.y + head * T.exp_head_stride + b] = (uint8_t)e;
        }
    }
}

// A thread per eight values; grid y: tensors.
__global__ void __launch_bounds__(WT) kv8_read_kernel(const __grid_constant__ Kv8Args A) {
    grid_launch_dependents();
    grid_wait_prior();
    const plm_kv8_tensor& T = A.t[blockIdx.y];
    const int blocks = A.d >> 5, parts = 4 * blocks;
    const long long units = A.tokens * T.heads * parts;
    for (long long u = (long long)blockIdx.x * WT + threadIdx.x; u < units; u += (long long)gridDim.x * WT) {
        const long long row = u / parts, t = row / T.heads;
        const int i = 8 * (int)(u - row * parts), head = (int)(row - t * T.heads);
        const longlong2 at = kv8_place(T, __ldg(reinterpret_cast<const long long*>(T.slots) + t), blocks);
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
        if (at.x >= 0) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(T.codes + at.x + head * T.head_stride + i);
            const uint32_t w0 = w[0], w1 = w[1];
            const float s = __uint_as_float((uint32_t)T.exps[at.y + head * T.exp_head_stride + (i >> 5)] << 23);
            auto code = [](uint32_t x, int k) { return (float)(int)(int8_t)(x >> (8 * k)); };
            a = make_float4(code(w0, 0) * s, code(w0, 1) * s, code(w0, 2) * s, code(w0, 3) * s);
            b = make_float4(code(w1, 0) * s, code(w1, 1) * s, code(w1, 2) * s, code(w1, 3) * s);
        }
        const long long to = t * T.row_token_stride + head * T.row_head_stride + i;
        store_four(T.rows, T.type, to, 4, A.four[blockIdx.y], a);
        store_four(T.rows, T.type, to + 4, 4, A.four[blockIdx.y], b);
    }
}

Kv8Args kv8_args(const plm_kv8_tensor* tensors, int count, long long tokens, int head_dim) {
    Kv8Args A = {};
    A.count = count;
    A.tokens = tokens;
    A.d = head_dim;
    for (int j = 0; j < count; ++j) {
        const plm_kv8_tensor& t = A.t[j] = tensors[j];
        A.four[j] = four_aligned(t.rows, t.row_token_stride, t.type) && t.row_head_stride % 4 == 0;
    }
    return A;
}

}  // namespace

cudaError_t launch_kv8_write(const plm_kv8_tensor* tensors, int count, const int32_t* positions, const uint64_t* freqs,
                             long long tokens, int head_dim, int rotary_dim, int layout, float scale, cudaStream_t stream) {
    Kv8Args A = kv8_args(tensors, count, tokens, head_dim);
    A.positions = positions;
    A.freqs = reinterpret_cast<const unsigned long long*>(freqs);
    A.r = rotary_dim;
    A.half = layout == PLM_ROPE_HALF;
    A.scale = scale;
    for (int j = 0; j < count; ++j) A.turned |= tensors[j].rotate != 0;
    const int sms = num_sms();
    int tb = KV8_TB;
    if (tb > tokens / (2 * sms)) tb = (int)(tokens / (2 * sms));
    if (tb < 1) tb = 1;
    A.tb = tb;
    const long long gx = (tokens + tb - 1) / tb;
    const int pitch = A.turned ? (rotary_dim / 2 + 3) & ~3 : 0;
    return launch_kernel(kv8_write_kernel, dim3((unsigned)gx, gx < 2 * sms ? (unsigned)count : 1u), dim3(WT),
                         (size_t)tb * pitch * 2 * sizeof(float), stream, A);
}

cudaError_t launch_kv8_read(const plm_kv8_tensor* tensors, int count, long long tokens, int head_dim, cudaStream_t stream) {
    const Kv8Args A = kv8_args(tensors, count, tokens, head_dim);
    long long most = 0;
    for (int j = 0; j < count; ++j) most = tensors[j].heads > most ? tensors[j].heads : most;
    long long ctas = (tokens * most * (head_dim / 8) + WT - 1) / WT;
    const long long cap = 64LL * num_sms();
    if (ctas > cap) ctas = cap;
    return launch_kernel(kv8_read_kernel, dim3((unsigned)ctas, (unsigned)count), dim3(WT), 0, stream, A);
}

}  // namespace plm

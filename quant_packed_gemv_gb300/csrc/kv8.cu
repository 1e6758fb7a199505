// A cache in 8 bits: rows turned by their positions and written as blocks of
// 32 codes with a power of two (plm_kv8_write), and read back (plm_kv8_read).
//
// Mathematics.  A block's power of two is 2^j, the smallest with amax 2^-j <
// 127.5: with amax = f 2^k, 1 <= f < 2, j = k - 6, or k - 5 where 64 f >= 127.5.
// Scaling by it is exact, so a code is one rounding, and the value code 2^j is
// exact in f32 and bf16.  The turning is plm_rope's (csrc/rope.cu).
//
// Layout.  A CTA takes a few tokens: where each goes, and the cosines and sines of
// its pairs, are worked out once, in shared memory.  A warp takes some heads of a
// token: written, eight values a lane and four lanes a block; read back, sixteen a
// lane.  The rows of a lane differ by the head alone, so their places are one
// addition apart, and their loads are issued together.  The values that a lane's are
// paired with come from another lane.
//
// Bound: HBM (a value's bytes and 33 / 32 of a byte), for writing after the issue of ~10
// instructions a value.  One GB300, 8 heads of 128, keys and values: 8191 tokens from f32,
// interleaved pairs, half of each head turned, 18.5 us (4.5 TB/s), all of it 18.9; halves 20.6
// and 21.1, whose kernels spill 28 to 36 bytes at their 80 registers; 48000 tokens of scattered
// slots into bf16 52 us (5.6 TB/s); 61 tokens written in 3.8 us and read in 2.2, which is latency.
#include <type_traits>

#include "plm_device.cuh"
#include "plm_internal.h"
#include "values.cuh"

namespace plm {

namespace {

constexpr int WT = 256;          // threads per CTA
// Tokens of a CTA at most (4: 59 us for the 48000 instead of 52, 24.9 for the 8191 instead of 18.5;
// 16: 50 and 20.0).
constexpr int KV8_TB = 8;
// Rows that a lane has in flight.  8 heads of 128, 48000 tokens read: 52 us with one, 61
// with two, 69 with four (registers, and longer runs of a CTA); 8191 written, interleaved and in
// halves: 21 and 29 with one, 22 and 23 with two, 18.5 and 20.6 with four, 27 and 42 with eight.
constexpr int READ_ROWS = 1, WRITE_ROWS = 4;
constexpr float LARGEST = 0x1p120f;

struct Kv8Args {
    plm_kv8_tensor t[PLM_ROPE_MAX_TENSORS];
    bool eight[PLM_ROPE_MAX_TENSORS];    // rows in accesses of 16 bytes
    bool wide[PLM_ROPE_MAX_TENSORS];     // and codes (written: 8 bytes)
    int groups[PLM_ROPE_MAX_TENSORS];    // of heads that a warp takes at a time
    int shift[PLM_ROPE_MAX_TENSORS];     // their logarithm, -1: they are no power of two
    int lanes, rows, passes;             // of a warp: lanes a row, rows at once, passes over longer rows
    int count;
    const int32_t* positions;
    const unsigned long long* freqs;
    long long tokens;
    int d, r, tb, half, turned;          // turned: a tensor rotates
    float scale;
};

// Where a token's codes and exponents begin; x = -1: nowhere.
__device__ __forceinline__ longlong2 kv8_place(const plm_kv8_tensor& T, long long slot, int blocks) {
    if (slot < 0 || slot >= T.pages * T.page_tokens) return make_longlong2(-1, 0);
    // (a division of 32 bits where that does: the whole CTA waits for it)
    const long long page = (slot | T.page_tokens) >> 32 ? slot / T.page_tokens : (uint32_t)slot / (uint32_t)T.page_tokens;
    const long long at = slot - page * T.page_tokens;
    return make_longlong2(page * T.page_stride + at * T.token_stride, page * T.exp_page_stride + at * blocks);
}
using Places = longlong2[PLM_ROPE_MAX_TENSORS][KV8_TB];

// The places of the CTA's tokens in `count` tensors.
__device__ __forceinline__ void find_places(const Kv8Args& A, Places& place, long long t0, int nt, int first, int count) {
    if ((int)threadIdx.x < nt * count) {   // (64 at most)
        const int j = first + threadIdx.x / nt, t = threadIdx.x % nt;
        place[j][t] = kv8_place(A.t[j], __ldg(reinterpret_cast<const long long*>(A.t[j].slots) + t0 + t), A.d >> 5);
    }
}

// The lane's part of a warp's item: token, part of the row (of `parts`), first of its heads
// (the next is A.rows on); there: a part of the row.  The warp's items are N rows a lane.
struct Item {
    int t, part, h;
    bool there;
    template <int N> static __device__ __forceinline__ Item of(const Kv8Args& A, int j, int item, int parts, int lane, int row, std::integral_constant<int, N>) {
        int pass = 0;
        if (A.passes > 1) {
            pass = item % A.passes;
            item /= A.passes;
        }
        Item I;
        I.t = A.shift[j] >= 0 ? item >> A.shift[j] : item / A.groups[j];
        I.part = 32 * pass + lane - row * A.lanes;
        I.h = (item - I.t * A.groups[j]) * N * A.rows + row;
        I.there = row < A.rows && I.part < parts;
        return I;
    }
};

__device__ __forceinline__ float cut(float v) {   // NaN: 0
    return v != v ? 0.0f : fminf(fmaxf(v, -LARGEST), LARGEST);
}
__device__ __forceinline__ float larger(float a, float b) {   // of the sizes; NaN if one is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
__device__ __forceinline__ float block_top(const float (&v)[8]) {   // of four lanes
    float top = larger(larger(larger(v[0], v[1]), larger(v[2], v[3])), larger(larger(v[4], v[5]), larger(v[6], v[7])));
    top = larger(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    return larger(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
}

// Eight values from i on, as whole accesses.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <class E> __device__ __forceinline__ void load8(const E* p, float (&v)[8]) {
    union { uint4 u; E e[8]; } x = {*reinterpret_cast<const uint4*>(p)};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)x.e[i];
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

// A block's part of eight values into its codes, and the block's exponent.
__device__ __forceinline__ void put_part(int8_t* codes, uint8_t* exps, bool in, bool first, bool wide, float (&v)[8]) {
    float most = block_top(v);
    if (__any_sync(0xFFFFFFFFu, !(most <= LARGEST))) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = cut(v[k]);
        most = block_top(v);
    }
    const uint32_t top = __float_as_uint(most);
    if (!in) return;
    // e = 127 + j, at least 27; zeros: 0
    int e = max((int)(top >> 23) - 6 + ((top & 0x7FFFFFu) >= 0x7F0000u ? 1 : 0), 27);
    if (top == 0) e = 0;
    const float back = e == 0 ? 0.0f : __uint_as_float((uint32_t)(254 - e) << 23);   // 2^-j
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        // rounded by adding 1.5 2^23; the code is the low byte
        uint32_t q[4];
#pragma unroll
        for (int l = 0; l < 4; ++l) q[l] = __float_as_uint(fmaf(v[4 * k + l], back, 12582912.0f));
        w[k] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    }
    if (wide) {
        *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
    } else {
        reinterpret_cast<uint32_t*>(codes)[0] = w[0];
        reinterpret_cast<uint32_t*>(codes)[1] = w[1];
    }
    if (first) *exps = (uint8_t)e;
}

// The rows of one tensor.  WHOLE: in accesses of 16 bytes, a turned row's pairs in
// parts, laid out as HALF says; else value by value.
template <class X, bool WHOLE, bool HALF>
__device__ __forceinline__ void write_rows(const Kv8Args& A, int j, int row0, const longlong2* place, long long t0, int nt,
                                           const float* cs_c, const float* cs_s, int pitch, bool wide) {
    const plm_kv8_tensor& T = A.t[j];
    const int lane = threadIdx.x & 31, h = A.r >> 1, heads = (int)T.heads;
    const bool turns = T.rotate != 0;
    const int parts = A.d >> 3, items = nt * A.groups[j] * A.passes;
    for (int item = threadIdx.x >> 5; item < items; item += WT / 32) {
        const Item at = Item::of(A, j, item, parts, lane, row0, std::integral_constant<int, WRITE_ROWS>());
        const longlong2 to = place[at.t];
        const int i = 8 * at.part;
        const long long from = (t0 + at.t) * T.row_token_stride + at.h * T.row_head_stride;
        const long long head_step = A.rows * T.row_head_stride;
        const bool there = at.there && to.x >= 0, turned = there && turns && i < A.r, second = i >= h;
        float v[WRITE_ROWS][8], c[8], s[8];
        bool in[WRITE_ROWS];
#pragma unroll
        for (int k = 0; k < WRITE_ROWS; ++k) {
            in[k] = there && at.h + k * A.rows < heads;
#pragma unroll
            for (int l = 0; l < 8; ++l) v[k][l] = 0.0f;
            if (!in[k]) continue;
            const long long row = from + k * head_step;
            if constexpr (WHOLE) {
                load8(static_cast<const X*>(T.rows) + row + i, v[k]);
            } else {
#pragma unroll
                for (int l = 0; l < 8; ++l)
                    v[k][l] = turned ? turned_at(A, T, row, i + l, cs_c + at.t * pitch, cs_s + at.t * pitch) : value_at(T.rows, T.type, row + i + l);
            }
        }
        if (WHOLE && turns) {
            if (turned) {
                const int p = at.t * pitch + (HALF ? (second ? i - h : i) : i >> 1);
                if constexpr (HALF) {
                    load8(cs_c + p, c);
                    load8(cs_s + p, s);
#pragma unroll
                    for (int l = 0; l < 8; ++l) s[l] = second ? s[l] : -s[l];
                } else {
                    const float4 c4 = *reinterpret_cast<const float4*>(cs_c + p), s4 = *reinterpret_cast<const float4*>(cs_s + p);
                    c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
                    s[0] = s4.x; s[1] = s4.y; s[2] = s4.z; s[3] = s4.w;
                }
            }
            // the values that a lane's are paired with: another lane has them, or (rows of several passes) L1
            const int mate = turned ? (second ? lane - (h >> 3) : lane + (h >> 3)) : lane;
#pragma unroll
            for (int k = 0; k < WRITE_ROWS; ++k) {
                if constexpr (HALF) {
                    float z[8];
                    if (A.passes == 1) {
#pragma unroll
                        for (int l = 0; l < 8; ++l) z[l] = __shfl_sync(0xFFFFFFFFu, v[k][l], mate);
                    } else if (turned && in[k]) {
                        load8(static_cast<const X*>(T.rows) + from + k * head_step + (second ? i - h : i + h), z);
                    }
                    if (turned && in[k])
#pragma unroll
                        for (int l = 0; l < 8; ++l) v[k][l] = v[k][l] * c[l] + z[l] * s[l];
                } else if (turned) {
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        const float a = v[k][2 * l], b = v[k][2 * l + 1];
                        v[k][2 * l] = a * c[l] - b * s[l];
                        v[k][2 * l + 1] = b * c[l] + a * s[l];
                    }
                }
            }
        }
        int8_t* codes = T.codes + to.x + at.h * T.head_stride + i;
        uint8_t* exps = T.exps + to.y + at.h * T.exp_head_stride + (i >> 5);
#pragma unroll
        for (int k = 0; k < WRITE_ROWS; ++k) {
            put_part(codes, exps, in[k], (i & 31) == 0, wide, v[k]);
            codes += A.rows * T.head_stride;
            exps += A.rows * T.exp_head_stride;
        }
    }
}

// CTA (x, y): tokens x * tb .., tensors y, y + gridDim.y, ..
template <class X, bool WHOLE, bool HALF>
__global__ void __launch_bounds__(WT, 3) kv8_write_kernel(const __grid_constant__ Kv8Args A) {
    extern __shared__ __align__(16) float cs[];   // cosines, then sines, of the tokens' pairs
    __shared__ Places place;
    grid_launch_dependents();
    grid_wait_prior();
    const long long t0 = (long long)blockIdx.x * A.tb;
    const int nt = (int)min((long long)A.tb, A.tokens - t0), row0 = (threadIdx.x & 31) / A.lanes;   // the lane's row among those of a warp
    const int pairs = A.turned ? A.r >> 1 : 0, pitch = (pairs + 3) & ~3;   // rows of the table stay 16-byte aligned
    float* const cs_s = cs + nt * pitch;
    for (int i = threadIdx.x; i < nt * pairs; i += WT) {
        const int t = i / pairs, p = i - t * pairs;
        const unsigned long long turn = (unsigned long long)(long long)__ldg(A.positions + t0 + t) * __ldg(A.freqs + p);
        float s, c;
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
        cs[t * pitch + p] = c * A.scale;
        cs_s[t * pitch + p] = s * A.scale;
    }
    find_places(A, place, t0, nt, 0, A.count);
    __syncthreads();
#pragma unroll 1
    for (int j = blockIdx.y; j < A.count; j += gridDim.y) write_rows<X, WHOLE, HALF>(A, j, row0, place[j], t0, nt, cs, cs_s, pitch, A.wide[j]);
}

// Sixteen values from their codes, into rows of type E.
__device__ __forceinline__ float value_of(uint32_t w, int i, float s) {   // w: codes + 128
    // 2^23 + (c + 128), less 2^23 + 128 (before the product: 2^23 s may be too large)
    return (__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 | i)) - 8388736.0f) * s;
}
template <class Y> __device__ __forceinline__ void put_values(Y* y, const uint32_t (&q)[4], float s) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t r[4];
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            const uint32_t w = q[2 * k + (l >> 1)];
            const float a = value_of(w, 2 * (l & 1), s), b = value_of(w, 2 * (l & 1) + 1, s);
            if constexpr (std::is_same<Y, __half>::value) {
                const __half2 x = __floats2half2_rn(a, b);
                r[l] = *reinterpret_cast<const uint32_t*>(&x);
            } else {
                const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
                r[l] = *reinterpret_cast<const uint32_t*>(&x);
            }
        }
        *reinterpret_cast<uint4*>(y + 8 * k) = make_uint4(r[0], r[1], r[2], r[3]);
    }
}
template <> __device__ __forceinline__ void put_values<float>(float* y, const uint32_t (&q)[4], float s) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<float4*>(y + 4 * k) = make_float4(value_of(q[k], 0, s), value_of(q[k], 1, s), value_of(q[k], 2, s), value_of(q[k], 3, s));
}

template <class Y, bool WHOLE>
__device__ __forceinline__ void read_rows(const Kv8Args& A, int j, int row0, const longlong2* place, long long t0, int nt, bool wide) {
    const plm_kv8_tensor& T = A.t[j];
    const int lane = threadIdx.x & 31, heads = (int)T.heads;
    const int parts = A.d >> 4, items = nt * A.groups[j] * A.passes;
    for (int item = threadIdx.x >> 5; item < items; item += WT / 32) {
        const Item at = Item::of(A, j, item, parts, lane, row0, std::integral_constant<int, READ_ROWS>());
        const longlong2 from = place[at.t];
        const int i = 16 * at.part;
        const int8_t* codes = T.codes + from.x + at.h * T.head_stride + i;
        const uint8_t* exps = T.exps + from.y + at.h * T.exp_head_stride + (i >> 5);
        uint32_t q[READ_ROWS][4], e[READ_ROWS];
        bool in[READ_ROWS];
#pragma unroll
        for (int k = 0; k < READ_ROWS; ++k) {
            in[k] = at.there && at.h + k * A.rows < heads;
            q[k][0] = q[k][1] = q[k][2] = q[k][3] = e[k] = 0;
            if (in[k] && from.x >= 0) {
                if (wide) {
                    const uint4 v = *reinterpret_cast<const uint4*>(codes);
                    q[k][0] = v.x; q[k][1] = v.y; q[k][2] = v.z; q[k][3] = v.w;
                } else {
#pragma unroll
                    for (int l = 0; l < 4; ++l) q[k][l] = reinterpret_cast<const uint32_t*>(codes)[l];
                }
                e[k] = *exps;
            }
            codes += A.rows * T.head_stride;
            exps += A.rows * T.exp_head_stride;
        }
        long long to = (t0 + at.t) * T.row_token_stride + at.h * T.row_head_stride + i;
#pragma unroll
        for (int k = 0; k < READ_ROWS; ++k) {
            const float s = __uint_as_float(e[k] << 23);
#pragma unroll
            for (int l = 0; l < 4; ++l) q[k][l] ^= 0x80808080u;
            if (in[k]) {
                if constexpr (WHOLE) {
                    put_values(static_cast<Y*>(T.rows) + to, q[k], s);
                } else {
#pragma unroll
                    for (int l = 0; l < 16; ++l) value_put(T.rows, T.type, to + l, value_of(q[k][l >> 2], l & 3, s));
                }
            }
            to += A.rows * T.row_head_stride;
        }
    }
}

// CTA (x, y): tokens x * tb .. of tensor y.
template <class Y, bool WHOLE>
__global__ void __launch_bounds__(WT) kv8_read_kernel(const __grid_constant__ Kv8Args A) {
    __shared__ Places place;
    grid_launch_dependents();
    grid_wait_prior();
    const int j = blockIdx.y, row0 = (threadIdx.x & 31) / A.lanes;
    const long long t0 = (long long)blockIdx.x * A.tb;
    const int nt = (int)min((long long)A.tb, A.tokens - t0);
    find_places(A, place, t0, nt, j, 1);
    __syncthreads();
    read_rows<Y, WHOLE>(A, j, row0, place[j], t0, nt, A.wide[j]);
}

// per: values of a lane; rows: of a lane at a time
Kv8Args kv8_args(const plm_kv8_tensor* tensors, int count, long long tokens, int head_dim, int per, int rows) {
    Kv8Args A = {};
    A.count = count;
    A.tokens = tokens;
    A.d = head_dim;
    const int parts = head_dim / per;
    A.passes = (parts + 31) / 32;
    A.lanes = parts < 32 ? parts : 32;
    A.rows = 32 / A.lanes;
    for (int j = 0; j < count; ++j) {
        const plm_kv8_tensor& t = A.t[j] = tensors[j];
        A.eight[j] = (uintptr_t)t.rows % 16 == 0 && t.row_token_stride * type_bytes(t.type) % 16 == 0 &&
                     t.row_head_stride * type_bytes(t.type) % 16 == 0;
        A.groups[j] = (int)(t.heads + rows * A.rows - 1) / (rows * A.rows);
        A.shift[j] = -1;
        for (int k = 0; k < 20; ++k)
            if (A.groups[j] == 1 << k) A.shift[j] = k;
        A.wide[j] = (uintptr_t)t.codes % 16 == 0 && t.page_stride % 16 == 0 && t.head_stride % 16 == 0 && t.token_stride % 16 == 0;
    }
    return A;
}

// Tokens per CTA, while every SM still gets some.
int kv8_tokens(long long tokens) {
    const long long tb = tokens / (2 * num_sms());
    return tb > KV8_TB ? KV8_TB : tb < 1 ? 1 : (int)tb;
}

}  // namespace

cudaError_t launch_kv8_write(const plm_kv8_tensor* tensors, int count, const int32_t* positions, const uint64_t* freqs,
                             long long tokens, int head_dim, int rotary_dim, int layout, float scale, cudaStream_t stream) {
    Kv8Args A = kv8_args(tensors, count, tokens, head_dim, 8, WRITE_ROWS);
    A.positions = positions;
    A.freqs = reinterpret_cast<const unsigned long long*>(freqs);
    A.r = rotary_dim;
    A.half = layout == PLM_ROPE_HALF;
    A.scale = scale;
    for (int j = 0; j < count; ++j) A.turned |= tensors[j].rotate != 0;
    A.tb = kv8_tokens(tokens);
    const long long ctas = (tokens + A.tb - 1) / A.tb;
    const int pitch = A.turned ? (rotary_dim / 2 + 3) & ~3 : 0;
    const dim3 grid((unsigned)ctas, ctas < 2 * num_sms() ? (unsigned)count : 1u);
    const size_t bytes = (size_t)A.tb * pitch * 2 * sizeof(float);
    // whole accesses: all rows of one type, and of turned ones the rotary part, for halves each half, made of parts
    const int type = tensors[0].type;
    bool whole = !A.turned || rotary_dim % (A.half ? 16 : 8) == 0;
    for (int j = 0; j < count; ++j) whole = whole && A.eight[j] && tensors[j].type == type;
    auto run = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(WT), bytes, stream, A); };
    if (!whole) return run(kv8_write_kernel<float, false, false>);
    if (type == PLM_F32) return A.half ? run(kv8_write_kernel<float, true, true>) : run(kv8_write_kernel<float, true, false>);
    if (type == PLM_F16) return A.half ? run(kv8_write_kernel<__half, true, true>) : run(kv8_write_kernel<__half, true, false>);
    return A.half ? run(kv8_write_kernel<__nv_bfloat16, true, true>) : run(kv8_write_kernel<__nv_bfloat16, true, false>);
}

cudaError_t launch_kv8_read(const plm_kv8_tensor* tensors, int count, long long tokens, int head_dim, cudaStream_t stream) {
    Kv8Args A = kv8_args(tensors, count, tokens, head_dim, 16, READ_ROWS);
    A.tb = kv8_tokens(tokens);
    const dim3 grid((unsigned)((tokens + A.tb - 1) / A.tb), (unsigned)count);
    const int type = tensors[0].type;
    bool whole = true;   // accesses of 16 bytes: all rows of one type
    for (int j = 0; j < count; ++j) whole = whole && A.eight[j] && tensors[j].type == type;
    auto run = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(WT), 0, stream, A); };
    if (!whole) return run(kv8_read_kernel<float, false>);
    return type == PLM_F32 ? run(kv8_read_kernel<float, true>) : type == PLM_F16 ? run(kv8_read_kernel<__half, true>) : run(kv8_read_kernel<__nv_bfloat16, true>);
}

}  // namespace plm

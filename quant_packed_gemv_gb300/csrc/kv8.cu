// A cache in 8 bits: rows turned by their positions and written as blocks of
// 32 codes with a power of two (plm_kv8_write), and read back (plm_kv8_read).
//
// Mathematics.  A block's power of two is 2^j, the smallest with amax 2^-j <
// 127.5: with amax = f 2^k, 1 <= f < 2, j = k - 6, or k - 5 where 64 f >= 127.5.
// Scaling by it is exact, so a code is one rounding, and the value code 2^j is
// exact in f32 and bf16.  The turning is plm_rope's (csrc/rope.cu).
//
// Layout.  A CTA takes a few tokens: where each goes, and the cosines and sines of
// its pairs, are worked out once, in shared memory.  Four lanes take a block, eight
// values each; a thread has two such parts in flight and steps from part to part by
// additions.  A lane of a turned row also loads the eight values that its own are
// paired with (they are in L1).
#include "plm_device.cuh"
#include "plm_internal.h"
#include "values.cuh"

namespace plm {

namespace {

constexpr int WT = 256;          // threads per CTA
constexpr int KV8_TB = 8;        // tokens of a CTA at most
constexpr int AT_ONCE = 2;       // parts of eight values that a thread has in flight
constexpr float LARGEST = 0x1p120f;

struct Kv8Args {
    plm_kv8_tensor t[PLM_ROPE_MAX_TENSORS];
    bool eight[PLM_ROPE_MAX_TENSORS];    // eight values of a row in whole accesses
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
    const long long page = slot / T.page_tokens, at = slot - page * T.page_tokens;
    return make_longlong2(page * T.page_stride + at * T.token_stride, page * T.exp_page_stride + at * blocks);
}
using Places = longlong2[PLM_ROPE_MAX_TENSORS][KV8_TB];
__device__ __forceinline__ void find_places(const Kv8Args& A, Places& place, long long t0, int nt, int first, int tensors) {
    for (int i = threadIdx.x; i < nt * tensors; i += WT) {
        const int j = first + i / nt, t = i % nt;
        place[j][t] = kv8_place(A.t[j], __ldg(reinterpret_cast<const long long*>(A.t[j].slots) + t0 + t), A.d >> 5);
    }
}

// The parts of a CTA's tokens: part of a row, head, token; WT parts on at a time.
struct Walk {
    int part, h, t, parts, heads, part_step, h_step, t_step;
    __device__ Walk(int parts_, int heads_) : parts(parts_), heads(heads_) {
        int row = threadIdx.x / parts;
        part = threadIdx.x - row * parts;
        t = row / heads;
        h = row - t * heads;
        row = WT / parts;
        part_step = WT - row * parts;
        t_step = row / heads;
        h_step = row - t_step * heads;
    }
    __device__ __forceinline__ void next() {
        part += part_step;
        h += h_step;
        t += t_step;
        if (part >= parts) { part -= parts; ++h; }
        if (h >= heads) { h -= heads; ++t; }
    }
};

__device__ __forceinline__ float cut(float v) {   // NaN: 0
    return v != v ? 0.0f : fminf(fmaxf(v, -LARGEST), LARGEST);
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
__device__ __forceinline__ void put_part(const plm_kv8_tensor& T, longlong2 at, int head, int i, bool in, float (&v)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        v[k] = cut(v[k]);
        top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    }
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
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
    int8_t* const to = T.codes + at.x + head * T.head_stride + i;
    if ((reinterpret_cast<uintptr_t>(to) & 7) == 0) {
        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    } else {
        reinterpret_cast<uint32_t*>(to)[0] = w[0];
        reinterpret_cast<uint32_t*>(to)[1] = w[1];
    }
    if ((i & 31) == 0) T.exps[at.y + head * T.exp_head_stride + (i >> 5)] = (uint8_t)e;
}

// The rows of one tensor, in whole accesses; a turned one's pairs lie in parts.
template <class X>
__device__ __forceinline__ void write_rows(const Kv8Args& A, const plm_kv8_tensor& T, const longlong2* place, long long t0, int nt,
                                           const float* cs_c, const float* cs_s, int pitch) {
    const int units = nt * (int)T.heads * (A.d >> 3), h = A.r >> 1;
    const bool turns = T.rotate != 0;
    Walk at(A.d >> 3, (int)T.heads);
    for (int u = 0; u < units; u += AT_ONCE * WT) {
        float v[AT_ONCE][8], z[AT_ONCE][8];
        Walk w[AT_ONCE] = {at, at};
        bool in[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            w[k] = at;
            at.next();
            in[k] = u + k * WT + (int)threadIdx.x < units && place[min(w[k].t, nt - 1)].x >= 0;
            const X* row = static_cast<const X*>(T.rows) + (t0 + w[k].t) * T.row_token_stride + w[k].h * T.row_head_stride;
            const int i = 8 * w[k].part;
#pragma unroll
            for (int l = 0; l < 8; ++l) v[k][l] = 0.0f;
            if (in[k]) {
                load8(row + i, v[k]);
                if (turns && A.half && i < A.r) load8(row + (i >= h ? i - h : i + h), z[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int i = 8 * w[k].part;
            if (in[k] && turns && i < A.r) {
                const float* c = cs_c + w[k].t * pitch;
                const float* s = cs_s + w[k].t * pitch;
                float cc[8], ss[8];
                if (A.half) {
                    const bool second = i >= h;
                    const int p = second ? i - h : i;
                    load8(c + p, cc);
                    load8(s + p, ss);
#pragma unroll
                    for (int l = 0; l < 8; ++l) v[k][l] = v[k][l] * cc[l] + z[k][l] * (second ? ss[l] : -ss[l]);
                } else {
                    const float4 c4 = *reinterpret_cast<const float4*>(c + (i >> 1)), s4 = *reinterpret_cast<const float4*>(s + (i >> 1));
                    cc[0] = c4.x; cc[1] = c4.y; cc[2] = c4.z; cc[3] = c4.w;
                    ss[0] = s4.x; ss[1] = s4.y; ss[2] = s4.z; ss[3] = s4.w;
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        const float a = v[k][2 * l], b = v[k][2 * l + 1];
                        v[k][2 * l] = a * cc[l] - b * ss[l];
                        v[k][2 * l + 1] = b * cc[l] + a * ss[l];
                    }
                }
            }
            put_part(T, place[min(w[k].t, nt - 1)], w[k].h, i, in[k], v[k]);
        }
    }
}

// The same value by value: other alignments, pairs and sizes.
__device__ __noinline__ void write_rows_slowly(const Kv8Args& A, const plm_kv8_tensor& T, const longlong2* place, long long t0, int nt,
                                               const float* cs_c, const float* cs_s, int pitch) {
    const int units = nt * (int)T.heads * (A.d >> 3);
    Walk at(A.d >> 3, (int)T.heads);
#pragma unroll 1
    for (int u = 0; u < units; u += WT, at.next()) {
        const longlong2 to = place[min(at.t, nt - 1)];
        const bool in = u + (int)threadIdx.x < units && to.x >= 0;
        const long long row = (t0 + at.t) * T.row_token_stride + at.h * T.row_head_stride;
        float v[8];
#pragma unroll
        for (int l = 0; l < 8; ++l) {
            const int i = 8 * at.part + l;
            v[l] = !in ? 0.0f : T.rotate ? turned_at(A, T, row, i, cs_c + at.t * pitch, cs_s + at.t * pitch) : value_at(T.rows, T.type, row + i);
        }
        put_part(T, to, at.h, 8 * at.part, in, v);
    }
}

// CTA (x, y): tokens x * tb .., tensors y, y + gridDim.y, ..
__global__ void __launch_bounds__(WT) kv8_write_kernel(const __grid_constant__ Kv8Args A) {
    extern __shared__ __align__(16) float cs[];   // cosines then sines of the tokens' pairs
    __shared__ Places place;
    grid_launch_dependents();
    grid_wait_prior();
    const long long t0 = (long long)blockIdx.x * A.tb;
    const int nt = (int)min((long long)A.tb, A.tokens - t0);
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
    find_places(A, place, t0, nt, 0, A.count);
    __syncthreads();
#pragma unroll 1
    for (int j = blockIdx.y; j < A.count; j += gridDim.y) {
        const plm_kv8_tensor& T = A.t[j];
        // whole accesses of a turned row: the rotary part, and for halves each half, is made of parts
        const bool whole = A.eight[j] && (!T.rotate || A.r % (A.half ? 16 : 8) == 0);
        if (!whole) write_rows_slowly(A, T, place[j], t0, nt, cs_c, cs_s, pitch);
        else if (T.type == PLM_F32) write_rows<float>(A, T, place[j], t0, nt, cs_c, cs_s, pitch);
        else if (T.type == PLM_F16) write_rows<__half>(A, T, place[j], t0, nt, cs_c, cs_s, pitch);
        else write_rows<__nv_bfloat16>(A, T, place[j], t0, nt, cs_c, cs_s, pitch);
    }
}

// CTA (x, y): tokens x * tb .. of tensor y.
__global__ void __launch_bounds__(WT) kv8_read_kernel(const __grid_constant__ Kv8Args A) {
    __shared__ Places place;
    grid_launch_dependents();
    grid_wait_prior();
    const int j = blockIdx.y;
    const plm_kv8_tensor& T = A.t[j];
    const long long t0 = (long long)blockIdx.x * A.tb;
    const int nt = (int)min((long long)A.tb, A.tokens - t0);
    find_places(A, place, t0, nt, j, 1);
    __syncthreads();
    const int units = nt * (int)T.heads * (A.d >> 3);
    const bool eight = A.eight[j];
    Walk at(A.d >> 3, (int)T.heads);
    for (int u = 0; u < units; u += AT_ONCE * WT) {
        uint32_t q[AT_ONCE][2], e[AT_ONCE];
        Walk w[AT_ONCE] = {at, at};
        bool in[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            w[k] = at;
            at.next();
            in[k] = u + k * WT + (int)threadIdx.x < units;
            const longlong2 from = place[j][min(w[k].t, nt - 1)];
            q[k][0] = q[k][1] = e[k] = 0;
            if (in[k] && from.x >= 0) {
                const int8_t* codes = T.codes + from.x + w[k].h * T.head_stride + 8 * w[k].part;
                if ((reinterpret_cast<uintptr_t>(codes) & 7) == 0) {
                    const uint2 v = *reinterpret_cast<const uint2*>(codes);
                    q[k][0] = v.x;
                    q[k][1] = v.y;
                } else {
                    q[k][0] = reinterpret_cast<const uint32_t*>(codes)[0];
                    q[k][1] = reinterpret_cast<const uint32_t*>(codes)[1];
                }
                e[k] = T.exps[from.y + w[k].h * T.exp_head_stride + (w[k].part >> 2)];
            }
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            if (!in[k]) continue;
            const float s = __uint_as_float(e[k] << 23);
            // a code as 2^23 + (c + 128), less 2^23 + 128
            auto code = [&](int i) {
                return (__uint_as_float(__byte_perm(q[k][i >> 2] ^ 0x80808080u, 0x4B000000u, 0x7650 | (i & 3))) - 8388736.0f) * s;
            };
            const long long to = (t0 + w[k].t) * T.row_token_stride + w[k].h * T.row_head_stride + 8 * w[k].part;
            if (eight && T.type != PLM_F32) {
                uint32_t r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (T.type == PLM_F16) {
                        const __half2 x = __floats2half2_rn(code(2 * i), code(2 * i + 1));
                        r[i] = *reinterpret_cast<const uint32_t*>(&x);
                    } else {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(code(2 * i), code(2 * i + 1));
                        r[i] = *reinterpret_cast<const uint32_t*>(&x);
                    }
                }
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(T.rows) + to) = make_uint4(r[0], r[1], r[2], r[3]);
            } else {
                store_four(T.rows, T.type, to, 4, eight, make_float4(code(0), code(1), code(2), code(3)));
                store_four(T.rows, T.type, to + 4, 4, eight, make_float4(code(4), code(5), code(6), code(7)));
            }
        }
    }
}

Kv8Args kv8_args(const plm_kv8_tensor* tensors, int count, long long tokens, int head_dim) {
    Kv8Args A = {};
    A.count = count;
    A.tokens = tokens;
    A.d = head_dim;
    for (int j = 0; j < count; ++j) {
        const plm_kv8_tensor& t = A.t[j] = tensors[j];
        A.eight[j] = (uintptr_t)t.rows % 16 == 0 && t.row_token_stride * type_bytes(t.type) % 16 == 0 &&
                     t.row_head_stride * type_bytes(t.type) % 16 == 0;
    }
    return A;
}

// Tokens per CTA: some parts for each thread, while every SM still gets CTAs.
int kv8_tokens(const Kv8Args& A, long long tokens) {
    long long tb = 8 * WT / ((A.d >> 3) * A.t[0].heads);
    if (tb > KV8_TB) tb = KV8_TB;
    if (tb > tokens / (2 * num_sms())) tb = tokens / (2 * num_sms());
    return tb < 1 ? 1 : (int)tb;
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
    A.tb = kv8_tokens(A, tokens);
    const long long gx = (tokens + A.tb - 1) / A.tb;
    const int pitch = A.turned ? (rotary_dim / 2 + 3) & ~3 : 0;
    return launch_kernel(kv8_write_kernel, dim3((unsigned)gx, gx < 2 * num_sms() ? (unsigned)count : 1u), dim3(WT),
                         (size_t)A.tb * pitch * 2 * sizeof(float), stream, A);
}

cudaError_t launch_kv8_read(const plm_kv8_tensor* tensors, int count, long long tokens, int head_dim, cudaStream_t stream) {
    Kv8Args A = kv8_args(tensors, count, tokens, head_dim);
    A.tb = kv8_tokens(A, tokens);
    return launch_kernel(kv8_read_kernel, dim3((unsigned)((tokens + A.tb - 1) / A.tb), (unsigned)count), dim3(WT), 0, stream, A);
}

}  // namespace plm

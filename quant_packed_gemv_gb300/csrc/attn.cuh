// What the attention kernels share: the problem as they see it, the visible
// lengths, element conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/plm.h"
#include "plm_device.cuh"
#include "plm_internal.h"

namespace plm {

struct AttnArgs {
    const void* q;
    void* o;
    float* lse;
    const void* k;
    const void* v;
    const int* table;
    const int* lens;
    const int* seqs;
    int batch, nq, heads, kv_heads, group;   // group = heads / kv_heads
    long long q_ts, q_hs, o_ts, o_hs;
    long long page_stride, kv_hs, kv_ts, table_stride;
    int page_shift, pages, rows;
    int prefix, cap;                         // prefix_len; lengths are cut to cap
    float scale;
    int o_f32;
};

// Table row of sequence b, or -1.
__device__ __forceinline__ int attn_row(const AttnArgs& A, int b) {
    const int r = A.seqs ? A.seqs[b] : b;
    return r >= 0 && r < A.rows ? r : -1;
}
__device__ __forceinline__ int attn_len(const AttnArgs& A, int row) {
    return row < 0 ? 0 : max(0, min(A.lens[row], A.cap));
}
// Keys that query t of a sequence of len tokens sees.
__device__ __forceinline__ int attn_seen(const AttnArgs& A, int len, int t) { return max(0, len - A.nq + t + 1); }

template <class E> __device__ __forceinline__ float2 pair_to_f32(uint32_t u);
template <> __device__ __forceinline__ float2 pair_to_f32<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<__half2*>(&u));
}
template <> __device__ __forceinline__ float2 pair_to_f32<__nv_bfloat16>(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

}  // namespace plm

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
    unsigned group_inv;                      // 65536 / group, rounded up: r / group for r, group < 256
    long long q_ts, q_hs, o_ts, o_hs;
    long long page_stride, kv_hs, kv_ts, table_stride;
    int page_shift, pages, rows;
    int prefix, cap;                         // prefix_len; lengths are cut to cap
    float scale;
    int o_f32;
};

// r / group for r < 256 (an integer division is ~100 cycles in a row).
__device__ __forceinline__ int small_row(const AttnArgs& A, int r) { return (int)(((unsigned)r * A.group_inv) >> 16); }

// Table row of sequence b, or -1; its length.
__device__ __forceinline__ int attn_row_of(const AttnArgs& A, int r) { return r >= 0 && r < A.rows ? r : -1; }
__device__ __forceinline__ int attn_row(const AttnArgs& A, int b) { return attn_row_of(A, A.seqs ? A.seqs[b] : b); }
__device__ __forceinline__ int attn_cut(const AttnArgs& A, int len) { return max(0, min(len, A.cap)); }
__device__ __forceinline__ int attn_len(const AttnArgs& A, int row) { return row < 0 ? 0 : attn_cut(A, A.lens[row]); }
// Keys that query t of a sequence of len tokens sees.
__device__ __forceinline__ int attn_seen(const AttnArgs& A, int len, int t) { return max(0, len - A.nq + t + 1); }

template <class E> __device__ __forceinline__ float2 pair_to_f32(uint32_t u);
template <> __device__ __forceinline__ float2 pair_to_f32<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<__half2*>(&u));
}
template <> __device__ __forceinline__ float2 pair_to_f32<__nv_bfloat16>(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

// Two f32 rounded to the cache's type, the first in the low half: p for the second
// product, and O.  The tensor cores take both operands of a product in one type, V's;
// p in f32 would be two products, of its upper and its lower bits, and the second
// product is half of the work.  Each p is off by 2^-8 of itself at most in bf16 (2^-11
// in f16), in either direction: over the cases of perf/operators.py the outputs' error
// is 0.0022 of their size in bf16 and 0.00027 in f16, where p in f32 gives 0.0017 and
// 0.00021, mostly the output's own rounding.
template <class E> __device__ __forceinline__ uint32_t pack_pair(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack_pair<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <> __device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four values of an output row, at element offset off (a multiple of 4).
template <class E>
__device__ __forceinline__ void attn_store4(const AttnArgs& A, long long off, float4 v) {
    if (A.o_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(A.o) + off) = v;
    else
        *reinterpret_cast<uint2*>(static_cast<E*>(A.o) + off) = make_uint2(pack_pair<E>(v.x, v.y), pack_pair<E>(v.z, v.w));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The cluster's CTAs: a barrier over all their threads, and shared memory of
// the CTA of rank z at the place of `p` here.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, int z) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(z));
    return a;
}
__device__ __forceinline__ float peer_f32(const float* p, int z) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_addr(p, z)) : "memory");
    return v;
}
__device__ __forceinline__ float4 peer_f32x4(const float* p, int z) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer_addr(p, z)) : "memory");
    return v;
}

}  // namespace plm

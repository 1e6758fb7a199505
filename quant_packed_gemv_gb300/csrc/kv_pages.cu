// Pages of a key/value cache, kept on the device (plm_kv_*): sequences grow
// (reserve), split (fork), end (free); a sparse pool is packed (compact).
//
// A page is free when its reference count is 0; there is no free list to keep
// in step.  A call that hands out pages counts what its items need (a prefix
// sum over the items), then walks the counts in index order until it has
// found that many free pages.  Both are done by one CTA: 1024 threads read
// 64 K counts (256 KB) in a few microseconds.  As the lowest free pages are handed
// out, those below are in use, and the walk reads about as many counts as there are
// live pages; packing reads all.  (Millions of small pages would take one CTA a
// millisecond.)  What follows touches each item, table row and page independently and runs on the
// whole GPU; reference counts change by integer atomics, whose order does not
// show.  Bound: HBM for the calls that move pages (each moved page read and
// written once), launch latency for the others.  One GB300: packing 3000 pages of
// 1.8 MB, 55 % in use: 420 us, 6.5 TB/s; 37 sequences into 8 each, such pages: 115 us
// (5.0 TB/s of distinct bytes); 61 sequences grow by a token: 8.6 us; 300 end: 4.3.
#include <cstdint>

#include "../../include/plm.h"
#include "plm_device.cuh"
#include "plm_internal.h"

namespace plm {

namespace {

constexpr int PT = 1024;     // threads of the planning CTA
constexpr int AT = 256;      // threads of the others
constexpr int CHUNK = 4096;  // bytes a warp copies at a time

// Workspace: counters, per item (first new page, number of new pages), then
// two page lists.
struct Plan {
    int* head;     // [0] pages to move (fork: last pages; compact), [1] 1 if the call is done, 0 if out of pages
    int* first;    // [n] index of the item's first new page in `fresh`
    int* need;     // [n] new pages of the item; -1: a bad item
    int* fresh;    // [pages] new pages in ascending order; compact: the holes
    int* src;      // [max(pages, n)] pages to copy from; reserve: [n] the items' lengths before
    int* dst;      // fork: [n] pages to copy to; compact: map of moved pages [pages]
};

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

size_t plan_bytes(long long pages, long long n) {
    const long long m = pages > n ? pages : n;
    return up256(64) + 2 * up256(4 * (size_t)n) + up256(4 * (size_t)pages) + 2 * up256(4 * (size_t)m);
}

Plan plan_at(void* ws, long long pages, long long n) {
    const long long m = pages > n ? pages : n;
    uint8_t* p = static_cast<uint8_t*>(ws);
    Plan P;
    auto take = [&](size_t b) { int* r = reinterpret_cast<int*>(p); p += up256(b); return r; };
    P.head = take(64);
    P.first = take(4 * (size_t)n);
    P.need = take(4 * (size_t)n);
    P.fresh = take(4 * (size_t)pages);
    P.src = take(4 * (size_t)m);
    P.dst = take(4 * (size_t)m);
    return P;
}

// Exclusive prefix sum of v over the CTA's PT threads; total gets the sum.
template <class T> __device__ T cta_scan(T v, T& total) {
    __shared__ T sums[33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // sums of an earlier scan have been read
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T w = sums[lane], z = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xFFFFFFFFu, z, o);
            if (lane >= o) z += y;
        }
        sums[lane] = z - w;
        if (lane == 31) sums[32] = z;
    }
    __syncthreads();
    total = sums[32];
    return sums[warp] + x - v;
}

__device__ __forceinline__ void flag(const plm_kv_state& S, int bit) {
    if (S.status) atomicOr(S.status, bit);
}

__device__ __forceinline__ long long pages_for(long long tokens, long long per) { return (tokens + per - 1) / per; }

// The first `want` free pages in ascending order; returns how many there are
// (at most want).
__device__ int find_free(const plm_kv_state& S, int want, int* fresh) {
    int have = 0;
    for (long long p0 = 0; p0 < S.pages && have < want; p0 += 4 * PT) {
        const long long p = p0 + 4 * threadIdx.x;
        int r[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] = p + i < S.pages ? S.refs[p + i] : 1;
            mine += r[i] == 0;
        }
        int total;
        int at = have + cta_scan(mine, total);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] == 0) {
                if (at < want) fresh[at] = (int)(p + i);
                ++at;
            }
        have += total;
    }
    return have < want ? have : want;
}

// ---------------------------------------------------------------- reserve
struct ReserveArgs {
    plm_kv_state S;
    Plan P;
    const int* seqs;
    const int* add;
    long long n;
    long long* slots;
    long long slots_stride;
};

// One item, by a warp: its new table entries, counts, length and slots.  The length
// before is the plan's, for which the row was found long enough: of a sequence listed
// twice, the other item may have raised it since.
__device__ void reserve_item(const ReserveArgs& A, long long i, bool done, int lane) {
    const plm_kv_state& S = A.S;
    const int need = A.P.need[i];
    long long* slots = A.slots ? A.slots + i * A.slots_stride : nullptr;
    if (!done || need < 0) {
        if (slots)
            for (long long j = lane; j < A.slots_stride; j += 32) slots[j] = -1;
        return;
    }
    const int s = A.seqs[i];
    const long long old = A.P.src[i], add = A.add[i];
    int* row = S.table + (long long)s * S.max_pages;
    const long long have = pages_for(old, S.page_tokens);
    const int* fresh = A.P.fresh + A.P.first[i];
    for (int k = lane; k < need; k += 32) {
        row[have + k] = fresh[k];
        S.refs[fresh[k]] = 1;
    }
    if (slots)
        for (long long j = lane; j < A.slots_stride; j += 32) {
            long long v = -1;
            if (j < add) {
                const long long pos = old + j, col = pos / S.page_tokens;
                const int page = col < have ? row[col] : fresh[col - have];
                v = (long long)page * S.page_tokens + (pos - col * S.page_tokens);
            }
            slots[j] = v;
        }
    __syncwarp();
    if (lane == 0) S.lens[s] = (int)(old + add);
}

// apply != 0: the CTA also does the items (small calls: one launch).
__global__ void __launch_bounds__(PT) reserve_plan_kernel(const __grid_constant__ ReserveArgs A, int apply) {
    grid_launch_dependents();
    grid_wait_prior();
    const plm_kv_state& S = A.S;
    long long want = 0;   // rows of 2^21 pages: 1024 items can ask for 2^31
    for (long long i0 = 0; i0 < A.n; i0 += PT) {
        const long long i = i0 + threadIdx.x;
        int need = 0;
        if (i < A.n) {
            const int s = A.seqs[i], add = A.add[i];
            need = -1;
            if (s >= 0 && s < S.max_seqs && add >= 0) {
                const long long old = S.lens[s], now = old + add;
                A.P.src[i] = (int)old;
                if (old >= 0 && now <= 0x7FFFFFFFLL && pages_for(now, S.page_tokens) <= S.max_pages &&
                    (!A.slots || add <= A.slots_stride))
                    need = (int)(pages_for(now, S.page_tokens) - pages_for(old, S.page_tokens));
            }
            A.P.need[i] = need;
            if (need < 0) flag(S, PLM_KV_BAD_ITEM);
        }
        long long total;
        const long long at = want + cta_scan<long long>(max(need, 0), total);
        if (i < A.n) A.P.first[i] = (int)at;   // read only if all fit: it is at most S.pages then
        want += total;
    }
    const bool done = want <= S.pages && find_free(S, (int)want, A.P.fresh) == want;
    if (threadIdx.x == 0) {
        if (!done) flag(S, PLM_KV_OUT_OF_PAGES);
        A.P.head[1] = done;
    }
    if (!apply) return;
    __syncthreads();
    for (long long i = threadIdx.x >> 5; i < A.n; i += PT / 32) reserve_item(A, i, done, threadIdx.x & 31);
}

__global__ void __launch_bounds__(AT) reserve_apply_kernel(const __grid_constant__ ReserveArgs A) {
    grid_launch_dependents();
    grid_wait_prior();
    const bool done = A.P.head[1] != 0;
    for (long long i = ((long long)blockIdx.x * AT + threadIdx.x) >> 5; i < A.n; i += (long long)gridDim.x * (AT / 32))
        reserve_item(A, i, done, threadIdx.x & 31);
}

// ------------------------------------------------------------------- moves
// Pages src[k] -> dst[k], k < count: a warp moves CHUNK bytes at a time with
// 16-byte accesses, all its loads before its stores.
__device__ void copy_pages(const plm_kv_state& S, const int* src, const int* dst, long long count) {
    const long long per = (S.page_bytes + CHUNK - 1) / CHUNK;
    const int lane = threadIdx.x & 31;
    uint8_t* pool = static_cast<uint8_t*>(S.pool);
    const long long nw = (long long)gridDim.x * (AT / 32);
    for (long long u = ((long long)blockIdx.x * AT + threadIdx.x) >> 5; u < count * per; u += nw) {
        const long long k = u / per;
        const int from = src[k], to = dst[k];
        if (from < 0 || from >= S.pages || to < 0 || to >= S.pages) continue;
        const long long off = (u - k * per) * CHUNK + 16 * lane;
        const uint8_t* a = pool + from * S.page_bytes;
        uint8_t* b = pool + to * S.page_bytes;
        uint4 v[CHUNK / 512];
#pragma unroll
        for (int i = 0; i < CHUNK / 512; ++i)
            if (off + 512 * i < S.page_bytes) v[i] = *reinterpret_cast<const uint4*>(a + off + 512 * i);
#pragma unroll
        for (int i = 0; i < CHUNK / 512; ++i)
            if (off + 512 * i < S.page_bytes) *reinterpret_cast<uint4*>(b + off + 512 * i) = v[i];
    }
}

__global__ void __launch_bounds__(AT) copy_kernel(const __grid_constant__ plm_kv_state S, const int* src,
                                                  const int* dst, long long n) {
    grid_launch_dependents();
    grid_wait_prior();
    copy_pages(S, src, dst, n);
}

// -------------------------------------------------------------------- fork
struct ForkArgs {
    plm_kv_state S;
    Plan P;
    const int* parents;
    const int* children;
    const int* keep;
    long long n;
};

__device__ __forceinline__ long long fork_len(const ForkArgs& A, long long i) {
    const long long len = A.S.lens[A.parents[i]];
    return A.keep ? min(len, (long long)A.keep[i]) : len;
}

__global__ void __launch_bounds__(PT) fork_plan_kernel(const __grid_constant__ ForkArgs A) {
    grid_launch_dependents();
    grid_wait_prior();
    const plm_kv_state& S = A.S;
    int want = 0;
    for (long long i0 = 0; i0 < A.n; i0 += PT) {
        const long long i = i0 + threadIdx.x;
        int need = 0, last = -1;
        if (i < A.n) {
            const int p = A.parents[i], c = A.children[i];
            need = -1;
            if (p >= 0 && p < S.max_seqs && c >= 0 && c < S.max_seqs && c != p && S.lens[c] == 0 &&
                (!A.keep || A.keep[i] >= 0)) {
                const long long len = fork_len(A, i), full = len / S.page_tokens;
                if (len >= 0 && pages_for(len, S.page_tokens) <= S.max_pages) {
                    need = len % S.page_tokens != 0;
                    if (need) last = S.table[(long long)p * S.max_pages + full];
                }
            }
            A.P.need[i] = need;
            if (need < 0) flag(S, PLM_KV_BAD_ITEM);
        }
        int total;
        const int at = want + cta_scan<int>(need > 0, total);
        if (i < A.n) {
            A.P.first[i] = at;
            if (need > 0) A.P.src[at] = last;
        }
        want += total;
    }
    const bool done = find_free(S, want, A.P.fresh) == want;
    if (threadIdx.x == 0) {
        if (!done) flag(S, PLM_KV_OUT_OF_PAGES);
        A.P.head[0] = done ? want : 0;
        A.P.head[1] = done;
    }
}

__global__ void __launch_bounds__(AT) fork_apply_kernel(const __grid_constant__ ForkArgs A) {
    grid_launch_dependents();
    grid_wait_prior();
    const plm_kv_state& S = A.S;
    if (!A.P.head[1]) return;
    for (long long i = blockIdx.x; i < A.n; i += gridDim.x) {
        const int need = A.P.need[i];
        if (need < 0) continue;
        const long long len = fork_len(A, i), full = len / S.page_tokens;
        const int* from = S.table + (long long)A.parents[i] * S.max_pages;
        int* to = S.table + (long long)A.children[i] * S.max_pages;
        const int own = need ? A.P.fresh[A.P.first[i]] : -1;
        for (long long j = threadIdx.x; j < S.max_pages; j += AT) {
            int v = -1;
            if (j < full) {
                v = from[j];
                if (v >= 0 && v < S.pages) atomicAdd(S.refs + v, 1);
            } else if (j == full) {
                v = own;
            }
            to[j] = v;
        }
        if (threadIdx.x == 0) {
            S.lens[A.children[i]] = (int)len;
            if (need) S.refs[own] = 1;
        }
    }
    copy_pages(S, A.P.src, A.P.fresh, A.P.head[0]);
}

// -------------------------------------------------------------------- free
// One CTA per sequence.  An entry is taken out of the row by an exchange, so
// that a page is given back once even for a sequence listed twice.
__global__ void __launch_bounds__(AT) free_kernel(const __grid_constant__ plm_kv_state S, const int* seqs, long long n) {
    grid_launch_dependents();
    grid_wait_prior();
    for (long long i = blockIdx.x; i < n; i += gridDim.x) {
        const int s = seqs[i];
        if (s < 0 || s >= S.max_seqs) {
            if (threadIdx.x == 0) flag(S, PLM_KV_BAD_ITEM);
            continue;
        }
        int* row = S.table + (long long)s * S.max_pages;
        for (long long j = threadIdx.x; j < S.max_pages; j += AT) {
            const int p = atomicExch(row + j, -1);
            if (p >= 0 && p < S.pages) atomicSub(S.refs + p, 1);
        }
        if (threadIdx.x == 0) S.lens[s] = 0;
    }
}

// ----------------------------------------------------------------- compact
struct CompactArgs {
    plm_kv_state S;
    Plan P;
    int* live;
};

__global__ void __launch_bounds__(PT) compact_plan_kernel(const __grid_constant__ CompactArgs A) {
    grid_launch_dependents();
    grid_wait_prior();
    const plm_kv_state& S = A.S;
    int mine = 0, live;
    for (long long p = threadIdx.x; p < S.pages; p += PT) mine += S.refs[p] > 0;
    cta_scan(mine, live);
    int holes = 0, high = 0;
    for (long long p0 = 0; p0 < S.pages; p0 += PT) {
        const long long p = p0 + threadIdx.x;
        const bool in = p < S.pages, used = in && S.refs[p] > 0;
        const bool hole = in && !used && p < live, move = used && p >= live;
        int total;
        int at = holes + cta_scan<int>(hole, total);
        if (hole) A.P.fresh[at] = (int)p;
        holes += total;
        at = high + cta_scan<int>(move, total);
        if (move) A.P.src[at] = (int)p;
        high += total;
    }
    __syncthreads();   // the lists are complete: holes = high
    for (int k = threadIdx.x; k < high; k += PT) A.P.dst[A.P.src[k]] = A.P.fresh[k];
    if (threadIdx.x == 0) {
        A.P.head[0] = high;
        A.P.head[2] = live;
        if (A.live) *A.live = live;
    }
}

__global__ void __launch_bounds__(AT) compact_apply_kernel(const __grid_constant__ CompactArgs A) {
    grid_launch_dependents();
    grid_wait_prior();
    const plm_kv_state& S = A.S;
    const int moved = A.P.head[0], live = A.P.head[2];
    const long long me = (long long)blockIdx.x * AT + threadIdx.x, all = (long long)gridDim.x * AT;
    for (long long k = me; k < moved; k += all) {
        S.refs[A.P.fresh[k]] = S.refs[A.P.src[k]];
        S.refs[A.P.src[k]] = 0;
    }
    for (long long e = me; e < S.max_seqs * S.max_pages; e += all) {
        const int p = S.table[e];
        if (p >= live && p < S.pages) S.table[e] = A.P.dst[p];
    }
    copy_pages(S, A.P.src, A.P.fresh, moved);
}

unsigned grid_for(long long ctas, int per_sm) {
    const long long cap = (long long)num_sms() * per_sm;
    if (ctas > cap) ctas = cap;
    return (unsigned)(ctas < 1 ? 1 : ctas);
}

// CTAs that copy up to n pages.
unsigned copy_grid(const plm_kv_state& S, long long n) {
    const long long per = (S.page_bytes + CHUNK - 1) / CHUNK, warps = AT / 32;
    const long long most = (long long)num_sms() * 8;
    if (per > most * warps || n > most * warps) return (unsigned)most;
    return grid_for((n * per + warps - 1) / warps, 8);
}

}  // namespace

size_t kv_workspace_bytes(long long pages, long long n) { return plan_bytes(pages, n); }

cudaError_t launch_kv_reserve(const plm_kv_state& S, const int* seqs, const int* add, long long n, long long* slots,
                              long long slots_stride, void* ws, cudaStream_t stream) {
    const ReserveArgs A = {S, plan_at(ws, S.pages, n), seqs, add, n, slots, slots_stride};
    // up to 32 slots rows per warp, the planning CTA does the items itself
    const int apply = n * (slots ? slots_stride + 32 : 32) <= 1 << 16;
    cudaError_t e = launch_kernel(reserve_plan_kernel, dim3(1), dim3(PT), 0, stream, A, apply);
    if (e != cudaSuccess || apply) return e;
    return launch_kernel(reserve_apply_kernel, dim3(grid_for((n + AT / 32 - 1) / (AT / 32), 8)), dim3(AT), 0, stream, A);
}

cudaError_t launch_kv_fork(const plm_kv_state& S, const int* parents, const int* children, const int* keep, long long n,
                           void* ws, cudaStream_t stream) {
    const ForkArgs A = {S, plan_at(ws, S.pages, n), parents, children, keep, n};
    cudaError_t e = launch_kernel(fork_plan_kernel, dim3(1), dim3(PT), 0, stream, A);
    if (e != cudaSuccess) return e;
    const unsigned rows = grid_for(n, 8), copies = copy_grid(S, n);
    return launch_kernel(fork_apply_kernel, dim3(rows > copies ? rows : copies), dim3(AT), 0, stream, A);
}

cudaError_t launch_kv_free(const plm_kv_state& S, const int* seqs, long long n, cudaStream_t stream) {
    return launch_kernel(free_kernel, dim3(grid_for(n, 64)), dim3(AT), 0, stream, S, seqs, n);
}

cudaError_t launch_kv_compact(const plm_kv_state& S, int* live, void* ws, cudaStream_t stream) {
    const CompactArgs A = {S, plan_at(ws, S.pages, 0), live};
    cudaError_t e = launch_kernel(compact_plan_kernel, dim3(1), dim3(PT), 0, stream, A);
    if (e != cudaSuccess) return e;
    const unsigned copies = copy_grid(S, S.pages / 2 + 1);
    const unsigned rows = grid_for((S.max_seqs * S.max_pages + AT - 1) / AT, 8);
    return launch_kernel(compact_apply_kernel, dim3(rows > copies ? rows : copies), dim3(AT), 0, stream, A);
}

cudaError_t launch_kv_copy_pages(const plm_kv_state& S, const int* src, const int* dst, long long n,
                                 cudaStream_t stream) {
    return launch_kernel(copy_kernel, dim3(copy_grid(S, n)), dim3(AT), 0, stream, S, src, dst, n);
}

}  // namespace plm

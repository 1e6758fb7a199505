// The next token of each row of logits (plm_sample): temperature, top-k, top-p
// and min-p from one given random number a row.
//
// Mathematics.  w = 2^-t, t = (max - x) log2(e) / T, in fixed point: 2^40 for
// the largest logit, nothing from t = 40 on.  t is formed as f / 64 + r with a
// whole f: f from the f32 product p of x and c = log2(e) / T, r from what is left,
// which f32 subtraction gives exactly, and p's own rounding error.  2^-t is a
// table's 2^(-i/64), a shift, and the series of 2^-r (a table-driven exponential as
// in P. T. P. Tang, ACM TOMS 15, 1989), to 2^-28 of itself.  Sums of whole numbers
// do not depend on their order, so which token is met does not depend on the launch.
//   A border (the k-th largest logit; the one at which the sum of the w's in
// descending order reaches p of all) is found without sorting the row: f is the
// bin of a histogram, which says in which bins the border lies.  If few logits lie
// from there upwards they are sorted and everything is decided among them (the
// rule for top-k).  Else the logits of the border's bin are, and the sum of those
// above it is formed exactly (a top-p of flat rows).  Where neither applies the
// bins are cut again by the logits' bits until a bin is a single value.
//
// Layout.  A cluster of CTAs takes a row, each a piece of it in shared memory as
// integers that order as the logits do; so the row is read once.  What does not
// fit is read again from L2.  A warp has consecutive logits, so the sums of the
// warps say in which of them the token is.
#include "plm_device.cuh"
#include "plm_internal.h"
#include "values.cuh"

namespace plm {

namespace {

using u64 = unsigned long long;

constexpr int MOST_THREADS = 1024, MOST_WARPS = MOST_THREADS / 32;
constexpr int BINS = 2560;                   // f of a logit with a weight: t below 40
constexpr int LIST = 1024;                   // logits that are sorted at most
constexpr int MOST_CS = 8;                   // CTAs of a row at most
constexpr uint32_t LOWEST = 0x007FFFFFu;     // the key of -inf; 0: no logit
constexpr float MAGIC = 12582912.0f;         // 1.5 2^23: adding it rounds to a whole number

struct SampleArgs {
    plm_sample_problem p;
    int seg, held;                           // logits of a warp (a multiple of 128), of which in shared memory
    bool four;                               // rows in accesses of four
};

// 2^(40 - i/64)
__device__ const u64 EXP_TABLE[64] = {
    0x10000000000ULL, 0x0FD3E0C0CF5ULL, 0x0FA83B2DB72ULL, 0x0F7D0DF730BULL, 0x0F5257D1525ULL, 0x0F281773C5AULL,
    0x0EFE4B99BDDULL, 0x0ED4F301EDAULL, 0x0EAC0C6E7DDULL, 0x0E8396A503CULL, 0x0E5B906E77DULL, 0x0E33F8972BFULL,
    0x0E0CCDEEC2BULL, 0x0DE60F4825EULL, 0x0DBFBB797DBULL, 0x0D99D15C279ULL, 0x0D744FCCAD7ULL, 0x0D4F35AABD0ULL,
    0x0D2A81D91F1ULL, 0x0D06333DAEFULL, 0x0CE248C1520ULL, 0x0CBEC14FEF2ULL, 0x0C9B9BD866EULL, 0x0C78D74C8ACULL,
    0x0C5672A1155ULL, 0x0C346CCDA25ULL, 0x0C12C4CCA66ULL, 0x0BF1799B67AULL, 0x0BD08A39F58ULL, 0x0BAFF5AB213ULL,
    0x0B8FBAF4763ULL, 0x0B6FD91E329ULL, 0x0B504F333FAULL, 0x0B311C412A9ULL, 0x0B123F581D3ULL, 0x0AF3B78AD69ULL,
    0x0AD583EEA43ULL, 0x0AB7A39B5A9ULL, 0x0A9A15AB4EAULL, 0x0A7CD93B4E9ULL, 0x0A5FED6A9B1ULL, 0x0A43515AE0AULL,
    0x0A27043030CULL, 0x0A0B0510FB9ULL, 0x09EF5326092ULL, 0x09D3ED9A72DULL, 0x09B8D39B9D5ULL, 0x099E0459321ULL,
    0x09837F0518EULL, 0x096942D3720ULL, 0x094F4EFA8FFULL, 0x0935A2B2F14ULL, 0x091C3D373ABULL, 0x09031DC4314ULL,
    0x08EA4398B46ULL, 0x08D1ADF5B7EULL, 0x08B95C1E3EBULL, 0x08A14D57549ULL, 0x088980E8093ULL, 0x0871F61969FULL,
    0x085AAC367CCULL, 0x0843A28C3ADULL, 0x082CD8698ACULL, 0x08164D1F3BCULL,
};

// Logits as integers in their order; NaN is -inf, -0 is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return x != x ? LOWEST : b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {   // of 0: NaN
    return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

struct alignas(16) SampleSmem {
    u64 table[64];
    u64 part[2][MOST_WARPS], slot[2][MOST_CS];   // of an exchange, in turn
    u64 own[MOST_WARPS];                         // the warps' sums of kept w's
    u64 scan[2][MOST_WARPS];
    u64 sums[MOST_CS * MOST_WARPS];              // the same of all warps of the row
    u64 found_sum;
    uint32_t found[8];
    int listed;                                  // logits in `list`
    alignas(16) uint32_t hist[BINS];
    u64 list[LIST], sorted[LIST];                // key, and the index's complement below
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ u64 warp_max64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = w > v ? w : v;
    }
    return v;
}
__device__ __forceinline__ u64 warp_scan64(u64 v, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 w = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

__device__ __forceinline__ uint32_t at_peer(const void* p, int z) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(z));
    return a;
}
__device__ __forceinline__ u64 peer64(const u64* p, int z) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at_peer(p, z)) : "memory");
    return v;
}
__device__ __forceinline__ void to_peer64(u64* p, int z, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(at_peer(p, z)), "l"(v) : "memory");
}
__device__ __forceinline__ uint4 peer128(const uint32_t* p, int z) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at_peer(p, z)) : "memory");
    return v;
}
__device__ __forceinline__ int peer_int(const int* p, int z) {
    int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at_peer(p, z)) : "memory");
    return v;
}

// v part of 1: floor and ceiling of v a for 0 <= a < 1 (f32), v below 2^63.
__device__ __forceinline__ u64 share_of(u64 v, float a, bool up) {
    const uint32_t b = __float_as_uint(a);
    const int e = (int)(b >> 23);                       // a = m 2^(e - 150)
    const u64 m = e ? (b & 0x7FFFFFu) | 0x800000u : b;
    const int s = 150 - (e ? e : 1);                    // 24 at least
    const u64 lo = v * m, hi = __umul64hi(v, m);        // v m < 2^87
    u64 q, rest;
    if (s >= 87) {
        q = 0;
        rest = lo | hi;
    } else if (s >= 64) {
        q = hi >> (s - 64);
        rest = lo | (s > 64 ? hi << (128 - s) : 0);
    } else {
        q = hi << (64 - s) | lo >> s;
        rest = lo << (64 - s);
    }
    return q + (up && rest);
}

// A row as one CTA of its cluster sees it.
struct Sampler {
    const SampleArgs& A;
    SampleSmem& sm;
    uint32_t* keys;             // of this warp's logits, the first `held`
    long long row;
    int lane, warp, nw, nt, cs, rank, first, turn;   // first: index of the warp's first logit
    uint32_t kmax;
    float base, c_hi, c_lo, ref, ref64;              // t = ref - (x - base) (c_hi + c_lo)
    bool infinite;                                   // the largest logits are +inf: they are 0, the others no logits

    // Four logits from index i on, as keys
    __device__ __forceinline__ uint4 load(int i) const {
        const long long n = A.p.n - i;
        const float4 v = load_four(A.p.logits, A.p.type, row * A.p.stride + i, n < 4 ? (int)n : 4, A.four && n >= 4);
        return make_uint4(n > 0 ? key_of(v.x) : 0, n > 1 ? key_of(v.y) : 0, n > 2 ? key_of(v.z) : 0, n > 3 ? key_of(v.w) : 0);
    }
    __device__ __forceinline__ uint32_t finite(uint32_t k) const { return k == key_of(INFINITY) ? key_of(0.0f) : 0; }
    // The lane's four of the warp's 128 from place i on
    __device__ __forceinline__ uint4 four(int i) const {
        if (i < A.held) return *reinterpret_cast<const uint4*>(keys + i + 4 * lane);
        uint4 k = load(first + i + 4 * lane);
        if (infinite) k = make_uint4(finite(k.x), finite(k.y), finite(k.z), finite(k.w));
        return k;
    }
    template <class F> __device__ __forceinline__ void each(F f) const {
        const int end = (int)min((long long)A.seg, (long long)A.p.n - first);
#pragma unroll 2
        for (int i = 0; i < end; i += 128) {
            const uint4 k = four(i);
            f(k.x, i + 4 * lane);
            f(k.y, i + 4 * lane + 1);
            f(k.z, i + 4 * lane + 2);
            f(k.w, i + 4 * lane + 3);
        }
    }
    __device__ __forceinline__ void together() const {
        __syncwarp();
        if (cs > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else __syncthreads();
    }

    // 64 t rounded, MAGIC added: its bits count in steps of 1.  No less for a smaller logit.
    __device__ __forceinline__ float steps(float p) const { return fmaf(p, -64.0f, ref64); }
    __device__ __forceinline__ float product(uint32_t k) const { return (logit_of(k) - base) * c_hi; }
    __device__ __forceinline__ bool weighs(float s) const { return s < MAGIC + (float)BINS; }   // (false for NaN)
    __device__ __forceinline__ int bin(uint32_t k) const {   // BINS where there is no weight
        const float s = steps(product(k));
        return weighs(s) ? (int)(__float_as_uint(s) - __float_as_uint(MAGIC)) : BINS;
    }
    // 2^(40 - f/64 - r)
    __device__ __forceinline__ u64 power(uint32_t f, float r) const {
        const float e = r * fmaf(r, fmaf(r, -0.0555041087f, 0.240226507f), -0.693147181f);   // 2^-r - 1
        const u64 v = sm.table[f & 63];
        // v e in steps of 2^11: below 2^22 of them
        const float s = fmaf((float)(uint32_t)(v >> 17) * 64.0f, e, MAGIC);
        return (v + (u64)((long long)(int)(__float_as_uint(s) - __float_as_uint(MAGIC)) * 2048)) >> (f >> 6);
    }
    __device__ __forceinline__ u64 weight(uint32_t k) const {   // 0 where there is none
        const float x = logit_of(k) - base, p = x * c_hi, s = steps(p);
        if (!weighs(s)) return 0;
        const float y = fmaf(s - MAGIC, -0.015625f, ref);       // ref - f/64, exact
        const float r = fmaf(x, -c_lo, (y - p) - fmaf(x, c_hi, -p));
        return power(__float_as_uint(s) - __float_as_uint(MAGIC), r);
    }

    // Sum or maximum of the threads' v over the row.
    template <bool MAX> __device__ u64 exchange(u64 v) {
        const int b = turn & 1;
        ++turn;
        v = MAX ? warp_max64(v) : warp_sum64(v);
        if (lane == 0) sm.part[b][warp] = v;
        __syncthreads();
        if (cs == 1 || warp == 0) {
            v = lane < nw ? sm.part[b][lane] : 0;
            v = MAX ? warp_max64(v) : warp_sum64(v);
        }
        if (cs == 1) return v;
        if (warp == 0 && lane < cs) to_peer64(&sm.slot[b][rank], lane, v);
        together();
        v = lane < cs ? sm.slot[b][lane] : 0;
        return MAX ? warp_max64(v) : warp_sum64(v);
    }

    // The largest (up) or smallest key in [lo, hi] whose bin is >= b (<= b), of
    // which there is one: the bins fall as the keys rise.  A lane tries a key each.
    __device__ uint32_t edge(int b, uint32_t lo, uint32_t hi, bool up) const {
        while (lo < hi) {
            const uint32_t step = (hi - lo) / 32 + 1, off = step * lane;   // (below 2^32)
            const bool in = off <= hi - lo;
            const uint32_t k = up ? hi - off : lo + off;
            const unsigned yes = __ballot_sync(0xFFFFFFFFu, in && (up ? bin(k) >= b : bin(k) <= b));
            const int first_yes = __ffs(yes) - 1;
            // the one looked for lies at that key, or between it and the one tried before
            if (first_yes < 0) {   // beyond the last key tried
                const uint32_t far = (hi - lo) / step * step;
                if (up) hi -= far;
                else lo += far;
                if (step == 1) break;
            } else {
                const uint32_t at = step * first_yes, before = first_yes ? at - step + 1 : 0;
                const uint32_t a = up ? hi - at : lo + before, z = up ? hi - before : lo + at;
                lo = a;
                hi = z;
                if (first_yes == 0) return up ? hi : lo;
            }
        }
        return lo;
    }

    // Empties the histogram, once every CTA has read it.
    __device__ __forceinline__ void empty() const {
        together();
        for (int i = threadIdx.x; i < BINS / 4; i += nt) reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    // Four bins of the row's histogram (after a barrier)
    __device__ __forceinline__ uint4 counts(int b) const {
        if (cs == 1) return *reinterpret_cast<const uint4*>(sm.hist + b);
        uint4 c = make_uint4(0, 0, 0, 0);
#pragma unroll 4
        for (int z = 0; z < cs; ++z) {
            const uint4 v = peer128(sm.hist + b, z);
            c.x += v.x;
            c.y += v.y;
            c.z += v.z;
            c.w += v.w;
        }
        return c;
    }
    __device__ __forceinline__ uint32_t count_of(int b) const {
        const uint4 c = counts(b & ~3);
        return (b & 3) == 0 ? c.x : (b & 3) == 1 ? c.y : (b & 3) == 2 ? c.z : c.w;
    }
    // Exclusive sums of the threads' pair over the CTA.
    __device__ __forceinline__ void block_scan(u64& a, u64& b) {
        const u64 ai = warp_scan64(a, lane), bi = warp_scan64(b, lane);
        __syncthreads();   // (what was there has been read)
        if (lane == 31) {
            sm.scan[0][warp] = ai;
            sm.scan[1][warp] = bi;
        }
        __syncthreads();
        u64 x = lane < warp ? sm.scan[0][lane] : 0, y = lane < warp ? sm.scan[1][lane] : 0;
        a = ai - a + warp_sum64(x);
        b = bi - b + warp_sum64(y);
    }

    struct Border { uint32_t key; uint32_t ties, of; };   // ties kept of `of`

    // The border of the row at which the count (mass = false) or the w's sum of
    // the logits in descending order reaches `target` >= 1 (which they do).  Below
    // `floor_` nothing counts, and of the logits equal to it `missing` do not.
    __device__ Border select(bool mass, u64 target, uint32_t floor_, uint32_t missing) {
        uint32_t hi = kmax, lo = floor_;
        bool by_t = true;
        for (;;) {
            int shift = 0;
            while (((hi - lo) >> shift) >= (uint32_t)BINS) ++shift;
            auto place = [&](uint32_t k) { return by_t ? min(bin(k), BINS - 1) : (int)((hi - k) >> shift); };
            empty();
            u64 mine = 0;
            each([&](uint32_t k, int) {
                if (k > hi) mine += mass ? weight(k) : 1;
                else if (k >= lo) atomicAdd(&sm.hist[place(k)], 1u);
            });
            const u64 above = exchange<false>(mine);
            // a thread's bins, four at a time: how many, and the bounds of their sums
            u64 up_run = above, down_run = above;
            if (threadIdx.x == 0) { sm.found[0] = BINS; sm.found[1] = BINS; sm.found[4] = 0; }
            for (int at = 0; at < BINS; at += 4 * nt) {
                const int b0 = at + 4 * (int)threadIdx.x;
                uint32_t n[4] = {0, 0, 0, 0};
                u64 most[4], least[4], up = 0, down = 0;
                if (b0 < BINS) {
                    const uint4 c = counts(b0);
                    n[0] = c.x; n[1] = c.y; n[2] = c.z; n[3] = c.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int b = b0 + j;
                    if (n[j] && missing && lo == floor_ && b == place(lo)) n[j] -= missing;
                    most[j] = least[j] = n[j];
                    if (mass && n[j]) {
                        u64 w1, w0;
                        if (by_t) {   // r is within half a step, give or take rounding
                            w1 = power(b, -0.0079f) + 1;
                            w0 = power(b, 0.0079f);
                        } else {
                            const uint32_t k1 = hi - ((uint32_t)b << shift), left = k1 - lo, k0 = left >> shift ? k1 - (1u << shift) + 1 : lo;
                            w1 = weight(k1);
                            w0 = k0 == k1 ? w1 : weight(k0);
                            if (k0 != k1) {   // w is right to 2^-28, and may fall by that where it should rise
                                w1 += (w1 >> 26) + 1;
                                w0 -= w0 >> 26;
                            }
                        }
                        most[j] = n[j] * w1;
                        least[j] = n[j] * w0;
                    }
                    up += most[j];
                    down += least[j];
                }
                u64 up_at = up, down_at = down;
                block_scan(up_at, down_at);
                if (threadIdx.x == nt - 1) { sm.sums[0] = up_at + up; sm.sums[1] = down_at + down; }
                up_at += up_run;
                down_at += down_run;
                // the first bin whose upper bound reaches the target, the first whose lower bound does
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (n[j]) {
                        if (up_at < target && up_at + most[j] >= target) {
                            sm.found[0] = b0 + j;
                            sm.found[2] = n[j];
                            sm.found_sum = up_at;
                        }
                        if (down_at < target && down_at + least[j] >= target) sm.found[1] = b0 + j;
                        atomicMax(&sm.found[4], (uint32_t)(b0 + j));
                    }
                    up_at += most[j];
                    down_at += least[j];
                }
                __syncthreads();
                up_run += sm.sums[0];
                down_run += sm.sums[1];
            }
            const int last = (int)sm.found[4], b1 = min((int)sm.found[0], last), b2 = min((int)sm.found[1], last);
            const uint32_t count = sm.found[2];
            const u64 before = sm.found_sum;
            __syncthreads();
            if (!by_t && shift == 0) {
                Border B;
                B.key = hi - b1;
                B.of = count;
                const u64 w = mass ? weight(B.key) : 1;
                const u64 need = target > before && w ? (target - before + w - 1) / w : 1;
                B.ties = (uint32_t)(need < 1 ? 1 : need > count ? count : need);
                return B;
            }
            const uint32_t wide = hi - lo;
            if (by_t) {
                const uint32_t top = edge(b1, lo, hi, true);
                if (b2 < BINS - 1) lo = edge(b2, lo, hi, false);
                hi = top;
                by_t = false;
                continue;
            }
            const uint32_t top = hi - ((uint32_t)b1 << shift), k2 = hi - ((uint32_t)b2 << shift);
            lo = (k2 - lo) >> shift ? k2 - (1u << shift) + 1 : lo;
            hi = top;
            if (hi - lo > wide / 4) {   // bounds that tell the bins apart badly: halve what is left
                const uint32_t mid = lo + (hi - lo) / 2;
                u64 v = 0;
                each([&](uint32_t k, int) {
                    if (k > mid) v += mass ? weight(k) : 1;
                });
                if (exchange<false>(v) >= target) lo = mid + 1;
                else hi = mid;
            }
        }
    }

    // The w's sum of the logits from `from` on.
    __device__ u64 total(uint32_t from) {
        u64 v = 0;
        each([&](uint32_t k, int) {
            if (k >= from) v += weight(k);
        });
        return exchange<false>(v);
    }

    // The index of the logit equal to `key` that `before` equal ones precede.
    __device__ int tie_at(uint32_t key, u64 before) {
        u64 mine = 0;
        each([&](uint32_t k, int) { mine += k == key; });
        mine = warp_sum64(mine);
        tell(mine);
        u64 pre = 0;
        for (int i = lane; i < rank * nw + warp; i += 32) pre += sm.sums[i];
        pre = warp_sum64(pre);
        int at = 0x7FFFFFFF;
        if (before >= pre && before < pre + mine)
            at = find([&](uint32_t k, int) -> u64 { return k == key; }, before - pre);
        return (int)(0xFFFFFFFFu - (uint32_t)exchange<true>(at == 0x7FFFFFFF ? 0 : 0xFFFFFFFFu - (uint32_t)at));
    }

    // The warps' sums of the whole row into sm.sums.
    __device__ void tell(u64 mine) {
        if (lane == 0) sm.own[warp] = mine;
        together();
        gather();
        together();   // (sm.own may be written again)
    }
    __device__ void gather() {
        for (int i = threadIdx.x; i < cs * nw; i += nt) {
            const int z = i / nw;
            sm.sums[i] = cs > 1 ? peer64(&sm.own[i - z * nw], z) : sm.own[i];
        }
        __syncthreads();
    }

    // The index at which the sum of f over this warp's logits exceeds `target`.
    template <class F> __device__ int find(F f, u64 target) const {
        const int end = (int)min((long long)A.seg, (long long)A.p.n - first);
        u64 pre = 0;
        for (int i = 0; i < end; i += 128) {
            const uint4 k = four(i);
            const u64 a = f(k.x, i + 4 * lane), b = f(k.y, i + 4 * lane + 1), c = f(k.z, i + 4 * lane + 2), d = f(k.w, i + 4 * lane + 3);
            const u64 in = warp_scan64(a + b + c + d, lane);
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, pre + in > target);
            if (hit) {
                const int l = __ffs(hit) - 1;
                const u64 before = pre + in - (a + b + c + d);
                const int j = before + a > target ? 0 : before + a + b > target ? 1 : before + a + b + c > target ? 2 : 3;
                return first + i + __shfl_sync(0xFFFFFFFFu, 4 * lane + j, l);
            }
            pre += __shfl_sync(0xFFFFFFFFu, in, 31);
        }
        return 0x7FFFFFFF;
    }

    __device__ void put(int token, float prob) const {
        A.p.tokens[row] = token;
        if (A.p.prob) A.p.prob[row] = prob;
    }
    __device__ u64 target_of(u64 all) const {   // the place in the kept w's that u points at
        const float u = fmaxf(A.p.u[row], 0.0f);
        return u < 1.0f ? share_of(all, u, false) : all - 1;
    }

    // The token, of the logits above `key` and those equal to it up to index
    // `last`; the warps' sums of their w's are in sm.sums.
    __device__ void finish(uint32_t key, int last) {
        u64 all = 0;
        for (int i = lane; i < cs * nw; i += 32) all += sm.sums[i];
        all = warp_sum64(all);
        const u64 target = target_of(all);
        u64 pre = 0;
        for (int i = lane; i < rank * nw + warp; i += 32) pre += sm.sums[i];
        pre = warp_sum64(pre);
        if (target < pre || target >= pre + sm.sums[rank * nw + warp]) return;
        const int at = find([&](uint32_t k, int i) -> u64 { return k > key || (k == key && first + i <= last) ? weight(k) : 0; }, target - pre);
        if (lane == 0) {
            uint32_t k = key_of(value_at(A.p.logits, A.p.type, row * A.p.stride + at));
            if (infinite) k = finite(k);
            put(at, (float)((double)weight(k) / (double)all));
        }
    }

    // Sorts sm.sorted[0 .. n), n a power of two of 32 .. LIST, downwards.
    __device__ void sort(int n) {
        // a thread has the values at threadIdx.x and, where nt < n, threadIdx.x + nt
        const int i0 = threadIdx.x, i1 = i0 + nt;
        u64 a = i0 < n ? sm.sorted[i0] : 0, b = i1 < n ? sm.sorted[i1] : 0;
        auto keep = [](u64 mine, u64 other, bool larger) { return (mine > other) == larger ? mine : other; };
        for (int k = 2; k <= n; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                const bool a_max = ((i0 & k) == 0) == ((i0 & j) == 0), b_max = ((i1 & k) == 0) == ((i1 & j) == 0);
                if (j < 32) {
                    const u64 x = __shfl_xor_sync(0xFFFFFFFFu, a, j), y = __shfl_xor_sync(0xFFFFFFFFu, b, j);
                    a = keep(a, x, a_max);
                    b = keep(b, y, b_max);
                } else {
                    __syncthreads();
                    if (i0 < n) sm.sorted[i0] = a;
                    if (i1 < n) sm.sorted[i1] = b;
                    __syncthreads();
                    if (i0 < n) a = keep(a, sm.sorted[i0 ^ j], a_max);
                    if (i1 < n) b = keep(b, sm.sorted[i1 ^ j], b_max);
                }
            }
        __syncthreads();
        if (i0 < n) sm.sorted[i0] = a;
        if (i1 < n) sm.sorted[i1] = b;
        __syncthreads();
    }
    static __device__ __forceinline__ int rounded_up(int n) { return n <= 32 ? 32 : 1 << (32 - __clz(n - 1)); }

    // Puts the logits of [lo, hi] on this CTA's list, and the w's of those above
    // into the warps' sums; the logits on all lists (more than LIST: they are not whole).
    __device__ int collect(uint32_t lo, uint32_t hi) {
        u64 above = 0;
        const int end = (int)min((long long)A.seg, (long long)A.p.n - first);
        for (int i = 0; i < end; i += 128) {
            const uint4 v = four(i);
            const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (k[j] > hi) above += weight(k[j]);
                const bool in = k[j] >= lo && k[j] <= hi;
                const unsigned who = __ballot_sync(0xFFFFFFFFu, in);
                if (!who) continue;
                int at = 0;
                if (lane == 0) at = atomicAdd(&sm.listed, __popc(who));
                at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(who & ((1u << lane) - 1));
                if (in && at < LIST) sm.list[at] = (u64)k[j] << 32 | (0xFFFFFFFFu - (uint32_t)(first + i + 4 * lane + j));
            }
        }
        above = warp_sum64(above);
        if (lane == 0) sm.own[warp] = above;
        together();
        int n = lane < cs ? (cs > 1 ? peer_int(&sm.listed, lane) : sm.listed) : 0;
        return __reduce_add_sync(0xFFFFFFFFu, min(n, LIST + 1));
    }
    // All lists into sm.sorted, sorted; the place after the last.
    __device__ int bring(int n) {
        const int size = rounded_up(n);
        int at = 0;
        for (int z = 0; z < cs; ++z) {
            const int m = cs > 1 ? peer_int(&sm.listed, z) : sm.listed;
            for (int i = threadIdx.x; i < m; i += nt) sm.sorted[at + i] = cs > 1 ? peer64(&sm.list[i], z) : sm.list[i];
            at += m;
        }
        for (int i = n + threadIdx.x; i < size; i += nt) sm.sorted[i] = 0;
        __syncthreads();
        sort(size);
        return size;
    }
};

// CTA (row, , rank in the row's cluster).
__global__ void __launch_bounds__(MOST_THREADS) sample_kernel(const __grid_constant__ SampleArgs A) {
    extern __shared__ __align__(16) uint8_t sample_raw[];
    SampleSmem& sm = *reinterpret_cast<SampleSmem*>(sample_raw);
    grid_launch_dependents();
    Sampler S{A, sm};
    S.row = blockIdx.x;
    S.lane = threadIdx.x & 31;
    S.warp = threadIdx.x >> 5;
    S.nt = blockDim.x;
    S.nw = S.nt >> 5;
    S.cs = gridDim.z;
    S.rank = blockIdx.z;
    S.first = (int)min((long long)(S.rank * S.nw + S.warp) * A.seg, (long long)A.p.n);
    S.turn = 0;
    S.infinite = false;
    S.keys = reinterpret_cast<uint32_t*>(sample_raw + sizeof(SampleSmem)) + S.warp * A.held;
    if (threadIdx.x < 64) sm.table[threadIdx.x] = EXP_TABLE[threadIdx.x];
    if (threadIdx.x == 0) sm.listed = 0;
    for (int i = threadIdx.x; i < BINS / 4; i += S.nt) reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0, 0, 0, 0);
    grid_wait_prior();
    // the row, and its largest logit
    uint32_t best = 0;
    {
        const int end = (int)min((long long)A.seg, (long long)A.p.n - S.first);
#pragma unroll 4
        for (int i = 0; i < end; i += 128) {
            const uint4 k = S.load(S.first + i + 4 * S.lane);
            if (i < A.held) *reinterpret_cast<uint4*>(S.keys + i + 4 * S.lane) = k;
            best = max(best, max(max(k.x, k.y), max(k.z, k.w)));
        }
    }
    S.kmax = (uint32_t)S.exchange<true>(best);
    const bool leader = S.rank == 0 && threadIdx.x == 0;
    const float T = A.p.temperature ? A.p.temperature[S.row] : 1.0f;
    if (S.kmax <= LOWEST) {
        if (leader) S.put(-1, 0.0f);
    } else if (!(T > 0.0f) || !A.p.u) {
        uint32_t at = 0;   // the first index, as its complement
        S.each([&](uint32_t k, int i) {
            if (k == S.kmax) at = max(at, 0xFFFFFFFFu - (uint32_t)(S.first + i));
        });
        at = (uint32_t)S.exchange<true>(at);
        if (leader) S.put((int)(0xFFFFFFFFu - at), 1.0f);
    } else {
        if (S.kmax == key_of(INFINITY)) {
            S.infinite = true;
            const int end = min(A.held, (int)min((long long)A.seg, (long long)A.p.n - S.first));
            for (int i = 4 * S.lane; i < end; i += 128)
                for (int j = i; j < i + 4; ++j) S.keys[j] = S.finite(S.keys[j]);
            S.kmax = key_of(0.0f);
            __syncwarp();
        }
        const float top = logit_of(S.kmax);
        {   // c = log2(e) / T as a pair of f32: the quotient and what it leaves
            const float l_hi = 1.44269502f, l_lo = 1.92596299e-8f;   // log2(e)
            const float q = fminf(__fdiv_rn(l_hi, T), 3e38f);
            S.c_hi = q;
            S.c_lo = q < 1e37f && T < 1e37f && T > 1e-30f ? __fdiv_rn(fmaf(-q, T, l_hi) + l_lo, T) : 0.0f;
        }
        // Logits near the top differ from it exactly; else the reference is 0
        S.base = fabsf(top * S.c_hi) < 80.0f ? 0.0f : top;
        S.ref = ceilf((top - S.base) * S.c_hi * 64.0f) * 0.015625f;
        S.ref64 = S.ref * 64.0f + MAGIC;
        const int k = A.p.top_k ? A.p.top_k[S.row] : 0;
        const float p = A.p.top_p ? A.p.top_p[S.row] : 1.0f, low = A.p.min_p ? A.p.min_p[S.row] : 0.0f;
        const bool by_k = k > 0 && k < A.p.n, by_p = p < 1.0f;
        // the lowest key with a weight; min_p: of the smallest f32 that is at least max + T ln(min_p)
        uint32_t floor_ = S.edge(BINS - 1, LOWEST + 1, S.kmax, false);
        if (low > 0.0f) {
            if (threadIdx.x == 0)
                sm.found[7] = S.infinite ? S.kmax : min(key_of(__double2float_ru((double)top + (double)T * log((double)fminf(low, 1.0f)))), S.kmax);
            __syncthreads();
            floor_ = max(floor_, sm.found[7]);
            __syncthreads();
        }
        uint32_t border = floor_;   // what is kept: the keys above, and those equal up to index `last`
        int last = 0x7FFFFFFF;
        enum { AGAIN, LISTED, WIDE, DONE } how = DONE;
        u64 sum = 0;
        if (by_k || by_p) {
            // The histogram; for top_p alone also the sum of all w's
            u64 mine = 0;
            S.each([&](uint32_t x, int) {
                const int b = S.bin(x);
                if (b < BINS) atomicAdd(&sm.hist[b], 1u);
                if (!by_k) mine += S.weight(x);
            });
            sum = S.exchange<false>(mine);
            u64 target = by_k ? k : share_of(sum, fmaxf(p, 0.0f), true);
            if (target < 1) target = 1;
            if (target > sum && !by_k) target = sum;
            // the bin in which the count, or by the bins' middles the sum, reaches it
            if (threadIdx.x == 0) { sm.found[0] = BINS; sm.found[1] = 0; sm.found[2] = 0; sm.found[3] = 0; }
            u64 run = 0, run_n = 0;
            for (int at = 0; at < BINS; at += 4 * S.nt) {
                const int b0 = at + 4 * (int)threadIdx.x;
                const uint4 c = b0 < BINS ? S.counts(b0) : make_uint4(0, 0, 0, 0);
                const uint32_t n[4] = {c.x, c.y, c.z, c.w};
                u64 v[4], in = 0, in_n = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = by_k ? n[j] : n[j] ? n[j] * S.power(b0 + j, 0.0f) : 0;
                    in += v[j];
                    in_n += n[j];
                }
                u64 pre = in, pre_n = in_n;
                S.block_scan(pre, pre_n);
                if (threadIdx.x == S.nt - 1) { sm.sums[0] = pre + in; sm.sums[1] = pre_n + in_n; }
                pre += run;
                pre_n += run_n;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    pre_n += n[j];
                    if (n[j] && pre < target && pre + v[j] >= target) {
                        sm.found[0] = b0 + j;
                        sm.found[1] = (uint32_t)pre_n;   // logits down to this bin
                        sm.found[2] = n[j];
                    }
                    pre += v[j];
                }
                __syncthreads();
                run += sm.sums[0];
                run_n += sm.sums[1];
            }
            const int b = (int)sm.found[0];
            const uint32_t down_to = sm.found[1], there = sm.found[2];
            if (by_k && run_n <= (u64)k) {
                how = by_p ? AGAIN : DONE;                 // top_k leaves all that have a weight
            } else if (b >= BINS) {
                how = AGAIN;                               // (rounding has put it past the last bin)
            } else {
                // for top_p the border may be a bin further down, or up, than the middles say
                uint32_t lo = S.edge(b, LOWEST + 1, S.kmax, false), hi = S.kmax;
                how = LISTED;
                if (!by_k) {
                    const uint32_t below = b + 1 < BINS ? S.count_of(b + 1) : 0, above = b ? S.count_of(b - 1) : 0;
                    if (down_to + below <= (uint32_t)LIST) {
                        lo = S.edge(min(b + 1, BINS - 1), LOWEST + 1, S.kmax, false);
                    } else {
                        how = WIDE;
                        const bool three = below + there + above <= (uint32_t)LIST;
                        if (three) lo = S.edge(min(b + 1, BINS - 1), LOWEST + 1, S.kmax, false);
                        hi = S.edge(three ? max(b - 1, 0) : b, LOWEST + 1, S.kmax, true);
                    }
                }
                // what min_p leaves out need not be looked at, but counts in what top_p is of
                if (!(by_k && by_p) && floor_ > lo) lo = floor_;
                if (lo > hi) {                             // min_p seems to leave less than top_p
                    how = S.total(floor_) <= target ? DONE : AGAIN;
                } else if (by_k && down_to > (uint32_t)LIST) {
                    how = AGAIN;
                } else {
                    const int n = S.collect(lo, hi);
                    if (n > LIST || n == 0) {
                        how = AGAIN;
                    } else {
                        S.bring(n);
                        u64 above = 0;
                        if (how == WIDE) {
                            S.gather();
                            for (int i = S.lane; i < S.cs * S.nw; i += 32) above += sm.sums[i];
                            above = warp_sum64(above);
                        }
                        // a thread's values of the list, in descending order
                        u64 w[2], key[2];
                        for (int round = 0; round < 2; ++round) {
                            const int i = 2 * threadIdx.x + round;
                            key[round] = i < n ? sm.sorted[i] : 0;
                            w[round] = i < n && (!by_k || i < k) ? S.weight((uint32_t)(key[round] >> 32)) : 0;
                        }
                        u64 pre = w[0] + w[1], none = 0;
                        const u64 pair = pre;
                        S.block_scan(pre, none);
                        if (threadIdx.x == S.nt - 1) sm.found_sum = pre + pair;
                        __syncthreads();
                        const u64 listed = sm.found_sum;
                        if (by_k) {
                            sum = listed;
                            target = by_p ? share_of(sum, fmaxf(p, 0.0f), true) : sum;
                            if (target < 1) target = 1;
                        }
                        // (by the middles of the bins the border may seem to lie where it does not; a list that min_p
                        // has cut short need not reach it)
                        if (!by_k && (above >= target || (above + listed < target && lo > floor_))) {
                            how = AGAIN;
                        } else {
                            const bool keep0 = w[0] && above + pre < target && (uint32_t)(key[0] >> 32) >= floor_;
                            const bool keep1 = w[1] && above + pre + w[0] < target && (uint32_t)(key[1] >> 32) >= floor_;
                            const int kept = __syncthreads_count(keep0) + __syncthreads_count(keep1);   // the first so many
                            if (how == WIDE) {
                                // each of them adds to its warp's sum
                                for (int round = 0; round < 2; ++round)
                                    if (round ? keep1 : keep0)
                                        atomicAdd(&sm.sums[(0xFFFFFFFFu - (uint32_t)key[round]) / A.seg], w[round]);
                                __syncthreads();
                                if (kept) {
                                    const u64 end = sm.sorted[kept - 1];
                                    border = (uint32_t)(end >> 32);
                                    last = (int)(0xFFFFFFFFu - (uint32_t)end);
                                } else {
                                    border = hi + 1;   // (none: those above alone)
                                }
                                S.finish(border, last);
                            } else if (S.rank == 0) {
                                // in the order of the indices: the index's complement first, downwards
                                const int size = Sampler::rounded_up(kept);
                                __syncthreads();
                                for (int round = 0; round < 2; ++round) {
                                    const int i = 2 * threadIdx.x + round;
                                    if (i < size) sm.sorted[i] = i < kept ? key[round] << 32 | key[round] >> 32 : 0;
                                }
                                __syncthreads();
                                S.sort(size);
                                for (int round = 0; round < 2; ++round) {
                                    const int i = 2 * threadIdx.x + round;
                                    key[round] = i < kept ? sm.sorted[i] : 0;
                                    w[round] = i < kept ? S.weight((uint32_t)key[round]) : 0;
                                }
                                u64 up = w[0] + w[1];
                                const u64 both = up;
                                S.block_scan(up, none);
                                if (threadIdx.x == S.nt - 1) sm.found_sum = up + both;
                                __syncthreads();
                                const u64 all = sm.found_sum, at = S.target_of(all);
                                for (int round = 0; round < 2; ++round) {
                                    if (at >= up && at < up + w[round])
                                        S.put((int)(0xFFFFFFFFu - (uint32_t)(key[round] >> 32)), (float)((double)w[round] / (double)all));
                                    up += w[round];
                                }
                            }
                        }
                    }
                }
            }
            if (how == AGAIN) {
                const uint32_t live = S.edge(BINS - 1, LOWEST + 1, S.kmax, false);
                Sampler::Border B = {live, 0, 0};
                bool cut = false;
                if (by_k && run_n > (u64)k) {
                    B = S.select(false, k, live, 0);
                    cut = true;
                }
                if (by_p) {
                    u64 all = S.total(B.key);
                    if (cut) all -= (B.of - B.ties) * S.weight(B.key);
                    u64 reach = share_of(all, fmaxf(p, 0.0f), true);
                    if (reach < 1) reach = 1;
                    B = S.select(true, reach, B.key, cut ? B.of - B.ties : 0);
                    cut = true;
                }
                if (cut && B.key >= floor_) {
                    border = B.key;
                    last = S.tie_at(border, B.ties - 1);
                }
                how = DONE;
            }
        }
        if (how == DONE) {
            u64 v = 0;
            S.each([&](uint32_t x, int i) {
                if (x > border || (x == border && S.first + i <= last)) v += S.weight(x);
            });
            S.tell(warp_sum64(v));
            S.finish(border, last);
        }
    }
    if (S.cs > 1) S.together();   // no CTA leaves while its shared memory is read
}

}  // namespace

cudaError_t launch_sample(const plm_sample_problem& p, cudaStream_t stream) {
    SampleArgs A = {};
    A.p = p;
    A.four = four_aligned(p.logits, p.m > 1 ? p.stride : 0, p.type);
    constexpr int room = 227 * 1024 - (int)sizeof(SampleSmem);
    const int sms = num_sms();
    // CTAs of a row: two of 16 warps an SM, with all the row in shared memory; few rows
    // are spread further
    int cs = 1, nt = 512;
    const int half = 113 * 1024 - (int)sizeof(SampleSmem);
    while (cs < 8 && p.n * 4 > (long long)cs * half) cs *= 2;
    while (cs < 8 && p.n > 4096LL * cs && p.m * cs * 2 <= sms) cs *= 2;
    if (p.m * cs <= sms) nt = 1024;
    const int warps = cs * nt / 32;
    A.seg = (int)((p.n + 128LL * warps - 1) / (128LL * warps)) * 128;
    const int most = (nt == 512 && 4LL * A.seg * (nt / 32) <= half ? half : room) / 4 / (nt / 32) / 128 * 128;
    A.held = A.seg < most ? A.seg : most;
    const size_t bytes = sizeof(SampleSmem) + 4 * (size_t)A.held * (nt / 32);
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)p.m, 1, (unsigned)cs);
    if (cs == 1) return launch_kernel(sample_kernel, grid, dim3(nt), bytes, stream, A);
    return launch_kernel_cluster(sample_kernel, grid, dim3(nt), bytes, stream, (unsigned)cs, A);
}

}  // namespace plm

// The next token of each row of logits (plm_sample): temperature, top-k, top-p
// and min-p from one given random number a row.
//
// Mathematics.  w = 2^-t, t = (max - x) log2(e) / T, in fixed point: 2^40 for
// the largest logit, nothing from t = 40 on.  t is formed as f / 64 + r with a
// whole f: f from the f32 product p of x and c = log2(e) / T, r from what is left,
// which f32 subtraction gives exactly, and p's own rounding error.  2^-t is a
// table's 2^(-i/64), a shift, and the series of 2^-r (a table-driven exponential as
// in P. T. P. Tang, ACM TOMS 15, 1989), to 2^-29 of itself.  Sums of whole numbers
// do not depend on their order, so which token is met does not depend on the launch.
//   A border (the k-th largest logit; the one at which the sum of the w's in
// descending order reaches p of all) is found without sorting the row: f is the
// bin of a histogram, which says in which bins the border lies.  If few logits lie
// from there upwards they are put in order and everything is decided among them
// (the rule for top-k).  Else the logits of the border's bin are, and the sum of
// those above it is formed exactly (a top-p of flat rows).  Where neither applies
// the bins are cut again by the logits' bits until a bin is a single value.
//
// Layout.  A cluster of CTAs takes a row, each a piece of it in shared memory, so
// the row is read once.  What does not fit is read again from L2.  A warp has
// consecutive logits, so the sums of the warps, which every CTA gets, say in which of
// them the token is.
//   What bounds it.  A row takes 2 (greedy) to 10 barriers of its cluster and 40
// instructions a logit for each time its weights are formed (once without top-k and
// top-p, up to three times with a top-p of many tokens); the read of the row hides behind
// that.  One row is held by 8 SMs, 19000 logits each: a pass that forms weights is 3 us of
// issue there.  One GB300, f32 logits, spread 2.5, us: 256 rows of 151936 (23 for the read alone)
// greedy 47, no limits 114, min-p 75, top-k 146, with top-p and min-p 156, top-p 0.9 alone
// 250 (spread 4: 193); one row of them 4.3, 10, 9, 15, 17, 25; 64 rows of 32000 greedy 4.3,
// top-k 15, top-p 26.  At the 64 registers that two CTAs leave, 100 bytes are spilled.
#include "plm_device.cuh"
#include "plm_internal.h"
#include "sample_keys.cuh"
#include "values.cuh"

namespace plm {

namespace {

using u64 = unsigned long long;

constexpr int NT = 512, NW = NT / 32;         // threads and warps of a CTA
static_assert(BINS == 64 * 40);               // f of a logit with a weight: t below 40
constexpr int COARSE = 16, GROUPS = BINS / COARSE;   // bins that are first looked at together
constexpr int LIST = 1024;                   // logits that are put in order at most
constexpr int BUCKETS = 512;
constexpr int MOST_CS = 8;                   // CTAs of a row at most
constexpr float MAGIC = 12582912.0f;         // 1.5 2^23: adding it rounds to a whole number

struct SampleArgs {
    plm_sample_problem p;
    int seg, held;                           // logits of a warp (a multiple of 128), of which in shared memory
    bool four;                               // rows in accesses of four
};

// 2^(40 - i/64), less 2^-41 of it, so that all are below 2^40
__device__ const u64 EXP_TABLE[64] = {
    0xFFFFFFFFFFull, 0xFD3E0C0CF4ull, 0xFA83B2DB71ull, 0xF7D0DF730Aull, 0xF5257D1524ull, 0xF281773C59ull,
    0xEFE4B99BDCull, 0xED4F301ED9ull, 0xEAC0C6E7DCull, 0xE8396A503Bull, 0xE5B906E77Cull, 0xE33F8972BEull,
    0xE0CCDEEC2Aull, 0xDE60F4825Dull, 0xDBFBB797DAull, 0xD99D15C278ull, 0xD744FCCAD6ull, 0xD4F35AABCFull,
    0xD2A81D91F0ull, 0xD06333DAEEull, 0xCE248C151Full, 0xCBEC14FEF2ull, 0xC9B9BD866Dull, 0xC78D74C8ABull,
    0xC5672A1154ull, 0xC346CCDA24ull, 0xC12C4CCA66ull, 0xBF1799B67Aull, 0xBD08A39F57ull, 0xBAFF5AB212ull,
    0xB8FBAF4762ull, 0xB6FD91E328ull, 0xB504F333F9ull, 0xB311C412A8ull, 0xB123F581D2ull, 0xAF3B78AD68ull,
    0xAD583EEA42ull, 0xAB7A39B5A8ull, 0xA9A15AB4EAull, 0xA7CD93B4E9ull, 0xA5FED6A9B0ull, 0xA43515AE09ull,
    0xA27043030Bull, 0xA0B0510FB9ull, 0x9EF5326091ull, 0x9D3ED9A72Cull, 0x9B8D39B9D5ull, 0x99E0459320ull,
    0x9837F0518Dull, 0x96942D371Full, 0x94F4EFA8FEull, 0x935A2B2F13ull, 0x91C3D373AAull, 0x9031DC4314ull,
    0x8EA4398B45ull, 0x8D1ADF5B7Eull, 0x8B95C1E3EAull, 0x8A14D57549ull, 0x88980E8092ull, 0x871F61969Eull,
    0x85AAC367CCull, 0x843A28C3ACull, 0x82CD8698ABull, 0x8164D1F3BBull,
};

__device__ __forceinline__ float nothing() { return __uint_as_float(0x7FFFFFFFu); }   // NaN: no logit

struct alignas(16) SampleSmem {
    u64 table[64][16];                           // a copy for every pair of banks
    u64 part[2][NW], slot[2][MOST_CS];   // of an exchange, in turn
    u64 scan[2][NW];
    u64 group_sum[GROUPS];                       // of the row's logits, by the bins' middles
    u64 found_sum, run[2];
    uint32_t group[GROUPS];                      // the row's logits
    uint32_t near[MOST_CS][32];                  // of a group's bins and those beside it, by CTA
    uint32_t found[8];
    int listed;                                  // logits in `list`
    union {
        alignas(16) uint32_t hist[BINS];
        struct {
            u64 sorted[LIST];                    // key, and the index's complement below
            uint32_t bucket[BUCKETS];
        };
    };
    u64 list[LIST];
    // behind it: the sums of the row's warps, in turn; the row
};
__host__ __device__ constexpr size_t fixed_bytes(int warps) { return sizeof(SampleSmem) + 2 * sizeof(u64) * warps; }   // warps: of the row

// (in parts whose sums fit 32 bits: an instruction each)
__device__ __forceinline__ u64 warp_sum64(u64 v) {
    const uint32_t a = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)v & 0x7FFFFFFu);
    const uint32_t b = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)(v >> 27) & 0x7FFFFFFu);
    const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)(v >> 54));
    return a + ((u64)b << 27) + ((u64)c << 54);
}
template <class T> __device__ __forceinline__ T warp_scan(T v, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T w = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

// Shared memory of CTA z of the cluster.
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
__device__ __forceinline__ uint32_t peer32(const void* p, int z) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at_peer(p, z)) : "memory");
    return v;
}
__device__ __forceinline__ uint4 peer128(const uint32_t* p, int z) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at_peer(p, z)) : "memory");
    return v;
}
__device__ __forceinline__ void to_peer64(u64* p, int z, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(at_peer(p, z)), "l"(v) : "memory");
}
__device__ __forceinline__ void add_at_peer(u64* p, int z, u64 v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" :: "r"(at_peer(p, z)), "l"(v) : "memory");
}
__device__ __forceinline__ void add_at_peer(uint32_t* p, int z, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" :: "r"(at_peer(p, z)), "r"(v) : "memory");
}

// Sixteen bytes from global memory, on their way
__device__ __forceinline__ void cp_async16(float* to, const float* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(to)), "l"(from) : "memory");
}

// Floor and ceiling of v a for 0 <= a < 1, v below 2^63.
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
// w / all, w below 2^63: the f32 quotient, corrected once.
__device__ __forceinline__ float quotient(u64 w, u64 all) {
    const float w1 = __ull2float_rn(w), w2 = __ll2float_rn((long long)(w - (u64)w1));
    const float a1 = __ull2float_rn(all), a2 = __ll2float_rn((long long)(all - (u64)a1));
    const float q = __fdiv_rn(w1, a1), rest = fmaf(-q, a1, w1) + fmaf(-q, a2, w2);
    return q + __fdiv_rn(rest, a1);
}

// A row as one CTA of its cluster sees it.
struct Sampler {
    const SampleArgs& A;
    SampleSmem& sm;
    float* held;                // this warp's logits, the first A.held
    long long row;
    int lane, warp, cs, rank, first;                 // first: index of the warp's first logit
    int turn, owned;
    float top, u;
    float base, c_hi, c_lo, ref, ref64;              // t = ref - (x - base) (c_hi + c_lo)
    bool infinite;                                   // the largest logits are +inf: they are 0, the others nothing

    // Four logits from index i on
    __device__ __forceinline__ float4 load(int i) const {
        const long long n = A.p.n - i;
        float4 v = load_four(A.p.logits, A.p.type, row * A.p.stride + i, n < 4 ? (int)n : 4, A.four && n >= 4);
        v.x = n > 0 ? v.x : nothing();
        v.y = n > 1 ? v.y : nothing();
        v.z = n > 2 ? v.z : nothing();
        v.w = n > 3 ? v.w : nothing();
        return v;
    }
    __device__ __forceinline__ float finite(float x) const { return x == INFINITY ? 0.0f : nothing(); }
    // The lane's four of a warp's 128 from place i on; that warp's first logit has index `from`
    __device__ __forceinline__ float4 four(const float* theirs, int from, int i) const {
        if (i < A.held) return *reinterpret_cast<const float4*>(theirs + i + 4 * lane);
        float4 v = load(from + i + 4 * lane);
        if (infinite) v = make_float4(finite(v.x), finite(v.y), finite(v.z), finite(v.w));
        return v;
    }
    __device__ __forceinline__ int length(int from) const { return (int)min((long long)A.seg, (long long)A.p.n - from); }
    // f(logit, index) of all of this warp's
    template <class F> __device__ __forceinline__ void each(F f) const {
        const int end = length(first);
#pragma unroll 2
        for (int i = 0; i < end; i += 128) {
            const float4 v = four(held, first, i);
            const int j = first + i + 4 * lane;
            f(v.x, j);
            f(v.y, j + 1);
            f(v.z, j + 2);
            f(v.w, j + 3);
        }
    }
    __device__ __forceinline__ void together() const {
        __syncwarp();
        if (cs > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else __syncthreads();
    }

    // p is the rounded product wherever it is formed, and what is taken from it is taken from the rounded
    // one: left to the compiler, some of these may be fused, and a weight be off by p's own rounding
    __device__ __forceinline__ float less_base(float logit) const { return __fsub_rn(logit, base); }
    __device__ __forceinline__ float times_c(float x) const { return __fmul_rn(x, c_hi); }
    // 64 t rounded, MAGIC added: its bits count in steps of 1.  No less for a smaller
    // logit; NaN for none.  (x: less base; p: times c_hi)
    __device__ __forceinline__ float steps(float p) const { return fmaf(p, -64.0f, ref64); }
    __device__ __forceinline__ bool weighs(float s) const { return s < MAGIC + (float)BINS; }   // (false for NaN)
    __device__ __forceinline__ int bin_of(float s) const { return (int)(__float_as_uint(s) - __float_as_uint(MAGIC)); }
    __device__ __forceinline__ int bin(float x) const {   // BINS where there is no weight
        const float s = steps(times_c(less_base(x)));
        return weighs(s) ? bin_of(s) : BINS;
    }
    // 2^(60 - (f mod 64)/64 - r), and 2^(40 - f/64 - r).  2^-r - 1 (below 2^-7) in steps of 2^-29 is the rounding that
    // counts: 2^-30; the series before it is good to 2^-31, the 28 bits of the table that it is multiplied by to 2^-34
    __device__ __forceinline__ u64 power_of_rest(uint32_t f, float r) const {
        constexpr float S = 536870912.0f;   // 2^29
        const float s = fmaf(r, fmaf(r, fmaf(r, -0.0555041087f * S, 0.240226507f * S), -0.693147181f * S), MAGIC);
        const u64 v = sm.table[f & 63][lane & 15];
        return v + (u64)((long long)(int)(v >> 32) * (8 * bin_of(s)));
    }
    __device__ __forceinline__ u64 power(uint32_t f, float r) const { return power_of_rest(f, r) >> (20 + (f >> 6)); }
    __device__ __forceinline__ u64 middle(int f) const { return sm.table[f & 63][lane & 15] >> (20 + (f >> 6)); }
    __device__ __forceinline__ float rest(float x, float p, float s) const {
        const float y = fmaf(s - MAGIC, -0.015625f, ref);       // ref - f/64, exact
        return fmaf(x, -c_lo, __fsub_rn(__fsub_rn(y, p), fmaf(x, c_hi, -p)));
    }
    // w of any logit, to be used where `there`: without a branch, so that those of
    // several logits are worked out side by side
    __device__ __forceinline__ u64 weight(float logit, bool& there, int& b) const {
        const float x = less_base(logit), p = times_c(x), s = steps(p), in = fminf(s, MAGIC + (float)BINS);   // (NaN: BINS)
        there = weighs(s);
        b = bin_of(in);
        return power(b, rest(x, p, in));
    }
    __device__ __forceinline__ u64 weight(float logit, bool& there) const {
        int b;
        return weight(logit, there, b);
    }
    __device__ __forceinline__ u64 weight(float logit) const {   // 0 where there is none
        bool there;
        const u64 w = weight(logit, there);
        return there ? w : 0;
    }
    // The sum of the w's of this warp's logits that keep(logit, index) takes, a lane's part of it
    template <class F> __device__ __forceinline__ u64 weights(F keep) const {
        const int end = length(first);
        u64 sum = 0;
#pragma unroll 2
        for (int i = 0; i < end; i += 128) {
            const float4 v = four(held, first, i);
            const float x[4] = {v.x, v.y, v.z, v.w};
            const int at = first + i + 4 * lane;
            bool in[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) in[j] = keep(x[j], at + j);
            if (!__any_sync(0xFFFFFFFFu, in[0] || in[1] || in[2] || in[3])) continue;   // (min_p leaves few)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bool there;
                const u64 w = weight(x[j], there);
                if (there && in[j]) sum += w;
            }
        }
        return sum;
    }
    // The share of a logit that has a weight in `all`.  Of a small w the bits below 1,
    // which the sums leave out, count here.
    __device__ __forceinline__ float chance(float logit, u64 all) const {
        const float x = less_base(logit), p = times_c(x), s = steps(p);
        const int f = bin_of(s);
        return quotient(power_of_rest(f, rest(x, p, s)), all) * __uint_as_float((uint32_t)(127 - 20 - (f >> 6)) << 23);
    }

    // Sum, or maximum (of 32 bits), of the threads' v over the row.
    template <bool MAX> __device__ u64 exchange(u64 v) {
        const int b = turn & 1;
        ++turn;
        auto warps = [](u64 x) { return MAX ? (u64)__reduce_max_sync(0xFFFFFFFFu, (uint32_t)x) : warp_sum64(x); };
        v = warps(v);
        if (lane == 0) sm.part[b][warp] = v;
        __syncthreads();
        if (cs == 1 || warp == 0) v = warps(lane < NW ? sm.part[b][lane] : 0);
        if (cs == 1) return v;
        if (warp == 0 && lane < cs) to_peer64(&sm.slot[b][rank], lane, v);
        together();
        return warps(lane < cs ? sm.slot[b][lane] : 0);
    }
    // Exclusive sum of the threads' value over the CTA, and the sum of all.
    __device__ __forceinline__ u64 block_scan(u64 v, u64& all) {
        const u64 in = warp_scan(v, lane);
        __syncthreads();   // (what was there has been read)
        if (lane == 31) sm.scan[0][warp] = in;
        __syncthreads();
        const u64 x = lane < NW ? sm.scan[0][lane] : 0;
        all = warp_sum64(x);
        return in - v + warp_sum64(lane < warp ? x : 0);
    }

    // The key of the largest logit whose bin is >= b (the bins fall as the keys
    // rise), b <= BINS.  It lies close to where f32 arithmetic puts it; a lane tries
    // a key each.
    __device__ uint32_t up_to(int b) const {
        if (bin(top) >= b) return key_of(top);
        uint32_t lo = LOWEST, hi = key_of(top);      // it is lo or above, and below hi
        auto reaches = [&](uint32_t k) { return bin(logit_of(k)) >= b; };
        const uint32_t guess = min(max(key_of(base + (ref - ((float)b - 0.5f) * 0.015625f) / c_hi), LOWEST + 32), 0xFF800000u);
        const uint32_t k = guess + 15 - lane;
        int yes = __ffs(__ballot_sync(0xFFFFFFFFu, k < hi && reaches(k))) - 1;
        if (guess < hi) {
            if (yes > 0) return guess + 15 - yes;
            if (yes == 0) lo = guess + 15;
            else hi = guess - 16;
        }
        while (hi - lo > 1) {
            const uint32_t far = hi - lo, step = (far + 31) / 32, off = step * (lane + 1);   // (far < 2^32 - 2^23)
            yes = __ffs(__ballot_sync(0xFFFFFFFFu, off >= far || reaches(hi - off))) - 1;
            const uint32_t z = hi - step * yes;
            lo = (uint32_t)(max((u64)lo + step, (u64)z) - step);
            hi = z;
        }
        return lo;
    }

    // Adds the histogram's bins up in groups, at every CTA (complete after a barrier).
    __device__ __forceinline__ void add_groups(bool sum) {
        __syncthreads();
        for (int at = 0; at < BINS; at += 4 * NT) {   // four bins a thread, a group in four lanes
            const int b = at + 4 * (int)threadIdx.x;
            if (b >= BINS) break;                     // (whole warps)
            const uint4 c = *reinterpret_cast<const uint4*>(sm.hist + b);
            uint32_t n = c.x + c.y + c.z + c.w;
            u64 v = 0;
            if (sum && n) v = c.x * middle(b) + c.y * middle(b + 1) + c.z * middle(b + 2) + c.w * middle(b + 3);
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
                if (sum) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            }
            for (int z = lane & 3; n && z < cs; z += 4)   // (a lane of the group for every fourth CTA)
                if (cs == 1) {
                    sm.group[b / COARSE] = n;
                    sm.group_sum[b / COARSE] = v;
                } else {
                    add_at_peer(&sm.group[b / COARSE], z, n);
                    if (sum) add_at_peer(&sm.group_sum[b / COARSE], z, v);
                }
        }
    }
    // Where the histogram has the border (by the bins' middles, for sums): its bin (BINS:
    // nowhere), the logits down to it and in it, and in its neighbours; for warp 0.
    struct Place { int b; uint32_t live, down_to, there, above, below; };
    // For sums the border may be some bins off, the more so the fewer logits have most of
    // the sum (a bin's w's are up to 2^(1/128) off its middle).  So the list takes in groups of bins
    // around, as far as they fit: `wide` not from the top.  False: nothing fits.
    __device__ bool window(const Place& P, int& first_bin, int& last_bin, bool& wide) const {
        constexpr int AROUND = 8;
        const int g = P.b / COARSE;
        // lanes 0 .. 7: groups g + lane + 1 and what is down to them; lanes 8 .. 15: g - 1 - (lane - 8)
        const int mine = lane < AROUND ? g + 1 + lane : g - 1 - (lane - AROUND);
        const uint32_t n = lane < 2 * AROUND && mine >= 0 && mine < GROUPS ? sm.group[mine] : 0;
        const uint32_t in = warp_scan(n, lane), up = in - __shfl_sync(0xFFFFFFFFu, in, AROUND - 1);   // of each side, to the lane
        uint32_t to_end = 0;   // from the border's bin to its group's end
        for (int i = lane; i < GROUPS; i += 32) to_end += i <= g ? sm.group[i] : 0;
        to_end = __reduce_add_sync(0xFFFFFFFFu, to_end) - P.down_to;
        const uint32_t down = P.down_to + to_end;   // logits to the end of the border's group
        wide = P.down_to + P.below > (uint32_t)LIST;
        if (!wide) {
            first_bin = 0;
            last_bin = P.b + 1;
            if (down <= (uint32_t)LIST) {
                const int more = __popc(__ballot_sync(0xFFFFFFFFu, lane < AROUND && down + in <= (uint32_t)LIST));
                last_bin = max(last_bin, (g + more) * COARSE + COARSE - 1);
            }
        } else {
            const uint32_t group = sm.group[g];
            if (group <= (uint32_t)LIST) {
                // as many groups on both sides as fit together
                const uint32_t below = __shfl_sync(0xFFFFFFFFu, in, lane & (AROUND - 1)), above = __shfl_sync(0xFFFFFFFFu, up, AROUND + (lane & (AROUND - 1)));
                const int more = __popc(__ballot_sync(0xFFFFFFFFu, lane < AROUND && group + below + above <= (uint32_t)LIST));
                first_bin = (g - more) * COARSE;
                last_bin = (g + more) * COARSE + COARSE - 1;
                if (more == 0) {   // the neighbours, where the border is at the group's end
                    if (P.b == first_bin && group + P.above <= (uint32_t)LIST) first_bin = P.b - 1;
                    if (P.b == last_bin && group + P.below <= (uint32_t)LIST) last_bin = P.b + 1;
                }
            } else {
                const bool one = P.below + P.there + P.above > (uint32_t)LIST;
                if (P.there > (uint32_t)LIST) return false;
                first_bin = one ? P.b : P.b - 1;
                last_bin = one ? P.b : P.b + 1;
            }
        }
        first_bin = max(first_bin, 0);
        last_bin = min(last_bin, BINS - 1);
        return true;
    }
    __device__ Place locate(bool sum, u64 target) const {
        constexpr int L = GROUPS / 32;
        Place P = {BINS, 0, 0, 0, 0, 0};
        int group = -1;
        u64 at = 0;
        uint32_t at_n = 0;
        if (warp < cs) {   // the group; its bins of CTA `warp`, in lanes 1 .. 16, the neighbours beside them
            uint32_t n[L], mine_n = 0;
            u64 v[L], mine = 0;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                n[i] = sm.group[lane * L + i];
                v[i] = sum ? sm.group_sum[lane * L + i] : n[i];
                mine += v[i];
                mine_n += n[i];
            }
            const u64 in = warp_scan(mine, lane);
            u64 pre = in - mine;
            int found = -1;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (found < 0 && n[i] && pre < target && pre + v[i] >= target) found = i;
                if (found < 0) pre += v[i];
            }
            const unsigned who = __ballot_sync(0xFFFFFFFFu, found >= 0);
            P.live = __reduce_add_sync(0xFFFFFFFFu, mine_n);
            if (who) {
                const int l = __ffs(who) - 1, i = __shfl_sync(0xFFFFFFFFu, found, l);
                at = __shfl_sync(0xFFFFFFFFu, pre, l);
                group = l * L + i;
                uint32_t above = lane < l ? mine_n : 0;
#pragma unroll
                for (int k = 0; k < L; ++k) above += lane == l && k < i ? n[k] : 0;
                at_n = __reduce_add_sync(0xFFFFFFFFu, above);
                const int b = group * COARSE + lane - 1;
                uint32_t c = 0;
                if (lane < COARSE + 2 && b >= 0 && b < BINS) c = cs > 1 ? peer32(&sm.hist[b], warp) : sm.hist[b];
                sm.near[warp][lane] = c;
            }
        }
        __syncthreads();
        if (warp == 0 && group >= 0) {
            uint32_t c = 0;
#pragma unroll
            for (int z = 0; z < MOST_CS; ++z) c += z < cs ? sm.near[z][lane] : 0;
            sm.near[0][lane] = c;   // (of the row now)
            const bool inside = lane >= 1 && lane <= COARSE;
            const u64 w = inside && c ? (sum ? c * middle(group * COARSE + lane - 1) : c) : 0, down = warp_scan(w, lane);
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, inside && c && at + down - w < target && at + down >= target);
            if (hit) {
                const int h = __ffs(hit) - 1;
                P.b = group * COARSE + h - 1;
                P.there = __shfl_sync(0xFFFFFFFFu, c, h);
                P.above = __shfl_sync(0xFFFFFFFFu, c, h - 1);
                P.below = __shfl_sync(0xFFFFFFFFu, c, h + 1);
                P.down_to = at_n + __reduce_add_sync(0xFFFFFFFFu, inside && lane <= h ? c : 0);
            }
        }
        return P;
    }

    // The sum, by the middles, of the bins before bin b; P: what was located last (warp 0)
    __device__ u64 estimate(const Place& P, int b) const {
        const int g = b / COARSE;
        u64 v = 0;
        for (int i = lane; i < g; i += 32) v += sm.group_sum[i];
        const int at = g * COARSE + lane;
        if (at < b) {   // bins of its own group
            uint32_t c = 0;
            if (g == P.b / COARSE) c = sm.near[0][lane + 1];
            else
                for (int z = 0; z < cs; ++z) c += cs > 1 ? peer32(&sm.hist[at], z) : sm.hist[at];
            v += c * middle(at);
        }
        return warp_sum64(v);
    }

    // Puts the logits of lo .. hi on this CTA's list, and the w's of those above
    // into the warps' sums; the logits on all lists (more than LIST: they are not whole),
    // and on that of CTA `lane`.
    __device__ int collect(float lo, float hi, int& parts) {
        u64 above = 0;
        const int end = length(first);
        for (int i = 0; i < end; i += 128) {
            const float4 v = four(held, first, i);
            const float x[4] = {v.x, v.y, v.z, v.w};
            if (!__any_sync(0xFFFFFFFFu, v.x >= lo || v.y >= lo || v.z >= lo || v.w >= lo)) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (x[j] > hi) above += weight(x[j]);
                const bool in = x[j] >= lo && x[j] <= hi;
                const unsigned who = __ballot_sync(0xFFFFFFFFu, in);
                if (!who) continue;
                int at = 0;
                if (lane == 0) at = atomicAdd(&sm.listed, __popc(who));
                at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(who & ((1u << lane) - 1));
                if (in && at < LIST) sm.list[at] = (u64)key_of(x[j] + 0.0f) << 32 | (0xFFFFFFFFu - (uint32_t)(first + i + 4 * lane + j));
            }
        }
        put_own(warp_sum64(above));
        together();
        const int n = lane < cs ? (cs > 1 ? (int)peer32(&sm.listed, lane) : sm.listed) : 0;
        parts = min(n, LIST + 1);
        return __reduce_add_sync(0xFFFFFFFFu, parts);
    }
    // Values threadIdx.x and threadIdx.x + NT of all lists (0 past the n)
    __device__ void bring(int n, int parts, u64 (&e)[2]) const {
        int end[MOST_CS];   // of the lists, one after the other
#pragma unroll
        for (int z = 0; z < MOST_CS; ++z) end[z] = __shfl_sync(0xFFFFFFFFu, parts, z) + (z ? end[z ? z - 1 : 0] : 0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = threadIdx.x + k * NT;
            int z = 0, from = 0;
#pragma unroll
            for (int j = 0; j < MOST_CS - 1; ++j)
                if (i >= end[j]) {
                    z = j + 1;
                    from = end[j];
                }
            e[k] = i >= n ? 0 : cs > 1 ? peer64(&sm.list[i - from], z) : sm.list[i];
        }
    }
    // The n <= LIST distinct values that the threads hold into sm.sorted, in descending
    // order.  bucket: of a value, BUCKETS of them, no less for a smaller one.
    template <class B> __device__ void order(int n, const u64 (&e)[2], B bucket) {
        __syncthreads();
        if (threadIdx.x < BUCKETS) sm.bucket[threadIdx.x] = 0;
        __syncthreads();
        int b[2];
        uint32_t place[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            b[k] = e[k] ? bucket(e[k]) : 0;
            place[k] = e[k] ? atomicAdd(&sm.bucket[b[k]], 1u) : 0;
        }
        __syncthreads();
        const uint32_t c = threadIdx.x < BUCKETS ? sm.bucket[threadIdx.x] : 0, in = warp_scan(c, lane);
        if (lane == 31) sm.scan[0][warp] = in;
        __syncthreads();
        if (threadIdx.x < BUCKETS) sm.bucket[threadIdx.x] = in - c + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? (uint32_t)sm.scan[0][lane] : 0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (e[k]) sm.sorted[sm.bucket[b[k]] + place[k]] = e[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (e[k]) {   // its place in its bucket
                const uint32_t from = sm.bucket[b[k]], to = b[k] + 1 < BUCKETS ? sm.bucket[b[k] + 1] : n;
                place[k] = from;
                for (uint32_t i = from; i < to; ++i) place[k] += sm.sorted[i] > e[k];
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (e[k]) sm.sorted[place[k]] = e[k];
        __syncthreads();
    }

    // The warps' sums into every CTA's sums() (complete once all are together; what was
    // there a turn ago may still be read).
    __device__ void put_own(u64 mine) {
        ++owned;
        u64* at = &sums()[rank * NW + warp];
        if (cs == 1 && lane == 0) *at = mine;
        if (cs > 1 && lane < cs) to_peer64(at, lane, mine);
    }
    __device__ __forceinline__ u64* sums() const { return reinterpret_cast<u64*>(&sm + 1) + (owned & 1 ? cs * NW : 0); }
    __device__ void tell(u64 mine) {
        put_own(mine);
        together();
    }
    // The first index at which the sum of f over the row exceeds target_of(the whole),
    // which is less than that; in all lanes of one warp, -1 in the others.  The warps'
    // sums are in sums().  f: logit, index.
    template <class F, class G> __device__ int find(F f, G target_of) {
        // the warp that has it: a lane adds up neighbouring ones
        const int per = (cs * NW + 31) / 32;
        u64 v = 0, pre;
        for (int i = lane * per; i < min((lane + 1) * per, cs * NW); ++i) v += sums()[i];
        const u64 in = warp_scan(v, lane);
        const u64 target = target_of(__shfl_sync(0xFFFFFFFFu, in, 31));
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, in > target);
        int who = -1;
        if (hit) {
            const int l = __ffs(hit) - 1;
            who = l * per;
            pre = __shfl_sync(0xFFFFFFFFu, in - v, l);
            while (pre + sums()[who] <= target) pre += sums()[who++];
        }
        if (who < 0 || who / NW != rank) return -1;
        // its logits: 128 a warp of this CTA, in rounds
        const int w = who - rank * NW, at = who * A.seg, end = length(at);
        const float* const theirs = held + (w - warp) * A.held;
        for (int i0 = 0; i0 < end; i0 += 128 * NW) {
            const int i = i0 + 128 * warp, j = at + i + 4 * lane;
            float4 x = make_float4(nothing(), nothing(), nothing(), nothing());
            if (i < end) x = four(theirs, at, i);
            const u64 a = f(x.x, j), b = f(x.y, j + 1), c = f(x.z, j + 2), d = f(x.w, j + 3), mine = warp_sum64(a + b + c + d);
            __syncthreads();   // (what was there has been read)
            if (lane == 0) sm.scan[0][warp] = mine;
            __syncthreads();
            const u64 part = lane < NW ? sm.scan[0][lane] : 0, here = pre + warp_sum64(lane < warp ? part : 0);
            if (here <= target && target < here + mine) {
                const u64 in = warp_scan(a + b + c + d, lane), before = here + in - (a + b + c + d);
                const int l = __ffs(__ballot_sync(0xFFFFFFFFu, here + in > target)) - 1;
                const int k = before + a > target ? 0 : before + a + b > target ? 1 : before + a + b + c > target ? 2 : 3;
                return __shfl_sync(0xFFFFFFFFu, j + k, l);
            }
            const u64 round = warp_sum64(part);
            if (pre + round > target) return -1;   // (in another warp)
            pre += round;
        }
        return -1;
    }
    // The place in the kept w's that u points at
    __device__ u64 target_of(u64 all) const { return u < 1.0f ? share_of(all, u, false) : all - 1; }
    __device__ void put(int token, float prob) const {
        A.p.tokens[row] = token;
        if (A.p.prob) A.p.prob[row] = prob;
    }
    // The token, of the logits above `border` and those equal to it up to index
    // `last`; the warps' sums of their w's are in sums().
    __device__ void finish(float border, int last) {
        u64 all = 0;
        const int at = find([&](float x, int i) -> u64 { return x > border || (x == border && i <= last) ? weight(x) : 0; },
                            [&](u64 sum) { all = sum; return target_of(sum); });
        if (at >= 0 && lane == 0) {
            float x = value_at(A.p.logits, A.p.type, row * A.p.stride + at) + 0.0f;
            if (infinite) x = finite(x);
            put(at, chance(x, all));
        }
    }

    // ------------------------------------------------ rows that the histogram does not settle
    // The w's sum of the logits from `from` on.
    __device__ u64 total(float from) {
        return exchange<false>(weights([&](float x, int) { return x >= from; }));
    }
    // The index of the logit equal to `border` that `before` equal ones precede.
    __device__ int tie_at(float border, u64 before) {
        u64 mine = 0;
        each([&](float x, int) { mine += x == border; });
        tell(warp_sum64(mine));
        const int at = find([&](float x, int) -> u64 { return x == border; }, [&](u64) { return before; });
        return (int)(0xFFFFFFFFu - (uint32_t)exchange<true>(at < 0 ? 0 : 0xFFFFFFFFu - (uint32_t)at));
    }
    // Empties the histogram, once every CTA has read it.
    __device__ __forceinline__ void empty() const {
        together();
        for (int i = threadIdx.x; i < BINS / 4; i += NT) reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    // Four bins of the row's histogram (after a barrier)
    __device__ __forceinline__ uint4 counts(int b) const {
        if (cs == 1) return *reinterpret_cast<const uint4*>(sm.hist + b);
        uint4 c = make_uint4(0, 0, 0, 0);
        for (int z = 0; z < cs; ++z) {
            const uint4 v = peer128(sm.hist + b, z);
            c.x += v.x;
            c.y += v.y;
            c.z += v.z;
            c.w += v.w;
        }
        return c;
    }
    // Exclusive sums of the threads' pair over the CTA.
    __device__ __forceinline__ void block_scan_two(u64& a, u64& b) {
        const u64 ai = warp_scan(a, lane), bi = warp_scan(b, lane);
        __syncthreads();   // (what was there has been read)
        if (lane == 31) {
            sm.scan[0][warp] = ai;
            sm.scan[1][warp] = bi;
        }
        __syncthreads();
        const u64 x = lane < warp ? sm.scan[0][lane] : 0, y = lane < warp ? sm.scan[1][lane] : 0;
        a = ai - a + warp_sum64(x);
        b = bi - b + warp_sum64(y);
    }

    struct Border { uint32_t key, ties, of; };   // ties kept of `of`

    // The border of the row at which the count (mass = false) or the w's sum of
    // the logits in descending order reaches `target` >= 1 (which they do).  Below
    // `floor_` nothing counts, and of the logits equal to it `missing` do not.
    __device__ Border select(bool mass, u64 target, uint32_t floor_, uint32_t missing) {
        uint32_t hi = key_of(top), lo = floor_;
        bool by_t = true;
        for (;;) {
            hi = range_end(hi);
            const KeyBins K(lo, hi);
            auto place = [&](uint32_t k) { return by_t ? min(bin(logit_of(k)), BINS - 1) : K.bin(k); };
            empty();
            u64 mine = 0;
            const float hi_x = logit_of(hi), lo_x = logit_of(lo);
            each([&](float x, int) {
                if (x > hi_x) mine += mass ? weight(x) : 1;
                else if (x >= lo_x) atomicAdd(&sm.hist[place(key_of(x + 0.0f))], 1u);
            });
            const u64 above = exchange<false>(mine);
            // a thread's bins, four at a time: how many, and the bounds of their sums
            u64 up_run = above, down_run = above;
            if (threadIdx.x == 0) { sm.found[0] = BINS; sm.found[1] = BINS; sm.found[4] = 0; }
            for (int at = 0; at < BINS; at += 4 * NT) {
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
                            const uint32_t k1 = K.first(b), k0 = K.last(b);
                            w1 = weight(logit_of(k1));
                            w0 = k0 == k1 ? w1 : weight(logit_of(k0));
                            if (k0 != k1) {   // w is right to 2^-29, and may fall by that where it should rise
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
                block_scan_two(up_at, down_at);
                if (threadIdx.x == NT - 1) { sm.run[0] = up_at + up; sm.run[1] = down_at + down; }
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
                up_run += sm.run[0];
                down_run += sm.run[1];
            }
            const int last = (int)sm.found[4], b1 = min((int)sm.found[0], last), b2 = min((int)sm.found[1], last);
            const uint32_t count = sm.found[2];
            const u64 before = sm.found_sum;
            __syncthreads();
            if (!by_t && K.shift == 0) {
                Border B;
                B.key = hi - b1;
                B.of = count;
                const u64 w = mass ? weight(logit_of(B.key)) : 1;
                const u64 need = target > before && w ? (target - before + w - 1) / w : 1;
                B.ties = (uint32_t)(need < 1 ? 1 : need > count ? count : need);
                return B;
            }
            const uint32_t wide = hi - lo;
            if (by_t) {
                hi = up_to(b1);
                lo = max(lo, up_to(b2 + 1) + 1);
                by_t = false;
                continue;
            }
            lo = K.last(b2);
            hi = K.first(b1);
            if (hi - lo > wide / 4) {   // bounds that tell the bins apart badly: halve what is left
                const uint32_t mid = range_end(lo + (hi - lo) / 2);
                const float mid_x = logit_of(mid);
                u64 v = 0;
                each([&](float x, int) {
                    if (x > mid_x) v += mass ? weight(x) : 1;
                });
                if (exchange<false>(v) >= target) lo = mid + 1;
                else hi = mid;
            }
        }
    }
};

// CTA (row, , rank in the row's cluster).
__global__ void __launch_bounds__(NT, 2) sample_kernel(const __grid_constant__ SampleArgs A) {
    extern __shared__ __align__(16) uint8_t sample_raw[];
    SampleSmem& sm = *reinterpret_cast<SampleSmem*>(sample_raw);
    grid_launch_dependents();
    if (gridDim.z > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // waited for before peers are written to
    Sampler S{A, sm};
    S.row = blockIdx.x;
    S.lane = threadIdx.x & 31;
    S.warp = threadIdx.x >> 5;
    S.cs = gridDim.z;
    S.rank = blockIdx.z;
    S.first = (int)min((long long)(S.rank * NW + S.warp) * A.seg, (long long)A.p.n);
    S.turn = S.owned = 0;
    S.infinite = false;
    S.held = reinterpret_cast<float*>(sample_raw + fixed_bytes(S.cs * NW)) + S.warp * A.held;
    // The row's copy into shared memory, under way while the rest of it is made ready
    const int end = S.length(S.first), copied = A.four && A.p.type == PLM_F32 ? min(end, A.held) : 0;
    grid_wait_prior();
    {
        const float* const from = static_cast<const float*>(A.p.logits) + S.row * A.p.stride + S.first;
        for (int i = 4 * S.lane; i < ((copied + 127) & ~127); i += 128)
            if (i + 4 <= copied) cp_async16(S.held + i, from + i);
            else
                for (int j = i; j < i + 4; ++j) S.held[j] = j < copied ? from[j] : nothing();
    }
    for (int i = threadIdx.x; i < 64 * 16; i += NT) sm.table[i / 16][i % 16] = EXP_TABLE[i / 16] << 20;
    for (int i = threadIdx.x; i < GROUPS; i += NT) sm.group[i] = sm.group_sum[i] = 0;
    if (threadIdx.x == 0) sm.listed = 0;
    for (int i = threadIdx.x; i < BINS / 4; i += NT) reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0, 0, 0, 0);
    const float T = A.p.temperature ? A.p.temperature[S.row] : 1.0f;
    const int k = A.p.top_k ? A.p.top_k[S.row] : 0;
    const float p = A.p.top_p ? A.p.top_p[S.row] : 1.0f, low = A.p.min_p ? A.p.min_p[S.row] : 0.0f;
    S.u = A.p.u ? fmaxf(A.p.u[S.row], 0.0f) : 0.0f;
    // the row, and its largest logit
    float best = -INFINITY;
    {
        constexpr int AHEAD = 5;   // loads in flight
#pragma unroll 1
        for (int i0 = (copied + 127) & ~127; i0 < end; i0 += 128 * AHEAD) {
            float4 v[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                v[j] = i0 + 128 * j < end ? S.load(S.first + i0 + 128 * j + 4 * S.lane) : make_float4(nothing(), nothing(), nothing(), nothing());
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int i = i0 + 128 * j;
                if (i < min(end, A.held)) *reinterpret_cast<float4*>(S.held + i + 4 * S.lane) = v[j];
                best = fmaxf(fmaxf(best, fmaxf(v[j].x, v[j].y)), fmaxf(v[j].z, v[j].w));   // (NaN counts for nothing)
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < copied; i += 128) {
            const float4 v = *reinterpret_cast<const float4*>(S.held + i + 4 * S.lane);
            best = fmaxf(fmaxf(best, fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
        }
    }
    if (S.cs > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // all CTAs of the row have begun
    const uint32_t most = (uint32_t)S.exchange<true>(key_of(best + 0.0f));
    S.top = logit_of(most);
    const bool leader = S.rank == 0 && threadIdx.x == 0;
    if (most <= LOWEST) {
        if (leader) S.put(-1, 0.0f);
    } else if (!(T > 0.0f) || !A.p.u) {
        uint32_t at = 0;   // the first index, as its complement
        if (__any_sync(0xFFFFFFFFu, best == S.top))   // (few warps)
            S.each([&](float x, int i) {
                if (x == S.top) at = max(at, 0xFFFFFFFFu - (uint32_t)i);
            });
        at = (uint32_t)S.exchange<true>(at);
        if (leader) S.put((int)(0xFFFFFFFFu - at), 1.0f);
    } else {
        if (S.top == INFINITY) {
            S.infinite = true;
            const int end = min(A.held, S.length(S.first));
            for (int i = 4 * S.lane; i < end; i += 128)
                for (int j = i; j < i + 4; ++j) S.held[j] = S.finite(S.held[j]);
            S.top = 0.0f;
            __syncwarp();
        }
        {   // c = log2(e) / T as a pair of f32: the quotient and what it leaves
            const float l_hi = 1.44269502f, l_lo = 1.92596299e-8f;   // log2(e)
            const float q = fminf(__fdiv_rn(l_hi, T), 3e38f);
            S.c_hi = q;
            S.c_lo = q < 1e37f && T < 1e37f && T > 1e-30f ? __fdiv_rn(fmaf(-q, T, l_hi) + l_lo, T) : 0.0f;
        }
        // Logits near the top differ from it exactly; else the reference is 0
        S.base = fabsf(S.top * S.c_hi) < 80.0f ? 0.0f : S.top;
        S.ref = ceilf((S.top - S.base) * S.c_hi * 64.0f) * 0.015625f;
        S.ref64 = S.ref * 64.0f + MAGIC;
        const bool by_k = k > 0 && k < A.p.n, by_p = p < 1.0f;
        // min_p: the smallest f32 that is at least max + T ln(min_p)
        uint32_t floor_ = LOWEST + 1;
        if (low > 0.0f) {
            if (threadIdx.x == 0) {
                const double at = (double)S.top + (double)T * log((double)fminf(low, 1.0f));   // (NaN: T is infinite, min_p 1)
                sm.found[7] = S.infinite ? key_of(0.0f) : at == at ? min(key_of(__double2float_ru(at) + 0.0f), key_of(S.top)) : floor_;
            }
            __syncthreads();
            floor_ = sm.found[7];
            __syncthreads();
        }
        uint32_t border = floor_;   // what is kept: the keys above, and those equal up to index `last`
        int last = 0x7FFFFFFF;
        enum { AGAIN, LISTED, WIDE, DONE } how = DONE;
        if (by_k || by_p) {
            // The histogram; for top_p alone also the sum of all w's
            u64 mine = 0;
            if (by_k) {
                S.each([&](float x, int) {
                    const float s = S.steps(S.times_c(S.less_base(x)));
                    if (S.weighs(s)) atomicAdd(&sm.hist[S.bin_of(s)], 1u);
                });
            } else {
                S.each([&](float x, int) {
                    bool there;
                    int b;
                    const u64 w = S.weight(x, there, b);
                    if (there) {
                        atomicAdd(&sm.hist[b], 1u);
                        mine += w;
                    }
                });
            }
            S.add_groups(!by_k);
            const u64 sum = S.exchange<false>(mine);
            u64 target = by_k ? k : share_of(sum, fmaxf(p, 0.0f), true);
            if (target < 1) target = 1;
            u64 aim = target;   // the target in what the middles say
            uint32_t live = 0;
            // By the middles the border may seem to lie where it does not.  Then the sum of what lies above the window,
            // which is exact, says how far off they are.
            for (int attempt = 0;; ++attempt) {
                const Sampler::Place P = S.locate(!by_k, aim);
                if (S.warp == 0) {
                    // The list: down to the border's bin for top_k, with what is around for top_p
                    uint32_t lo = LOWEST + 1, hi = key_of(S.top);
                    int first_bin = 0, last_bin = P.b;
                    bool wide = false, far = P.b >= BINS || (by_k && P.down_to > (uint32_t)LIST);
                    if (!far && !by_k) far = !S.window(P, first_bin, last_bin, wide);
                    u64 before = 0;
                    if (!far) {
                        lo = S.up_to(last_bin + 1) + 1;
                        if (wide) {
                            hi = S.up_to(first_bin);
                            before = S.estimate(P, first_bin);
                        }
                    }
                    if (S.lane == 0) {
                        sm.found[0] = lo;
                        sm.found[1] = hi;
                        sm.found[2] = wide;
                        sm.found[3] = far;
                        sm.found[4] = P.live;
                        sm.found[5] = last_bin;
                        sm.found_sum = before;
                    }
                }
                __syncthreads();
                uint32_t lo = sm.found[0];
                const uint32_t hi = sm.found[1], bins = sm.found[5] + 1;
                const u64 before = sm.found_sum;
                live = sm.found[4];
                how = sm.found[3] ? AGAIN : sm.found[2] ? WIDE : LISTED;
                __syncthreads();
                if (by_k && live <= (uint32_t)k) {
                    how = by_p ? AGAIN : DONE;                 // top_k leaves all that have a weight
                    break;
                }
                if (how == AGAIN) break;
                // what min_p leaves out need not be looked at, but counts in what top_p is of
                if (!(by_k && by_p) && floor_ > lo) lo = floor_;
                if (lo > hi) {                                 // min_p seems to leave less than top_p
                    how = S.total(logit_of(floor_)) <= target ? DONE : AGAIN;
                    break;
                }
                int parts;
                const int n = S.collect(logit_of(lo), logit_of(hi), parts);
                if (n > LIST || n == 0) {
                    how = AGAIN;
                    break;
                }
                u64 e[2], w[2], above = 0, listed;
                S.bring(n, parts, e);
                if (!by_k) {
                    if (how == WIDE) {
                        for (int i = S.lane; i < S.cs * NW; i += 32) above += S.sums()[i];
                        above = warp_sum64(above);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) w[j] = e[j] ? S.weight(logit_of((uint32_t)(e[j] >> 32))) : 0;
                    S.block_scan(w[0] + w[1], listed);
                    // (a list that min_p has cut short need not reach the target)
                    if (above >= target || (above + listed < target && lo > floor_)) {
                        how = AGAIN;
                        if (attempt == 2) break;
                        if (above >= target) {
                            aim = target + before - above;
                        } else {                               // what the list reaches, by the middles
                            if (S.warp == 0) {
                                const u64 end = S.estimate(P, (int)bins);
                                if (S.lane == 0) sm.found_sum = end;
                            }
                            __syncthreads();
                            aim = target + sm.found_sum - (above + listed);
                        }
                        if ((long long)aim < 1) break;         // (the estimate was worth nothing)
                        S.together();                          // every CTA has read the lists and histograms
                        if (threadIdx.x == 0) sm.listed = 0;
                        __syncthreads();
                        continue;
                    }
                }
                if (how == WIDE) {
                    const uint32_t step = (hi - lo) / BUCKETS + 1;
                    S.order(n, e, [&](u64 v) { return (int)((hi - (uint32_t)(v >> 32)) / step); });
                } else {
                    const uint32_t step = (bins + BUCKETS - 1) / BUCKETS;
                    S.order(n, e, [&](u64 v) { return min(S.bin(logit_of((uint32_t)(v >> 32))) / (int)step, BUCKETS - 1); });
                }
                // a thread's two values of the list, in descending order
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int i = 2 * threadIdx.x + j;
                    e[j] = i < n ? sm.sorted[i] : 0;
                    w[j] = i < n && (!by_k || i < k) ? S.weight(logit_of((uint32_t)(e[j] >> 32))) : 0;
                }
                const u64 pre = S.block_scan(w[0] + w[1], listed);
                if (by_k) {
                    target = by_p ? share_of(listed, fmaxf(p, 0.0f), true) : listed;
                    if (target < 1) target = 1;
                }
                const bool keep0 = w[0] && above + pre < target && (uint32_t)(e[0] >> 32) >= floor_;
                const bool keep1 = w[1] && above + pre + w[0] < target && (uint32_t)(e[1] >> 32) >= floor_;
                const int kept = __syncthreads_count(keep0) + __syncthreads_count(keep1);   // the first so many
                if (how == WIDE) {
                    // each of them adds to its warp's sum
                    if (keep0) atomicAdd(&S.sums()[(0xFFFFFFFFu - (uint32_t)e[0]) / A.seg], w[0]);
                    if (keep1) atomicAdd(&S.sums()[(0xFFFFFFFFu - (uint32_t)e[1]) / A.seg], w[1]);
                    __syncthreads();
                    border = hi + 1;                           // none of them: those above alone
                    if (kept) {
                        const u64 end = sm.sorted[kept - 1];
                        border = (uint32_t)(end >> 32);
                        last = (int)(0xFFFFFFFFu - (uint32_t)end);
                    }
                    S.finish(logit_of(border), last);
                } else if (S.rank == 0) {
                    // in the order of the indices: the index's complement first, downwards
                    e[0] = keep0 ? e[0] << 32 | e[0] >> 32 : 0;
                    e[1] = keep1 ? e[1] << 32 | e[1] >> 32 : 0;
                    const uint32_t step = (uint32_t)(A.p.n - 1) / BUCKETS + 1;
                    S.order(kept, e, [&](u64 v) { return (int)((0xFFFFFFFFu - (uint32_t)(v >> 32)) / step); });
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int i = 2 * threadIdx.x + j;
                        e[j] = i < kept ? sm.sorted[i] : 0;
                        w[j] = i < kept ? S.weight(logit_of((uint32_t)e[j])) : 0;
                    }
                    u64 all, up = S.block_scan(w[0] + w[1], all);
                    const u64 at = S.target_of(all);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (at >= up && at < up + w[j]) S.put((int)(0xFFFFFFFFu - (uint32_t)(e[j] >> 32)), S.chance(logit_of((uint32_t)e[j]), all));
                        up += w[j];
                    }
                }
                break;
            }
            if (how == AGAIN) {
                Sampler::Border B = {S.up_to(BINS) + 1, 0, 0};   // the lowest key with a weight
                bool cut = false;
                if (by_k && live > (uint32_t)k) {
                    B = S.select(false, k, B.key, 0);
                    cut = true;
                }
                if (by_p) {
                    u64 all = S.total(logit_of(B.key));
                    if (cut) all -= (B.of - B.ties) * S.weight(logit_of(B.key));
                    u64 reach = share_of(all, fmaxf(p, 0.0f), true);
                    if (reach < 1) reach = 1;
                    B = S.select(true, reach, B.key, cut ? B.of - B.ties : 0);
                    cut = true;
                }
                if (cut && B.key >= floor_) {
                    border = B.key;
                    last = S.tie_at(logit_of(border), B.ties - 1);
                }
                how = DONE;
            }
        }
        if (how == DONE) {
            const float edge = logit_of(border);
            const u64 v = last == 0x7FFFFFFF ? S.weights([&](float x, int) { return x >= edge; })
                                             : S.weights([&](float x, int i) { return x > edge || (x == edge && i <= last); });
            S.tell(warp_sum64(v));
            S.finish(edge, last);
        }
        if (S.cs > 1 && (by_k || by_p)) S.together();   // no CTA leaves while its list is read
    }
}

}  // namespace

cudaError_t launch_sample(const plm_sample_problem& p, cudaStream_t stream) {
    SampleArgs A = {};
    A.p = p;
    A.four = four_aligned(p.logits, p.m > 1 ? p.stride : 0, p.type);
    const int sms = num_sms();
    // Two CTAs an SM, 8 a row at most: what of a row does not fit half the SM's shared
    // memory is left in L2.  256 rows of 200064 take 152 us so, top-k 182, and 241 and 322
    // with all of the row in one CTA of 32 warps an SM.  Few rows are spread further, over
    // CTAs with 4096 logits: 64 of 32000 with top-p 26 us, and 33 while only half as many
    // CTAs were made; with 2048 or 8192 logits a CTA one row of 32000 takes 6.7 and 7.1
    // (4096: 6.7), 16 of them 8.4 and 7.9 (8.3).
    int cs = 1;
    constexpr int HALF = 113 * 1024, WHOLE = 227 * 1024;   // bytes of a CTA
    const auto room = [&](int bytes) { return bytes - (int)fixed_bytes(cs * NW); };   // for its part of the row
    while (cs < MOST_CS && p.n * 4 > (long long)cs * room(HALF)) cs *= 2;
    while (cs < MOST_CS && p.n > 4096LL * cs && p.m * cs <= sms) cs *= 2;
    A.seg = (int)((p.n + 128LL * cs * NW - 1) / (128LL * cs * NW)) * 128;
    const int most = room(p.m * cs <= sms ? WHOLE : HALF) / (4 * NW) / 128 * 128;
    A.held = A.seg < most ? A.seg : most;
    const size_t bytes = fixed_bytes(cs * NW) + 4 * (size_t)A.held * NW;
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)p.m, 1, (unsigned)cs);
    if (cs == 1) return launch_kernel(sample_kernel, grid, dim3(NT), bytes, stream, A);
    return launch_kernel_cluster(sample_kernel, grid, dim3(NT), bytes, stream, (unsigned)cs, A);
}

}  // namespace plm

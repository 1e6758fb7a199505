// The next token of each row of logits (plm_sample): temperature, top-k, top-p
// and min-p from one given random number a row.
//
// Mathematics.  w = 2^-t, t = (max - x) log2(e) / T, in fixed point: 2^40 for the
// largest logit, nothing from t = 40 on.  t is formed in pairs of f32; 2^-t by a
// table of 2^(-i/64) and the series of the rest (a table-driven exponential as
// in P. T. P. Tang, ACM TOMS 15, 1989), to 2^-30 of itself.  Sums of whole
// numbers do not depend on their order, so which token is met does not depend
// on the launch.
//   A border (the k-th largest logit; the one at which the sum of the w's in
// descending order reaches p of all) is found without sorting: a histogram of
// how many logits lie in each of 2048 bins of t; what the w's of a bin add up to
// is bounded by its edges, so the border lies in one bin or a few; these are cut
// again, by the logits' bits now, until a bin is a single value.  The sum of what
// lies above the bins in question is formed exactly on each level.
//
// Layout.  A cluster of CTAs takes a row, each a piece of it in shared memory as
// integers that order as the logits do; so the row is read once.  What does not
// fit is read again from L2.
#include "plm_device.cuh"
#include "plm_internal.h"
#include "values.cuh"

namespace plm {

namespace {

using u64 = unsigned long long;

constexpr int ST = 512, SW = ST / 32;        // threads, warps per CTA
constexpr int BINS = 2048, PER = BINS / ST;  // of the histogram; of a thread
constexpr int MOST_CS = 8;                   // CTAs of a row at most
constexpr float SPAN = 40.0f;                // t from which on a logit has no weight
constexpr uint32_t LOWEST = 0x007FFFFFu;     // the key of -inf

struct SampleArgs {
    plm_sample_problem p;
    int slice, held;                         // logits of a CTA, of which in shared memory
};

// Logits as integers in their order; NaN is -inf, -0 is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return x != x ? LOWEST : b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

struct Exchange {           // what the CTAs of a row tell each other
    u64 sum[2][SW], top[2][SW];
};

struct SampleSmem {
    u64 table[64];          // 2^(40 - i/64)
    u64 scan[2][SW + 1];
    Exchange ex[2];         // in turn
    uint32_t hist[3][BINS];   // in turn: one is filled, one may still be read by others, one is emptied
    uint32_t found[8];
    u64 found_sum[4];
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
__device__ __forceinline__ uint32_t peer32(const uint32_t* p, int z) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at_peer(p, z)) : "memory");
    return v;
}

// A row as one CTA of its cluster sees it.
struct Sampler {
    const SampleArgs& A;
    SampleSmem& sm;
    const uint32_t* keys;       // of this CTA's logits, the first `held`
    long long row;
    int lane, warp, cs, rank, first, len, turn;   // turn: of sm.ex
    uint32_t kmax;
    float half_max, c_hi, c_lo, per_t;
    bool infinite;

    __device__ uint32_t key(int i) const {
        if (i < A.held) return keys[i];
        return key_of(value_at(A.p.logits, A.p.type, row * A.p.stride + first + i));
    }
    __device__ void together() const {
        __syncwarp();
        if (cs > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else __syncthreads();
    }

    // t of a logit: high part, and what is missing to it
    __device__ __forceinline__ float t_of(uint32_t k) const {
        return fmaf(logit_of(k), -0.5f, half_max) * c_hi;
    }
    // whether the logit has a weight
    __device__ __forceinline__ bool live(uint32_t k) const { return infinite ? k == kmax : k > LOWEST && t_of(k) < SPAN; }
    __device__ __forceinline__ u64 weight_t(float t, float rest) const {
        const float f = rintf(t * 64.0f);
        const int i = (int)f;
        const float r = (fmaf(f, -0.015625f, t) + rest) * -0.693147180559945f;   // 2^-(t - i/64) = e^r
        const float e = r * fmaf(r, fmaf(r, fmaf(r, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f), 1.0f);
        const u64 v = sm.table[i & 63];
        // v e in units of 2^8 (v up to 2^40, e up to 0.006)
        const int more = __float2int_rn((float)(uint32_t)(v >> 16) * 256.0f * e);
        return (u64)((long long)v + (long long)more * 256) >> (i >> 6);
    }
    __device__ __forceinline__ u64 weight(uint32_t k) const {   // of one that is live
        if (infinite) return 1ull << 40;
        const float x = logit_of(k), b = 0.5f * x, d = fmaf(x, -0.5f, half_max);
        const float bb = half_max - d, low = (half_max - (d + bb)) + (bb - b);   // (max - x) / 2 = d + low
        const float t = d * c_hi;
        return weight_t(t, fmaf(d, c_hi, -t) + fmaf(low, c_hi, d * c_lo));
    }
    __device__ __forceinline__ int bin_t(uint32_t k) const { return (int)(t_of(k) * per_t); }   // not increasing in k

    // Sums of v (and maxima of w) over the row.  The sums of the CTAs before this one: *before.
    __device__ u64 sum_all(u64 v, u64* before = nullptr) {
        Exchange& ex = sm.ex[turn & 1];
        ++turn;
        v = warp_sum64(v);
        if (lane == 0) ex.sum[0][warp] = v;
        together();
        u64 all = 0, pre = 0;
        for (int z = 0; z < cs; ++z) {
            u64 s = lane < SW ? (cs > 1 ? peer64(&ex.sum[0][lane], z) : ex.sum[0][lane]) : 0;
            s = warp_sum64(s);
            all += s;
            if (z < rank) pre += s;
        }
        if (before) *before = pre;
        return all;
    }
    __device__ u64 max_all(u64 v) {
        Exchange& ex = sm.ex[turn & 1];
        ++turn;
        v = warp_max64(v);
        if (lane == 0) ex.top[0][warp] = v;
        together();
        u64 all = 0;
        for (int z = 0; z < cs; ++z) {
            const u64 s = lane < SW ? (cs > 1 ? peer64(&ex.top[0][lane], z) : ex.top[0][lane]) : 0;
            all = s > all ? s : all;
        }
        return warp_max64(all);
    }

    // The largest (up) or smallest key in [lo, hi] whose bin is >= b (<= b): the
    // bins fall as the keys rise.
    __device__ uint32_t edge(int b, uint32_t lo, uint32_t hi, bool up) const {
        while (lo < hi) {
            const uint32_t mid = up ? lo + (hi - lo + 1) / 2 : lo + (hi - lo) / 2;
            const int at = bin_t(mid);
            if (up) {
                if (at >= b) lo = mid;
                else hi = mid - 1;
            } else {
                if (at <= b) hi = mid;
                else lo = mid + 1;
            }
        }
        return lo;
    }

    struct Border { uint32_t key; uint32_t ties, of; u64 above; };   // ties kept of `of`; what lies above

    // The border of the row at which the count (mass = false) or the w's sum of
    // the logits in descending order reaches `target` >= 1 (which they do).  Below
    // `floor_` nothing counts, and of the logits equal to it `missing` do not.
    __device__ Border select(bool mass, u64 target, uint32_t floor_, uint32_t missing, int& buffer) {
        uint32_t hi = kmax, lo = floor_;
        bool by_t = !infinite;
        u64 above = 0;
        for (;;) {
            int shift = 0;
            while (((hi - lo) >> shift) >= (uint32_t)BINS) ++shift;
            uint32_t* h = sm.hist[buffer];
            buffer = buffer == 2 ? 0 : buffer + 1;
            uint32_t* next = sm.hist[buffer];
            auto bin = [&](uint32_t k) { return by_t ? min(bin_t(k), BINS - 1) : (int)((hi - k) >> shift); };
            // (h is empty: it was emptied a level ago)
            u64 mine = 0;
            for (int i = threadIdx.x; i < len; i += ST) {
                const uint32_t k = key(i);
                if (k > hi) mine += mass ? weight(k) : 1;
                else if (k >= lo) atomicAdd(&h[bin(k)], 1u);
            }
            for (int i = threadIdx.x; i < BINS; i += ST) next[i] = 0;
            above = sum_all(mine);
            // a thread's bins: how many, and the bounds of their sums
            uint32_t n[PER];
            u64 most[PER], least[PER], up = 0, down = 0;
            const int b0 = threadIdx.x * PER;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int b = b0 + j;
                uint32_t c = h[b];
                if (cs > 1) {
                    c = 0;
                    for (int z = 0; z < cs; ++z) c += peer32(&h[b], z);
                }
                if (missing && b == bin(lo) && lo == floor_) c -= missing;
                n[j] = c;
                most[j] = least[j] = c;
                if (mass && c) {
                    u64 w1, w0;
                    if (by_t) {   // by the bin's edges, and what rounding may add
                        const float t1 = (float)b / per_t, t0 = (float)(b + 1) / per_t;
                        w1 = weight_t(fmaxf(t1 - 1e-4f, 0.0f), 0.0f) + 1;
                        w0 = weight_t(fminf(t0 + 1e-4f, SPAN), 0.0f);
                    } else {
                        const uint32_t k1 = hi - ((uint32_t)b << shift), left = k1 - lo, k0 = left >> shift ? k1 - (1u << shift) + 1 : lo;
                        w1 = weight(k1);
                        w0 = k0 == k1 ? w1 : weight(k0);
                        if (k0 != k1) {   // w is right to 2^-30, and may fall by that where it should rise
                            w1 += (w1 >> 28) + 1;
                            w0 -= w0 >> 28;
                        }
                    }
                    most[j] = c * w1;
                    least[j] = c * w0;
                }
                up += most[j];
                down += least[j];
            }
            const u64 up_in = warp_scan64(up, lane), down_in = warp_scan64(down, lane);
            if (lane == 31) { sm.scan[0][warp] = up_in; sm.scan[1][warp] = down_in; }
            if (threadIdx.x == 0) { sm.found[0] = BINS; sm.found[1] = BINS; sm.found[4] = 0; }
            __syncthreads();
            u64 up_at = above + up_in - up, down_at = above + down_in - down;
            for (int w = 0; w < warp; ++w) { up_at += sm.scan[0][w]; down_at += sm.scan[1][w]; }
            // the first bin whose upper bound reaches the target, the first whose lower bound does
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int b = b0 + j;
                if (n[j]) {
                    if (up_at < target && up_at + most[j] >= target) {
                        sm.found[0] = b;
                        sm.found[2] = n[j];
                        sm.found_sum[0] = up_at;
                    }
                    if (down_at < target && down_at + least[j] >= target) sm.found[1] = b;
                    atomicMax(&sm.found[4], (uint32_t)b);
                }
                up_at += most[j];
                down_at += least[j];
            }
            __syncthreads();
            const int last = (int)sm.found[4];
            const int b1 = min((int)sm.found[0], last), b2 = min((int)sm.found[1], last);
            const uint32_t count = sm.found[2];
            const u64 before = sm.found_sum[0];
            __syncthreads();
            if (!by_t && shift == 0) {
                Border B;
                B.key = hi - b1;
                B.of = count;
                B.above = before;
                const u64 w = mass ? weight(B.key) : 1;
                const u64 need = target > before ? (target - before + w - 1) / (w ? w : 1) : 1;
                B.ties = (uint32_t)(need < 1 ? 1 : need > count ? count : need);
                return B;
            }
            const uint32_t wide = hi - lo;
            if (by_t) {
                if (threadIdx.x < 2) sm.found[5 + threadIdx.x] = threadIdx.x == 0 ? edge(b1, lo, hi, true) : (b2 >= BINS - 1 ? lo : edge(b2, lo, hi, false));
                __syncthreads();
                hi = sm.found[5];
                lo = sm.found[6];
                by_t = false;
                continue;
            } else {
                const uint32_t top = hi - ((uint32_t)b1 << shift), k2 = hi - ((uint32_t)b2 << shift);
                lo = (k2 - lo) >> shift ? k2 - (1u << shift) + 1 : lo;
                hi = top;
            }
            if (hi - lo > wide / 4) {   // bounds that tell the bins apart badly: halve what is left
                const uint32_t mid = lo + (hi - lo) / 2;
                u64 v = 0;
                for (int i = threadIdx.x; i < len; i += ST) {
                    const uint32_t k = key(i);
                    if (k > mid) v += mass ? weight(k) : 1;
                }
                if (sum_all(v) >= target) lo = mid + 1;
                else hi = mid;
            }
        }
    }

    // The first index at which the sum of f over the indices exceeds target(sum of
    // all), which is less than that; -1 where another warp has it.  f: key, index.
    template <class F, class G> __device__ int pick(F f, G target_of, u64* all) {
        const int seg = (len + SW - 1) / SW, i0 = warp * seg, i1 = min(i0 + seg, len);
        u64 mine = 0;
        for (int i = i0 + lane; i < i1; i += 32) mine += f(key(i), i);
        mine = warp_sum64(mine);
        u64 pre;
        *all = sum_all(lane == 0 ? mine : 0, &pre);
        const u64 target = target_of(*all);
        if (lane == 0) sm.scan[0][warp] = mine;
        __syncthreads();
        for (int w = 0; w < warp; ++w) pre += sm.scan[0][w];
        __syncthreads();
        if (target < pre || target >= pre + mine) return -1;
        for (int i = i0; i < i1; i += 32) {
            const u64 v = i + lane < i1 ? f(key(i + lane), i + lane) : 0, in = warp_scan64(v, lane);
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, pre + in > target);
            if (hit) return i + __ffs(hit) - 1;
            pre += __shfl_sync(0xFFFFFFFFu, in, 31);
        }
        return -1;
    }

    __device__ void put(int token, float prob) const {
        A.p.tokens[row] = token;
        if (A.p.prob) A.p.prob[row] = prob;
    }
};

// CTA (row, , rank in the row's cluster).
__global__ void __launch_bounds__(ST) sample_kernel(const __grid_constant__ SampleArgs A) {
    extern __shared__ __align__(16) uint8_t sample_raw[];
    SampleSmem& sm = *reinterpret_cast<SampleSmem*>(sample_raw);
    uint32_t* keys = reinterpret_cast<uint32_t*>(sample_raw + sizeof(SampleSmem));
    grid_launch_dependents();
    if (threadIdx.x < 64) sm.table[threadIdx.x] = (u64)llrint(exp2(40.0 - threadIdx.x / 64.0));
    for (int i = threadIdx.x; i < 3 * BINS; i += ST) (&sm.hist[0][0])[i] = 0;
    grid_wait_prior();
    Sampler S{A, sm, keys};
    S.row = blockIdx.x;
    S.lane = threadIdx.x & 31;
    S.warp = threadIdx.x >> 5;
    S.cs = gridDim.z;
    S.rank = blockIdx.z;
    S.first = S.rank * A.slice;
    S.len = max(0, min(A.slice, (int)A.p.n - S.first));
    S.turn = 0;
    // the row's largest logit, the lowest index of it
    u64 best = 0;
    for (int i = threadIdx.x; i < S.len; i += ST) {
        const uint32_t k = key_of(value_at(A.p.logits, A.p.type, S.row * A.p.stride + S.first + i));
        if (i < A.held) keys[i] = k;
        const u64 v = (u64)k << 32 | (0xFFFFFFFFu - (uint32_t)(S.first + i));
        best = v > best ? v : best;
    }
    best = S.max_all(best);
    S.kmax = (uint32_t)(best >> 32);
    const bool leader = S.rank == 0 && threadIdx.x == 0;
    const float T = A.p.temperature ? A.p.temperature[S.row] : 1.0f;
    if (S.kmax <= LOWEST) {
        if (leader) S.put(-1, 0.0f);
    } else if (!(T > 0.0f) || !A.p.u) {
        if (leader) S.put((int)(0xFFFFFFFFu - (uint32_t)best), 1.0f);
    } else {
        const float top = logit_of(S.kmax);
        S.infinite = isinf(top);
        // t = (max - x) / 2 * (2 log2(e) / T)
        const double c = 2.0 * 1.4426950408889634 / (double)T;
        S.c_hi = c < 3e38 ? (float)c : 3e38f;
        S.c_lo = c < 3e38 ? (float)(c - (double)S.c_hi) : 0.0f;
        S.half_max = 0.5f * top;
        S.per_t = BINS / SPAN;
        // the lowest key with a weight
        uint32_t floor_ = S.kmax;
        if (!S.infinite) {
            uint32_t lo = LOWEST + 1, hi = S.kmax;
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2;
                if (S.live(mid)) hi = mid;
                else lo = mid + 1;
            }
            floor_ = lo;
        }
        const int k = A.p.top_k ? A.p.top_k[S.row] : 0;
        const float p = A.p.top_p ? A.p.top_p[S.row] : 1.0f, low = A.p.min_p ? A.p.min_p[S.row] : 0.0f;
        int buffer = 0;
        Sampler::Border B = {floor_, 0, 0, 0};
        bool all_ties = true;
        auto total = [&](uint32_t from, u64* count) {   // the w's sum, and how many, of the keys >= from
            u64 v = 0, n = 0;
            for (int i = threadIdx.x; i < S.len; i += ST) {
                const uint32_t x = S.key(i);
                if (x >= from) {
                    v += S.weight(x);
                    ++n;
                }
            }
            if (count) *count = S.sum_all(n);
            return S.sum_all(v);
        };
        u64 sum = 0;
        bool summed = false;
        if (k > 0 && k < A.p.n) {
            u64 count;
            sum = total(floor_, &count);
            summed = true;
            if (count > (u64)k) {
                B = S.select(false, k, floor_, 0, buffer);
                all_ties = B.ties == B.of;
                summed = false;
            }
        }
        if (p < 1.0f) {
            if (!summed) {
                sum = total(B.key, nullptr);
                if (!all_ties) sum -= (B.of - B.ties) * S.weight(B.key);
            }
            const double want = ceil((double)fmaxf(p, 0.0f) * (double)sum);
            u64 target = want < 1.0 ? 1 : (u64)want;
            if (target > sum) target = sum;
            B = S.select(true, target, B.key, all_ties ? 0 : B.of - B.ties, buffer);
            all_ties = false;   // (of may count ties that top_k has left out)
        }
        int last_tie = 0x7FFFFFFF;   // the index of the last tie that is kept
        if (low > 0.0f) {
            // the smallest f32 that is at least max + T ln(min_p)
            const double at = S.infinite ? 0.0 : (double)top + (double)T * log((double)fminf(low, 1.0f));
            const uint32_t kl = S.infinite ? S.kmax : min(key_of(__double2float_ru(at)), S.kmax);
            if (kl > B.key) {
                B.key = kl;
                all_ties = true;
            }
        }
        if (!all_ties) {
            const uint32_t border = B.key;
            const u64 before = B.ties - 1;
            u64 ties;
            const int at = S.pick([&](uint32_t x, int) -> u64 { return x == border; }, [&](u64) { return before; }, &ties);
            last_tie = (int)(0xFFFFFFFFu - (uint32_t)S.max_all(at < 0 ? 0 : 0xFFFFFFFFu - (uint32_t)(S.first + at)));
        }
        const uint32_t border = B.key;
        auto kept = [&](uint32_t x, int i) -> u64 {
            return x > border || (x == border && S.first + i <= last_tie) ? S.weight(x) : 0;
        };
        const double u = fminf(fmaxf(A.p.u[S.row], 0.0f), 1.0f);
        const int at = S.pick(kept, [&](u64 all) {
            const u64 part = (u64)floor(u * (double)all);
            return part < all ? part : all - 1;
        }, &sum);
        if (at >= 0 && S.lane == 0) S.put(S.first + at, (float)((double)S.weight(S.key(at)) / (double)sum));
    }
    if (S.cs > 1) S.together();   // no CTA leaves while its shared memory is read
}

}  // namespace

cudaError_t launch_sample(const plm_sample_problem& p, cudaStream_t stream) {
    SampleArgs A = {};
    A.p = p;
    const int most_held = (200 * 1024 - (int)sizeof(SampleSmem)) / 4;
    int cs = 1;
    const int sms = num_sms();
    while (cs < MOST_CS && p.n > 4096 * cs && (p.m * cs * 2 <= 2 * sms || (p.n + cs - 1) / cs > most_held / 2)) cs *= 2;
    A.slice = (int)((p.n + cs - 1) / cs);
    A.held = A.slice < most_held ? A.slice : most_held;
    const size_t bytes = sizeof(SampleSmem) + 4 * (size_t)A.held;
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(200 * 1024));
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)p.m, 1, (unsigned)cs);
    if (cs == 1) return launch_kernel(sample_kernel, grid, dim3(ST), bytes, stream, A);
    return launch_kernel_cluster(sample_kernel, grid, dim3(ST), bytes, stream, (unsigned)cs, A);
}

}  // namespace plm

// Attention over 8-bit pages (plm_attn_kv8): which kernels a call runs.
//
// Few rows per sequence and head: the rows kernel, which turns codes into
// values as it takes them from shared memory.  A prefix that is done apart, and
// more rows, go through the tile kernel, whose operands come by TMA as they
// are: their pages are read back into the workspace first, as 16-bit pages of
// 128 tokens (once for all row tiles, and a shared prefix once for the batch).
#include "attn_tile.cuh"

namespace plm {

namespace {

constexpr int PT = 128;   // tokens of a page in the workspace

// The workspace's pages: `shared` of the prefix, then `each` a sequence.
struct Back {
    uint16_t* k;
    uint16_t* v;
    int* table;      // [batch][each], or the prefix's alone
    int* lens;       // [batch]
    int shared, each, own;   // own: sequences have pages besides
    size_t bytes;
};

// Reads pages back.  A CTA a page of the workspace and head.
template <class E, int D>
__global__ void __launch_bounds__(256) kv8_pages_kernel(const __grid_constant__ AttnArgs8 A, const __grid_constant__ Back W) {
    __shared__ int first;
    grid_launch_dependents();
    grid_wait_prior();
    const int at_page = (int)(blockIdx.x / (unsigned)A.kv_heads), h = (int)(blockIdx.x - (unsigned)at_page * A.kv_heads);
    int b, j;                             // sequence, page of it
    const bool common = at_page < W.shared;
    if (common) {   // of the first sequence that sees all of the prefix
        j = at_page;
        if (threadIdx.x == 0) first = A.batch;
        __syncthreads();
        for (int i = threadIdx.x; i < A.batch; i += 256)
            if (attn_len(A, attn_row(A, i)) - A.nq + 1 >= A.prefix) {
                atomicMin(&first, i);
                break;
            }
        __syncthreads();
        b = first;
        if (threadIdx.x == 0 && h == 0 && !W.own) W.table[j] = j;
        if (b == A.batch) return;         // nobody reads it
    } else {
        b = (at_page - W.shared) / W.each;
        j = at_page - W.shared - b * W.each;
    }
    const int row = attn_row(A, b), len = attn_len(A, row), end = common ? A.prefix : len;
    if (!common) {
        const bool shares = j < W.shared && len - A.nq + 1 >= A.prefix;
        if (threadIdx.x == 0 && h == 0) {
            W.table[(long long)b * W.each + j] = shares ? j : at_page;
            if (j == 0) W.lens[b] = len;
        }
        if (shares) return;
    }
    if (j * PT >= end) return;
    const int* tab = A.table + (long long)row * A.table_stride;
    constexpr int CH = D / 16;            // 16 codes a thread
    const int mask = (1 << A.page_shift) - 1;
    const long long to = (long long)blockIdx.x * PT * D;
#pragma unroll 2
    for (int u = threadIdx.x; u < 2 * PT * CH; u += 256) {
        const bool value = u >= PT * CH;
        const int i = value ? u - PT * CH : u, t = i / CH, c = i - t * CH, tok = j * PT + t;
        uint4 x = make_uint4(0, 0, 0, 0);
        uint32_t e = 0;
        const int page = tok < end ? tab[tok >> A.page_shift] : -1;
        if (page >= 0 && page < A.pages) {
            const int at = tok & mask;
            const int8_t* codes = static_cast<const int8_t*>(value ? A.v : A.k) + page * A.page_stride + h * A.kv_hs + at * A.kv_ts + 16 * c;
            x = *reinterpret_cast<const uint4*>(codes);
            e = (value ? A.v_exps : A.k_exps)[page * A.exp_page + h * A.exp_hs + at * (D / 32) + (c >> 1)];
        }
        const uint32_t f = exps_to_pair<E>(e, e), w[4] = {x.x, x.y, x.z, x.w};
        uint32_t r[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            codes_to_pairs<E>(w[k], r[2 * k], r[2 * k + 1]);
            r[2 * k] = finite_pair<E>(mul_pairs<E>(r[2 * k], f));
            r[2 * k + 1] = finite_pair<E>(mul_pairs<E>(r[2 * k + 1], f));
        }
        uint4* out = reinterpret_cast<uint4*>((value ? W.v : W.k) + to + (long long)t * D + 16 * c);
        out[0] = make_uint4(r[0], r[1], r[2], r[3]);
        out[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

template <class E, int D> cudaError_t pages_launch(const AttnArgs8& A, const Back& W, cudaStream_t stream) {
    const long long pages = W.shared + (W.own ? (long long)A.batch * W.each : 0);
    return launch_kernel(kv8_pages_kernel<E, D>, dim3((unsigned)(pages * A.kv_heads)), dim3(256), 0, stream, A, W);
}
cudaError_t launch_pages(const AttnArgs8& A, const Back& W, int type, int d, cudaStream_t stream) {
    if (type == PLM_F16) return d == 64 ? pages_launch<__half, 64>(A, W, stream) : pages_launch<__half, 128>(A, W, stream);
    return d == 64 ? pages_launch<__nv_bfloat16, 64>(A, W, stream) : pages_launch<__nv_bfloat16, 128>(A, W, stream);
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// The pages of the prefix (own: of whole sequences, what is shared once) in a workspace.
Back back_plan(const AttnArgs& A, int d, bool own, long long bound, uint8_t* ws) {
    Back W = {};
    W.own = own;
    // of a prefix read by every sequence whole pages are shared, for the tables' sake
    W.shared = own ? (A.batch > 1 ? A.prefix / PT : 0) : (A.prefix + PT - 1) / PT;
    W.each = (int)((bound + PT - 1) / PT);
    const long long pages = W.shared + (own ? (long long)A.batch * W.each : 0);
    if (pages > 0x7FFFFFFFLL / A.kv_heads) {   // (a CTA each)
        W.bytes = SIZE_MAX;
        return W;
    }
    const size_t part = up256((size_t)pages * A.kv_heads * PT * d * 2);
    const size_t table = up256(4 * (own ? (size_t)A.batch * W.each : (size_t)W.shared)), lens = own ? up256(4 * (size_t)A.batch) : 0;
    W.bytes = 2 * part + table + lens;
    if (!ws) return W;
    W.k = reinterpret_cast<uint16_t*>(ws);
    W.v = reinterpret_cast<uint16_t*>(ws + part);
    W.table = reinterpret_cast<int*>(ws + 2 * part);
    W.lens = reinterpret_cast<int*>(ws + 2 * part + table);
    return W;
}

// The problem over the workspace's pages.
AttnArgs over(const AttnArgs8& A8, const Back& W, int d) {
    AttnArgs A = A8;
    A.k = W.k;
    A.v = W.v;
    A.table = W.table;
    A.kv_ts = d;
    A.kv_hs = (long long)PT * d;
    A.page_stride = A.kv_hs * A.kv_heads;
    A.page_shift = 7;
    if (W.own) {
        A.pages = W.shared + A.batch * W.each;
        A.table_stride = W.each;
        A.lens = W.lens;
        A.seqs = nullptr;
        A.rows = A.batch;
        A.prefix = 0;
    } else {
        A.pages = W.shared;
        A.table_stride = 0;   // the same for all rows
    }
    return A;
}

struct Choice8 {
    bool rows, share;
    TilePlan plan;     // of the prefix apart (share), or of all keys (not rows)
    Back back;
    size_t bytes;
};

// bound: what the lengths are bounded by (A.cap may be less).
Choice8 choose8(const AttnArgs& A, int d, long long bound, void* ws) {
    const long long mine = (long long)A.nq * A.group;
    Choice8 c = {};
    // Beyond 32 rows the rows kernel goes over the keys again for each chunk of 32; the tile
    // kernel needs them read back first.  One GB300, 24 sequences, 8 heads of 128, us here and
    // there: 40 rows over 500 keys 21 and 59, over 4000 79 and 152; 64 over 500 34 and 60, 3000
    // 111 and 128, 12000 378 and 312 (2 sequences, 4000: 24 and 38); 96 over 400 44 and 53, 1000
    // 67 and 77, 3000 153 and 137.
    c.rows = mine <= 48 || (mine <= 64 && bound <= 5120) || (mine <= 96 && bound <= 2048);
    if (c.rows) {
        // The prefix apart costs two launches, a trip of every row's O through memory, and
        // reading it back.  It saves what every other sequence would read of it (~35 keys and
        // heads a ns; more than 16 rows take twice as long), or the blocks that a warp of a full
        // cluster goes through.  One GB300, us unshared and shared, a token each on 8 heads of
        // 128: 16 behind 1024 14 and 26, 64 behind 512 23 and 29, behind 1024 34 and 34, 128 58
        // and 47, behind 2048 96 and 51, 24 behind 4096 54 and 33, 2 behind 16384 34 and 51; 61
        // on 2 heads of 64 behind 8176 39 and 30; 2 x 28 rows behind 8192 57 and 47, 4 behind
        // 16384 80 and 60, 12 behind 2048 (not taken apart) 52 and 48, 48 x 20 behind 8192 255 and 84.
        const double others = (A.batch - 1.0) * A.prefix * A.kv_heads * ((mine + 31) / 32) * (mine > 16 ? 2.2 : 1.0) / 35e3;
        const double chain = A.prefix / 512.0 * (mine > 16 ? 1.4 : 0.7), back = 6.0 * A.prefix * A.kv_heads * d / 5.5e6;
        c.share = A.prefix > 0 && A.batch > 1 && (others > chain ? others : chain) > 13.0 + back;
        if (!c.share) return c;
    }
    size_t plan = 0;
    AttnArgs T = A;
    if (!c.rows) T.prefix = 0;
    c.plan = tile_plan(T, d, c.rows ? 0 : 1, c.rows, ws, &plan);
    if (plan == SIZE_MAX) { c.bytes = plan; return c; }
    c.back = back_plan(A, d, !c.rows, bound, ws ? static_cast<uint8_t*>(ws) + plan : nullptr);
    c.bytes = c.back.bytes == SIZE_MAX ? SIZE_MAX : plan + c.back.bytes;
    return c;
}

}  // namespace

size_t attn_kv8_workspace_bytes(long long batch, long long tokens, long long heads, long long kv_heads, long long head_dim,
                                long long prefix_len, long long max_len) {
    AttnArgs A = {};
    A.batch = (int)batch; A.nq = (int)tokens; A.heads = (int)heads; A.kv_heads = (int)kv_heads;
    A.group = A.heads / A.kv_heads;
    A.prefix = (int)prefix_len;
    A.cap = (int)max_len;
    return choose8(A, (int)head_dim, max_len, nullptr).bytes;
}

cudaError_t launch_attn_kv8(const plm_attn_kv8_problem& p, void* ws, cudaStream_t stream) {
    AttnArgs8 A = {};
    A.q = p.q; A.o = p.o; A.lse = p.lse; A.k = p.k; A.v = p.v; A.k_exps = p.k_exps; A.v_exps = p.v_exps;
    A.table = p.table; A.lens = p.lens; A.seqs = p.seqs;
    A.batch = (int)p.batch; A.nq = (int)p.tokens; A.heads = (int)p.heads; A.kv_heads = (int)p.kv_heads;
    A.group = A.heads / A.kv_heads;
    A.group_inv = (65536u + A.group - 1) / A.group;
    A.q_ts = p.q_token_stride; A.q_hs = p.q_head_stride; A.o_ts = p.o_token_stride; A.o_hs = p.o_head_stride;
    A.page_stride = p.page_stride; A.kv_hs = p.kv_head_stride; A.kv_ts = p.kv_token_stride;
    A.exp_page = p.exp_page_stride; A.exp_hs = p.exp_head_stride;
    A.table_stride = p.table_stride;
    while ((1LL << A.page_shift) < p.page_tokens) ++A.page_shift;
    A.pages = (int)p.pages; A.rows = (int)p.rows;
    A.prefix = (int)p.prefix_len;
    const long long room = p.table_stride * p.page_tokens;
    A.cap = (int)(p.max_len < room ? p.max_len : room);
    A.scale = p.scale;
    A.o_f32 = p.o_type == PLM_F32;
    const int d = (int)p.head_dim;
    const Choice8 c = choose8(A, d, p.max_len, ws);
    if (c.rows && !c.share) return launch_attn_rows8(A, nullptr, p.type, d, stream);
    cudaError_t e = launch_pages(A, c.back, p.type, d, stream);
    if (e == cudaSuccess) e = launch_attn_tile(over(A, c.back, d), c.plan, p.type, d, stream);
    return e == cudaSuccess && c.rows ? launch_attn_rows8(A, &c.plan, p.type, d, stream) : e;
}

}  // namespace plm

// Attention over a paged cache (plm_attn_shared_prefix): which kernels a call
// runs.
//
// Few rows per sequence and head (decode, drafted tokens: up to 32, up to 96 over
// few keys): attn_rows.cu, a cluster per (sequence, head).  More rows: the tile kernel
// (attn_tile.cu), and a last kernel that adds what was cut.  A shared prefix goes
// either with each sequence's own keys or, where that pays, first and for the whole
// batch through the tile kernel; its results are then added at the end.
#include "attn_tile.cuh"

namespace plm {

namespace {

AttnArgs attn_args(const plm_attn_problem& p) {
    AttnArgs A = {};
    A.q = p.q; A.o = p.o; A.lse = p.lse; A.k = p.k; A.v = p.v;
    A.table = p.table; A.lens = p.lens; A.seqs = p.seqs;
    A.batch = (int)p.batch; A.nq = (int)p.tokens; A.heads = (int)p.heads; A.kv_heads = (int)p.kv_heads;
    A.group = A.heads / A.kv_heads;
    A.group_inv = (65536u + A.group - 1) / A.group;
    A.q_ts = p.q_token_stride; A.q_hs = p.q_head_stride; A.o_ts = p.o_token_stride; A.o_hs = p.o_head_stride;
    A.page_stride = p.page_stride; A.kv_hs = p.kv_head_stride; A.kv_ts = p.kv_token_stride;
    A.table_stride = p.table_stride;
    while ((1LL << A.page_shift) < p.page_tokens) ++A.page_shift;
    A.pages = (int)p.pages; A.rows = (int)p.rows;
    A.prefix = (int)p.prefix_len;
    const long long room = p.table_stride * p.page_tokens;
    A.cap = (int)(p.max_len < room ? p.max_len : room);
    A.scale = p.scale;
    A.o_f32 = p.o_type == PLM_F32;
    return A;
}

// A call's kernels and their plans.
struct Choice {
    bool rows;     // own keys in the rows kernel, else in the tile kernel
    bool share;    // the prefix apart, for the whole batch
    TilePlan prefix, own;
    size_t bytes;  // workspace, SIZE_MAX: too many units
};

// bound: what the lengths are bounded by (A.cap may be less: the table's rows end
// first; the workspace is sized without knowing them).
Choice choose(const AttnArgs& A, int d, long long bound, void* ws) {
    const long long mine = (long long)A.nq * A.group;
    const bool common = A.prefix > 0 && A.batch > 1;
    Choice c = {};
    if (mine <= 96) {
        // The prefix apart costs a launch and longer sums, ~7 us.  Read by every sequence
        // it takes its bytes at ~6 TB/s, or the 16-key blocks that a warp of a full
        // cluster goes through.  One GB300, us unshared and shared: 4 streams behind 1024
        // tokens 9.8 and 11.1, 149 behind 64 16 and 25; 16 behind 1024 15.9 and 11.6, 2
        // behind 8192 22 and 19, 12 x 28 rows behind 3072 59 and 32.
        const double bytes = (A.batch - 1.0) * A.prefix * A.kv_heads * 4 * d * ((mine + 31) / 32);
        const double chain = A.prefix / 512.0 * (mine > 16 ? 1.4 : 0.7);
        c.share = common && (bytes / 6e6 > chain ? bytes / 6e6 : chain) > 7.0;
        // Beyond 32 rows the rows kernel goes over the keys again for each chunk of 32, which
        // pays as long as they are few, and for longer where its CTAs leave room on the GPU;
        // the prefix apart, and its sums, count as 512 keys.  One GB300, 8 heads of 128, us
        // here and in the tile kernel: 24 x 40 rows over 4000 keys 74 and 97, over 16000 254 and
        // 178; 24 x 64 over 2000 74 and 81, over 3000 101 and 81; 60 x 72 over 2000 136 and 137,
        // over 3000 184 and 152; 2 x 64 over 4000 23 and 27, 5 x 72 over 3000 24 and 28; 60 x 80
        // over 1000 154 and 114, 8 x 80 27 and 30, over 3000 56 and 39; 8 x 96 behind 4096 51
        // and 41.  Heads of 64: 24 x 64 over 4000 57 and 71, 24 x 80 over 1000 31 and 40, over
        // 4000 82 and 68, 3 x 80 19 and 22.
        c.rows = true;
        if (mine > 32) {
            const long long keys = c.share ? bound - A.prefix + 512 : bound, pairs = (long long)A.batch * A.kv_heads;
            const long long ctas = (mine + 31) / 32 * pairs, room = attn_rows_room(d, (int)mine);
            const bool half = 2 * ctas <= room, whole = ctas <= room && !c.share;
            const int most = mine <= 48 ? 4096 : mine <= 72 ? (half ? 4096 : 2048) : half && d == 64 ? 3072 : whole ? 1536 : 512;
            // (what the tile kernel cannot count the rows kernel can)
            c.rows = keys <= most * (128 / d) || pairs * ((bound + TK - 1) / TK) > 0x7FFFFFFFLL;
        }
    }
    if (!c.rows) {
        // What it saves: the prefix's units in every sequence's own tiles, less those of the
        // batch's rows together.  A unit of two row tiles takes the whole GPU 8 + d / 32 ns,
        // one of a single tile 0.57 of that.  What it costs: a launch, and two more trips of
        // every row's O through memory.  So it pays where a sequence's rows fill its tiles
        // badly.  One GB300, us unshared and shared; 8 heads of 128: 24 x 140 rows behind 8192
        // 173 and 158, behind 2048 78 and 98; 24 x 180 behind 8192 176 and 180; 24 x 112 97 and
        // 113 (4096); 60 x 128 97 and 182 (2048); 96 x 490 2105 and 2442 (15360), on 2 heads 528
        // and 628; 40 x 130 on 2 103 and 90 (10240); 60 x 100 on 2 204 and 182 (32768); 8 heads
        // of 64, 60 x 140 behind 8192 320 and 255.
        const long long tile = mine > 128 ? 256 : 128, each = (mine + tile - 1) / tile, all = (mine * A.batch + 255) / 256;
        const double unit = 1e-3 * (8 + d / 32.0) * A.kv_heads * A.prefix / TK;
        const double saved = unit * (A.batch * each * (tile == 256 ? 1.0 : 0.57) - all);
        c.share = common && saved > 6.0 + 1.25e-5 * d * A.batch * mine * A.kv_heads;
    }
    size_t a = 0, b = 0;
    if (c.share) c.prefix = tile_plan(A, d, 0, true, ws, &a);
    if (a == SIZE_MAX) { c.bytes = a; return c; }
    if (!c.rows) c.own = tile_plan(A, d, 1, c.share, ws ? static_cast<uint8_t*>(ws) + a : nullptr, &b);
    c.bytes = b == SIZE_MAX ? b : a + b;
    return c;
}

}  // namespace

size_t attn_workspace_bytes(long long batch, long long tokens, long long heads, long long kv_heads, long long head_dim,
                            long long prefix_len, long long max_len) {
    AttnArgs A = {};
    A.batch = (int)batch; A.nq = (int)tokens; A.heads = (int)heads; A.kv_heads = (int)kv_heads;
    A.group = A.heads / A.kv_heads;
    A.prefix = (int)prefix_len;
    A.cap = (int)max_len;
    return choose(A, (int)head_dim, max_len, nullptr).bytes;
}

cudaError_t launch_attn(const plm_attn_problem& p, void* ws, cudaStream_t stream) {
    const AttnArgs A = attn_args(p);
    const int d = (int)p.head_dim;
    const Choice c = choose(A, d, p.max_len, ws);
    if (c.share) {
        const cudaError_t e = launch_attn_tile(A, c.prefix, p.type, d, stream);
        if (e != cudaSuccess) return e;
    }
    if (c.rows) return launch_attn_rows(A, c.share ? &c.prefix : nullptr, p.type, d, stream);
    const cudaError_t e = launch_attn_tile(A, c.own, p.type, d, stream);
    return e == cudaSuccess && c.share ? launch_attn_merge(A, c.prefix, c.own, p.type, d, stream) : e;
}

}  // namespace plm

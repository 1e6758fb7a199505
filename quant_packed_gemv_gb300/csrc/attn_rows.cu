// Paged attention for few query rows over 16-bit pages, and how many CTAs take
// a (sequence, key/value head): the kernel is in attn_rows.cuh.
#include "attn_rows.cuh"

namespace plm {

// CTAs of a pair (at most 8: 32 warps): as many as the GPU holds at once (a second
// wave costs a whole start and end: 12 x 36 rows over up to 812 keys, 28 us where one
// wave takes 24), while every warp still gets two blocks of 16 keys.  Long rows up to 16
// are cut into CTAs of 1024 keys and more whatever their number: the GPU hands them
// out as others end, so that sequences of unequal lengths even out (20 of up to
// 16000 keys, 8 heads of 128: 116 us in one wave, 105 so; 128 of up to 6000: 255 and
// 241; 64 of up to 4000: 84 and 82; 4 tokens each, 3000: 76 and 72).  8-bit pages are
// cut at 3000 keys: 20 of up to 16000 114 and 76 (cut at 4096: 85, at 2048: 76), 128 of
// up to 6000 179 and 158 (158, 168), 64 of up to 4000 81 and 61 (81, 61).
int rows_cluster(const AttnArgs& A, int d, int chunks, int keys, bool kv8) {
    const int rows = A.nq * A.group, cut = rows <= 16 ? (kv8 ? 3000 : 2048) : 0x7FFFFFFF;
    const long long pairs = (long long)A.batch * A.kv_heads * chunks, room = attn_rows_room(d, rows, kv8);
    int cs = 1;
    while (cs < 8 && keys > 2 * 16 * DW * cs && (pairs * cs * 2 <= room || keys / cs > cut)) cs *= 2;
    return cs;
}

// Where an SM holds one CTA (25 to 32 rows of 128), a third more than fit at once
// still pays, as those of short sequences end early, and more does not.  Sequences x
// tokens, 4 query heads each on 8 heads, up to 3000 keys: 12 x 8 as 96 CTAs 45 us, as
// 192 35; 8 x 8 as 128 26, as 256 31; 18 x 8 as 144 46, as 288 49; 4 x 8 over 8000 as
// 128 37, as 256 70; 7 heads on 2, over 2000: 40 x 4 as 80 35, as 160 26; 60 x 4 as
// 120 35, as 240 38.  8-bit pages, the first three: 52 and 35, 30 and 32, 53 and 53.
long long attn_rows_room(int d, int rows, bool kv8) {
    const int chunks = (rows + 31) / 32, ctas = rows_ctas(d, ((rows + chunks - 1) / chunks + 7) / 8, kv8), sms = num_sms();
    return ctas == 1 ? sms + sms / 3 : (long long)ctas * sms;
}

cudaError_t launch_attn_rows(const AttnArgs& A, const TilePlan* plan, int type, int d, cudaStream_t stream) {
    return rows_any(A, plan, type, d, stream);
}

}  // namespace plm

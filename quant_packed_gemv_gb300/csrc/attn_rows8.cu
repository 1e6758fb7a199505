// Paged attention for few query rows over 8-bit pages: the kernel is in
// attn_rows.cuh.
#include "attn_rows.cuh"

namespace plm {

cudaError_t launch_attn_rows8(const AttnArgs8& A, const TilePlan* plan, int type, int d, cudaStream_t stream) {
    return rows_any(A, plan, type, d, stream);
}

}  // namespace plm

// The residual norm with dropout, rows loaded straight into registers (the rows of
// kda_norm_ring.cu are streamed with dropout there).
#include "kda_norm_rows.cuh"

namespace kda {

cudaError_t launch_norm_drop(const NormArgs &a, bool bwd, int size, const Shape &s, cudaStream_t st) {
    return bwd ? launch_op<OP_DROP, true>(a, size, s, st) : launch_op<OP_DROP, false>(a, size, s, st);
}

}  // namespace kda

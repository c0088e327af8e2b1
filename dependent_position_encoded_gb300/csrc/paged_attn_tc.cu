// The attention of plain steps, bf16 (paged_attn_tc.cuh).
#include "paged_attn_tc.cuh"

namespace path {
namespace paged {

size_t tc_ws_bytes(const Cache &c, int N, int max_chunk, int d, bool fox) {
    return tc_layout(c, N, max_chunk, d, fox).total;
}

template cudaError_t launch_tc(const Step &, int, void *, float *, float *, void *, uint64_t, cudaStream_t);

}  // namespace paged
}  // namespace path

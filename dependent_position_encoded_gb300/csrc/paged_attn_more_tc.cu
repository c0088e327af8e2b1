// The attention of steps through a window or behind prefixes, bf16 (paged_attn_tc.cuh).
#include "paged_attn_tc.cuh"

namespace path {
namespace paged {

template cudaError_t launch_tc(const StepMore &, int, void *, float *, float *, void *, uint64_t, cudaStream_t);

}  // namespace paged
}  // namespace path

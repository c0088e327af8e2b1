// The kernels of paged_prep_tc.cuh for plain steps.
#include "paged_prep_tc.cuh"

namespace path {
namespace paged {

template cudaError_t launch_tc_prep<64>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_prep<128>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_carry<64>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_carry<128>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_finish<64>(const Step &, const TcWs &, const Behind &, cudaStream_t);
template cudaError_t launch_tc_finish<128>(const Step &, const TcWs &, const Behind &, cudaStream_t);

}  // namespace paged
}  // namespace path

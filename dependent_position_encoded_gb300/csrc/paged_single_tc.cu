// The pass of single tokens over their cached keys (paged_cached_tc.cuh).
#include "paged_cached_tc.cuh"

namespace path {
namespace paged {

ONE_PASS(PASS)

}  // namespace paged
}  // namespace path

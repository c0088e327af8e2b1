// The pass of a step with a window over its cached keys (paged_cached_tc.cuh).
#include "paged_cached_tc.cuh"

namespace path {
namespace paged {

EACH_PASS(PASS, Pass::window)

}  // namespace paged
}  // namespace path

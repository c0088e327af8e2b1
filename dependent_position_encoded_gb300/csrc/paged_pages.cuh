// Sequence rows that the host names to the page kernels, passed by value (no copy of a host
// list has to outlive the call, and a captured call keeps them).
#pragma once

namespace path {
namespace paged {

constexpr int kMaxRows = 1024;
template <int N>
struct Rows {
    int n;
    int row[N];
};

}  // namespace paged
}  // namespace path

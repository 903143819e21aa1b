// Kernels of shared prefixes for head dim 64.
#include "fa2_paged_shared.cuh"

namespace fa2 {
int launch_paged_shared_d64(const PagedLaunchArgs& shared, const PagedLaunchArgs& own) {
  return launch_paged_shared<64>(shared, own);
}
}  // namespace fa2

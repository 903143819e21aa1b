// Kernels of shared prefixes for head dim 256.
#include "fa2_paged_shared.cuh"

namespace fa2 {
int launch_paged_shared_d256(const PagedLaunchArgs& shared, const PagedLaunchArgs& own) {
  return launch_paged_shared<256>(shared, own);
}
}  // namespace fa2

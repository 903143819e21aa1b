// Paged attention kernels for head dim 256 (fp16 and bf16, with and without a band).
#include "fa2_paged.cuh"

namespace fa2 {
int launch_paged_d256(const PagedLaunchArgs& a) { return launch_paged<256>(a); }
}  // namespace fa2

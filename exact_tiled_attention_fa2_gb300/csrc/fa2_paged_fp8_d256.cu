// Attention kernels on 8-bit paged rows for head dim 256.
#include "fa2_paged_fp8.cuh"

namespace fa2 {
int launch_paged_fp8_d256(const PagedFp8LaunchArgs& a) { return launch_paged_fp8<256>(a); }
}  // namespace fa2

// Attention kernels on 8-bit paged rows for head dim 64.
#include "fa2_paged_fp8.cuh"

namespace fa2 {
int launch_paged_fp8_d64(const PagedFp8LaunchArgs& a) { return launch_paged_fp8<64>(a); }
}  // namespace fa2

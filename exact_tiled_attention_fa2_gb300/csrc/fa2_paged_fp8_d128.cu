// Attention kernels on 8-bit paged rows for head dim 128.
#include "fa2_paged_fp8.cuh"

namespace fa2 {
int launch_paged_fp8_d128(const PagedFp8LaunchArgs& a) { return launch_paged_fp8<128>(a); }
}  // namespace fa2

// Paged attention kernels for head dim 128 (fp16 and bf16, with and without a band).
#include "fa2_paged.cuh"

namespace fa2 {
int launch_paged_d128(const PagedLaunchArgs& a) { return launch_paged<128>(a); }
}  // namespace fa2

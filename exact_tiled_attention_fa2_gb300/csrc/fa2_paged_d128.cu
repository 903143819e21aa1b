// Paged attention kernels for head dim 128 (fp16 and bf16, with and without a band).
#include "fa2_paged.cuh"

namespace fa2 {
int launch_paged_d128(const PagedLaunchArgs& a) { return launch_paged<128>(a); }
int launch_paged_merge_d128(const PagedParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_paged_merge<128, true>(p, stream) : launch_paged_merge<128, false>(p, stream);
}
}  // namespace fa2

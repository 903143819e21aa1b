// Paged attention kernels for head dim 64 (fp16 and bf16, with and without a band).
#include "fa2_paged.cuh"

namespace fa2 {
int launch_paged_d64(const PagedLaunchArgs& a) { return launch_paged<64>(a); }
int launch_paged_merge_d64(const PagedParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_paged_merge<64, true>(p, stream) : launch_paged_merge<64, false>(p, stream);
}
}  // namespace fa2

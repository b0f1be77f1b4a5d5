// Attention over the paged 8-bit cache (sm_103a): capped scores, with or without a bias and masks.
#include "kvq_paged_launch.cuh"

namespace kvq {

kvq_status launch_paged_capped(const PagedAttnArgs& a, cudaStream_t stream) { return launch_paged_mode<kCapped>(a, stream); }

}  // namespace kvq

// Attention over the paged 8-bit cache (sm_103a): scores with a distance bias, and the masks beyond
// causal and window.
#include "kvq_paged_launch.cuh"

namespace kvq {

kvq_status launch_paged_biased(const PagedAttnArgs& a, cudaStream_t stream) { return launch_paged_mode<kBiased>(a, stream); }

}  // namespace kvq

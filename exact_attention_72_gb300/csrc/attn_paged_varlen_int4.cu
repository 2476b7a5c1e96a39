// Instances of the attention of chunks over a paged cache: 4 bits.
#include "attn_paged_varlen_impl.cuh"

namespace gb300 {
template cudaError_t launch_paged_varlen<64, true>(const PagedVarlenLaunch&, cudaStream_t);
template cudaError_t launch_paged_varlen<128, true>(const PagedVarlenLaunch&, cudaStream_t);
template cudaError_t launch_paged_varlen<256, true>(const PagedVarlenLaunch&, cudaStream_t);
}  // namespace gb300

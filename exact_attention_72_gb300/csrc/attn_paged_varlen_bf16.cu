// Instances of the attention of chunks over a paged cache: bf16.
#include "attn_paged_varlen_impl.cuh"

namespace gb300 {
template cudaError_t launch_paged_varlen<64, false>(const PagedVarlenLaunch&, cudaStream_t);
template cudaError_t launch_paged_varlen<128, false>(const PagedVarlenLaunch&, cudaStream_t);
template cudaError_t launch_paged_varlen<256, false>(const PagedVarlenLaunch&, cudaStream_t);
}  // namespace gb300

// Launchers of attn_paged_varlen_kernel, one for each head dim and cache type.
#pragma once
#include "attn_paged_varlen.cuh"

namespace gb300 {

struct PagedVarlenLaunch {
  CUtensorMap tm_q, tm_k, tm_v;   // bf16 cache only
  PagedVarlenParams params;
  int grid;
  unsigned long long context;
};

template <int D, bool INT4>
cudaError_t launch_paged_varlen(const PagedVarlenLaunch& a, cudaStream_t stream);

extern template cudaError_t launch_paged_varlen<64, false>(const PagedVarlenLaunch&, cudaStream_t);
extern template cudaError_t launch_paged_varlen<128, false>(const PagedVarlenLaunch&, cudaStream_t);
extern template cudaError_t launch_paged_varlen<256, false>(const PagedVarlenLaunch&, cudaStream_t);
extern template cudaError_t launch_paged_varlen<64, true>(const PagedVarlenLaunch&, cudaStream_t);
extern template cudaError_t launch_paged_varlen<128, true>(const PagedVarlenLaunch&, cudaStream_t);
extern template cudaError_t launch_paged_varlen<256, true>(const PagedVarlenLaunch&, cudaStream_t);

}  // namespace gb300

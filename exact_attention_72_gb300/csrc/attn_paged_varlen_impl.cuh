// Definition of the launchers; included by the instantiation units only.
#pragma once
#include <atomic>

#include "attn_paged_varlen.h"

namespace gb300 {

template <int D, bool INT4>
cudaError_t launch_paged_varlen(const PagedVarlenLaunch& a, cudaStream_t stream) {
  using C = PagedVarlenCfg<D, INT4>;
  auto kernel = attn_paged_varlen_kernel<C>;
  // The attribute stays with the context; setting it on every call would cost the host 1 us.
  static std::atomic<unsigned long long> set_for{0};
  if (a.context == 0 || set_for.load(std::memory_order_relaxed) != a.context) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // setmaxnreg deals out the registers that the block was launched with: refuse a launch with fewer than the split needs.
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
    if (fa.numRegs * C::THREADS < C::REGS_NEEDED) return cudaErrorInvalidConfiguration;
    set_for.store(a.context, std::memory_order_relaxed);
  }
  return launch_dependent(kernel, dim3((unsigned)a.grid), dim3(C::THREADS), (size_t)C::SMEM_BYTES, stream, a.tm_q, a.tm_k, a.tm_v,
                          a.params);
}

}  // namespace gb300

// Attention of the sequences of one query token in a packed batch over a 4-bit cache (attn_paged.cu), for attn_fwd_paged_varlen.
#pragma once
#include "attn.h"
#include "paged.cuh"

namespace gb300 {

struct PagedSingles {
  PagedCache c;
  const __nv_bfloat16* q;   // [total, H, d]
  __nv_bfloat16* o;
  float* lse;               // [H, total]
  const int *table, *lens, *cu;
  long long total, table_stride;
  int B, H, d, max_pages, sms;
  float scale;
  void* workspace;          // 256-byte aligned, paged_singles_workspace_bytes(H / Hkv, d, sms)
  uint32_t* status;
  unsigned long long context;
};

attn_status_t launch_paged_singles(const PagedSingles& a, cudaStream_t stream);
size_t paged_singles_workspace_bytes(int G, int d, int sms);

}  // namespace gb300

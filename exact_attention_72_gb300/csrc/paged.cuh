// Paged key/value cache: addressing, the 4-bit row format and the search of a packed token's
// sequence, shared by the kernels that fill, read back and attend to the cache.
//
// 4-bit rows ("int4"): the d values of one token and kv head are cut into groups of 64. A group
// with least value lo and greatest hi has
//   zero  = lo rounded down to bf16,
//   scale = max((hi - zero) / 15, 2^-20 max(|lo|, |hi|), 2^-100) rounded up to bf16,
//   code  = rint((x - zero) / scale) in 0 .. 15,      x ~ zero + scale * code,
// so no value is clipped and |x - (zero + scale code)| <= scale / 2 up to fp32 rounding. The two
// floors keep scale positive and |zero| / scale within 2^20: the first lies far below bf16's own
// resolution of the group (2^-9 of its greatest value), the second counts only for groups whose values
// all stay below 15 2^-100. Codes of dims 2i and 2i + 1
// share byte i (even dim in the low half); (scale, zero) is a bf16 pair, scale first.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace gb300 {

constexpr int kInt4Group = 64;
constexpr uint32_t kStatusBadPage = 0x20000000u | 13u;       // paged cache: page, position (angles too) or offsets
constexpr uint32_t kStatusBadPosition = 0x20000000u | 14u;   // norm and rotation: position outside the tables

// Cache of one layer, in bytes: row (page, token in page, kv head) of k starts at
// k + page * page_b + token * token_b + head * head_b; its (scale, zero) pairs at k_sz + ...
struct PagedCache {
  uint8_t *k, *v, *k_sz, *v_sz;
  long long page_b, token_b, head_b;
  long long sz_page_b, sz_token_b, sz_head_b;
  int num_pages, page_size, Hkv;
};

// The sequence that packed token t lies in: the b with cu[b] <= t < cu[b + 1], found by the LPR
// lanes of one row together (LPR probes a step; one step for B <= LPR). All lanes of the warp call
// this. Offsets that do not ascend give some b in 0 .. B; the caller checks cu[b] <= t < cu[b + 1].
template <int LPR>
__device__ __forceinline__ int find_sequence(const int* __restrict__ cu, int B, int t) {
  const int lane = threadIdx.x & 31, j = lane % LPR, shift = lane / LPR * LPR;
  const uint32_t mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u);
  int lo = 0, n = B;
  while (true) {
    const int step = (n + LPR - 1) / LPR;
    const long long idx = (long long)lo + (long long)(j + 1) * step - 1;    // last sequence of my part
    const bool behind = idx < B && cu[idx + 1] <= t;
    const uint32_t bal = (__ballot_sync(0xffffffffu, behind) >> shift) & mask;
    // parts wholly behind t come first; a part cut off by B counts as not behind
    lo += __popc(bal) * step;
    if (step == 1) return lo < B ? lo : B;
    n = step;
    if (lo > B) lo = B;
  }
}

}  // namespace gb300

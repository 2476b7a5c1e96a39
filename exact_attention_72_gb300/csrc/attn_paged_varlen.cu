// Entry point of the attention of chunks over a paged cache, and the kernel that joins the parts of units that several CTAs
// have worked on.
#include <algorithm>
#include <climits>
#include <cmath>

#include "attn.h"
#include "attn_paged_varlen.h"
#include "paged_host.h"
#include "paged_singles.h"

namespace gb300 {
namespace {

constexpr int kJoinWarps = 8;

// O = sum 2^(LSE_i - LSE) O_i, LSE = log2 sum 2^LSE_i over the parts of the unit that CTA blockIdx.x of the grid before has
// begun and not ended: its slot 2 x + 1, then slots 2 (x + 1), 2 (x + 2), .. A warp takes one row. Parts without keys have
// LSE -inf and no O.
template <int D, int ROWS>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_paged_varlen_join_kernel(const PagedVarlenParams p) {
  griddep_wait();
  const int4 cut = p.cut[blockIdx.x];
  const int parts = cut.w;
  if (parts == 0) return;
  const int row = blockIdx.y * kJoinWarps + threadIdx.x / 32, lane = threadIdx.x % 32, r = row % 128;
  const int pos_r = (uint32_t)r / p.div_g, g = r - pos_r * p.G, pos = row / 128 * p.P + pos_r;
  if (r >= p.P * p.G || pos >= cut.z) return;
  constexpr int V = D / 32;   // values of a lane
  auto at = [&](int i) { return (i == 0 ? 2LL * blockIdx.x + 1 : 2LL * (blockIdx.x + i)) * ROWS + row; };
  float top = -INFINITY;
  bool any = false;   // a part that has keys, or is NaN
  for (int i = lane; i < parts; i += 32) {
    const float x = p.part_lse[at(i)];
    top = fmaxf(top, x);
    any = any || !(x == -INFINITY);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  any = __any_sync(0xffffffffu, any);
  float sum = 0.f, x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = 0.f;
  if (any) {
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float lse2 = p.part_lse[at(i)];
      if (lse2 == -INFINITY) continue;
      const float f = ex2(lse2 - top);
      sum += f;
      const float* from = p.part_o + at(i) * D + lane * V;
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(from + v));
        x[v] = fmaf(f, y.x, x[v]), x[v + 1] = fmaf(f, y.y, x[v + 1]);
      }
    }
  }
  const float inv = any ? 1.f / sum : 0.f;
  const int h = cut.y * p.G + g;
  const long long to = (long long)(cut.x + pos) * p.H + h;
  uint32_t* o = reinterpret_cast<uint32_t*>(p.o + to * D + lane * V);
#pragma unroll
  for (int v = 0; v < V; v += 2) o[v / 2] = pack_bf16x2(x[v] * inv, x[v + 1] * inv);
  if (lane == 0) p.lse[(long long)h * p.total_q + cut.x + pos] = any ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <int D, bool INT4>
cudaError_t launch(const PagedVarlenLaunch& a, cudaStream_t s) {
  constexpr int ROWS = PagedVarlenCfg<D, INT4>::ROWS;
  const cudaError_t e = launch_paged_varlen<D, INT4>(a, s);
  if (e != cudaSuccess || a.grid == 1) return e;   // one CTA cuts nothing
  return launch_dependent(attn_paged_varlen_join_kernel<D, ROWS>, dim3((unsigned)a.grid, ROWS / kJoinWarps), dim3(32 * kJoinWarps),
                          0, s, a.params);
}

// Over 4-bit caches a chunk's kernel unpacks every key for its tensor cores, 2.3 us a tile of 128 whatever its rows, where the
// kernel of attn_fwd_paged multiplies the codes as they are. It takes sequences of one token (of at most kSinglesRows rows a kv
// head, which read the cache once) in batches of kSinglesBatch and more. Which sequences have one token is known on the GPU only, and
// its two launches cost 8 to 10 us if there is none: so a rule on the size of the batch, where single tokens are likely, and neither
// side of it is always right. H 32, Hkv 8, d 128, us unpacked and so:
//   all single tokens:  B 30, up to 16384 keys 367, 106;  B 8, 8000 keys 69, 36, 500 keys 24 to 26, 26
//     below the rule:   B 4, 65536 keys 224, 73;  B 7 384, 110;  B 4, 8000 keys 42, 32;  up to 2000 keys 24 to 32, 24 to 30
//   no single token:    8 chunks of 4 over 500 keys 28, 36;  of 60 over 2000 58, 67;  30 of 100 over 8000 443, 454
constexpr int kSinglesRows = 16, kSinglesBatch = 8;

int unit_rows(int d) { return d <= 128 ? 256 : 128; }
size_t pad(size_t x) { return (x + 255) / 256 * 256; }

// Bytes of the parts, of their LSE, and of the cut units.
void workspace_parts(int sms, int d, size_t (&n)[3]) {
  n[0] = pad((size_t)2 * sms * unit_rows(d) * d * 4);
  n[1] = pad((size_t)2 * sms * unit_rows(d) * 4);
  n[2] = pad((size_t)sms * sizeof(int4));
}

// Bytes of a call's workspace: the kernels that share it run one after the other.
size_t workspace_need(int sms, int d, int G, attn_cache_type_t type) {
  size_t n[3];
  workspace_parts(sms, d, n);
  const size_t parts = n[0] + n[1] + n[2];
  return type == ATTN_CACHE_INT4 ? std::max(parts, paged_singles_workspace_bytes(std::min(G, kSinglesRows), d, sms)) : parts;
}

// bf16 cache -> 4-D map (d, token of a page, kv head, page), box 64 columns of `rows` tokens. The stride of a single page,
// token or head says nothing, and may be 0.
bool cache_map(CUtensorMap* m, const void* base, const PagedCache& c, int d, int rows) {
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)c.page_size, (uint64_t)c.Hkv, (uint64_t)c.num_pages};
  const uint64_t strides[3] = {(uint64_t)c.token_b, (uint64_t)(c.Hkv > 1 ? c.head_b : 2 * d), (uint64_t)(c.num_pages > 1 ? c.page_b : 2 * d)};
  const uint32_t box[4] = {64, (uint32_t)rows, 1, 1};
  return encode_bf16_map(m, base, 4, dims, strides, box);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" size_t attn_fwd_paged_varlen_workspace_bytes(int B, int H, int Hkv, int total_q, int d, attn_cache_type_t type) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || total_q < 0 || (d != 64 && d != 128 && d != 256)) return 0;
  if (type != ATTN_CACHE_BF16 && type != ATTN_CACHE_INT4) return 0;
  int sms = 152;
  uint32_t* status;
  device_state(&sms, &status);
  return workspace_need(sms, d, H / Hkv, type);
}

extern "C" attn_status_t attn_fwd_paged_varlen(const void* q, const attn_paged_cache_t* cache, void* o, float* lse,
                                               const int* page_table, long long table_stride, int max_pages,
                                               const int* cu_seqlens_q, const int* seqlens, int B, int H, int total_q, float scale,
                                               int causal, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  PagedVarlenLaunch a = {};
  PagedVarlenParams& p = a.params;
  const attn_status_t st = paged_cache_args(cache, &p.c);
  if (st != ATTN_OK) return st;
  const int d = cache->d, Hkv = cache->Hkv;
  if (B < 1 || H < 1 || H % Hkv || total_q < 0 || max_pages < 1 || table_stride < 0 || !std::isfinite(scale))
    return ATTN_ERR_INVALID_ARG;
  if (!q || !o || !lse || !page_table || !cu_seqlens_q || !seqlens || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(o, 16) || !is_aligned(lse, 4) || !is_aligned(page_table, 4) || !is_aligned(cu_seqlens_q, 4) ||
      !is_aligned(seqlens, 4) || !is_aligned(workspace, 256))
    return ATTN_ERR_INVALID_ARG;
  if (scale == 0.f) return ATTN_ERR_UNSUPPORTED;   // as attn_fwd
  const int G = H / Hkv;
  constexpr long long kMaxKeys = INT_MAX - 1023;   // keys and positions are counted in 32 bits
  const long long keys = (long long)max_pages * cache->page_size;
  if (G > 128 || total_q > kMaxKeys || keys > kMaxKeys) return ATTN_ERR_UNSUPPORTED;
  const int P = 128 / G, RP = P * (unit_rows(d) / 128);
  // Work of all units, as the kernel adds it up.
  const double most = ((double)total_q / RP + std::min(B, total_q)) * Hkv * (4. * keys + kUnitOverhead);
  if (most > (double)kMostWork) return ATTN_ERR_UNSUPPORTED;
  if (!device_state(&a.grid, &p.status, &a.context)) return ATTN_ERR_CUDA;
  size_t n[3];
  workspace_parts(a.grid, d, n);
  const size_t need = workspace_need(a.grid, d, G, cache->type);
  if (workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
  struct {
    const void* b;
    size_t n;
  } x[4] = {{o, (size_t)total_q * H * d * 2}, {lse, (size_t)total_q * H * 4}, {workspace, need}, {q, (size_t)total_q * H * d * 2}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 4; ++j) {
      const uintptr_t u = (uintptr_t)x[i].b, v = (uintptr_t)x[j].b;
      if (u < v + x[j].n && v < u + x[i].n) return ATTN_ERR_INVALID_ARG;
    }
  if (total_q == 0) return ATTN_OK;   // no query rows: nothing to write
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.table = page_table, p.table_stride = table_stride, p.cu = cu_seqlens_q, p.lens = seqlens;
  p.B = B, p.H = H, p.G = G, p.P = P, p.total_q = total_q, p.max_pages = max_pages, p.causal = causal != 0;
  p.div_g = fast_div((uint32_t)G), p.div_page = fast_div((uint32_t)cache->page_size);
  p.scale_log2 = std::fabs(scale) * 1.4426950408889634f;
  p.qk_negate = scale < 0.f ? kIdescNegateA : 0u;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + n[0]);
  p.cut = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + n[0] + n[1]);
  p.o_v8 = is_aligned(o, 32);
  p.timeout_ns = wait_timeout_ns();
  p.debug_skip_load = debug_skip_load();
  p.box_rows = 16;
  while (p.box_rows < 128 && cache->page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
  const bool int4 = cache->type == ATTN_CACHE_INT4;
  // (that kernel counts its tiles of 32 keys, and 4 more, of at most two blocks of rows, in 32 bits)
  p.skip_singles = int4 && B >= kSinglesBatch && G <= kSinglesRows && 2LL * B * Hkv * (keys / 32 + 5) <= INT_MAX;
  const int sms = a.grid;
  a.grid = (int)std::clamp<double>(most / kLeastShare, 1., a.grid);
  if (!int4) {
    const uint64_t dims[4] = {(uint64_t)d, (uint64_t)G, (uint64_t)total_q, (uint64_t)Hkv};
    const uint64_t strides[3] = {(uint64_t)2 * d, (uint64_t)2 * H * d, (uint64_t)2 * G * d};
    const uint32_t box[4] = {64, (uint32_t)G, (uint32_t)P, 1};
    if (std::max({p.c.page_b, p.c.token_b, p.c.head_b}) >= (1LL << 40)) return ATTN_ERR_UNSUPPORTED;
    if (!encode_bf16_map(&a.tm_q, q, 4, dims, strides, box)) return ATTN_ERR_CUDA;
    if (!cache_map(&a.tm_k, p.c.k, p.c, d, p.box_rows) || !cache_map(&a.tm_v, p.c.v, p.c, d, p.box_rows)) return ATTN_ERR_UNSUPPORTED;
  }
  cudaError_t e;
  switch (d) {
    case 64: e = int4 ? launch<64, true>(a, stream) : launch<64, false>(a, stream); break;
    case 128: e = int4 ? launch<128, true>(a, stream) : launch<128, false>(a, stream); break;
    default: e = int4 ? launch<256, true>(a, stream) : launch<256, false>(a, stream); break;
  }
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  if (!p.skip_singles) return ATTN_OK;
  return launch_paged_singles({p.c, p.q, p.o, lse, page_table, seqlens, cu_seqlens_q, total_q, table_stride, B, H, d, max_pages, sms,
                               scale, workspace, p.status, a.context},
                              stream);
}

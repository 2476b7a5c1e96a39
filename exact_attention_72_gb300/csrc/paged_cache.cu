// Filling a paged key/value cache and reading it back.
//
// attn_paged_append: token i of sequence b (row cu[b] + i of the packed k and v) goes to position
// p = len[b] + i, that is row p % page_size of page table[b, p / page_size]. Keys are turned by their
// position's angles on the way; rows are stored as bf16 or in the 4-bit format of paged.cuh.
// attn_paged_gather: rows 0 .. n_b - 1 of every sequence into packed bf16 k and v, the layout the
// ragged-batch forward reads.
//
// A lane reads the values that its own are paired with from the same row (a second load of a line already in L1) instead
// of exchanging them, and a group of 64 values is 4 neighbouring lanes, so its least and greatest value take two
// exchanges. Rotation and quantisation round every step as written here (no contraction into fused multiply-adds): a
// code must not depend on how the compiler schedules, or a value at a border between two codes would change with it.
//
// Measured on a GB300, 8 kv heads, d 128, 4 bits: append of 12.4k tokens 24.5 us (66 MB; arithmetic and the chain of
// offsets, page and angles; 49 us with IEEE divisions and 8 values a lane), gather of 29.4k tokens 24.4 us (154 MB, 93% of
// the copy bandwidth; 29.5 us with values converted one by one).
#include <algorithm>
#include <climits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "fastdiv.cuh"
#include "ops.h"
#include "paged.cuh"
#include "paged_host.h"

namespace gb300 {
namespace {

constexpr int kThreads = 128;

struct AppendParams {
  PagedCache c;
  const __nv_bfloat16 *k, *v;
  long long k_st, k_sh, v_st, v_sh;
  const int *cu, *len, *table;
  long long table_stride;
  const float *cos, *sin;
  int B, total, max_pages, half, rope_dim, max_pos;
  FastDiv parts, page_size;   // parts: tasks of a token
  uint32_t* status;
};

struct GatherParams {
  PagedCache c;
  __nv_bfloat16 *k, *v;
  const int *cu, *table;
  long long table_stride;
  int B, total, max_pages;
  FastDiv parts, page_size;
  uint32_t* status;
};

__device__ __forceinline__ void unpack8(float (&x)[8], const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// fp32 to the bf16 not above it (UP false) or not below it, as fp32.
template <bool UP>
__device__ __forceinline__ float bf16_toward(float x) {
  const uint32_t bits = __float_as_uint(x), cut = bits & 0xffff0000u;
  const bool away = cut != bits && ((bits >> 31) != 0) != UP;
  return __uint_as_float(cut + (away ? 0x10000u : 0u));
}

// x / y, correctly rounded, from the correctly rounded reciprocal of y (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor"): the remainder of the first product is exact.
__device__ __forceinline__ float divide(float x, float y, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, y, x), inv, q);
}

// 16 of a group's 64 values (4 neighbouring lanes) as codes; sz: its (scale, zero) pair.
__device__ __forceinline__ uint2 quantise16(const float (&x)[16], uint32_t& sz) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float zero = bf16_toward<false>(lo);
  const float least = fmaxf(fmaxf(fabsf(lo), fabsf(hi)) * 0x1p-20f, 0x1p-100f);
  const float scale = bf16_toward<true>(fmaxf(divide(__fsub_rn(hi, zero), 15.f, 1.f / 15.f), least));
  sz = (__float_as_uint(scale) >> 16) | (__float_as_uint(zero) & 0xffff0000u);
  // 0 <= quotient <= 15, as scale >= (hi - zero) / 15. Adding 2^23 rounds it to a whole number, which then stands in the
  // low bits; the exponents that the sum of the shifted words carries with it are taken off at the end.
  const float inv = __frcp_rn(scale);
  uint32_t codes[2] = {0, 0}, exponents = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      codes[s] = codes[s] * 16 + __float_as_uint(__fadd_rn(divide(__fsub_rn(x[8 * s + i], zero), scale, inv), 0x1p23f));
    exponents = exponents * 16 + 0x4b000000u;
  }
  return make_uint2(codes[0] - exponents, codes[1] - exponents);
}

// Where position pos of sequence b lies, or false where the table does not lead into the pool.
__device__ __forceinline__ bool find_row(const PagedCache& c, const FastDiv& page_size,
                                         const int* __restrict__ table, long long table_stride, int max_pages, int b,
                                         int pos, int& page, int& at) {
  if (pos < 0) return false;
  const int e = (uint32_t)pos / page_size;
  if (e >= max_pages) return false;
  page = table[b * table_stride + e];
  at = pos - e * c.page_size;
  return page >= 0 && page < c.num_pages;
}

// d / 16 lanes hold a row; a task is one head of one token, key and value.
template <int D, bool INT4, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendParams p) {
  constexpr int LPR = D / 16;
  const int l = threadIdx.x % LPR;
  const uint32_t task = blockIdx.x * (uint32_t)(kThreads / LPR) + threadIdx.x / LPR, token = task / p.parts;
  const int t = min(token, (uint32_t)p.total - 1u), h = task - token * p.parts.v;
  bool good = token < (uint32_t)p.total;
  // This lane's dims in eights, 16l and 16l + 8, and for each where the values begin that they are paired with.
  const __nv_bfloat16 *k = p.k + t * p.k_st + h * p.k_sh, *v = p.v + t * p.v_st + h * p.v_sh;
  uint4 raw[2][2], raw_mate[2];
  bool turned[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int d0 = 16 * l + 8 * s;
    raw[0][s] = *reinterpret_cast<const uint4*>(k + d0);
    raw[1][s] = *reinterpret_cast<const uint4*>(v + d0);
    turned[s] = p.cos && d0 < p.rope_dim;
    raw_mate[s] = make_uint4(0, 0, 0, 0);
    if (!INTERLEAVED && turned[s])
      raw_mate[s] = *reinterpret_cast<const uint4*>(k + (d0 < p.half ? d0 + p.half : d0 - p.half));
  }
  const int b = find_sequence<LPR>(p.cu, p.B, t);
  int page = 0, at = 0, pos = 0;
  if (b >= p.B) {
    good = false;   // behind the last sequence: not stored
  } else {
    const int first = p.cu[b], past = p.len[b];
    pos = past + (t - first);
    const bool in = t >= first && t < p.cu[b + 1] && past >= 0 && pos >= 0 &&
                    find_row(p.c, p.page_size, p.table, p.table_stride, p.max_pages, b, pos, page, at) &&
                    (!p.cos || pos < p.max_pos);
    if (good && !in && l == 0) atomicCAS(p.status, 0u, kStatusBadPage);
    good = good && in;
    if (!in) pos = 0;
  }
  float y[2][16];   // key, value
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float x[8], m[8], cs[8], sn[8];
    unpack8(x, raw[1][s]);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[1][8 * s + j] = x[j];
    unpack8(x, raw[0][s]);
    if (turned[s]) {
      // pair of dim j: j mod half, or j / 2 when interleaved
      const int d0 = 16 * l + 8 * s, pair = INTERLEAVED ? d0 / 2 : (d0 < p.half ? d0 : d0 - p.half);
      const float* ct = p.cos + (long long)pos * p.half + pair;
      const float* st = p.sin + (long long)pos * p.half + pair;
#pragma unroll
      for (int i = 0; i < (INTERLEAVED ? 4 : 8); i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(ct + i), b = *reinterpret_cast<const float4*>(st + i);
        cs[i] = a.x, cs[i + 1] = a.y, cs[i + 2] = a.z, cs[i + 3] = a.w;
        sn[i] = b.x, sn[i + 1] = b.y, sn[i + 2] = b.z, sn[i + 3] = b.w;
      }
      if (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u = x[2 * j], w = x[2 * j + 1];
          x[2 * j] = __fsub_rn(__fmul_rn(u, cs[j]), __fmul_rn(w, sn[j]));
          x[2 * j + 1] = __fadd_rn(__fmul_rn(w, cs[j]), __fmul_rn(u, sn[j]));
        }
      } else {
        unpack8(m, raw_mate[s]);
        // the first half subtracts: a product with the sine's sign turned has the other sign, bit for bit
        const float sign = d0 < p.half ? -1.f : 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], cs[j]), __fmul_rn(m[j], __fmul_rn(sn[j], sign)));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) y[0][8 * s + j] = x[j];
  }
  const PagedCache& c = p.c;
  const long long row = page * c.page_b + at * c.token_b + h * c.head_b;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint8_t* base = (i ? c.v : c.k) + row;
    if constexpr (INT4) {
      uint32_t sz;
      const uint2 codes = quantise16(y[i], sz);
      if (good) {
        *reinterpret_cast<uint2*>(base + 8 * l) = codes;
        const long long sz_row = page * c.sz_page_b + at * c.sz_token_b + h * c.sz_head_b;
        if (l % 4 == 0) *reinterpret_cast<uint32_t*>((i ? c.v_sz : c.k_sz) + sz_row + l) = sz;
      }
    } else if (good) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {   // values no rotation touches keep their bits
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = y[i][8 * s + j];
        *reinterpret_cast<uint4*>(base + 32 * l + 16 * s) = i == 0 && turned[s] ? pack8(x) : raw[i][s];
      }
    }
  }
}

constexpr int kGatherRows = 2;   // heads of one token, keys and values

// The values of 8 codes as bf16. A code in the low bits of bf16 128 is 128 + code; scale * code + zero is rounded once.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t sz) {
  const uint32_t scale = __byte_perm(sz, 0, 0x1010), zero = __byte_perm(sz, 0, 0x3232);
  uint32_t x[4];   // codes (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((codes >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("{\n .reg .b32 c;\n sub.rn.bf16x2 c, %1, %2;\n fma.rn.bf16x2 %0, c, %3, %4;\n}"
        : "=r"(x[i])
        : "r"(c), "r"(0x43004300u), "r"(scale), "r"(zero));
  }
  return make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                    __byte_perm(x[2], x[3], 0x7632));
}

template <int D, bool INT4>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(const GatherParams p) {
  constexpr int LPR = D / 8;
  const int l = threadIdx.x % LPR;
  const uint32_t task = blockIdx.x * (uint32_t)(kThreads / LPR) + threadIdx.x / LPR, token = task / p.parts;
  const int t = min(token, (uint32_t)p.total - 1u), h0 = (task - token * p.parts.v) * kGatherRows, heads = p.c.Hkv;
  const bool mine = token < (uint32_t)p.total;
  const int b = find_sequence<LPR>(p.cu, p.B, t);
  if (b >= p.B || !mine) return;   // behind the last sequence: left as it was
  const int first = p.cu[b];
  int page, at;
  if (t < first || t >= p.cu[b + 1] ||
      !find_row(p.c, p.page_size, p.table, p.table_stride, p.max_pages, b, t - first, page, at)) {
    if (l == 0) atomicCAS(p.status, 0u, kStatusBadPage);
    return;
  }
  const PagedCache& c = p.c;
  const long long row0 = page * c.page_b + at * c.token_b, out = ((long long)t * heads + h0) * D + 8 * l;
  if constexpr (INT4) {
    const long long sz0 = page * c.sz_page_b + at * c.sz_token_b + l / 8 * 4;
    uint32_t codes[2][kGatherRows], sz[2][kGatherRows];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      const int h = min(h0 + i, heads - 1);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        codes[v][i] = *reinterpret_cast<const uint32_t*>((v ? c.v : c.k) + row0 + h * c.head_b + 4 * l);
        sz[v][i] = *reinterpret_cast<const uint32_t*>((v ? c.v_sz : c.k_sz) + sz0 + h * c.sz_head_b);
      }
    }
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      if (h0 + i >= heads) break;
      *reinterpret_cast<uint4*>(p.k + out + i * D) = values8(codes[0][i], sz[0][i]);
      *reinterpret_cast<uint4*>(p.v + out + i * D) = values8(codes[1][i], sz[1][i]);
    }
  } else {
    uint4 raw[2][kGatherRows];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      const long long row = row0 + min(h0 + i, heads - 1) * c.head_b + 16 * l;
      raw[0][i] = *reinterpret_cast<const uint4*>(c.k + row);
      raw[1][i] = *reinterpret_cast<const uint4*>(c.v + row);
    }
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      if (h0 + i >= heads) break;
      *reinterpret_cast<uint4*>(p.k + out + i * D) = raw[0][i];
      *reinterpret_cast<uint4*>(p.v + out + i * D) = raw[1][i];
    }
  }
}

template <int D, bool INT4>
cudaError_t launch_append(const AppendParams& p, bool interleaved, cudaStream_t s) {
  const unsigned rows = kThreads / (D / 16);
  const unsigned grid = ((unsigned)p.total * p.parts.v + rows - 1) / rows;
  if (interleaved) paged_append_kernel<D, INT4, true><<<grid, kThreads, 0, s>>>(p);
  else paged_append_kernel<D, INT4, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D, bool INT4>
cudaError_t launch_gather(const GatherParams& p, cudaStream_t s) {
  const unsigned rows = kThreads / (D / 8);
  paged_gather_kernel<D, INT4><<<((unsigned)p.total * p.parts.v + rows - 1) / rows, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" attn_status_t attn_paged_append(const attn_paged_cache_t* cache, const void* k, const void* v,
                                           long long k_stride_t, long long k_stride_h, long long v_stride_t,
                                           long long v_stride_h, const int* cu_seqlens, const int* cache_lens,
                                           const int* page_table, long long table_stride, int max_pages, int B,
                                           int total, const float* cos, const float* sin, int rope_dim, int max_pos,
                                           int interleaved, cudaStream_t stream) {
  AppendParams p = {};
  const attn_status_t st = paged_cache_args(cache, &p.c);
  if (st != ATTN_OK) return st;
  if (B < 1 || total < 0 || max_pages < 1 || table_stride < 0) return ATTN_ERR_INVALID_ARG;
  if (!k || !v || !cu_seqlens || !cache_lens || !page_table) return ATTN_ERR_INVALID_ARG;
  if (!is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(cu_seqlens, 4) || !is_aligned(cache_lens, 4) ||
      !is_aligned(page_table, 4))
    return ATTN_ERR_INVALID_ARG;
  for (const long long s : {k_stride_t, k_stride_h, v_stride_t, v_stride_h})
    if (s < 0 || s % 8 || s > (1LL << 40)) return ATTN_ERR_INVALID_ARG;
  if ((cos != nullptr) != (sin != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (cos) {
    if (!is_aligned(cos, 16) || !is_aligned(sin, 16) || max_pos < 1) return ATTN_ERR_INVALID_ARG;
    if (rope_dim < 16 || rope_dim % 16 || rope_dim > cache->d) return ATTN_ERR_INVALID_ARG;
  }
  p.parts = fast_div((uint32_t)cache->Hkv);
  p.page_size = fast_div((uint32_t)cache->page_size);
  if ((long long)total * p.parts.v > INT_MAX - kThreads) return ATTN_ERR_UNSUPPORTED;   // tasks are counted in 31 bits
  if (total == 0) return ATTN_OK;
  int sms;
  if (!device_state(&sms, &p.status)) return ATTN_ERR_CUDA;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_st = k_stride_t, p.k_sh = k_stride_h, p.v_st = v_stride_t, p.v_sh = v_stride_h;
  p.cu = cu_seqlens, p.len = cache_lens, p.table = page_table, p.table_stride = table_stride;
  p.cos = cos, p.sin = sin;
  p.B = B, p.total = total, p.max_pages = max_pages, p.max_pos = max_pos;
  p.rope_dim = cos ? rope_dim : 0, p.half = p.rope_dim / 2;
  const bool int4 = cache->type == ATTN_CACHE_INT4, il = interleaved != 0;
  cudaError_t e;
  switch (cache->d) {
    case 64: e = int4 ? launch_append<64, true>(p, il, stream) : launch_append<64, false>(p, il, stream); break;
    case 128: e = int4 ? launch_append<128, true>(p, il, stream) : launch_append<128, false>(p, il, stream); break;
    default: e = int4 ? launch_append<256, true>(p, il, stream) : launch_append<256, false>(p, il, stream); break;
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t attn_paged_gather(const attn_paged_cache_t* cache, void* k, void* v, const int* cu_seqlens,
                                           const int* page_table, long long table_stride, int max_pages, int B,
                                           int total, cudaStream_t stream) {
  GatherParams p = {};
  const attn_status_t st = paged_cache_args(cache, &p.c);
  if (st != ATTN_OK) return st;
  if (B < 1 || total < 0 || max_pages < 1 || table_stride < 0) return ATTN_ERR_INVALID_ARG;
  if (!k || !v || !cu_seqlens || !page_table) return ATTN_ERR_INVALID_ARG;
  if (!is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(cu_seqlens, 4) || !is_aligned(page_table, 4))
    return ATTN_ERR_INVALID_ARG;
  const uintptr_t bytes = (uintptr_t)total * cache->Hkv * cache->d * 2, kb = (uintptr_t)k, vb = (uintptr_t)v;
  if (kb < vb + bytes && vb < kb + bytes) return ATTN_ERR_INVALID_ARG;
  p.parts = fast_div((uint32_t)(((long long)cache->Hkv + kGatherRows - 1) / kGatherRows));
  p.page_size = fast_div((uint32_t)cache->page_size);
  if ((long long)total * p.parts.v > INT_MAX - kThreads) return ATTN_ERR_UNSUPPORTED;
  if (total == 0) return ATTN_OK;
  int sms;
  if (!device_state(&sms, &p.status)) return ATTN_ERR_CUDA;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.cu = cu_seqlens, p.table = page_table, p.table_stride = table_stride;
  p.B = B, p.total = total, p.max_pages = max_pages;
  const bool int4 = cache->type == ATTN_CACHE_INT4;
  cudaError_t e;
  switch (cache->d) {
    case 64: e = int4 ? launch_gather<64, true>(p, stream) : launch_gather<64, false>(p, stream); break;
    case 128: e = int4 ? launch_gather<128, true>(p, stream) : launch_gather<128, false>(p, stream); break;
    default: e = int4 ? launch_gather<256, true>(p, stream) : launch_gather<256, false>(p, stream); break;
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Filling a paged key/value cache and reading it back.
//
// attn_paged_append: token i of sequence b (row cu[b] + i of the packed k and v) goes to position
// p = len[b] + i, that is row p % page_size of page table[b, p / page_size]. Keys are turned by their
// position's angles on the way; rows are stored as bf16 or in the 4-bit format of paged.cuh.
// attn_paged_gather: rows 0 .. n_b - 1 of every sequence into packed bf16 k and v, the layout the
// ragged-batch forward reads.
//
// A lane holds 8 values of a row's first half and the 8 half a row on: the pairs of a fully turned row lie in one lane,
// and loads and stores are whole sectors (16 neighbouring values a lane took 14.1 instead of 11.8 us for 12.4k bf16 tokens).
// Rows turned in part read the paired values a second time, out of L1. Rotation and quantisation round every step as
// written here (no contraction into fused multiply-adds): a code must not depend on how the compiler schedules, or a value
// at a border between two codes would change with it.
//
// Measured on a GB300, 8 kv heads, d 128, 4 bits: append of 12.4k tokens 20 us (66 MB; arithmetic, 60% of the issue slots,
// and the chain of offsets, page and angles; 49 us with IEEE divisions, 24.5 us one value an instruction), gather of 29.4k
// tokens 24.4 us (154 MB, 93% of the copy bandwidth; 29.5 us with values converted one by one). Two heads a lane, sharing
// the look-ups, are no faster (45.3 against 45.0 us for both), nor are more CTAs an SM.
#include <algorithm>
#include <climits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "fastdiv.cuh"
#include "ops.h"
#include "paged.cuh"
#include "paged_host.h"
#include "ptx.cuh"

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
  uint64_t one, minus_one;    // pairs of them, where the compiler does not see the value
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

// Two values in a register pair: the arithmetic below works on two at a time (FFMA2 and its kin, half the issue slots).
__device__ __forceinline__ void unpack8(uint64_t* x, const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_pack(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}

__device__ __forceinline__ void load8(uint64_t (&x)[4], const float* from) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(from + 2 * i);
    x[i] = a.x, x[i + 1] = a.y;
  }
}

__device__ __forceinline__ uint4 pack8(const uint64_t* x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(x[i], lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// A lane's 16 values of a row as codes, dims 8l .. 8l + 7 in codes[0] and D / 2 on in codes[1]; sz: a (scale, zero) pair.
// d = 64: one group in 4 lanes. Above: the two eights lie in two groups of 8 lanes; lanes 0 to 3 of the eight finish the
// first one's least and greatest value, scale and reciprocal, lanes 4 to 7 the second's, and they swap what they found.
template <int D>
__device__ __forceinline__ void quantise16(const uint64_t (&x)[8], uint32_t (&codes)[2], uint32_t& sz) {
  constexpr bool TWO = D > 64;
  float lo[2], hi[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float a, b;
    f2_unpack(x[4 * s], a, b);
    lo[s] = fminf(a, b), hi[s] = fmaxf(a, b);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      f2_unpack(x[4 * s + i], a, b);
      lo[s] = fmin3(lo[s], a, b), hi[s] = fmax3(hi[s], a, b);
    }
  }
  const bool second = TWO && (threadIdx.x & 4);
  float least, greatest;
  if (TWO) {
    least = fminf(second ? lo[1] : lo[0], __shfl_xor_sync(0xffffffffu, second ? lo[0] : lo[1], 4));
    greatest = fmaxf(second ? hi[1] : hi[0], __shfl_xor_sync(0xffffffffu, second ? hi[0] : hi[1], 4));
  } else {
    least = fminf(lo[0], lo[1]), greatest = fmaxf(hi[0], hi[1]);
  }
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) {
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    greatest = fmaxf(greatest, __shfl_xor_sync(0xffffffffu, greatest, o));
  }
  const float zero = bf16_toward<false>(least);
  const float floor = fmaxf(fmaxf(fabsf(least), fabsf(greatest)) * 0x1p-20f, 0x1p-100f);
  const float scale = bf16_toward<true>(fmaxf(divide(__fsub_rn(greatest, zero), 15.f, 1.f / 15.f), floor));
  const float inv = __frcp_rn(scale);
  sz = (__float_as_uint(scale) >> 16) | (__float_as_uint(zero) & 0xffff0000u);
  uint32_t sz_of[2] = {sz, sz};
  float inv_of[2] = {inv, inv};
  if (TWO) {
    const uint32_t o_sz = __shfl_xor_sync(0xffffffffu, sz, 4);
    const float o_inv = __shfl_xor_sync(0xffffffffu, inv, 4);
    sz_of[0] = second ? o_sz : sz, sz_of[1] = second ? sz : o_sz;
    inv_of[0] = second ? o_inv : inv, inv_of[1] = second ? inv : o_inv;
  }
  // 0 <= quotient <= 15, as scale >= (greatest - zero) / 15. Adding 2^23 rounds it to a whole number, which then stands in
  // the low bits; the exponents that the sum of the shifted words carries with it are taken off at the end.
  const uint64_t whole2 = f2_pack(0x1p23f, 0x1p23f);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float z = __uint_as_float(sz_of[s] & 0xffff0000u), m = -__uint_as_float(sz_of[s] << 16);
    const uint64_t zero2 = f2_pack(z, z), inv2 = f2_pack(inv_of[s], inv_of[s]), minus_scale2 = f2_pack(m, m);
    uint32_t word = 0, exponents = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      // divide() by the scale, two at a time: the remainder is x - q scale = q (-scale) + x
      const uint64_t n = f2_sub(x[4 * s + i], zero2), q = f2_mul(n, inv2);
      float even, odd;
      f2_unpack(f2_add(f2_fma(f2_fma(q, minus_scale2, n), inv2, q), whole2), even, odd);
      word = (word * 16 + __float_as_uint(odd)) * 16 + __float_as_uint(even);
      exponents = (exponents * 16 + 0x4b000000u) * 16 + 0x4b000000u;
    }
    codes[s] = word - exponents;
  }
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

enum Rope { kNone, kFull, kPart, kInterleaved };   // rotation: none, of half-split pairs over the row or a part, of neighbours

// d / 16 lanes hold a row, dims 8l .. 8l + 7 and d / 2 on each (the pairs of a fully turned row, and loads and stores of
// whole sectors); a task is one head of one token, key and value.
template <int D, bool INT4, int ROPE>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();   // of the next kernel only the launch may overlap: it waits for this one's end
  constexpr int LPR = D / 16;
  const int l = threadIdx.x % LPR;
  const uint32_t task = blockIdx.x * (uint32_t)(kThreads / LPR) + threadIdx.x / LPR, token = task / p.parts;
  const int t = min(token, (uint32_t)p.total - 1u), h = task - token * p.parts.v;
  bool good = token < (uint32_t)p.total;
  const __nv_bfloat16 *k = p.k + t * p.k_st + h * p.k_sh, *v = p.v + t * p.v_st + h * p.v_sh;
  uint4 raw[2][2], raw_mate[2];
  bool turned[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int d0 = 8 * l + s * (D / 2);
    raw[0][s] = *reinterpret_cast<const uint4*>(k + d0);
    raw[1][s] = *reinterpret_cast<const uint4*>(v + d0);
    turned[s] = ROPE != kNone && (ROPE == kFull || d0 < p.rope_dim);
    raw_mate[s] = make_uint4(0, 0, 0, 0);
    if (ROPE == kPart && turned[s])
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
  // Rotation rounds both products, then their sum or difference: an addition of a product in a register pair may be fused
  // with it even where both are written with a rounding of their own, a product with +-1 out of memory may not (and is exact).
  uint64_t y[2][8];   // key, value
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 0; s < 2; ++s) unpack8(y[i] + 4 * s, raw[i][s]);
  if constexpr (ROPE == kFull) {
    uint64_t cs[4], sn[4];
    load8(cs, p.cos + (long long)pos * (D / 2) + 8 * l);
    load8(sn, p.sin + (long long)pos * (D / 2) + 8 * l);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t a = y[0][j], b = y[0][4 + j];
      y[0][j] = f2_fma(f2_mul(b, sn[j]), p.minus_one, f2_mul(a, cs[j]));
      y[0][4 + j] = f2_fma(f2_mul(a, sn[j]), p.one, f2_mul(b, cs[j]));
    }
  } else if constexpr (ROPE != kNone) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (!turned[s]) continue;
      // x cos -+ mate sin. Pair of dim j: j mod half, or j / 2 when interleaved
      const int d0 = 8 * l + s * (D / 2), pair = ROPE == kInterleaved ? d0 / 2 : (d0 < p.half ? d0 : d0 - p.half);
      const float* ct = p.cos + (long long)pos * p.half + pair;
      const float* st = p.sin + (long long)pos * p.half + pair;
      uint64_t* x = y[0] + 4 * s;
      uint64_t m[4], cs[4], sn[4], sign;
      if constexpr (ROPE == kInterleaved) {
        const float4 a = *reinterpret_cast<const float4*>(ct), b = *reinterpret_cast<const float4*>(st);
        const float ca[4] = {a.x, a.y, a.z, a.w}, sa[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float u, w;
          f2_unpack(x[j], u, w);
          m[j] = f2_pack(w, u), cs[j] = f2_pack(ca[j], ca[j]), sn[j] = f2_pack(sa[j], sa[j]);
        }
        float plus, minus, unused;
        f2_unpack(p.one, plus, unused);
        f2_unpack(p.minus_one, minus, unused);
        sign = f2_pack(minus, plus);
      } else {
        load8(cs, ct);
        load8(sn, st);
        unpack8(m, raw_mate[s]);
        sign = d0 < p.half ? p.minus_one : p.one;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = f2_fma(f2_mul(m[j], sn[j]), sign, f2_mul(x[j], cs[j]));
    }
  }
  const PagedCache& c = p.c;
  const long long row = page * c.page_b + at * c.token_b + h * c.head_b;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint8_t* base = (i ? c.v : c.k) + row;
    if constexpr (INT4) {
      uint32_t sz, codes[2];
      quantise16<D>(y[i], codes, sz);
      if (good) {
        *reinterpret_cast<uint32_t*>(base + 4 * l) = codes[0];
        *reinterpret_cast<uint32_t*>(base + D / 4 + 4 * l) = codes[1];
        const long long sz_row = page * c.sz_page_b + at * c.sz_token_b + h * c.sz_head_b;
        const int group = D == 64 ? 0 : l / 8 + (l & 4 ? D / 128 : 0);
        if (l % 4 == 0) *reinterpret_cast<uint32_t*>((i ? c.v_sz : c.k_sz) + sz_row + 4 * group) = sz;
      }
    } else if (good) {
#pragma unroll
      for (int s = 0; s < 2; ++s)   // values no rotation touches keep their bits
        *reinterpret_cast<uint4*>(base + D * s + 16 * l) = i == 0 && turned[s] ? pack8(y[i] + 4 * s) : raw[i][s];
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
  griddep_wait();
  griddep_launch_dependents();   // of the next kernel only the launch may overlap: it waits for this one's end
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
  auto kernel = !p.cos          ? paged_append_kernel<D, INT4, kNone>
                : interleaved     ? paged_append_kernel<D, INT4, kInterleaved>
                : p.rope_dim == D ? paged_append_kernel<D, INT4, kFull>
                                  : paged_append_kernel<D, INT4, kPart>;
  return launch_dependent(kernel, dim3(grid), dim3(kThreads), 0, s, p);
}

template <int D, bool INT4>
cudaError_t launch_gather(const GatherParams& p, cudaStream_t s) {
  const unsigned rows = kThreads / (D / 8);
  const unsigned grid = ((unsigned)p.total * p.parts.v + rows - 1) / rows;
  return launch_dependent(paged_gather_kernel<D, INT4>, dim3(grid), dim3(kThreads), 0, s, p);
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
  p.one = 0x3f8000003f800000u, p.minus_one = 0xbf800000bf800000u;
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

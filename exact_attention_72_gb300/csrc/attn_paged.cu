// Attention over a paged key/value cache in bf16 or 4 bits, for few query rows a sequence (decode,
// drafted tokens):  S = scale q k^T over the keys a row sees,  O = softmax(S) V,  LSE.
//
// The cache is read once and that bounds the call: 2 d / 2 + d / 4 bytes a key and kv head in 4 bits.
// All query rows that share a kv head (Nq tokens x H / Hkv heads) are columns of one narrow product,
//   S^T [keys x rows] = K [keys x d] q^T,     O^T [d x rows] = V^T [d x keys] P^T,
// with m16n8k16: the long dims (keys, d) fill the 16 and a call pads its rows only to 8. tcgen05 would
// pad them to 128 and needs unpacked operands in shared memory, more traffic than the cache itself.
//
// 4-bit codes go to the tensor cores as they are. A code c in the low bits of a half is the
// subnormal fp16 number c 2^-24, and 4 bits higher it is 16 c 2^-24: a pair of operands costs one AND.
// For keys the factor 16 is taken out of the query's matching values; for values it falls on
// separate output rows. Scale and zero stay outside the products, in fp32:
//   q.k = sum over groups  scale (codes . q) + zero sum(q),
//   O   = (sum_j (p_j scale_j) codes_j + sum_j p_j zero_j) / sum_j p_j.
// q is scaled by a power of two per row, so fp16 holds it exactly where it counts (2^-25 of the row's
// greatest value); p_j scale_j is rounded to fp16, 2^-12 of itself, and bf16 caches round p_j to bf16,
// 2^-9, both averaged over the keys. For p_j scale_j to stay within fp16 at any scale, the running
// maximum is taken over S + log2 of the key's scale (its exponent) instead of S.
//
// Work: sequences are cut into pieces of SPLIT keys; all pieces of all (sequence, kv head, row block)
// units in order are dealt to the CTAs in equal contiguous shares, so ragged batches load every SM
// alike. A unit inside one share is finished there; one cut across CTAs leaves normalised parts with
// their LSE, joined by a second, dependent launch. The shares follow from the lengths alone: the same
// bits on every run, no atomics.
//
// In a CTA each of the 4 warps takes every fourth tile of KT keys through a ring of its own in shared
// memory, filled by 16-byte asynchronous copies; warps meet only at the end of a unit. Keys are
// assigned to the MMA's rows in the order 0 4 1 5 2 6 3 7 so that a lane's four V rows are 4 apart
// and the loads of both products meet every bank once.
#include <algorithm>
#include <climits>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "fastdiv.cuh"
#include "ops.h"
#include "paged.cuh"
#include "paged_host.h"

namespace gb300 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kMinExp = -100.f;   // least scale exponent that counts in the running maximum

template <int D_, bool INT4_, int NT_>
struct Cfg {
  static constexpr int D = D_, NT = NT_;
  static constexpr bool INT4 = INT4_;
  static constexpr int KT = INT4 ? 32 : 16;              // keys of a warp's tile
  static constexpr int SPLIT = KT * kWarps;              // keys of a piece of work
  static constexpr int ROWS = 8 * NT;                    // query rows of a unit
  static constexpr int GROUPS = D / kInt4Group;
  static constexpr int ROWB = INT4 ? D / 2 : 2 * D;      // bytes of a key's row
  static constexpr int SZB = INT4 ? 4 * GROUPS : 0;      // bytes of its (scale, zero) pairs
  static constexpr int V_OFF = KT * ROWB, KSZ_OFF = 2 * KT * ROWB, VSZ_OFF = KSZ_OFF + KT * SZB;
  static constexpr int STAGE = VSZ_OFF + KT * SZB;
  static constexpr int STAGES = 3;
  static constexpr int WARP_BYTES = STAGES * STAGE;
  static constexpr int SMEM = kWarps * WARP_BYTES;
  static constexpr int CTAS = std::min(D * NT >= 256 ? 2 : 4, 233472 / (SMEM + 1024 + 1600));
  static_assert(WARP_BYTES >= ROWS * D * 4, "a warp's part of O is joined in its ring");
  static_assert(CTAS >= 1 && STAGE % 16 == 0, "ring");
};

struct Params {
  PagedCache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int *table, *lens;
  long long table_stride;
  int B, H, G, Nq, max_pages, row_blocks, causal;
  FastDiv blocks_per_page;   // 16-key blocks
  float scale_log2;
  float* part_o;     // [2 CTAs, ROWS, D] normalised O of a cut unit's parts
  float* part_lse;   // [2 CTAs, ROWS] their log2-sum-exp2
  int4* cut;         // [CTAs]: the unit that begins in this CTA and ends in a later one (z; -1: none)
  uint32_t* status;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(in ? N : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 x;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
  return x;
}

// The (scale, zero) pairs of a row.
template <int N>
__device__ __forceinline__ void load_pairs(uint32_t (&x)[N], uint32_t a) {
  if constexpr (N == 1) {
    x[0] = lds32(a);
  } else if constexpr (N == 2) {
    const uint2 w = lds64(a);
    x[0] = w.x, x[1] = w.y;
  } else {
    const uint4 w = lds128(a);
    x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
  }
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf162(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of row r in a tile of rows of ROWB bytes. A K load takes rows 0 4 1 5
// (2 6 3 7) at one place, a V load rows 0 1 2 3 (4 5 6 7): rows whose lines coincide are moved by 32
// or 64 bytes so that either set covers all banks.
template <int ROWB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  const int h = ((r >> 1) ^ (r >> 2)) & 1;
  if constexpr (ROWB == 32) return (uint32_t)((r ^ ((r >> 1) & 2)) * 32 + c * 16);
  else if constexpr (ROWB == 64) return (uint32_t)(r * 64 + ((c ^ (h << 1)) * 16));
  else return (uint32_t)(r * ROWB + ((c ^ (((r & 1) << 1) | (h << 2))) * 16));
}

// Key of the 16-key block that the MMA's row i stands for.
__device__ __forceinline__ int key_of_row(int i) { return (i & 8) | ((i & 7) >> 1) | ((i & 1) << 2); }

// Keys that some row of sequence b sees at most, and its pieces of work (at least one: a unit without
// keys still writes its zeros).
__device__ __forceinline__ int sequence_keys(const Params& p, int b) {
  const long long cap = min((long long)p.max_pages * p.c.page_size, (long long)INT_MAX);
  const int n = p.lens[b];
  return n < 0 ? 0 : (int)min((long long)n, cap);
}

template <class C>
__device__ __forceinline__ int pieces(int keys) { return max(1, (keys + C::SPLIT - 1) / C::SPLIT); }

template <class C>
__global__ void __launch_bounds__(kThreads, C::CTAS) attn_paged_kernel(const Params p) {
  constexpr int D = C::D, NT = C::NT, KT = C::KT, KB = KT / 16, GROUPS = C::GROUPS;
  constexpr bool INT4 = C::INT4;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ long long s_scan[kThreads];
  __shared__ long long s_base;
  __shared__ int s_first;
  __shared__ float s_m[kWarps][C::ROWS], s_l[kWarps][C::ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int per_seq = p.c.Hkv * p.row_blocks;   // units of a sequence

  // My share of all pieces: total and, for its first piece, the sequence it lies in.
  long long mine = 0;
  const int each = (p.B + kThreads - 1) / kThreads;
  for (int b = tid * each; b < min(p.B, (tid + 1) * each); ++b) mine += (long long)pieces<C>(sequence_keys(p, b)) * per_seq;
  s_scan[tid] = mine;
  __syncthreads();
  for (int o = 1; o < kThreads; o <<= 1) {
    const long long x = tid >= o ? s_scan[tid - o] : 0;
    __syncthreads();
    s_scan[tid] += x;
    __syncthreads();
  }
  const long long total = s_scan[kThreads - 1];
  const long long ctas = min((long long)gridDim.x, total);
  const long long cta = blockIdx.x;
  if (tid == 0) p.cut[cta] = make_int4(0, 0, -1, 0);
  if (cta >= ctas) return;
  const long long first = cta * total / ctas, last = (cta + 1) * total / ctas;
  {
    long long base = s_scan[tid] - mine;
    if (mine > 0 && base <= first && first < base + mine) {
      int b = tid * each;
      for (;; ++b) {
        const long long n = (long long)pieces<C>(sequence_keys(p, b)) * per_seq;
        if (first < base + n) break;
        base += n;
      }
      s_first = b;
      s_base = base;
    }
  }
  __syncthreads();
  int b = s_first;
  long long seq_base = s_base;
  const uint32_t buf = smem_u32(ring) + warp * C::WARP_BYTES;
  float* part_of_warp = reinterpret_cast<float*>(ring + warp * C::WARP_BYTES);

  for (long long at = first; at < last;) {
    // The unit that piece `at` belongs to, and my pieces [p0, p1) of it.
    int keys = sequence_keys(p, b), np = pieces<C>(keys);
    while (at >= seq_base + (long long)np * per_seq) {
      seq_base += (long long)np * per_seq;
      ++b;
      keys = sequence_keys(p, b);
      np = pieces<C>(keys);
    }
    if (keys < p.lens[b] || p.lens[b] < 0)
      if (tid == 0) atomicCAS(p.status, 0u, kStatusBadPage);
    const int unit = (int)((at - seq_base) / np);
    const long long unit_base = seq_base + (long long)unit * np;
    const int p0 = (int)(at - unit_base), p1 = (int)min((long long)np, last - unit_base);
    const int hkv = unit / p.row_blocks, row0 = unit % p.row_blocks * C::ROWS, rows = p.Nq * p.G;
    const int key0 = p0 * C::SPLIT + warp * KT, tiles = p1 - p0;
    const uint8_t* kbase = p.c.k + hkv * p.c.head_b;
    const uint8_t* vbase = p.c.v + hkv * p.c.head_b;
    const uint8_t* ksz = p.c.k_sz + hkv * p.c.sz_head_b;
    const uint8_t* vsz = p.c.v_sz + hkv * p.c.sz_head_b;
    const int* pages = p.table + b * p.table_stride;

    // A tile's copies: lane i < KB finds where 16-key block i begins (bytes into k and v, and into the
    // pairs; -1: nowhere), one tile ahead of the copies themselves.
    struct Place {
      long long row, sz;
    };
    auto look_up = [&](int n) -> Place {
      const int key = key0 + n * C::SPLIT + lane * 16;
      Place at{-1, -1};
      if (lane < KB && n < tiles && key < keys) {
        const uint32_t block = key >> 4, e = block / p.blocks_per_page;
        const int page = pages[e], in_page = (block - e * p.blocks_per_page.v) << 4;
        if (page >= 0 && page < p.c.num_pages) {
          at.row = page * p.c.page_b + in_page * p.c.token_b;
          if (INT4) at.sz = page * p.c.sz_page_b + in_page * p.c.sz_token_b;
        } else {
          atomicCAS(p.status, 0u, kStatusBadPage);
        }
      }
      return at;
    };
    constexpr int CH = C::ROWB / 16, RPI = 32 / CH;   // chunks of a row, rows of one copy instruction
    const long long my_row = (lane / CH) * p.c.token_b + lane % CH * 16;
    auto fetch = [&](int n, const Place& place) {
      if (n < tiles) {
        const uint32_t dst = buf + n % C::STAGES * C::STAGE;
        const int valid = keys - (key0 + n * C::SPLIT);
#pragma unroll
        for (int i = 0; i < KT / RPI; ++i) {
          const int r = i * RPI + lane / CH;
          const long long base = __shfl_sync(0xffffffffu, place.row, i * RPI / 16);
          const bool in = base >= 0 && r < valid;
          const long long row = in ? base + my_row + i * RPI % 16 * p.c.token_b : 0;
          const uint32_t d = dst + chunk_at<C::ROWB>(r, lane % CH);
          copy16(d, kbase + row, in);
          copy16(d + C::V_OFF, vbase + row, in);
        }
        if constexpr (INT4) {
          const long long base = __shfl_sync(0xffffffffu, place.sz, lane / 16);
          const bool in = base >= 0 && lane < valid;
          const long long row = in ? base + lane % 16 * p.c.sz_token_b : 0;
          copy_small<C::SZB>(dst + C::KSZ_OFF + lane * C::SZB, ksz + row, in);
          copy_small<C::SZB>(dst + C::VSZ_OFF + lane * C::SZB, vsz + row, in);
        }
      }
      copies_commit();
    };

    Place page = look_up(0);
#pragma unroll
    for (int n = 0; n < C::STAGES - 1; ++n) {
      const Place next = look_up(n + 1);
      fetch(n, page);
      page = next;
    }

    // Query rows as the B operand: lane (g, t) holds row g's values that its K bytes are paired with.
    constexpr int QR = D / 16;
    uint32_t qf[NT][QR][2];
    float mult[NT][2];            // S = mult * (what the products give), per column 2t, 2t + 1
    float qsum[NT][GROUPS][2];    // 4 bits: sums of q over a group, in units of the products
    float out[NT][2];             // what a masked product is set to, so that S is -inf
    int limit[NT][2];             // keys the column's row sees: key < limit
    int least = INT_MAX;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      const bool in = r < rows;
      const __nv_bfloat16* src =
          p.q + (((long long)b * p.Nq + (in ? r / p.G : 0)) * p.H + hkv * p.G + (in ? r % p.G : 0)) * D;
      if constexpr (INT4) {
        uint4 raw[GROUPS][2];
        float top = 0.f, sum[GROUPS];
#pragma unroll
        for (int gr = 0; gr < GROUPS; ++gr) {
          sum[gr] = 0.f;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            raw[gr][w] = in ? *reinterpret_cast<const uint4*>(src + gr * 64 + 16 * t + 8 * w) : make_uint4(0, 0, 0, 0);
            const uint32_t u[4] = {raw[gr][w].x, raw[gr][w].y, raw[gr][w].z, raw[gr][w].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = __uint_as_float(u[i] << 16), y = __uint_as_float(u[i] & 0xffff0000u);
              sum[gr] += x + y;
              top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
            }
          }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
          for (int gr = 0; gr < GROUPS; ++gr) sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], o);
        }
        // q 2^-e has its greatest value in [2^11, 2^12): normal in fp16 down to 2^-21 of it after the 1/16
        const int e = top > 0.f ? min(max((int)(__float_as_uint(top) >> 23) - 127 - 11, -120), 120) : 0;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int gr = 0; gr < GROUPS; ++gr) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t u[4] = {raw[gr][w].x, raw[gr][w].y, raw[gr][w].z, raw[gr][w].w};
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[2 * i] = __uint_as_float(u[i] << 16) * down;
              x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u) * down;
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {   // word's codes (0, 4), (1, 5) then (2, 6), (3, 7)
              qf[nt][gr * 4 + 2 * w + s][0] = pack_half2(x[2 * s], x[2 * s + 4]);
              qf[nt][gr * 4 + 2 * w + s][1] = pack_half2(x[2 * s + 1] * 0.0625f, x[2 * s + 5] * 0.0625f);
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) qsum[nt][gr][j] = __shfl_sync(0xffffffffu, sum[gr] * down * 0x1p-24f, (2 * t + j) * 4);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) mult[nt][j] = __shfl_sync(0xffffffffu, up, (2 * t + j) * 4) * p.scale_log2 * 0x1p24f;
      } else {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 x = in ? *reinterpret_cast<const uint4*>(src + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
          qf[nt][2 * j][0] = x.x;
          qf[nt][2 * j][1] = x.y;
          qf[nt][2 * j + 1][0] = x.z;
          qf[nt][2 * j + 1][1] = x.w;
        }
        mult[nt][0] = mult[nt][1] = p.scale_log2;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = row0 + nt * 8 + 2 * t + j;
        if (mult[nt][j] == 0.f) mult[nt][j] = 0x1p-126f;   // 0 times the masked infinity would be NaN
        out[nt][j] = mult[nt][j] < 0.f ? INFINITY : -INFINITY;
        limit[nt][j] = p.causal ? (c < rows ? keys - p.Nq + 1 + c / p.G : keys) : keys;
        least = min(least, limit[nt][j]);
      }
    }
    least = min(least, __shfl_xor_sync(0xffffffffu, least, 1));
    least = min(least, __shfl_xor_sync(0xffffffffu, least, 2));

    float acc[NT][D / 16][4];
    float m[NT][2], l[NT][2], z[NT][INT4 ? GROUPS : 1][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[nt][i][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
#pragma unroll
        for (int gr = 0; gr < (INT4 ? GROUPS : 1); ++gr) z[nt][gr][j] = 0.f;
      }
    }

    for (int n = 0; n < tiles; ++n) {
      copies_wait<C::STAGES - 2>();
      __syncwarp();
      {
        const Place next = look_up(n + C::STAGES);
        fetch(n + C::STAGES - 1, page);
        page = next;
      }
      const uint32_t tile = buf + n % C::STAGES * C::STAGE;
      const int tile_key = key0 + n * C::SPLIT;
      float s[KB][NT][4], ev[KB][2];
      uint32_t vs[KB][2][GROUPS];   // (scale, zero) of my two values' rows
      // S^T = K q^T
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int r0 = kb * 16 + key_of_row(g), r1 = r0 + 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[kb][nt][j] = 0.f;
        if constexpr (INT4) {
          uint32_t ks[2][GROUPS];
          load_pairs<GROUPS>(ks[0], tile + C::KSZ_OFF + r0 * C::SZB);
          load_pairs<GROUPS>(ks[1], tile + C::KSZ_OFF + r1 * C::SZB);
          load_pairs<GROUPS>(vs[kb][0], tile + C::VSZ_OFF + r0 * C::SZB);
          load_pairs<GROUPS>(vs[kb][1], tile + C::VSZ_OFF + r1 * C::SZB);
#pragma unroll
          for (int gr = 0; gr < GROUPS; ++gr) {
            const uint32_t place = (t & 1) * 8;
            const uint2 w0 = lds64(tile + chunk_at<C::ROWB>(r0, gr * 2 + (t >> 1)) + place);
            const uint2 w1 = lds64(tile + chunk_at<C::ROWB>(r1, gr * 2 + (t >> 1)) + place);
            float c[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) c[nt][j] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t x0 = (k < 2 ? w0.x : w0.y) >> (k % 2 * 8), x1 = (k < 2 ? w1.x : w1.y) >> (k % 2 * 8);
              const uint32_t a0 = x0 & 0x000f000fu, a1 = x1 & 0x000f000fu, a2 = x0 & 0x00f000f0u, a3 = x1 & 0x00f000f0u;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<true>(c[nt], a0, a1, a2, a3, qf[nt][gr * 4 + k][0], qf[nt][gr * 4 + k][1]);
            }
            const float sc0 = __uint_as_float(ks[0][gr] << 16), zr0 = __uint_as_float(ks[0][gr] & 0xffff0000u);
            const float sc1 = __uint_as_float(ks[1][gr] << 16), zr1 = __uint_as_float(ks[1][gr] & 0xffff0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                s[kb][nt][j] = fmaf(c[nt][j], sc0, fmaf(zr0, qsum[nt][gr][j], s[kb][nt][j]));
                s[kb][nt][2 + j] = fmaf(c[nt][2 + j], sc1, fmaf(zr1, qsum[nt][gr][j], s[kb][nt][2 + j]));
              }
          }
          // exponent of the greatest value scale, one more so that scale 2^-e < 1
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t e = 0;
#pragma unroll
            for (int gr = 0; gr < GROUPS; ++gr) e = max(e, vs[kb][i][gr] & 0x7f80u);
            ev[kb][i] = fmaxf(__uint_as_float(0x4b000000u | (e >> 7)) - (0x1p23f + 126.f), kMinExp);
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 x0 = lds128(tile + chunk_at<C::ROWB>(r0, 4 * j + t)), x1 = lds128(tile + chunk_at<C::ROWB>(r1, 4 * j + t));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<false>(s[kb][nt], x0.x, x1.x, x0.y, x1.y, qf[nt][2 * j][0], qf[nt][2 * j][1]);
              mma<false>(s[kb][nt], x0.z, x1.z, x0.w, x1.w, qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
            }
          }
          ev[kb][0] = ev[kb][1] = 0.f;
        }
        if (tile_key + KT > least) {   // the same for the whole warp
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (tile_key + r0 >= limit[nt][j]) s[kb][nt][j] = out[nt][j];
              if (tile_key + r1 >= limit[nt][j]) s[kb][nt][2 + j] = out[nt][j];
            }
        }
      }
      // Running maximum of S + exponent, rescale of what was summed under an older one.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = -INFINITY;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            x = fmaxf(x, fmaxf(fmaf(s[kb][nt][j], mult[nt][j], ev[kb][0]), fmaf(s[kb][nt][2 + j], mult[nt][j], ev[kb][1])));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
          top[j] = fmaxf(x, m[nt][j]);
        }
        if (__any_sync(0xffffffffu, top[0] != m[nt][0] || top[1] != m[nt][1])) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = m[nt][j] == -INFINITY ? 0.f : exp2_fast(m[nt][j] - top[j]);
            m[nt][j] = top[j];
            l[nt][j] *= f;
#pragma unroll
            for (int gr = 0; gr < (INT4 ? GROUPS : 1); ++gr) z[nt][gr][j] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              acc[nt][i][j] *= f;
              acc[nt][i][2 + j] *= f;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float ref = m[nt][j] == -INFINITY ? 0.f : m[nt][j];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            s[kb][nt][j] = exp2_fast(fmaf(s[kb][nt][j], mult[nt][j], -ref));
            s[kb][nt][2 + j] = exp2_fast(fmaf(s[kb][nt][2 + j], mult[nt][j], -ref));
            l[nt][j] += s[kb][nt][j] + s[kb][nt][2 + j];
          }
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int v0 = kb * 16 + t;
        if constexpr (INT4) {
#pragma unroll
          for (int gr = 0; gr < GROUPS; ++gr) {
            const uint32_t sv0 = vs[kb][0][gr], sv1 = vs[kb][1][gr];
            const float sc0 = __uint_as_float(sv0 << 16), zr0 = __uint_as_float(sv0 & 0xffff0000u);
            const float sc1 = __uint_as_float(sv1 << 16), zr1 = __uint_as_float(sv1 & 0xffff0000u);
            uint32_t b0[NT], b1[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float(&q)[4] = s[kb][nt];
              b0[nt] = transpose8x8(pack_half2(q[0] * sc0, q[1] * sc0));
              b1[nt] = transpose8x8(pack_half2(q[2] * sc1, q[3] * sc1));
              z[nt][gr][0] += q[0] * zr0 + q[2] * zr1;
              z[nt][gr][1] += q[1] * zr0 + q[3] * zr1;
            }
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = lds32(tile + C::V_OFF + chunk_at<C::ROWB>(v0 + 4 * i, gr * 2 + (g >> 2)) + (g & 3) * 4);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t sel = half ? 0x7632u : 0x5410u;
              const uint32_t x = __byte_perm(w[0], w[1], sel), y = __byte_perm(w[2], w[3], sel);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t xs = x >> (8 * k), ys = y >> (8 * k);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma<true>(acc[nt][gr * 4 + 2 * half + k], xs & 0x000f000fu, xs & 0x00f000f0u, ys & 0x000f000fu,
                            ys & 0x00f000f0u, b0[nt], b1[nt]);
              }
            }
          }
        } else {
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            b0[nt] = transpose8x8(pack_bf162(s[kb][nt][0], s[kb][nt][1]));
            b1[nt] = transpose8x8(pack_bf162(s[kb][nt][2], s[kb][nt][3]));
          }
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = lds128(tile + C::V_OFF + chunk_at<C::ROWB>(v0 + 4 * i, 8 * j + g));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u0 = i == 0 ? w[0].x : i == 1 ? w[0].y : i == 2 ? w[0].z : w[0].w;
              const uint32_t u1 = i == 0 ? w[1].x : i == 1 ? w[1].y : i == 2 ? w[1].z : w[1].w;
              const uint32_t u2 = i == 0 ? w[2].x : i == 1 ? w[2].y : i == 2 ? w[2].z : w[2].w;
              const uint32_t u3 = i == 0 ? w[3].x : i == 1 ? w[3].y : i == 2 ? w[3].z : w[3].w;
              const uint32_t a0 = __byte_perm(u0, u1, 0x5410), a1 = __byte_perm(u0, u1, 0x7632);
              const uint32_t a2 = __byte_perm(u2, u3, 0x5410), a3 = __byte_perm(u2, u3, 0x7632);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<false>(acc[nt][j * 4 + i], a0, a1, a2, a3, b0[nt], b1[nt]);
            }
          }
        }
      }
      __syncwarp();   // all lanes have read the tile before its slot is filled again
    }
    copies_wait<0>();
    __syncthreads();

    // Join the warps: each weighs its part by exp2(its maximum - the CTA's).
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], o);
          if constexpr (INT4) {
#pragma unroll
            for (int gr = 0; gr < GROUPS; ++gr) z[nt][gr][j] += __shfl_xor_sync(0xffffffffu, z[nt][gr][j], o);
          }
        }
        if (g == 0) {
          s_m[warp][nt * 8 + 2 * t + j] = m[nt][j];
          s_l[warp][nt * 8 + 2 * t + j] = l[nt][j];
        }
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = nt * 8 + 2 * t + j;
        float top = s_m[0][c];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][c]);
        const float f = m[nt][j] == -INFINITY ? 0.f : exp2_fast(m[nt][j] - top);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          float x = acc[nt][i][j], y = acc[nt][i][2 + j];
          if constexpr (INT4) {
            x = x * 0x1p24f + z[nt][i / 4][j];
            y = y * 0x1p20f + z[nt][i / 4][j];
          }
          // MMA rows g, g + 8 of tile i are dims 64 (i / 4) + 8 g + 2 (i % 4) and the next
          *reinterpret_cast<float2*>(part_of_warp + c * D + i / 4 * 64 + 8 * g + i % 4 * 2) = make_float2(x * f, y * f);
        }
      }
    __syncthreads();
    const bool whole = p0 == 0 && p1 == np;
    const long long slot = 2 * cta + (p0 == 0 ? 1 : 0);
    for (int i = tid; i < C::ROWS * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float top = s_m[0][r], sum = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (s_m[w][r] > -INFINITY) sum += s_l[w][r] * exp2_fast(s_m[w][r] - top);
        const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring + w * C::WARP_BYTES) + r * D + c);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
      const float lse2 = sum > 0.f ? top + log2f(sum) : -INFINITY;
      if (!whole) {
        *reinterpret_cast<float4*>(p.part_o + (slot * C::ROWS + r) * D + c) = x;
        if (c == 0) p.part_lse[slot * C::ROWS + r] = lse2;
      } else if (row0 + r < rows) {
        const int qi = (row0 + r) / p.G, h = hkv * p.G + (row0 + r) % p.G;
        uint2 y;
        y.x = pack_bf162(x.x, x.y);
        y.y = pack_bf162(x.z, x.w);
        *reinterpret_cast<uint2*>(p.o + (((long long)b * p.Nq + qi) * p.H + h) * D + c) = y;
        if (c == 0) p.lse[((long long)b * p.H + h) * p.Nq + qi] = lse2 * 0.69314718055994531f;
      }
    }
    if (p0 == 0 && !whole && tid == 0) {
      // the CTA that holds the unit's last piece: the last c with c total / ctas < its end
      const long long end = unit_base + np - 1;
      long long c = (end * ctas) / total;
      while ((c + 1) * total / ctas <= end) ++c;
      while (c * total / ctas > end) --c;
      p.cut[cta] = make_int4(b, unit, (int)c, 0);
    }
    __syncthreads();   // the ring is free again
    at = unit_base + p1;
  }
}

// Joins the parts of the units that were cut: CTA (c, r) takes row r of the unit that begins in CTA c.
// LSE = log2 sum 2^LSE_i,  O = sum 2^(LSE_i - LSE) O_i.
template <int D>
__global__ void __launch_bounds__(128) attn_paged_join_kernel(const Params p, int rows_per_unit) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int LANES = D / 4, WAYS = 128 / LANES;
  const int4 cut = p.cut[blockIdx.x];
  const int r = blockIdx.y, hkv = cut.y / p.row_blocks, row = cut.y % p.row_blocks * rows_per_unit + r;
  if (cut.z < 0 || row >= p.Nq * p.G) return;
  const int parts = cut.z - (int)blockIdx.x + 1;
  const int tid = threadIdx.x, c = tid % LANES * 4, way = tid / LANES;
  // part 0 is slot 2c + 1 of CTA c, part i > 0 slot 2 (c + i)
  auto at = [&](int i) -> long long {
    return ((i == 0 ? 2LL * blockIdx.x + 1 : 2LL * (blockIdx.x + i)) * rows_per_unit + r);
  };
  __shared__ float s_top[128], s_sum[WAYS];
  __shared__ float4 s_x[128];
  float top = -INFINITY;
  for (int i = tid; i < parts; i += 128) top = fmaxf(top, p.part_lse[at(i)]);
  s_top[tid] = top;
  __syncthreads();
  for (int o = 64; o > 0; o >>= 1) {
    if (tid < o) s_top[tid] = fmaxf(s_top[tid], s_top[tid + o]);
    __syncthreads();
  }
  top = s_top[0];
  float sum = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (top > -INFINITY) {
#pragma unroll 4
    for (int i = way; i < parts; i += WAYS) {
      const float f = exp2_fast(p.part_lse[at(i)] - top);
      const float4 y = *reinterpret_cast<const float4*>(p.part_o + at(i) * D + c);
      sum += f;
      x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
    }
  }
  s_x[tid] = x;
  if (c == 0) s_sum[way] = sum;
  __syncthreads();
  if (way == 0) {
    for (int w = 1; w < WAYS; ++w) {
      const float4 y = s_x[w * LANES + tid];
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      sum += s_sum[w];
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int qi = row / p.G, h = hkv * p.G + row % p.G;
    uint2 y;
    y.x = pack_bf162(x.x * inv, x.y * inv);
    y.y = pack_bf162(x.z * inv, x.w * inv);
    *reinterpret_cast<uint2*>(p.o + (((long long)cut.x * p.Nq + qi) * p.H + h) * D + c) = y;
    if (c == 0)
      p.lse[((long long)cut.x * p.H + h) * p.Nq + qi] = sum > 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
  }
}

struct Plan {
  int rows_per_unit, row_blocks, grid, split;
};

// Rows a unit holds (8, or 16 at d <= 128 when a call has more than 8: d = 256 has no registers for
// them) and the CTAs that fill the device.
template <int D, bool INT4>
Plan plan_for(int rows, int sms) {
  constexpr int NT2 = D <= 128 ? 2 : 1;
  const bool two = rows > 8 && NT2 == 2;
  const int per = two ? 16 : 8;
  return {per, (rows + per - 1) / per, sms * (two ? Cfg<D, INT4, NT2>::CTAS : Cfg<D, INT4, 1>::CTAS), Cfg<D, INT4, 1>::SPLIT};
}

Plan make_plan(int d, bool int4, int rows, int sms) {
  switch (d) {
    case 64: return int4 ? plan_for<64, true>(rows, sms) : plan_for<64, false>(rows, sms);
    case 128: return int4 ? plan_for<128, true>(rows, sms) : plan_for<128, false>(rows, sms);
    default: return int4 ? plan_for<256, true>(rows, sms) : plan_for<256, false>(rows, sms);
  }
}

template <class C>
cudaError_t launch(const Params& p, int grid, cudaStream_t s) {
  auto kernel = attn_paged_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, C::SMEM, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)std::min(C::ROWS, p.Nq * p.G));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<C::D>, p, C::ROWS);
}

template <int D, bool INT4>
cudaError_t launch_rows(const Params& p, int rows_per_unit, int grid, cudaStream_t s) {
  if constexpr (D <= 128) {
    if (rows_per_unit == 16) return launch<Cfg<D, INT4, 2>>(p, grid, s);
  }
  return launch<Cfg<D, INT4, 1>>(p, grid, s);
}

size_t pad(size_t x) { return (x + 255) / 256 * 256; }

// Bytes of the parts, of their LSE, and of the cut units.
void workspace_parts(const Plan& pl, int d, size_t (&n)[3]) {
  n[0] = pad((size_t)2 * pl.grid * pl.rows_per_unit * d * 4);
  n[1] = pad((size_t)2 * pl.grid * pl.rows_per_unit * 4);
  n[2] = pad((size_t)pl.grid * sizeof(int4));
}

bool shape_ok(int B, int H, int Hkv, int Nq) { return B >= 1 && H >= 1 && Hkv >= 1 && Nq >= 1 && H % Hkv == 0; }

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" size_t attn_fwd_paged_workspace_bytes(int B, int H, int Hkv, int Nq, int d, attn_cache_type_t type) {
  if (!shape_ok(B, H, Hkv, Nq) || (d != 64 && d != 128 && d != 256)) return 0;
  if (type != ATTN_CACHE_BF16 && type != ATTN_CACHE_INT4) return 0;
  if ((long long)Nq * (H / Hkv) > INT_MAX / 2) return 0;
  int sms = 152;
  uint32_t* status;
  device_state(&sms, &status);
  size_t n[3];
  workspace_parts(make_plan(d, type == ATTN_CACHE_INT4, Nq * (H / Hkv), sms), d, n);
  return n[0] + n[1] + n[2];
}

extern "C" attn_status_t attn_fwd_paged(const void* q, const attn_paged_cache_t* cache, void* o, float* lse,
                                        const int* page_table, long long table_stride, int max_pages,
                                        const int* seqlens, int B, int H, int Nq, float scale, int causal,
                                        void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  Params p = {};
  const attn_status_t st = paged_cache_args(cache, &p.c);
  if (st != ATTN_OK) return st;
  const int d = cache->d, Hkv = cache->Hkv;
  if (!shape_ok(B, H, Hkv, Nq) || max_pages < 1 || table_stride < 0 || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (!q || !o || !lse || !page_table || !seqlens || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(o, 16) || !is_aligned(lse, 4) || !is_aligned(page_table, 4) ||
      !is_aligned(seqlens, 4) || !is_aligned(workspace, 256))
    return ATTN_ERR_INVALID_ARG;
  if (scale == 0.f) return ATTN_ERR_UNSUPPORTED;   // as attn_fwd
  const long long rows = (long long)Nq * (H / Hkv);
  if (rows > INT_MAX / 2 || (long long)B * H * Nq > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  int sms;
  if (!device_state(&sms, &p.status)) return ATTN_ERR_CUDA;
  const bool bits4 = cache->type == ATTN_CACHE_INT4;
  const Plan pl = make_plan(d, bits4, (int)rows, sms);
  size_t n[3];
  workspace_parts(pl, d, n);
  if (workspace_bytes < n[0] + n[1] + n[2]) return ATTN_ERR_INVALID_ARG;
  if ((long long)Hkv * pl.row_blocks > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  struct {
    const void* b;
    size_t n;
  } x[4] = {{o, (size_t)B * Nq * H * d * 2}, {lse, (size_t)B * Nq * H * 4}, {workspace, n[0] + n[1] + n[2]}, {q, (size_t)B * Nq * H * d * 2}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 4; ++j) {
      const uintptr_t a = (uintptr_t)x[i].b, b = (uintptr_t)x[j].b;
      if (a < b + x[j].n && b < a + x[i].n) return ATTN_ERR_INVALID_ARG;
    }
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.table = page_table, p.table_stride = table_stride, p.lens = seqlens;
  p.B = B, p.H = H, p.G = H / Hkv, p.Nq = Nq, p.max_pages = max_pages, p.row_blocks = pl.row_blocks;
  p.causal = causal != 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.blocks_per_page = fast_div((uint32_t)cache->page_size / 16);
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + n[0]);
  p.cut = reinterpret_cast<::int4*>(static_cast<uint8_t*>(workspace) + n[0] + n[1]);
  // No more CTAs than pieces of work there can be.
  const long long most = (long long)B * Hkv * pl.row_blocks * std::max<long long>(1, ((long long)max_pages * cache->page_size + pl.split - 1) / pl.split);
  const int grid = (int)std::min<long long>(pl.grid, most);
  cudaError_t e;
  switch (d) {
    case 64: e = bits4 ? launch_rows<64, true>(p, pl.rows_per_unit, grid, stream) : launch_rows<64, false>(p, pl.rows_per_unit, grid, stream); break;
    case 128: e = bits4 ? launch_rows<128, true>(p, pl.rows_per_unit, grid, stream) : launch_rows<128, false>(p, pl.rows_per_unit, grid, stream); break;
    default: e = bits4 ? launch_rows<256, true>(p, pl.rows_per_unit, grid, stream) : launch_rows<256, false>(p, pl.rows_per_unit, grid, stream); break;
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

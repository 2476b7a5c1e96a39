// Attention over a paged key/value cache in bf16 or 4 bits, for few query rows a sequence (decode, drafted tokens):
//   S = scale q k^T over the keys a row sees,  O = softmax(S) V,  LSE.
//
// The cache is read once and that bounds the call: 4 d bytes a key and kv head in bf16, d + d / 8 in 4 bits. All query
// rows that share a kv head (Nq tokens x H / Hkv heads) are columns of one narrow product,
//   S^T [keys x rows] = K [keys x d] q^T,     O^T [d x rows] = V^T [d x keys] P^T,
// with m16n8k16: the long dims (keys, d) fill the 16 and a call pads its rows only to 8. tcgen05 would pad them to 128
// and needs unpacked operands in shared memory, more traffic than the cache itself.
//
// 4-bit codes go to the tensor cores as they are. A code c in the low bits of a half is the subnormal fp16 number
// c 2^-24, and 4 bits higher it is 16 c 2^-24: a pair of operands costs one AND. For keys the factor 16 is taken out of
// the query's matching values; for values a pair of rows sums low codes and whole bytes, low + 16 high, whose difference
// is taken once at the end. Scale and zero stay outside the products, in fp32:
//   q.k = sum over groups  scale (codes . q) + zero sum(q),
//   O   = (sum_j (p_j scale_j) codes_j + sum_j p_j zero_j) / sum_j p_j.
// Roundings: q is scaled by a power of two per row, so fp16 holds it exactly where it counts (2^-25 of the row's greatest
// value). Weights go into the second product as a sum of two numbers. In one bf16 number, 2^-8 off, p_j would add as much to
// O's error as its own rounding (0.0023 instead of 0.0017 of its norm); two are 2^-16 off, and the second product costs
// nothing beside the cache's bytes. p_j scale_j in one fp16 number, 2^-11 off, moves O by 0.0011 of its norm (codes are
// summed with their offset apart, so that a weight's rounding counts twice the value's size) and by any share of it where
// zero and codes cancel; two are 2^-22 off and cost 12% with 5 to 8 rows, 19% with more. With at most 4 rows they cost 2%:
// half the columns would be padding, so that columns c and c + 4 take one query row, and the first takes the weights'
// first number, the second the other (B 8, 16384 keys, 4 rows: 34.8 us in one number, 35.5 so, 38.7 with two products;
// B 32, up to 32768 keys: 98.7, 100.2, 112.4).
// For p_j scale_j to stay within fp16 at any scale, the running maximum is taken over S + log2 of the key's scale (its exponent)
// instead of S; with several groups of dims, each has a power of two of its own that follows its own scales, so that a group
// keeps its bits beside one far larger (5% with 4 rows, 35.6 -> 37.2 and 100.3 -> 106 us, 1% with more; one factor for all
// lost the codes of a group 2^-14 as large).
// Products of 16 keys are added up outside the tensor cores: chained, they left an error of 0.0065 of O's norm at 48 sequences
// of 32768 keys and 0.026 at 64 of 65536, added 0.0016 (at most 4 rows 1% slower, 8 rows 39.7 -> 42.4 us, 12 rows 68.5 -> 72.5).
//
// Work: a sequence's keys are cut into tiles of KT; a unit is the tiles of one (sequence, kv head, block of query rows).
// All units in order, each OVERHEAD tiles longer than it is, are dealt to all warps in equal contiguous shares, so ragged
// batches load every SM alike. A warp streams through its share alone: query rows, keys and values go through a ring of
// its own in shared memory, filled by 16-byte asynchronous copies that run ahead across the ends of units. A unit inside
// one share is finished by its warp. One that is cut leaves normalised parts with their LSE: what the warps of a CTA hold
// of one unit when their shares end is joined there, the rest by a second, dependent launch. The shares follow from the
// lengths alone: the same bits on every run, no atomics.
//
// Matrix loads hand out the operands, those of V transposed: a 16-bit unit of them is one bf16 value or four codes.
//
// Measured on a GB300 (us in a CUDA graph, share of the copy bandwidth; H 32, Hkv 8, d 128 if not said otherwise):
//   bf16, B 8, 16384 keys                85.5  93%
//   4 bits, B 8, 16384 keys              37.5  59%: about 5 us until the first tiles are there and 5 us to join the parts
//   4 bits, B 32, up to 32768 keys       106   79%: issue slots 60%, ALU 53%; three warps a scheduler wait for their own results
//   4 bits, B 16, H 96 (12 rows), 13400 keys  92    40%: two warps a scheduler, 254 registers
//   bf16, d 256, B 13, up to 5000 keys, 12 rows (two blocks, the second out of L2)  35    52%
// What it took before weights came in two numbers, at B 8 and 16384 keys in 4 bits: tiles of one CTA with lane-wise operand
// loads 61; pages looked up once a tile 48.6; matrix loads, shares by warp, a vote instead of the maximum's exchanges 40; one
// wave of shorter launches 36.
// OVERHEAD sets how even the shares are where units are short: a warp that got a sequence's empty units at one tile each held
// up a batch of 16 (4 bits, H 96, 165 to 20539 keys, one empty: 99 us, 72 at 4 tiles; the same sizes at equal lengths 74).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>
#include <utility>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "fastdiv.cuh"
#include "ops.h"
#include "paged.cuh"
#include "paged_host.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Least scale that counts in the running maximum: a weight then stays below 2^84, sums of weights and of weight
// times zero (at most 2^20 scales) far from overflow.
constexpr float kLeastScale = 0x1p-70f;

constexpr long long kMaxKeys = INT_MAX - 1023;   // keys a page table may hold: they are counted in 32 bits
constexpr float kNone = -1e30f;     // running maximum before the first key
constexpr float kHeadroom = 0x1p14f;   // weights of a bf16 cache may grow to this before the maximum is moved
// 4 bits: a move sets the greatest weight times scale below 2^6 (a group's own, where there are several); it may grow to
// 2^15 before the next. fp16 may lose 2^-25 of each: 2^-29 of the greatest, which is 2^4 at least.
constexpr float kTop = 6.f, kScaledHeadroom = 0x1p15f;

template <int D_, bool INT4_, int NT_, bool TWIN_ = false>
struct Cfg {
  static constexpr int D = D_, NT = NT_;
  static constexpr bool INT4 = INT4_, TWIN = TWIN_;      // TWIN: columns c and c + 4 hold one query row (at most 4 rows)
  static constexpr int KT = INT4 ? 32 : 16;              // keys of a tile
  static constexpr int OVERHEAD = INT4 ? 4 : 8;          // what beginning and ending a unit costs, in tiles
  static constexpr int ROWS = 8 * NT;                    // query rows of a unit
  static constexpr int GROUPS = D / kInt4Group;
  static constexpr bool UP = INT4 && GROUPS > 1;         // groups have powers of two of their own
  static constexpr int ROWB = INT4 ? D / 2 : 2 * D;      // bytes of a key's row
  static constexpr int SZB = INT4 ? 4 * GROUPS : 0;      // bytes of its (scale, zero) pairs
  // A slot of the ring: a tile's keys and values, or 8 query rows. At d = 256 in bf16 a tile takes two slots, keys then
  // values: two CTAs of four warps would not fit otherwise.
  static constexpr bool PAIR = INT4 || D < 256;
  static constexpr int V_OFF = PAIR ? KT * ROWB : 0, SZ_OFF = V_OFF + KT * ROWB, SZV_OFF = SZ_OFF + KT * SZB;
  static constexpr int SLOT = PAIR ? SZV_OFF + KT * SZB : KT * ROWB;
  static constexpr int SLOTS = 3;
  static constexpr int WARP_BYTES = SLOTS * SLOT;
  static constexpr int SMEM = kWarps * WARP_BYTES;
  static constexpr int CTAS = std::min(D * NT >= 256 ? 2 : 3, 233472 / (SMEM + 1024 + 2048));
  static_assert(WARP_BYTES >= ROWS * D * 4, "a warp's part of O is joined in its ring");
  static_assert(SLOT >= 16 * D && CTAS >= 1 && SLOT % 16 == 0, "ring");
};

struct Params {
  PagedCache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int *table, *lens;
  long long table_stride;
  int B, H, G, Nq, max_pages, row_blocks, causal;
  int table_lines;   // of 32 entries, of a sequence; 0 for tables of more than a line a thread, or 1 MB
  FastDiv blocks_per_page, div_g, div_blocks;   // 16-key blocks; heads of a group; row blocks of a kv head
  float scale_log2;
  // Parts of cut units, by warp w of the grid: 2w the one whose unit ends inside its share, 2w + 1 the one that the share
  // ends in, joined over the warps of the CTA from w on that hold the same unit.
  float* part_o;     // [2 warps, ROWS, D] normalised O
  float* part_lse;   // [2 warps, ROWS] log2-sum-exp2
  int4* cut;         // [warps]: (sequence, unit in it, warp with its last tile, whether that ends inside a share; -1: none)
  uint32_t* status;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Copies to dst + OFF in shared memory; zeros instead where `in` is false (the address must be readable all the same).
template <int OFF>
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0+%2], [%1], 16;" ::"r"(dst), "l"(src), "n"(OFF) : "memory");
}
template <int OFF>
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0+%3], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0), "n"(OFF)
               : "memory");
}
template <int OFF, int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0+%4], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(in ? N : 0), "n"(OFF)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Four 8x8 matrices of 16-bit values at a + OFF; lanes 8i .. 8i + 7 give the rows of matrix i. Lane (g, t) gets values 2t,
// 2t + 1 of row g, or with TRANS of column g.
template <bool TRANS, int OFF>
__device__ __forceinline__ uint4 load_matrices(uint32_t a) {
  uint4 x;
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a), "n"(OFF) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a), "n"(OFF) : "memory");
  return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
  return x;
}

// The (scale, zero) pairs of a row at a + OFF.
template <int OFF, int N>
__device__ __forceinline__ void load_pairs(uint32_t (&x)[N], uint32_t a) {
  if constexpr (N == 1)
    asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(x[0]) : "r"(a), "n"(OFF) : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2+%3];" : "=r"(x[0]), "=r"(x[1]) : "r"(a), "n"(OFF) : "memory");
  else
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(a), "n"(OFF) : "memory");
}

// Calls f with the constants 0 .. N - 1, for addresses that take them as immediates.
template <class F, int... I>
__device__ __forceinline__ void each_in(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each_of(F&& f) {
  each_in(f, std::make_integer_sequence<int, N>{});
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing summed yet.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bytes 1 and 3 as two 16-bit values.
__device__ __forceinline__ uint32_t high_bytes(uint32_t x) { return __byte_perm(x, 0, 0x4341); }
__device__ __forceinline__ uint32_t subtract_half2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_half2(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return pack_half2(a, b);
}
__device__ __forceinline__ uint64_t unpack_half2(uint32_t x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return f2_pack(f.x, f.y);
}
__device__ __forceinline__ uint32_t pack_bf162(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void add(float4& x, float f, const float4& y) {
  x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
}

__device__ __forceinline__ void add(float (&x)[4], const float (&y)[4]) {
  f2_unpack(f2_add(f2_pack(x[0], x[1]), f2_pack(y[0], y[1])), x[0], x[1]);
  f2_unpack(f2_add(f2_pack(x[2], x[3]), f2_pack(y[2], y[3])), x[2], x[3]);
}

// Byte offset of 16-byte chunk c of row r in a tile of rows of ROWB bytes: one chunk of 8 neighbouring rows, what a
// matrix load takes, meets every bank once.
template <int ROWB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  constexpr int LINE = ROWB < 128 ? 128 / ROWB : 1;               // rows of 128 bytes
  constexpr int MASK = ROWB < 128 ? ROWB / 16 - 1 : 7;
  return (uint32_t)(r * ROWB + ((c ^ (r / LINE & MASK)) * 16));
}

// Keys that some row of sequence b sees at most, and its pieces of work (at least one: a unit without
// keys still writes its zeros).
__device__ __forceinline__ int sequence_keys(const Params& p, int b) {
  const int n = p.lens[b];
  return min(max(n, 0), p.max_pages * p.c.page_size);   // a call with more than kMaxKeys is refused
}

// Which block of query rows the unit of a sequence has.
__device__ __forceinline__ int row_block(const Params& p, uint32_t unit) {
  return unit - unit / p.div_blocks * p.row_blocks;
}

template <class C>
__device__ __forceinline__ int tiles_of(int keys) { return (keys - 1) / C::KT + 1; }   // at least 1

// Where a warp is in its share: the next tile to plan for, its sequence, what that begins with; of the unit that is being
// copied the sequence, the first query row of its heads and of its block.
struct Cursor {
  int at, last, seq, seq_base, b, hkv, row0;
  long long q_row;
};

struct Unit {   // what a warp has to do of one unit: tiles [t0, t1) of nt
  int b, unit, t0, t1, nt, keys, end;
};

template <class C>
__global__ void __launch_bounds__(kThreads, C::CTAS) attn_paged_kernel(const Params p) {
  constexpr int D = C::D, NT = C::NT, KT = C::KT, KB = KT / 16, GROUPS = C::GROUPS, OV = C::OVERHEAD;
  constexpr bool INT4 = C::INT4;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int s_upto[kThreads];        // tiles of this warp's threads' sequences, up to each
  __shared__ Unit s_units[kWarps][4];     // units whose copies have begun, by turn
  __shared__ Cursor s_cursor[kWarps];     // here, not in registers: needed once a unit
  __shared__ int s_id[kWarps], s_open[kWarps];
  __shared__ float s_m[kWarps][C::ROWS], s_l[kWarps][C::ROWS];
  griddep_wait();   // launched early: what it reads may be a previous kernel's
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int per_seq = p.c.Hkv * p.row_blocks;   // units of a sequence

  // My share of all tiles: total and, for its beginning, the sequence it lies in.
  int mine = 0;
  const int each = (p.B + kThreads - 1) / kThreads;
  for (int b = tid * each; b < min(p.B, (tid + 1) * each); ++b) mine += (tiles_of<C>(sequence_keys(p, b)) + OV) * per_seq;
  // The tables are read a little later, by single lanes one entry after the other: small ones go into L2 meanwhile.
  const int line = blockIdx.x * kThreads + tid;
  if (line < p.B * p.table_lines) {
    const int b = line / p.table_lines;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + b * p.table_stride + (line - b * p.table_lines) * 32));
  }
  int upto = mine;   // of this warp's threads up to me
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  s_upto[tid] = upto;
  if (lane == 0) s_id[warp] = -1;
  __syncthreads();
  int total = 0, before[kWarps];   // of the warps before each
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before[w] = total;
    total += s_upto[32 * w + 31];
  }
  const int warps = min((int)gridDim.x * kWarps, total), me = blockIdx.x * kWarps + warp;
  const int part = total / warps, more = total - part * warps;         // the first `more` shares have one tile more
  auto share = [&](int w) { return w * part + min(w, more); };         // where warp w's begins
  if (lane == 0) p.cut[me] = make_int4(0, 0, -1, 0);

  const uint32_t buf = smem_u32(ring) + warp * C::WARP_BYTES, ring_end = buf + C::WARP_BYTES;
  if (me < warps) {
    // ---- copies: units in turn; of each its query rows (a slot for every 8), then keys and values of every tile
    volatile Cursor& cur = s_cursor[warp];
    {
      // The thread above whose sequences hold the share's beginning, and the tiles before them.
      const int first = share(me);
      int owner = 0;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) owner = first >= before[w] ? w : owner;
      const int base = before[0] + (owner == 0 ? 0 : owner == 1 ? before[1] : owner == 2 ? before[2] : before[3]);
      const uint32_t behind = __ballot_sync(0xffffffffu, base + s_upto[32 * owner + lane] <= first);
      const int j = __popc(behind);   // lanes whose sequences all end before
      if (lane == 0) {
        cur.at = first, cur.last = share(me + 1), cur.seq = (32 * owner + j) * each;
        cur.seq_base = base + (j > 0 ? s_upto[32 * owner + j - 1] : 0);
      }
    }
    __syncwarp();
    int f_turn = 0;              // units entered
    int f_q = NT, f_tile = 0, f_end = 0, f_keys = 0, f_rel = 0;   // query slots done; tile; its unit's last, keys; in a batch
    bool f_values = false, f_unit = false;
    long long at_row = -1, at_sz = -1;   // lane i: 16-key block i % KB of tile i / KB of a batch (bytes; -1: nowhere)
    int next_pages = -1;
    constexpr int PER = 32 / KB, CH = C::ROWB / 16, RPI = 32 / CH;   // tiles of a batch; chunks of a row, rows of a copy
    const long long my_row = (lane / CH) * p.c.token_b + lane % CH * 16, my_sz = lane % 16 * p.c.sz_token_b;
    uint32_t fill = buf;                 // slot that the next copies go to
    const uint32_t my_dst = chunk_at<C::ROWB>(lane / CH, lane % CH);

    auto look_up = [&](int first) -> int {   // pages of a batch of tiles, read one batch ahead
      const int tile = first + lane / KB, key = tile * KT + lane % KB * 16;
      if (tile >= f_end || key >= f_keys) return -1;
      return p.table[cur.b * p.table_stride + (uint32_t)(key >> 4) / p.blocks_per_page];
    };
    auto next_batch = [&]() {
      const int tile = f_tile + lane / KB, key = tile * KT + lane % KB * 16;
      const int page = next_pages;
      at_row = at_sz = -1;
      if (tile < f_end && key < f_keys) {
        const uint32_t block = key >> 4;
        const int in_page = (block - block / p.blocks_per_page * p.blocks_per_page.v) << 4, hkv = cur.hkv;
        if (page >= 0 && page < p.c.num_pages) {
          at_row = page * p.c.page_b + in_page * p.c.token_b + hkv * p.c.head_b;
          if (INT4) at_sz = page * p.c.sz_page_b + in_page * p.c.sz_token_b + hkv * p.c.sz_head_b;
        } else {
          atomicCAS(p.status, 0u, kStatusBadPage);
        }
      }
      next_pages = look_up(f_tile + PER);
    };
    // The next unit of my share that has tiles in it; f_unit false when there is none.
    auto enter = [&]() {
      f_unit = false;
      const int at = cur.at, last = cur.last;
      if (at >= last) return;
      int seq = cur.seq, seq_base = cur.seq_base, keys = sequence_keys(p, seq), nt = tiles_of<C>(keys);
      while (seq + 1 < p.B && at >= seq_base + (nt + OV) * per_seq) {
        seq_base += (nt + OV) * per_seq;
        ++seq;
        keys = sequence_keys(p, seq);
        nt = tiles_of<C>(keys);
      }
      if (p.lens[seq] != keys && lane == 0) atomicCAS(p.status, 0u, kStatusBadPage);
      const int unit = (at - seq_base) / (nt + OV), base = seq_base + unit * (nt + OV) + OV;   // its first tile
      const int t0 = max(at - base, 0), t1 = min(nt, last - base), hkv = (uint32_t)unit / p.div_blocks;
      __syncwarp();
      if (lane == 0) {
        cur.at = base + nt, cur.seq = seq, cur.seq_base = seq_base, cur.b = seq, cur.hkv = hkv;
        cur.row0 = (unit - hkv * p.row_blocks) * C::ROWS, cur.q_row = (long long)seq * p.Nq * p.H + hkv * p.G;
        s_units[warp][f_turn & 3] = Unit{seq, unit, t0, t1, nt, keys, base + nt};
      }
      __syncwarp();
      if (t1 <= t0) return;   // my share ends before the unit's first tile
      f_unit = true;
      f_keys = keys, f_tile = t0, f_end = t1, f_q = 0, f_rel = 0, f_values = false;
      next_pages = look_up(t0);
      ++f_turn;
    };
    auto step = [&]() {
      if (f_unit) {
        if (f_q < NT) {
          constexpr int QCH = D / 8, QRPI = 32 / QCH;   // 16-byte chunks of a query row, rows of a copy
#pragma unroll
          for (int i = 0; i < 8 / QRPI; ++i) {
            const int r = i * QRPI + lane / QCH;
            const uint32_t row = cur.row0 + f_q * 8 + (C::TWIN ? r & 3 : r), qi = row / p.div_g;
            const bool in = row < (uint32_t)(p.Nq * p.G);
            const long long from = in ? cur.q_row + (long long)qi * p.H + (row - qi * p.G) : 0;
            copy16<0>(fill + chunk_at<2 * D>(r, lane % QCH), p.q + from * D + lane % QCH * 8, in);
          }
          ++f_q;
        } else {
          if (f_rel == 0 && (C::PAIR || !f_values)) next_batch();
          const int valid = f_keys - f_tile * KT, from = f_rel * KB;
          const uint8_t* src = (!C::PAIR && f_values ? p.c.v : p.c.k) + my_row;
          const long long to_v = p.c.v - p.c.k;
          const uint32_t dst = fill + my_dst;
          long long base[KB];
          bool full = valid >= KT;
#pragma unroll
          for (int i = 0; i < KB; ++i) {
            base[i] = __shfl_sync(0xffffffffu, at_row, from + i);
            full = full && base[i] >= 0;
          }
          // Copies of one place of chunk_at's 8-row pattern share an address but for a constant.
          auto copy_rows = [&](auto copy) {
            each_of<KT / RPI>([&](auto index) {
              constexpr int I = decltype(index)::value, R = I * RPI, FIRST = R % 8;
              uint32_t to = dst;
              if constexpr (FIRST != 0) to = fill + chunk_at<C::ROWB>(FIRST + lane / CH, lane % CH) - FIRST * C::ROWB;
              copy(std::integral_constant<int, R>{}, std::integral_constant<int, R * C::ROWB>{}, to);
            });
          };
          if (full) {   // the same for the whole warp
            copy_rows([&](auto row, auto off, uint32_t to) {
              constexpr int R = decltype(row)::value, OFF = decltype(off)::value;
              const uint8_t* from = src + base[R / 16] + R % 16 * p.c.token_b;
              copy16<OFF>(to, from);
              if (C::PAIR) copy16<C::V_OFF + OFF>(to, from + to_v);
            });
          } else {      // rows behind the last key, or without a page, become zeros
            copy_rows([&](auto row, auto off, uint32_t to) {
              constexpr int R = decltype(row)::value, OFF = decltype(off)::value;
              const bool in = base[R / 16] >= 0 && R + lane / CH < valid;
              const uint8_t* from = src + (in ? base[R / 16] + R % 16 * p.c.token_b : -my_row);
              copy16<OFF>(to, from, in);
              if (C::PAIR) copy16<C::V_OFF + OFF>(to, from + to_v, in);
            });
          }
          if constexpr (INT4) {
            const long long base = __shfl_sync(0xffffffffu, at_sz, from + lane / 16);
            const bool in = base >= 0 && lane < valid;
            const uint8_t* sz = p.c.k_sz + (in ? my_sz + base : 0);
            copy_small<C::SZ_OFF, C::SZB>(fill + lane * C::SZB, sz, in);
            copy_small<C::SZV_OFF, C::SZB>(fill + lane * C::SZB, sz + (p.c.v_sz - p.c.k_sz), in);
          }
          if (!C::PAIR && !f_values) {
            f_values = true;
          } else {
            f_values = false;
            f_rel = (f_rel + 1) % PER;
            if (++f_tile == f_end) enter();
          }
        }
      }
      copies_commit();
      fill += C::SLOT;
      if (fill == ring_end) fill = buf;
    };
    enter();
#pragma unroll 1
    for (int i = 0; i < C::SLOTS - 1; ++i) step();

    // ---- products
    uint32_t slot = buf;   // slot that is read
    // Its copies are here, and the slot read before, which all lanes are past, takes the next ones.
    auto turn_to = [&]() {
      copies_wait<C::SLOTS - 2>();
      __syncwarp();
      step();
    };
    auto leave = [&]() {
      slot += C::SLOT;
      if (slot == ring_end) slot = buf;
    };
    // Twin columns: the second ones' weights are without their first number.
    [[maybe_unused]] const uint64_t minus_hi = t < 2 ? f2_pack(0.f, 0.f) : f2_pack(-1.f, -1.f);
    // Where this lane's row of a matrix load lies: lanes 0-7 and 8-15 rows 0-7 and 8-15 of a 16-row block's first
    // chunk, lanes 16-31 of its second. Further pairs of chunks differ in bits 5 and up.
    const uint32_t my_chunk = chunk_at<C::ROWB>(lane & 15, lane >> 4);
    for (int turn = 0; turn < f_turn; ++turn) {
      constexpr int QR = D / 16;
      // Query rows as the B operand: lane (g, t) holds row g's values that its K bytes are paired with.
      uint32_t qf[NT][QR][2];
      float mult[NT][2];            // S = mult * (what the products give), per column 2t, 2t + 1
      float qsum[NT][GROUPS][2];    // 4 bits: sums of q over a group, in units of the products
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        turn_to();
        if constexpr (INT4) {
          uint4 raw[GROUPS][2];
          float top = 0.f, sum[GROUPS];
#pragma unroll
          for (int gr = 0; gr < GROUPS; ++gr) {
            sum[gr] = 0.f;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              raw[gr][w] = lds128(slot + chunk_at<2 * D>(g, gr * 8 + 4 * w + t));   // dims 64 gr + 32 w + 8 t
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
              for (int i = 0; i < 2; ++i) {   // word's codes (0, 4), (1, 5) then (2, 6), (3, 7)
                qf[nt][gr * 4 + 2 * w + i][0] = pack_half2(x[2 * i], x[2 * i + 4]);
                qf[nt][gr * 4 + 2 * w + i][1] = pack_half2(x[2 * i + 1] * 0.0625f, x[2 * i + 5] * 0.0625f);
              }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) qsum[nt][gr][j] = __shfl_sync(0xffffffffu, sum[gr] * down * 0x1p-24f, (2 * t + j) * 4);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) mult[nt][j] = __shfl_sync(0xffffffffu, up, (2 * t + j) * 4) * p.scale_log2 * 0x1p24f;
        } else {
#pragma unroll
          for (int k = 0; k < QR; k += 2) {   // matrices: 8 rows of four neighbouring chunks
            const uint4 x = load_matrices<false, 0>(slot + chunk_at<2 * D>(lane & 7, 2 * k + (lane >> 3)));
            qf[nt][k][0] = x.x;
            qf[nt][k][1] = x.y;
            qf[nt][k + 1][0] = x.z;
            qf[nt][k + 1][1] = x.w;
          }
          mult[nt][0] = mult[nt][1] = p.scale_log2;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (mult[nt][j] == 0.f) mult[nt][j] = 0x1p-126f;   // 0 times a masked key's infinity would be NaN
        leave();
      }
      const volatile Unit& unit = s_units[warp][turn & 3];
      const int keys = unit.keys, t1 = unit.t1, rows = p.Nq * p.G;
      const int row0 = row_block(p, unit.unit) * C::ROWS;
      int limit[NT][2], least = INT_MAX;   // the column's row sees keys < limit
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = row0 + nt * 8 + (C::TWIN ? 2 * t & 3 : 2 * t) + j;
          limit[nt][j] = p.causal && c < rows ? keys - p.Nq + 1 + (int)((uint32_t)c / p.div_g) : keys;
          least = min(least, limit[nt][j]);
        }
      least = min(least, __shfl_xor_sync(0xffffffffu, least, 1));
      least = min(least, __shfl_xor_sync(0xffffffffu, least, 2));

      float acc[NT][D / 16][4];
      float m[NT][2], l[NT][2];
      uint64_t z[NT][INT4 ? GROUPS : 1];    // 4 bits, a pair of columns: sums of weight times zero,
      [[maybe_unused]] uint64_t up[NT][C::UP ? GROUPS : 1];   // and what a group's weights times scale are multiplied with
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[nt][i][j] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          m[nt][j] = kNone;
          l[nt][j] = 0.f;
#pragma unroll
          for (int gr = 0; gr < (INT4 ? GROUPS : 1); ++gr) z[nt][gr] = f2_pack(0.f, 0.f);
#pragma unroll
          for (int gr = 0; gr < (C::UP ? GROUPS : 1); ++gr) up[nt][gr] = f2_pack(1.f, 1.f);
        }
      }
#pragma unroll 1
      for (int n = unit.t0; n < t1; ++n) {
        turn_to();
        const int tile_key = n * KT;
        float s[KB][NT][4];
        // S^T = K q^T
        each_of<KB>([&](auto block) {
          constexpr int kb = decltype(block)::value;
          [[maybe_unused]] const uint32_t pairs = slot + g * C::SZB;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[kb][nt][j] = 0.f;
          if constexpr (INT4) {
            uint32_t ks[2][GROUPS];
            load_pairs<C::SZ_OFF + kb * 16 * C::SZB>(ks[0], pairs);
            load_pairs<C::SZ_OFF + (kb * 16 + 8) * C::SZB>(ks[1], pairs);
#pragma unroll
            for (int gr = 0; gr < GROUPS; ++gr) {
              // rows g and g + 8: dims 8t .. 8t + 7 of the group's first 32, then of its second
              const uint4 x = load_matrices<false, kb * 16 * C::ROWB>(slot + (my_chunk ^ gr * 32));
              float c[NT][4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t x0 = k < 2 ? x.x : x.z, x1 = k < 2 ? x.y : x.w;
                uint32_t a0, a1, a2, a3;   // low codes of both rows, high codes
                if (k % 2 == 0) {
                  a0 = x0 & 0x000f000fu, a1 = x1 & 0x000f000fu, a2 = x0 & 0x00f000f0u, a3 = x1 & 0x00f000f0u;
                } else {
                  const uint32_t y0 = high_bytes(x0), y1 = high_bytes(x1);
                  a0 = y0 & 0x000f000fu, a1 = y1 & 0x000f000fu, a2 = subtract_half2(y0, a0), a3 = subtract_half2(y1, a1);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint32_t(&q)[2] = qf[nt][gr * 4 + k];
                  if (k == 0) mma_first(c[nt], a0, a1, a2, a3, q[0], q[1]);
                  else mma<true>(c[nt], a0, a1, a2, a3, q[0], q[1]);
                }
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
          } else {
            each_of<QR>([&](auto step) {
              constexpr int k = decltype(step)::value;
              const uint4 x = load_matrices<false, kb * 16 * C::ROWB + k / 4 * 128>(slot + (my_chunk ^ k % 4 * 32));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<false>(s[kb][nt], x.x, x.y, x.z, x.w, qf[nt][k][0], qf[nt][k][1]);
            });
          }
          if (tile_key + KT > least) {   // the same for the whole warp
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float out = mult[nt][j] < 0.f ? INFINITY : -INFINITY;   // so that S is -inf
                if (tile_key + kb * 16 + g >= limit[nt][j]) s[kb][nt][j] = out;
                if (tile_key + kb * 16 + g + 8 >= limit[nt][j]) s[kb][nt][2 + j] = out;
              }
          }
        });
        if constexpr (!C::PAIR) {
          leave();
          turn_to();
        }
        // Weights p = 2^(S - m). The maximum m moves only when a weight outgrows its room: rarely after the first tile, so
        // that a tile costs a vote instead of the exchanges of a maximum. In 4 bits a weight times scale has to stay within
        // fp16. With one group of dims m is taken over S + log2 scale (its exponent). With several it is taken over S, and each
        // group of a column has a power of two that its weights times scale are multiplied with: one factor for all would
        // follow the greatest scale and lose the codes of a group 2^-14 as large, or less beside one early key's.
        [[maybe_unused]] uint32_t vs[KB][2][INT4 ? GROUPS : 1];   // (scale, zero) of my two values of a block
        float w[KB][NT][4], high[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          high[nt][0] = high[nt][1] = 0.f;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[kb][nt][j] = exp2_fast(fmaf(s[kb][nt][j], mult[nt][j & 1], -m[nt][j & 1]));
#pragma unroll
            for (int j = 0; j < 2; ++j) high[nt][j] = fmax3(high[nt][j], w[kb][nt][j], w[kb][nt][2 + j]);
          }
        }
        float most = 0.f;
        if constexpr (!INT4 || C::UP) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) most = fmax3(most, high[nt][0], high[nt][1]);
        }
        if constexpr (INT4) {
          each_of<KB * 2>([&](auto index) {
            constexpr int kb = decltype(index)::value / 2, i = decltype(index)::value % 2;
            load_pairs<C::SZV_OFF + (kb * 16 + i * 8) * C::SZB>(vs[kb][i], slot + g * C::SZB);
          });
          most *= 0x1p-25f;   // with several groups: weights themselves stay far from overflow
#pragma unroll
          for (int gr = 0; gr < GROUPS; ++gr) {
            float top = kLeastScale;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int i = 0; i < 2; ++i) top = fmaxf(top, fabsf(__uint_as_float(vs[kb][i][gr] << 16)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float a = high[nt][0] * top, b = high[nt][1] * top;
              if constexpr (C::UP) f2_unpack(f2_mul(f2_pack(a, b), up[nt][gr]), a, b);
              most = fmax3(most, a, b);
            }
          }
        }
        if (__any_sync(0xffffffffu, most > (INT4 ? kScaledHeadroom : kHeadroom))) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float x = m[nt][j];
              [[maybe_unused]] float y[C::UP ? GROUPS : 1];   // the same of S + log2 scale
#pragma unroll
              for (int gr = 0; gr < (C::UP ? GROUPS : 1); ++gr) y[gr] = -INFINITY;
#pragma unroll
              for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  // exponent of the scale, one more so that scale 2^-e < 1
                  auto exponent = [&](int gr) {
                    const float sc = fmaxf(fabsf(__uint_as_float(vs[kb][i][gr] << 16)), kLeastScale);
                    return (float)((int)(__float_as_uint(sc) >> 23) - 126);
                  };
                  const float score = s[kb][nt][2 * i + j];
                  if constexpr (C::UP) {
                    x = fmaxf(x, score * mult[nt][j]);
#pragma unroll
                    for (int gr = 0; gr < GROUPS; ++gr) y[gr] = fmaxf(y[gr], fmaf(score, mult[nt][j], exponent(gr)));
                  } else {
                    x = fmaxf(x, fmaf(score, mult[nt][j], INT4 ? exponent(0) - kTop : 1.f));
                  }
                }
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) {
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                if constexpr (C::UP) {
#pragma unroll
                  for (int gr = 0; gr < GROUPS; ++gr) y[gr] = fmaxf(y[gr], __shfl_xor_sync(0xffffffffu, y[gr], o));
                }
              }
              const float down = m[nt][j] - x, f = exp2_fast(down);
              m[nt][j] = x;
              l[nt][j] *= f;
#pragma unroll
              for (int gr = 0; gr < (INT4 ? GROUPS : 1); ++gr) z[nt][gr] = f2_mul(z[nt][gr], j ? f2_pack(1.f, f) : f2_pack(f, 1.f));
              if constexpr (C::UP) {
#pragma unroll
                for (int gr = 0; gr < GROUPS; ++gr) {
                  float u[2];
                  f2_unpack(up[nt][gr], u[0], u[1]);
                  const int was = (int)(__float_as_uint(u[j]) >> 23) - 127;
                  // as far up as this tile allows, and what is summed already (its greatest stays where it was)
                  const int now = (int)fmaxf(fminf(fminf(floorf(kTop + x - y[gr]), was + floorf(-down)), 125.f), -125.f);
                  u[j] = __uint_as_float((uint32_t)(now + 127) << 23);
                  up[nt][gr] = f2_pack(u[0], u[1]);
                  const float fg = exp2_fast(down + (float)(now - was));
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    acc[nt][gr * 4 + i][j] *= fg;
                    acc[nt][gr * 4 + i][2 + j] *= fg;
                  }
                }
              } else {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  acc[nt][i][j] *= f;
                  acc[nt][i][2 + j] *= f;
                }
              }
#pragma unroll
              for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int i = 0; i < 2; ++i) w[kb][nt][2 * i + j] = exp2_fast(fmaf(s[kb][nt][2 * i + j], mult[nt][j], -x));
            }
        }
        // O^T += V^T P^T
        each_of<KB>([&](auto block) {
          constexpr int kb = decltype(block)::value;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) l[nt][j] += w[kb][nt][j] + w[kb][nt][2 + j];
          if constexpr (INT4) {
#pragma unroll
            for (int gr = 0; gr < GROUPS; ++gr) {
              uint64_t sc[2], zr[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float a = __uint_as_float(vs[kb][i][gr] << 16), b = __uint_as_float(vs[kb][i][gr] & 0xffff0000u);
                sc[i] = f2_pack(a, a), zr[i] = f2_pack(b, b);
              }
              // Weights times scale rounded to fp16, and what that left; of twin columns the first takes one, the second
              // the other.
              uint32_t hi[2][NT];
              [[maybe_unused]] uint32_t lo[2][NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint64_t q = f2_pack(w[kb][nt][2 * i], w[kb][nt][2 * i + 1]);
                  const uint64_t x = f2_mul(C::UP ? f2_mul(q, up[nt][gr]) : q, sc[i]);
                  const uint32_t h = pack_half2(x);
                  if constexpr (C::TWIN) {
                    hi[i][nt] = transpose8x8(pack_half2(f2_fma(unpack_half2(h), minus_hi, x)));
                  } else {
                    hi[i][nt] = transpose8x8(h);
                    lo[i][nt] = transpose8x8(pack_half2(f2_sub(x, unpack_half2(h))));
                  }
                  z[nt][gr] = f2_fma(q, zr[i], z[nt][gr]);
                }
              // lane (g, t): of keys 2t, 2t + 1 (and 8 further) dims 4g .. 4g + 3 of the group's two halves
              const uint4 x = load_matrices<true, C::V_OFF + kb * 16 * C::ROWB>(slot + (my_chunk ^ gr * 32));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t x0 = i < 2 ? x.x : x.z, x1 = i < 2 ? x.y : x.w;
                const uint32_t y0 = i % 2 ? high_bytes(x0) : x0 & 0x00ff00ffu, y1 = i % 2 ? high_bytes(x1) : x1 & 0x00ff00ffu;
                const uint32_t c0 = y0 & 0x000f000fu, c1 = y1 & 0x000f000fu;   // low codes, and low + 16 high
                // A matrix product cuts what it adds up, towards 0. In a chain over all keys that is a drift of the codes'
                // offset, hundreds of times O where many keys share the weight: products start from 0, sums round to nearest.
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float p[4];
                  mma_first(p, c0, y0, c1, y1, hi[0][nt], hi[1][nt]);
                  if constexpr (!C::TWIN) mma<true>(p, c0, y0, c1, y1, lo[0][nt], lo[1][nt]);
                  add(acc[nt][gr * 4 + i], p);
                }
              }
            }
          } else {
            uint32_t b0[NT], b1[NT], c0[NT], c1[NT];   // weights rounded to bf16, and what that left
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float(&q)[4] = w[kb][nt];
              const uint32_t p0 = pack_bf162(q[0], q[1]), p1 = pack_bf162(q[2], q[3]);
              b0[nt] = transpose8x8(p0);
              b1[nt] = transpose8x8(p1);
              c0[nt] = transpose8x8(pack_bf162(q[0] - __uint_as_float(p0 << 16), q[1] - __uint_as_float(p0 & 0xffff0000u)));
              c1[nt] = transpose8x8(pack_bf162(q[2] - __uint_as_float(p1 << 16), q[3] - __uint_as_float(p1 & 0xffff0000u)));
            }
            each_of<D / 16>([&](auto index) {
              constexpr int i = decltype(index)::value;
              const uint4 x = load_matrices<true, C::V_OFF + kb * 16 * C::ROWB + i / 4 * 128>(slot + (my_chunk ^ i % 4 * 32));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma<false>(acc[nt][i], x.x, x.z, x.y, x.w, b0[nt], b1[nt]);
                mma<false>(acc[nt][i], x.x, x.z, x.y, x.w, c0[nt], c1[nt]);
              }
            });
          }
        });
        leave();
      }

      // The unit is done, or my share is. Column sums over the lanes that hold its keys.
      const bool head = unit.t0 == 0, tail = t1 == unit.nt;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], o);
            if constexpr (INT4) {
#pragma unroll
              for (int gr = 0; gr < GROUPS; ++gr)
                if (j == 0) z[nt][gr] = f2_add(z[nt][gr], __shfl_xor_sync(0xffffffffu, (unsigned long long)z[nt][gr], o));
            }
          }
        }
      if constexpr (C::TWIN) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[0][i][j] += __shfl_xor_sync(0xffffffffu, acc[0][i][j], 2);
      }
      // O^T of column c, dims d(i) and d(i) + 1 (4 bits) or + 8: MMA rows g and g + 8 of tile i
      auto value = [&](int nt, int i, int j) -> float2 {
        const float x = acc[nt][i][j], y = acc[nt][i][2 + j];
        if constexpr (INT4) {
          float z0, z1, back = 1.f;
          f2_unpack(z[nt][i / 4], z0, z1);
          if constexpr (C::UP) {
            float u0, u1;
            f2_unpack(up[nt][i / 4], u0, u1);
            back = __uint_as_float((254u << 23) - __float_as_uint(j ? u1 : u0));   // 1 / u, a power of two
          }
          return make_float2(x * back * 0x1p24f + (j ? z1 : z0), (y - x) * back * 0x1p20f + (j ? z1 : z0));
        }
        else return make_float2(x, y);
      };
      auto dim = [&](int i) { return INT4 ? i / 2 * 32 + 4 * g + i % 2 * 2 : 16 * i + g; };
      const bool whole = head && tail;
      if (whole || turn + 1 < f_turn) {   // finished, or the last part of a unit that other warps have begun
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = nt * 8 + 2 * t + j, row = row0 + c;
            const float inv = l[nt][j] != 0.f ? 1.f / l[nt][j] : 0.f;
            const float lse2 = l[nt][j] != 0.f ? m[nt][j] + log2f(l[nt][j]) : -INFINITY;
            if (!whole) {
              float* to = p.part_o + ((long long)(2 * me) * C::ROWS + c) * D;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const float2 x = value(nt, i, j);
                if constexpr (INT4) *reinterpret_cast<float2*>(to + dim(i)) = make_float2(x.x * inv, x.y * inv);
                else to[dim(i)] = x.x * inv, to[dim(i) + 8] = x.y * inv;
              }
              if (g == 0) p.part_lse[2 * me * C::ROWS + c] = lse2;
            } else if (row < rows) {
              const int qi = (uint32_t)row / p.div_g, h = (uint32_t)unit.unit / p.div_blocks * p.G + row - qi * p.G;
              __nv_bfloat16* to = p.o + (((long long)unit.b * p.Nq + qi) * p.H + h) * D;
              if constexpr (INT4) {
#pragma unroll
                for (int i = 0; i < D / 16; i += 2) {
                  const float2 x = value(nt, i, j), y = value(nt, i + 1, j);
                  *reinterpret_cast<uint2*>(to + dim(i)) =
                      make_uint2(pack_bf162(x.x * inv, x.y * inv), pack_bf162(y.x * inv, y.y * inv));
                }
              } else {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  const float2 x = value(nt, i, j);
                  to[dim(i)] = __float2bfloat16_rn(x.x * inv), to[dim(i) + 8] = __float2bfloat16_rn(x.y * inv);
                }
              }
              if (g == 0) p.lse[((long long)unit.b * p.H + h) * p.Nq + qi] = lse2 * 0.69314718055994531f;
            }
          }
      } else {   // my share ends in this unit: joined with the CTA's other warps in it, below
        copies_wait<0>();
        __syncwarp();
        float* part = reinterpret_cast<float*>(ring + warp * C::WARP_BYTES);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = nt * 8 + 2 * t + j;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const float2 x = value(nt, i, j);
              if constexpr (INT4) *reinterpret_cast<float2*>(part + c * D + dim(i)) = x;
              else part[c * D + dim(i)] = x.x, part[c * D + dim(i) + 8] = x.y;
            }
            if (g == 0) {
              s_m[warp][c] = m[nt][j];
              s_l[warp][c] = l[nt][j];
            }
          }
        if (lane == 0) {
          s_units[warp][0] = Unit{unit.b, unit.unit, unit.t0, t1, unit.nt, keys, unit.end};
          s_id[warp] = unit.end;   // no two units end at one place
          s_open[warp] = (head ? 1 : 0) | (tail ? 2 : 0);
        }
      }
    }
    copies_wait<0>();
  }
  // The joining kernel's CTAs may take the room that CTAs of this one leave; they wait for all of its results.
  griddep_launch_dependents();
  __syncthreads();

  // Warps [w0, w1) of this CTA whose shares end in one unit.
  for (int w0 = 0; w0 < kWarps;) {
    int w1 = w0 + 1;
    while (w1 < kWarps && s_id[w1] == s_id[w0]) ++w1;
    if (s_id[w0] >= 0) {
      const Unit unit = s_units[w0][0];
      const int first = blockIdx.x * kWarps + w0, rows = p.Nq * p.G, row0 = row_block(p, unit.unit) * C::ROWS;
      const bool head = s_open[w0] & 1, whole = head && (s_open[w1 - 1] & 2);
#pragma unroll
      for (int n = 0; n < C::ROWS * (D / 4) / kThreads; ++n) {
        const int i = n * kThreads + tid, r = i / (D / 4), c = i % (D / 4) * 4, row = row0 + r;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, w >= w0 && w < w1 ? s_m[w][r] : -INFINITY);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w < w0 || w >= w1) continue;
          const float f = exp2_fast(s_m[w][r] - top);
          const float4 y = *reinterpret_cast<const float4*>(ring + w * C::WARP_BYTES + (r * D + c) * 4);
          sum += s_l[w][r] * f;
          add(x, f, y);
        }
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
        const float lse2 = sum != 0.f ? top + log2f(sum) : -INFINITY;
        if (!whole) {
          const long long to = (long long)(2 * first + 1) * C::ROWS + r;
          *reinterpret_cast<float4*>(p.part_o + to * D + c) = x;
          if (c == 0) p.part_lse[to] = lse2;
        } else if (row < rows) {
          const int qi = (uint32_t)row / p.div_g, h = (uint32_t)unit.unit / p.div_blocks * p.G + row - qi * p.G;
          *reinterpret_cast<uint2*>(p.o + (((long long)unit.b * p.Nq + qi) * p.H + h) * D + c) =
              make_uint2(pack_bf162(x.x, x.y), pack_bf162(x.z, x.w));
          if (c == 0) p.lse[((long long)unit.b * p.H + h) * p.Nq + qi] = lse2 * 0.69314718055994531f;
        }
      }
      if (head && !whole && tid == 0) {
        // The warp with the unit's last tile; whether it goes on to the tiles of a next unit.
        const int end = unit.end - 1, long_ones = more * (part + 1);
        const int w = end < long_ones ? end / (part + 1) : more + (end - long_ones) / part;
        p.cut[first] = make_int4(unit.b, unit.unit, w, share(w + 1) > unit.end + OV ? 1 : 0);
      }
    }
    w0 = w1;
  }
}

// Joins the parts of the units that were cut: CTA (c, r) takes row r of the units that begin in warps c span to
// (c + 1) span - 1 of the grid before. With a unit a warp or so (span = kWarps, "alone") a warp takes one if it has few
// parts; otherwise all warps share the parts of one after the other.
// LSE = log2 sum 2^LSE_i,  O = sum 2^(LSE_i - LSE) O_i.
constexpr int kFewParts = 8;
constexpr int kManyWarps = 16;   // of a CTA when units have many parts

template <int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) attn_paged_join_kernel(const Params p, int rows_per_unit, int span, int records) {
  griddep_wait();
  const bool alone = WARPS == kWarps && span == kWarps;   // a record a warp
  constexpr int LANES = D / 4;                // lanes of a row
  constexpr int STEP = LANES < 32 ? LANES : 32, V = LANES / STEP, WAYS = 32 / STEP;   // of a warp: values each, rows at once
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = lane % STEP * 4, way = lane / STEP, r = blockIdx.y;
  struct Cut {
    int4 cut;
    int from;   // the warp that it begins in
  };
  __shared__ Cut cuts[32 * WARPS];   // units left to the whole CTA, in order
  __shared__ int counts[WARPS];
  Cut own{make_int4(0, 0, -1, 0), (int)(blockIdx.x * span + (alone ? warp : threadIdx.x))};
  if ((alone || (int)threadIdx.x < span) && own.from < records) own.cut = p.cut[own.from];
  bool mine = own.cut.z >= 0 && own.cut.y % p.row_blocks * rows_per_unit + r < p.Nq * p.G;
  // Parts of a unit that begins in warp `from`: slot 2 from + 1, one of each later CTA's first warp, and of the last warp its
  // slot for a unit that ends inside a share (then the last CTA's first warp has one only if it is not that warp).
  auto joined_of = [&](const Cut& x) {
    return max(x.cut.z / kWarps - x.from / kWarps - (x.cut.w && x.cut.z % kWarps == 0 ? 1 : 0), 0);
  };
  auto parts_of = [&](const Cut& x) { return 1 + joined_of(x) + x.cut.w; };
  auto slot_of = [&](const Cut& x, int joined, int i) -> long long {
    return i == 0 ? 2LL * x.from + 1 : i <= joined ? 2LL * kWarps * (x.from / kWarps + i) + 1 : 2LL * x.cut.z;
  };
  struct Sum {
    float top, sum;
    float4 x[V];
  };
  // Parts first, first + stride, .. of a unit: their weighted sums for this lane, and the weights'.
  auto gather = [&](const Cut& x, float top, int first, int stride) {
    const int joined = joined_of(x), parts = parts_of(x);
    auto at = [&](int i) -> long long { return slot_of(x, joined, i) * rows_per_unit + r; };
    Sum s{top, 0.f, {}};
#pragma unroll 4
    for (int i = first * WAYS + way; i < parts; i += stride * WAYS) {
      const float f = exp2_fast(p.part_lse[at(i)] - s.top);
      s.sum += f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        add(s.x[v], f, *reinterpret_cast<const float4*>(p.part_o + at(i) * D + v * 128 + c));
      }
    }
    if constexpr (WAYS > 1) {
#pragma unroll
      for (int o = STEP; o < 32; o <<= 1) {
        s.sum += __shfl_xor_sync(0xffffffffu, s.sum, o);
        s.x[0].x += __shfl_xor_sync(0xffffffffu, s.x[0].x, o);
        s.x[0].y += __shfl_xor_sync(0xffffffffu, s.x[0].y, o);
        s.x[0].z += __shfl_xor_sync(0xffffffffu, s.x[0].z, o);
        s.x[0].w += __shfl_xor_sync(0xffffffffu, s.x[0].w, o);
      }
    }
    return s;
  };
  auto store = [&](const int4& cut, const Sum& s) {
    const int hkv = cut.y / p.row_blocks, row = (cut.y - hkv * p.row_blocks) * rows_per_unit + r;
    const int qi = (uint32_t)row / p.div_g, h = hkv * p.G + row - qi * p.G;
    const float inv = s.sum != 0.f ? 1.f / s.sum : 0.f;
    if (way == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        *reinterpret_cast<uint2*>(p.o + (((long long)cut.x * p.Nq + qi) * p.H + h) * D + v * 128 + c) =
            make_uint2(pack_bf162(s.x[v].x * inv, s.x[v].y * inv), pack_bf162(s.x[v].z * inv, s.x[v].w * inv));
    }
    if (lane == 0)
      p.lse[((long long)cut.x * p.H + h) * p.Nq + qi] = s.sum != 0.f ? (s.top + log2f(s.sum)) * 0.69314718055994531f : -INFINITY;
  };
  // A few parts: everything is loaded at once.
  auto gather_few = [&](const Cut& cut) {
    const int joined = joined_of(cut), parts = parts_of(cut);
    float lse[kFewParts];
    float4 x[kFewParts][V];
#pragma unroll
    for (int i = 0; i < kFewParts; ++i) {
      const long long at = slot_of(cut, joined, i) * rows_per_unit + r;
      lse[i] = i < parts ? p.part_lse[at] : -INFINITY;
#pragma unroll
      for (int v = 0; v < V; ++v)
        x[i][v] = i < parts ? *reinterpret_cast<const float4*>(p.part_o + at * D + v * 128 + c) : float4{};
    }
    Sum s{-INFINITY, 0.f, {}};
    bool any = false;
#pragma unroll
    for (int i = 0; i < kFewParts; ++i) {
      s.top = fmaxf(s.top, lse[i]);
      any = any || !(lse[i] == -INFINITY);
    }
    if (!any) return s;
#pragma unroll
    for (int i = 0; i < kFewParts; ++i) {
      const float f = i < parts ? exp2_fast(lse[i] - s.top) : 0.f;
      s.sum += f;
#pragma unroll
      for (int v = 0; v < V; ++v) add(s.x[v], f, x[i][v]);
    }
    return s;
  };
  if (alone) {
    if (mine && parts_of(own) <= kFewParts) {
      store(own.cut, gather_few(own));
      mine = false;
    }
    mine = mine && lane == 0;
  }
  const uint32_t ballot = __ballot_sync(0xffffffffu, mine);
  if (lane == 0) counts[warp] = __popc(ballot);
  if (!__syncthreads_or(mine)) return;
  int n = 0, before = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    before += w < warp ? counts[w] : 0;
    n += counts[w];
  }
  if (mine) cuts[before + __popc(ballot & ((1u << lane) - 1u))] = own;
  __syncthreads();
  __shared__ Sum sums[WARPS][32];
  __shared__ float tops[WARPS];
  for (int i = 0; i < n; ++i) {   // the same for the whole CTA
    const Cut x = cuts[i];
    const int joined = joined_of(x), parts = parts_of(x);
    float top = -INFINITY;
    bool any = false;   // a part that has keys, or is NaN
    for (int j = threadIdx.x; j < parts; j += 32 * WARPS) {
      const float lse = p.part_lse[slot_of(x, joined, j) * rows_per_unit + r];
      top = fmaxf(top, lse);
      any = any || !(lse == -INFINITY);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    const bool some = __syncthreads_or(any);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, tops[w]);
    sums[warp][lane] = some ? gather(x, top, warp, WARPS) : Sum{-INFINITY, 0.f, {}};
    __syncthreads();
    if (warp == 0) {
      Sum s = sums[0][lane];
      for (int w = 1; w < WARPS; ++w) {
        const Sum& y = sums[w][lane];
        s.sum += y.sum;
#pragma unroll
        for (int v = 0; v < V; ++v) add(s.x[v], 1.f, y.x[v]);
      }
      store(x.cut, s);
    }
    __syncthreads();   // the sums are free again
  }
}

struct Plan {
  int rows_per_unit, row_blocks, grid, tile, overhead;
};

// Rows a unit holds (8, or 16 at d <= 128 when a call has more: d = 256 has no registers for them) and the CTAs that fill
// the device.
template <int D, bool INT4>
Plan plan_for(int rows, int sms) {
  constexpr int NT2 = D <= 128 ? 2 : 1;
  const int per = rows > 8 ? 8 * NT2 : 8;
  return {per, (rows + per - 1) / per, sms * (per == 16 ? Cfg<D, INT4, NT2>::CTAS : Cfg<D, INT4, 1>::CTAS),
          Cfg<D, INT4, 1>::KT, Cfg<D, INT4, 1>::OVERHEAD};
}

Plan make_plan(int d, bool int4, int rows, int sms) {
  switch (d) {
    case 64: return int4 ? plan_for<64, true>(rows, sms) : plan_for<64, false>(rows, sms);
    case 128: return int4 ? plan_for<128, true>(rows, sms) : plan_for<128, false>(rows, sms);
    default: return int4 ? plan_for<256, true>(rows, sms) : plan_for<256, false>(rows, sms);
  }
}

template <class C>
cudaError_t launch(const Params& p, int grid, unsigned long long context, cudaStream_t s) {
  auto kernel = attn_paged_kernel<C>;
  cudaError_t e;
  // The attribute stays with the context; setting it on every call would cost the host 1 us of 7.6.
  static std::atomic<unsigned long long> set_for{0};
  if (context == 0 || set_for.load(std::memory_order_relaxed) != context) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
    set_for.store(context, std::memory_order_relaxed);
  }
  if ((e = launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), C::SMEM, s, p)) != cudaSuccess) return e;
  // At most a unit a CTA, as a rule: with few units most warps begin none, and CTAs that find nothing cost more than a look at
  // more warps does (B 4, one kv head, 12 rows, 6161 keys: 13.5 us with 4 warps a CTA always, 11.3 so; twice or four times
  // as many warps a CTA leave some with two units, one after the other, 1 us more at B 2).
  const int records = grid * kWarps;
  const long long units = (long long)p.B * p.c.Hkv * p.row_blocks;
  const int span = (int)std::clamp<long long>(records / (4 * units), kWarps, kThreads);
  // 32 parts a unit and more: 16 warps (one sequence of 60871 keys, d 256 in bf16, one kv head: 25.5 us, with 4 warps 32.4;
  // at 16 parts, B 28 of up to 1166 keys, 17 against 10.4).
  const bool many = grid >= 32 * units;
  auto join = many ? attn_paged_join_kernel<C::D, kManyWarps> : attn_paged_join_kernel<C::D, kWarps>;
  return launch_dependent(join, dim3((unsigned)((records + span - 1) / span), (unsigned)std::min(C::ROWS, p.Nq * p.G)),
                          dim3(many ? 32 * kManyWarps : kThreads), 0, s, p, (int)C::ROWS, span, records);
}

template <int D, bool INT4>
cudaError_t launch_rows(const Params& p, int rows_per_unit, int grid, unsigned long long context, cudaStream_t s) {
  if constexpr (D <= 128) {
    if (rows_per_unit == 16) return launch<Cfg<D, INT4, 2>>(p, grid, context, s);
  }
  if constexpr (INT4) {
    if (p.Nq * p.G <= 4) return launch<Cfg<D, true, 1, true>>(p, grid, context, s);
  }
  return launch<Cfg<D, INT4, 1>>(p, grid, context, s);
}

template <int D>
cudaError_t launch_dim(const Params& p, bool bits4, int rows_per_unit, int grid, unsigned long long context, cudaStream_t s) {
  return bits4 ? launch_rows<D, true>(p, rows_per_unit, grid, context, s)
               : launch_rows<D, false>(p, rows_per_unit, grid, context, s);
}

size_t pad(size_t x) { return (x + 255) / 256 * 256; }

// Bytes of the parts, of their LSE, and of the cut units.
void workspace_parts(const Plan& pl, int d, size_t (&n)[3]) {
  const size_t warps = (size_t)pl.grid * kWarps;
  n[0] = pad(2 * warps * pl.rows_per_unit * d * 4);
  n[1] = pad(2 * warps * pl.rows_per_unit * 4);
  n[2] = pad(warps * sizeof(int4));
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
  if (rows > INT_MAX / 2 || (long long)B * H * Nq > INT_MAX || (long long)max_pages * cache->page_size > kMaxKeys)
    return ATTN_ERR_UNSUPPORTED;
  int sms;
  unsigned long long context;
  if (!device_state(&sms, &p.status, &context)) return ATTN_ERR_CUDA;
  const bool bits4 = cache->type == ATTN_CACHE_INT4;
  const Plan pl = make_plan(d, bits4, (int)rows, sms);
  size_t n[3];
  workspace_parts(pl, d, n);
  if (workspace_bytes < n[0] + n[1] + n[2]) return ATTN_ERR_INVALID_ARG;
  if ((long long)Hkv * pl.row_blocks > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  struct {
    const void* b;
    size_t n;
  } x[4] = {{o, (size_t)B * Nq * H * d * 2},
            {lse, (size_t)B * Nq * H * 4},
            {workspace, n[0] + n[1] + n[2]},
            {q, (size_t)B * Nq * H * d * 2}};
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
  p.div_g = fast_div((uint32_t)p.G), p.div_blocks = fast_div((uint32_t)pl.row_blocks);
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + n[0]);
  p.cut = reinterpret_cast<::int4*>(static_cast<uint8_t*>(workspace) + n[0] + n[1]);
  // No more warps than tiles there can be; tiles are counted in 32 bits.
  const long long most = (long long)B * Hkv * pl.row_blocks *
                         (((long long)max_pages * cache->page_size - 1) / pl.tile + 1 + pl.overhead);
  if (most > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  const int grid = (int)std::min<long long>(pl.grid, (most + kWarps - 1) / kWarps);
  const long long lines = (max_pages + 31LL) / 32;
  p.table_lines = lines * B <= std::min(8192, grid * kThreads) ? (int)lines : 0;
  const cudaError_t e = d == 64    ? launch_dim<64>(p, bits4, pl.rows_per_unit, grid, context, stream)
                        : d == 128 ? launch_dim<128>(p, bits4, pl.rows_per_unit, grid, context, stream)
                                   : launch_dim<256>(p, bits4, pl.rows_per_unit, grid, context, stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

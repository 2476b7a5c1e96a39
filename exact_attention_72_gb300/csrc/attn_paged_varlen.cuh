// Attention of chunks of new tokens over a paged key/value cache in bf16 or 4 bits, any ragged batch:
//   S = scale q k^T over the keys a row sees,  O = softmax(S) V,  LSE,
// with the queries of sequence b packed from row cu[b] on and its keys, the new ones among them, in pages.
//
// The G query heads of a kv head share its keys, so 128 rows of a tile are P = 128 / G positions times G heads: a decoding sequence
// reads its cache once. A CTA has two such tiles (one at d = 256, where O fills tensor memory), tcgen05 for both products, P in
// tensor memory, the scores' buffer shared by both tiles, and a softmax warpgroup for each.
//
// Work: units of (sequence, kv head, tiles of positions) times KV tiles. Lengths are known on the GPU only, and differ by orders:
// so all work, in weighted keys, is dealt to the CTAs, one an SM, in equal contiguous shares, whatever unit their ends fall into. A unit
// that is cut leaves normalised parts in fp32, at most two a CTA, which a second kernel joins. A chunk of 300 tokens over 65k keys
// fills the GPU like 34 sequences, and the workspace depends on neither. Finding its share takes a CTA some 2 us.
//
// What bounds it (GB300, H 32, Hkv 8, d 128, times of a call in a graph):
//   bf16, 4 chunks of up to 4096 tokens over 8192: 1183 us, 1640 TFLOP/s (85% of measured; another card 1230), and 1380 in calls
//     without a pause, at the power cap. A tile of 2 x 128 rows takes 1.65 us, in which the tensor core waits for the softmax of the
//     one buffer of scores; 1509 us at first: copies issued by four warps, MMAs by warps that run as one, and maxima taken by the
//     loads of the scores made it so.
//   the same at d 64: 923 us, 1050 TFLOP/s (54%). Exponentials take 46% of the special-function units and products as much of the
//     tensor pipe; 54% of the issue slots are taken: as many scores a tile as at d = 128, for half the products.
//   bf16, 30 decoding sequences of up to 16k keys: 243 us, 6200 GB/s (91%). A CTA by itself takes 1.2 us a tile, 64 KB that come 2 us after
//     their copy was issued; with fewer CTAs at it neither a fifth stage, tiles fetched into the L2 ahead (they take the copies' turns: 20%
//     slower), nor both tiles' warps on one unit made it faster.
//   bf16, d 256: 5 sequences, 777 tokens over 5000, H 16, Hkv 4: 149 us. 128 KB of keys and values for 128 rows come out of the
//     L2 at 40 bytes a cycle and SM, 11.5 TB/s in all. Halves of keys in more stages: 155 us.
//   4 bits, the first case: 1676 us. Unpacking, 2.3 us a tile of 128 keys and values by 4 warps; see unpack_role. (1833 us with a
//     branch around each arrival, which only one lane makes.)
#pragma once
#include <cuda_fp16.h>

#include "attn_fwd_kernel.cuh"
#include "fastdiv.cuh"
#include "ops.h"
#include "paged.cuh"

namespace gb300 {

struct PagedVarlenParams {
  PagedCache c;
  const __nv_bfloat16* q;   // [total_q, H, D]
  __nv_bfloat16* o;
  float* lse;               // [H, total_q]
  const int *table, *cu, *lens;
  long long table_stride;
  int B, H, G, P;           // G query heads a kv head, P = 128 / G positions a Q tile
  int total_q, max_pages, box_rows, causal;
  int skip_singles;         // sequences of one query are another kernel's
  FastDiv div_g, div_page;  // by G and by the page size
  float scale_log2;         // |scale| log2(e)
  uint32_t qk_negate;       // as AttnParams
  // Parts of cut units: slot 2c the one that CTA c continues, 2c + 1 the one that it begins and does not end.
  float* part_o;            // [2 CTAs, ROWS, D] normalised O
  float* part_lse;          // [2 CTAs, ROWS] log2-sum-exp2
  int4* cut;                // [CTAs]: (first packed row, kv head, positions, parts) of the unit that CTA c begins; parts 0: none
  int o_v8;                 // rows of o are 32-byte aligned
  uint32_t* status;
  unsigned long long timeout_ns;
  int debug_skip_load;
};

// A unit: the P * NQ positions of one (sequence, kv head) whose G heads fill the CTA's Q tiles; a piece: what one CTA does
// of it, KV tiles t0 .. t0 + max(n0, n1) - 1.
struct Piece {
  int work;                 // 0: no more pieces
  int q_row, n_pos;         // first packed row of the unit, its positions
  int kvh, b;
  int vis;                  // keys that its first query sees, less one (causal)
  int nk;                   // keys of the sequence
  int t0, n0, n1;           // first KV tile; tiles that Q tile 0 and 1 visit from there
  int slot;                 // of its part; -1: the piece is the whole unit
};

template <int D_, bool INT4_>
struct PagedVarlenCfg {
  static constexpr int D = D_;
  static constexpr bool INT4 = INT4_;
  static constexpr int NQ = D <= 128 ? 2 : 1;             // 128-row Q tiles of a CTA
  static constexpr int ROWS = 128 * NQ;                   // rows of a unit
  // Operands: 16-bit, K-major (V: MN-major) tiles of 128 rows in chunks of 64 columns with the 128-byte swizzle.
  static constexpr int SWZ = 128, SBO = 1024, CHUNK_BYTES = 128 * 128, NCH = D / 64;
  static constexpr int TILE_BYTES = NCH * CHUNK_BYTES;
  static constexpr int KSTEPS_QK = D / 16, KSTEPS_PV = 8, PV_ROWS = 16;
  static constexpr int EXT_BYTES = INT4 ? 128 * 32 : 0;   // 16 more columns of Q and K for the zeros of 4-bit keys
  static constexpr int NK = D == 64 ? 4 : D == 128 ? 2 : 1, NV = NK;   // stages of K and of V
  static constexpr int Q_BYTES = NQ * TILE_BYTES;
  static constexpr int SMEM_BYTES = Q_BYTES + NQ * EXT_BYTES + NK * (TILE_BYTES + EXT_BYTES) + NV * TILE_BYTES + 1024;
  // TMEM: S buffers, then a P area and an O tile of each Q tile.
  static constexpr int NSB = D == 64 ? 2 : 1;
  static constexpr int P_COL = 128 * NSB, P_COLS = 64, O_COL = D == 64 ? 384 : 256, TMEM_COLS = 512;
  static_assert(P_COL + NQ * P_COLS <= O_COL && O_COL + NQ * D <= TMEM_COLS, "TMEM budget");
  static constexpr uint32_t FMT = INT4 ? kFmtF16 : kFmtBF16;
  static constexpr uint32_t IDESC_QK = make_idesc(FMT, 128, 128, false, false);
  static constexpr uint32_t IDESC_PV = make_idesc(FMT, 128, D, false, true);
  // Warps: softmax (a warpgroup for each Q tile), then a warpgroup of PV issuers, scheduler and S issuer, then one that feeds
  // the stages: bf16, two warps issue the copies of keys and two those of values (a page of 16 keys takes a copy for every 64
  // dims, and a copy 70 cycles of a warp: one warp for all bounded the kernel); 4 bits, all unpack keys, then values.
  static constexpr int SOFTMAX_WARPS = 4 * NQ, WARP_PV = SOFTMAX_WARPS, WARP_PLAN = WARP_PV + 2, WARP_S = WARP_PV + 3;
  static constexpr int FEED_WARPS = INT4 && D == 256 ? 8 : 4;   // 8: four for keys, four for values
  static constexpr int WARP_FEED = WARP_PV + 4, THREADS = 32 * (WARP_FEED + FEED_WARPS);
  // Registers, of the launch's 512 x 128 (one Q tile over bf16: 384 x 168).
  static constexpr uint32_t REGS_SOFTMAX = INT4 && NQ == 2 ? 184 : 200;
  static constexpr uint32_t REGS_ROLES = NQ == 1 ? 64 : 56, REGS_FEED = NQ == 1 ? 96 : INT4 ? 88 : 56;
  static constexpr int REGS_NEEDED = SOFTMAX_WARPS * 32 * REGS_SOFTMAX + 128 * REGS_ROLES + 32 * FEED_WARPS * REGS_FEED;
  static constexpr int FEEDERS = INT4 ? 4 : 2;            // warps that fill a stage
  // Work of a key in a unit of one Q tile and of two. bf16: a tile of a decoding sequence takes 1.2 us, of a chunk 1.65. 4 bits:
  // unpacking bounds both.
  static constexpr int ONE = 3, TWO = INT4 || NQ == 1 ? 3 : 4;
  static constexpr int PIECES = 4;                        // pieces that the scheduler may be ahead
  static constexpr int CONSUMERS = SOFTMAX_WARPS + NQ + 1 + FEED_WARPS;
  // Tiles whose powers of two are kept, and pieces whose query rows' are: K_{j + METAS} waits for S_{j + NK}, which comes after
  // the softmax has taken S_j from its buffer, and with it all of these; likewise the query rows QFS pieces later.
  static constexpr int METAS = 2 * NK, QFS = NSB + 1;
};

constexpr long long kMostWork = 1LL << 52;   // of a call: 64 bits hold it times the number of CTAs
constexpr int kUnitOverhead = 6 * 128;       // work (see UnitWork) of beginning and ending a unit
// Least work of a CTA: about a tile, since less might lie within a unit's beginning and have nothing to do. 61 tokens over 1000, H 16,
// Hkv 4, d 64: 13.8 us, with 12 * 128 14.6, with 24 * 128 17.8.
constexpr long long kLeastShare = 8 * 128;

// Descriptor of an operand without swizzle: 8 x 16-byte core matrices, lbo apart along K, sbo along the rows.
__device__ __forceinline__ uint64_t make_sdesc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return make_sdesc_swz(saddr, lbo, sbo, 64u) & ~((uint64_t)7 << 61);
}

__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t a, uint4 x) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// Work of the units of one (sequence, kv head), P * NQ = RP positions each, off = nk - nq: unit m needs the keys that its last query
// sees, `one` for each if its rows fill one Q tile at most and `two` if they fill two, and kUnitOverhead.
struct UnitWork {
  int nq, nk, M, RP, one, two, causal;
  __device__ int keys(int m) const {
    if (!causal) return nk;
    const long long last = (long long)min((long long)(m + 1) * RP, (long long)nq) + nk - nq;
    return last > 0 ? (int)last : 0;
  }
  __device__ int a_key(int m) const { return nq - m * RP > RP / 2 ? two : one; }
  __device__ long long upto(int k) const {   // of units 0 .. k - 1
    long long s = (long long)k * kUnitOverhead;
    if (k == M && M > 0) {   // the last unit ends with the last query, which sees all keys
      --k;
      s += (long long)a_key(k) * nk;
    }
    if (!causal) return s + (long long)k * two * nk;
    const long long off = (long long)nk - nq;
    const long long m0 = off >= 0 ? 0 : -off / RP;   // units before see nothing
    if (k > m0) s += two * ((k - m0) * off + RP * ((long long)k * (k + 1) / 2 - m0 * (m0 + 1) / 2));
    return s;
  }
};

// Wait sites of this kernel besides those of the forward (SITE_*).
enum : uint32_t { SITE_PIECE_FULL = 16, SITE_PIECE_EMPTY = 17, SITE_META = 18 };

// A load that is not to be moved behind a wait: what it reads is used a step later.
__device__ __forceinline__ uint4 load_ahead(const void* p) {
  uint4 x;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}

// 2^e of a float's exponent bits: 1 <= bits <= 254.
__device__ __forceinline__ float power_of_bits(uint32_t bits) { return __uint_as_float(bits << 23); }
__device__ __forceinline__ uint32_t half2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float half_round(float x) { return __half2float(__float2half_rn(x)); }

// tcgen05 operations that a warp runs as one, of which the one lane with `on` issues them: what they take is then the same for the
// warp and stays in uniform registers (in a branch of one lane every descriptor was moved there anew).
__device__ __forceinline__ void warp_mma_ss(bool on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void warp_mma_ts(bool on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void warp_commit(bool on, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"((uint32_t)on)
      : "memory");
}

// One lane's arrival, as above.
__device__ __forceinline__ void warp_arrive(bool on, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar),
      "r"((uint32_t)on)
      : "memory");
}

// Waits, with a limit, until the copies that a phase counts have landed.
__device__ __forceinline__ void land(uint64_t* bar, uint32_t phase, unsigned long long timeout_ns) {
  const uint64_t t = global_timer_ns();
  while (!mbar_try_wait(smem_addr(bar), phase & 1) && global_timer_ns() - t < timeout_ns) {}
}

// The bf16 cache's keys or values, by one warp of the two that share the work. Lane i copies box 2 i + half of a tile: 64 columns
// (box % NCH) of box_rows neighbouring keys (box / NCH), which lie in one page.
template <class C, bool IS_V, class F>
__device__ __forceinline__ void load_role(const PagedVarlenParams& p, int half, const CUtensorMap* map, uint32_t tiles,
                                          uint64_t* bar_full, uint64_t* bar_empty, uint64_t* bar_patch, const WaitCtl& ctl,
                                          F& piece_of_warp) {
  constexpr int NCH = C::NCH, NS = IS_V ? C::NV : C::NK;
  const int lane = threadIdx.x & 31, rows = p.box_rows, boxes = 128 / rows * NCH;
  const int box = 2 * lane + half, chunk = box % NCH, at = box / NCH * rows;
  const bool mine = box < boxes;
  const uint32_t dst = chunk * C::CHUNK_BYTES + at * 128, bytes = (uint32_t)((boxes + 1 - half) / 2 * rows * 128);
  if (lane == 0) tma_prefetch_desc(map);
  uint32_t n_t = 0, n_patch = 0;   // tiles, patched ones
  Piece pc;
  bool ok = true;
  for (uint32_t it = 0; ok && piece_of_warp(it, pc); ++it) {
    const int n = max(pc.n0, pc.n1);
    const int* table = p.table + pc.b * p.table_stride;
    auto look_up = [&](int t) {
      const int key = t * 128 + at;
      return mine && key < pc.nk ? __ldg(table + (uint32_t)key / p.div_page) : -1;
    };
    int page = n > 0 ? look_up(pc.t0) : -1;
    for (int j = 0; j < n; ++j) {
      const int key0 = (pc.t0 + j) * 128, key = key0 + at, tok = key - (int)((uint32_t)key / p.div_page) * p.c.page_size;
      if (mine && key < pc.nk && (page < 0 || page >= p.c.num_pages)) {
        atomicCAS(p.status, 0u, kStatusBadPage);
        page = -1;   // outside the map: zeros, as for keys behind the last
      }
      const int from = page;
      if (j + 1 < n) page = look_up(pc.t0 + j + 1);
      const uint32_t stage = n_t % NS, tile = tiles + stage * C::TILE_BYTES;
      bool w = n_t < (uint32_t)NS || mbar_wait(smem_addr(&bar_empty[stage]), (n_t / NS - 1) & 1, ctl, SITE_KV_EMPTY);
      if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
      ++n_t;
      if (IS_V && p.debug_skip_load && blockIdx.x == 0 && n_t == 1) continue;
      // Values of the last page's rows behind the sequence's end may be anything, and 0 times NaN is NaN: they are cleared.
      const bool patch = IS_V && pc.nk - key0 < 128 && pc.nk % rows != 0;
      const uint32_t bar = smem_addr(patch ? bar_patch : &bar_full[stage]);
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (mine) tma_load_4d(tile + dst, map, bar, chunk * 64, tok, pc.kvh, from);
      if (patch) {
        ++n_patch;
        w = mbar_wait(bar, (n_patch - 1) & 1, ctl, SITE_KV_FULL);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        const int r0 = pc.nk - key0, last = r0 / rows, n_rows = (last + 1) * rows - r0;
        for (int i = lane; i < n_rows * 8 * NCH; i += 32) {
          const int r = i / (8 * NCH), c = i % (8 * NCH);
          if ((last * NCH + c / 8) % 2 == half)   // of a box of mine
            sts128(tile + c / 8 * C::CHUNK_BYTES + (r0 + r) * 128 + c % 8 * 16, make_uint4(0u, 0u, 0u, 0u));
        }
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bar_full[stage]));
      }
    }
  }
  if (!ok || *ctl.abort_flag) {   // unwinding: let every copy still in flight land before the CTA exits
    for (uint32_t i = n_t > (uint32_t)NS ? n_t - NS : 0u; i < n_t; ++i) land(&bar_full[i % NS], i / NS, p.timeout_ns);
    if (n_patch > 0) land(bar_patch, n_patch - 1, p.timeout_ns);
  }
}

// The 4-bit cache's operands. Thread r of the warpgroup has query row r of each Q tile and key r of each KV tile; at d = 256 one
// warpgroup has the keys and one the values, and each half of the query rows: with one stage of each, values that wait for their stage
// must not hold up the next keys (5 sequences of up to 777 over 5000 tokens, 16 heads on 4: 219 us; in turns, with branches, 292, each for itself 237).
//
// A code in the high bits of fp16's mantissa is 1 + c / 16: a shift and a three-input logic operation, and a fused multiply-add makes
// the operand of it.
// Keys: zero + scale c = scale (c - 8) + zero', zero' = zero + 8 scale. The first term, 16 scale (1 + c / 16) - 24 scale, has 11
// bits (8 of scale, 3 of c - 8), so fp16 holds it; the second is one value a group of dims, which S takes in as a product of 16
// more columns,
//   zero' sum(q) = (zh + zl) (Qh + Ql),    zh + zl and Qh + Ql the two values in 22 bits each.
// So S is what fp32 would give. In bf16 the keys would be 2^-8 off, and LSE with them (2e-5 of it over 1000 keys).
// Values: 16 scale (1 + c / 16) + (zero - 16 scale), the sum and its second term rounded to fp16: off by 2^-11 of the value and by
// 2^-11 |zero - 16 scale|, which for a group around zero (zero = -7.5 scale) is 3 * 2^-11 of its greatest value, and the same for all
// values of a group, whatever their size. With P's 2^-11, O's error is 0.0017 of its norm, as that of its own rounding alone; in
// bf16 the two would add as much again.
// fp16's range: every 32 keys (a warp's) of a tile are divided by a power of two that brings the greatest of them below 2^15, a
// query row by one that brings its greatest value into [2^7, 2^8). Full precision is left to values 2^-29 of the greatest of
// their 32 keys (query rows: 2^-21), others are off by 2^-40 (2^-33) of it. The softmax puts the keys' power back into the
// scores, and the values' into the weights' exponents: the running maximum is over weights times those powers, and the weights
// are summed without them.
template <class C, class F>
__device__ __forceinline__ void unpack_role(const PagedVarlenParams& p, int thread, int PG, uint32_t sQ, uint32_t sQx, uint32_t sK,
                                            uint32_t sKx, uint32_t sV, uint64_t* bar_q_full, uint64_t* bar_q_empty,
                                            uint64_t* bar_k_full, uint64_t* bar_k_empty, uint64_t* bar_v_full,
                                            uint64_t* bar_v_empty, uint64_t* bar_meta, float4* s_kf, float4* s_ve, float* s_qf,
                                            const WaitCtl& ctl, F& piece_of_warp) {
  constexpr int D = C::D, NQ = C::NQ, NK = C::NK, NV = C::NV, GROUPS = D / kInt4Group;
  constexpr bool SPLIT = D == 256;              // keys and values have a warpgroup each
  constexpr int WORDS = D >= 128 ? 16 : 8;      // 8 codes each, of a step: a key's or a value's, or with SPLIT half of them
  constexpr int STEP_GROUPS = WORDS / 8;        // groups of dims of a step
  const int r = thread & 127, role = thread >> 7, lane = r & 31, w = r >> 5;   // role: 1 for the values' warpgroup
  const uint32_t swz = (uint32_t)(r & 7), row_at = (uint32_t)r * 128, ext_at = (uint32_t)(r >> 3) * 256 + (r & 7) * 16;
  uint32_t n_q = 0, n_k = 0;                    // pieces with work, tiles
  Piece pc;
  for (uint32_t it = 0; piece_of_warp(it, pc); ++it) {
    const int n = max(pc.n0, pc.n1), nk = pc.nk, t0 = pc.t0;
    if (n == 0) continue;
    // My key's page in the page table, and where its codes and pairs begin. A key behind the last, or without a page, has scale and
    // zero 0 and any codes.
    const int* table = p.table + pc.b * p.table_stride;
    const long long head = pc.kvh * p.c.head_b, sz_head = pc.kvh * p.c.sz_head_b;
    int page = 0, tok = 0;   // of my key in the tile behind the one that is located; tok < 0: no key
    auto look_up = [&](int t) {
      const int key = t * 128 + r, i = (uint32_t)min(key, nk - 1) / p.div_page;
      page = __ldg(table + i);
      tok = key < nk ? key - i * p.c.page_size : -1;
    };
    uint32_t ksz[GROUPS], vsz[GROUPS];
    if (SPLIT) {   // a role has one of them
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) ksz[g] = vsz[g] = 0u;
    }
    auto fetch_pairs = [&](uint32_t (&x)[GROUPS], const uint8_t* from) {
      if constexpr (GROUPS == 1) {
        x[0] = __ldg(reinterpret_cast<const uint32_t*>(from));
      } else if constexpr (GROUPS == 2) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(from));
        x[0] = u.x, x[1] = u.y;
      } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(from));
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
      }
    };
    long long at = 0;
    bool held = false;   // my key of the located tile is there
    auto locate = [&]() {
      const bool sound = (uint32_t)page < (uint32_t)p.c.num_pages;
      if (tok >= 0 && !sound) atomicCAS(p.status, 0u, kStatusBadPage);
      held = tok >= 0 && sound;
      const int pg = held ? page : 0, tk = held ? tok : 0;   // else the cache's first row
      at = pg * p.c.page_b + tk * p.c.token_b + head;
      const long long sz = pg * p.c.sz_page_b + tk * p.c.sz_token_b + sz_head;
      if (!SPLIT || role == 0) fetch_pairs(ksz, p.c.k_sz + sz);
      if (!SPLIT || role == 1) fetch_pairs(vsz, p.c.v_sz + sz);
    };
    // Codes of two steps, which make a tile: those that are unpacked next, and the ones behind them, on their way.
    uint32_t now[WORDS], next[WORDS];
    auto fetch = [&](uint32_t (&x)[WORDS], int step) {
      const uint8_t* from = ((SPLIT ? role : step) ? p.c.v : p.c.k) + at + (SPLIT ? step * (WORDS * 4) : 0);
#pragma unroll
      for (int i = 0; i < WORDS / 4; ++i) {
        const uint4 u = load_ahead(from + i * 16);
        x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
      }
    };
    look_up(t0);
    locate();
    fetch(now, 0);
    fetch(next, 1);
    if (n > 1) look_up(t0 + 1);

    // Query rows, once the S products of the last piece have read theirs.
    bool ok = n_q == 0 || mbar_wait(smem_addr(bar_q_empty), (n_q - 1) & 1, ctl, SITE_Q_EMPTY);
    if (!__all_sync(0xffffffffu, ok)) return;
    const int pos_r = (uint32_t)r / p.div_g, g_r = r - pos_r * p.G;
#pragma unroll 1
    for (int q = 0; q < NQ; ++q) {
      if ((q ? pc.n1 : pc.n0) == 0) continue;
      const int pos = q * p.P + pos_r;
      const bool valid = r < PG && pos < pc.n_pos;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + ((long long)(pc.q_row + (valid ? pos : 0)) * p.H + pc.kvh * p.G + (valid ? g_r : 0)) * D);
      uint32_t most = 0;
#pragma unroll 8
      for (int i = 0; i < D / 8; ++i) {
        const uint4 u = __ldg(src + i);
        most = max_u16x2(max_u16x2(most, u.x & 0x7fff7fffu), max_u16x2(u.y & 0x7fff7fffu, max_u16x2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
      }
      const uint32_t bits = max(max(most & 0xffffu, most >> 16) >> 7, 8u);   // exponent of the greatest
      const float f = valid ? power_of_bits(261u - bits) : 0.f;
      s_qf[n_q % C::QFS * C::ROWS + q * 128 + r] = power_of_bits(bits - 7u);
      uint32_t ext[4] = {0u, 0u, 0u, 0u};
      const uint32_t to = sQ + q * C::TILE_BYTES + row_at;
#pragma unroll
      for (int g = 0; g < STEP_GROUPS; ++g) {
        const int ch = role * STEP_GROUPS + g;
        float sum = 0.f;
#pragma unroll 2
        for (uint32_t u8 = 0; u8 < 8; ++u8) {
          const uint4 u = valid ? __ldg(src + ch * 8 + u8) : make_uint4(0u, 0u, 0u, 0u);
          const float d0 = __uint_as_float(u.x << 16) * f, d1 = __uint_as_float(u.x & 0xffff0000u) * f;
          const float d2 = __uint_as_float(u.y << 16) * f, d3 = __uint_as_float(u.y & 0xffff0000u) * f;
          const float d4 = __uint_as_float(u.z << 16) * f, d5 = __uint_as_float(u.z & 0xffff0000u) * f;
          const float d6 = __uint_as_float(u.w << 16) * f, d7 = __uint_as_float(u.w & 0xffff0000u) * f;
          sum += ((d0 + d1) + (d2 + d3)) + ((d4 + d5) + (d6 + d7));
          sts128(to + ch * C::CHUNK_BYTES + ((u8 ^ (uint32_t)(r & 7)) << 4),
                 make_uint4(f16x2_pack(d0, d4), f16x2_pack(d1, d5), f16x2_pack(d2, d6), f16x2_pack(d3, d7)));
        }
        const float hi = half_round(sum), lo = sum - hi;
        ext[2 * g] = f16x2_pack(hi, hi), ext[2 * g + 1] = f16x2_pack(lo, lo);
      }
      // 4 more columns of each group, 16 in two core matrices; with SPLIT a thread has one of them
      sts128(sQx + q * C::EXT_BYTES + ext_at + role * 128, make_uint4(ext[0], ext[1], ext[2], ext[3]));
      if (!SPLIT) sts128(sQx + q * C::EXT_BYTES + ext_at + 128, make_uint4(0u, 0u, 0u, 0u));
    }
    fence_async_proxy();
    __syncwarp();
    warp_arrive(lane == 0, smem_addr(bar_q_full));
    ++n_q;

    for (int j = 0; j < n; ++j, ++n_k) {
      const uint32_t ks = n_k % NK, vs = n_k % NV, meta = n_k % C::METAS;
      // Powers of two of my warp's keys and values.
      uint32_t mk = 0, mv = 0;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        if (!SPLIT || role == 0) ksz[g] = held ? ksz[g] : 0u;
        if (!SPLIT || role == 1) vsz[g] = held ? vsz[g] : 0u;
        const float scale = __uint_as_float(ksz[g] << 16), zero = __uint_as_float(ksz[g] & 0xffff0000u);
        mk = max(mk, __float_as_uint(fmaxf(fabsf(scale) * 24.f, fabsf(fmaf(8.f, scale, zero)))));
        const float vscale = __uint_as_float(vsz[g] << 16), vzero = __uint_as_float(vsz[g] & 0xffff0000u);
        mv = max(mv, __float_as_uint(fmaf(16.f, fabsf(vscale), fabsf(vzero))));
      }
      const uint32_t bk = min(max(__reduce_max_sync(0xffffffffu, mk) >> 23, 15u), 254u);
      // Not below 2^-80: weights without their powers are summed in fp32.
      const uint32_t bv = min(max(__reduce_max_sync(0xffffffffu, mv) >> 23, 61u), 254u);
      const float fk = power_of_bits(268u - bk), fv = power_of_bits(268u - bv);
      auto publish = [&](bool keys, bool values) {
        // by all lanes: the same value
        if (keys) reinterpret_cast<float*>(s_kf + meta)[w] = power_of_bits(bk - 14u);
        if (values) reinterpret_cast<float*>(s_ve + meta)[w] = (float)((int)bv - 141);
        warp_arrive(lane == 0, smem_addr(&bar_meta[meta]));
      };
      // The softmax needs the values' powers before their stage is free. (It has read this slot's last: that tile's PV is done.)
      if (SPLIT && role) publish(false, true);
      {
        const bool values = SPLIT && role;
        uint64_t* bar = values ? &bar_v_empty[vs] : &bar_k_empty[ks];
        ok = n_k < (uint32_t)NK || mbar_wait(smem_addr(bar), (n_k / NK - 1) & 1, ctl, SITE_KV_EMPTY);
        if (!__all_sync(0xffffffffu, ok)) return;
      }
      if (!SPLIT || !role) publish(true, !SPLIT);
      // What codes are multiplied with and what is added, a pair of fp16 of each group.
      uint32_t kpair[GROUPS], vpair[GROUPS], ext[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) ext[i] = 0u;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const float scale = __uint_as_float(ksz[g] << 16) * fk, zero = __uint_as_float(ksz[g] & 0xffff0000u) * fk;
        const float z = fmaf(8.f, scale, zero), hi = half_round(z);
        kpair[g] = f16x2_pack(16.f * scale, -24.f * scale);
        ext[2 * g] = ext[2 * g + 1] = f16x2_pack(hi, z - hi);
        const float vscale = __uint_as_float(vsz[g] << 16) * fv, vzero = __uint_as_float(vsz[g] & 0xffff0000u) * fv;
        vpair[g] = f16x2_pack(16.f * vscale, fmaf(-16.f, vscale, vzero));
      }
      if (!SPLIT || !role) {
        sts128(sKx + ks * C::EXT_BYTES + ext_at, make_uint4(ext[0], ext[1], ext[2], ext[3]));
        sts128(sKx + ks * C::EXT_BYTES + ext_at + 128, make_uint4(ext[4], ext[5], ext[6], ext[7]));
      }
      // The next tile's pairs, and its row for the codes.
      if (j + 1 < n) {
        locate();
        if (j + 2 < n) look_up(t0 + j + 2);
      }
      // One loop for keys and values: the roles' code would not stay in the instruction caches (with both unrolled, 0.8 warps a
      // scheduler waited for instructions at any time).
#pragma unroll 1
      for (int step = 0; step < 2; ++step) {
        const bool is_v = (SPLIT ? role : step) != 0;
        if (!SPLIT && is_v) {
          ok = n_k < (uint32_t)NV || mbar_wait(smem_addr(&bar_v_empty[vs]), (n_k / NV - 1) & 1, ctl, SITE_KV_EMPTY);
          if (!__all_sync(0xffffffffu, ok)) return;
        }
        uint32_t s2[STEP_GROUPS], z2[STEP_GROUPS];
#pragma unroll
        for (int g = 0; g < STEP_GROUPS; ++g) {
          const int at_g = (g + STEP_GROUPS) % GROUPS;   // SPLIT: of the second half
          const uint32_t kk = SPLIT && step ? kpair[at_g] : kpair[g], vv = SPLIT && step ? vpair[at_g] : vpair[g];
          const uint32_t pair = is_v ? vv : kk;
          s2[g] = __byte_perm(pair, 0, 0x1010), z2[g] = __byte_perm(pair, 0, 0x3232);
        }
        const uint32_t stage = is_v ? sV + vs * C::TILE_BYTES : sK + ks * C::TILE_BYTES;
        const uint32_t to = (stage + row_at + (SPLIT ? step * (STEP_GROUPS * C::CHUNK_BYTES) : 0)) | swz << 4;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
          // Codes m and m + 4 in the high bits of fp16's mantissa, 1 + code / 16.
          const uint32_t x = now[i], mask = 0x03c003c0u, one = 0x3c003c00u, s = s2[i / 8], z = z2[i / 8];
          sts128((to ^ i % 8 << 4) + i / 8 * C::CHUNK_BYTES,
                 make_uint4(half2_fma((x << 6 & mask) | one, s, z), half2_fma((x << 2 & mask) | one, s, z),
                            half2_fma((x >> 2 & mask) | one, s, z), half2_fma((x >> 6 & mask) | one, s, z)));
        }
        if (!SPLIT || step) {
          fence_async_proxy();
          __syncwarp();
          warp_arrive(lane == 0, smem_addr(is_v ? &bar_v_full[vs] : &bar_k_full[ks]));
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i) now[i] = next[i];
        if (j + 1 < n) fetch(next, step);   // of the next tile
      }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
attn_paged_varlen_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedVarlenParams p) {
  constexpr int D = C::D, NQ = C::NQ, NCH = C::NCH, NK = C::NK, NV = C::NV, NSB = C::NSB;
  constexpr bool INT4 = C::INT4;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q_full, bar_q_empty, bar_k_full[NK], bar_k_empty[NK], bar_v_full[NV], bar_v_empty[NV];
  __shared__ __align__(8) uint64_t bar_s_full[NQ * NSB], bar_s_free[NSB], bar_p_half[NQ][2], bar_o_done[NQ], bar_o_full[NQ];
  __shared__ __align__(8) uint64_t bar_piece_full[C::PIECES], bar_piece_empty[C::PIECES], bar_patch[2], bar_drain[NQ + 1];
  __shared__ __align__(8) uint64_t bar_meta[C::METAS];
  __shared__ Piece s_pieces[C::PIECES];
  // 4 bits: powers of two of the keys (as factors of S) and values (as exponents) of every 32 keys of a tile, and of the
  // query rows.
  __shared__ float4 s_kf[INT4 ? C::METAS : 1], s_ve[INT4 ? C::METAS : 1];
  __shared__ float s_qf[INT4 ? C::QFS * C::ROWS : 1];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem_base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = smem_base, sK = sQ + C::Q_BYTES, sV = sK + NK * C::TILE_BYTES;
  const uint32_t sQx = sV + NV * C::TILE_BYTES, sKx = sQx + NQ * C::EXT_BYTES;
  const WaitCtl ctl{&abort_flag, p.status, p.timeout_ns};

  if (tid == 0) {
    abort_flag = 0u;
    mbar_init(smem_addr(&bar_q_full), INT4 ? C::FEED_WARPS : 1);
    mbar_init(smem_addr(&bar_q_empty), 1);
    for (int i = 0; i < NK; ++i) mbar_init(smem_addr(&bar_k_full[i]), C::FEEDERS), mbar_init(smem_addr(&bar_k_empty[i]), 1);
    for (int i = 0; i < NV; ++i) mbar_init(smem_addr(&bar_v_full[i]), C::FEEDERS), mbar_init(smem_addr(&bar_v_empty[i]), NQ);
    for (int i = 0; i < NQ * NSB; ++i) mbar_init(smem_addr(&bar_s_full[i]), 1);
    for (int i = 0; i < NSB; ++i) mbar_init(smem_addr(&bar_s_free[i]), 4);
    for (int i = 0; i < NQ; ++i) {
      mbar_init(smem_addr(&bar_p_half[i][0]), 4);
      mbar_init(smem_addr(&bar_p_half[i][1]), 4);
      mbar_init(smem_addr(&bar_o_done[i]), 1);
      mbar_init(smem_addr(&bar_o_full[i]), 1);
    }
    for (int i = 0; i < C::PIECES; ++i) {
      mbar_init(smem_addr(&bar_piece_full[i]), 1);
      mbar_init(smem_addr(&bar_piece_empty[i]), C::CONSUMERS);
    }
    for (int i = 0; i < C::METAS; ++i) mbar_init(smem_addr(&bar_meta[i]), C::FEED_WARPS);
    for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&bar_patch[i]), 1);
    for (int i = 0; i < NQ + 1; ++i) mbar_init(smem_addr(&bar_drain[i]), 1);
    fence_mbar_init();
  }
  if (warp == C::WARP_PV) {
    tmem_alloc(smem_addr(&tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (!INT4 && p.P * p.G < 128) {   // rows of the Q tiles that no load writes
    for (int i = tid; i < C::Q_BYTES / 16; i += C::THREADS) sts128(sQ + 16 * i, make_uint4(0u, 0u, 0u, 0u));
    fence_async_proxy();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();   // launched early: what it reads may be a previous kernel's
  griddep_launch_dependents();   // the joining kernel's CTAs come where these end (each has nearly all registers of its SM)
  const uint32_t tmem = tmem_slot;
  const int PG = p.P * p.G, RP = p.P * NQ;

  auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {   // by a whole warp
    const bool w = mbar_wait(bar, parity, ctl, site);
    return __all_sync(0xffffffffu, w) != 0;
  };
  // Pieces as their consumers see them; `it` counts those taken.
  auto wait_piece = [&](uint32_t it) {
    const uint32_t i = it % C::PIECES;
    const bool w = mbar_wait(smem_addr(&bar_piece_full[i]), (it / C::PIECES) & 1, ctl, SITE_PIECE_FULL);
    return __all_sync(0xffffffffu, w) && s_pieces[i].work != 0;
  };
  auto release_piece = [&](uint32_t it) {
    __syncwarp();
    warp_arrive(lane == 0, smem_addr(&bar_piece_empty[it % C::PIECES]));
  };
  auto piece_of_warp = [&](uint32_t it, Piece& pc) {
    if (!wait_piece(it)) return false;
    pc = s_pieces[it % C::PIECES];
    release_piece(it);
    return true;
  };

  if (warp == C::WARP_PLAN) {
    // ------------------------------------------------------------------ scheduler, and copies of queries over a bf16 cache
    setmaxnreg_dec<C::REGS_ROLES>();
    if (!INT4 && lane == 0) tma_prefetch_desc(&tm_q);
    uint32_t n_pieces = 0, n_q = 0;   // published, Q loads
    bool ok = true;
    // Publishes a piece; its consumers are at most PIECES behind.
    auto publish = [&](const Piece& pc) {
      const uint32_t i = n_pieces % C::PIECES;
      if (n_pieces >= (uint32_t)C::PIECES) {
        const bool w = mbar_wait(smem_addr(&bar_piece_empty[i]), (n_pieces / C::PIECES - 1) & 1, ctl, SITE_PIECE_EMPTY);
        if (!__all_sync(0xffffffffu, w)) return false;
      }
      if (lane == 0) {
        s_pieces[i] = pc;
        mbar_arrive(smem_addr(&bar_piece_full[i]));
      }
      __syncwarp();
      ++n_pieces;
      return true;
    };
    // The query rows of a piece, once the S products of the last one have read theirs.
    auto load_queries = [&](const Piece& pc) {
      if (INT4 || (pc.n0 == 0 && pc.n1 == 0)) return true;
      const bool w = n_q == 0 || mbar_wait(smem_addr(&bar_q_empty), (n_q - 1) & 1, ctl, SITE_Q_EMPTY);
      if (!__all_sync(0xffffffffu, w)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_addr(&bar_q_full), ((pc.n0 > 0) + (pc.n1 > 0)) * NCH * PG * 128);
        for (int q = 0; q < NQ; ++q) {
          if ((q ? pc.n1 : pc.n0) == 0) continue;
          for (int ch = 0; ch < NCH; ++ch)
            tma_load_4d(sQ + (q * NCH + ch) * C::CHUNK_BYTES, &tm_q, smem_addr(&bar_q_full), ch * 64, 0, pc.q_row + q * p.P, pc.kvh);
        }
      }
      ++n_q;
      return true;
    };

    // Sequence b as far as the offsets and lengths are sound; nq = 0 otherwise.
    auto sequence = [&](int b, int& q_base) {
      UnitWork s{0, 0, 0, RP, C::ONE, C::TWO, p.causal};
      q_base = 0;
      if (b < p.B) {
        const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), n = __ldg(p.lens + b);
        const int nk = min(max(n, 0), p.max_pages * p.c.page_size);   // the host refuses tables of more
        const bool good = c0 >= 0 && c1 >= c0 && c1 <= p.total_q;
        if (!good || nk != n) atomicCAS(p.status, 0u, kStatusBadPage);
        if (good && !(p.skip_singles && c1 - c0 == 1)) q_base = c0, s.nq = c1 - c0, s.nk = nk, s.M = (s.nq + RP - 1) / RP;
      }
      return s;
    };
    // Sequence b0 + lane; work of a kv head of it, of all its heads, and of all 32 sequences up to it.
    UnitWork s;
    int q_base;
    long long per, mine, upto;
    auto costs = [&](int b0) {
      s = sequence(b0 + lane, q_base);
      per = s.upto(s.M);
      mine = p.c.Hkv * per;
      upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
    };
    // All work, dealt to the CTAs in equal contiguous shares: mine is [x0, x1).
    long long W = 0, x0 = 0, x1 = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) costs(b0), W = min(W + __shfl_sync(0xffffffffu, upto, 31), 2 * kMostWork);
    if (W > kMostWork) {   // the host refuses calls of more: offsets whose sequences share rows
      if (lane == 0) atomicCAS(p.status, 0u, kStatusBadPage);
      W = 0;
    }
    const int shares = (int)max(1LL, min((long long)gridDim.x, W / kLeastShare)), me = blockIdx.x;
    int4 cut0 = make_int4(0, 0, 0, 0);
    if (me < shares && W > 0) {
      // Divisions in 64 bits, some 500 cycles each, go to lanes that do them at once.
      x0 = (me + (lane & 1)) * W / shares;
      x1 = __shfl_sync(0xffffffffu, x0, 1);
      x0 = __shfl_sync(0xffffffffu, x0, 0);
      // The sequence, kv head and unit that x0 lies in.
      int b = 0, kvh = 0, m = 0;
      long long before = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        if (p.B > 32) costs(b0);   // else still those of the first look
        const long long all = __shfl_sync(0xffffffffu, upto, 31);
        if (before + all > x0) {
          const int i = __popc(__ballot_sync(0xffffffffu, before + upto <= x0));
          b = b0 + i;
          before += __shfl_sync(0xffffffffu, upto - mine, i);
          per = __shfl_sync(0xffffffffu, per, i);
          q_base = __shfl_sync(0xffffffffu, q_base, i);
          s.nq = __shfl_sync(0xffffffffu, s.nq, i), s.nk = __shfl_sync(0xffffffffu, s.nk, i), s.M = __shfl_sync(0xffffffffu, s.M, i);
          break;
        }
        before += all;
      }
      {
        const long long rest = x0 - before;
        for (int ended = 32, k0 = 0; ended == 32; k0 += 32) {   // kv heads that end at x0 or before
          ended = __popc(__ballot_sync(0xffffffffu, (k0 + lane + 1) * per <= rest));
          kvh += ended;
        }
        const long long in = rest - kvh * per;
        int n = s.M;   // the last unit that begins at `in` or before
        while (n > 1) {
          const int step = (n + 31) / 32, i = m + lane * step;
          const uint32_t ballot = __ballot_sync(0xffffffffu, lane * step < n && s.upto(i) <= in);
          const int k = __popc(ballot) - 1;
          m += k * step;
          n = min(step, n - k * step);
        }
        before += kvh * per + s.upto(m);
      }
      while (ok && before < x1) {
        const int keys = s.keys(m), n = (keys + 127) / 128, per = 128 * s.a_key(m);   // per: work of a tile
        const long long end = before + kUnitOverhead + keys * (long long)(per / 128);
        // The tiles that places x0 and x1 of all work lie at, by lanes 0 and 1. Lane 2: the share that begins at or behind the place
        // where the last tile is reached.
        const long long place = min(end, before + kUnitOverhead + (long long)per * n - per / 2);
        const long long from = (lane == 1 ? x1 : x0) - before - kUnitOverhead + per / 2;
        const long long quotient = (lane == 2 ? place * shares + W - 1 : max(from, 0LL)) / (lane == 2 ? W : (long long)per);
        const int at = (int)min(quotient, (long long)(lane == 2 ? shares : n));
        const int at0 = __shfl_sync(0xffffffffu, at, 0), at1 = __shfl_sync(0xffffffffu, at, 1), at2 = __shfl_sync(0xffffffffu, at, 2);
        const int t0 = x0 > before ? at0 : 0, t1 = x1 >= end ? n : at1;
        if (t1 > t0 || (n == 0 && before >= x0)) {
          const bool whole = t0 == 0 && t1 == n;
          Piece pc = {};
          pc.work = 1;
          pc.q_row = q_base + m * RP;
          pc.n_pos = min(RP, s.nq - m * RP);
          pc.kvh = kvh, pc.b = b, pc.nk = s.nk, pc.t0 = t0;
          pc.vis = m * RP + s.nk - s.nq;
          auto tiles_of = [&](int q) {
            const int last = min((q + 1) * p.P, pc.n_pos);   // positions up to the end of Q tile q
            if (last <= q * p.P) return 0;
            const int seen = p.causal ? pc.vis + last : s.nk;
            return seen <= 0 ? 0 : max(min((seen + 127) / 128, t1) - t0, 0);
          };
          pc.n0 = tiles_of(0);
          pc.n1 = NQ == 2 ? tiles_of(1) : 0;
          pc.slot = whole ? -1 : t0 > 0 ? 2 * me : 2 * me + 1;
          if (t0 == 0 && !whole) {
            // Parts: mine, and one of each CTA whose share begins before the place where the last tile is reached.
            cut0 = make_int4(pc.q_row, pc.kvh, pc.n_pos, at2 - me);
          }
          ok = publish(pc) && load_queries(pc);
        }
        before = end;
        if (++m == s.M) {
          m = 0;
          if (++kvh == p.c.Hkv) {
            kvh = 0;
            // The next sequence with queries.
            int b0 = b + 1;
            b = p.B;
            for (; b0 < p.B; b0 += 32) {
              const int i = b0 + lane;
              const bool any = i < p.B && __ldg(p.cu + i + 1) > __ldg(p.cu + i);
              const uint32_t ballot = __ballot_sync(0xffffffffu, any);
              if (ballot) {
                b = b0 + __ffs(ballot) - 1;
                s = sequence(b, q_base);
                if (s.M > 0) break;
                b0 = b - 31;   // unsound: on behind it
                b = p.B;
              }
            }
            if (b == p.B) break;
          }
        }
      }
    }
    if (lane == 0) p.cut[me] = cut0;
    if (ok) {
      Piece none = {};
      publish(none);
    } else if (n_q > 0) {   // unwinding: let the copies still in flight land before the CTA exits
      land(&bar_q_full, n_q - 1, p.timeout_ns);
    }
  } else if (warp >= C::WARP_PV && warp < C::WARP_PV + NQ) {
    // ------------------------------------------------------------------ PV issuer, one per Q tile
    setmaxnreg_dec<C::REGS_ROLES>();
    const bool on = elect_one();
    const int q = warp - C::WARP_PV;
    const uint32_t d_o = tmem + C::O_COL + q * D, a_p = tmem + C::P_COL + C::P_COLS * q;
    uint32_t n_v = 0, g = 0;   // V tiles of the CTA, products of this Q tile
    bool ok = true;
    Piece pc;
    for (uint32_t it = 0; ok && piece_of_warp(it, pc); ++it) {
      const int n = q ? pc.n1 : pc.n0, n_all = max(pc.n0, pc.n1);
      for (int j = 0; ok && j < n_all; ++j, ++n_v) {
        const uint32_t vs = n_v % NV;
        if (!wait(smem_addr(&bar_v_full[vs]), (n_v / NV) & 1, SITE_KV_FULL)) { ok = false; break; }
        if (j < n) {
          const uint64_t b_v = make_sdesc_swz(sV + vs * C::TILE_BYTES, C::CHUNK_BYTES, C::SBO, C::SWZ);
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // as the softmax hands P over
            if (!wait(smem_addr(&bar_p_half[q][h]), g & 1, SITE_P_FULL)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < C::KSTEPS_PV / 2; ++i) {
              const int k = h * (C::KSTEPS_PV / 2) + i;
              warp_mma_ts(on, d_o, a_p + k * 8, b_v + (uint64_t)((k * C::PV_ROWS * C::SWZ) >> 4), C::IDESC_PV, k > 0 || j > 0 ? 1u : 0u);
            }
          }
          if (!ok) break;
          warp_commit(on, smem_addr(&bar_o_done[q]));
          if (j + 1 == n) warp_commit(on, smem_addr(&bar_o_full[q]));
          warp_commit(on, smem_addr(&bar_v_empty[vs]));
          ++g;
        } else {
          warp_arrive(lane == 0, smem_addr(&bar_v_empty[vs]));
        }
      }
    }
    // Every MMA this warp issued must finish before TMEM is released.
    warp_commit(on, smem_addr(&bar_drain[q]));
    land(&bar_drain[q], 0, p.timeout_ns);
  } else if (warp == C::WARP_S) {
    // ------------------------------------------------------------------ S issuer
    setmaxnreg_dec<C::REGS_ROLES>();
    const bool on = elect_one();
    const uint32_t idesc = C::IDESC_QK | p.qk_negate;
    uint32_t n_k = 0, n_q = 0, k = 0, g0 = 0, g1 = 0;   // K tiles, Q loads, S products of the CTA and of each Q tile
    bool ok = true;
    Piece pc;
    for (uint32_t it = 0; ok && piece_of_warp(it, pc); ++it) {
      const int n_all = max(pc.n0, pc.n1);
      if (n_all == 0) continue;
      if (!wait(smem_addr(&bar_q_full), n_q & 1, SITE_Q_FULL)) { ok = false; break; }
      ++n_q;
      for (int j = 0; ok && j < n_all; ++j, ++n_k) {
        const uint32_t ks = n_k % NK;
        if (!wait(smem_addr(&bar_k_full[ks]), (n_k / NK) & 1, SITE_KV_FULL)) { ok = false; break; }
        for (int q = 0; ok && q < NQ; ++q) {
          if (j >= (q ? pc.n1 : pc.n0)) continue;
          uint32_t& g = q ? g1 : g0;
          const uint32_t b = k % NSB;
          if (k >= (uint32_t)NSB && !wait(smem_addr(&bar_s_free[b]), (k / NSB - 1) & 1, SITE_S_FREE)) { ok = false; break; }
          tc_fence_after();
          const uint64_t dq = make_sdesc_swz(sQ + q * C::TILE_BYTES, 16, C::SBO, C::SWZ);
          const uint64_t dk = make_sdesc_swz(sK + ks * C::TILE_BYTES, 16, C::SBO, C::SWZ);
#pragma unroll
          for (int i = 0; i < C::KSTEPS_QK; ++i) {   // 4 steps of 32 bytes to a swizzle row
            const uint64_t off = (uint64_t)(((i / 4) * C::CHUNK_BYTES + (i % 4) * 32) >> 4);
            warp_mma_ss(on, tmem + b * 128u, dq + off, dk + off, idesc, i > 0 ? 1u : 0u);
          }
          if constexpr (INT4)
            warp_mma_ss(on, tmem + b * 128u, make_sdesc_plain(sQx + q * C::EXT_BYTES, 128, 256),
                        make_sdesc_plain(sKx + ks * C::EXT_BYTES, 128, 256), idesc, 1u);
          warp_commit(on, smem_addr(&bar_s_full[q * NSB + g % NSB]));
          ++g;
          ++k;
        }
        if (!ok) break;
        warp_commit(on, smem_addr(&bar_k_empty[ks]));
        if (j + 1 == n_all) warp_commit(on, smem_addr(&bar_q_empty));
      }
    }
    warp_commit(on, smem_addr(&bar_drain[NQ]));
    land(&bar_drain[NQ], 0, p.timeout_ns);
  } else if (warp >= C::WARP_FEED) {
    // ------------------------------------------------------------------ bf16: copies of keys and values. 4 bits: query rows, keys and
    // values to fp16
    setmaxnreg_dec<C::REGS_FEED>();
    if constexpr (!INT4) {
      if (warp < C::WARP_FEED + 2)
        load_role<C, false>(p, warp & 1, &tm_k, sK, bar_k_full, bar_k_empty, &bar_patch[warp & 1], ctl, piece_of_warp);
      else
        load_role<C, true>(p, warp & 1, &tm_v, sV, bar_v_full, bar_v_empty, &bar_patch[warp & 1], ctl, piece_of_warp);
    } else {
      unpack_role<C>(p, tid - 32 * C::WARP_FEED, PG, sQ, sQx, sK, sKx, sV, &bar_q_full, &bar_q_empty, bar_k_full, bar_k_empty,
                     bar_v_full, bar_v_empty, bar_meta, s_kf, s_ve, s_qf, ctl, piece_of_warp);
    }
  } else if (warp < C::SOFTMAX_WARPS) {
    // ------------------------------------------------------------------ softmax + epilogue
    setmaxnreg_inc<C::REGS_SOFTMAX>();
    const int qt = warp >> 2, r = ((warp & 3) << 5) + lane;   // Q tile; row in it == TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) << 5) << 16;
    const uint32_t tP = tmem + lane_base + C::P_COL + C::P_COLS * qt, tO = tmem + lane_base + C::O_COL + qt * D;
    // S products of the CTA, of this tile; KV tiles; pieces with work, of the CTA and of this tile
    uint32_t sbase = 0, g = 0, n_kv = 0, n_q = 0, done = 0;
    bool ok = true;
    // P is 2^kUp times larger over 4-bit caches: fp16 then loses 2^-32 of a row's greatest weight times value at most.
    constexpr float kUp = INT4 ? 7.0f : 0.0f;
    auto s_ready = [&](uint32_t n) {   // S product number n of this tile
      return mbar_wait(smem_addr(&bar_s_full[qt * NSB + n % NSB]), (n / NSB) & 1, ctl, SITE_S_FULL);
    };
    for (uint32_t it = 0; ok && wait_piece(it); ++it) {
      const Piece& pc = s_pieces[it % C::PIECES];   // read where it is: registers are short
      const int n0 = pc.n0, n1 = pc.n1, n = qt ? n1 : n0, key_first = pc.t0 * 128, nk = pc.nk;
      const uint32_t sb = sbase, gb = g, kvb = n_kv;
      sbase += (uint32_t)(n0 + n1);
      g += (uint32_t)n;
      n_kv += (uint32_t)max(n0, n1);
      const int vis_first = pc.vis + qt * p.P;   // keys that the tile's first query sees, less one
      const int seen = p.causal ? min(nk, vis_first + (int)((uint32_t)r / p.div_g) + 1) : nk;   // this row: the first so many
      float s = p.scale_log2;
      if (INT4 && n > 0) {
        // The rows' powers of two come with the query rows.
        const bool w = s_ready(gb);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        s *= s_qf[n_q % C::QFS * C::ROWS + qt * 128 + r];
      }
      n_q += n0 > 0 || n1 > 0;
      float m = -INFINITY;   // running max (log2 units), the exponents' shift
      float l = 0.0f;        // running sum of exp2(s x - m)
      for (int j = 0; j < n; ++j) {
        const uint32_t gj = gb + j;
        float sc[4], ve[4];   // scale of the scores and, over 4 bits, exponent of the values, of 32 keys each
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = s, ve[i] = 0.f;
        if constexpr (INT4) {
          const uint32_t t = kvb + j, meta = t % C::METAS;
          const bool w = mbar_wait(smem_addr(&bar_meta[meta]), (t / C::METAS) & 1, ctl, SITE_META);
          if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
          const float4 f = s_kf[meta], e = s_ve[meta];
          // never 0, which would make NaN of a masked score; scores that small are 0 either way
          constexpr float kLeast = 0x1p-126f;
          sc[0] = fmaxf(s * f.x, kLeast), sc[1] = fmaxf(s * f.y, kLeast), sc[2] = fmaxf(s * f.z, kLeast), sc[3] = fmaxf(s * f.w, kLeast);
          ve[0] = e.x, ve[1] = e.y, ve[2] = e.z, ve[3] = e.w;
        }
        const bool w = s_ready(gj);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        const int key0 = key_first + j * 128;
        const bool masked = key0 + 128 > nk || (p.causal && key0 + 127 > vis_first);
        tc_fence_after();
        const uint32_t sbuf = NSB == 1 ? 0u : s_number(sb, qt, j, n0, n1) % NSB;
        const uint32_t tS = tmem + lane_base + sbuf * 128u;
        const int lim = seen - key0;   // keys of the tile that the row sees
        // COLS columns of S from column c0 on and the maxima of every 32 of them, which the load takes on the way (NaN ignored);
        // columns that the row does not see are -inf.
        auto load_scores = [&](int c0, auto& x, float* top) {
          constexpr int COLS = sizeof(x) / 4;
          uint32_t* bits = reinterpret_cast<uint32_t*>(x);
#pragma unroll
          for (int i = 0; i < COLS / 32; ++i) tmem_ld_32cols_max(tS + c0 + 32 * i, bits + 32 * i, top[i]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < COLS / 32; ++i) {
            reg_fence32(bits + 32 * i);
            asm volatile("" : "+f"(top[i]));
          }
        };
        auto mask_scores = [&](int c0, auto& x, float* top) {
          constexpr int COLS = sizeof(x) / 4;
#pragma unroll
          for (int c = 0; c < COLS; ++c)
            if (c0 + c >= lim) x[c] = -INFINITY;
#pragma unroll
          for (int i = 0; i < COLS / 32; ++i) {
            const float* y = x + 32 * i;
            float a[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) a[c] = fmax3(y[c], y[c + 4], y[c + 8]);
#pragma unroll
            for (int c = 12; c + 8 <= 32; c += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) a[k] = fmax3(a[k], y[c + k], y[c + 4 + k]);
#pragma unroll
            for (int c = 0; c < 4; ++c) a[c] = fmaxf(a[c], y[28 + c]);
            top[i] = fmaxf(fmax3(a[0], a[1], a[2]), a[3]);
          }
        };
        auto scores_taken = [&]() {   // S is in registers: its buffer may take the next
          tc_fence_before();
          __syncwarp();
          warp_arrive(lane == 0, smem_addr(&bar_s_free[sbuf]));
        };
        // P = exp2(s x + ve - m) of 64 keys, in pairs; their sum, in fp32, without the values' powers. P is rounded to the values' type, as
        // a product has one: bf16, 2^-8 off (O's error 0.0023 of its norm, 0.0017 without; a second number for the rest would be the
        // second product again), or fp16, 2^-11.
        auto exp_half = [&](const float* x, float s_lo, float s_hi, float e_lo, float e_hi, uint32_t* pk) {
          float sum = 0.f;
          if constexpr (INT4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float e = i ? e_hi : e_lo, add = e - m + kUp, f = i ? s_hi : s_lo;
              const uint64_t s2 = f2_pack(f, f), a2 = f2_pack(add, add);
              uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const float* y = x + 32 * i + c;
                float t0, t1, t2, t3;
                f2_unpack(f2_fma(f2_pack(y[0], y[1]), s2, a2), t0, t1);
                f2_unpack(f2_fma(f2_pack(y[2], y[3]), s2, a2), t2, t3);
                const float p0 = ex2(t0), p1 = ex2(t1), p2 = ex2(t2), p3 = ex2(t3);
                acc0 = c ? f2_add(acc0, f2_pack(p0, p1)) : f2_pack(p0, p1);
                acc1 = c ? f2_add(acc1, f2_pack(p2, p3)) : f2_pack(p2, p3);
                pk[i * 16 + (c >> 1)] = f16x2_pack(p0, p1);
                pk[i * 16 + (c >> 1) + 1] = f16x2_pack(p2, p3);
              }
              float l0, l1;
              f2_unpack(f2_add(acc0, acc1), l0, l1);
              sum = fmaf(l0 + l1, ex2(-e), sum);
            }
          } else {
            const uint64_t s2 = f2_pack(s, s), a2 = f2_pack(-m, -m);
            uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              float t0, t1, t2, t3;
              f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), s2, a2), t0, t1);
              f2_unpack(f2_fma(f2_pack(x[c + 2], x[c + 3]), s2, a2), t2, t3);
              const float p0 = ex2(t0), p1 = ex2(t1), p2 = ex2(t2), p3 = ex2(t3);
              acc0 = c ? f2_add(acc0, f2_pack(p0, p1)) : f2_pack(p0, p1);
              acc1 = c ? f2_add(acc1, f2_pack(p2, p3)) : f2_pack(p2, p3);
              pk[c >> 1] = pack_bf16x2(p0, p1);
              pk[(c >> 1) + 1] = pack_bf16x2(p2, p3);
            }
            float l0, l1;
            f2_unpack(f2_add(acc0, acc1), l0, l1);
            sum = l0 + l1;
          }
          return sum;
        };
        auto store_half = [&](int h, const uint32_t* pk) {
          tmem_st_32cols(tP + h * 32, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          warp_arrive(lane == 0, smem_addr(&bar_p_half[qt][h]));
        };
        // PV_{j-1} reads the last P, and adds to O, which a rescale changes.
        bool pv_done = j == 0;
        auto wait_pv = [&]() {
          const bool done_ = pv_done || mbar_wait(smem_addr(&bar_o_done[qt]), (gj - 1) & 1, ctl, SITE_O_DONE);
          pv_done = true;
          return __all_sync(0xffffffffu, done_);
        };
        float alpha = 1.0f, sum = 0.f;
        auto move_max = [&](float m_tile) {
          bool rescale = false;
          if (m_tile > m + 8.0f) {
            alpha = ex2(m - m_tile);   // 0 on the first tile
            m = m_tile;
            rescale = true;
          }
          if (__any_sync(0xffffffffu, rescale) && j > 0) {
            if (!wait_pv()) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t ov[32];
              tmem_ld_32cols(tO + c0, ov);
              tmem_ld_wait();
              reg_fence32(ov);
#pragma unroll
              for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
              tmem_st_32cols(tO + c0, ov);
            }
          }
          return true;
        };
        uint32_t pk[32];
        float x[128], top[4];
        load_scores(0, x, top);
        scores_taken();
        if (masked) mask_scores(0, x, top);
        float m_tile;
        if constexpr (INT4)
          m_tile = fmaxf(fmaxf(fmaf(top[0], sc[0], ve[0]), fmaf(top[1], sc[1], ve[1])),
                         fmaxf(fmaf(top[2], sc[2], ve[2]), fmaf(top[3], sc[3], ve[3])));
        else
          m_tile = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * s;
        if (!move_max(m_tile)) { ok = false; break; }
        sum = exp_half(x, sc[0], sc[1], ve[0], ve[1], pk);
        if (!wait_pv()) { ok = false; break; }
        store_half(0, pk);
        sum += exp_half(x + 64, sc[2], sc[3], ve[2], ve[3], pk);
        store_half(1, pk);
        l = l * alpha + sum;
      }
      if (!ok) break;
      // Epilogue: O / l, LSE. A row that sees no key of the piece gives 0 and -inf; its accumulator holds nothing.
      if (n > 0) {
        const bool w = mbar_wait(smem_addr(&bar_o_full[qt]), done & 1, ctl, SITE_O_FULL);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        ++done;
        tc_fence_after();
      }
      const int pos_r = (uint32_t)r / p.div_g, g_r = r - pos_r * p.G, pos = qt * p.P + pos_r;   // position in the unit, head
      const bool valid = r < PG && pos < pc.n_pos;
      const int slot = pc.slot, q_row = pc.q_row, head = pc.kvh * p.G + g_r;
      release_piece(it);   // before the stores, which a later arrival would wait for
      const bool none = seen <= key_first || n == 0;   // no key of the piece
      const float inv_l = 1.0f / l, lse2 = none ? -INFINITY : m + log2f(l) - kUp;
      // Column of dim i of a group of 8: 4-bit codes are unpacked in the order 0 4 1 5 2 6 3 7.
      auto col = [](int c) { return INT4 ? (c & ~7) | ((c & 3) << 1) | ((c >> 2) & 1) : c; };
      if (slot < 0) {
        const long long row = (long long)(q_row + pos) * p.H + head;
        __nv_bfloat16* orow = p.o + row * D;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 64) {
          uint32_t pk[32];
          if (n > 0) {   // the same for the whole warp
            uint32_t ov[64];
            tmem_ld_32cols(tO + c0, ov);
            tmem_ld_32cols(tO + c0 + 32, ov + 32);
            tmem_ld_wait();
            reg_fence32(ov);
            reg_fence32(ov + 32);
#pragma unroll
            for (int c = 0; c < 64; c += 2)
              pk[c >> 1] = none ? 0u
                                : pack_bf16x2(__uint_as_float(ov[col(c)]) * inv_l, __uint_as_float(ov[col(c + 1)]) * inv_l);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = 0u;
          }
          if (valid) {
            if (p.o_v8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) st_global_v8(orow + c0 + 16 * i, pk + 8 * i);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(orow + c0);
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
            }
          }
        }
        if (valid) p.lse[(long long)head * p.total_q + q_row + pos] = lse2 * 0.69314718055994531f;
      } else {
        const long long row = (long long)slot * C::ROWS + qt * 128 + r;
        float* orow = p.part_o + row * D;
        if (n > 0) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t ov[32], out[32];
            tmem_ld_32cols(tO + c0, ov);
            tmem_ld_wait();
            reg_fence32(ov);
#pragma unroll
            for (int c = 0; c < 32; ++c) out[c] = __float_as_uint(__uint_as_float(ov[col(c)]) * inv_l);
            if (valid && !none) {
#pragma unroll
              for (int i = 0; i < 4; ++i) st_global_v8(orow + c0 + 8 * i, out + 8 * i);
            }
          }
        }
        if (valid) p.part_lse[row] = lse2;
      }
      tc_fence_before();
    }
  } else {   // one Q tile: the second PV issuer's warp
    setmaxnreg_dec<C::REGS_ROLES>();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::WARP_PV) tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace gb300

// RMS norm of every head of q and k, then the rotation by position, in one pass; and its gradient.
//
// One row is one token of one head, x of d values:
//   n = x r, r = (mean x^2 + eps)^(-1/2);   u = n w;   y = R u,
// where R turns the pairs (a, b) of the first rope_dim values by the position's angles:
//   y_a = u_a cos - u_b sin,   y_b = u_b cos + u_a sin.
// Pairs are (i, i + rope_dim / 2), or (2i, 2i + 1) when interleaved. The gradient turns back
// (R is orthogonal), du = R^T dy, and with g = du w:
//   dw = sum over rows of du n,   dx = r (g - n mean(g n)).
//
// d / 8 lanes hold a row, 8 values each as two chunks of 4 that hold both members of their pairs, so
// the rotation needs no exchange and only the row sums cross lanes. A task is one token and up to
// 4 heads of q or of k: the angles and weights are loaded once per task, and the 4 rows' loads are in
// flight together, those of the next task behind them. Everything is fp32 between the bf16 loads and the
// one rounding at the store.
//
// With several axes (time, height and width of images and video) a token has a position on each, and pair i turns by the angle
// of column i at its axis' position: cos[pos[axis(i)], i]. The axes of the pairs are 2 bits each in the launch's parameters. A
// lane's 4 columns come as one 16-byte load where their positions agree (one axis' block of columns, or text, whose axes
// agree), and as 4-byte loads otherwise (axes that take turns). Where every lane's columns have one axis (blocks of whole fours), a
// kernel of its own needs only that axis' position.
//
// Memory bounds both. At B 2, N 8192, 32 + 8 heads, d 128 on a GB300 (share of the copy bandwidth): forward 55.8 us
// (90%; 102 with rows unpacked at the load and a CTA per 16 tasks, 70 with rows held packed, 56.7 one value an
// instruction), backward 89.7 us (83%; 155 at first; 114 with 2 heads a task, 92.2 one value an instruction). Angles
// loaded before the next task's rows cost 2 to 5 us, a ring of asynchronous copies in shared memory 24: 8-byte copies, what
// a half-split pair leaves a lane, take more of the load unit than 8-byte loads.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "fastdiv.cuh"
#include "ops.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;   // rows of a task
constexpr int kFwdCtasPerSm = 3, kBwdCtasPerSm = 2;

struct NormRopeParams {
  const __nv_bfloat16 *q, *k;      // inputs (or x of the backward)
  const __nv_bfloat16 *dyq, *dyk;  // backward: gradients of the outputs, contiguous
  __nv_bfloat16 *oq, *ok;          // outputs (or dx), contiguous
  long long q_st, q_sh, k_st, k_sh;
  const float *wq, *wk, *cos, *sin;
  const int* positions;
  float* part;                     // backward: [CTAs, d] sums of du n
  float eps;
  int T, H, Hkv, half, max_pos, seq_len, parts_q, parts_k, ctas_q, w_vec;
  FastDiv parts, div_q, div_k;     // tasks of a token: all, of q, of k
  FastDiv div_seq;
  uint32_t* status;
  // Several axes: positions [axes, T], axis_st apart, and the axis of every pair in 2 bits.
  long long axis_st;
  uint32_t axes, axis_of[8];       // axes: an Axis
};

// A lane's 8 values of a row: pairs of neighbours, 0 and 1 of its first chunk, 2 and 3 of its second. The arithmetic works
// on a register pair at a time (FFMA2 and its kin).
struct Chunks {
  uint64_t v[4];
};

// A lane's values of a row as they lie in memory: held like this while other rows' loads are under way.
struct Raw {
  uint2 a, b;
};

__device__ __forceinline__ Raw load_raw(const __nv_bfloat16* row, int da, int db) {
  return {*reinterpret_cast<const uint2*>(row + da), *reinterpret_cast<const uint2*>(row + db)};
}

__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ Chunks unpack(const Raw& r) {
  return {{unpack2(r.a.x), unpack2(r.a.y), unpack2(r.b.x), unpack2(r.b.y)}};
}

__device__ __forceinline__ uint32_t pack2(uint64_t x) {
  float lo, hi;
  f2_unpack(x, lo, hi);
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, uint64_t x, uint64_t y) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x), pack2(y));
}

__device__ __forceinline__ uint64_t twice(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float sum2(uint64_t x) {
  float lo, hi;
  f2_unpack(x, lo, hi);
  return lo + hi;
}

// Whether a lane holds rotated pairs. The others' values stay as they are, rather than turned by 0: 0 times an infinite one
// would make its neighbour NaN.
__device__ __forceinline__ bool turns(int l, int half) { return 4 * l < half; }

// First dims of a lane's two chunks. half = rope_dim / 2; lanes behind the rotated dims hold 8
// neighbouring values, as all lanes do when pairs are interleaved.
template <bool INTERLEAVED>
__device__ __forceinline__ void chunk_dims(int l, int half, int& da, int& db) {
  const bool split = !INTERLEAVED && turns(l, half);
  da = split ? 4 * l : 8 * l;
  db = split ? half + 4 * l : 8 * l + 4;
}

// Angles of a lane's pairs at one position, as turn() multiplies with them: cosines, sines for the second member of a pair
// and, with the sign turned, for the first. When interleaved a register pair is a rotated pair: (cos, cos), (-sin, sin).
template <bool INTERLEAVED>
struct Angles {
  uint64_t c[INTERLEAVED ? 4 : 2], s[INTERLEAVED ? 4 : 2], n[INTERLEAVED ? 1 : 2];
};

template <bool INTERLEAVED>
__device__ __forceinline__ void turn(Chunks& x, const Angles<INTERLEAVED>& r) {
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u, w;
      f2_unpack(x.v[i], u, w);
      x.v[i] = f2_fma(x.v[i], r.c[i], f2_mul(f2_pack(w, u), r.s[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t a = x.v[i], b = x.v[2 + i];
      x.v[i] = f2_fma(a, r.c[i], f2_mul(b, r.n[i]));
      x.v[2 + i] = f2_fma(b, r.c[i], f2_mul(a, r.s[i]));
    }
  }
}

// Of a lane whose values are rotated. PART: some lanes' are not, in a row that is rotated in part or not at all. They choose
// rather than branch, which would keep the rows of a task apart (half of each row rotated, B 2, N 8192: forward 57.7 us, with a
// branch 60.1, with values turned by 0 56.5; whole rows, that do not ask, 55.9, with a branch 59.2).
template <bool INTERLEAVED, bool PART>
__device__ __forceinline__ void turn_lane(Chunks& x, const Angles<INTERLEAVED>& r, bool rotated) {
  Chunks y = x;
  turn<INTERLEAVED>(y, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = !PART || rotated ? y.v[i] : x.v[i];
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// How a token's positions are given: one; one for each axis, of which a lane's 4 pairs need one; or up to four.
enum Axis { kOneAxis, kAxisOfLane, kAxesOfLane };

template <Axis AXES>
struct Positions {
  int v[AXES == kAxesOfLane ? 4 : 1];   // of this lane's pairs; v[0] = -1: nothing to store
};

// Positions of token t for a lane of its row of LPR; v[0] = -1 in every lane of the row where one that some pair turns by lies
// outside the tables. mine: the axes of the lane's pairs. With several axes the lanes of a row agree by a vote.
template <Axis AXES, int LPR>
__device__ __forceinline__ Positions<AXES> position(const NormRopeParams& p, int t, uint32_t mine, int l) {
  Positions<AXES> r;
  if constexpr (AXES == kOneAxis) {
    r.v[0] = 0;
    if (!p.cos) return r;
    const int pos = p.positions ? p.positions[t] : t - (int)((uint32_t)t / p.div_seq) * p.seq_len;
    if (pos >= 0 && pos < p.max_pos) {
      r.v[0] = pos;
      return r;
    }
    if (l == 0) atomicCAS(p.status, 0u, kStatusBadPosition);
    r.v[0] = -1;
  } else {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < (AXES == kAxesOfLane ? 4 : 1); ++i) {
      r.v[i] = turns(l, p.half) ? p.positions[(mine >> (2 * i) & 3u) * p.axis_st + t] : 0;
      bad = bad || r.v[i] < 0 || r.v[i] >= p.max_pos;
    }
    const uint32_t row = (LPR == 32 ? 0xffffffffu : (1u << (LPR & 31)) - 1u) << (threadIdx.x & 31) / LPR * LPR;
    if (__ballot_sync(0xffffffffu, bad) & row) {
      if (l == 0) atomicCAS(p.status, 0u, kStatusBadPosition);
      r.v[0] = -1;
    }
  }
  return r;
}

// Angles at these positions; back: for the turn back.
template <bool INTERLEAVED, Axis AXES>
__device__ __forceinline__ Angles<INTERLEAVED> load_angles(const NormRopeParams& p, const Positions<AXES>& pos, int l, bool back) {
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turns(l, p.half) && pos.v[0] >= 0) {
    bool same = true;
    if constexpr (AXES == kAxesOfLane) same = pos.v[1] == pos.v[0] && pos.v[2] == pos.v[0] && pos.v[3] == pos.v[0];
    if (same) {
      const long long at = (long long)pos.v[0] * p.half + 4 * l;
      c = *reinterpret_cast<const float4*>(p.cos + at), s = *reinterpret_cast<const float4*>(p.sin + at);
    } else if constexpr (AXES == kAxesOfLane) {
      float cs[4], sn[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long at = (long long)pos.v[i] * p.half + 4 * l + i;
        cs[i] = p.cos[at], sn[i] = p.sin[at];
      }
      c = make_float4(cs[0], cs[1], cs[2], cs[3]), s = make_float4(sn[0], sn[1], sn[2], sn[3]);
    }
  }
  if (back) s = make_float4(-s.x, -s.y, -s.z, -s.w);
  Angles<INTERLEAVED> r;
  if constexpr (INTERLEAVED) {
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) r.c[i] = twice(cs[i]), r.s[i] = f2_pack(-sn[i], sn[i]);
  } else {
    r.c[0] = f2_pack(c.x, c.y), r.c[1] = f2_pack(c.z, c.w);
    r.s[0] = f2_pack(s.x, s.y), r.s[1] = f2_pack(s.z, s.w);
    r.n[0] = f2_pack(-s.x, -s.y), r.n[1] = f2_pack(-s.z, -s.w);
  }
  return r;
}

__device__ __forceinline__ void load_weights4(uint64_t* x, const float* w, bool vec) {
  const float4 y = vec ? *reinterpret_cast<const float4*>(w) : make_float4(w[0], w[1], w[2], w[3]);
  x[0] = f2_pack(y.x, y.y), x[1] = f2_pack(y.z, y.w);
}

// vec: the weights are 16-byte aligned.
__device__ __forceinline__ Chunks load_weights(const float* w, int da, int db, bool vec) {
  Chunks x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = twice(1.f);
  if (w) {
    load_weights4(x.v, w + da, vec);
    load_weights4(x.v + 2, w + db, vec);
  }
  return x;
}

// CTAs walk the tasks of all tokens, one wave of them; a thread has the rows of its next task on their
// way while it turns those of this one, so that loads are always in flight.
template <int D, bool NORM, bool INTERLEAVED, bool PART, Axis AXES>
__global__ void __launch_bounds__(kThreads, kFwdCtasPerSm) qk_norm_rope_kernel(const NormRopeParams p) {
  griddep_wait();
  griddep_launch_dependents();   // of the next kernel only the launch may overlap: it waits for this one's end
  constexpr int LPR = D / 8, ROWS = kThreads / LPR;
  const int l = threadIdx.x % LPR;
  const uint32_t axes = AXES != kOneAxis ? p.axis_of[l / 4] >> (8 * (l % 4)) : 0u;
  int da, db;
  chunk_dims<INTERLEAVED>(l, p.half, da, db);
  struct Task {
    int t, h0;
    Positions<AXES> pos;
    bool is_k;
    Raw raw[kHeads];
  };
  const uint32_t tasks = (uint32_t)p.T * p.parts.v, stride = gridDim.x * ROWS;
  auto load = [&](uint32_t id) {
    Task w;
    const uint32_t token = id / p.parts;
    const int part = id - token * p.parts.v;
    w.t = token;
    w.pos = position<AXES, LPR>(p, w.t, axes, l);
    w.is_k = part >= p.parts_q;
    w.h0 = (w.is_k ? part - p.parts_q : part) * kHeads;
    const __nv_bfloat16* x = w.is_k ? p.k + w.t * p.k_st : p.q + w.t * p.q_st;
    const long long sh = w.is_k ? p.k_sh : p.q_sh;
    const int last = (w.is_k ? p.Hkv : p.H) - 1;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) w.raw[i] = load_raw(x + min(w.h0 + i, last) * sh, da, db);   // the last row again
    return w;
  };
  // Every thread of the CTA makes the same number of turns: row sums take whole warps.
  const uint32_t slot = threadIdx.x / LPR;
  uint32_t id = blockIdx.x * ROWS + slot;
  Task now = load(min(id, tasks - 1));
  for (uint32_t first = blockIdx.x * ROWS; first < tasks; first += stride, id += stride) {
    Task next = now;
    if (first + stride < tasks) next = load(min(id + stride, tasks - 1));
    const Angles<INTERLEAVED> r = load_angles<INTERLEAVED, AXES>(p, now.pos, l, false);
    Chunks w;
    if (NORM) w = load_weights(now.is_k ? p.wk : p.wq, da, db, p.w_vec);
    const int heads = now.is_k ? p.Hkv : p.H, last = id < tasks && now.pos.v[0] >= 0 ? heads : 0;
    __nv_bfloat16* y = (now.is_k ? p.ok : p.oq) + ((long long)now.t * heads + now.h0) * D;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      Chunks v = unpack(now.raw[i]);
      if (NORM) {
        uint64_t s = f2_mul(v.v[0], v.v[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) s = f2_fma(v.v[j], v.v[j], s);
        const uint64_t rs = twice(rsqrtf(row_sum<LPR>(sum2(s)) * (1.f / D) + p.eps));
#pragma unroll
        for (int j = 0; j < 4; ++j) v.v[j] = f2_mul(f2_mul(v.v[j], rs), w.v[j]);
      }
      turn_lane<INTERLEAVED, PART>(v, r, turns(l, p.half));
      if (now.h0 + i < last) {
        store4(y + i * D + da, v.v[0], v.v[1]);
        store4(y + i * D + db, v.v[2], v.v[3]);
      }
    }
    now = next;
  }
}

// The gradient. CTAs 0 .. ctas_q - 1 walk the tasks of q, the others those of k, so a thread sums the
// weight gradient of its 8 dims in registers; a CTA adds its rows' sums in a fixed order and leaves
// [d] in part, which dw_kernel adds up: the same bits every time.
template <int D, bool NORM, bool INTERLEAVED, bool PART, Axis AXES>
__global__ void __launch_bounds__(kThreads, kBwdCtasPerSm) qk_norm_rope_bwd_kernel(const NormRopeParams p) {
  griddep_wait();
  griddep_launch_dependents();   // of the next kernel only the launch may overlap: it waits for this one's end
  constexpr int LPR = D / 8, ROWS = kThreads / LPR;
  const int l = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const bool is_k = blockIdx.x >= (unsigned)p.ctas_q;
  const int cta = is_k ? (int)blockIdx.x - p.ctas_q : blockIdx.x, ctas = is_k ? (int)gridDim.x - p.ctas_q : p.ctas_q;
  const int heads = is_k ? p.Hkv : p.H;
  const FastDiv parts = is_k ? p.div_k : p.div_q;
  const float* wp = is_k ? p.wk : p.wq;
  const long long sh = is_k ? p.k_sh : p.q_sh;
  const uint32_t axes = AXES != kOneAxis ? p.axis_of[l / 4] >> (8 * (l % 4)) : 0u;
  int da, db;
  chunk_dims<INTERLEAVED>(l, p.half, da, db);
  Chunks w, dw;
  if (NORM) w = load_weights(wp, da, db, p.w_vec);
#pragma unroll
  for (int j = 0; j < 4; ++j) dw.v[j] = twice(0.f);
  struct Task {
    int t, h0;
    Positions<AXES> pos;
    Raw x[kHeads], g[kHeads];
  };
  auto load = [&](uint32_t id) {
    Task w;
    w.t = id / parts;
    w.h0 = (id - w.t * parts.v) * kHeads;
    w.pos = position<AXES, LPR>(p, w.t, axes, l);
    const __nv_bfloat16* x = is_k ? p.k + w.t * p.k_st : p.q + w.t * p.q_st;
    const __nv_bfloat16* dy = (is_k ? p.dyk : p.dyq) + (long long)w.t * heads * D;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = min(w.h0 + i, heads - 1);   // the last row again
      if (NORM) w.x[i] = load_raw(x + h * sh, da, db);
      w.g[i] = load_raw(dy + h * D, da, db);
    }
    return w;
  };
  const uint32_t tasks = (uint32_t)p.T * parts.v, stride = (uint32_t)ctas * ROWS;
  uint32_t id = (uint32_t)cta * ROWS + slot;
  Task now = load(min(id, tasks - 1));
  // Every thread of the CTA makes the same number of turns: row sums take whole warps.
  for (uint32_t first = (uint32_t)cta * ROWS; first < tasks; first += stride, id += stride) {
    Task next = now;
    if (first + stride < tasks) next = load(min(id + stride, tasks - 1));
    const Angles<INTERLEAVED> r = load_angles<INTERLEAVED, AXES>(p, now.pos, l, true);
    const int last = id < tasks && now.pos.v[0] >= 0 ? heads : 0;
    __nv_bfloat16* dx = (is_k ? p.ok : p.oq) + ((long long)now.t * heads + now.h0) * D;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      Chunks g = unpack(now.g[i]);
      turn_lane<INTERLEAVED, PART>(g, r, turns(l, p.half));
      if (NORM) {
        const Chunks v = unpack(now.x[i]);
        Chunks gw;
        uint64_t s2 = 0, m2 = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          gw.v[j] = f2_mul(g.v[j], w.v[j]);
          s2 = j ? f2_fma(v.v[j], v.v[j], s2) : f2_mul(v.v[j], v.v[j]);
          m2 = j ? f2_fma(gw.v[j], v.v[j], m2) : f2_mul(gw.v[j], v.v[j]);
        }
        const float s = row_sum<LPR>(sum2(s2)), m = row_sum<LPR>(sum2(m2));
        const float rs = rsqrtf(s * (1.f / D) + p.eps), c = m * (1.f / D) * rs * rs;
        const uint64_t rs2 = twice(rs), c2 = twice(-c);
        if (now.h0 + i < last) {   // not the repeated rows, nor a row without a position, which may hold anything
#pragma unroll
          for (int j = 0; j < 4; ++j) dw.v[j] = f2_fma(g.v[j], f2_mul(v.v[j], rs2), dw.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) g.v[j] = f2_mul(f2_fma(v.v[j], c2, gw.v[j]), rs2);
      }
      if (now.h0 + i < last) {
        store4(dx + i * D + da, g.v[0], g.v[1]);
        store4(dx + i * D + db, g.v[2], g.v[3]);
      }
    }
    now = next;
  }
  if (NORM && wp) {
    __shared__ float sums[ROWS][D];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = (j < 2 ? da : db) + j % 2 * 2;
      f2_unpack(dw.v[j], sums[slot][at], sums[slot][at + 1]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) s += sums[r][i];
      p.part[(long long)blockIdx.x * D + i] = s;
    }
  }
}

// dw[i] = sum over CTAs of part[cta][i]; block x is 32 dims of q's (y = 0) or k's (y = 1) weight.
__global__ void __launch_bounds__(1024) dw_kernel(const float* __restrict__ part, float* dwq, float* dwk, int d,
                                                  int ctas_q, int ctas) {
  griddep_wait();
  float* dw = blockIdx.y ? dwk : dwq;
  if (!dw) return;
  const int first = blockIdx.y ? ctas_q : 0, last = blockIdx.y ? ctas : ctas_q;
  const int i = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
#pragma unroll 8
  for (int c = first + threadIdx.y; c < last; c += 32) s += part[(long long)c * d + i];
  __shared__ float sums[32][33];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0) {
    s = 0.f;
    for (int r = 0; r < 32; ++r) s += sums[r][threadIdx.x];
    dw[i] = s;
  }
}

// f with the constants of the kernel that p and the flags ask for.
template <int D, class F>
cudaError_t with_kind(const NormRopeParams& p, bool norm, bool interleaved, F&& f) {
  const bool part = 2 * p.half != D;
  auto go = [&](auto n, auto i) {
    auto axes = [&](auto a) { return part ? f(n, i, std::true_type{}, a) : f(n, i, std::false_type{}, a); };
    if (p.axes == kAxisOfLane) return axes(std::integral_constant<Axis, kAxisOfLane>{});
    if (p.axes == kAxesOfLane) return axes(std::integral_constant<Axis, kAxesOfLane>{});
    return axes(std::integral_constant<Axis, kOneAxis>{});
  };
  if (norm) return interleaved ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  return interleaved ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
}

template <int D>
cudaError_t launch_forward(const NormRopeParams& p, bool norm, bool interleaved, int sms, cudaStream_t s) {
  const long long tasks = (long long)p.T * (p.parts_q + p.parts_k), rows = kThreads / (D / 8);
  const unsigned grid = (unsigned)std::min<long long>((tasks + rows - 1) / rows, (long long)kFwdCtasPerSm * sms);
  return with_kind<D>(p, norm, interleaved, [&](auto n, auto i, auto part, auto axes) {
    return launch_dependent(qk_norm_rope_kernel<D, n(), i(), part(), axes()>, dim3(grid), dim3(kThreads), 0, s, p);
  });
}

template <int D>
cudaError_t launch_backward(const NormRopeParams& p, bool norm, bool interleaved, int grid, cudaStream_t s) {
  return with_kind<D>(p, norm, interleaved, [&](auto n, auto i, auto part, auto axes) {
    return launch_dependent(qk_norm_rope_bwd_kernel<D, n(), i(), part(), axes()>, dim3((unsigned)grid), dim3(kThreads), 0, s, p);
  });
}

// CTAs of the backward: one wave, shared between q and k by their tasks.
struct BwdGrid {
  int ctas_q, ctas;
};

BwdGrid bwd_grid(int T, int H, int Hkv, int d, int sms) {
  const long long rows = kThreads / (d / 8);
  const long long tq = (long long)T * ((H + kHeads - 1) / kHeads), tk = (long long)T * ((Hkv + kHeads - 1) / kHeads);
  const long long need_q = (tq + rows - 1) / rows, need_k = (tk + rows - 1) / rows, cap = (long long)kBwdCtasPerSm * sms;
  if (need_q + need_k <= cap) return {(int)need_q, (int)(need_q + need_k)};
  long long cq = cap * tq / (tq + tk);
  cq = std::max<long long>(1, std::min(cq, cap - (tk ? 1 : 0)));
  return {(int)cq, (int)(tk ? cap : cq)};
}

struct Range {
  uintptr_t b, e;
};

Range rows_range(const void* p, long long T, long long heads, long long st, long long sh, int d) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + 2 * ((uintptr_t)(T - 1) * st + (uintptr_t)(heads - 1) * sh + d)};
}

bool meet(const Range& a, const Range& b) { return a.b < b.e && b.b < a.e; }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// Checks that the forward and the backward share; x are the strided inputs (null: not read).
attn_status_t check(const void* xq, const void* xk, const void* oq, const void* ok, int T, int H, int Hkv, int d,
                    long long q_st, long long q_sh, long long k_st, long long k_sh, int norm, const float* wq,
                    const float* wk, float eps, const float* cos, const float* sin, int rope_dim, int max_pos,
                    const int* positions, int seq_len) {
  if (T < 1 || H < 1 || Hkv < 0 || d < 1) return ATTN_ERR_INVALID_ARG;
  if (!oq || (Hkv > 0) != (ok != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(xk) || !aligned16(oq) || !aligned16(ok)) return ATTN_ERR_INVALID_ARG;
  if (q_st < 0 || q_sh < 0 || k_st < 0 || k_sh < 0 || q_st % 8 || q_sh % 8 || k_st % 8 || k_sh % 8)
    return ATTN_ERR_INVALID_ARG;
  if (q_st > (1LL << 40) || q_sh > (1LL << 40) || k_st > (1LL << 40) || k_sh > (1LL << 40)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
  if (norm && !(eps >= 0.f && std::isfinite(eps))) return ATTN_ERR_INVALID_ARG;
  if (!norm && (wq || wk)) return ATTN_ERR_INVALID_ARG;
  if (!aligned4(wq) || !aligned4(wk)) return ATTN_ERR_INVALID_ARG;
  if ((cos != nullptr) != (sin != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (cos) {
    if (!aligned16(cos) || !aligned16(sin) || max_pos < 1 || !aligned4(positions)) return ATTN_ERR_INVALID_ARG;
    if (!positions && seq_len < 1) return ATTN_ERR_INVALID_ARG;
    if (rope_dim < 16 || rope_dim % 16 || rope_dim > d) return ATTN_ERR_INVALID_ARG;
  }
  const long long parts = (H + (long long)kHeads - 1) / kHeads + (Hkv + (long long)kHeads - 1) / kHeads;
  if (T * parts > INT_MAX) return ATTN_ERR_UNSUPPORTED;   // tasks are counted in 32 bits
  return ATTN_OK;
}

// Positions on several axes: what an _axes entry is given besides.
struct Axes {
  long long stride;
  int n;
  const unsigned char* of;   // host, of every pair
};

// Checks them (the tables and rope_dim have passed check) and puts them into p.
attn_status_t put_axes(const Axes& a, int T, const float* cos, int rope_dim, const int* positions, NormRopeParams& p) {
  if (!cos || !positions || !a.of || a.n < 1 || a.n > 4) return ATTN_ERR_INVALID_ARG;
  if (a.n > 1 && (a.stride < T || a.stride > (1LL << 40))) return ATTN_ERR_INVALID_ARG;
  p.axis_st = a.n > 1 ? a.stride : 0;
  for (int i = 0; i < rope_dim / 2; ++i) {
    if (a.of[i] >= a.n) return ATTN_ERR_INVALID_ARG;
    p.axis_of[i / 16] |= (uint32_t)a.of[i] << (2 * (i % 16));
    if (i % 4 == 0 && p.axes == kOneAxis) p.axes = kAxisOfLane;
    if (a.of[i] != a.of[i / 4 * 4]) p.axes = kAxesOfLane;   // within the 4 pairs of a lane
  }
  return ATTN_OK;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

static attn_status_t norm_rope(const void* q, const void* k, void* q_out, void* k_out, int T, int H, int Hkv, int d,
                               long long q_stride_t, long long q_stride_h, long long k_stride_t, long long k_stride_h,
                               int norm, const float* wq, const float* wk, float eps, const float* cos, const float* sin,
                               int rope_dim, int max_pos, int interleaved, const int* positions, int seq_len,
                               const Axes* axes, cudaStream_t stream) {
  const attn_status_t st = check(q, k, q_out, k_out, T, H, Hkv, d, q_stride_t, q_stride_h, k_stride_t, k_stride_h,
                                 norm, wq, wk, eps, cos, sin, rope_dim, max_pos, positions, seq_len);
  if (st != ATTN_OK) return st;
  if (!q || (Hkv > 0) != (k != nullptr)) return ATTN_ERR_INVALID_ARG;
  NormRopeParams p = {};
  if (axes) {
    const attn_status_t sa = put_axes(*axes, T, cos, rope_dim, positions, p);
    if (sa != ATTN_OK) return sa;
  }
  // An output may be its own contiguous input (a row is read before it is written); otherwise
  // outputs meet neither the inputs nor each other.
  const Range rq = rows_range(q, T, H, q_stride_t, q_stride_h, d), oq = rows_range(q_out, T, H, (long long)H * d, d, d);
  const bool same_q = q == q_out && q_stride_h == d && q_stride_t == (long long)H * d;
  if (!same_q && meet(oq, rq)) return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0) {
    const Range rk = rows_range(k, T, Hkv, k_stride_t, k_stride_h, d),
                ok = rows_range(k_out, T, Hkv, (long long)Hkv * d, d, d);
    const bool same_k = k == k_out && k_stride_h == d && k_stride_t == (long long)Hkv * d;
    if ((!same_k && meet(ok, rk)) || meet(oq, rk) || meet(ok, rq) || meet(oq, ok)) return ATTN_ERR_INVALID_ARG;
  }
  int sms;
  uint32_t* status;
  if (!device_state(&sms, &status)) return ATTN_ERR_CUDA;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.oq = static_cast<__nv_bfloat16*>(q_out);
  p.ok = static_cast<__nv_bfloat16*>(k_out);
  p.q_st = q_stride_t, p.q_sh = q_stride_h, p.k_st = k_stride_t, p.k_sh = k_stride_h;
  p.wq = wq, p.wk = wk, p.cos = cos, p.sin = sin, p.positions = positions;
  p.eps = eps;
  p.T = T, p.H = H, p.Hkv = Hkv, p.half = cos ? rope_dim / 2 : 0, p.max_pos = max_pos, p.seq_len = seq_len;
  p.parts_q = (H + kHeads - 1) / kHeads, p.parts_k = (Hkv + kHeads - 1) / kHeads;
  p.parts = fast_div(p.parts_q + p.parts_k), p.div_q = fast_div(p.parts_q), p.div_k = fast_div(std::max(p.parts_k, 1));
  p.div_seq = fast_div(std::max(seq_len, 1));
  p.w_vec = aligned16(wq) && aligned16(wk);
  p.status = status;
  cudaError_t e;
  switch (d) {
    case 64: e = launch_forward<64>(p, norm != 0, interleaved != 0, sms, stream); break;
    case 128: e = launch_forward<128>(p, norm != 0, interleaved != 0, sms, stream); break;
    default: e = launch_forward<256>(p, norm != 0, interleaved != 0, sms, stream); break;
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t attn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int T, int H,
                                           int Hkv, int d, long long q_stride_t, long long q_stride_h,
                                           long long k_stride_t, long long k_stride_h, int norm, const float* wq,
                                           const float* wk, float eps, const float* cos, const float* sin,
                                           int rope_dim, int max_pos, int interleaved, const int* positions,
                                           int seq_len, cudaStream_t stream) {
  return norm_rope(q, k, q_out, k_out, T, H, Hkv, d, q_stride_t, q_stride_h, k_stride_t, k_stride_h, norm, wq, wk, eps, cos,
                   sin, rope_dim, max_pos, interleaved, positions, seq_len, nullptr, stream);
}

extern "C" attn_status_t attn_qk_norm_rope_axes(const void* q, const void* k, void* q_out, void* k_out, int T, int H,
                                                int Hkv, int d, long long q_stride_t, long long q_stride_h,
                                                long long k_stride_t, long long k_stride_h, int norm, const float* wq,
                                                const float* wk, float eps, const float* cos, const float* sin,
                                                int rope_dim, int max_pos, int interleaved, const int* positions,
                                                long long axis_stride, int axes, const unsigned char* pair_axis,
                                                cudaStream_t stream) {
  const Axes a{axis_stride, axes, pair_axis};
  return norm_rope(q, k, q_out, k_out, T, H, Hkv, d, q_stride_t, q_stride_h, k_stride_t, k_stride_h, norm, wq, wk, eps, cos,
                   sin, rope_dim, max_pos, interleaved, positions, 1, &a, stream);
}

extern "C" size_t attn_qk_norm_rope_bwd_workspace_bytes(int T, int H, int Hkv, int d) {
  if (T < 1 || H < 1 || Hkv < 0 || (d != 64 && d != 128 && d != 256)) return 0;
  int sms = 152;
  uint32_t* status;
  device_state(&sms, &status);
  return (size_t)bwd_grid(T, H, Hkv, d, sms).ctas * d * 4;
}

static attn_status_t norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                                   float* dwq, float* dwk, int T, int H, int Hkv, int d, long long q_stride_t,
                                   long long q_stride_h, long long k_stride_t, long long k_stride_h, int norm,
                                   const float* wq, const float* wk, float eps, const float* cos, const float* sin,
                                   int rope_dim, int max_pos, int interleaved, const int* positions, int seq_len,
                                   const Axes* axes, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const attn_status_t st = check(norm ? q : nullptr, norm ? k : nullptr, dq, dk, T, H, Hkv, d, q_stride_t, q_stride_h,
                                 k_stride_t, k_stride_h, norm, wq, wk, eps, cos, sin, rope_dim, max_pos, positions,
                                 seq_len);
  if (st != ATTN_OK) return st;
  if (!dq_out || (Hkv > 0) != (dk_out != nullptr) || (norm && (!q || (Hkv > 0) != (k != nullptr))))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(dq_out) || !aligned16(dk_out)) return ATTN_ERR_INVALID_ARG;
  NormRopeParams p = {};
  if (axes) {
    const attn_status_t sa = put_axes(*axes, T, cos, rope_dim, positions, p);
    if (sa != ATTN_OK) return sa;
  }
  // weight gradients come with their weights
  if ((dwq != nullptr) != (wq != nullptr) || (dwk != nullptr) != (wk != nullptr) || !aligned4(dwq) || !aligned4(dwk))
    return ATTN_ERR_INVALID_ARG;
  const size_t need = attn_qk_norm_rope_bwd_workspace_bytes(T, H, Hkv, d);
  const bool dw = dwq || dwk;
  if (dw && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return ATTN_ERR_INVALID_ARG;
  // Outputs: dq and dk may be the gradients they are made from, and nothing else.
  Range outs[5], ins[4];
  int no = 0, ni = 0;
  auto bytes = [](const void* p, size_t n) {
    return Range{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + n};
  };
  const Range oq = rows_range(dq, T, H, (long long)H * d, d, d);
  outs[no++] = oq;
  if (Hkv > 0) outs[no++] = rows_range(dk, T, Hkv, (long long)Hkv * d, d, d);
  if (dwq) outs[no++] = bytes(dwq, (size_t)d * 4);
  if (dwk) outs[no++] = bytes(dwk, (size_t)d * 4);
  if (dw) outs[no++] = bytes(workspace, need);
  if (norm) {
    ins[ni++] = rows_range(q, T, H, q_stride_t, q_stride_h, d);
    if (Hkv > 0) ins[ni++] = rows_range(k, T, Hkv, k_stride_t, k_stride_h, d);
  }
  ins[ni++] = rows_range(dq_out, T, H, (long long)H * d, d, d);
  if (Hkv > 0) ins[ni++] = rows_range(dk_out, T, Hkv, (long long)Hkv * d, d, d);
  for (int i = 0; i < no; ++i) {
    for (int j = i + 1; j < no; ++j)
      if (meet(outs[i], outs[j])) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < ni; ++j) {
      const bool in_place = (i == 0 && dq == dq_out && j == (norm ? (Hkv > 0 ? 2 : 1) : 0)) ||
                            (i == 1 && Hkv > 0 && dk == dk_out && j == ni - 1);
      if (!in_place && meet(outs[i], ins[j])) return ATTN_ERR_INVALID_ARG;
    }
  }
  int sms;
  uint32_t* status;
  if (!device_state(&sms, &status)) return ATTN_ERR_CUDA;
  const BwdGrid g = bwd_grid(T, H, Hkv, d, sms);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.dyq = static_cast<const __nv_bfloat16*>(dq_out);
  p.dyk = static_cast<const __nv_bfloat16*>(dk_out);
  p.oq = static_cast<__nv_bfloat16*>(dq);
  p.ok = static_cast<__nv_bfloat16*>(dk);
  p.q_st = q_stride_t, p.q_sh = q_stride_h, p.k_st = k_stride_t, p.k_sh = k_stride_h;
  p.wq = wq, p.wk = wk, p.cos = cos, p.sin = sin, p.positions = positions;
  p.part = static_cast<float*>(workspace);
  p.eps = eps;
  p.T = T, p.H = H, p.Hkv = Hkv, p.half = cos ? rope_dim / 2 : 0, p.max_pos = max_pos, p.seq_len = seq_len;
  p.parts_q = (H + kHeads - 1) / kHeads, p.parts_k = (Hkv + kHeads - 1) / kHeads, p.ctas_q = g.ctas_q;
  p.parts = fast_div(p.parts_q + p.parts_k), p.div_q = fast_div(p.parts_q), p.div_k = fast_div(std::max(p.parts_k, 1));
  p.div_seq = fast_div(std::max(seq_len, 1));
  p.w_vec = aligned16(wq) && aligned16(wk);
  p.status = status;
  cudaError_t e;
  switch (d) {
    case 64: e = launch_backward<64>(p, norm != 0, interleaved != 0, g.ctas, stream); break;
    case 128: e = launch_backward<128>(p, norm != 0, interleaved != 0, g.ctas, stream); break;
    default: e = launch_backward<256>(p, norm != 0, interleaved != 0, g.ctas, stream); break;
  }
  if (e == cudaSuccess && dw) {
    e = launch_dependent(dw_kernel, dim3((unsigned)d / 32, 2), dim3(32, 32), 0, stream, (const float*)p.part, dwq, dwk, d,
                         g.ctas_q, g.ctas);
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t attn_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                                               void* dq, void* dk, float* dwq, float* dwk, int T, int H, int Hkv,
                                               int d, long long q_stride_t, long long q_stride_h,
                                               long long k_stride_t, long long k_stride_h, int norm, const float* wq,
                                               const float* wk, float eps, const float* cos, const float* sin,
                                               int rope_dim, int max_pos, int interleaved, const int* positions,
                                               int seq_len, void* workspace, size_t workspace_bytes,
                                               cudaStream_t stream) {
  return norm_rope_bwd(q, k, dq_out, dk_out, dq, dk, dwq, dwk, T, H, Hkv, d, q_stride_t, q_stride_h, k_stride_t, k_stride_h,
                       norm, wq, wk, eps, cos, sin, rope_dim, max_pos, interleaved, positions, seq_len, nullptr, workspace,
                       workspace_bytes, stream);
}

extern "C" attn_status_t attn_qk_norm_rope_axes_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                                                    void* dq, void* dk, float* dwq, float* dwk, int T, int H, int Hkv,
                                                    int d, long long q_stride_t, long long q_stride_h,
                                                    long long k_stride_t, long long k_stride_h, int norm,
                                                    const float* wq, const float* wk, float eps, const float* cos,
                                                    const float* sin, int rope_dim, int max_pos, int interleaved,
                                                    const int* positions, long long axis_stride, int axes,
                                                    const unsigned char* pair_axis, void* workspace,
                                                    size_t workspace_bytes, cudaStream_t stream) {
  const Axes a{axis_stride, axes, pair_axis};
  return norm_rope_bwd(q, k, dq_out, dk_out, dq, dk, dwq, dwk, T, H, Hkv, d, q_stride_t, q_stride_h, k_stride_t, k_stride_h,
                       norm, wq, wk, eps, cos, sin, rope_dim, max_pos, interleaved, positions, 1, &a, workspace,
                       workspace_bytes, stream);
}

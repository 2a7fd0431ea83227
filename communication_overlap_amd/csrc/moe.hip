// A whole mixture-of-experts layer for a few tokens: routing, the experts'
// two products, the gate-weighted sum.  What it must read is the chosen
// experts' weights; everything else is small, so the experts' products are
// rows.h's streams, spread over the chip by (chosen expert, columns, range of
// k), a workgroup a compute unit taking items in turn.  Partial sums meet in a
// fixed order, at whichever workgroup arrives last or in a launch of their own.
//  1. Routing (with a router), two launches: logits of ranges of hidden x
//     groups of 4 tokens, in float64 so that a choice between two near logits
//     does not hang on the order of a sum; then each token's ranges added up
//     and its experts picked.  (One launch, the last range picking, took 0.4 us
//     more for a token and 5 more for 64.)  One token's experts every workgroup
//     of 2 picks for itself (33.4 us for the layer, 34.5 with the launch): it
//     reads at most 64 logits a range, from its die's cache.
//  2. Up: u = x w1, then h = act(gate) * up as bf16 planes (see ovl.h).
//  3. Down: h w2 per (token, choice) pair in float32, and the sum of each
//     token's choices with their gates, in order: by the last workgroup of a
//     column tile, over all experts and ranges, for at most 8 tokens in few
//     tiles, else by a launch of its own.
// Every workgroup of 2 and 3 lists the distinct experts itself, from the at
// most 1024 chosen ids, and finds its items' pairs there.
//
// Measured (4096 x 1408, 64 experts, gated): one token, top 2, bf16 33.5 us, of
// which 12 is the 70 MB stream and the rest the three launches' starts and ends;
// 64 tokens, top 2, bf16 345-368 us (HBM: 1.85 GB, up 5.6 and down 5.4 TB/s), 128
// tokens 408; 9 tokens, top 4, FP8 92-104 us by how many experts they choose (HBM:
// 437 MB, up 4.8 and down 4.0 TB/s).
#include <algorithm>

#include "epilogue.h"
#include "host.h"
#include "moe_ranges.h"
#include "rows.h"

namespace ovl {

namespace {

constexpr int kMoeTokens = 128, kMoeExperts = 256, kMoeTopk = 8;
constexpr int kMoeRouteRows = 64;    // rows of the router a workgroup sums (128: 8.8 against 3.4 us for a token)
constexpr int kMoeRouteTokens = 4;   // tokens of a routing group (1 where there is one)
// Arrival counters: down tiles, then (expert, up tile).
constexpr int32_t kMoeDownCounters = 1024;
constexpr int kMoePlanes = 3;    // of h: 24 bits, as many as a float32 has

struct MoeArgs {
  const uint16_t* x;
  const uint16_t* router;
  int32_t* topk;
  float* gates;
  const uint8_t* w1;
  const float* s1;
  const uint8_t* w2;
  const float* s2;
  void* out;
  uint16_t* h;      // [planes][pairs][inter]
  float* up;        // [up_max][pairs][n1] when up_max > 1
  float* down;      // [down_max][pairs][hidden]
  double* logits;   // [chunks][tokens][experts]
  int32_t* down_counters;
  int32_t* up_counters;
  int64_t hidden, inter, n1;
  int32_t tokens, experts, topk_n, pairs, act, out_type, norm_topk;
  int32_t up_tiles, up_max, up_steps;  // column tiles, most ranges of k, steps of k
  int32_t down_tiles, down_max, down_steps;
  int32_t chunks;
  int32_t fused;  // the down launch sums the choices itself
  int32_t pick;   // the up launch picks the one token's experts itself
};

// ---------------------------------------------------------------- routing

// exp(x) of a float64 x <= 0 to 1e-12 of itself, so that a gate is rounded
// once: x = n ln 2 + r with |r| <= ln 2 / 2, and the exponential series of r up
// to r^10 / 10!, whose next term is below 3e-13.  (The device library's float64
// exp is exact to the last bits, and its code is long to fetch.)
__device__ inline double moe_exp(double x) {
  if (x < -740.0) return 0.0;
  const double n = rint(x * 1.4426950408889634074);
  const double r = fma(-n, 0.69314718055994530942, x);
  double p = 1.0 / 3628800;
  constexpr double kTerms[] = {1.0 / 362880, 1.0 / 40320, 1.0 / 5040, 1.0 / 720, 1.0 / 120,
                               1.0 / 24,     1.0 / 6,     0.5,        1.0,       1.0};
#pragma unroll
  for (int i = 0; i < 10; ++i) p = fma(p, r, kTerms[i]);
  return ldexp(p, (int)n);
}

__device__ inline double moe_wave_max(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d, 64));
  return v;
}

// A token's choices from its logits in LDS, by one wavefront: the largest
// remaining one, topk times; among equals the lowest id, a NaN when nothing
// else remains (fmax passes NaN over).  Lane j holds choice j and its gate.
struct MoeChoice {
  int32_t id;
  float gate;
};
__device__ inline MoeChoice moe_pick(const MoeArgs& a, const double* logits) {
  const int lane = lane_id();
  double v[4];
  bool have[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    have[i] = lane + 64 * i < a.experts;
    v[i] = have[i] ? logits[lane + 64 * i] : 0.0;
  }
  double first = 0;  // the first choice's logit
  double chosen = 0, mine = 0;
  int my_id = 0;
  for (int j = 0; j < a.topk_n; ++j) {
    double m = -HUGE_VAL;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (have[i]) m = fmax(m, v[i]);
    m = moe_wave_max(m);
    int id = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t eq = __ballot(have[i] && v[i] == m);
      if (id < 0 && eq) id = 64 * i + __ffsll((unsigned long long)eq) - 1;
    }
    if (id < 0) {  // only NaN left
      m = __builtin_nan("");
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t left = __ballot(have[i]);
        if (id < 0 && left) id = 64 * i + __ffsll((unsigned long long)left) - 1;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i == id) have[i] = false;
    if (j == 0) first = m;
    const double p = moe_exp(m - first);
    chosen += p;
    if (lane == j) {
      mine = p;
      my_id = id;
    }
  }
  if (!a.norm_topk) {
    chosen = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < a.experts) chosen += moe_exp(v[i] - first);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) chosen += __shfl_xor(chosen, d, 64);
  }
  return {my_id, (float)(mine / chosen)};
}

// Workgroup (range of hidden, TT tokens): EP lanes across the experts, 256 /
// EP rows of the router at a time, x from LDS; float64 sums of the range.
template <int EP, int TT>
__global__ __launch_bounds__(kThreads) void moe_logits_kernel(MoeArgs a) {
  constexpr int R = kThreads / EP, U = 16;
  __shared__ float xs[TT][kMoeRouteRows];
  __shared__ double part[R][TT][EP];
  const int chunk = blockIdx.x % a.chunks, tg = blockIdx.x / a.chunks;
  const int t0 = tg * TT, nt = min(TT, a.tokens - t0);
  const int64_t r0 = (int64_t)chunk * kMoeRouteRows;
  const int nr = (int)min((int64_t)kMoeRouteRows, a.hidden - r0);
  const int e = threadIdx.x % EP, rr = threadIdx.x / EP;
  const uint16_t* w = a.router + r0 * a.experts + min(e, a.experts - 1);
  for (int i = threadIdx.x; i < TT * kMoeRouteRows; i += kThreads) {
    const int t = i / kMoeRouteRows, r = i % kMoeRouteRows;
    const float v = bf16_lo_f(a.x[(t0 + min(t, nt - 1)) * a.hidden + r0 + min(r, nr - 1)]);
    xs[t][r] = t < nt && r < nr ? v : 0.f;
  }
  __syncthreads();
  double acc[TT] = {};
  for (int r = rr; r < kMoeRouteRows; r += R * U) {
    uint16_t q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) q[u] = w[(int64_t)min(r + u * R, nr - 1) * a.experts];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const double d = r + u * R < nr ? bf16_lo_f(q[u]) : 0.f;
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] += d * xs[t][min(r + u * R, kMoeRouteRows - 1)];
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) part[rr][t][e] = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < nt * EP; i += kThreads) {
    const int t = i / EP, x = i % EP;
    if (x >= a.experts) continue;
    double s = part[0][t][x];
#pragma unroll
    for (int q = 1; q < R; ++q) s += part[q][t][x];
    a.logits[((int64_t)chunk * a.tokens + t0 + t) * a.experts + x] = s;
  }
}

// Token t's logits into LDS [256 / EP][EP]: the ranges' sums, 256 / EP threads
// a logit, those in order.
template <int EP>
__device__ inline void moe_logits(const MoeArgs& a, int t, double* part) {
  constexpr int R = kThreads / EP, U = 8;
  const int e = threadIdx.x % EP, rr = threadIdx.x / EP;
  const double* p = a.logits + (int64_t)t * a.experts + min(e, a.experts - 1);
  const int64_t step = (int64_t)a.tokens * a.experts;
  double s = 0;
  for (int c = rr; c < a.chunks; c += R * U) {
    double q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) q[u] = p[min(c + u * R, a.chunks - 1) * step];
#pragma unroll
    for (int u = 0; u < U; ++u) s += c + u * R < a.chunks ? q[u] : 0.0;
  }
  part[rr * EP + e] = s;
  __syncthreads();
  if (rr == 0) {
#pragma unroll
    for (int q = 1; q < R; ++q) s += part[q * EP + e];
    part[e] = s;
  }
  __syncthreads();
}

// One token a workgroup.
template <int EP>
__global__ __launch_bounds__(kThreads) void moe_pick_kernel(MoeArgs a) {
  __shared__ double part[kThreads];
  moe_logits<EP>(a, blockIdx.x, part);
  if (threadIdx.x < 64) {
    const MoeChoice c = moe_pick(a, part);
    if (lane_id() < a.topk_n) {
      a.topk[blockIdx.x * a.topk_n + lane_id()] = c.id;
      a.gates[blockIdx.x * a.topk_n + lane_id()] = c.gate;
    }
  }
}

// ---------------------------------------------------------------- experts

// What a workgroup of the experts' launches knows of the routing.
template <int N>  // rows of a unit
struct MoeLds {
  int32_t ids[kMoeTokens * kMoeTopk];
  int32_t experts[kMoeExperts];  // the distinct experts chosen, ascending
  uint64_t mask[4];
  int32_t rows[2][kRowWaves][N];  // pairs of even and odd units, one table a wavefront
  int32_t flag;
};

// Codes: the column scales of the last four units, gate's (or all) and up's.
// Wavefront 0 fetches a unit's ahead of its steps, straight into LDS: loads of
// them behind the products would wait for the next unit's weights.  It may be
// one unit ahead of the unit whose steps run, and a slower wavefront one
// behind: three are in use at a time.
struct MoeScales {
  float s[4][256];
};

// (Shared memory reached through the generator is named as such: a generic
// load counts as a global one, and a wait for it would empty the rings.)
__device__ inline int32_t lds_word(const int32_t* p) { return *OVL_LDS(const int32_t, p); }

// Reads the chosen ids and lists the distinct experts among them; returns how
// many there are.  id: this thread's choice of the only token, else null.
template <int N>
__device__ inline int moe_begin(const MoeArgs& a, MoeLds<N>& s, const int32_t* id = nullptr) {
  if (threadIdx.x < 4) s.mask[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.pairs; i += kThreads) {
    const int e = id ? *id : a.topk[i];
    const bool here = e >= 0 && e < a.experts;
    s.ids[i] = here ? e : -1;
    if (here) atomicOr(reinterpret_cast<unsigned long long*>(&s.mask[e >> 6]), 1ull << (e & 63));
  }
  __syncthreads();
  int n = 0, below = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint64_t m = s.mask[w];
    if (w < (int)threadIdx.x >> 6) below += __popcll(m);
    if (w == (int)threadIdx.x >> 6) below += __popcll(m & ((1ull << (threadIdx.x & 63)) - 1));
    n += __popcll(m);
  }
  static_assert(kThreads == kMoeExperts, "one thread an expert");
  if (s.mask[threadIdx.x >> 6] >> (threadIdx.x & 63) & 1) s.experts[below] = threadIdx.x;
  __syncthreads();
  return uniform(n);
}

// Pairs first .. first + N - 1 of expert e, in order, into this wavefront's
// table (-1 past the last); returns how many pairs e has.
template <int N>
__device__ inline int moe_rows(const MoeArgs& a, const int32_t* ids, int e, int first, int32_t* rows) {
  const int lane = lane_id();
  if (lane < N) *OVL_LDS(int32_t, rows + lane) = -1;
  int n = 0;
  for (int i = 0; i < a.pairs; i += 64) {
    const bool hit = i + lane < a.pairs && lds_word(ids + min(i + lane, kMoeTokens * kMoeTopk - 1)) == e;
    const uint64_t m = __ballot(hit);
    const int at = n + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
    if (hit && at >= first && at < first + N) *OVL_LDS(int32_t, rows + at - first) = i + lane;
    n += __popcll(m);
  }
  return uniform(n);
}

// Ranges of k that a launch cuts its items into: as many as weigh least.  Lane l
// weighs l % 16 + 1.
__device__ inline int moe_ranges(int items, int steps, int most) {
  int best = moe_range_weight(items, steps, most, (int)lane_id() % kMoeMostRanges + 1);
#pragma unroll
  for (int d = kMoeMostRanges / 2; d >= 1; d >>= 1) best = min(best, __shfl_xor(best, d, 64));
  return uniform(moe_weight_ranges(best));
}

// The units of a workgroup: its items (expert, column tile, range of k) in
// turn, each as often as the expert's rows fill a table.
template <class C, bool UP>
struct MoeGen {
  static constexpr int N = C::ROWS;
  const MoeArgs& a;
  MoeLds<N>& s;
  MoeScales* scales;  // codes only
  RowOperands o;
  int32_t tiles, ranges, steps, per, items;
  // The unit being loaded, and the unit being added up.
  int32_t l_item, l_first, l_count, l_unit;
  int32_t c_item, c_first, c_count, c_unit;

  __device__ inline MoeGen(const MoeArgs& args, MoeLds<N>& lds, MoeScales* sc, int active)
      : a(args), s(lds), scales(sc), o{} {
    tiles = UP ? a.up_tiles : a.down_tiles;
    steps = UP ? a.up_steps : a.down_steps;
    ranges = moe_ranges(active * tiles, steps, UP ? a.up_max : a.down_max);
    per = (steps + ranges - 1) / ranges;
    items = active * tiles * ranges;
    const int64_t rows = UP ? a.hidden : a.inter, cols = UP ? a.n1 : a.hidden;
    o.w_bytes = rows * cols * (C::FP8 ? 1 : 2);
    o.ldw = C::FP8 ? rows : cols;
    o.cols = UP ? a.inter : a.hidden;
    o.pair = a.inter;
    o.x = UP ? a.x : a.h;
    o.plane = UP ? 0 : a.pairs * a.inter;
    o.x_bytes = UP ? a.tokens * a.hidden * 2 : C::PL * o.plane * 2;
    o.ldx = rows;
    o.k = rows;
    l_item = c_item = blockIdx.x;
    l_first = c_first = 0;
    l_count = c_count = 0;
    l_unit = c_unit = 0;
  }
  // Item = (expert * ranges + range) * tiles + tile.
  __device__ inline int tile(int item) const { return item % tiles; }
  __device__ inline int range_of(int item) const { return item / tiles % ranges; }
  __device__ inline int slot(int item) const { return item / (tiles * ranges); }
  __device__ inline void steps_of(int item, int32_t& s0, int32_t& s1) const {
    s0 = min(range_of(item) * per, steps);
    s1 = min(s0 + per, steps);
  }
  __device__ inline const int32_t* rows(int unit) const { return s.rows[unit & 1][threadIdx.x >> 6]; }

  __device__ inline bool begin(int32_t u, RowLoads<C>& ld, int32_t& s0, int32_t& s1) {
    if (u) {
      l_first += N;
      if (l_first >= l_count) {
        l_first = 0;
        l_item += gridDim.x;
      }
    }
    if (l_item >= items) return false;
    const int e = uniform(lds_word(s.experts + slot(l_item)));
    int32_t* table = s.rows[u & 1][threadIdx.x >> 6];
    l_count = moe_rows<N>(a, s.ids, e, l_first, table);
    o.w = (UP ? a.w1 : a.w2) + e * o.w_bytes;
    o.col0 = (int64_t)tile(l_item) * C::COLS;
    ld.init(o, table, UP ? a.topk_n : 1);
    if constexpr (C::FP8) {
      static_assert((C::PAIR ? 2 : 1) * C::COLS <= 256, "a unit's scales fit one load");
      if (uniform((int)(threadIdx.x >> 6)) == 0) {
        const int64_t n = UP ? a.n1 : a.hidden;
        const u32x4 srd = make_srd((UP ? a.s1 : a.s2) + e * n, n * 4);
        const int half = lane_id() / (C::COLS / 4), c = lane_id() % (C::COLS / 4) * 4;
        const bool there = half < (C::PAIR ? 2 : 1) && o.col0 + c < o.cols;
        load_to_lds(srd, lds_addr(scales->s[u & 3]), there ? (uint32_t)(half * o.pair + o.col0 + c) * 4 : kOOB);
      }
    }
    steps_of(l_item, s0, s1);
    return true;
  }
  __device__ inline bool range(int32_t u, int32_t& s0, int32_t& s1) {
    if (u) {
      c_first += N;
      if (c_first >= c_count) {
        c_first = 0;
        c_item += gridDim.x;
      }
    }
    if (c_item >= items) return false;
    const int e = uniform(lds_word(s.experts + slot(c_item)));
    // Only the count matters here: where the table holds every pair it is the
    // table's own.
    int n = 0;
    for (int i = 0; i < a.pairs; i += 64)
      n += __popcll(__ballot(i + lane_id() < a.pairs &&
                             lds_word(s.ids + min(i + lane_id(), kMoeTokens * kMoeTopk - 1)) == e));
    c_count = uniform(n);
    c_unit = u;
    steps_of(c_item, s0, s1);
    return true;
  }
  // Codes: units start at different places of their range.
  __device__ inline int32_t turn(int32_t n) const { return C::FP8 ? tile(l_item) * 5 % n : 0; }
  __device__ inline bool last_of_item() const { return c_first + N >= c_count; }
};

// h as three bf16 planes that add up to it: the upper 16 bits of what is left,
// cut off and not rounded, so that every plane has h's sign and none is larger
// than h.  Where nothing is left, the planes before it are halved (a quarter and
// a quarter where there is one): none is zero unless h is, and an infinite
// weight times each of them is the infinity that it is times h.  (Two planes, 16
// bits, left 0.2% of the bf16 outputs a step off; the third costs the down
// launch nothing where a unit holds few rows, and where codes have many rows an
// expert, whose units then hold 8 instead of 16, 64 tokens, top 2 of 16, 97 us
// instead of 86.)
__device__ inline float moe_top(float x) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xFFFF0000u); }

__device__ inline void moe_store_h(const MoeArgs& a, int pair, int64_t col, const float (&h)[8]) {
  float p[kMoePlanes][8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float x = h[c], p0 = moe_top(x), r1 = x - p0, p1 = moe_top(r1), r2 = r1 - p1;
    const bool one = !(r1 != 0.f) || !isfinite(x), two = r2 == 0.f;
    p[0][c] = one ? 0.5f * x : p0;
    p[1][c] = one ? 0.25f * x : (two ? 0.5f * p1 : p1);
    p[2][c] = one ? 0.25f * x : (two ? 0.5f * p1 : r2);
  }
#pragma unroll
  for (int q = 0; q < kMoePlanes; ++q) store8(p[q], a.h, ((int64_t)q * a.pairs + pair) * a.inter + col, OVL_BF16);
}

// One pair's eight columns of the up product: scale, activation, h.
template <class C>
__device__ inline void moe_act(const MoeArgs& a, int pair, int64_t col, float (&g)[8], float (&u)[8]) {
  act8(g, a.act);
  if (C::PAIR)
#pragma unroll
    for (int c = 0; c < 8; ++c) g[c] *= u[c];
  moe_store_h(a, pair, col, g);
}

// v times the scales of columns col .. of half `half` of unit u.
template <class C>
__device__ inline void moe_scale(float (&v)[8], const MoeScales* sc, int32_t u, int half, int col) {
  if constexpr (C::FP8) {
    const float* p = sc->s[u & 3] + half * C::COLS + col;
    const f32x4 a = *OVL_LDS(const f32x4, p), b = *OVL_LDS(const f32x4, p + 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[c] *= a[c];
      v[4 + c] *= b[c];
    }
  }
}

template <class C>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a) {
  extern __shared__ __align__(16) uint8_t moe_lds[];
  __shared__ MoeLds<C::ROWS> s;
  __shared__ __align__(16) uint8_t sc[C::FP8 ? sizeof(MoeScales) : 16];
  MoeScales* scales = reinterpret_cast<MoeScales*>(sc);
  constexpr int PR = C::COLS / 8;  // pieces of a row
  int active;
  if (a.pick) {
    double* part = reinterpret_cast<double*>(moe_lds);
    moe_logits<64>(a, 0, part);
    MoeChoice c = {-1, 0.f};
    if (threadIdx.x < 64) c = moe_pick(a, part);
    if (blockIdx.x == 0 && (int)threadIdx.x < a.topk_n) {
      a.topk[threadIdx.x] = c.id;
      a.gates[threadIdx.x] = c.gate;
    }
    active = moe_begin(a, s, &c.id);
  } else {
    active = moe_begin(a, s);
  }
  MoeGen<C, true> gen(a, s, scales, active);
  row_stream<C>(gen, moe_lds, [&](int32_t u, const float* st) {
    const int item = gen.c_item, sp = gen.range_of(item), tile = gen.tile(item);
    const int e = uniform(lds_word(s.experts + gen.slot(item)));
    const int64_t col0 = (int64_t)tile * C::COLS;
    const int32_t* rows = gen.rows(u);
    for (int i = threadIdx.x; i < C::PIECES; i += kThreads) {
      const int pair = lds_word(rows + i / PR);
      const int64_t col = col0 + (i % PR) * 8;
      if (pair < 0 || col >= a.inter) continue;
      float g[8], v[8];
      row_sums8<C>(g, st, 0, i / PR, (i % PR) * 8);
      moe_scale<C>(g, scales, u, 0, (i % PR) * 8);
      if (C::PAIR) {
        row_sums8<C>(v, st, 1, i / PR, (i % PR) * 8);
        moe_scale<C>(v, scales, u, 1, (i % PR) * 8);
      }
      if (gen.ranges > 1) {
        float* p = a.up + ((int64_t)sp * a.pairs + pair) * a.n1 + col;
        store8_agent(g, p);
        if (C::PAIR) store8_agent(v, p + a.inter);
      } else {
        moe_act<C>(a, pair, col, g, v);
      }
    }
    if (gen.ranges == 1 || !gen.last_of_item()) return;
    if (!row_arrive_last(a.up_counters + (gen.slot(item) * gen.tiles + tile) * kCounterStride, gen.ranges, &s.flag)) return;
    // All the expert's pairs, in the order of their ids.
    for (int i = threadIdx.x; i < a.pairs * PR; i += kThreads) {
      const int pair = i / PR;
      const int64_t col = col0 + (i % PR) * 8;
      if (lds_word(s.ids + pair) != e || col >= a.inter) continue;
      float v[C::PAIR ? 2 : 1][8];
      row_ranges8(v, a.up + pair * a.n1 + col, gen.ranges, a.pairs * a.n1, a.inter);
      moe_act<C>(a, pair, col, v[0], v[C::PAIR ? 1 : 0]);
    }
    wave_drain();
  });
}

// Eight columns of a token's output: its choices in order, each the sum of its
// ranges in order; eight loads of (choice, range) go out together.
__device__ inline void moe_out8(const MoeArgs& a, const int32_t* ids, int ranges, int t, int64_t col) {
  constexpr int U = 8;
  float v[8] = {}, y[8] = {};
  int lj = 0, ls = 0, cj = 0, cs = 0;  // the (choice, range) loaded next and added next
  while (cj < a.topk_n) {
    RowPart q[U];
    float gate[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int pair = t * a.topk_n + lj;
      if (lj < a.topk_n && lds_word(ids + pair) >= 0) {
        q[u] = load8_agent(a.down + ((int64_t)ls * a.pairs + pair) * a.hidden + col);
        gate[u] = a.gates[pair];
      }
      if (++ls == ranges) ls = 0, ++lj;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int pair = t * a.topk_n + cj;
      if (cj < a.topk_n && lds_word(ids + pair) >= 0) {
        add8(y, q[u]);
        if (cs + 1 == ranges) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            v[c] += gate[u] * y[c];
            y[c] = 0.f;
          }
        }
      }
      if (++cs == ranges) cs = 0, ++cj;
    }
  }
  store8(v, a.out, t * a.hidden + col, a.out_type);
}

// out of one column tile.
template <int PR>
__device__ inline void moe_out(const MoeArgs& a, const int32_t* ids, int ranges, int64_t col0) {
  for (int i = threadIdx.x; i < a.tokens * PR; i += kThreads)
    if (col0 + (i % PR) * 8 < a.hidden) moe_out8(a, ids, ranges, i / PR, col0 + (i % PR) * 8);
}

// FUSED: the launch sums the choices itself.
template <class C, bool FUSED>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
  extern __shared__ __align__(16) uint8_t moe_lds[];
  __shared__ MoeLds<C::ROWS> s;
  __shared__ __align__(16) uint8_t sc[C::FP8 ? sizeof(MoeScales) : 16];
  MoeScales* scales = reinterpret_cast<MoeScales*>(sc);
  constexpr int PR = C::COLS / 8;
  const int active = moe_begin(a, s);
  if (FUSED && active == 0)  // no expert of this rank: zeros
    for (int t = blockIdx.x; t < a.down_tiles; t += gridDim.x) moe_out<PR>(a, s.ids, 1, (int64_t)t * C::COLS);
  MoeGen<C, false> gen(a, s, scales, active);
  row_stream<C>(gen, moe_lds, [&](int32_t u, const float* st) {
    const int item = gen.c_item, sp = gen.range_of(item), tile = gen.tile(item);
    const int64_t col0 = (int64_t)tile * C::COLS;
    const int32_t* rows = gen.rows(u);
    for (int i = threadIdx.x; i < C::PIECES; i += kThreads) {
      const int pair = lds_word(rows + i / PR);
      const int64_t col = col0 + (i % PR) * 8;
      if (pair < 0 || col >= a.hidden) continue;
      float v[8];
      row_sums8<C>(v, st, 0, i / PR, (i % PR) * 8);
      moe_scale<C>(v, scales, u, 0, (i % PR) * 8);
      float* p = a.down + ((int64_t)sp * a.pairs + pair) * a.hidden + col;
      if (FUSED)
        store8_agent(v, p);
      else
        store8(v, p, 0, OVL_F32);
    }
    if (FUSED && gen.last_of_item() && row_arrive_last(a.down_counters + tile * kCounterStride, active * gen.ranges, &s.flag)) {
      moe_out<PR>(a, s.ids, gen.ranges, col0);
      wave_drain();
    }
  });
}

// The sum on its own, where the down launch has many units a workgroup and an
// arrival after each would hold up its stream.
template <class C>
__global__ __launch_bounds__(kThreads) void moe_sum_kernel(MoeArgs a) {
  __shared__ MoeLds<C::ROWS> s;
  const int active = moe_begin(a, s);
  const int ranges = moe_ranges(active * a.down_tiles, a.down_steps, a.down_max);
  const int per = (int)(a.hidden / 8);
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.tokens * per; i += gridDim.x * kThreads)
    moe_out8(a, s.ids, ranges, i / per, (int64_t)(i % per) * 8);
}

// ---------------------------------------------------------------- host

struct MoeShape {
  int32_t pairs, chunks;
  bool few, many;  // pairs an expert: at most 1.5, more than 6
  int32_t up_tiles, up_max, up_steps;
  int32_t down_tiles, down_max, down_steps;
  size_t h_off, up_off, down_off, logits_off, bytes;
};

// A wavefront's ring: what the staged sums and the tables leave of LDS.
constexpr int kMoeRing = 34 * 1024;
constexpr int64_t kMoePartial = 64 << 20;  // bytes that the ranges of k may take

// Most ranges of k: 16, at least 4 steps each, within the partial products'
// room and the counters.
int32_t moe_most(int32_t steps, int64_t floats, bool counted) {
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>({counted ? 16 : 1, steps / 4, kMoePartial / (floats * 4)}));
}

MoeShape moe_shape(const moe_layer_desc& d) {
  MoeShape s = {};
  const bool fp8 = d.w_type == OVL_FP8;
  const int ks = fp8 ? 128 : 32;
  s.pairs = (int32_t)(d.tokens * d.topk);
  s.chunks = (int32_t)ceil_div(d.hidden, kMoeRouteRows);
  s.few = 2 * s.pairs <= 3 * d.experts;
  s.many = s.pairs > 6 * d.experts;
  s.up_tiles = (int32_t)ceil_div(d.inter, fp8 && d.gated ? 32 : 64);
  s.down_tiles = (int32_t)ceil_div(d.hidden, fp8 ? 64 : 128);
  s.up_steps = (int32_t)ceil_div(d.hidden, ks);
  s.down_steps = (int32_t)ceil_div(d.inter, ks);
  const int64_t n1 = d.gated ? 2 * d.inter : d.inter, pairs = std::max(s.pairs, 1);
  const int64_t up_items = std::min<int64_t>(d.experts, pairs) * s.up_tiles;
  s.up_max = moe_most(s.up_steps, pairs * n1, up_items <= kCounters - kMoeDownCounters);
  s.down_max = moe_most(s.down_steps, pairs * d.hidden, true);
  size_t off = kCounterBytes;
  const auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += aligned_up((size_t)bytes, 256);
    return at;
  };
  s.h_off = take(kMoePlanes * pairs * d.inter * 2);
  s.up_off = take(s.up_max > 1 ? s.up_max * pairs * n1 * 4 : 0);
  s.down_off = take(s.down_max * pairs * d.hidden * 4);
  s.logits_off = take((int64_t)s.chunks * d.tokens * d.experts * 8);
  s.bytes = off;
  return s;
}

ovl_status moe_check(const moe_layer_desc& d) {
  if (d.reserved || d.act < OVL_ACT_NONE || d.act > OVL_ACT_SILU || (d.gated & ~1) || (d.norm_topk & ~1) ||
      (d.w_type != OVL_BF16 && d.w_type != OVL_FP8) || (d.out_type != OVL_BF16 && d.out_type != OVL_F32))
    return OVL_EINVAL;
  if (d.tokens < 0 || d.hidden < 8 || d.inter < 8 || d.experts < 1 || d.topk < 1 || d.topk > d.experts)
    return OVL_ESHAPE;
  const int mult = d.w_type == OVL_FP8 ? 16 : 8;
  if (d.hidden % mult || d.inter % mult) return OVL_EALIGN;
  if (d.tokens > kMoeTokens || d.experts > kMoeExperts || d.topk > kMoeTopk || d.hidden > (1 << 16) ||
      d.inter > (1 << 16))
    return OVL_EUNSUPPORTED;
  // An expert's matrix stays within 32-bit buffer offsets.
  if (d.hidden * d.inter * (d.gated ? 2 : 1) * (d.w_type == OVL_FP8 ? 1 : 2) > (1ll << 30)) return OVL_EUNSUPPORTED;
  return OVL_OK;
}

template <class C>
ovl_status moe_up(const MoeArgs& a, hipStream_t stream) {
  ovl_status st = allow_lds(reinterpret_cast<const void*>(&moe_up_kernel<C>), C::LDS);
  if (st) return st;
  hipLaunchKernelGGL((moe_up_kernel<C>), dim3(kMoeGroups), dim3(kThreads), C::LDS, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  return OVL_OK;
}

template <class C>
ovl_status moe_down(const MoeArgs& a, hipStream_t stream) {
  const auto kernel = a.fused ? &moe_down_kernel<C, true> : &moe_down_kernel<C, false>;
  ovl_status st = allow_lds(reinterpret_cast<const void*>(kernel), C::LDS);
  if (st) return st;
  hipLaunchKernelGGL(kernel, dim3(kMoeGroups), dim3(kThreads), C::LDS, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  if (!a.fused) {
    hipLaunchKernelGGL((moe_sum_kernel<C>), dim3(ceil_div(a.tokens * a.hidden / 8, kThreads)), dim3(kThreads), 0, stream,
                       a);
    OVL_HIP_TRY(hipGetLastError());
  }
  return OVL_OK;
}

template <int EP>
ovl_status moe_route(const MoeArgs& a, hipStream_t stream) {
  if (a.tokens == 1)
    hipLaunchKernelGGL((moe_logits_kernel<EP, 1>), dim3(a.chunks), dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((moe_logits_kernel<EP, kMoeRouteTokens>), dim3(a.chunks * ceil_div(a.tokens, kMoeRouteTokens)),
                       dim3(kThreads), 0, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  if (a.pick) return OVL_OK;
  hipLaunchKernelGGL((moe_pick_kernel<EP>), dim3(a.tokens), dim3(kThreads), 0, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  return OVL_OK;
}

// bf16 weights: NB blocks of 16 rows a unit.  Two where experts have many
// tokens; their rows take a slot from the down launch's ring (64 tokens, top 2
// of 64: 134 us with two blocks, 115 with one).
template <int NB>
ovl_status moe_bf16(const MoeArgs& a, bool gated, hipStream_t stream) {
  const ovl_status st = gated ? moe_up<RowCfg<false, true, 1, NB, 1, kMoeRing>>(a, stream)
                              : moe_up<RowCfg<false, false, 1, NB, 1, kMoeRing>>(a, stream);
  return st ? st : moe_down<RowCfg<false, false, kMoePlanes, NB, 2, kMoeRing>>(a, stream);
}

// Codes: a step's rows take as much LDS as its weights, so that few rows leave
// a deeper ring: 4 a unit where an expert has few tokens, else what fits.
ovl_status moe_fp8(const MoeArgs& a, bool gated, bool few, hipStream_t stream) {
  if (few) {
    const ovl_status st = gated ? moe_up<RowCfg<true, true, 1, 1, 1, kMoeRing, 4>>(a, stream)
                                : moe_up<RowCfg<true, false, 1, 1, 2, kMoeRing, 4>>(a, stream);
    return st ? st : moe_down<RowCfg<true, false, kMoePlanes, 1, 2, kMoeRing, 4>>(a, stream);
  }
  const ovl_status st = gated ? moe_up<RowCfg<true, true, 1, 2, 1, kMoeRing>>(a, stream)
                              : moe_up<RowCfg<true, false, 1, 2, 2, kMoeRing>>(a, stream);
  return st ? st : moe_down<RowCfg<true, false, kMoePlanes, 1, 2, kMoeRing, 8>>(a, stream);
}

}  // namespace

}  // namespace ovl

using namespace ovl;

extern "C" size_t moe_layer_workspace_bytes(const moe_layer_desc* d) {
  if (!d || moe_check(*d)) return 0;
  return moe_shape(*d).bytes;
}

extern "C" ovl_status moe_layer_run(const moe_layer_desc* d, const void* x, const void* router, int32_t* topk_idx,
                                    float* gates, const void* w1, const float* w1_scale, const void* w2,
                                    const float* w2_scale, void* out, void* workspace, hipStream_t stream) {
  if (!d || !workspace) return OVL_EINVAL;
  ovl_status st = moe_check(*d);
  if (st) return st;
  if (!aligned16(workspace)) return OVL_EALIGN;
  if (d->tokens == 0) return OVL_OK;
  if (!x || !topk_idx || !gates || !w1 || !w2 || !out) return OVL_EINVAL;
  const bool fp8 = d->w_type == OVL_FP8;
  if (fp8 != (w1_scale != nullptr) || fp8 != (w2_scale != nullptr)) return OVL_EINVAL;
  if (!aligned16(x) || !aligned16(w1) || !aligned16(w2) || !aligned16(w1_scale) || !aligned16(w2_scale) ||
      !aligned16(out) || !aligned16(router) || (reinterpret_cast<uintptr_t>(topk_idx) & 3u) ||
      (reinterpret_cast<uintptr_t>(gates) & 3u))
    return OVL_EALIGN;
  const bool routed = router != nullptr;
  const CallBuffer buffers[] = {{x, false},        {router, false}, {topk_idx, routed}, {gates, routed}, {w1, false},
                                {w1_scale, false}, {w2, false},     {w2_scale, false},  {out, true},     {workspace, true}};
  if (begins_alike(buffers, {{-1, -1}})) return OVL_EINVAL;
  const MoeShape s = moe_shape(*d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MoeArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.router = static_cast<const uint16_t*>(router);
  a.topk = topk_idx;
  a.gates = gates;
  a.w1 = static_cast<const uint8_t*>(w1);
  a.s1 = w1_scale;
  a.w2 = static_cast<const uint8_t*>(w2);
  a.s2 = w2_scale;
  a.out = out;
  a.h = reinterpret_cast<uint16_t*>(ws + s.h_off);
  a.up = reinterpret_cast<float*>(ws + s.up_off);
  a.down = reinterpret_cast<float*>(ws + s.down_off);
  a.logits = reinterpret_cast<double*>(ws + s.logits_off);
  a.down_counters = reinterpret_cast<int32_t*>(ws + OVL_ERROR_RECORD_BYTES);
  a.up_counters = a.down_counters + kMoeDownCounters * kCounterStride;
  a.hidden = d->hidden;
  a.inter = d->inter;
  a.n1 = d->gated ? 2 * d->inter : d->inter;
  a.tokens = (int32_t)d->tokens;
  a.experts = d->experts;
  a.topk_n = d->topk;
  a.pairs = s.pairs;
  a.act = d->act;
  a.out_type = d->out_type;
  a.norm_topk = d->norm_topk;
  a.up_tiles = s.up_tiles;
  a.up_max = s.up_max;
  a.up_steps = s.up_steps;
  a.down_tiles = s.down_tiles;
  a.down_max = s.down_max;
  a.down_steps = s.down_steps;
  a.chunks = s.chunks;
  // At most one unit a workgroup, and no more tokens than one workgroup sums at
  // once (40 tokens, 112 x 400, top 4 of 16: 33 us the layer so, 24 with a launch
  // for the sum).
  a.fused = (int64_t)s.pairs * s.down_tiles <= kMoeGroups && s.pairs <= 8 * d->topk;
  a.pick = router && d->tokens == 1 && d->experts <= 64;
  if (router) {
    st = d->experts <= 64 ? moe_route<64>(a, stream)
                          : (d->experts <= 128 ? moe_route<128>(a, stream) : moe_route<256>(a, stream));
    if (st) return st;
  }
  if (fp8) return moe_fp8(a, d->gated, s.few, stream);
  return s.many ? moe_bf16<2>(a, d->gated, stream) : moe_bf16<1>(a, d->gated, stream);
}

// A whole mixture-of-experts layer for a few tokens: routing, the experts'
// two products, the gate-weighted sum.  What it must read is the chosen
// experts' weights; everything else is small, so the experts' products are
// rows.h's streams, spread over the chip by (chosen expert, 64 columns,
// range of k), and every reduction is done by whichever workgroup arrives
// last, in a fixed order.
//  1. Routing (with a router): ranges of hidden x groups of 16 tokens, sums
//     in float64 so that a choice between two near logits does not hang on
//     the order of a sum; the last range of a token group picks.
//  2. Up: u = x w1, then h = act(gate) * up as bf16 planes (see ovl.h).
//  3. Down: h w2 per (token, choice) pair in float32; the last workgroup of a
//     column tile, over all experts and ranges, sums each token's choices
//     with their gates, in order, and stores out.
// Every workgroup of 2 and 3 finds its expert itself: the chosen ids are at
// most 1024 words, from which it takes the set of distinct experts and its
// own expert's pairs.
#include <algorithm>

#include "epilogue.h"
#include "host.h"
#include "rows.h"

namespace ovl {

namespace {

constexpr int kMoeTokens = 128, kMoeExperts = 256, kMoeTopk = 8;
constexpr int kMoeRouteRows = 128;   // rows of the router a workgroup sums
constexpr int kMoeRouteTokens = 16;  // tokens of a routing group
constexpr int32_t kMoeDownCounters = 1024, kMoeRouteCounters = 16;  // then the up counters

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
  float* up;        // [up_splits][pairs][n1] when up_splits > 1
  float* down;      // [down_splits][pairs][hidden]
  double* logits;   // [chunks][tokens][experts]
  int32_t* down_counters;
  int32_t* route_counters;
  int32_t* up_counters;
  int64_t hidden, inter, n1;
  int32_t tokens, experts, topk_n, pairs, act, out_type, norm_topk;
  int32_t slots;  // a bound on the distinct experts chosen
  int32_t up_tiles, up_splits, up_steps, up_split_steps;
  int32_t down_tiles, down_splits, down_steps, down_split_steps;
  int32_t chunks;
};

// ---------------------------------------------------------------- routing

// a before b: the larger logit, NaN behind everything, then the lower id.
__device__ inline bool moe_before(double a, int ia, double b, int ib) {
  const bool na = isnan(a), nb = isnan(b);
  if (na != nb) return nb;
  if (!na && a != b) return a > b;
  return ia < ib;
}

// Token t's choices, by one wavefront.
__device__ inline void moe_pick(const MoeArgs& a, int t) {
  const int lane = lane_id();
  double v[4];
  bool have[4];
  double top = -HUGE_VAL;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    have[i] = e < a.experts;
    v[i] = 0;
    if (have[i]) {
      for (int c = 0; c < a.chunks; ++c) v[i] += a.logits[((int64_t)c * a.tokens + t) * a.experts + e];
      top = fmax(top, v[i]);
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = fmax(top, __shfl_xor(top, d, 64));
  double sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (have[i]) sum += exp(v[i] - top);
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
  double picked[kMoeTopk], chosen = 0;
#pragma unroll
  for (int j = 0; j < kMoeTopk; ++j) {
    picked[j] = 0;
    if (j >= a.topk_n) continue;
    double b = 0;
    int id = INT32_MAX;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (have[i] && (id == INT32_MAX || moe_before(v[i], lane + 64 * i, b, id))) {
        b = v[i];
        id = lane + 64 * i;
      }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const double ob = __shfl_xor(b, d, 64);
      const int oi = __shfl_xor(id, d, 64);
      if (oi != INT32_MAX && (id == INT32_MAX || moe_before(ob, oi, b, id))) {
        b = ob;
        id = oi;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i == id) have[i] = false;
    picked[j] = exp(b - top);
    chosen += picked[j];
    if (lane == 0) a.topk[t * a.topk_n + j] = id;
  }
  const double den = a.norm_topk ? chosen : sum;
#pragma unroll
  for (int j = 0; j < kMoeTopk; ++j)
    if (j < a.topk_n && lane == 0) a.gates[t * a.topk_n + j] = (float)(picked[j] / den);
}

// Workgroup (range of hidden, 16 tokens): EP lanes across the experts, 256 /
// EP rows of the router at a time, x from LDS.
template <int EP>
__global__ __launch_bounds__(kThreads) void moe_route_kernel(MoeArgs a) {
  constexpr int R = kThreads / EP;
  __shared__ float xs[kMoeRouteTokens][kMoeRouteRows];
  __shared__ double part[R][kMoeRouteTokens][EP];
  __shared__ int32_t flag;
  const int chunk = blockIdx.x % a.chunks, tg = blockIdx.x / a.chunks;
  const int t0 = tg * kMoeRouteTokens, nt = min(kMoeRouteTokens, a.tokens - t0);
  const int64_t r0 = (int64_t)chunk * kMoeRouteRows;
  const int nr = (int)min((int64_t)kMoeRouteRows, a.hidden - r0);
#pragma unroll
  for (int j = 0; j < kMoeRouteTokens * kMoeRouteRows / kThreads; ++j) {
    const int i = j * kThreads + threadIdx.x, t = i / kMoeRouteRows, r = i % kMoeRouteRows;
    const float v = bf16_lo_f(a.x[(t0 + min(t, nt - 1)) * a.hidden + r0 + min(r, nr - 1)]);
    xs[t][r] = t < nt && r < nr ? v : 0.f;
  }
  __syncthreads();
  const int e = threadIdx.x % EP, rr = threadIdx.x / EP;
  double acc[kMoeRouteTokens] = {};
  if (e < a.experts)
    for (int r = rr; r < nr; r += R) {
      const double w = bf16_lo_f(a.router[(r0 + r) * a.experts + e]);
#pragma unroll
      for (int t = 0; t < kMoeRouteTokens; ++t) acc[t] += w * xs[t][r];
    }
#pragma unroll
  for (int t = 0; t < kMoeRouteTokens; ++t) part[rr][t][e] = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < nt * EP; i += kThreads) {
    const int t = i / EP, x = i % EP;
    if (x >= a.experts) continue;
    double s = part[0][t][x];
#pragma unroll
    for (int q = 1; q < R; ++q) s += part[q][t][x];
    st8_agent(reinterpret_cast<uint64_t*>(a.logits + ((int64_t)chunk * a.tokens + t0 + t) * a.experts + x),
              __builtin_bit_cast(uint64_t, s));
  }
  if (!row_arrive_last(a.route_counters + tg, a.chunks, &flag)) return;
  for (int t = uniform(threadIdx.x >> 6); t < nt; t += kThreads / 64) moe_pick(a, t0 + t);
}

// ---------------------------------------------------------------- experts

// The distinct experts among the chosen ids: returns the slot-th of them, in
// ascending order (-1: fewer), and their number.
__device__ inline int moe_expert(const MoeArgs& a, int slot, uint64_t* mask, int* active) {
  if (threadIdx.x < 4) mask[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.pairs; i += kThreads) {
    const int e = a.topk[i];
    if (e >= 0 && e < a.experts)
      atomicOr(reinterpret_cast<unsigned long long*>(&mask[e >> 6]), 1ull << (e & 63));
  }
  __syncthreads();
  int n = 0, found = -1;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint64_t m = mask[w];
    const int c = __popcll(m);
    if (slot >= n && slot < n + c) {
      uint64_t r = m;
      for (int i = slot - n; i > 0; --i) r &= r - 1;
      found = 64 * w + __ffsll((unsigned long long)r) - 1;
    }
    n += c;
  }
  *active = uniform(n);
  return uniform(found);
}

// Pairs first .. first + N - 1 of expert e, in order, into the LDS table
// (-1 past the last); returns how many pairs e has.  By wavefront 0, between
// barriers.
template <int N>
__device__ inline int moe_rows(const MoeArgs& a, int e, int first, int32_t* rows, int32_t* count) {
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = lane_id();
    if (lane < N) rows[lane] = -1;
    int n = 0;
    for (int i = 0; i < a.pairs; i += 64) {
      const bool hit = i + lane < a.pairs && a.topk[i + lane] == e;
      const uint64_t m = __ballot(hit);
      const int at = n + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
      if (hit && at >= first && at < first + N) rows[at - first] = i + lane;
      n += __popcll(m);
    }
    if (lane == 0) *count = n;
  }
  __syncthreads();
  return uniform(*count);
}

// h as bf16 planes whose sum is h to 8 bits a plane.
__device__ inline void moe_store_h(const MoeArgs& a, int planes, int pair, int64_t col, float (&h)[8]) {
  for (int p = 0; p < planes; ++p) {
    store8(h, a.h, ((int64_t)p * a.pairs + pair) * a.inter + col, OVL_BF16);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float b = bf16_lo_f(bf16_bits(h[c]));
      h[c] = isfinite(b) ? h[c] - b : 0.f;  // an infinity or NaN stands in the first plane alone
    }
  }
}

// One pair's eight columns of the up product: scale, activation, h.
template <class C>
__device__ inline void moe_act(const MoeArgs& a, int planes, int pair, int64_t col, float (&g)[8], float (&u)[8]) {
  act8(g, a.act);
  if (C::PAIR)
#pragma unroll
    for (int c = 0; c < 8; ++c) g[c] *= u[c];
  moe_store_h(a, planes, pair, col, g);
}

template <class C>
__device__ inline void moe_scale(float (&v)[8], const float* s, int64_t i) {
  if (C::FP8) {
    float w[8];
    load8(w, s, i, OVL_F32);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] *= w[c];
  }
}

template <class C>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a, int planes) {
  extern __shared__ __align__(16) uint8_t moe_lds[];
  __shared__ int32_t rows[16 * C::NB], toks[16 * C::NB];
  __shared__ uint64_t mask[4];
  __shared__ int32_t flag, count;
  const int tile = blockIdx.x % a.up_tiles, sp = blockIdx.x / a.up_tiles % a.up_splits;
  const int slot = blockIdx.x / (a.up_tiles * a.up_splits);
  int active;
  const int e = moe_expert(a, slot, mask, &active);
  if (e < 0) return;
  RowOperands o = {};
  o.w_bytes = a.hidden * a.n1 * (C::FP8 ? 1 : 2);
  o.w = a.w1 + e * o.w_bytes;
  o.ldw = C::FP8 ? a.hidden : a.n1;
  o.col0 = (int64_t)tile * kRowCols;
  o.cols = a.inter;
  o.pair = a.inter;
  o.x = a.x;
  o.x_bytes = a.tokens * a.hidden * 2;
  o.ldx = a.hidden;
  o.k = a.hidden;
  const int s0 = min(sp * a.up_split_steps, a.up_steps), s1 = min(s0 + a.up_split_steps, a.up_steps);
  int n = 1;
  for (int first = 0; first < n; first += 16 * C::NB) {
    n = moe_rows<16 * C::NB>(a, e, first, rows, &count);
    if (threadIdx.x < 16 * C::NB) toks[threadIdx.x] = rows[threadIdx.x] < 0 ? -1 : rows[threadIdx.x] / a.topk_n;
    __syncthreads();
    const float* st = row_product<C>(o, toks, s0, s1, moe_lds);
    for (int i = threadIdx.x; i < 16 * C::NB * 8; i += kThreads) {
      const int pair = rows[i / 8];
      const int64_t col = o.col0 + (i % 8) * 8;
      if (pair < 0 || col >= a.inter) continue;
      float g[8], u[8];
      row_sums8<C>(g, st, 0, i / 8, (i % 8) * 8);
      moe_scale<C>(g, a.s1, e * a.n1 + col);
      if (C::PAIR) {
        row_sums8<C>(u, st, C::WT - 1, i / 8, (i % 8) * 8);
        moe_scale<C>(u, a.s1, e * a.n1 + a.inter + col);
      }
      if (a.up_splits > 1) {
        float* p = a.up + ((int64_t)sp * a.pairs + pair) * a.n1 + col;
        store8_agent(g, p);
        if (C::PAIR) store8_agent(u, p + a.inter);
      } else {
        moe_act<C>(a, planes, pair, col, g, u);
      }
    }
  }
  if (a.up_splits == 1) return;
  if (!row_arrive_last(a.up_counters + slot * a.up_tiles + tile, a.up_splits, &flag)) return;
  for (int first = 0; first < n; first += 16 * C::NB) {
    moe_rows<16 * C::NB>(a, e, first, rows, &count);
    for (int i = threadIdx.x; i < 16 * C::NB * 8; i += kThreads) {
      const int pair = rows[i / 8];
      const int64_t col = o.col0 + (i % 8) * 8;
      if (pair < 0 || col >= a.inter) continue;
      float g[8] = {}, u[8] = {};
      for (int s = 0; s < a.up_splits; ++s) {
        float q[8];
        const int64_t at = ((int64_t)s * a.pairs + pair) * a.n1 + col;
        load8(q, a.up, at, OVL_F32);
#pragma unroll
        for (int c = 0; c < 8; ++c) g[c] += q[c];
        if (C::PAIR) {
          load8(q, a.up, at + a.inter, OVL_F32);
#pragma unroll
          for (int c = 0; c < 8; ++c) u[c] += q[c];
        }
      }
      moe_act<C>(a, planes, pair, col, g, u);
    }
  }
}

// out of one column tile: every token's choices in order.
__device__ inline void moe_out(const MoeArgs& a, int64_t col0) {
  for (int i = threadIdx.x; i < a.tokens * 8; i += kThreads) {
    const int t = i / 8;
    const int64_t col = col0 + (i % 8) * 8;
    if (col >= a.hidden) continue;
    float v[8] = {};
    for (int j = 0; j < a.topk_n; ++j) {
      const int pair = t * a.topk_n + j, e = a.topk[pair];
      if (e < 0 || e >= a.experts) continue;
      float y[8] = {};
      for (int s = 0; s < a.down_splits; ++s) {
        float q[8];
        load8(q, a.down, ((int64_t)s * a.pairs + pair) * a.hidden + col, OVL_F32);
#pragma unroll
        for (int c = 0; c < 8; ++c) y[c] += q[c];
      }
      const float g = a.gates[pair];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] += g * y[c];
    }
    store8(v, a.out, t * a.hidden + col, a.out_type);
  }
}

template <class C>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
  extern __shared__ __align__(16) uint8_t moe_lds[];
  __shared__ int32_t rows[16 * C::NB];
  __shared__ uint64_t mask[4];
  __shared__ int32_t flag, count;
  const int tile = blockIdx.x % a.down_tiles, sp = blockIdx.x / a.down_tiles % a.down_splits;
  const int slot = blockIdx.x / (a.down_tiles * a.down_splits);
  int active;
  const int e = moe_expert(a, slot, mask, &active);
  if (active == 0 && slot == 0 && sp == 0) moe_out(a, (int64_t)tile * kRowCols);  // zeros
  if (e < 0) return;
  RowOperands o = {};
  o.w_bytes = a.hidden * a.inter * (C::FP8 ? 1 : 2);
  o.w = a.w2 + e * o.w_bytes;
  o.ldw = C::FP8 ? a.inter : a.hidden;
  o.col0 = (int64_t)tile * kRowCols;
  o.cols = a.hidden;
  o.x = a.h;
  o.plane = a.pairs * a.inter;
  o.x_bytes = C::PL * o.plane * 2;
  o.ldx = a.inter;
  o.k = a.inter;
  const int s0 = min(sp * a.down_split_steps, a.down_steps), s1 = min(s0 + a.down_split_steps, a.down_steps);
  int n = 1;
  for (int first = 0; first < n; first += 16 * C::NB) {
    n = moe_rows<16 * C::NB>(a, e, first, rows, &count);
    const float* st = row_product<C>(o, rows, s0, s1, moe_lds);
    for (int i = threadIdx.x; i < 16 * C::NB * 8; i += kThreads) {
      const int pair = rows[i / 8];
      const int64_t col = o.col0 + (i % 8) * 8;
      if (pair < 0 || col >= a.hidden) continue;
      float v[8];
      row_sums8<C>(v, st, 0, i / 8, (i % 8) * 8);
      moe_scale<C>(v, a.s2, e * a.hidden + col);
      store8_agent(v, a.down + ((int64_t)sp * a.pairs + pair) * a.hidden + col);
    }
  }
  if (row_arrive_last(a.down_counters + tile, active * a.down_splits, &flag)) moe_out(a, o.col0);
}

// ---------------------------------------------------------------- host

struct MoeShape {
  int32_t slots, pairs, planes, chunks, groups;
  int32_t up_tiles, up_splits, up_steps, up_split_steps;
  int32_t down_tiles, down_splits, down_steps, down_split_steps;
  size_t h_off, up_off, down_off, logits_off, bytes;
};

constexpr int kMoeTarget = 512;  // workgroups that fill the chip

void moe_split(int64_t k, int ks, int64_t items, int max_splits, int32_t* steps, int32_t* splits, int32_t* per) {
  *steps = (int32_t)ceil_div(k, ks);
  int64_t sp = std::min<int64_t>({(int64_t)max_splits, ceil_div(kMoeTarget, items), *steps / 8});
  sp = std::max<int64_t>(sp, 1);
  *per = (int32_t)ceil_div(*steps, sp);
  *splits = (int32_t)ceil_div(*steps, *per);
}

MoeShape moe_shape(const moe_layer_desc& d) {
  MoeShape s = {};
  const int ks = d.w_type == OVL_FP8 ? 64 : 32;
  s.pairs = (int32_t)(d.tokens * d.topk);
  s.slots = std::max(1, std::min(d.experts, s.pairs));
  s.planes = d.out_type == OVL_F32 ? 3 : 2;
  s.chunks = (int32_t)ceil_div(d.hidden, kMoeRouteRows);
  s.groups = (int32_t)ceil_div(d.tokens, kMoeRouteTokens);
  s.up_tiles = (int32_t)ceil_div(d.inter, kRowCols);
  s.down_tiles = (int32_t)ceil_div(d.hidden, kRowCols);
  const int64_t up_items = (int64_t)s.slots * s.up_tiles;
  const bool up_counted = up_items <= kCounters - kMoeDownCounters - kMoeRouteCounters;
  moe_split(d.hidden, ks, up_items, up_counted ? 16 : 1, &s.up_steps, &s.up_splits, &s.up_split_steps);
  moe_split(d.inter, ks, (int64_t)s.slots * s.down_tiles, 16, &s.down_steps, &s.down_splits, &s.down_split_steps);
  const int64_t n1 = d.gated ? 2 * d.inter : d.inter;
  size_t off = kCounterBytes;
  const auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += aligned_up((size_t)bytes, 256);
    return at;
  };
  s.h_off = take((int64_t)s.planes * s.pairs * d.inter * 2);
  s.up_off = take(s.up_splits > 1 ? (int64_t)s.up_splits * s.pairs * n1 * 4 : 0);
  s.down_off = take((int64_t)s.down_splits * s.pairs * d.hidden * 4);
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
ovl_status moe_up(const MoeArgs& a, int planes, hipStream_t stream) {
  ovl_status st = allow_lds(reinterpret_cast<const void*>(&moe_up_kernel<C>), C::LDS);
  if (st) return st;
  hipLaunchKernelGGL((moe_up_kernel<C>), dim3(a.slots * a.up_tiles * a.up_splits), dim3(kThreads), C::LDS, stream, a,
                     planes);
  OVL_HIP_TRY(hipGetLastError());
  return OVL_OK;
}

template <class C>
ovl_status moe_down(const MoeArgs& a, hipStream_t stream) {
  ovl_status st = allow_lds(reinterpret_cast<const void*>(&moe_down_kernel<C>), C::LDS);
  if (st) return st;
  hipLaunchKernelGGL((moe_down_kernel<C>), dim3(a.slots * a.down_tiles * a.down_splits), dim3(kThreads), C::LDS,
                     stream, a);
  OVL_HIP_TRY(hipGetLastError());
  return OVL_OK;
}

template <int EP>
ovl_status moe_route(const MoeArgs& a, int groups, hipStream_t stream) {
  hipLaunchKernelGGL((moe_route_kernel<EP>), dim3(a.chunks * groups), dim3(kThreads), 0, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  return OVL_OK;
}

template <bool FP8, int NB>
ovl_status moe_experts(const MoeArgs& a, bool gated, int planes, hipStream_t stream) {
  const ovl_status st = gated ? moe_up<RowCfg<FP8, true, 1, NB>>(a, planes, stream)
                              : moe_up<RowCfg<FP8, false, 1, NB>>(a, planes, stream);
  if (st) return st;
  return planes == 2 ? moe_down<RowCfg<FP8, false, 2, NB>>(a, stream) : moe_down<RowCfg<FP8, false, 3, NB>>(a, stream);
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
  a.route_counters = a.down_counters + kMoeDownCounters;
  a.up_counters = a.route_counters + kMoeRouteCounters;
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
  a.slots = s.slots;
  a.up_tiles = s.up_tiles;
  a.up_splits = s.up_splits;
  a.up_steps = s.up_steps;
  a.up_split_steps = s.up_split_steps;
  a.down_tiles = s.down_tiles;
  a.down_splits = s.down_splits;
  a.down_steps = s.down_steps;
  a.down_split_steps = s.down_split_steps;
  a.chunks = s.chunks;
  if (router) {
    st = d->experts <= 64 ? moe_route<64>(a, s.groups, stream)
                          : (d->experts <= 128 ? moe_route<128>(a, s.groups, stream)
                                               : moe_route<256>(a, s.groups, stream));
    if (st) return st;
  }
  // Groups of 32 rows only where more than 16 tokens can meet at an expert.
  if (fp8)
    return d->tokens <= 16 ? moe_experts<true, 1>(a, d->gated, s.planes, stream)
                           : moe_experts<true, 2>(a, d->gated, s.planes, stream);
  return d->tokens <= 16 ? moe_experts<false, 1>(a, d->gated, s.planes, stream)
                         : moe_experts<false, 2>(a, d->gated, s.planes, stream);
}

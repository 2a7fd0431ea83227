// Product with bias, activation and residual in its epilogue, and its
// gradient:
//   forward:  z = A B + bias, out = act(z) + residual;
//   gradient: dA = (dZ B^T) * act_in'(z_in), dB = dB_in + A^T dZ,
//             dbias = dbias_in + column sums of dZ.
// The products are gemm_any.h's tiles.  A tile's sums leave through LDS in
// 8-column pieces, so that bias, residual and outputs move in 16-byte
// vectors and the pre-activation is rounded from the same float32 sums as
// the output.  The gradient's two products and its column sums are the items
// of one launch: they share nothing but their inputs, and each fills the
// compute units that the others' last rounds leave idle.  Where tiles are
// few, K is split: the ranges' float32 products go to the workspace and a
// second launch sums them in range order and applies the epilogue.
//
// Measured, with what bounds them: forward 8192 x 3584 x 4096 with bias and
// GELU 236 us (matrix units and power); gradient 8192 x 4096 x 1792 239 us (the
// same, 1.01 PFLOP/s over both products; with the activation of the call's own,
// a launch before it, 268); 1000 x 2056 x 520 13.3 us and the gradient of 700 x
// 2056 x 520 16.6 us (latency: a launch, 9 and 11 K steps, an epilogue, a second
// launch in the latter); 1 x 7168 x 8192 24.3 us (HBM, 117 MB at 4.8 TB/s with
// start and end, which take about 5 us of it); 1 x 50304 x 4096 74 us and 1 x
// 36864 x 4096 75 us (HBM at 5.5 and 4.0 TB/s: one workgroup a column tile, 393
// and 288 of them, so that the second round is half and an eighth full).
#include <algorithm>

#include "epilogue.h"
#include "gemm_any.h"
#include "host.h"
#include "rows.h"

namespace ovl {

namespace {

constexpr int kLinMaxSplits = 16;

// One product's tiles: tiles_m * tiles_n * splits items.
struct LinJob {
  AnyOperand a, b;
  Epilogue epi;
  float* partial;     // [splits][m][n] when splits > 1
  int64_t m, n;       // output
  int32_t steps;      // K steps of 64
  int32_t split_steps;
  int32_t tiles_m, tiles_n, splits;
  int32_t items;
};

// Column sums of dz, strips of 64 columns x ranges of rows.
struct LinSum {
  const uint16_t* dz;
  const float* in;
  float* out;
  float* partial;  // [splits][n] when splits > 1
  int64_t ld, m, n, rows;  // rows of a range
  int32_t strips, splits;
  int32_t items;
};

struct LinArgs {
  LinJob job[2];
  LinSum sum;
  int32_t second_first;  // job 1's tiles are the longer ones
};

// Items of die x (workgroup b runs on die b % 8): a consecutive share, so that
// a die's tiles share operand panels in its L2.
__host__ __device__ inline int lin_share(int items, int x) { return items / 8 + (x < items % 8); }
__device__ inline int lin_item(int items, int x, int q) { return x * (items / 8) + min(x, items % 8) + q; }

template <class T>
__device__ inline void lin_tile(const LinJob& j, int item, uint8_t* lds) {
  // Tiles in groups of 4 tile rows, column by column within a group; the K
  // ranges of a tile lie tiles apart, so that a die's tiles read the same
  // range.
  const int tiles = j.tiles_m * j.tiles_n;
  const int sp = item / tiles, t = item % tiles;
  constexpr int G = 4;
  const int g = t / (G * j.tiles_n), rows = min(G, j.tiles_m - g * G), r = t % (G * j.tiles_n);
  const int64_t m0 = (int64_t)(g * G + r % rows) * T::BM, n0 = (int64_t)(r / rows) * T::BN;
  const int s0 = min(sp * j.split_steps, j.steps), s1 = min(s0 + j.split_steps, j.steps);
  typename T::Acc acc;
  any_tile<T>(acc, j.a, j.b, m0, n0, s0, s1, lds);
  if (j.splits > 1) {
    float* p = j.partial + (int64_t)sp * j.m * j.n;
    any_rows<T>(acc, lds, [](int, int) { return 0; }, [&](int row, int col, float (&v)[8], int) {
      if (m0 + row < j.m && n0 + col < j.n) store8(v, p, (m0 + row) * j.n + n0 + col, OVL_F32);
    });
  } else {
    const auto there = [&](int row, int col) { return m0 + row < j.m && n0 + col < j.n; };
    float bias[8];
    epilogue_bias(bias, j.epi, n0 + any_col<T>(), there(0, any_col<T>()));
    any_rows<T>(acc, lds,
                [&](int row, int col) {
                  return there(row, col) ? epilogue_load(j.epi, m0 + row, n0 + col) : EpilogueIn{};
                },
                [&](int row, int col, float (&v)[8], const EpilogueIn& x) {
                  if (there(row, col)) epilogue8(j.epi, m0 + row, n0 + col, v, bias, x);
                });
  }
}

// Columns [64 strip, +64) of rows [r0, r1): eight lanes across the strip,
// NT / 8 rows at a time, each thread adding its rows in order, then the
// threads of a column through LDS in a fixed tree.
template <int NT>
__device__ inline void lin_sum(const LinSum& s, int item, uint8_t* lds) {
  constexpr int ROWS = NT / 8;
  const int strip = item % s.strips, sp = item / s.strips;
  const int64_t r0 = sp * s.rows, r1 = min(r0 + s.rows, s.m);
  const int64_t col = (int64_t)strip * 64 + (threadIdx.x % 8) * 8;
  const int tr = threadIdx.x / 8;
  float v[8] = {};
  if (col < s.n) {
    const uint16_t* p = s.dz + col;
    int64_t r = r0 + tr;
    for (; r + 3 * ROWS < r1; r += 4 * ROWS) {
      u32x4 w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = ld16(p + (r + u * ROWS) * s.ld);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[2 * c] += bf16_lo_f(w[u][c]);
          v[2 * c + 1] += bf16_hi_f(w[u][c]);
        }
    }
    for (; r < r1; r += ROWS) {
      const u32x4 w = ld16(p + r * s.ld);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[2 * c] += bf16_lo_f(w[c]);
        v[2 * c + 1] += bf16_hi_f(w[c]);
      }
    }
  }
  float* area = reinterpret_cast<float*>(lds);  // [ROWS][64]
#pragma unroll
  for (int c = 0; c < 8; ++c) area[tr * 64 + (threadIdx.x % 8) * 8 + c] = v[c];
  __syncthreads();
  if (threadIdx.x < 64) {
    const int64_t c = (int64_t)strip * 64 + threadIdx.x;
    float t[4] = {};
    for (int i = 0; i < ROWS; i += 4)
#pragma unroll
      for (int u = 0; u < 4; ++u) t[u] += area[(i + u) * 64 + threadIdx.x];
    const float total = (t[0] + t[1]) + (t[2] + t[3]);
    if (c < s.n) {
      if (s.splits > 1)
        s.partial[(int64_t)sp * s.n + c] = total;
      else
        s.out[c] = s.in ? s.in[c] + total : total;
    }
  }
}

// One item a workgroup.  TA is job 0's tile, TB job 1's.
template <class T>
__global__ __launch_bounds__(64 * T::NW, T::NW == 4 ? 2 : 1) void lin_fwd_kernel(LinJob j) {
  extern __shared__ __align__(16) uint8_t lin_lds[];
  lin_tile<T>(j, lin_item(j.items, blockIdx.x % 8, blockIdx.x / 8), lin_lds);
}

template <class TA, class TB>
__global__ __launch_bounds__(64 * TA::NW, TA::NW == 4 ? 2 : 1) void lin_grad_kernel(LinArgs a) {
  extern __shared__ __align__(16) uint8_t lin_lds[];
  // Every die takes its share of each product and of the sums, the product
  // with the longer tiles first (a die's last round is then short tiles and
  // sums: 8192 x 4096 x 1792 ran in 405 us with the items of the one product
  // all on the first dies).
  const int x = blockIdx.x % 8;
  int q = blockIdx.x / 8;
  const int n0 = lin_share(a.job[0].items, x), n1 = lin_share(a.job[1].items, x);
  if (a.second_first) q = q < n1 ? q + n0 : (q < n0 + n1 ? q - n1 : q);
  if (q < n0)
    lin_tile<TA>(a.job[0], lin_item(a.job[0].items, x, q), lin_lds);
  else if (q < n0 + n1)
    lin_tile<TB>(a.job[1], lin_item(a.job[1].items, x, q - n0), lin_lds);
  else if (q - n0 - n1 < lin_share(a.sum.items, x))
    lin_sum<64 * TA::NW>(a.sum, lin_item(a.sum.items, x, q - n0 - n1), lin_lds);
}

struct LinReduceArgs {
  LinJob job[2];
  LinSum sum;
  int64_t pieces[2];  // 8-column pieces of each split job's output
};

// The second launch of split products: every 8-column piece's partial sums
// in range order, then the epilogue.
__global__ __launch_bounds__(kThreads) void lin_reduce_kernel(LinReduceArgs a) {
  const int64_t total = a.pieces[0] + a.pieces[1];
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t i = first; i < total; i += stride) {
    const int w = i >= a.pieces[0];
    const LinJob& j = a.job[w];
    const int64_t p = w ? i - a.pieces[0] : i;
    const int64_t per = j.n / 8, row = p / per, col = (p - row * per) * 8;
    float v[8];
    load8(v, j.partial, row * j.n + col, OVL_F32);
    for (int s = 1; s < j.splits; ++s) {
      float q[8];
      load8(q, j.partial, ((int64_t)s * j.m + row) * j.n + col, OVL_F32);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] += q[c];
    }
    epilogue8(j.epi, row, col, v);
  }
  if (a.sum.splits > 1)
    for (int64_t c = first; c < a.sum.n; c += stride) {
      float t = 0.f;
      for (int s = 0; s < a.sum.splits; ++s) t += a.sum.partial[(int64_t)s * a.sum.n + c];
      a.sum.out[c] = a.sum.in ? a.sum.in[c] + t : t;
    }
}

// Few rows (decoding): column tiles of 128 x K ranges, rows.h's stream.  The
// last range of a tile to arrive sums the ranges' partial products in range
// order and applies the epilogue.
struct LinRowArgs {
  RowOperands o;
  Epilogue epi;
  float* partial;  // [splits][m][n]
  int32_t* counters;
  int64_t m, n;
  int32_t tiles, splits, steps, split_steps;
};

// One unit a workgroup.
template <class C>
struct LinRowGen {
  const RowOperands* o;
  const int32_t* rows;
  int32_t s0, s1;
  __device__ inline bool range(int32_t u, int32_t& a, int32_t& b) const {
    a = s0;
    b = s1;
    return u == 0;
  }
  __device__ inline bool begin(int32_t u, RowLoads<C>& ld, int32_t& a, int32_t& b) const {
    if (u == 0) ld.init(*o, rows);
    return range(u, a, b);
  }
  __device__ inline int32_t turn(int32_t) const { return 0; }
};

template <class C>
__global__ __launch_bounds__(kThreads) void lin_row_kernel(LinRowArgs a) {
  extern __shared__ __align__(16) uint8_t row_lds[];
  __shared__ int32_t rows[16 * C::NB];
  __shared__ int32_t flag;
  constexpr int PR = C::COLS / 8;  // pieces of a row
  const int tile = blockIdx.x % a.tiles, sp = blockIdx.x / a.tiles;
  if (threadIdx.x < 16 * C::NB) rows[threadIdx.x] = (int)threadIdx.x < a.m ? (int)threadIdx.x : -1;
  __syncthreads();
  RowOperands o = a.o;
  o.col0 = (int64_t)tile * C::COLS;
  const int s0 = min(sp * a.split_steps, a.steps);
  LinRowGen<C> gen{&o, rows, s0, min(s0 + a.split_steps, a.steps)};
  const int pieces = (int)a.m * PR;
  row_stream<C>(gen, row_lds, [&](int32_t, const float* st) {
    if (a.splits > 1) {
      float* p = a.partial + (int64_t)sp * a.m * a.n;
      for (int i = threadIdx.x; i < pieces; i += kThreads) {
        const int row = i / PR;
        const int64_t col = o.col0 + (i % PR) * 8;
        if (col >= a.n) continue;
        float v[8];
        row_sums8<C>(v, st, 0, row, (i % PR) * 8);
        store8_agent(v, p + row * a.n + col);
      }
      if (!row_arrive_last(a.counters + tile * kCounterStride, a.splits, &flag)) return;
    }
    for (int i = threadIdx.x; i < pieces; i += kThreads) {
      const int row = i / PR;
      const int64_t col = o.col0 + (i % PR) * 8;
      if (col >= a.n) continue;
      float v[1][8], bias[8];
      // The epilogue's own loads go out with the sums'.
      epilogue_bias(bias, a.epi, col, true);
      const EpilogueIn x = epilogue_load(a.epi, row, col);
      if (a.splits > 1)
        row_ranges8(v, a.partial + row * a.n + col, a.splits, a.m * a.n, 0);
      else
        row_sums8<C>(v[0], st, 0, row, (i % PR) * 8);
      epilogue8(a.epi, row, col, v[0], bias, x);
    }
    wave_drain();
  });
}

// dz = bf16(dy * act'(z)), rows x cols with row strides.
struct LinDactArgs {
  const void* dy;
  const uint16_t* z;
  uint16_t* dz;
  int64_t ld_dy, ld_z, ld_dz, m, n;
  int32_t dy_type, act;
};

__global__ __launch_bounds__(kThreads) void lin_dact_kernel(LinDactArgs a) {
  const int64_t per = a.n / 8, total = a.m * per, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += stride) {
    const int64_t row = i / per, col = (i - row * per) * 8;
    float d[8], z[8];
    load8(d, a.dy, row * a.ld_dy + col, a.dy_type);
    load8(z, a.z, row * a.ld_z + col, OVL_BF16);
    act_grad8(d, z, a.act);
    store8(d, a.dz, row * a.ld_dz + col, OVL_BF16);
  }
}

using Fwd256 = AnyTile<256, 256, 8, true, false>;
using Fwd128 = AnyTile<128, 128, 4, true, false>;
using Da256 = AnyTile<256, 256, 8, true, true>;
using Da128 = AnyTile<128, 128, 4, true, true>;
using Db256 = AnyTile<256, 256, 8, false, false>;
using Db128 = AnyTile<128, 128, 4, false, false>;
// Few tiles: half the rows, three stages deep, two workgroups a compute unit
// (1000 x 2056 x 520: 13.5 us against 14.6 with 128 x 128 tiles four deep; the
// gradient of 128 x 256 x 256, captured, 6.1 against 8.5).
using Fwd64 = AnyTile<64, 128, 4, true, false, 3>;
using Da64 = AnyTile<64, 128, 4, true, true, 3>;
using Db64 = AnyTile<64, 128, 4, false, false, 3>;

// Tile edge and K splits of the products of one launch.  Both the size
// queries and the launches use this.
struct LinShape {
  int tile_m, tile_n;  // 256 x 256, 128 x 128 or 64 x 128
  int32_t splits[2];
  int32_t sum_splits;
  size_t partial_off[2], sum_off, bytes;
};

constexpr int kLinCus = 256;  // the plan is made for a whole MI355X, so that sizes do not hang on the device

// What cutting K costs and saves, in microseconds: a step of a 64 x 128 tile,
// two on a compute unit, a second launch, and a float32 partial product's way
// to memory and back (8 bytes an element at 4 TB/s).  The operands' own way from
// memory is not in it, and a gradient without da or db is cut as the whole one.
// The three are fitted together to the times of calls, and the launch's is not
// what a trace gives it (4 us, the second kernel's own work included).
// Captured, us as this cuts and whole: forward 40 x 512 x 4096 12.9 and 27.8,
// 512 x 1024 x 2048 14.1 and 18.2, 256 x 1024 x 1024 11.2 and 12.3, 256 x 4096 x
// 1792 16.4 and 17.2; gradient of 700 x 2056 x 520 18.6 and 21.8, of 4000 x 264 x
// 264 19.1 and 31.1, but of 1000 x 264 x 264 13.7 and 11.1.  With 4 us for the
// launch the last one runs whole, and so do the two forward ones before.
constexpr double kLinStepUs = 0.4, kLinLaunchUs = 1.0, kLinPartialUs = 8.0 / 4e6;

LinShape lin_shape(const int64_t (*mnk)[3], int jobs, int64_t sum_m, int64_t sum_n) {
  LinShape s = {};
  const auto tiles_of = [&](int j, int64_t tm, int64_t tn) {
    return ceil_div(mnk[j][0], tm) * ceil_div(mnk[j][1], tn);
  };
  int64_t t256 = 0, t64 = 0, steps[2] = {1, 1}, tiles[2] = {}, longest = 1;
  for (int j = 0; j < jobs; ++j) {
    t256 += tiles_of(j, 256, 256);
    t64 += tiles_of(j, 64, 128);
    steps[j] = std::max<int64_t>(1, ceil_div(mnk[j][2], kAnyBK));
    if (mnk[j][0]) longest = std::max(longest, steps[j]);
  }
  // 256 x 256 where such tiles fill half the chip; 64 x 128 where even those
  // run all at once; 128 x 128 between.
  const bool few = t64 <= 2 * kLinCus;
  s.tile_m = t256 >= kLinCus / 2 ? 256 : (few ? 64 : 128);
  s.tile_n = s.tile_m == 256 ? 256 : 128;
  for (int j = 0; j < jobs; ++j) tiles[j] = tiles_of(j, s.tile_m, s.tile_n);
  // Cut K where few tiles have many steps.  Items that all run at once: into
  // the length that costs least.  More of them: a product whose tiles are over
  // half again as long as a compute unit's share of all the work is cut to that
  // share (64 x 7168 x 8192, gradient: 32 tiles of 112 steps beside 896 of one;
  // 183 us whole, 91 cut).
  int64_t len = longest;
  if (s.tile_m == 64) {
    double best = kLinStepUs * longest;
    for (int64_t c = 2; c <= kLinMaxSplits; ++c) {
      const int64_t l = ceil_div(longest, c);
      int64_t items = 0;
      double cost = kLinStepUs * l + kLinLaunchUs;
      for (int j = 0; j < jobs; ++j) {
        const int64_t cuts = ceil_div(steps[j], l);
        items += tiles[j] * cuts;
        if (cuts > 1) cost += kLinPartialUs * cuts * mnk[j][0] * mnk[j][1];
      }
      if (items > 2 * kLinCus) break;
      if (cost < best) {
        best = cost;
        len = l;
      }
    }
  } else {
    int64_t work = 0;
    for (int j = 0; j < jobs; ++j) work += tiles[j] * steps[j];
    const int64_t share = std::max<int64_t>({8, ceil_div(work, s.tile_m == 256 ? kLinCus : 2 * kLinCus),
                                             ceil_div(longest, kLinMaxSplits)});
    if (2 * longest > 3 * share) len = share;
  }
  size_t off = kCounterBytes;
  for (int j = 0; j < jobs; ++j) {
    int64_t sp = ceil_div(steps[j], len);
    sp = ceil_div(steps[j], ceil_div(steps[j], sp));  // no empty range
    s.splits[j] = (int32_t)sp;
    s.partial_off[j] = off;
    if (sp > 1) off += aligned_up((size_t)(sp * mnk[j][0] * mnk[j][1]) * 4, 256);
  }
  // Column sums: a workgroup adds a strip's rows at the latency of its loads, so
  // few strips are cut into ranges of rows (7936 x 16 x 64, gradient: 24 us in one,
  // 14 cut).
  const int64_t strips = std::max<int64_t>(1, ceil_div(sum_n, 64));
  s.sum_splits = (int32_t)std::max<int64_t>({1, std::min<int64_t>(sum_m / 1024, 64 / strips), std::min<int64_t>(sum_m / 16384, 64)});
  s.sum_off = off;
  if (s.sum_splits > 1) off += aligned_up((size_t)s.sum_splits * sum_n * 4, 256);
  s.bytes = off;
  return s;
}

LinJob lin_job(const LinShape& s, int j, const AnyOperand& a, const AnyOperand& b, const Epilogue& epi, void* ws) {
  LinJob r = {};
  r.a = a;
  r.b = b;
  r.epi = epi;
  r.m = a.rows;
  r.n = b.rows;
  r.steps = (int32_t)ceil_div(a.k, kAnyBK);
  r.splits = s.splits[j];
  r.split_steps = (int32_t)ceil_div(std::max(r.steps, 1), r.splits);
  r.tiles_m = (int32_t)ceil_div(r.m, s.tile_m);
  r.tiles_n = (int32_t)ceil_div(r.n, s.tile_n);
  r.items = r.tiles_m * r.tiles_n * r.splits;
  r.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + s.partial_off[j]);
  return r;
}

ovl_status lin_reduce(const LinArgs& a, hipStream_t stream);

template <class T>
ovl_status lin_fwd_launch(const LinArgs& a, hipStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(&lin_fwd_kernel<T>);
  ovl_status st = allow_lds(fn, T::LDS_BYTES);
  if (st) return st;
  hipLaunchKernelGGL((lin_fwd_kernel<T>), dim3(a.job[0].items), dim3(64 * T::NW), T::LDS_BYTES, stream, a.job[0]);
  OVL_HIP_TRY(hipGetLastError());
  return lin_reduce(a, stream);
}

template <class TA, class TB>
ovl_status lin_grad_launch(LinArgs& a, hipStream_t stream) {
  a.second_first = a.job[1].split_steps > a.job[0].split_steps;
  int per = 0;
  for (int x = 0; x < 8; ++x)
    per = std::max(per, lin_share(a.job[0].items, x) + lin_share(a.job[1].items, x) + lin_share(a.sum.items, x));
  if (!per) return OVL_OK;
  const void* fn = reinterpret_cast<const void*>(&lin_grad_kernel<TA, TB>);
  const int lds = std::max(TA::LDS_BYTES, TB::LDS_BYTES);
  ovl_status st = allow_lds(fn, lds);
  if (st) return st;
  hipLaunchKernelGGL((lin_grad_kernel<TA, TB>), dim3(8 * per), dim3(64 * TA::NW), lds, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  return lin_reduce(a, stream);
}

ovl_status lin_reduce(const LinArgs& a, hipStream_t stream) {
  LinReduceArgs r = {};
  for (int j = 0; j < 2; ++j) {
    r.job[j] = a.job[j];
    r.pieces[j] = a.job[j].items && a.job[j].splits > 1 ? a.job[j].m * (a.job[j].n / 8) : 0;
  }
  r.sum = a.sum;
  if (!a.sum.items) r.sum.splits = 1;
  const int64_t work = r.pieces[0] + r.pieces[1] + (r.sum.splits > 1 ? r.sum.n : 0);
  if (work) {
    hipLaunchKernelGGL(lin_reduce_kernel, dim3((uint32_t)std::min<int64_t>(2048, ceil_div(work, kThreads))),
                       dim3(kThreads), 0, stream, r);
    OVL_HIP_TRY(hipGetLastError());
  }
  return OVL_OK;
}

bool is_type(int32_t t) { return t == OVL_BF16 || t == OVL_F32; }
bool is_act(int32_t a) { return a >= OVL_ACT_NONE && a <= OVL_ACT_SILU; }

// A row stride: 0 stands for `len`.
ovl_status lin_ld(int64_t* ld, int64_t len) {
  if (*ld == 0) *ld = len;
  if (*ld < len) return OVL_ESHAPE;
  if (*ld % 8) return OVL_EALIGN;
  if (*ld > (1 << 20)) return OVL_EUNSUPPORTED;
  return OVL_OK;
}

constexpr int64_t kLinSpan = 1ll << 30;  // an operand's bytes, so that 32-bit buffer offsets never wrap

ovl_status lin_sizes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 8 || k < 8) return OVL_ESHAPE;
  if (n % 8 || k % 8) return OVL_EALIGN;
  if (m > (1 << 20) || n > (1 << 20) || k > (1 << 20)) return OVL_EUNSUPPORTED;
  return OVL_OK;
}

// The checked descriptor with every stride filled in.
ovl_status lin_fwd_desc(gemm_epilogue_desc* d) {
  ovl_status st = lin_sizes(d->m, d->n, d->k);
  if (st) return st;
  if (!is_act(d->act) || !is_type(d->out_type) || !is_type(d->res_type) || d->reserved) return OVL_EINVAL;
  if ((st = lin_ld(&d->lda, d->k)) || (st = lin_ld(&d->ldb, d->n)) || (st = lin_ld(&d->ldo, d->n)) ||
      (st = lin_ld(&d->ldz, d->n)) || (st = lin_ld(&d->ldr, d->n)))
    return st;
  if (d->m * d->lda * 2 > kLinSpan || d->k * d->ldb * 2 > kLinSpan) return OVL_EUNSUPPORTED;
  return OVL_OK;
}

ovl_status lin_grad_desc(gemm_epilogue_grad_desc* d) {
  ovl_status st = lin_sizes(d->m, d->n, d->k);
  if (st) return st;
  if (!is_act(d->act) || !is_act(d->act_in) || !is_type(d->dy_type) || !is_type(d->da_type) ||
      !is_type(d->db_type) || d->reserved)
    return OVL_EINVAL;
  if ((st = lin_ld(&d->lda, d->k)) || (st = lin_ld(&d->ldb, d->n)) || (st = lin_ld(&d->lddz, d->n)) ||
      (st = lin_ld(&d->lddy, d->n)) || (st = lin_ld(&d->ldz, d->n)) || (st = lin_ld(&d->ldz_in, d->k)) ||
      (st = lin_ld(&d->ldda, d->k)) || (st = lin_ld(&d->lddb, d->n)))
    return st;
  if (d->m * d->lda * 2 > kLinSpan || d->k * d->ldb * 2 > kLinSpan || d->m * d->lddz * 2 > kLinSpan)
    return OVL_EUNSUPPORTED;
  return OVL_OK;
}

// Rows that go to the streaming kernel: as many as two blocks of the matrix
// instruction's columns.  It reads a weight once for all of them.
constexpr int64_t kLinRows = 32;

using LinRow1 = RowCfg<false, false, 1, 1, 2, 36 * 1024>;
using LinRow2 = RowCfg<false, false, 1, 2, 2, 36 * 1024>;

struct LinRowShape {
  int32_t tiles, splits, steps, split_steps;
  size_t bytes;
};

LinRowShape row_shape(const gemm_epilogue_desc& d) {
  LinRowShape s = {};
  s.tiles = (int32_t)ceil_div(d.n, LinRow1::COLS);
  s.steps = (int32_t)ceil_div(d.k, 32);
  int64_t sp = std::min<int64_t>({kLinMaxSplits, kLinCus / s.tiles, s.steps / 8});
  sp = std::max<int64_t>(sp, 1);
  s.split_steps = (int32_t)ceil_div(s.steps, sp);
  s.splits = (int32_t)ceil_div(s.steps, s.split_steps);
  s.bytes = kCounterBytes + (s.splits > 1 ? aligned_up((size_t)(s.splits * d.m * d.n) * 4, 256) : 0);
  return s;
}

template <class C>
ovl_status row_launch(const LinRowArgs& a, hipStream_t stream) {
  ovl_status st = allow_lds(reinterpret_cast<const void*>(&lin_row_kernel<C>), C::LDS);
  if (st) return st;
  hipLaunchKernelGGL((lin_row_kernel<C>), dim3(a.tiles * a.splits), dim3(kThreads), C::LDS, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  return OVL_OK;
}

LinShape fwd_shape(const gemm_epilogue_desc& d) {
  const int64_t mnk[1][3] = {{d.m, d.n, d.k}};
  return lin_shape(mnk, 1, 0, 0);
}
LinShape grad_shape(const gemm_epilogue_grad_desc& d) {
  const int64_t mnk[2][3] = {{d.k, d.n, d.m}, {d.m, d.k, d.n}};
  return lin_shape(mnk, 2, d.m, d.n);
}

}  // namespace

}  // namespace ovl

using namespace ovl;

extern "C" size_t gemm_epilogue_workspace_bytes(const gemm_epilogue_desc* desc) {
  if (!desc) return 0;
  gemm_epilogue_desc d = *desc;
  if (lin_fwd_desc(&d)) return 0;
  return d.m <= kLinRows ? row_shape(d).bytes : fwd_shape(d).bytes;
}

extern "C" ovl_status gemm_epilogue_run(const gemm_epilogue_desc* desc, const void* a, const void* b,
                                        const float* bias, const void* residual, void* out, void* z,
                                        void* workspace, hipStream_t stream) {
  if (!desc || !workspace) return OVL_EINVAL;
  gemm_epilogue_desc d = *desc;
  ovl_status st = lin_fwd_desc(&d);
  if (st) return st;
  if (!aligned16(workspace)) return OVL_EALIGN;
  if (d.m == 0) return OVL_OK;
  if (!a || !b || !out) return OVL_EINVAL;
  if (!aligned16(a) || !aligned16(b) || !aligned16(bias) || !aligned16(residual) || !aligned16(out) || !aligned16(z))
    return OVL_EALIGN;
  // In place only where each piece is read by the thread that writes it.
  if (residual == out && (d.res_type != d.out_type || d.ldr != d.ldo)) return OVL_EINVAL;
  const CallBuffer buffers[] = {{residual, false}, {out, true}, {z, true},        {a, false},
                                {b, false},        {bias, false}, {workspace, true}};
  if (begins_alike(buffers, {{0, 1}})) return OVL_EINVAL;
  Epilogue e = {};
  e.out = out;
  e.z_out = z;
  e.bias = bias;
  e.residual = residual;
  e.ld_out = d.ldo;
  e.ld_z = d.ldz;
  e.ld_res = d.ldr;
  e.out_type = d.out_type;
  e.res_type = d.res_type;
  e.act = d.act;
  if (d.m <= kLinRows) {
    const LinRowShape rs = row_shape(d);
    LinRowArgs r = {};
    r.o.w = b;
    r.o.ldw = d.ldb;
    r.o.w_bytes = ((d.k - 1) * d.ldb + d.n) * 2;
    r.o.cols = d.n;
    r.o.x = static_cast<const uint16_t*>(a);
    r.o.x_bytes = ((d.m - 1) * d.lda + d.k) * 2;
    r.o.ldx = d.lda;
    r.o.k = d.k;
    r.epi = e;
    r.counters = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + OVL_ERROR_RECORD_BYTES);
    r.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
    r.m = d.m;
    r.n = d.n;
    r.tiles = rs.tiles;
    r.splits = rs.splits;
    r.steps = rs.steps;
    r.split_steps = rs.split_steps;
    return d.m <= 16 ? row_launch<LinRow1>(r, stream) : row_launch<LinRow2>(r, stream);
  }
  const LinShape s = fwd_shape(d);
  LinArgs args = {};
  args.job[0] = lin_job(s, 0, {static_cast<const uint16_t*>(a), d.lda, d.m, d.k},
                        {static_cast<const uint16_t*>(b), d.ldb, d.n, d.k}, e, workspace);
  args.sum.splits = 1;
  if (s.tile_m == 64) return lin_fwd_launch<Fwd64>(args, stream);
  return s.tile_m == 256 ? lin_fwd_launch<Fwd256>(args, stream) : lin_fwd_launch<Fwd128>(args, stream);
}

extern "C" size_t gemm_epilogue_grad_workspace_bytes(const gemm_epilogue_grad_desc* desc) {
  if (!desc) return 0;
  gemm_epilogue_grad_desc d = *desc;
  if (lin_grad_desc(&d)) return 0;
  return grad_shape(d).bytes;
}

extern "C" ovl_status gemm_epilogue_grad_run(const gemm_epilogue_grad_desc* desc, const void* dy, const void* z,
                                             void* dz, const void* a, const void* b, const void* z_in, void* da,
                                             void* db, const void* db_in, float* dbias, const float* dbias_in,
                                             void* workspace, hipStream_t stream) {
  if (!desc || !workspace) return OVL_EINVAL;
  gemm_epilogue_grad_desc d = *desc;
  ovl_status st = lin_grad_desc(&d);
  if (st) return st;
  const bool dact = d.act != OVL_ACT_NONE;
  if (!aligned16(workspace)) return OVL_EALIGN;
  if ((db_in && !db) || (dbias_in && !dbias)) return OVL_EINVAL;
  if (d.m) {
    if (!dz || (dact && (!dy || !z)) || (!dact && (dy || z))) return OVL_EINVAL;
    if (da && !b) return OVL_EINVAL;
    if (db && !a) return OVL_EINVAL;
    if (da && (d.act_in != OVL_ACT_NONE) != (z_in != nullptr)) return OVL_EINVAL;
  }
  for (const void* p : {dy, z, static_cast<const void*>(dz), a, b, z_in, static_cast<const void*>(da),
                        static_cast<const void*>(db), db_in, static_cast<const void*>(dbias),
                        static_cast<const void*>(dbias_in)})
    if (!aligned16(p)) return OVL_EALIGN;
  // (Without rows only db and dbias are written, and what they add is read; z_in
  // is read for da alone.)
  const auto rows = [&](const void* p) { return d.m ? p : nullptr; };
  const CallBuffer buffers[] = {{rows(dy), false}, {rows(z), false}, {rows(dz), dact},  {rows(da ? z_in : nullptr), false},
                                {rows(da), true},  {db_in, false},   {db, true},        {dbias_in, false},
                                {dbias, true},     {rows(a), false}, {rows(b), false},  {workspace, true}};
  if (begins_alike(buffers, {{0, 2}, {1, 2}, {3, 4}, {5, 6}, {7, 8}})) return OVL_EINVAL;
  if (d.m) {
    // In place only where each piece is read by the thread that writes it.
    if (dact && ((dz == dy && (d.dy_type != OVL_BF16 || d.lddy != d.lddz)) || (dz == z && d.ldz != d.lddz)))
      return OVL_EINVAL;
    if (da && da == z_in && (d.da_type != OVL_BF16 || d.ldda != d.ldz_in)) return OVL_EINVAL;
  }
  if (dact && d.m) {
    LinDactArgs g = {dy, static_cast<const uint16_t*>(z), static_cast<uint16_t*>(dz), d.lddy, d.ldz, d.lddz,
                     d.m, d.n, d.dy_type, d.act};
    const int64_t pieces = d.m * (d.n / 8);
    hipLaunchKernelGGL(lin_dact_kernel, dim3((uint32_t)std::min<int64_t>(2048, ceil_div(pieces, kThreads))),
                       dim3(kThreads), 0, stream, g);
    OVL_HIP_TRY(hipGetLastError());
  }
  const LinShape s = grad_shape(d);
  const uint16_t *pz = static_cast<const uint16_t*>(dz), *pa = static_cast<const uint16_t*>(a),
                 *pb = static_cast<const uint16_t*>(b);
  LinArgs args = {};
  if (db) {
    Epilogue e = {};
    e.out = db;
    e.residual = db_in;
    e.ld_out = e.ld_res = d.lddb;
    e.out_type = e.res_type = d.db_type;
    args.job[0] = lin_job(s, 0, {pa, d.lda, d.k, d.m}, {pz, d.lddz, d.n, d.m}, e, workspace);
  }
  if (da && d.m) {
    Epilogue e = {};
    e.out = da;
    e.z_in = d.act_in != OVL_ACT_NONE ? z_in : nullptr;
    e.ld_out = d.ldda;
    e.ld_z = d.ldz_in;
    e.out_type = d.da_type;
    e.act = d.act_in;
    args.job[1] = lin_job(s, 1, {pz, d.lddz, d.m, d.n}, {pb, d.ldb, d.k, d.n}, e, workspace);
  }
  args.sum.splits = 1;
  if (dbias) {
    LinSum& u = args.sum;
    u.dz = pz;
    u.in = dbias_in;
    u.out = dbias;
    u.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.sum_off);
    u.ld = d.lddz;
    u.m = d.m;
    u.n = d.n;
    u.splits = s.sum_splits;
    u.rows = ceil_div(d.m, u.splits);
    u.strips = (int32_t)ceil_div(d.n, 64);
    u.items = u.strips * u.splits;
  }
  if (s.tile_m == 64) return lin_grad_launch<Db64, Da64>(args, stream);
  return s.tile_m == 256 ? lin_grad_launch<Db256, Da256>(args, stream) : lin_grad_launch<Db128, Da128>(args, stream);
}

// A few rows times a streamed weight: y[r][c] = sum_k x[r][k] w[k][c] for at
// most 16 * NB rows, 64 columns (PAIR: and 64 more, `pair` columns further
// on) and a range of k, by one workgroup of four wavefronts.
//
// Every weight is read once and used for few rows, so the bound is HBM: what
// counts is bytes in flight.  The wavefronts split the range of k and share
// nothing while they stream: each has its own LDS ring of D steps, filled by
// buffer loads that write LDS directly, and waits on its own load counter
// only (no barrier in the loop).  The weight is the matrix instruction's A
// operand and the rows its B operand (v_mfma_f32_16x16x32_bf16: 16 columns x
// 16 rows, k 32 at a time), which leaves the matrix units nearly idle and
// the vector units out of the loop:
//   bf16 weights [k][n]: steps of 32 k; LDS rows of 64 columns, fragments by
//     the transposing read ds_read_b64_tr_b16;
//   E4M3 weights [n][k]: steps of 64 k; LDS rows of 64 codes, 16 codes a
//     lane, widened to bf16 (exact) in front of the matrix instruction.  A
//     lane group's 16 codes serve two instructions of 8 k each; the rows'
//     fragments take the same k.
// PL: x comes as that many bf16 planes whose sum is the value, each
// multiplied on its own (a float32 h as 2 or 3 planes: 16 or 24 bits).
// LDS rows are XOR-permuted in 16-byte chunks, as in gemm_core.h.
#pragma once

#include "device.h"
#include "gemm_core.h"

namespace ovl {

constexpr int kRowWaves = 4;
constexpr int kRowCols = 64;

template <bool FP8_, bool PAIR_, int PL_, int NB_>
struct RowCfg {
  static constexpr bool FP8 = FP8_, PAIR = PAIR_;
  static constexpr int PL = PL_, NB = NB_;
  static constexpr int KS = FP8 ? 64 : 32;             // k of a step
  static constexpr int WT = PAIR ? 2 : 1;              // weight tiles of a step
  static constexpr int XB = 16 * KS * 2;               // bytes of a step's 16 rows
  static constexpr int XQ = XB / 1024;                 // load instructions of them
  static constexpr int LPS = 4 * WT + XQ * PL * NB;    // load instructions of a step
  static constexpr int STEP = LPS * 1024;
  static constexpr int D = 20 * 1024 / STEP >= 2 ? 20 * 1024 / STEP : 2;  // steps in the ring
  static constexpr int WAVE_LDS = D * STEP;
  static constexpr int SUMS = kRowWaves * WT * 16 * NB * (kRowCols + 4) * 4;  // the waves' sums, staged over the rings
  static constexpr int LDS = kRowWaves * WAVE_LDS > SUMS ? kRowWaves * WAVE_LDS : SUMS;
  static_assert((D - 1) * LPS <= 63, "the load counter holds 63 loads");
};

struct RowOperands {
  const void* w;     // this expert's weight: bf16 [k][ldw] or codes [n][ldw]
  int64_t ldw;       // elements between its memory rows
  int64_t w_bytes;   // of the weight, from w on
  int64_t col0;      // first column
  int64_t cols;      // columns that exist (of either half)
  int64_t pair;      // PAIR: the second tile's columns are col0 + pair ..
  const uint16_t* x; // rows, plane by plane
  int64_t x_bytes;
  int64_t ldx;       // elements between rows
  int64_t plane;     // elements between planes
  int64_t k;         // contraction length
};

template <class C>
struct RowLoads {
  u32x4 sw[C::WT], sx;
  uint32_t w_off[4];            // this lane's offsets at k = 0, or kOOB
  uint32_t w_k;                 // FP8: the lane's first k in a step
  uint32_t x_off[C::NB * C::XQ];
  uint32_t x_k[C::XQ];
  uint32_t w_step, plane_b;
  int32_t k;

  // rows: LDS table of 16 * NB row numbers, -1 for none.
  __device__ inline void init(const RowOperands& o, const int32_t* rows) {
    const uint32_t l = lane_id();
    k = (int32_t)o.k;
    plane_b = (uint32_t)(o.plane * 2);
    sx = make_srd(o.x, o.x_bytes);
#pragma unroll
    for (int t = 0; t < C::WT; ++t) {
      const int64_t c = o.col0 + t * o.pair;
      const int64_t skip = C::FP8 ? c * o.ldw : c * 2;
      sw[t] = make_srd(static_cast<const uint8_t*>(o.w) + skip, o.w_bytes - skip);
    }
    if constexpr (C::FP8) {
      w_step = C::KS;
      w_k = ((l & 3) ^ ((l >> 3) & 3)) * 16;  // row l/4 of an instruction's 16; chunk (l%4) ^ (row/2 % 4)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t row = q * 16 + l / 4;
        w_off[q] = o.col0 + row < o.cols ? (uint32_t)(row * o.ldw) + w_k : kOOB;
      }
    } else {
      w_step = (uint32_t)(C::KS * o.ldw * 2);
      w_k = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t row = q * 8 + l / 8, c = (l & 7) ^ swz_w(row);
        w_off[q] = o.col0 + c * 8 < o.cols ? row * (uint32_t)(o.ldw * 2) + c * 16 : kOOB;
      }
    }
#pragma unroll
    for (int q = 0; q < C::XQ; ++q) {
      const uint32_t row = C::FP8 ? q * 8 + l / 8 : l / 4;
      const uint32_t c = C::FP8 ? (l & 7) ^ (row & 7) : (l & 3) ^ ((row >> 1) & 3);
      x_k[q] = c * 8;
#pragma unroll
      for (int b = 0; b < C::NB; ++b) {
        const int32_t r = rows[b * 16 + row];
        x_off[b * C::XQ + q] = r >= 0 ? (uint32_t)(r * o.ldx * 2) + c * 16 : kOOB;
      }
    }
  }
  static __device__ inline uint32_t swz_w(uint32_t row) { return 2 * ((row & 3) ^ ((row >> 3) & 1)); }

  // Loads of the step at k0 into `slot` (LDS address): weight tiles, then the
  // rows plane by plane.
  __device__ inline void issue(uint32_t slot, int32_t k0) const {
#pragma unroll
    for (int t = 0; t < C::WT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t o = w_off[q] + (uint32_t)(k0 / C::KS) * w_step;
        if constexpr (C::FP8) o = k0 + (int32_t)w_k < k ? o : kOOB;
        load_to_lds(sw[t], slot + (t * 4 + q) * 1024, o);
      }
#pragma unroll
    for (int p = 0; p < C::PL; ++p)
#pragma unroll
      for (int i = 0; i < C::NB * C::XQ; ++i) {
        const uint32_t o = k0 + (int32_t)x_k[i % C::XQ] < k ? x_off[i] + p * plane_b + (uint32_t)k0 * 2 : kOOB;
        load_to_lds(sx, slot + (C::WT * 4 + p * C::NB * C::XQ + i) * 1024, o);
      }
  }
};

template <class C>
struct RowAcc {
  f32x4 v[C::WT][4][C::NB];  // [tile][16 columns][16 rows]: lane l holds row l%16, columns 4*(l/16) ..+3
};

// Eight E4M3 codes (two words) widened to bf16.
__device__ inline bf16x8 fp8_to_bf16(uint32_t a, uint32_t b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  bf16x8 r;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t c = w ? b : a;
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    r[4 * w] = (__bf16)lo[0];
    r[4 * w + 1] = (__bf16)lo[1];
    r[4 * w + 2] = (__bf16)hi[0];
    r[4 * w + 3] = (__bf16)hi[1];
  }
  return r;
}

template <class C>
__device__ inline void row_step(RowAcc<C>& acc, const uint8_t* slot) {
  const uint32_t l = lane_id(), g = l >> 4, r = l & 15;
  const uint8_t* xs = slot + C::WT * 4096;
  if constexpr (C::FP8) {
    bf16x8 x[C::PL][C::NB][2];
#pragma unroll
    for (int p = 0; p < C::PL; ++p)
#pragma unroll
      for (int b = 0; b < C::NB; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          x[p][b][s] = *OVL_LDS(const bf16x8, xs + (p * C::NB + b) * C::XB + r * 128 + (((2 * g + s) ^ (r & 7)) * 16));
#pragma unroll
    for (int t = 0; t < C::WT; ++t)
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) {
        const uint32_t row = cb * 16 + r;
        const u32x4 q = *OVL_LDS(const u32x4, slot + t * 4096 + row * 64 + ((g ^ ((row >> 1) & 3)) * 16));
        const bf16x8 w0 = fp8_to_bf16(q[0], q[1]), w1 = fp8_to_bf16(q[2], q[3]);
#pragma unroll
        for (int p = 0; p < C::PL; ++p)
#pragma unroll
          for (int b = 0; b < C::NB; ++b) {
            acc.v[t][cb][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, x[p][b][0], acc.v[t][cb][b], 0, 0, 0);
            acc.v[t][cb][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, x[p][b][1], acc.v[t][cb][b], 0, 0, 0);
          }
      }
  } else {
    bf16x8 x[C::PL][C::NB];
#pragma unroll
    for (int p = 0; p < C::PL; ++p)
#pragma unroll
      for (int b = 0; b < C::NB; ++b)
        x[p][b] = *OVL_LDS(const bf16x8, xs + (p * C::NB + b) * C::XB + r * 64 + ((g ^ ((r >> 1) & 3)) * 16));
    const uint32_t row = g * 8 + (r >> 2);
#pragma unroll
    for (int t = 0; t < C::WT; ++t)
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) {
        const uint32_t chunk = (cb * 2 + ((r & 3) >> 1)) ^ RowLoads<C>::swz_w(row);
        const uint8_t* p = slot + t * 4096 + row * 128 + chunk * 16 + (r & 1) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OVL_LDS(s16x4, p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OVL_LDS(s16x4, p + 4 * 128));
        const bf16x8 w = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
        for (int q = 0; q < C::PL; ++q)
#pragma unroll
          for (int b = 0; b < C::NB; ++b)
            acc.v[t][cb][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[q][b], acc.v[t][cb][b], 0, 0, 0);
      }
  }
}

// Waits until at most `steps` steps' loads of this wave are in flight, and
// for its LDS reads (a slot is refilled right afterwards).
template <int LPS, int P>
__device__ inline void row_wait(int steps) {
  if constexpr (P == 0) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  } else {
    if (steps >= P)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(P * LPS) : "memory");
    else
      row_wait<LPS, P - 1>(steps);
  }
}

// The sums over steps [s0, s1) of KS, all four wavefronts' together, staged
// in LDS: sums[tile][row][64 + 4], in every thread's sight when it returns.
// Every sum is made of the waves' in wave order, each in k order.  `rows` is
// an LDS table outside the ring; the ring must be free.
template <class C>
__device__ inline const float* row_product(const RowOperands& o, const int32_t* rows, int32_t s0, int32_t s1,
                                           uint8_t* lds) {
  const int wave = uniform((int)(threadIdx.x >> 6));
  RowAcc<C> acc;
#pragma unroll
  for (int t = 0; t < C::WT; ++t)
#pragma unroll
    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
      for (int b = 0; b < C::NB; ++b) acc.v[t][cb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  RowLoads<C> ld;
  ld.init(o, rows);
  const int32_t per = (s1 - s0 + kRowWaves - 1) / kRowWaves;
  const int32_t b = min(s0 + wave * per, s1), n = min(b + per, s1) - b;
  uint8_t* ring = lds + wave * C::WAVE_LDS;
  const uint32_t ring_a = lds_addr(ring);
  wave_drain();
  for (int32_t i = 0; i < C::D - 1 && i < n; ++i) ld.issue(ring_a + i * C::STEP, (b + i) * C::KS);
  row_wait<C::LPS, C::D - 2>(max(0, min(C::D - 2, n - 1)));
  int32_t slot = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t nxt = i + C::D - 1;
    const int32_t nslot = slot ? slot - 1 : C::D - 1;
    if (nxt < n) ld.issue(ring_a + nslot * C::STEP, (b + nxt) * C::KS);
    row_step<C>(acc, ring + slot * C::STEP);
    row_wait<C::LPS, C::D - 2>(max(0, min(nxt, n - 1) - (i + 1)));
    slot = slot + 1 == C::D ? 0 : slot + 1;
  }
  wave_drain();
  __syncthreads();  // every wave's ring is done with
  constexpr int P = kRowCols + 4, TILE = 16 * C::NB * P, ALL = C::WT * TILE;
  float* st = reinterpret_cast<float*>(lds);
  {
    const uint32_t l = lane_id();
#pragma unroll
    for (int t = 0; t < C::WT; ++t)
#pragma unroll
      for (int cb = 0; cb < 4; ++cb)
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb)
          *OVL_LDS(f32x4, st + wave * ALL + t * TILE + (nb * 16 + (l & 15)) * P + cb * 16 + 4 * (l >> 4)) =
              acc.v[t][cb][nb];
  }
  __syncthreads();
  for (int i = threadIdx.x * 4; i < ALL; i += kThreads * 4) {
    f32x4 v = *OVL_LDS(const f32x4, st + i);
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) v += *OVL_LDS(const f32x4, st + w * ALL + i);
    *OVL_LDS(f32x4, st + i) = v;
  }
  __syncthreads();
  return st;
}

// Eight sums of a staged tile.
template <class C>
__device__ inline void row_sums8(float (&v)[8], const float* st, int tile, int row, int col) {
  const float* p = st + (tile * 16 * C::NB + row) * (kRowCols + 4) + col;
  const f32x4 a = *OVL_LDS(const f32x4, p), b = *OVL_LDS(const f32x4, p + 4);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    v[c] = a[c];
    v[4 + c] = b[c];
  }
}

// Partial sums for a workgroup on another die: agent-scope stores, so that a
// drain, a barrier and a relaxed add publish them.
__device__ inline void store8_agent(const float (&v)[8], float* p) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st8_agent(reinterpret_cast<uint64_t*>(p) + c,
              (uint64_t)__builtin_bit_cast(uint32_t, v[2 * c]) | (uint64_t)__builtin_bit_cast(uint32_t, v[2 * c + 1]) << 32);
}

// Arrival at a counter of `expected` workgroups: true, in every thread, for
// the last one, which has acquired the others' stores and returned the
// counter to zero.
__device__ inline bool row_arrive_last(int32_t* counter, int expected, int32_t* lds_flag) {
  wave_drain();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int old = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *lds_flag = old + 1 == expected;
    if (old + 1 == expected) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  const bool last = uniform(*lds_flag);
  if (last) wave_acquire();
  return last;
}

}  // namespace ovl

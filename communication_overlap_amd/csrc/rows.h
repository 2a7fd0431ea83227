// A few rows times a streamed weight: y[r][c] = sum_k x[r][k] w[k][c] for at
// most ROWS rows, COLS columns (PAIR: and as many more, `pair` columns
// further on) and a range of k, by one workgroup of four wavefronts.
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
//   E4M3 weights [n][k]: steps of 128 k; LDS rows of 128 codes, 32 columns,
//     widened to bf16 (exact) in front of the matrix instruction.  A lane
//     reads 16 codes at a time, which serve two instructions of 8 k each; the
//     rows' fragments take the same k.
// Either way every row of the weight is read in whole 128-byte lines by one
// instruction: with steps of 64 codes, half a line each, the experts' launch
// streamed at 4.1 TB/s, with the next step's half just behind it.
// PL: x comes as that many bf16 planes whose sum is the value, each
// multiplied on its own (a float32 h as 3 planes: 24 bits).
// LDS rows are XOR-permuted in 16-byte chunks, as in gemm_core.h.
#pragma once

#include "device.h"
#include "gemm_core.h"

namespace ovl {

constexpr int kRowWaves = 4;
// AD: tiles of TC columns side by side.  XR: rows of x that a step holds, 16
// or, for codes, 4 or 8 (the matrix instruction's other columns then repeat
// them, and are not looked at).  RING: LDS bytes of a wavefront's ring, as
// deep as one workgroup a compute unit allows: two workgroups with 19 KiB
// rings took 48 us against 41 for the experts of one token.
template <bool FP8_, bool PAIR_, int PL_, int NB_, int AD_, int RING, int XR_ = 16>
struct RowCfg {
  static constexpr bool FP8 = FP8_, PAIR = PAIR_;
  static constexpr int PL = PL_, NB = NB_, AD = AD_;
  static constexpr int XR = XR_;
  static constexpr int ROWS = XR == 16 ? 16 * NB : XR;  // rows of a unit
  static constexpr int TC = FP8 ? 32 : 64;             // columns of a tile
  static constexpr int COLS = TC * AD;                 // columns of a workgroup (PAIR: of either half)
  static constexpr int PIECES = ROWS * COLS / 8;       // 8-column pieces of its rows
  static constexpr int KS = FP8 ? 128 : 32;            // k of a step
  static constexpr int WT = PAIR ? 2 * AD : AD;        // weight tiles of a step
  static constexpr int BLOCKS = WT * TC / 16;          // 16-column blocks of a step
  static constexpr int XB = XR * KS * 2;               // bytes of a step's block of rows
  static constexpr int XQ = XB / 1024;                 // load instructions of it
  static constexpr int LPS = 4 * WT + XQ * PL * NB;    // load instructions of a step
  static constexpr int STEP = LPS * 1024;
  static_assert(XB % 1024 == 0 && (XR == 16 || (XR <= 8 && NB == 1)), "whole load instructions");
  static_assert(BLOCKS % kRowWaves == 0, "the blocks divide over the waves");
  static constexpr int D = RING / STEP >= 2 ? RING / STEP : 2;  // steps in the ring
  static constexpr int WAVE_LDS = D * STEP;
  static constexpr int PITCH = TC + 4;                 // floats of a staged row
  static constexpr int LDS = kRowWaves * WAVE_LDS + WT * 16 * NB * PITCH * 4;  // the rings, then the staged sums
  static_assert((D - 1) * LPS <= 63, "the load counter holds 63 loads");
  static_assert(D * STEP <= RING, "the ring holds two steps");
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
  uint32_t w_off[C::AD][4];     // this lane's offsets at k = 0, or kOOB
  uint32_t w_k;                 // FP8: the lane's first k in a step
  uint32_t x_off[C::NB * C::XQ];
  uint32_t x_k[C::XQ];
  uint32_t w_step, plane_b;
  int32_t k;

  // rows: LDS table of ROWS numbers, -1 for none; number / div is the row.
  __device__ inline void init(const RowOperands& o, const int32_t* rows, int32_t div = 1) {
    const uint32_t l = lane_id();
    k = (int32_t)o.k;
    plane_b = (uint32_t)(o.plane * 2);
    sx = make_srd(o.x, o.x_bytes);
#pragma unroll
    for (int t = 0; t < C::WT; ++t) {
      const int64_t c = o.col0 + t / C::AD * o.pair + t % C::AD * C::TC;
      const int64_t skip = C::FP8 ? c * o.ldw : c * 2;
      sw[t] = make_srd(static_cast<const uint8_t*>(o.w) + skip, o.w_bytes - skip);
    }
    if constexpr (C::FP8) {
      w_step = C::KS;
      w_k = ((l & 7) ^ (l >> 3)) * 16;  // row l/8 of an instruction's 8; chunk (l%8) ^ (row % 8)
#pragma unroll
      for (int t = 0; t < C::AD; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t row = q * 8 + l / 8;
          w_off[t][q] = o.col0 + t * C::TC + row < o.cols ? (uint32_t)(row * o.ldw) + w_k : kOOB;
        }
    } else {
      w_step = (uint32_t)(C::KS * o.ldw * 2);
      w_k = 0;
#pragma unroll
      for (int t = 0; t < C::AD; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t row = q * 8 + l / 8, c = (l & 7) ^ swz_w(row);
          w_off[t][q] = o.col0 + t * C::TC + c * 8 < o.cols ? row * (uint32_t)(o.ldw * 2) + c * 16 : kOOB;
        }
    }
#pragma unroll
    for (int q = 0; q < C::XQ; ++q) {
      const uint32_t row = C::FP8 ? q * 4 + l / 16 : l / 4;
      const uint32_t c = C::FP8 ? (l & 15) ^ (row & 15) : (l & 3) ^ ((row >> 1) & 3);
      x_k[q] = c * 8;
#pragma unroll
      for (int b = 0; b < C::NB; ++b) {
        const int32_t r = *OVL_LDS(const int32_t, rows + b * 16 + row);
        x_off[b * C::XQ + q] = r >= 0 ? (uint32_t)(r / div * o.ldx * 2) + c * 16 : kOOB;
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
        uint32_t o = w_off[t % C::AD][q] + (uint32_t)(k0 / C::KS) * w_step;
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
  f32x4 v[C::BLOCKS][C::NB];  // [16 columns][16 rows]: lane l holds row l%16, columns 4*(l/16) ..+3
};

// Eight E4M3 codes (two words) widened to bf16, which holds them exactly.
__device__ inline bf16x8 fp8_to_bf16(uint32_t a, uint32_t b) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false);
  const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true);
  const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false);
  const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

template <class C>
__device__ inline void row_step(RowAcc<C>& acc, const uint8_t* slot) {
  const uint32_t l = lane_id(), g = l >> 4, r = l & 15;
  const uint8_t* xs = slot + C::WT * 4096;
  if constexpr (C::FP8) {
    const uint32_t xr = r % C::XR;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 64 codes at a time: lane group g holds k = 64 h + 16 g ..+15
      bf16x8 x[C::PL][C::NB][2];
#pragma unroll
      for (int p = 0; p < C::PL; ++p)
#pragma unroll
        for (int b = 0; b < C::NB; ++b)
#pragma unroll
          for (int s = 0; s < 2; ++s)
            x[p][b][s] = *OVL_LDS(const bf16x8, xs + (p * C::NB + b) * C::XB + xr * 256 +
                                                    (((8 * h + 2 * g + s) ^ xr) * 16));
#pragma unroll
      for (int t = 0; t < C::WT; ++t)
#pragma unroll
        for (int cb = 0; cb < 2; ++cb) {
          const uint32_t row = cb * 16 + r;
          const u32x4 q = *OVL_LDS(const u32x4, slot + t * 4096 + row * 128 + (((4 * h + g) ^ (row & 7)) * 16));
          const bf16x8 w0 = fp8_to_bf16(q[0], q[1]), w1 = fp8_to_bf16(q[2], q[3]);
#pragma unroll
          for (int p = 0; p < C::PL; ++p)
#pragma unroll
            for (int b = 0; b < C::NB; ++b) {
              f32x4& v = acc.v[t * 2 + cb][b];
              v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, x[p][b][0], v, 0, 0, 0);
              v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, x[p][b][1], v, 0, 0, 0);
            }
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
            acc.v[t * 4 + cb][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[q][b], acc.v[t * 4 + cb][b], 0, 0, 0);
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

// Streams the workgroup's units one after the other, a unit being one set of
// rows x columns x range of k.  The loads run ahead of the products by the
// ring's depth, across the end of a unit: while one unit's sums are added up
// and stored, the next one's weights are on their way.
//   gen.begin(u, ld, s0, s1): sets up the loads of unit u and its range of
//     steps; false when there is no such unit.  No global loads in it: it runs
//     inside the product loop, where a wait would empty the ring.
//     It is called at most one unit ahead of done().
//   gen.range(u, s0, s1): the range alone.
//   gen.turn(n): the step, of the range's n, that unit u begins with (the last
//     begun unit's).  Codes' rows of 128-byte pieces lie far apart, and units
//     that start alike crowd the same memory channels (9 tokens of FP8 experts:
//     104 us with units begun at different steps, 109 without).
//   done(u, sums): unit u's sums of all four wavefronts, staged in LDS as
//     sums[tile][row][TC + 4], in every thread's sight.  A path of it that
//     loads from global memory ends with wave_drain(): a load of which the
//     compiler cannot tell that it has landed would make it wait in the product
//     loop.
// Every sum is made of the waves' in an order fixed by its columns, each
// wave's in k order.
template <class C, class Gen, class Done>
__device__ inline void row_stream(Gen& gen, uint8_t* lds, Done done) {
  const int wave = uniform((int)(threadIdx.x >> 6));
  // The waves take steps in turn, so that the workgroup reads its range front
  // to back.
  const auto steps_of = [&](int32_t s0, int32_t s1) {
    return max(0, s1 - s0 - wave + kRowWaves - 1) / kRowWaves;
  };
  RowLoads<C> ld;
  const uint8_t* ring = lds + wave * C::WAVE_LDS;
  const uint32_t ring_a = lds_addr(ring);
  float* st = reinterpret_cast<float*>(lds + kRowWaves * C::WAVE_LDS);
  // The unit being loaded, its next step and how many this wave has of it.
  int32_t lu = 0, li = 0, ln = 0, l0 = 0, l1 = 0, turn = 0;
  bool more = gen.begin(0, ld, l0, l1);
  if (more) {
    ln = steps_of(l0, l1);
    turn = gen.turn(l1 - l0);
  }
  int32_t islot = 0, uslot = 0, ahead = 0;  // ahead: steps issued and not yet used
  int32_t u = 0;                            // the unit being added up
  const auto issue_next = [&]() {
    while (more && li == ln && lu <= u) {   // at most one unit ahead
      more = gen.begin(++lu, ld, l0, l1);
      li = 0;
      ln = more ? steps_of(l0, l1) : 0;
      turn = more ? gen.turn(l1 - l0) : 0;
    }
    if (!more || li == ln) return;
    int32_t at = wave + li * kRowWaves + turn;  // the range's steps from `turn` on, and round
    if (at >= l1 - l0) at -= l1 - l0;
    ld.issue(ring_a + islot * C::STEP, (l0 + at) * C::KS);
    islot = islot + 1 == C::D ? 0 : islot + 1;
    ++li;
    ++ahead;
  };
  wave_drain();
  int32_t s0, s1;
  for (; gen.range(u, s0, s1); ++u) {
    // Fill the ring and have the first step there; then every step of the
    // loop refills the slot used last and waits for the next one.
    for (int i = ahead; i < C::D - 1; ++i) issue_next();
    row_wait<C::LPS, C::D - 2>(min(C::D - 2, max(0, ahead - 1)));
    RowAcc<C> acc;
#pragma unroll
    for (int k = 0; k < C::BLOCKS; ++k)
#pragma unroll
      for (int b = 0; b < C::NB; ++b) acc.v[k][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int32_t n = steps_of(s0, s1);
    for (int32_t i = 0; i < n; ++i) {
      issue_next();
      row_step<C>(acc, ring + uslot * C::STEP);
      uslot = uslot + 1 == C::D ? 0 : uslot + 1;
      --ahead;
      row_wait<C::LPS, C::D - 2>(max(0, ahead - 1));
    }
    // Four rounds: in round r wave w puts in (round 0) or adds its blocks k
    // with k = w + r mod 4.
    __syncthreads();  // the staged sums of the unit before are done with
    const uint32_t l = lane_id();
#pragma unroll
    for (int r = 0; r < kRowWaves; ++r) {
#pragma unroll
      for (int k = 0; k < C::BLOCKS; ++k)
        if (((k - r) & 3) == wave) {
          constexpr int PB = C::TC / 16;  // blocks of a tile
#pragma unroll
          for (int b = 0; b < C::NB; ++b) {
            float* p = st + (k / PB * 16 * C::NB + b * 16 + (l & 15)) * C::PITCH + k % PB * 16 + 4 * (l >> 4);
            f32x4 v = acc.v[k][b];
            if (r) v += *OVL_LDS(const f32x4, p);
            *OVL_LDS(f32x4, p) = v;
          }
        }
      __syncthreads();
    }
    done(u, st);
  }
}

// Eight sums of a staged row, from column col (a multiple of 8) of half
// `half` (PAIR: 0 or 1).
template <class C>
__device__ inline void row_sums8(float (&v)[8], const float* st, int half, int row, int col) {
  const float* p = st + ((half * C::AD + col / C::TC) * 16 * C::NB + row) * C::PITCH + col % C::TC;
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

// Partial products written by other workgroups of the launch (store8_agent):
// agent-scope loads need no acquire, which would empty the die's caches.
struct RowPart {
  uint64_t q[4];
};
__device__ inline RowPart load8_agent(const float* p) {
  RowPart r;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    r.q[c] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p) + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return r;
}
__device__ inline void add8(float (&v)[8], const RowPart& r) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    v[2 * c] += __builtin_bit_cast(float, (uint32_t)r.q[c]);
    v[2 * c + 1] += __builtin_bit_cast(float, (uint32_t)(r.q[c] >> 32));
  }
}

// Eight sums of `ranges` partial products, `stride` floats apart, added in
// range order; H such sets, `half` floats apart.  Eight ranges' loads of all
// sets go out together: the reader's time is the latency of its batches.
template <int H>
__device__ inline void row_ranges8(float (&v)[H][8], const float* p, int ranges, int64_t stride, int64_t half) {
  constexpr int U = 8;
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int c = 0; c < 8; ++c) v[h][c] = 0.f;
  for (int s = 0; s < ranges; s += U) {
    RowPart q[U][H];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (s + u < ranges) q[u][h] = load8_agent(p + (s + u) * stride + h * half);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (s + u < ranges) add8(v[h], q[u][h]);
  }
}

// Arrival at a counter of `expected` workgroups: true, in every thread, for
// the last one, which has returned the counter to zero and finds the others'
// agent-scope stores with agent-scope loads.
__device__ inline bool row_arrive_last(int32_t* counter, int expected, int32_t* lds_flag) {
  wave_drain();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int old = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *lds_flag = old + 1 == expected;
    if (old + 1 == expected) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return uniform(*lds_flag);
}

}  // namespace ovl

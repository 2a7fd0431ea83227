// bf16 x bf16 -> fp32 tile GEMM on gfx950 matrix cores with either operand
// in either orientation, for the products of a layer's forward and backward
// pass:
//   forward  C = A B          A K-contiguous [m][k], B K-strided [k][n];
//   grad     dA = dZ B^T      both K-contiguous ([m][n], [k][n]: contraction over n);
//   grad     dB = A^T dZ      both K-strided ([m][k], [m][n]: contraction over m).
// One workgroup of NW = 4 or 8 wavefronts computes a BM x BN tile in 32 x 32
// blocks (v_mfma_f32_32x32x16_bf16), the waves forming a 2 x (NW/2) grid.  K
// advances in steps of 64 through NS LDS stages filled NS - 1 steps ahead by
// buffer loads that write LDS directly: two stages of 64 KiB for 256 x 256
// tiles, which keep the matrix units busy over a step, two of 32 KiB for 128 x
// 128, and three of 24 KiB for 64 x 128 tiles of few, where a step is shorter
// than a load takes and two workgroups share a compute unit.
//   K-contiguous operand: LDS [row][64 k], 128 bytes a row; a fragment is one
//   ds_read_b128 (8 consecutive k of one row).
//   K-strided operand: LDS [k][rows], a fragment is two ds_read_b64_tr_b16
//   (each transposes 4 x 4 blocks of 16-bit elements across 16 lanes).
// Each LDS row's 16-byte chunks are XOR-permuted so that fragment reads meet
// no bank twice; the permutation is applied to the global address a lane
// fetches.  Rows, columns and k past the operand's end read as zero: the
// buffer resource ends at the last valid element, and chunks that would run
// on into the next row get an offset past every buffer.
//
// Every output element is summed in one fixed order: k ascending, 16 at a
// time.
//
// Large products are bound by the matrix units at the clock their power
// allows: 8192 x 3584 x 4096, both sums and epilogue, 236 us (1.02 PFLOP/s),
// 207 us (1.16) with a plain store; the library's product alone 197 us.
#pragma once

#include "device.h"
#include "gemm_core.h"

namespace ovl {

// One operand of a tile: `rows` output rows (or columns) that exist, `k`
// contraction length, `ld` elements between its memory rows.  KC: element
// (row, k) at p[row * ld + k]; else at p[k * ld + row].
struct AnyOperand {
  const uint16_t* p;
  int64_t ld;
  int64_t rows;
  int64_t k;
};

constexpr int kAnyBK = 64;

// Chunk permutation of row k of a K-strided operand's LDS rows of R columns: a
// fragment read takes 4 rows x 2 chunks per 16 lanes, rows 8 apart in
// neighbouring groups of lanes.
template <int R>
__device__ inline uint32_t any_swz(uint32_t k) {
  return R >= 128 ? swz_b(k) : 2 * ((k & 3) ^ ((k >> 3) & 1));
}

template <int R, int NW, bool KC>
struct AnySide {
  static constexpr int BYTES = R * kAnyBK * 2;              // of one stage
  static constexpr int Q = BYTES / 1024 / NW;               // load instructions per wave per stage
  static constexpr int LPR = KC ? 8 : R / 8;                // lanes per LDS row in one instruction
  static constexpr int RPI = 64 / LPR;                      // LDS rows per instruction
  static constexpr int PITCH = KC ? kAnyBK * 2 : R * 2;     // bytes of an LDS row
  static constexpr int PIECES = KC ? 1 : 2;                 // LDS reads per fragment
  static_assert(BYTES % (1024 * NW) == 0 && Q >= 1, "loads divide over the waves");

  u32x4 srd;
  uint32_t off[2];   // lane offset at k = 0 of instructions of even / odd index, or kOOB
  uint32_t qstep;    // bytes between consecutive instructions
  uint32_t kstep;    // bytes a K step of 64 advances
  int32_t kc[2];     // KC: the lane's first k in a step
  int32_t k;
  uint32_t lds;      // byte offset of this wave's first block within a stage

  static __device__ inline uint32_t swz(uint32_t r) { return KC ? swz_a<64>(r) : any_swz<R>(r); }

  __device__ inline void init(const AnyOperand& o, int64_t r0, uint32_t wave) {
    const uint32_t l = lane_id();
    const uint32_t ld_b = (uint32_t)(o.ld * 2);
    k = (int32_t)o.k;
    lds = wave * Q * 1024;
    qstep = RPI * ld_b;
    if constexpr (KC) {
      // The resource ends with the last valid row's last k.
      srd = make_srd(o.p + r0 * o.ld, ((o.rows - r0 - 1) * o.ld + o.k) * 2);
      kstep = kAnyBK * 2;
    } else {
      srd = make_srd(o.p + r0, ((o.k - 1) * o.ld + o.rows - r0) * 2);
      kstep = kAnyBK * ld_b;
    }
#pragma unroll
    for (uint32_t par = 0; par < 2; ++par) {
      const uint32_t row = (wave * Q + par) * RPI + l / LPR;
      const uint32_t c = (l % LPR) ^ swz(row);
      kc[par] = (int32_t)c * 8;
      off[par] = row * ld_b + c * 16;
      if (!KC && r0 + (int64_t)c * 8 >= o.rows) off[par] = kOOB;
    }
  }
  template <int I>
  __device__ inline void issue(uint32_t stage, int32_t step) const {
    constexpr int par = I & 1;
    uint32_t o = off[par] + (I & ~1) * qstep + (uint32_t)step * kstep;
    if constexpr (KC) o = step * kAnyBK + kc[par] < k ? o : kOOB;
    load_to_lds(srd, stage + lds + I * 1024, o);
  }
};

// Per-lane LDS offsets of a wave's fragments of one operand (F blocks of 32
// rows from row w0).
template <int R, int F, bool KC>
struct AnyFrag {
  uint32_t o[KC ? kAnyBK / 16 : F];
  __device__ inline void init(uint32_t w0) {
    const uint32_t l = lane_id();
    if constexpr (KC) {
      const uint32_t row = w0 + (l & 31);
#pragma unroll
      for (uint32_t kk = 0; kk < kAnyBK / 16; ++kk)
        o[kk] = row * (kAnyBK * 2) + (((2 * kk) | (l >> 5)) ^ swz_a<64>(row)) * 16;
    } else {
      // Group g of 16 lanes, source lane s: row (g/2)*8 + s/4 (and +4),
      // columns (g%2)*16 + 4*(s%4) .. +3 of the block.
      const uint32_t g = l >> 4, s = l & 15, brow = (g >> 1) * 8 + (s >> 2);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const uint32_t col = w0 + f * 32 + (g & 1) * 16 + 4 * (s & 3);
        o[f] = brow * (R * 2) + ((col >> 3) ^ any_swz<R>(brow)) * 16 + (col & 4) * 2;
      }
    }
  }
};

union AnyFragData {
  bf16x8 v;
  s16x4 h[2];
};

template <int R, int F, bool KC, int PIECE>
__device__ inline void any_read(AnyFragData* d, const uint8_t* area, const AnyFrag<R, F, KC>& fa, int kk) {
  if constexpr (KC) {
    d[PIECE].v = *OVL_LDS(const bf16x8, area + fa.o[kk] + PIECE * 32 * (kAnyBK * 2));
  } else {
    constexpr int f = PIECE / 2, hi = PIECE & 1;
    d[f].h[hi] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OVL_LDS(s16x4, area + fa.o[f] + (kk * 16 + hi * 4) * (R * 2)));
  }
}

template <int BM_, int BN_, int NW_, bool AKC_, bool BKC_, int NS_ = 2>
struct AnyTile {
  static constexpr int BM = BM_, BN = BN_, NW = NW_, NS = NS_;
  static constexpr bool AKC = AKC_, BKC = BKC_;
  static constexpr int WN = NW / 2;
  static constexpr int FM = BM / 64, FN = BN / (32 * WN);
  using SA = AnySide<BM, NW, AKC>;
  using SB = AnySide<BN, NW, BKC>;
  static constexpr int STAGE = SA::BYTES + SB::BYTES;
  static constexpr int LPS = SA::Q + SB::Q;  // load instructions per wave per stage
  static constexpr int LDS_BYTES = NS * STAGE;
  static constexpr int READS = SB::PIECES * FN + SA::PIECES * FM;  // LDS reads of one sub-step
  struct Acc {
    f32x16 v[FM][FN];
  };
  struct Frags {
    AnyFragData a[FM], b[FN];
  };
};

template <class T>
struct AnyLoop {
  typename T::SA sa;
  typename T::SB sb;
  AnyFrag<T::BM, T::FM, T::AKC> fa;
  AnyFrag<T::BN, T::FN, T::BKC> fb;

  // Reads [P0, P1) of sub-step kk's fragments: B's first, then A's.
  template <int P0, int P1>
  __device__ inline void read(typename T::Frags& f, const uint8_t* stage, int kk) const {
    if constexpr (P0 < P1) {
      constexpr int NB = T::SB::PIECES * T::FN;
      if constexpr (P0 < NB)
        any_read<T::BN, T::FN, T::BKC, P0>(f.b, stage + T::SA::BYTES, fb, kk);
      else
        any_read<T::BM, T::FM, T::AKC, P0 - NB>(f.a, stage, fa, kk);
      read<P0 + 1, P1>(f, stage, kk);
    }
  }
  template <int I, int N>
  __device__ inline void issue_a(uint32_t stage, int32_t step) const {
    if constexpr (I < N) {
      sa.template issue<I>(stage, step);
      issue_a<I + 1, N>(stage, step);
    }
  }
  template <int I, int N>
  __device__ inline void issue_b(uint32_t stage, int32_t step) const {
    if constexpr (I < N) {
      sb.template issue<I>(stage + T::SA::BYTES, step);
      issue_b<I + 1, N>(stage, step);
    }
  }
  // MFMA group G of a stage: the FN blocks of A fragment G % FM in sub-step
  // G / FM, the next sub-step's fragment reads spread between them, then a
  // burst of the next stage's loads: B's behind the first group, A's behind
  // the first of the second sub-step.
  template <int G>
  __device__ inline void group(typename T::Acc& acc, const typename T::Frags& cur, typename T::Frags& nxt,
                               const uint8_t* stage, uint32_t next_stage, int32_t next_step, bool load) const {
    constexpr int KKI = G / T::FM, fm = G % T::FM;
    constexpr int per = (T::READS + T::FM - 1) / T::FM;
    constexpr int r0 = fm * per < T::READS ? fm * per : T::READS;
    constexpr int r1 = (fm + 1) * per < T::READS ? (fm + 1) * per : T::READS;
    constexpr int rd = KKI < 3 ? r1 - r0 : 0;
#pragma unroll
    for (int fn = 0; fn < T::FN; ++fn)
      acc.v[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cur.a[fm].v, cur.b[fn].v, acc.v[fm][fn], 0, 0, 0);
    if constexpr (KKI < 3) read<r0, r1>(nxt, stage, KKI + 1);
#pragma unroll
    for (int i = 0; i < T::FN; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
      if (i < rd) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // DS read
    }
    OVL_SCHED_FENCE();
    if constexpr (G == 0)
      if (load) issue_b<0, T::SB::Q>(next_stage, next_step);
    if constexpr (G == T::FM)
      if (load) issue_a<0, T::SA::Q>(next_stage, next_step);
    OVL_SCHED_FENCE();
  }
  template <int G, int N>
  __device__ inline void groups(typename T::Acc& acc, const typename T::Frags& cur, typename T::Frags& nxt,
                                const uint8_t* stage, uint32_t next_stage, int32_t next_step, bool load) const {
    if constexpr (N > 0) {
      group<G>(acc, cur, nxt, stage, next_stage, next_step, load);
      groups<G + 1, N - 1>(acc, cur, nxt, stage, next_stage, next_step, load);
    }
  }
};

// The K loop of one tile over steps [s0, s1) of 64.  Ends with a workgroup
// barrier: LDS may be reused at once.
template <class T>
__device__ inline void any_tile(typename T::Acc& acc, const AnyOperand& a, const AnyOperand& b, int64_t m0,
                                int64_t n0, int32_t s0, int32_t s1, uint8_t* lds) {
#pragma unroll
  for (int fm = 0; fm < T::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < T::FN; ++fn)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc.v[fm][fn][r] = 0.f;
  const uint32_t wave = (uint32_t)uniform((int)(threadIdx.x >> 6));
  AnyLoop<T> lp;
  lp.sa.init(a, m0, wave);
  lp.sb.init(b, n0, wave);
  lp.fa.init((wave / T::WN) * (T::BM / 2));
  lp.fb.init((wave % T::WN) * (T::BN / T::WN));
  const uint32_t base = lds_addr(lds);
  constexpr int NS = T::NS;
  const int32_t steps = s1 - s0;
  wave_drain();
  for (int32_t i = 0; i < NS - 1 && i < steps; ++i) {
    lp.template issue_a<0, T::SA::Q>(base + i * T::STAGE, s0 + i);
    lp.template issue_b<0, T::SB::Q>(base + i * T::STAGE, s0 + i);
  }
  wait_stage_loads<T::LPS, NS - 2>(max(0, min(NS - 2, steps - 1)));
  __syncthreads();
  int32_t cur = 0;
  for (int32_t s = 0; s < steps; ++s) {
    const uint8_t* stage = lds + cur * T::STAGE;
    const uint32_t nst = base + (cur ? cur - 1 : NS - 1) * T::STAGE;  // the stage of step s - 1, filled for s + NS - 1
    const int32_t nxt = s + NS - 1;
    const bool load = nxt < steps;
    typename T::Frags f0, f1;
    lp.template read<0, T::READS>(f0, stage, 0);
    OVL_SCHED_FENCE();
    lp.template groups<0, T::FM>(acc, f0, f1, stage, nst, s0 + nxt, load);
    lp.template groups<T::FM, T::FM>(acc, f1, f0, stage, nst, s0 + nxt, load);
    lp.template groups<2 * T::FM, T::FM>(acc, f0, f1, stage, nst, s0 + nxt, load);
    lp.template groups<3 * T::FM, T::FM>(acc, f1, f0, stage, nst, s0 + nxt, load);
    wait_stage_loads<T::LPS, NS - 2>(max(0, min(nxt, steps - 1) - (s + 1)));
    __syncthreads();
    cur = cur + 1 == NS ? 0 : cur + 1;
  }
}

// The tile through LDS, a wave's own part at a time, so that rows leave in
// 8-column pieces: f(row, col, v[8], x) for every piece of the wave's
// sub-tile, row/col relative to the tile (a lane's col is the same for all its
// pieces); x = load(row, col), what the epilogue reads beside the sums, is
// fetched for a block of 32 rows at once (one piece at a time, each waiting
// for its own load, 1000 x 2056 x 520 with a float32 residual took 20 us
// instead of 15).  The area must be free (any_tile's end) and holds 32 rows
// of a wave's columns for each wave.
template <class T>
__device__ inline int any_col() {  // the column of this lane's pieces
  constexpr int COLS = T::BN / T::WN;
  return uniform((int)(threadIdx.x >> 6)) % T::WN * COLS + lane_id() % (COLS / 8) * 8;
}

template <class T, class L, class F>
__device__ inline void any_rows(const typename T::Acc& acc, uint8_t* lds, L load, F f) {
  constexpr int COLS = T::BN / T::WN;           // a wave's columns: 64
  constexpr int PITCH = COLS + 4;               // floats of a staged row (the pad spreads the banks)
  constexpr int LPR = COLS / 8, RPI = 64 / LPR;  // lanes per row, rows per read
  constexpr int N = 32 / RPI;                   // pieces of a lane in a block
  static_assert(T::NW * 32 * PITCH * 4 <= T::LDS_BYTES, "the staged rows fit the stages");
  const int lane = lane_id();
  const int wave = uniform((int)(threadIdx.x >> 6));
  float* area = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  const int wm = (wave / T::WN) * (T::BM / 2), col = lane % LPR * 8, tcol = any_col<T>();
#pragma unroll
  for (int fm = 0; fm < T::FM; ++fm) {
    const int row0 = wm + fm * 32 + lane / LPR;
    decltype(load(0, 0)) x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = load(row0 + i * RPI, tcol);
#pragma unroll
    for (int fn = 0; fn < T::FN; ++fn)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        *OVL_LDS(float, area + ((r & 3) + 8 * (r >> 2) + 4 * (lane >> 5)) * PITCH + fn * 32 + (lane & 31)) =
            acc.v[fm][fn][r];
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const int row = i * RPI + lane / LPR;
      float v[8];
      const f32x4 lo = *OVL_LDS(const f32x4, area + row * PITCH + col);
      const f32x4 hi = *OVL_LDS(const f32x4, area + row * PITCH + col + 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = lo[c];
        v[4 + c] = hi[c];
      }
      f(wm + fm * 32 + row, tcol, v, x[0]);
      // The next piece's turn (moving the registers keeps the loop's body, with
      // every activation in it, from being laid out N times).
#pragma unroll
      for (int j = 0; j + 1 < N; ++j) x[j] = x[j + 1];
    }
  }
}

}  // namespace ovl

// Global gradient norm over many tensors, and clipping:
//   norm = sqrt(sum over tensors and elements of g^2),
//   coef = min(1, max_norm / (norm + 1e-6)),   dst = src * coef.
// Squares and sums are float64 throughout (a float32 square overflows at
// 1.8e19, and a float32 sum of 10^9 terms has lost its small ones); norm and
// coef are rounded to float32 once.
//
// The tensors are numbered through in 16-byte slots, a tensor's first slot
// being the one its first byte lies in (slots at multiples of 16 bytes of its
// source).  Every wavefront owns one contiguous range of slots, finds its
// first tensor with a 64-way search of the table, and walks on from there, so
// one launch is balanced whatever the lengths are.  Only a tensor's first and
// last slot can be partial; their elements go one per lane.
//
// Two launches: sums (one float64 a workgroup), then scaling, in which every
// workgroup adds the sums up again, all in the same order.  The second walks
// each range backwards with the same grid, so that it begins with what the
// first read last, which the caches still hold.  What a single workgroup can
// hold goes through one launch.
//
// Measured, with what bounds them: 384M elements in 60 tensors 556 us (HBM:
// 6.2 TB/s reading, then 5.3 reading and writing); 8M float32 17.6 us (the
// second launch's start, which adds up 1024 sums and searches the table, and
// memory), 8M bf16 13.6, in place 12.6, and 19.1 where outputs lie an element
// off their sources' alignment (element by element, 2 bytes a store); 8 tensors,
// 4099 elements, 6.3 us (one launch: a search, two rounds of loads, a barrier
// between them).
//
// The table lies in the caller's workspace between upload and run, and its
// entries are addresses: every entry carries a tag made of its contents, its
// number and its plan's, and a wavefront that meets one whose tag is wrong
// (never uploaded, another plan's, written over since) touches nothing that
// it names.  Its verdict travels apart from the sums (clip_sum.h), so that an
// infinity or a NaN among the gradients does not hide it.  The run then reports
// EINVAL, gives a NaN norm and scales nothing.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <memory>
#include <new>
#include <utility>
#include <vector>

#include "clip_sum.h"
#include "device.h"
#include "host.h"

namespace ovl {

namespace {

constexpr int kGcMaxGroups = 2048;  // workgroups of a launch, and float64 sums in the workspace
constexpr int kGcUpload = 80;       // table entries that travel as one launch's arguments
constexpr size_t kGcSums = kCounterBytes;
constexpr size_t kGcTable = kGcSums + kGcMaxGroups * sizeof(double);

struct GcEntry {
  uint64_t src, dst;  // dst 0: the tensor only counts in the norm
  int64_t first, end; // its slots
  int64_t count;      // 2 * elements + (1 for float32, 0 for bf16)
  uint64_t tag;
};

// Few instructions: a launch of a few microseconds also waits for its code.
// plan: random bits of the entry's plan.
__host__ __device__ inline uint64_t gc_tag(const GcEntry& e, int64_t i, uint64_t plan) {
  return (e.src + (e.dst << 1) + ((uint64_t)e.first << 2) + ((uint64_t)e.end << 3) + ((uint64_t)e.count << 4) +
          (uint64_t)i) ^ plan;
}

struct GcUpload {
  GcEntry e[kGcUpload];
  GcEntry* table;
  int32_t n;
};

struct GcArgs {
  const GcEntry* table;
  ErrRec* err;
  uint64_t plan;
  double* sums;
  float* norm;
  int64_t tensors, slots;
  int64_t per_wave;  // slots of a wavefront
  float max_norm;
};

__global__ __launch_bounds__(64) void gc_upload_kernel(GcUpload u) {
  for (int i = threadIdx.x; i < u.n; i += 64) u.table[i] = u.e[i];
}

__device__ inline float gc_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ inline float gc_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
// (Takes its word by value: a bit cast of a vector's element itself reads
// element 0.)
__device__ inline float gc_f32(uint32_t w) { return __builtin_bit_cast(float, w); }
// float32 to bf16 bits, nearest with ties to even; NaN stays NaN.
__device__ inline uint32_t gc_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__device__ inline double gc_square_sum(u32x4 v, bool f32) {
  double s = 0;
  if (f32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double d = gc_f32(v[i]);
      s += d * d;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double a = gc_lo(v[i]), b = gc_hi(v[i]);
      s += a * a;
      s += b * b;
    }
  }
  return s;
}

__device__ inline u32x4 gc_scaled(u32x4 v, bool f32, float coef) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = f32 ? __builtin_bit_cast(uint32_t, gc_f32(v[i]) * coef)
               : gc_bf16(gc_lo(v[i]) * coef) | gc_bf16(gc_hi(v[i]) * coef) << 16;
  return v;
}

__device__ inline uint64_t gc_lane(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}

// The last tensor whose first slot is <= v, the one that holds slot v, and its
// number.  The last round's lanes hold the entries that they look at, so that
// the one found needs no load of its own.
__device__ inline GcEntry gc_find(const GcEntry* table, int64_t tensors, int64_t v, int64_t& at) {
  int64_t lo = 0, n = tensors;
  while (n > 64) {
    const int64_t step = (n + 63) / 64, i = lane_id() * step;
    const bool le = i < n && table[lo + i].first <= v;
    // At least 1 in a sound table, and in any other: lo stays an entry's number.
    const int below = max(1, (int)__popcll(__ballot(le)));
    lo += (below - 1) * step;
    n = min(step, n - (below - 1) * step);
  }
  const GcEntry e = table[lo + min((int64_t)lane_id(), n - 1)];
  const int pick = uniform(max(1, (int)__popcll(__ballot(lane_id() < n && e.first <= v))) - 1);
  at = uniform64(lo + pick);
  return GcEntry{gc_lane(e.src, pick),           gc_lane(e.dst, pick),
                 (int64_t)gc_lane(e.first, pick), (int64_t)gc_lane(e.end, pick),
                 (int64_t)gc_lane(e.count, pick), gc_lane(e.tag, pick)};
}

// One tensor's slots, seen from the wavefront.
struct GcTensor {
  uint64_t src, dst;
  int64_t first, slots, count;
  bool f32;
  int head;  // bytes of slot 0 ahead of the tensor

  __device__ GcTensor(const GcEntry& e) {
    src = e.src;
    dst = e.dst;
    first = e.first;
    slots = e.end - e.first;
    count = e.count >> 1;
    f32 = e.count & 1;
    head = (int)(src & 15);
  }
  __device__ int shift() const { return f32 ? 2 : 1; }
  // Whole slots are [whole0, whole1); slot 0 and the last may be partial.
  __device__ int64_t whole0() const { return head ? 1 : 0; }
  __device__ int64_t whole1() const { return (head + (count << shift())) >> 4; }
  // Element of a partial slot that this lane holds, or -1.
  __device__ int64_t edge(int64_t slot) const {
    const int64_t i = ((slot * 16 - head) >> shift()) + lane_id();
    return lane_id() < (16 >> shift()) && i >= 0 && i < count ? i : -1;
  }
  __device__ float load(int64_t i) const {
    return f32 ? reinterpret_cast<const float*>(src)[i]
               : gc_lo(reinterpret_cast<const uint16_t*>(src)[i]);
  }
  __device__ void store(int64_t i, float v) const {
    if (f32)
      reinterpret_cast<float*>(dst)[i] = v;
    else
      reinterpret_cast<uint16_t*>(dst)[i] = (uint16_t)gc_bf16(v);
  }
  __device__ const u32x4* vec() const { return reinterpret_cast<const u32x4*>(src - head); }
};

constexpr int kGcU = 4;  // 16-byte loads in flight per lane

// Sum of squares over slots [v0, v1), this lane's share; kClipForeign, in every
// lane, where the table is not this plan's.  (Sound entries follow each other without a
// gap up to the last slot, so a walk from the one that holds v0 stays in the
// table.  Every entry holds slots, so that the launch looks at all of them.)
__device__ inline double gc_sum_range(const GcArgs& a, int64_t v0, int64_t v1) {
  double s = 0;
  if (v0 >= v1) return s;
  const int lane = lane_id();
  int64_t t;
  GcEntry entry = gc_find(a.table, a.tensors, v0, t);
  for (;;) {
    const uint64_t tag = gc_tag(entry, t, a.plan);
    if (entry.tag != tag || v0 < entry.first || v0 >= entry.end) {
      if (lane == 0) report_error(a.err, OVL_EINVAL, kSiteClip, t, (int64_t)entry.tag, (int64_t)tag);
      return kClipForeign;
    }
    const GcTensor g(entry);
    const int64_t b = v0 - g.first, e = min(v1 - g.first, g.slots);
    const int64_t w0 = max(b, g.whole0()), w1 = min(e, g.whole1());
    if (b < g.whole0() && b < e) {
      const int64_t i = g.edge(b);
      const double d = i >= 0 ? g.load(i) : 0.f;
      s += d * d;
    }
    const u32x4* p = g.vec();
    int64_t i = w0 + lane;
    for (; i + (kGcU - 1) * 64 < w1; i += kGcU * 64) {
      u32x4 v[kGcU];
#pragma unroll
      for (int u = 0; u < kGcU; ++u) v[u] = p[i + u * 64];
#pragma unroll
      for (int u = 0; u < kGcU; ++u) s += gc_square_sum(v[u], g.f32);
    }
    for (; i < w1; i += 64) s += gc_square_sum(p[i], g.f32);
    if (e > g.whole1() && e - 1 >= g.whole0() && b < e) {
      const int64_t j = g.edge(e - 1);
      const double d = j >= 0 ? g.load(j) : 0.f;
      s += d * d;
    }
    v0 = g.first + e;
    if (v0 >= v1) break;
    entry = a.table[++t];
  }
  return s;
}

__device__ inline void gc_scale_slot(const GcTensor& g, int64_t i, u32x4 v, float coef, bool vec) {
  if (vec) {
    __builtin_nontemporal_store(gc_scaled(v, g.f32, coef), reinterpret_cast<u32x4*>(g.dst - g.head) + i);
    return;
  }
  // dst lies differently within its 16 bytes than src: element by element.
  const int64_t e0 = (i * 16 - g.head) >> g.shift();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (g.f32) {
      g.store(e0 + k, gc_f32(v[k]) * coef);
    } else {
      g.store(e0 + 2 * k, gc_lo(v[k]) * coef);
      g.store(e0 + 2 * k + 1, gc_hi(v[k]) * coef);
    }
  }
}

// dst = src * coef over slots [v0, v1), from the last to the first.  Both
// streams are nontemporal (384M elements, both launches: 590 -> 553 us, of
// which 44 in the next call's first launch, behind ordinary stores; 32 MiB:
// 19.2 -> 18.1, in the second launch, which finds more of the first's reads).
__device__ inline void gc_scale_tensor(const GcTensor& g, int64_t b, int64_t e, float coef) {
  // In place with coef 1 nothing changes.
  if (!g.dst || (g.dst == g.src && coef == 1.f)) return;
  const int lane = lane_id();
  const bool vec = ((g.dst ^ g.src) & 15) == 0;
  const int64_t w0 = max(b, g.whole0()), w1 = min(e, g.whole1());
  if (e > g.whole1() && e - 1 >= g.whole0()) {
    const int64_t j = g.edge(e - 1);
    if (j >= 0) g.store(j, g.load(j) * coef);
  }
  const u32x4* p = g.vec();
  int64_t i = w1 - 1 - lane;
  for (; i - (kGcU - 1) * 64 >= w0; i -= kGcU * 64) {
    u32x4 v[kGcU];
#pragma unroll
    for (int u = 0; u < kGcU; ++u) v[u] = __builtin_nontemporal_load(p + i - u * 64);
#pragma unroll
    for (int u = 0; u < kGcU; ++u) gc_scale_slot(g, i - u * 64, v[u], coef, vec);
  }
  for (; i >= w0; i -= 64) gc_scale_slot(g, i, p[i], coef, vec);
  if (b < g.whole0()) {
    const int64_t j = g.edge(b);
    if (j >= 0) g.store(j, g.load(j) * coef);
  }
}

__device__ inline void gc_scale_range(const GcArgs& a, int64_t v0, int64_t v1, GcEntry entry, int64_t t, float coef) {
  if (v0 >= v1) return;
  for (;;) {
    const GcTensor g(entry);
    gc_scale_tensor(g, max(v0 - g.first, (int64_t)0), v1 - g.first, coef);
    v1 = g.first;
    if (v0 >= v1) break;
    entry = a.table[--t];
  }
}

__device__ inline double gc_wave_sum(double s) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
  return s;
}

// Total over the workgroup's threads, the same bits in every thread; s as
// ClipTotal::add takes it.
template <int NT>
__device__ inline ClipTotal gc_group_sum(double s, double* lds) {
  const bool foreign = __any(s < 0);
  s = gc_wave_sum(s);
  if (lane_id() == 0) lds[threadIdx.x >> 6] = foreign ? kClipForeign : s;
  __syncthreads();
  ClipTotal t;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) t.add(lds[w]);
  return t;
}

// norm by the first thread; NaN where the table is foreign.
__device__ inline float gc_coef(const GcArgs& a, const ClipTotal& t, bool first) {
  const double norm = t.foreign ? __builtin_nan("") : sqrt(t.sum);
  if (first) *a.norm = (float)norm;
  const double c = (double)a.max_norm / (norm + 1e-6);
  return c >= 1.0 || isinf(a.max_norm) ? 1.f : (float)c;  // a NaN norm gives a NaN coefficient
}

__global__ __launch_bounds__(kThreads) void gc_norm_kernel(GcArgs a) {
  __shared__ double lds[kThreads / 64];
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 64) + uniform(threadIdx.x >> 6);
  const int64_t v0 = min(w * a.per_wave, a.slots), v1 = min(v0 + a.per_wave, a.slots);
  const ClipTotal t = gc_group_sum<kThreads>(gc_sum_range(a, v0, v1), lds);
  if (threadIdx.x == 0) a.sums[blockIdx.x] = t.word();
}

__global__ __launch_bounds__(kThreads) void gc_scale_kernel(GcArgs a) {
  __shared__ double lds[kThreads / 64];
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 64) + uniform(threadIdx.x >> 6);
  const int64_t v0 = min(w * a.per_wave, a.slots), v1 = min(v0 + a.per_wave, a.slots);
  ClipTotal mine;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) mine.add(a.sums[i]);
  // (The search's loads are on their way with the sums'.)
  int64_t at = 0;
  GcEntry entry = gc_find(a.table, a.tensors, max(v1 - 1, (int64_t)0), at);
  const ClipTotal t = gc_group_sum<kThreads>(mine.word(), lds);
  const float coef = gc_coef(a, t, blockIdx.x == 0 && threadIdx.x == 0);
  if (t.foreign) return;
  gc_scale_range(a, v0, v1, entry, at, coef);
}

constexpr int kGcOneThreads = 1024;

__global__ __launch_bounds__(kGcOneThreads) void gc_one_kernel(GcArgs a) {
  __shared__ double lds[kGcOneThreads / 64];
  const int64_t w = uniform(threadIdx.x >> 6);
  const int64_t v0 = min(w * a.per_wave, a.slots), v1 = min(v0 + a.per_wave, a.slots);
  const ClipTotal t = gc_group_sum<kGcOneThreads>(gc_sum_range(a, v0, v1), lds);
  const float coef = gc_coef(a, t, threadIdx.x == 0);
  if (t.foreign) return;
  if (v0 >= v1) return;
  int64_t at;
  const GcEntry entry = gc_find(a.table, a.tensors, v1 - 1, at);
  gc_scale_range(a, v0, v1, entry, at, coef);
}

}  // namespace

}  // namespace ovl

using namespace ovl;

struct grad_clip_plan_s {
  std::vector<GcEntry> table;
  int64_t slots;
  uint64_t id;  // 64 bits that no other plan of this process has
  // What the tensors occupy, by beginning: [begin, the farthest end up to here).
  std::vector<std::pair<uint64_t, uint64_t>> spans;

  bool touches(const void* p, uint64_t bytes) const {
    const uint64_t lo = reinterpret_cast<uint64_t>(p), hi = lo + bytes;
    const auto behind = std::lower_bound(spans.begin(), spans.end(), hi,
                                         [](const std::pair<uint64_t, uint64_t>& s, uint64_t v) { return s.first < v; });
    return behind != spans.begin() && (behind - 1)->second > lo;
  }
};

static std::atomic<uint64_t> gc_plans{0};

extern "C" ovl_status grad_clip_plan(const grad_clip_tensor* tensors, int64_t num, grad_clip_plan_t* out) {
  if (!out) return OVL_EINVAL;
  *out = nullptr;
  if (num < 0 || (num && !tensors)) return OVL_EINVAL;
  if (num > (1 << 20)) return OVL_EUNSUPPORTED;
  try {
    struct Span {
      uint64_t lo, hi;
      int64_t owner;
      bool written;
    };
    std::vector<GcEntry> table;
    std::vector<Span> spans;
    table.reserve(num);
    int64_t slot = 0;
    for (int64_t i = 0; i < num; ++i) {
      const grad_clip_tensor& t = tensors[i];
      if ((t.type != OVL_BF16 && t.type != OVL_F32) || t.reserved) return OVL_EINVAL;
      if (t.count < 0) return OVL_ESHAPE;
      if (t.count > (1ll << 40)) return OVL_EUNSUPPORTED;
      const uint64_t src = reinterpret_cast<uint64_t>(t.src), dst = reinterpret_cast<uint64_t>(t.dst);
      const uint64_t size = t.type == OVL_F32 ? 4 : 2, bytes = (uint64_t)t.count * size;
      if (t.count && !src) return OVL_EINVAL;
      if ((src | dst) & (size - 1)) return OVL_EALIGN;
      if (!t.count) continue;
      const int64_t first = slot;
      slot += (int64_t)(((src & 15) + bytes + 15) / 16);
      table.push_back({src, dst, first, slot, 2 * t.count + (t.type == OVL_F32), 0});
      if (dst != src) spans.push_back({src, src + bytes, i, false});
      if (dst) spans.push_back({dst, dst + bytes, i, true});
    }
    // What is written may overlap nothing else that the call reads or writes
    // (a tensor clipped in place is one span).
    std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.lo < y.lo; });
    uint64_t end_any = 0, end_written = 0;
    for (const Span& s : spans) {
      if (s.lo < end_written || (s.written && s.lo < end_any)) return OVL_EINVAL;
      end_any = std::max(end_any, s.hi);
      if (s.written) end_written = std::max(end_written, s.hi);
    }
    std::unique_ptr<grad_clip_plan_s> p(new grad_clip_plan_s);
    p->spans.reserve(spans.size());
    p->slots = slot;
    for (const Span& s : spans) p->spans.emplace_back(s.lo, std::max(s.hi, p->spans.empty() ? 0 : p->spans.back().second));
    p->id = (++gc_plans + 1) * 0x9E3779B97F4A7C15ull;  // odd: a bijection of the plan's number
    for (size_t i = 0; i < table.size(); ++i) table[i].tag = gc_tag(table[i], (int64_t)i, p->id);
    p->table.swap(table);
    *out = p.release();
  } catch (const std::bad_alloc&) {
    return OVL_EUNSUPPORTED;
  }
  return OVL_OK;
}

extern "C" ovl_status grad_clip_plan_destroy(grad_clip_plan_t p) {
  delete p;
  return OVL_OK;
}

extern "C" size_t grad_clip_workspace_bytes(grad_clip_plan_t p) {
  return p ? kGcTable + aligned_up(p->table.size() * sizeof(GcEntry), 256) : 0;
}

extern "C" ovl_status grad_clip_upload(grad_clip_plan_t p, void* workspace, hipStream_t stream) {
  if (!p || !workspace) return OVL_EINVAL;
  if (!aligned16(workspace)) return OVL_EALIGN;
  if (p->touches(workspace, grad_clip_workspace_bytes(p))) return OVL_EINVAL;
  GcUpload u = {};
  GcEntry* table = reinterpret_cast<GcEntry*>(static_cast<uint8_t*>(workspace) + kGcTable);
  for (size_t i = 0; i < p->table.size(); i += kGcUpload) {
    u.n = (int32_t)std::min<size_t>(kGcUpload, p->table.size() - i);
    std::copy_n(p->table.begin() + i, u.n, u.e);
    u.table = table + i;
    hipLaunchKernelGGL(gc_upload_kernel, dim3(1), dim3(64), 0, stream, u);
    OVL_HIP_TRY(hipGetLastError());
  }
  return OVL_OK;
}

extern "C" ovl_status grad_norm_clip_run(grad_clip_plan_t p, float max_norm, float* norm, void* workspace,
                                         hipStream_t stream) {
  if (!p || !norm || !workspace) return OVL_EINVAL;
  if (!(max_norm >= 0.f)) return OVL_EINVAL;  // negative or NaN
  if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(norm) & 3u)) return OVL_EALIGN;
  const size_t bytes = grad_clip_workspace_bytes(p);
  const uint64_t at = reinterpret_cast<uint64_t>(norm), ws = reinterpret_cast<uint64_t>(workspace);
  if ((at < ws + bytes && at + 4 > ws) || p->touches(norm, 4) || p->touches(workspace, bytes)) return OVL_EINVAL;
  DeviceInfo di;
  ovl_status st = current_device_info(&di);
  if (st) return st;
  GcArgs a = {};
  a.table = reinterpret_cast<const GcEntry*>(static_cast<uint8_t*>(workspace) + kGcTable);
  a.sums = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + kGcSums);
  a.err = static_cast<ErrRec*>(workspace);
  a.plan = p->id;
  a.norm = norm;
  a.tensors = (int64_t)p->table.size();
  a.slots = p->slots;
  a.max_norm = max_norm;
  if (a.slots <= 8192) {
    a.per_wave = ceil_div(a.slots, kGcOneThreads / 64);
    hipLaunchKernelGGL(gc_one_kernel, dim3(1), dim3(kGcOneThreads), 0, stream, a);
    OVL_HIP_TRY(hipGetLastError());
    return OVL_OK;
  }
  const int64_t groups =
      std::min<int64_t>({kGcMaxGroups, (int64_t)di.cus * 4, ceil_div(a.slots, 64 * kGcU * (kThreads / 64))});
  a.per_wave = ceil_div(a.slots, groups * (kThreads / 64));
  hipLaunchKernelGGL(gc_norm_kernel, dim3((uint32_t)groups), dim3(kThreads), 0, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  hipLaunchKernelGGL(gc_scale_kernel, dim3((uint32_t)groups), dim3(kThreads), 0, stream, a);
  OVL_HIP_TRY(hipGetLastError());
  return OVL_OK;
}

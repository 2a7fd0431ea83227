// Drives the host code of the feed-forward calls for the sanitizers: size
// queries over random descriptors, plans of thousands of tensors, and the
// argument checks of the run calls, which refuse before any device work.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "ovl.h"

namespace {

int g_failures = 0;
#define EXPECT(c)                                                     \
  do {                                                                \
    if (!(c)) {                                                       \
      std::fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c);    \
      ++g_failures;                                                   \
    }                                                                 \
  } while (0)

void* fake(uint64_t a) { return reinterpret_cast<void*>(a << 12); }

int64_t size(std::mt19937_64& rng, int64_t most) {
  const int64_t edge[] = {-8, -1, 0, 1, 7, 8, 9, most, most + 8, INT64_MAX, INT64_MIN};
  if (rng() % 12 == 0) return edge[rng() % 11];
  const double l = std::log2((double)most / 8) * (double)(rng() % 1000) / 1000;
  return 8 * (int64_t)std::exp2(l);
}

void products(std::mt19937_64& rng) {
  int accepted = 0;
  for (int i = 0; i < 20000; ++i) {
    gemm_epilogue_desc d = {};
    d.m = rng() % 3 ? size(rng, 1 << 20) : (int64_t)(rng() % 40);
    d.n = size(rng, 1 << 20);
    d.k = size(rng, 1 << 20);
    if (rng() % 4 == 0) d.lda = size(rng, 1 << 20);
    if (rng() % 8 == 0) d.ldo = size(rng, 1 << 20);
    d.act = (int32_t)(rng() % 8) - 1;
    d.out_type = (int32_t)(rng() % 3);
    d.reserved = rng() % 50 == 0;
    const size_t bytes = gemm_epilogue_workspace_bytes(&d);
    EXPECT(!bytes || bytes > OVL_ERROR_RECORD_BYTES);
    accepted += bytes != 0;
    gemm_epilogue_grad_desc g = {};
    g.m = d.m;
    g.n = d.n;
    g.k = d.k;
    g.lda = d.lda;
    g.act_in = d.act;
    g.db_type = d.out_type;
    const size_t gb = gemm_epilogue_grad_workspace_bytes(&g);
    EXPECT(!gb || gb > OVL_ERROR_RECORD_BYTES);
    if (!bytes) EXPECT(gemm_epilogue_run(&d, fake(1), fake(2), nullptr, nullptr, fake(3), nullptr, fake(4), nullptr) != OVL_OK);
    if (!gb)
      EXPECT(gemm_epilogue_grad_run(&g, nullptr, nullptr, fake(1), fake(2), fake(3), nullptr, fake(5), fake(6), nullptr,
                                    nullptr, nullptr, fake(7), nullptr) != OVL_OK);
  }
  EXPECT(accepted > 1000);
}

void experts(std::mt19937_64& rng) {
  int accepted = 0;
  for (int i = 0; i < 20000; ++i) {
    moe_layer_desc d = {};
    d.tokens = rng() % 10 ? (int64_t)(rng() % 130) : size(rng, 128);
    d.hidden = size(rng, 1 << 16);
    d.inter = size(rng, 1 << 16);
    d.experts = (int32_t)(rng() % 259) - 1;
    d.topk = (int32_t)(rng() % 11) - 1;
    d.act = (int32_t)(rng() % 6);
    d.gated = rng() % 2;
    d.w_type = rng() % 2 ? OVL_FP8 : OVL_BF16;
    d.out_type = (int32_t)(rng() % 2);
    d.norm_topk = rng() % 2;
    const size_t bytes = moe_layer_workspace_bytes(&d);
    accepted += bytes != 0;
    if (!bytes)
      EXPECT(moe_layer_run(&d, fake(1), nullptr, (int32_t*)fake(2), (float*)fake(3), fake(4), nullptr, fake(5), nullptr,
                           fake(6), fake(7), nullptr) != OVL_OK);
  }
  EXPECT(accepted > 1000);
}

void clipping(std::mt19937_64& rng) {
  for (int n : {0, 1, 2, 80, 81, 5000, 1 << 16}) {
    std::vector<grad_clip_tensor> t(n);
    uint64_t at = 1 << 20;
    for (auto& x : t) {
      x.type = (int32_t)(rng() % 2);
      const uint64_t size = x.type == OVL_F32 ? 4 : 2;
      x.count = rng() % 5 ? (int64_t)(rng() % 5000) : 0;
      at = (at + rng() % 64) / size * size + size;
      x.src = reinterpret_cast<void*>(at);
      x.dst = rng() % 4 ? const_cast<void*>(x.src) : nullptr;
      at += (uint64_t)x.count * size;
      x.reserved = 0;
    }
    grad_clip_plan_t p = nullptr;
    EXPECT(grad_clip_plan(t.data(), n, &p) == OVL_OK && p);
    EXPECT(grad_clip_workspace_bytes(p) > OVL_ERROR_RECORD_BYTES);
    EXPECT(grad_norm_clip_run(p, -1.f, (float*)fake(1), fake(2), nullptr) == OVL_EINVAL);
    EXPECT(grad_clip_upload(p, (void*)8, nullptr) == OVL_EALIGN);
    EXPECT(grad_clip_plan_destroy(p) == OVL_OK);
    if (n > 1) {  // the last one written over the first one
      grad_clip_tensor& a = t[0];
      a.count = 64;
      t[n - 1] = a;
      t[n - 1].dst = const_cast<void*>(a.src);
      EXPECT(grad_clip_plan(t.data(), n, &p) == OVL_EINVAL && !p);
    }
  }
  grad_clip_plan_t p = nullptr;
  EXPECT(grad_clip_plan(nullptr, (1 << 20) + 1, &p) != OVL_OK);
  grad_clip_tensor huge[2] = {{fake(1), nullptr, 1ll << 40, OVL_F32, 0}, {fake(1), nullptr, 1ll << 40, OVL_F32, 0}};
  EXPECT(grad_clip_plan(huge, 2, &p) == OVL_OK);
  EXPECT(grad_clip_plan_destroy(p) == OVL_OK && grad_clip_plan_destroy(nullptr) == OVL_OK);
}

}  // namespace

int main() {
  std::mt19937_64 rng(2024);
  products(rng);
  experts(rng);
  clipping(rng);
  if (g_failures) {
    std::fprintf(stderr, "%d failed expectations\n", g_failures);
    return 1;
  }
  std::printf("host driver ok\n");
  return 0;
}

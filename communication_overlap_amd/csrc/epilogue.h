// What follows a product's float32 sums: bias, activation, residual, the
// activation's derivative, and the rounding into the output's type.  All of
// it is float32; an output is rounded once, to nearest with ties to even.
#pragma once

#include "device.h"
#include "ovl.h"

namespace ovl {

__device__ inline float bf16_lo_f(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ inline float bf16_hi_f(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
__device__ inline uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ inline uint32_t bf16_pair(float a, float b) { return bf16_bits(a) | bf16_bits(b) << 16; }

// sigma(x) = 1 / (1 + exp(-x)) from q = x log2(e) / 2, to a few float32 steps of
// itself on either side (2 |x| half steps come from the exponent's rounding): with
// e = exp(-|x|) = h^2, sigma is r = 1 / (1 + e) or e r, and sigma (1 - sigma) is
// (h r)^2.  A factor y goes in between h and h r, since e leaves float32's range
// before y e does.
struct Sigmoid {
  float h, r;
  bool up;
  __device__ inline explicit Sigmoid(float q) : up(q > 0.f) {
    h = __builtin_amdgcn_exp2f(-fabsf(q));
    r = __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.f));
  }
  // y sigma
  __device__ inline float times(float y) const {
    const float g = up ? 1.f : h;
    return (y * g) * (g * r);
  }
  // sigma + y sigma (1 - sigma)
  __device__ inline float slope(float y) const {
    const float m = h * r;
    return __builtin_fmaf(y * m, m, up ? r : h * m);
  }
};

constexpr float kHalfLog2e = 0.721347520444481704f;
// The tanh form of GELU, 0.5 z (1 + tanh u), u = sqrt(2 / pi) (z + 0.044715 z^3),
// is z sigma(2 u): no cancellation where tanh is near -1.  2 u is z times
constexpr float kGelu1 = 1.59576912160573071f, kGelu3 = 0.044715f * kGelu1;  // kGelu1 + kGelu3 z^2
__device__ inline float gelu_q(float z, float z2) {
  return z * __builtin_fmaf(kGelu3 * kHalfLog2e, z2, kGelu1 * kHalfLog2e);
}

// The normal distribution's tail beyond |z|, exp(-z^2 / 2) r, with r a
// polynomial in t = 1 / (1 + 0.3 |z|): the scaled complementary error function
// erfcx(|z| / sqrt 2) / 2 over |z| <= 13.6, fitted by weighted least squares to
// 2^-24 of itself (6 half steps in float32; the exponent's rounding adds 1.5 z^2
// of them).  (0.5 (1 + erf(z / sqrt 2)) has no digit of the tail left below z =
// -5.6; the device library's erfc has, and costs 8192 x 3584 x 4096 10 us and
// 1000 x 2056 x 520 3.3.)
struct NormalTail {
  float e, r;
  __device__ inline explicit NormalTail(float z) {
    constexpr float kC[] = {0.0383444632f, -0.169001593f, 0.228320013f, -0.0761172854f, 0.142266526f,
                            0.0947981873f, 0.121890982f,  0.119491808f, 6.92692344e-06f};
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, fabsf(z), 1.f));
    r = kC[0];
#pragma unroll
    for (int i = 1; i < 9; ++i) r = __builtin_fmaf(r, t, kC[i]);
    e = __builtin_amdgcn_exp2f(z * z * (-0.5f * 1.44269504088896341f));
  }
};

__device__ inline float act_f(float z, int kind) {
  switch (kind) {
    case OVL_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays
    case OVL_ACT_GELU: {
      const NormalTail n(z);
      return z * (z > 0.f ? 1.f - n.e * n.r : n.e * n.r);
    }
    default: return z;
  }
}

// z sigma(x), q = x log2(e) / 2 of eight z: by 1 / (1 + exp(-x)) itself, which is
// infinity's reciprocal below x = -88 where z sigma(x) still is a number, and
// from x = -44 down by the other form (for all of them that one takes 3 us more
// over the 8192 x 3584 outputs of a product with SiLU).
__device__ inline void times_sigma8(float (&z)[8], const float (&q)[8]) {
  float least = q[0];
#pragma unroll
  for (int c = 1; c < 8; ++c) least = fminf(least, q[c]);
  float v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) v[c] = z[c] * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-2.f * q[c]));
  if (least < -32.f)
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = q[c] < -32.f ? Sigmoid(q[c]).times(z[c]) : v[c];
#pragma unroll
  for (int c = 0; c < 8; ++c) z[c] = v[c];
}

// d act / dz.  A smooth one's factor z is taken at most so far out that the
// value has reached 1 there or, below, is under float32's least number (SiLU's: z
// exp(z), -1e-44 at z = -106; the GELUs': exp(-z^2 / 2)), which keeps infinity
// times zero out of the products.  NaN stays, by way of the exponential.
__device__ inline float act_grad_f(float z, int kind) {
  switch (kind) {
    case OVL_ACT_RELU: return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
    case OVL_ACT_GELU: {  // cdf + z pdf
      const NormalTail n(z);
      const float v = __builtin_amdgcn_fmed3f(z, -32.f, 32.f);
      return (z > 0.f ? 1.f : 0.f) + n.e * (0.398942280401432678f * v + (z > 0.f ? -n.r : n.r));
    }
    case OVL_ACT_GELU_TANH: {  // s + z s (1 - s) d(2 u) / dz
      const float z2 = fminf(z * z, 1024.f), v = __builtin_amdgcn_fmed3f(z, -32.f, 32.f);
      return Sigmoid(gelu_q(z, z2)).slope(v * __builtin_fmaf(3.f * kGelu3, z2, kGelu1));
    }
    case OVL_ACT_SILU:  // s + z s (1 - s)
      return Sigmoid(z * kHalfLog2e).slope(__builtin_amdgcn_fmed3f(z, -256.f, 256.f));
    default: return 1.f;
  }
}

// The same for eight values: one branch on the kind for all of them.
__device__ inline void act8(float (&v)[8], int kind) {
#define OVL_ACT8(K)                                    \
  case K:                                              \
    _Pragma("unroll") for (int c = 0; c < 8; ++c) v[c] = act_f(v[c], K); \
    break;
  switch (kind) {
    OVL_ACT8(OVL_ACT_RELU)
    OVL_ACT8(OVL_ACT_GELU)
    case OVL_ACT_GELU_TANH:
    case OVL_ACT_SILU: {
      float q[8];
      if (kind == OVL_ACT_SILU)
#pragma unroll
        for (int c = 0; c < 8; ++c) q[c] = v[c] * kHalfLog2e;
      else
#pragma unroll
        for (int c = 0; c < 8; ++c) q[c] = gelu_q(v[c], v[c] * v[c]);
      times_sigma8(v, q);
      break;
    }
    default: break;
  }
#undef OVL_ACT8
}

// v *= act'(z).
__device__ inline void act_grad8(float (&v)[8], const float (&z)[8], int kind) {
#define OVL_ACT8(K)                                    \
  case K:                                              \
    _Pragma("unroll") for (int c = 0; c < 8; ++c) v[c] *= act_grad_f(z[c], K); \
    break;
  switch (kind) {
    OVL_ACT8(OVL_ACT_RELU)
    OVL_ACT8(OVL_ACT_GELU)
    OVL_ACT8(OVL_ACT_GELU_TANH)
    OVL_ACT8(OVL_ACT_SILU)
    default: break;
  }
#undef OVL_ACT8
}

// Eight consecutive elements of a row in float32, from bf16 or float32.
__device__ inline void load8(float (&v)[8], const void* p, int64_t i, int type) {
  if (type == OVL_F32) {
    const f32x4 a = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i)[0];
    const f32x4 b = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i)[1];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[c] = a[c];
      v[4 + c] = b[c];
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[2 * c] = bf16_lo_f(w[c]);
      v[2 * c + 1] = bf16_hi_f(w[c]);
    }
  }
}

__device__ inline void store8(const float (&v)[8], void* p, int64_t i, int type) {
  if (type == OVL_F32) {
    reinterpret_cast<f32x4*>(static_cast<float*>(p) + i)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4*>(static_cast<float*>(p) + i)[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 w;
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = bf16_pair(v[2 * c], v[2 * c + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = w;
  }
}

// The epilogue of one product, columns n (a multiple of 8):
//   z = sum + bias;  out = act(z) + residual;  z_out = bf16(z)
// or, with z_in, out = sum * act'(z_in) (the gradient's).  A gradient's db_in is
// its residual.
struct Epilogue {
  void* out;
  void* z_out;           // bf16, or null
  const float* bias;     // [n], or null
  const void* residual;  // or null
  const void* z_in;      // bf16, or null: multiply by act'(z_in)
  int64_t ld_out, ld_z, ld_res;  // ld_z: of z_out or z_in
  int32_t out_type, res_type, act;
};

// What the epilogue of a piece reads beside the sums, as it lies in memory:
// eight elements of the residual or of z_in (a call has one of them at most).
struct EpilogueIn {
  u32x4 q[2];
};

__device__ inline void unpack8(float (&v)[8], const EpilogueIn& x, int type) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t a = x.q[0][c], b = x.q[1][c];
    if (type == OVL_F32) {
      v[c] = __builtin_bit_cast(float, a);
      v[4 + c] = __builtin_bit_cast(float, b);
    } else {
      v[2 * c] = bf16_lo_f(a);
      v[2 * c + 1] = bf16_hi_f(a);
    }
  }
}

__device__ inline EpilogueIn epilogue_load(const Epilogue& e, int64_t row, int64_t col) {
  EpilogueIn x = {};
  if (e.residual && e.res_type == OVL_F32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(e.residual) + row * e.ld_res + col);
    x.q[0] = p[0];
    x.q[1] = p[1];
  } else if (e.residual) {
    x.q[0] = ld16(static_cast<const uint16_t*>(e.residual) + row * e.ld_res + col);
  } else if (e.z_in) {
    x.q[0] = ld16(static_cast<const uint16_t*>(e.z_in) + row * e.ld_z + col);
  }
  return x;
}

// Eight columns' bias, or zeros.
__device__ inline void epilogue_bias(float (&b)[8], const Epilogue& e, int64_t col, bool there) {
#pragma unroll
  for (int c = 0; c < 8; ++c) b[c] = 0.f;
  if (e.bias && there) load8(b, e.bias, col, OVL_F32);
}

__device__ inline void epilogue8(const Epilogue& e, int64_t row, int64_t col, float (&v)[8], const float (&bias)[8],
                                 const EpilogueIn& x) {
  if (e.bias)
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] += bias[c];
  if (e.z_out) store8(v, e.z_out, row * e.ld_z + col, OVL_BF16);
  if (e.z_in) {
    float z[8];
    unpack8(z, x, OVL_BF16);
    act_grad8(v, z, e.act);
  } else {
    act8(v, e.act);
  }
  if (e.residual) {
    float r[8];
    unpack8(r, x, e.res_type);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] += r[c];
  }
  store8(v, e.out, row * e.ld_out + col, e.out_type);
}

__device__ inline void epilogue8(const Epilogue& e, int64_t row, int64_t col, float (&v)[8]) {
  float b[8];
  epilogue_bias(b, e, col, true);
  epilogue8(e, row, col, v, b, epilogue_load(e, row, col));
}

}  // namespace ovl

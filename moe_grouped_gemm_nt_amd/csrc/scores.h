// Scores of the router and its loss: exponentials, logits and sums over the lanes
// of a token.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cfloat>

namespace dg {

// e^x as 2^(x log2 e) with the product's rounding carried along: relative error
// below 2e-7 at any x the scores use (the bare product loses |x| units of the
// last place).  Results below 2^-126 are 0: exp_below has those.
__device__ __forceinline__ float exp_f32(float x) {
  const float log2e = 1.44269502f, log2e_lo = 1.92596303e-8f, ln2 = 0.693147182f;
  x = fmaxf(x, -150.0f);                 // 0 from here down; also keeps lo finite
  const float hi = x * log2e;
  const float lo = fmaf(x, log2e_lo, fmaf(x, log2e, -hi));
  const float r = __builtin_amdgcn_exp2f(hi);
  return hi < 127.0f ? fmaf(r * ln2, lo, r) : r;
}

// e^x below kLeastNormal, where the result may be subnormal, down to 2^-149: the
// hardware's exponential and reciprocal return 0 for those, so that it is taken
// 2^64 times as large and scaled by a product, which rounds once.
constexpr float kLeastNormal = -87.0f;   // e^-87 is 2^-125.5
__device__ __forceinline__ float exp_below(float x) {
  const float log2e = 1.44269502f, log2e_lo = 1.92596303e-8f, ln2 = 0.693147182f;
  x = fmaxf(x, -150.0f);
  const float hi = x * log2e;
  const float lo = fmaf(x, log2e_lo, fmaf(x, log2e, -hi));
  const float r = __builtin_amdgcn_exp2f(hi + 64.0f);
  return fmaf(r * ln2, lo, r) * 0x1p-64f;
}
// e^x of a single x <= 0
__device__ __forceinline__ float exp_any(float x) {
  const float r = exp_f32(x);
  return __builtin_expect(x < kLeastNormal, 0) ? exp_below(x) : r;
}

// The hardware reciprocal (1 unit of the last place) in place of a division: the
// scores stay within 3e-7.  Below kLeastNormal a sigmoid is e^x to 2^-125.
__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x)); }
__device__ __forceinline__ float sigmoid_any(float x) {
  const float r = sigmoid_f32(x);
  return __builtin_expect(x < kLeastNormal, 0) ? exp_below(x) : r;
}

template <bool BF16>
__device__ __forceinline__ float raw_logit(const void* p, size_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
}
// -inf for a masked expert (NaN or -inf), else the logit with +inf made finite
__device__ __forceinline__ float clean_logit(float x) { return x > -INFINITY ? fminf(x, FLT_MAX) : -INFINITY; }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// DPP controls that pair the sixteen lanes of a row in four steps
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ int row_max(int v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  return max(v, dpp<kMirror>(v));
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<kXor1>(v));
  v = fmaxf(v, dpp<kXor2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  return fmaxf(v, dpp<kMirror>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  return v + dpp<kMirror>(v);
}

}  // namespace dg

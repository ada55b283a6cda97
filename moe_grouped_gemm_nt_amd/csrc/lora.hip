// Low-rank adapters of many requests beside a shared projection (include/dg.h):
//   d[t] = c[t] + scales[i] * B[i] . (A[i] . x[t]),   i = adapter_ids[t]
#include <hip/hip_runtime.h>

#include "../../include/dg.h"
#include "dg_host.h"
#include "expert_rows.h"

namespace dg {
namespace {

constexpr int kMaxRank = 256;

struct LoraParams {
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const float* scales;
  const int32_t* ids;
  const uint16_t* c;
  uint16_t* d;
  int ldx, ldc, ldd;
  int T, N, K, R, L;
};

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf16_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ uint16_t f32_bf16(float x) {
  __bf16 h = static_cast<__bf16>(x);
  return __builtin_bit_cast(uint16_t, h);
}

// One workgroup per token.
__global__ __launch_bounds__(256) void lora_kernel(LoraParams p) {
  __shared__ float h[kMaxRank];
  const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int id = p.ids[t];
  const bool has = id >= 0 && id < p.L;
  if (has) {
    const float scale = p.scales ? p.scales[id] : 1.0f;
    for (int r = wave; r < p.R; r += 4) {
      const uint16_t* a = p.a + ((size_t)id * p.R + r) * p.K;
      float sum = 0.0f;
      for (int k = lane * 8; k < p.K; k += 512) {
        const u16x8 u = *reinterpret_cast<const u16x8*>(a + k);
        const u16x8 v = *reinterpret_cast<const u16x8*>(p.x + (size_t)t * p.ldx + k);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(bf16_f32(u[j]), bf16_f32(v[j]), sum);
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
      if (lane == 0) h[r] = sum * scale;
    }
  }
  __syncthreads();
  for (int n = threadIdx.x; n < p.N; n += 256) {
    float sum = p.c ? bf16_f32(p.c[(size_t)t * p.ldc + n]) : 0.0f;
    if (has) {
      const uint16_t* b = p.b + ((size_t)id * p.N + n) * p.R;
      for (int r = 0; r < p.R; r += 8) {
        const u16x8 v = *reinterpret_cast<const u16x8*>(b + r);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(bf16_f32(v[j]), h[r + j], sum);
      }
    }
    p.d[(size_t)t * p.ldd + n] = f32_bf16(sum);
  }
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" int dg_lora_bf16_nt(const void* x, int ldx, const void* a, const void* b, const float* scales,
                               const int32_t* adapter_ids, const void* c, int ldc, void* d, int ldd, int T, int N,
                               int K, int R, int num_adapters, void* stream) {
  if (T < 0 || N < 0 || K < 0 || R < 0) return fail(DG_ERR_INVALID_ARG, "negative size (T=%d N=%d K=%d R=%d)", T, N, K, R);
  if (num_adapters < 0) return fail(DG_ERR_INVALID_ARG, "num_adapters=%d must not be negative", num_adapters);
  if (K % 128 != 0) return fail(DG_ERR_INVALID_ARG, "K=%d is not a multiple of 128", K);
  if (R % 8 != 0) return fail(DG_ERR_INVALID_ARG, "R=%d is not a multiple of 8", R);
  if (R > kMaxRank) return fail(DG_ERR_UNSUPPORTED, "R=%d exceeds %d", R, kMaxRank);
  if (num_adapters > kMaxLayoutGroups)
    return fail(DG_ERR_UNSUPPORTED, "num_adapters=%d exceeds %d", num_adapters, kMaxLayoutGroups);
  if (T == 0 || N == 0) return DG_OK;
  if (!adapter_ids || !d) return fail(DG_ERR_INVALID_ARG, "adapter_ids and d must not be NULL");
  const bool terms = num_adapters > 0 && K > 0 && R > 0;     // without them d = c
  if (terms && (!x || !a || !b)) return fail(DG_ERR_INVALID_ARG, "x, a and b must not be NULL");
  if (terms && (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16)))
    return fail(DG_ERR_INVALID_ARG, "x, a and b must be 16-byte aligned");
  if (terms && (ldx < K || ldx % 8 != 0))
    return fail(DG_ERR_INVALID_ARG, "ldx=%d must be a multiple of 8 and at least K=%d", ldx, K);
  if (ldd < N || (c && ldc < N)) return fail(DG_ERR_INVALID_ARG, "ldc=%d and ldd=%d must be at least N=%d", ldc, ldd, N);
  if (c == d && ldc != ldd) return fail(DG_ERR_INVALID_ARG, "c may equal d only with ldc=%d equal to ldd=%d", ldc, ldd);
  if (!aligned(d, 2) || !aligned(c, 2) || !aligned(scales, 4) || !aligned(adapter_ids, 4))
    return fail(DG_ERR_INVALID_ARG, "c and d must be 2-byte, scales and adapter_ids 4-byte aligned");
  LoraParams p{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b),
               scales, adapter_ids, static_cast<const uint16_t*>(c), static_cast<uint16_t*>(d), ldx, ldc, ldd, T, N, K,
               R, terms ? num_adapters : 0};
  lora_kernel<<<T, 256, 0, static_cast<hipStream_t>(stream)>>>(p);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

// Routing to experts: scores, expert groups, top-k and weights, and the
// gradient of the weights with respect to the logits (include/dg.h).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <climits>

#include "../../include/dg.h"
#include "dg_host.h"

namespace dg {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kMaxExpertGroups = 64;
constexpr int WAVES = 4;                 // tokens per workgroup, one wave each

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  const float* grad_weights;
  void* grad_logits;
  int T, E, top_k;
  int num_groups, topk_groups, group_top;
  int renormalize;
  float scale;
};

// e^x as 2^(x log2 e) with the product's rounding carried along: relative error
// below 2e-7 at any x the scores use (the bare product loses |x| units of the
// last place).
__device__ __forceinline__ float exp_f32(float x) {
  const float log2e = 1.44269502f, log2e_lo = 1.92596303e-8f, ln2 = 0.693147182f;
  const float hi = x * log2e;
  const float lo = fmaf(x, log2e_lo, fmaf(x, log2e, -hi));
  const float r = __builtin_amdgcn_exp2f(hi);
  const float c = fmaf(r * ln2, lo, r);
  return hi < -126.0f ? (hi < -150.0f ? 0.0f : exp2f(hi)) : (hi > 127.9f ? INFINITY : c);
}

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + exp_f32(-x)); }

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

// The highest value of the wave and the lowest index that has it.
__device__ __forceinline__ void wave_argmax(float& v, int& at) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float w = __shfl_xor(v, o);
    const int j = __shfl_xor(at, o);
    const bool take = w > v || (w == v && j < at);
    v = take ? w : v;
    at = take ? j : at;
  }
}

// One wave per token; lane l holds experts l, l + 64, ...
template <int NI, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(64 * WAVES) void route_kernel(RouteParams p) {
  __shared__ float lds_key[WAVES][NI * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned t = blockIdx.x * WAVES + wave;
  const bool live = t < (unsigned)p.T;
  const size_t row = (size_t)(live ? t : 0) * p.E;
  float s[NI], key[NI];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    s[i] = e < p.E ? clean_logit(raw_logit<BF16>(p.logits, row + e)) : -INFINITY;
    key[i] = s[i];
    top = fmaxf(top, s[i]);
  }
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < NI; ++i) s[i] = sigmoid_f32(s[i]);
  } else {
    top = wave_max(top);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      s[i] = s[i] > -INFINITY ? exp_f32(s[i] - top) : 0.0f;
      total += s[i];
    }
    total = wave_sum(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) s[i] *= inv;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    float v = e < p.E && p.bias ? s[i] + p.bias[e] : s[i];
    key[i] = key[i] > -INFINITY && v > -INFINITY ? v : -INFINITY;    // NaN compares false
  }
  if (p.num_groups > 1) {
#pragma unroll
    for (int i = 0; i < NI; ++i) lds_key[wave][lane + 64 * i] = key[i];
    __syncthreads();
    const int per = p.E / p.num_groups;
    float a = -INFINITY, b = -INFINITY;          // the group's two highest keys
    if (lane < p.num_groups)
      for (int j = 0; j < per; ++j) {
        const float v = lds_key[wave][lane * per + j];
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
    float g = p.group_top > 1 && b > -INFINITY ? a + b : a;
    uint64_t kept = 0;
    for (int n = 0; n < p.topk_groups; ++n) {
      float v = (kept >> lane) & 1 || lane >= p.num_groups ? -INFINITY : g;
      int at = (kept >> lane) & 1 || lane >= p.num_groups ? INT_MAX : lane;
      wave_argmax(v, at);
      if (v == -INFINITY) break;
      kept |= 1ull << at;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = lane + 64 * i;
      if (e < p.E && !((kept >> (e / per)) & 1)) key[i] = -INFINITY;
    }
  }
  float mine = 0.0f, total = 0.0f;               // lane j keeps the j-th choice
  int mine_id = -1;
  for (int j = 0; j < p.top_k; ++j) {
    float v = -INFINITY;
    int at = INT_MAX;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (key[i] > v) {
        v = key[i];
        at = lane + 64 * i;
      }
    wave_argmax(v, at);
    if (v == -INFINITY) break;                   // nothing left: the remaining slots stay empty
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (at == lane + 64 * i) {
        w = s[i];
        key[i] = -INFINITY;
      }
    w = __shfl(w, at & 63);
    total += w;
    if (lane == j) {
      mine = w;
      mine_id = at;
    }
  }
  if (live && lane < p.top_k) {
    float w = p.scale * mine;
    if (p.renormalize) w = total > 0.0f ? p.scale * (mine / total) : 0.0f;
    p.ids[(size_t)t * p.top_k + lane] = mine_id;
    p.weights[(size_t)t * p.top_k + lane] = mine_id >= 0 ? w : 0.0f;
  }
}

// Gradient: with w_j = scale * s_j (/ sum of the chosen s) and u_j = g_j * w_j,
//   renormalised:  u_j -= (w_j / scale) * sum_i u_i
//   sigmoid:       dx_j = u_j * (1 - s_j), 0 elsewhere   (d log sigmoid = 1 - sigmoid)
//   softmax:       dx_i = [i chosen] u_i - p_i * sum_j u_j   (the sum is 0 when renormalised)
// One wave per token, lane j on the j-th choice; the chosen terms go through LDS.
template <int NI, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(64 * WAVES) void route_backward_kernel(RouteParams p) {
  __shared__ float lds_u[WAVES][NI * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned t = blockIdx.x * WAVES + wave;
  const bool live = t < (unsigned)p.T;
  const size_t row = (size_t)(live ? t : 0) * p.E;
  float x[NI];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < p.E ? clean_logit(raw_logit<BF16>(p.logits, row + e)) : -INFINITY;
    top = fmaxf(top, x[i]);
    lds_u[wave][lane + 64 * i] = 0.0f;
  }
  float inv = 0.0f;
  if constexpr (!SIGMOID) {
    top = wave_max(top);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      x[i] = x[i] > -INFINITY ? exp_f32(x[i] - top) : 0.0f;
      total += x[i];
    }
    total = wave_sum(total);
    inv = total > 0.0f ? 1.0f / total : 0.0f;
  }
  int id = -1;
  float s = 0.0f, g = 0.0f;
  if (live && lane < p.top_k) {
    id = p.ids[(size_t)t * p.top_k + lane];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      const float xi = clean_logit(raw_logit<BF16>(p.logits, row + id));
      if (xi > -INFINITY) {
        s = SIGMOID ? sigmoid_f32(xi) : exp_f32(xi - top) * inv;
        g = p.grad_weights[(size_t)t * p.top_k + lane] * p.scale;
      }
    }
  }
  float share = s;                                // w_j / scale
  if (p.renormalize) {
    const float total = wave_sum(s);
    share = total > 0.0f ? s / total : 0.0f;
  }
  float u = s > 0.0f ? g * share : 0.0f;
  const float sum = wave_sum(u);
  if (p.renormalize) u -= share * sum;
  __syncthreads();
  if (id >= 0) lds_u[wave][id] = SIGMOID ? u * (1.0f - s) : u;
  __syncthreads();
  if (!live) return;
  const float back = !SIGMOID && !p.renormalize ? sum : 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    if (e >= p.E) continue;
    float d = lds_u[wave][e];
    if constexpr (!SIGMOID) d -= x[i] * inv * back;
    if constexpr (BF16)
      static_cast<__bf16*>(p.grad_logits)[row + e] = static_cast<__bf16>(d);
    else
      static_cast<float*>(p.grad_logits)[row + e] = d;
  }
}

template <bool BACK, int NI, bool BF16>
void launch_score(const RouteParams& p, int score, int grid, hipStream_t st) {
  if constexpr (BACK) {
    if (score == DG_SCORE_SIGMOID)
      route_backward_kernel<NI, BF16, true><<<grid, 64 * WAVES, 0, st>>>(p);
    else
      route_backward_kernel<NI, BF16, false><<<grid, 64 * WAVES, 0, st>>>(p);
  } else {
    if (score == DG_SCORE_SIGMOID)
      route_kernel<NI, BF16, true><<<grid, 64 * WAVES, 0, st>>>(p);
    else
      route_kernel<NI, BF16, false><<<grid, 64 * WAVES, 0, st>>>(p);
  }
}

template <bool BACK>
int launch_route(const RouteParams& p, int logits_type, int score, hipStream_t st) {
  const int grid = (int)((p.T + (long long)WAVES - 1) / WAVES);
  const bool bf = logits_type == DG_BF16;
#define DG_ROUTE_CASE(NI)                                   \
  if (p.E <= 64 * (NI)) {                                   \
    if (bf)                                                 \
      launch_score<BACK, NI, true>(p, score, grid, st);     \
    else                                                    \
      launch_score<BACK, NI, false>(p, score, grid, st);    \
  } else
  DG_ROUTE_CASE(1) DG_ROUTE_CASE(2) DG_ROUTE_CASE(4) DG_ROUTE_CASE(8) DG_ROUTE_CASE(16) {}
#undef DG_ROUTE_CASE
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
  return DG_OK;
}

int check_route(const void* logits, int logits_type, int T, int E, int top_k, int score) {
  if (logits_type != DG_F32 && logits_type != DG_BF16)
    return fail(DG_ERR_INVALID_ARG, "logits_type=%d is neither DG_F32 nor DG_BF16", logits_type);
  if (score != DG_SCORE_SOFTMAX && score != DG_SCORE_SIGMOID)
    return fail(DG_ERR_INVALID_ARG, "score=%d is neither DG_SCORE_SOFTMAX nor DG_SCORE_SIGMOID", score);
  if (T < 0) return fail(DG_ERR_INVALID_ARG, "negative size (T=%d)", T);
  if (E < 1 || top_k < 1 || top_k > E)
    return fail(DG_ERR_INVALID_ARG, "top_k=%d must lie in [1, E=%d]", top_k, E);
  if (E > kMaxExperts || top_k > kMaxTopK)
    return fail(DG_ERR_UNSUPPORTED, "E=%d or top_k=%d exceeds %d experts and %d choices", E, top_k, kMaxExperts,
                kMaxTopK);
  if (T > 0 && !logits) return fail(DG_ERR_INVALID_ARG, "logits must not be NULL");
  if (!aligned(logits, logits_type == DG_F32 ? 4 : 2))
    return fail(DG_ERR_INVALID_ARG, "logits must be aligned to their type");
  return DG_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" int dg_route_topk(const void* logits, int logits_type, const float* bias, int32_t* topk_ids,
                             float* topk_weights, int T, int E, int top_k, int score, int num_groups, int topk_groups,
                             int group_top, int renormalize, float scale, void* stream) {
  int s = check_route(logits, logits_type, T, E, top_k, score);
  if (s != DG_OK) return s;
  if (num_groups < 1 || E % num_groups != 0)
    return fail(DG_ERR_INVALID_ARG, "num_groups=%d must divide E=%d", num_groups, E);
  if (num_groups > kMaxExpertGroups)
    return fail(DG_ERR_UNSUPPORTED, "num_groups=%d exceeds %d", num_groups, kMaxExpertGroups);
  if (topk_groups < 1 || topk_groups > num_groups)
    return fail(DG_ERR_INVALID_ARG, "topk_groups=%d must lie in [1, num_groups=%d]", topk_groups, num_groups);
  if (group_top != 1 && group_top != 2) return fail(DG_ERR_INVALID_ARG, "group_top=%d is neither 1 nor 2", group_top);
  if (top_k > topk_groups * (E / num_groups))
    return fail(DG_ERR_INVALID_ARG, "top_k=%d exceeds the %d experts of %d groups", top_k,
                topk_groups * (E / num_groups), topk_groups);
  if (T > 0 && (!topk_ids || !topk_weights))
    return fail(DG_ERR_INVALID_ARG, "topk_ids and topk_weights must not be NULL");
  if (!aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(bias, 4))
    return fail(DG_ERR_INVALID_ARG, "bias, topk_ids and topk_weights must be 4-byte aligned");
  if (T == 0) return DG_OK;
  RouteParams p{};
  p.logits = logits;
  p.bias = bias;
  p.ids = topk_ids;
  p.weights = topk_weights;
  p.T = T;
  p.E = E;
  p.top_k = top_k;
  p.num_groups = topk_groups == num_groups ? 1 : num_groups;     // every group stays: no group step
  p.topk_groups = topk_groups;
  p.group_top = group_top;
  p.renormalize = renormalize;
  p.scale = scale;
  return launch_route<false>(p, logits_type, score, static_cast<hipStream_t>(stream));
}

extern "C" int dg_route_topk_backward(const void* logits, int logits_type, const int32_t* topk_ids,
                                      const float* grad_weights, void* grad_logits, int T, int E, int top_k, int score,
                                      int renormalize, float scale, void* stream) {
  int s = check_route(logits, logits_type, T, E, top_k, score);
  if (s != DG_OK) return s;
  if (T > 0 && (!topk_ids || !grad_weights || !grad_logits))
    return fail(DG_ERR_INVALID_ARG, "topk_ids, grad_weights and grad_logits must not be NULL");
  if (!aligned(topk_ids, 4) || !aligned(grad_weights, 4) || !aligned(grad_logits, logits_type == DG_F32 ? 4 : 2))
    return fail(DG_ERR_INVALID_ARG, "topk_ids, grad_weights and grad_logits must be aligned to their types");
  if (T == 0) return DG_OK;
  RouteParams p{};
  p.logits = logits;
  p.ids = const_cast<int32_t*>(topk_ids);
  p.grad_weights = grad_weights;
  p.grad_logits = grad_logits;
  p.T = T;
  p.E = E;
  p.top_k = top_k;
  p.renormalize = renormalize;
  p.scale = scale;
  return launch_route<true>(p, logits_type, score, static_cast<hipStream_t>(stream));
}

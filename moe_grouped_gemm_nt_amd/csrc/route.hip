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

// The sum of the other lanes' values, added up as such: not a total less this
// lane's value, which has no digits left where that is nearly all of it.
__device__ __forceinline__ float wave_others(float v) {
  float others = 0.0f;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float w = __shfl_xor(v, o);
    others += w;
    v += w;
  }
  return others;
}

// The sum of a group's two highest keys: as an fp32 sum, but without its range, so
// that two keys of the lowest finite value still have a score (-inf would mask the
// group) and two of the highest do not tie with +inf.
__device__ __forceinline__ double group_sum(float a, float b) {
  uint64_t u = __builtin_bit_cast(uint64_t, (double)a + (double)b);    // exact but for bits that 24 do not see
  u += 0x0FFFFFFF + ((u >> 29) & 1);                                   // to nearest even at fp32's last place
  return __builtin_bit_cast(double, u & ~0x1FFFFFFFull);
}

// The highest value of the wave and the lowest index that has it.
template <typename F>
__device__ __forceinline__ void wave_argmax(F& v, int& at) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const F w = __shfl_xor(v, o);
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
    for (int i = 0; i < NI; ++i) s[i] = sigmoid_any(s[i]);
  } else {
    top = wave_max(top);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      s[i] = s[i] > -INFINITY ? exp_any(s[i] - top) : 0.0f;
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
    const double g = p.group_top > 1 && b > -INFINITY ? group_sum(a, b) : a;
    uint64_t kept = 0;
    for (int n = 0; n < p.topk_groups; ++n) {
      double v = (kept >> lane) & 1 || lane >= p.num_groups ? -INFINITY : g;
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

// Gradient: with the chosen scores' shares r_j = s_j (/ sum of the chosen s) and g_j
// the weights' gradients times scale,
//   renormalised:  u_j = r_j (g_j sum_{i != j} r_i - sum_{i != j} r_i g_i)
//   otherwise:     u_j = s_j g_j
//   sigmoid:       dx_j = u_j * sigmoid(-x_j), 0 elsewhere   (d log sigmoid(x) = 1 - sigmoid(x))
//   softmax:       renormalised dx_j = u_j, 0 elsewhere; otherwise, p the softmax,
//                  dx_j = p_j (g_j (1 - p_j) - sum_{i != j} p_i g_i) for the chosen,
//                  dx_e = -p_e sum_i p_i g_i elsewhere
// What a share leaves is summed from the others' (1 - p_j from p_j = 3/4 on, from
// the p up to 1/2), not subtracted from 1: where one choice takes nearly all, a
// difference has no digits left.
// The experts without a term of their own bear this mark, a NaN (a term that is the
// same NaN makes the sum, and so what stands for the mark, a NaN too).
constexpr uint32_t kNotChosen = 0x7FFFFFFF;
__device__ __forceinline__ float softmax_term(float s, float g, float rest, float others) {
  const float less = s > 0.75f ? rest : 1.0f - s;
  return s > 0.0f ? s * (g * less - others) : 0.0f;
}
// One wave per token, lane j on the j-th choice; the chosen terms go through LDS.
template <int NI, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(64 * WAVES) void route_backward_kernel(RouteParams p) {
  __shared__ float lds_u[WAVES][NI * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned t = blockIdx.x * WAVES + wave;
  const bool live = t < (unsigned)p.T;
  const size_t row = (size_t)(live ? t : 0) * p.E;
  const bool spread = !SIGMOID && !p.renormalize;        // every expert has a gradient
  float x[NI];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < p.E ? clean_logit(raw_logit<BF16>(p.logits, row + e)) : -INFINITY;
    top = fmaxf(top, x[i]);
    lds_u[wave][lane + 64 * i] = spread ? __uint_as_float(kNotChosen) : 0.0f;
  }
  float inv = 0.0f;
  if constexpr (!SIGMOID) {
    top = wave_max(top);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      x[i] = x[i] > -INFINITY ? exp_any(x[i] - top) : 0.0f;
      total += x[i];
    }
    total = wave_sum(total);
    inv = total > 0.0f ? 1.0f / total : 0.0f;
  }
  int id = -1;
  float s = 0.0f, g = 0.0f, xi = -INFINITY;
  if (live && lane < p.top_k) {
    id = p.ids[(size_t)t * p.top_k + lane];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      xi = clean_logit(raw_logit<BF16>(p.logits, row + id));
      if (xi > -INFINITY) {
        s = SIGMOID ? sigmoid_any(xi) : exp_any(xi - top) * inv;
        g = p.grad_weights[(size_t)t * p.top_k + lane] * p.scale;
      }
    }
  }
  float u = s > 0.0f ? g * s : 0.0f, sum = 0.0f;
  if (p.renormalize) {
    const float total = wave_sum(s);
    const float share = total > 0.0f ? s / total : 0.0f;
    const float less = wave_others(share), others = wave_others(s > 0.0f ? g * share : 0.0f);
    u = s > 0.0f ? share * (g * less - others) : 0.0f;
  } else if (spread) {
    float rest = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) rest += x[i] * inv <= 0.5f ? x[i] * inv : 0.0f;
    rest = wave_sum(rest);
    sum = wave_sum(u);
    u = softmax_term(s, g, rest, wave_others(u));
  }
  __syncthreads();
  if (id >= 0) lds_u[wave][id] = SIGMOID ? u * sigmoid_any(-xi) : u;
  __syncthreads();
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    if (e >= p.E) continue;
    float d = lds_u[wave][e];
    if constexpr (!SIGMOID) d = spread && __float_as_uint(d) == kNotChosen ? fmaf(-x[i] * inv, sum, 0.0f) : d;
    if constexpr (BF16)
      static_cast<__bf16*>(p.grad_logits)[row + e] = static_cast<__bf16>(d);
    else
      static_cast<float*>(p.grad_logits)[row + e] = d;
  }
}

// ---- the common sizes: sixteen lanes per token -------------------------------
// A key and its expert in one double: the fp32 key's value with the expert's
// index in low mantissa bits that the conversion leaves empty, so that doubles
// compare as (key, lowest index first) and no two are equal.  A comparison and
// exchange is then one v_max_f64 and one v_min_f64, which run at the rate of
// their fp32 forms here.
constexpr int kIndexBits = 11;

// max and min without the quieting of NaN that the C functions imply (keys are none)
__device__ __forceinline__ double max_f64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min_f64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

template <typename F>                    // float, or a group's score
__device__ __forceinline__ double pack_key(F key, int e) {
  const int rest = (1 << kIndexBits) - 1;
  // a lower index is greater: nearer to zero for negative keys, farther for others
  const int low = key < F(0) ? e : rest - e;
  const double d = min_f64((double)(key + F(0)), 0x1p130);        // -0 is 0; +inf is a finite value above all others
  const uint64_t u = __builtin_bit_cast(uint64_t, d) | (uint64_t)low;
  return key > -INFINITY ? __builtin_bit_cast(double, u) : -INFINITY;
}
__device__ __forceinline__ int key_index(double d) {
  const int low = (int)(__builtin_bit_cast(uint64_t, d) & ((1 << kIndexBits) - 1));
  return d < 0.0 ? low : (1 << kIndexBits) - 1 - low;
}

// DPP controls that pair the sixteen lanes of a row in four steps
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double row_max(double v) {
  v = max_f64(v, dpp<kXor1>(v));
  v = max_f64(v, dpp<kXor2>(v));
  v = max_f64(v, dpp<kHalfMirror>(v));
  return max_f64(v, dpp<kMirror>(v));
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

__device__ __forceinline__ float row_others(float v) {             // as wave_others, of sixteen lanes
  float w = dpp<kXor1>(v), others = w;
  v += w;
  w = dpp<kXor2>(v);
  others += w;
  v += w;
  w = dpp<kHalfMirror>(v);
  others += w;
  v += w;
  return others + dpp<kMirror>(v);
}

__device__ __forceinline__ void order(double& a, double& b) {     // a >= b afterwards
  const double hi = max_f64(a, b), lo = min_f64(a, b);
  a = hi;
  b = lo;
}

// Sorts v[LO .. LO + N) falling (N a power of two): Batcher's sort by merging odd
// and even positions.
template <int LO, int N, int R>
__device__ __forceinline__ void merge_falling(double* v) {
  if constexpr (2 * R < N) {
    merge_falling<LO, N, 2 * R>(v);
    merge_falling<LO + R, N, 2 * R>(v);
#pragma unroll
    for (int i = LO + R; i + R < LO + N; i += 2 * R) order(v[i], v[i + R]);
  } else {
    order(v[LO], v[LO + R]);
  }
}
template <int LO, int N>
__device__ __forceinline__ void sort_falling(double* v) {
  if constexpr (N > 1) {
    sort_falling<LO, N / 2>(v);
    sort_falling<LO + N / 2, N / 2>(v);
    merge_falling<LO, N, 1>(v);
  }
}

// The D highest of N values, sorted falling, into v[0..D): runs of D are sorted
// and merged; of two falling runs the D highest are max(a[i], b[D-1-i]), a
// rising-falling sequence that log2 D rounds put in order.
template <int N, int D>
__device__ __forceinline__ void top_falling(double* v) {
#pragma unroll
  for (int r = 0; r < N; r += D) sort_falling<0, D>(v + r);
#pragma unroll
  for (int r = D; r < N; r += D) {
#pragma unroll
    for (int i = 0; i < D; ++i) v[i] = max_f64(v[i], v[r + D - 1 - i]);
#pragma unroll
    for (int h = D / 2; h >= 1; h >>= 1)
#pragma unroll
      for (int i = 0; i < D; ++i)
        if ((i & h) == 0) order(v[i], v[i + h]);
  }
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef u16x4 u16x4_any __attribute__((aligned(2)));

// Sixteen lanes per token: lane l's logits, experts q * 64 + 4 l + i in x[4 q + i]
// (-inf for masked ones and beyond E).
template <bool BF16, int NI>
__device__ __forceinline__ void load16(const void* logits, size_t row, int E, int lane, float (&x)[NI]) {
#pragma unroll
  for (int q = 0; q < NI / 4; ++q) {
    const int e = q * 64 + lane * 4;
    if (e + 4 <= E) {
      if constexpr (BF16) {
        const u16x4 h = *reinterpret_cast<const u16x4_any*>(static_cast<const uint16_t*>(logits) + row + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * q + i] = __uint_as_float((uint32_t)h[i] << 16);
      } else {
        const f32x4 h = *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(logits) + row + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * q + i] = h[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * q + i] = e + i < E ? raw_logit<BF16>(logits, row + e + i) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) x[i] = clean_logit(x[i]);
}

// y[i] = e^(x[i] - top) again where that is below the normal range, in the waves
// that hold such a value (masked ones aside).  Counted from -inf's, the bits of a
// finite negative number are the greater the lower it is and above all others', so
// that one maximum finds the lowest (router of 64 tokens: 5.8 us against 6.0 with a
// comparison per value, 5.7 with neither).
template <int NI>
__device__ __forceinline__ void mend_below(const float (&x)[NI], float top, float (&y)[NI]) {
  auto mark = [](float v) { return __float_as_uint(v) - __float_as_uint(-INFINITY); };
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) most = max(most, mark(x[i] - top));
  if (__builtin_expect(__any(most > mark(kLeastNormal)), 0))
#pragma unroll
    for (int i = 0; i < NI; ++i) y[i] = x[i] - top < kLeastNormal ? exp_below(x[i] - top) : y[i];
}

// y = softmax(x) of the sixteen lanes' values; top and inv, the sum's reciprocal, for single values.
template <int NI>
__device__ __forceinline__ void softmax16(const float (&x)[NI], float (&y)[NI], float& top, float& inv) {
  top = x[0];
#pragma unroll
  for (int i = 1; i < NI; ++i) top = fmaxf(top, x[i]);
  top = row_max(top);
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    y[i] = x[i] > -INFINITY ? exp_f32(x[i] - top) : 0.0f;
    total += y[i];
  }
  mend_below(x, top, y);                 // the sum is at least 1: it does not see them
  total = row_sum(total);
  inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) y[i] *= inv;
}

// Sixteen lanes per token, four tokens per wave: lane l holds experts
// q * 64 + 4 l .. + 3, so that the sixteen read 256 (or, bf16, 128) contiguous
// bytes at a time and a lane's four neighbours are of one group (the groups'
// size is a multiple of 4 here).  Each lane sorts its own keys down to the D
// highest; a choice is then the highest head of the sixteen lists, four DPP
// steps, and its owner's list moves up.  Bound by the VALU at many tokens (16384
// tokens, 256 experts in 8 groups, 8 choices: 11.3 us, 1.5 TB/s; 1265 VALU
// instructions per wave fill four fifths of the SIMDs' cycles; one wave per token
// that searches all its keys for every choice took 44) and by the chain of loads
// and dependent instructions at few (64 tokens: 5.8 us, a third of it VALU issue;
// one wave per token took 11.9).
template <int NI, int D, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(256) void route16_kernel(RouteParams p) {
  constexpr int Q = NI / 4;
  __shared__ float2 lds_pair[16][16 * Q];      // [token of the workgroup][quad of experts]
  const int lane = threadIdx.x & 15, local = threadIdx.x >> 4;
  const size_t t = (size_t)blockIdx.x * 16 + local;
  const bool live = t < (size_t)p.T;
  const size_t row = (live ? t : (size_t)p.T - 1) * p.E;
  float s[NI];
  load16<BF16>(p.logits, row, p.E, lane, s);
  float top = 0.0f, inv = 1.0f, keys[NI];
  double v[NI];
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < NI; ++i) keys[i] = sigmoid_f32(s[i]);
    mend_below(s, 0.0f, keys);
  } else {
    softmax16(s, keys, top, inv);
  }
  if (p.bias) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = q * 64 + lane * 4;
      f32x4 b;
      if (e + 4 <= p.E)
        b = *reinterpret_cast<const f32x4_any*>(p.bias + e);
      else
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = e + i < p.E ? p.bias[e + i] : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) keys[4 * q + i] += b[i];
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)                       // NaN compares false
    keys[i] = s[i] > -INFINITY && keys[i] > -INFINITY ? keys[i] : -INFINITY;
  if (p.num_groups > 1) {
    const int per4 = p.E / p.num_groups / 4;         // quads per group
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float a = fmaxf(keys[4 * q], keys[4 * q + 1]), b = fminf(keys[4 * q], keys[4 * q + 1]);
      const float c = fmaxf(keys[4 * q + 2], keys[4 * q + 3]), d = fminf(keys[4 * q + 2], keys[4 * q + 3]);
      b = fmaxf(fminf(a, c), fmaxf(b, d));
      a = fmaxf(a, c);
      lds_pair[local][q * 16 + lane] = make_float2(a, b);
    }
    // the same wave wrote what these lanes read
    __builtin_amdgcn_wave_barrier();
    float a = -INFINITY, b = -INFINITY;
    if (lane < p.num_groups)
      for (int j = 0; j < per4; ++j) {
        const float2 c = lds_pair[local][lane * per4 + j];
        b = fmaxf(fminf(a, c.x), fmaxf(b, c.y));
        a = fmaxf(a, c.x);
      }
    const double sum = p.group_top > 1 && b > -INFINITY ? group_sum(a, b) : a;
    const double g = pack_key(lane < p.num_groups ? sum : -INFINITY, lane);
    // a group's place is the number of groups above it
    int above = 0;
    double other = g;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      other = dpp<0x121>(other);                     // the row turned by one lane
      above += other > g ? 1 : 0;
    }
    const uint64_t ballot = __ballot(above < p.topk_groups && g > -INFINITY);
    const uint32_t kept = (uint32_t)(ballot >> (threadIdx.x & 48)) & 0xFFFF;
    const uint32_t magic = 65536 / per4 + 1;         // quad / per4 for quads below 256
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint32_t group = ((uint32_t)(q * 16 + lane) * magic) >> 16;
      const bool in = (kept >> (group & 15)) & 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) keys[4 * q + i] = in ? keys[4 * q + i] : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) v[i] = pack_key(keys[i], (i >> 2) * 64 + lane * 4 + (i & 3));
  top_falling<NI, D>(v);
  double mine = -INFINITY;                           // lane j keeps the j-th choice
  for (int j = 0; j < p.top_k; ++j) {
    const double m = row_max(v[0]);
    if (lane == j) mine = m;
    const bool owner = v[0] == m;                    // keys differ, except where nothing is left
#pragma unroll
    for (int i = 0; i + 1 < D; ++i) {
      double next = v[i + 1];
      asm("" : "+v"(next));                          // two selects, and not a load at a selected index
      v[i] = owner ? next : v[i];
    }
    v[D - 1] = owner ? -INFINITY : v[D - 1];
  }
  const bool chosen = mine > -INFINITY;
  const int id = chosen ? key_index(mine) : -1;
  float w = 0.0f;
  if (chosen) {
    const float x = clean_logit(raw_logit<BF16>(p.logits, row + id));
    w = SIGMOID ? sigmoid_any(x) : exp_any(x - top) * inv;
  }
  if (p.renormalize) {
    const float total = row_sum(w);
    w = total > 0.0f ? w / total : 0.0f;
  }
  if (live && lane < p.top_k) {
    p.ids[t * p.top_k + lane] = id;
    p.weights[t * p.top_k + lane] = p.scale * w;
  }
}

// The gradient, sixteen lanes per token (formulas at route_backward_kernel): lane j
// on the j-th choice, whose term reaches the expert's lane through LDS.  Softmax
// over 60 bf16 logits of 20479 tokens: 4.5 us, of which the bytes need 1.1 and a
// launch about 2; one wave per token took 9.8.
template <int NI, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(256) void route16_backward_kernel(RouteParams p) {
  __shared__ f32x4 lds_u[16][NI * 4];          // [token of the workgroup][quad of experts]
  const int lane = threadIdx.x & 15, local = threadIdx.x >> 4;
  const size_t t = (size_t)blockIdx.x * 16 + local;
  const bool live = t < (size_t)p.T;
  const size_t row = (live ? t : (size_t)p.T - 1) * p.E;
  const bool spread = !SIGMOID && !p.renormalize;        // every expert has a gradient
  const float blank = spread ? __uint_as_float(kNotChosen) : 0.0f;
#pragma unroll
  for (int q = 0; q < NI / 4; ++q) lds_u[local][q * 16 + lane] = f32x4{blank, blank, blank, blank};
  int id = -1;
  float g = 0.0f, xi = -INFINITY;
  if (live && lane < p.top_k) {
    id = p.ids[t * p.top_k + lane];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      xi = clean_logit(raw_logit<BF16>(p.logits, row + id));
      g = p.grad_weights[t * p.top_k + lane] * p.scale;
    }
  }
  // a renormalised sigmoid needs the chosen logits only
  float y[NI], top = 0.0f, inv = 1.0f;
  if constexpr (!SIGMOID) {
    float x[NI];
    load16<BF16>(p.logits, row, p.E, lane, x);
    softmax16(x, y, top, inv);
  }
  const float s = xi > -INFINITY ? (SIGMOID ? sigmoid_any(xi) : exp_any(xi - top) * inv) : 0.0f;
  float u = s > 0.0f ? g * s : 0.0f, sum = 0.0f;
  if (p.renormalize) {
    const float total = row_sum(s);
    const float share = total > 0.0f ? s / total : 0.0f;
    const float less = row_others(share), others = row_others(s > 0.0f ? g * share : 0.0f);
    u = s > 0.0f ? share * (g * less - others) : 0.0f;
  } else if constexpr (!SIGMOID) {
    float rest = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) rest += y[i] <= 0.5f ? y[i] : 0.0f;
    rest = row_sum(rest);
    sum = row_sum(u);
    u = softmax_term(s, g, rest, row_others(u));
  }
  // one wave writes and reads a token's words: program order is enough
  __builtin_amdgcn_wave_barrier();
  if (id >= 0) reinterpret_cast<float*>(&lds_u[local][0])[id] = SIGMOID ? u * sigmoid_any(-xi) : u;
  __builtin_amdgcn_wave_barrier();
  if (!live) return;
#pragma unroll
  for (int q = 0; q < NI / 4; ++q) {
    const int e = q * 64 + lane * 4;
    if (e >= p.E) continue;
    f32x4 d = lds_u[local][q * 16 + lane];
    if constexpr (!SIGMOID)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = spread && __float_as_uint(d[i]) == kNotChosen ? fmaf(-y[4 * q + i], sum, 0.0f) : d[i];
    if constexpr (BF16) {
      u16x4 h;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(d[i]));
      uint16_t* out = static_cast<uint16_t*>(p.grad_logits) + row + e;
      if (e + 4 <= p.E)
        *reinterpret_cast<u16x4_any*>(out) = h;
      else
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (e + i < p.E) out[i] = h[i];
    } else {
      float* out = static_cast<float*>(p.grad_logits) + row + e;
      if (e + 4 <= p.E)
        *reinterpret_cast<f32x4_any*>(out) = d;
      else
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (e + i < p.E) out[i] = d[i];
    }
  }
}

template <int NI>
void launch_route16_backward(const RouteParams& p, bool bf, int score, hipStream_t st) {
  const int grid = (int)(((long long)p.T + 15) / 16);
  if (bf) {
    if (score == DG_SCORE_SIGMOID)
      route16_backward_kernel<NI, true, true><<<grid, 256, 0, st>>>(p);
    else
      route16_backward_kernel<NI, true, false><<<grid, 256, 0, st>>>(p);
  } else {
    if (score == DG_SCORE_SIGMOID)
      route16_backward_kernel<NI, false, true><<<grid, 256, 0, st>>>(p);
    else
      route16_backward_kernel<NI, false, false><<<grid, 256, 0, st>>>(p);
  }
}

template <int NI, int D>
void launch_route16(const RouteParams& p, bool bf, int score, hipStream_t st) {
  const int grid = (int)(((long long)p.T + 15) / 16);
  if (bf) {
    if (score == DG_SCORE_SIGMOID)
      route16_kernel<NI, D, true, true><<<grid, 256, 0, st>>>(p);
    else
      route16_kernel<NI, D, true, false><<<grid, 256, 0, st>>>(p);
  } else {
    if (score == DG_SCORE_SIGMOID)
      route16_kernel<NI, D, false, true><<<grid, 256, 0, st>>>(p);
    else
      route16_kernel<NI, D, false, false><<<grid, 256, 0, st>>>(p);
  }
}

// Whether sixteen lanes per token do it: up to 512 experts (32 keys a lane), 16
// choices (one a lane), 16 groups (one a lane) of whole quads.  Other calls take
// one wave per token.
bool fits_route16(const RouteParams& p) {
  return p.E <= 512 && p.top_k <= 16 &&
         (p.num_groups == 1 || (p.num_groups <= 16 && p.E / p.num_groups % 4 == 0));
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
int launch_tokens(const RouteParams& p, bool bf, int score, hipStream_t st) {
  if (!BACK && fits_route16(p)) {
    if (p.E <= 64)
      launch_route16<4, 4>(p, bf, score, st);
    else if (p.E <= 128)
      launch_route16<8, 8>(p, bf, score, st);
    else if (p.E <= 256)
      p.top_k <= 8 ? launch_route16<16, 8>(p, bf, score, st) : launch_route16<16, 16>(p, bf, score, st);
    else
      p.top_k <= 8 ? launch_route16<32, 8>(p, bf, score, st) : launch_route16<32, 16>(p, bf, score, st);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
  }
  if (BACK && p.E <= 512 && p.top_k <= 16) {
    if (p.E <= 64)
      launch_route16_backward<4>(p, bf, score, st);
    else if (p.E <= 128)
      launch_route16_backward<8>(p, bf, score, st);
    else if (p.E <= 256)
      launch_route16_backward<16>(p, bf, score, st);
    else
      launch_route16_backward<32>(p, bf, score, st);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
  }
  const int grid = (int)((p.T + (long long)WAVES - 1) / WAVES);
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

// A grid has fewer than 2^32 threads (a launch of more is cut short without an
// error): at 64 to a token, this many tokens per launch.
constexpr int kTokensPerLaunch = 1 << 25;

template <bool BACK>
int launch_route(RouteParams p, int logits_type, int score, hipStream_t st) {
  const bool bf = logits_type == DG_BF16;
  const int T = p.T;
  for (int t = 0; t < T; t += p.T) {
    p.T = T - t < kTokensPerLaunch ? T - t : kTokensPerLaunch;
    const int s = launch_tokens<BACK>(p, bf, score, st);
    if (s != DG_OK) return s;
    const size_t logits = (size_t)p.T * p.E * (bf ? 2 : 4), choices = (size_t)p.T * p.top_k;
    p.logits = static_cast<const uint8_t*>(p.logits) + logits;
    p.ids += choices;
    if constexpr (BACK) {
      p.grad_weights += choices;
      p.grad_logits = static_cast<uint8_t*>(p.grad_logits) + logits;
    } else {
      p.weights += choices;
    }
  }
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

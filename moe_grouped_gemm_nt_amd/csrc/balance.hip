// The router's balance loss with the experts' counts, and its gradient (include/dg.h):
//   p[t] = softmax(x[t]) or sigmoid(x[t]) / sum of the token's sigmoids
//   loss[s] = a_s sum_e counts[s][e] sum_{t in s} p[t][e],  a_s = scale E / (top_k n_s^2)
//   d loss[s] / d x[t][i] = a_s p_i r_i sum_e p_e (counts_i - counts_e),
//   r_i = 1 (softmax) or sigmoid(-x_i)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>

#include "../../include/dg.h"
#include "dg_host.h"
#include "scores.h"

namespace dg {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr long long kMaxChoices = 1LL << 30;
constexpr int THREADS = 256;
// One sequence of 16384 tokens of 256 experts, 8 of them, and 131072 tokens of 128
// experts in 16 sequences (sigmoids, replayed from a graph): 17.5, 13.5 and 24 us.  256
// threads per chunk make twice the sums for the second kernel (20.3, 16.4 and 33; with
// chunks of 32 tokens 24.1, 14.8 and 33), 1024 hold more tokens back behind a barrier
// (20.0, 16.2 and 26.6; with chunks of 128 17.1, 15.3 and 26.6).
constexpr int kSumThreads = 512;
constexpr long long kSequencesPerLaunch = 1 << 20;               // workgroups of up to 1024 threads: a grid has 2^32

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_u __attribute__((aligned(4)));               // at any address of its elements
typedef i32x4 i32x4_u __attribute__((aligned(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef u16x4 u16x4_u __attribute__((aligned(2)));

struct BalanceParams {
  const void* logits;
  const int32_t* ids;
  const int32_t* starts;   // [S + 1], or nullptr: one sequence of all tokens
  const float* grad_loss;  // [S], or nullptr: ones
  const void* c;
  void* grad_logits;
  float* loss;
  int32_t* counts;         // [S][E]
  int T, E, top_k, S;
  int chunk;               // tokens per workgroup
  int first, last;         // sequences of this launch (sums)
  float* part_sums;        // [chunks + last - first][row]
  int32_t* part_counts;
  int row;                 // E rounded up to 4
  float scale;
};

// A token's experts on LPT lanes, NV groups of four to a lane: column
// (v * LPT + lane) * 4 + i.  All loads and stores are of four columns, so that a
// token's lanes cover whole lines.
template <int LPT, int NV>
constexpr int kColumns = LPT * NV * 4;

template <bool BF16>
__device__ __forceinline__ f32x4 load4(const void* p, size_t row, int col, int E, float none) {
  f32x4 v = {none, none, none, none};
  if (col + 4 <= E) {
    if constexpr (BF16) {
      const u16x4 u = *reinterpret_cast<const u16x4_u*>(static_cast<const uint16_t*>(p) + row + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float((uint32_t)u[i] << 16);
    } else {
      v = *reinterpret_cast<const f32x4_u*>(static_cast<const float*>(p) + row + col);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (col + i < E) v[i] = raw_logit<BF16>(p, row + col + i);
  }
  return v;
}

__device__ __forceinline__ int start_of(const BalanceParams& p, int s) {
  return p.starts ? min(max(p.starts[s], 0), p.T) : (s == 0 ? 0 : p.T);
}

// The first sequence that ends behind token t: the number of those that end at or
// before it.  All threads of the workgroup call it; ends with a barrier.
template <int N>
__device__ __forceinline__ int sequence_at(const BalanceParams& p, int t, int* counter) {
  if (!p.starts) return 0;
  if (threadIdx.x == 0) *counter = 0;
  __syncthreads();
  int n = 0;
  for (int s = threadIdx.x; s < p.S; s += N) n += start_of(p, s + 1) <= t ? 1 : 0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  if ((threadIdx.x & 63) == 0 && n) atomicAdd(counter, n);
  __syncthreads();
  return *counter;
}

template <int LPT>
__device__ __forceinline__ float token_max(float v) {
  v = row_max(v);
  if constexpr (LPT > 16) v = fmaxf(v, __shfl_xor(v, 16));
  if constexpr (LPT > 32) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}
template <int LPT>
__device__ __forceinline__ int token_max(int v) {
  v = row_max(v);
  if constexpr (LPT > 16) v = max(v, __shfl_xor(v, 16));
  if constexpr (LPT > 32) v = max(v, __shfl_xor(v, 32));
  return v;
}
template <int LPT>
__device__ __forceinline__ float token_sum(float v) {
  v = row_sum(v);
  if constexpr (LPT > 16) v += __shfl_xor(v, 16);
  if constexpr (LPT > 32) v += __shfl_xor(v, 32);
  return v;
}

// exp_f32 of an x <= 0
__device__ __forceinline__ float exp_neg(float x) {
  const float log2e = 1.44269502f, log2e_lo = 1.92596303e-8f, ln2 = 0.693147182f;
  x = fmaxf(x, -150.0f);
  const float hi = x * log2e;
  const float lo = fmaf(x, log2e_lo, fmaf(x, log2e, -hi));
  const float r = __builtin_amdgcn_exp2f(hi);
  return fmaf(r * ln2, lo, r);
}

// x becomes the token's scores up to a factor, whose sum's reciprocal is returned
// (0 if nothing is left): e^(x - max), or sigmoids.  Where all of a token's logits
// are negative its sigmoids are taken e^-max times as large, so that far negative
// logits keep their shares.  rest: sigmoid(-x).  Shares below 2^-126 count as 0.
template <int LPT, int NV, bool SIGMOID>
__device__ __forceinline__ float scores(f32x4 (&x)[NV], f32x4 (&rest)[NV]) {
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[v][i] = clean_logit(x[v][i]);
      top = fmaxf(top, x[v][i]);
    }
  top = token_max<LPT>(top);
  float sum = 0.0f;
  if constexpr (SIGMOID) {
    const bool far = __any(top < 0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = x[v][i], b = exp_neg(-fabsf(y)), r = __builtin_amdgcn_rcpf(1.0f + b);
        float s = y >= 0.0f ? r : b * r;
        rest[v][i] = y >= 0.0f ? b * r : r;
        if (far) s = top < 0.0f ? (y > -INFINITY ? exp_neg(y - top) * r : 0.0f) : s;
        x[v][i] = s;
        sum += s;
      }
  } else {
    top = top > -INFINITY ? top : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[v][i] = exp_neg(x[v][i] - top);
        sum += x[v][i];
      }
  }
  sum = token_sum<LPT>(sum);
  return sum > 0.0f ? 1.0f / sum : 0.0f;
}

// The workgroup's sums and counts of sequence s to their row; they are zero again
// afterwards.
template <int LPT, int NV>
__device__ __forceinline__ void write_sums(const BalanceParams& p, int s, f32x4 (*sums)[LPT * NV], int* hist,
                                           f32x4 (&acc)[NV]) {
  constexpr int ROWS = kSumThreads / LPT;
  const int lane = threadIdx.x % LPT, row = threadIdx.x / LPT;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    sums[row][v * LPT + lane] = acc[v];
    acc[v] = f32x4{};
  }
  __syncthreads();
  const size_t to = (size_t)(blockIdx.x + s - p.first) * p.row;
  for (int e = threadIdx.x; e < p.row; e += kSumThreads) {
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) sum += reinterpret_cast<const float*>(&sums[r][0])[e];
    p.part_sums[to + e] = sum;
    p.part_counts[to + e] = hist[e];
    hist[e] = 0;
  }
  __syncthreads();
}

// The tokens' shares and choices, summed per chunk of tokens and sequence: the sums
// of chunk b and sequence s stand in row b + s, which no other chunk and sequence
// share, because along the tokens one of the two grows from piece to piece.
//
// A chunk is taken in blocks of two rounds of tokens, whose logits and choices are
// loaded before anything is known of the sequences.
template <int LPT, int NV, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kSumThreads) void balance_sums_kernel(BalanceParams p) {
  constexpr int ROWS = kSumThreads / LPT;          // tokens at a time
  constexpr int BLOCK = 2 * ROWS;
  __shared__ f32x4 sums[ROWS][LPT * NV];
  __shared__ int hist[kColumns<LPT, NV>];
  __shared__ int counter;
  const int lane = threadIdx.x % LPT, row = threadIdx.x / LPT;
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T - t0, p.chunk) + t0;
  f32x4 acc[NV] = {};
  bool some = false;                           // tokens since the last sums were written
  int s = -1;
  for (int tb = t0; tb < t1; tb += BLOCK) {
    const int te = min(t1 - tb, BLOCK) + tb;
    f32x4 x[2][NV], rest[NV];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        x[h][v] = load4<BF16>(p.logits, (size_t)min(tb + h * ROWS + row, te - 1) * p.E, (v * LPT + lane) * 4, p.E,
                              -INFINITY);
    const size_t first = (size_t)tb * p.top_k + threadIdx.x;     // of the choices; most often there are no more
    const int one = first < (size_t)te * p.top_k ? p.ids[first] : -1;
    if (s < 0) {
      for (int e = threadIdx.x; e < p.row; e += kSumThreads) hist[e] = 0;
      s = max(sequence_at<kSumThreads>(p, t0, &counter), p.first);
      __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float inv = scores<LPT, NV, SIGMOID>(x[h], rest);
#pragma unroll
      for (int v = 0; v < NV; ++v) x[h][v] *= inv;
    }
    for (; s < p.last; ++s) {
      const int from = start_of(p, s), to = start_of(p, s + 1);
      if (from >= te) break;
      const int a = max(from, tb), b = min(to, te);
      if (a < b) {
        some = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = tb + h * ROWS + row;
          const bool in = t >= a && t < b;
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[v][i] += in ? x[h][v][i] : 0.0f;
        }
        const size_t low = (size_t)a * p.top_k, high = (size_t)b * p.top_k;
        for (size_t i = first; i < high; i += kSumThreads) {
          if (i < low) continue;
          const int e = i == first ? one : p.ids[i];
          if ((unsigned)e < (unsigned)p.E) atomicAdd(&hist[e], 1);
        }
      }
      if (to > te || (to == te && te < t1)) break;               // it may go on in the next block
      if (some) {
        write_sums<LPT, NV>(p, s, sums, hist, acc);
        some = false;
      }
    }
  }
  if (some) write_sums<LPT, NV>(p, s, sums, hist, acc);
}

// The sum of a value over N threads, in thread 0
template <int N>
__device__ __forceinline__ double block_sum(double v, double* parts) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) parts[threadIdx.x / 64] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < N / 64; ++w) v += parts[w];
  return v;
}

// The loss of a sequence of n tokens from total = sum_e counts_e sum_t p_e
__device__ __forceinline__ void write_loss(const BalanceParams& p, int s, int n, double total) {
  p.loss[s] = n > 0 ? (float)((double)p.scale * p.E / ((double)p.top_k * n * n) * total) : 0.0f;
}

// One workgroup per sequence: its chunks' sums and counts, and the loss.
template <int N>
__global__ __launch_bounds__(N) void balance_loss_kernel(BalanceParams p) {
  __shared__ double lds_sum[N][4];
  __shared__ int lds_count[N][4];
  __shared__ double parts[N / 64];
  const int s = p.first + blockIdx.x;
  const int a = start_of(p, s), b = start_of(p, s + 1);
  const int n = max(b - a, 0);
  const int quads = p.row / 4, rows = N / quads;
  const int q = threadIdx.x % quads, r = threadIdx.x / quads;
  double sum[4] = {};
  int count[4] = {};
  if (n > 0 && r < rows) {
    const int c1 = (b - 1) / p.chunk;
#pragma unroll 8
    for (int c = a / p.chunk + r; c <= c1; c += rows) {
      const size_t at = (size_t)(c + blockIdx.x) * p.row + q * 4;
      const f32x4 v = *reinterpret_cast<const f32x4*>(p.part_sums + at);
      const i32x4 k = *reinterpret_cast<const i32x4*>(p.part_counts + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[i] += v[i];
        count[i] += k[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lds_sum[threadIdx.x][i] = sum[i];
    lds_count[threadIdx.x][i] = count[i];
  }
  // by halves down to eight rows: few experts leave many (8 of them 512, which a thread
  // each would take 13 us to add up)
  int left = rows;
  while (left > 8) {
    const int half = (left + 1) / 2;
    __syncthreads();
    if (r + half < left) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lds_sum[threadIdx.x][i] += lds_sum[threadIdx.x + half * quads][i];
        lds_count[threadIdx.x][i] += lds_count[threadIdx.x + half * quads][i];
      }
    }
    left = half;
  }
  __syncthreads();
  double total = 0.0;
  for (int e = threadIdx.x; e < p.E; e += N) {
    double v = 0.0;
    int k = 0;
#pragma unroll 4
    for (int j = 0; j < left; ++j) {
      v += lds_sum[j * quads + e / 4][e % 4];
      k += lds_count[j * quads + e / 4][e % 4];
    }
    p.counts[(size_t)s * p.E + e] = k;
    total += v * k;
  }
  total = block_sum<N>(total, parts);
  if (threadIdx.x == 0) write_loss(p, s, n, total);
}

// Few tokens: one workgroup per sequence does all of it, in one launch.
constexpr int kOneThreads = 1024;
template <int LPT, int NV, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kOneThreads) void balance_one_kernel(BalanceParams p) {
  constexpr int ROWS = kOneThreads / LPT;
  __shared__ f32x4 sums[kOneThreads / 64][LPT * NV];
  __shared__ int hist[kColumns<LPT, NV>];
  __shared__ double parts[kOneThreads / 64];
  const int lane = threadIdx.x % LPT, row = threadIdx.x / LPT;
  const int s = blockIdx.x;
  const int a = start_of(p, s), b = start_of(p, s + 1);
  for (int e = threadIdx.x; e < p.row; e += kOneThreads) hist[e] = 0;
  __syncthreads();
  const size_t last = (size_t)b * p.top_k;
  for (size_t i = (size_t)a * p.top_k + threadIdx.x; i < last; i += kOneThreads) {
    const int e = p.ids[i];
    if ((unsigned)e < (unsigned)p.E) atomicAdd(&hist[e], 1);
  }
  constexpr int ROUNDS = NV == 1 ? 8 : 16 / (NV * 2);            // whose logits are loaded together
  f32x4 acc[NV] = {};
  for (int base = a; base < b; base += ROUNDS * ROWS) {
    f32x4 x[ROUNDS][NV], rest[NV];
#pragma unroll
    for (int h = 0; h < ROUNDS; ++h)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        x[h][v] = load4<BF16>(p.logits, (size_t)min(base + h * ROWS + row, b - 1) * p.E, (v * LPT + lane) * 4, p.E,
                              -INFINITY);
#pragma unroll
    for (int h = 0; h < ROUNDS; ++h) {
      if (base + h * ROWS >= b) break;
      float inv = scores<LPT, NV, SIGMOID>(x[h], rest);
      inv = base + h * ROWS + row < b ? inv : 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) acc[v] += x[h][v] * inv;
    }
  }
  // a wave's rows are added in their registers, the waves' through shared memory
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (LPT <= 32) acc[v][i] += __shfl_xor(acc[v][i], 32);
      if constexpr (LPT <= 16) acc[v][i] += __shfl_xor(acc[v][i], 16);
    }
    if (threadIdx.x % 64 < LPT) sums[threadIdx.x / 64][v * LPT + lane] = acc[v];
  }
  __syncthreads();
  double total = 0.0;
  for (int e = threadIdx.x; e < p.E; e += kOneThreads) {
    double sum = 0.0;
#pragma unroll 8
    for (int r = 0; r < kOneThreads / 64; ++r) sum += reinterpret_cast<const float*>(&sums[r][0])[e];
    p.counts[(size_t)s * p.E + e] = hist[e];
    total += sum * hist[e];
  }
  total = block_sum<kOneThreads>(total, parts);
  if (threadIdx.x == 0) write_loss(p, s, b - a, total);
}

// The gradient.  All counts are taken less that of the token's highest logit: the
// differences are whole numbers, and a share of nearly 1 drops out of the sum over
// p_e (counts_i - counts_e) instead of cancelling in it.
template <int LPT, int NV, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(THREADS) void balance_backward_kernel(BalanceParams p) {
  constexpr int ROWS = THREADS / LPT;
  __shared__ int counter;
  const int lane = threadIdx.x % LPT, row = threadIdx.x / LPT;
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T - t0, p.chunk) + t0;
  f32x4 x[NV], rest[NV], c[NV];
  // tokens from base on, before anything is known of their sequences
  auto load = [&](int base) {
    const size_t at = (size_t)min(base + row, t1 - 1) * p.E;
#pragma unroll
    for (int v = 0; v < NV; ++v) x[v] = load4<BF16>(p.logits, at, (v * LPT + lane) * 4, p.E, -INFINITY);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      c[v] = f32x4{};
      if (p.c) c[v] = load4<BF16>(p.c, at, (v * LPT + lane) * 4, p.E, 0.0f);
    }
  };
  load(t0);
  int s = sequence_at<THREADS>(p, t0, &counter);
  for (int a = t0; a < t1;) {
    // the next tokens of one sequence, or of none (those keep c)
    const int from = s < p.S ? start_of(p, s) : t1;
    const bool in = from <= a;
    const int b = in ? min(start_of(p, s + 1), t1) : min(from, t1);
    i32x4 count[NV] = {};
    float weight = 0.0f;
    if (in && a < b) {
      const double n = start_of(p, s + 1) - from;
      weight = (float)((double)p.scale * p.E / (p.top_k * n * n) * (p.grad_loss ? p.grad_loss[s] : 1.0f));
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int col = (v * LPT + lane) * 4;
        const int32_t* k = p.counts + (size_t)s * p.E + col;
        if (col + 4 <= p.E)
          count[v] = *reinterpret_cast<const i32x4_u*>(k);
        else
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (col + i < p.E) count[v][i] = k[i];
      }
    }
    for (int base = a; base < b; base += ROWS) {
      const int t = base + row;
      const size_t at = (size_t)min(t, t1 - 1) * p.E;
      if (base != t0) load(base);
      float top = -INFINITY;
      int ref = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ref = x[v][i] > top ? count[v][i] : ref;
          top = fmaxf(x[v][i], top);           // (a NaN is neither)
        }
      const float highest = token_max<LPT>(top);
      // of lanes that share the highest, the largest count: one value for all lanes
      ref = token_max<LPT>(top == highest ? ref : INT_MIN);
      const float inv = scores<LPT, NV, SIGMOID>(x, rest);
      f32x4 d[NV];
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[v][i] = (float)(count[v][i] - ref);
          x[v][i] *= inv;
          sum = fmaf(x[v][i], d[v][i], sum);
        }
      sum = token_sum<LPT>(sum);
      if (t >= b) continue;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int col = (v * LPT + lane) * 4;
        f32x4 g;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = weight * x[v][i] * (d[v][i] - sum);
          if constexpr (SIGMOID) g[i] *= rest[v][i];
          g[i] = c[v][i] + (x[v][i] > 0.0f ? g[i] : 0.0f);
        }
        if constexpr (BF16) {
          uint16_t* out = static_cast<uint16_t*>(p.grad_logits) + at + col;
          u16x4 u;
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(g[i]));
          if (col + 4 <= p.E)
            *reinterpret_cast<u16x4_u*>(out) = u;
          else
#pragma unroll
            for (int i = 0; i < 3; ++i)
              if (col + i < p.E) out[i] = u[i];
        } else {
          float* out = static_cast<float*>(p.grad_logits) + at + col;
          if (col + 4 <= p.E)
            *reinterpret_cast<f32x4_u*>(out) = g;
          else
#pragma unroll
            for (int i = 0; i < 3; ++i)
              if (col + i < p.E) out[i] = g[i];
        }
      }
    }
    a = max(a, b);
    if (in) ++s;
  }
}

enum Kernel { kSums, kOne, kBackward };

template <Kernel WHICH, int LPT, int NV>
void launch_shape(const BalanceParams& p, bool bf, int score, int grid, hipStream_t st) {
#define DG_BALANCE(KERNEL, THREADS)                                   \
  if (score == DG_SCORE_SIGMOID) {                                    \
    if (bf)                                                           \
      KERNEL<LPT, NV, true, true><<<grid, THREADS, 0, st>>>(p);       \
    else                                                              \
      KERNEL<LPT, NV, false, true><<<grid, THREADS, 0, st>>>(p);      \
  } else {                                                            \
    if (bf)                                                           \
      KERNEL<LPT, NV, true, false><<<grid, THREADS, 0, st>>>(p);      \
    else                                                              \
      KERNEL<LPT, NV, false, false><<<grid, THREADS, 0, st>>>(p);     \
  }
  if constexpr (WHICH == kBackward) {
    DG_BALANCE(balance_backward_kernel, THREADS)
  } else if constexpr (WHICH == kOne) {
    DG_BALANCE(balance_one_kernel, kOneThreads)
  } else {
    DG_BALANCE(balance_sums_kernel, kSumThreads)
  }
#undef DG_BALANCE
}

template <Kernel WHICH>
void launch_kernel(const BalanceParams& p, bool bf, int score, int grid, hipStream_t st) {
  if (p.E <= 64)
    launch_shape<WHICH, 16, 1>(p, bf, score, grid, st);
  else if (p.E <= 128)
    launch_shape<WHICH, 16, 2>(p, bf, score, grid, st);
  else if (p.E <= 256)
    launch_shape<WHICH, 16, 4>(p, bf, score, grid, st);
  else if (p.E <= 512)
    launch_shape<WHICH, 32, 4>(p, bf, score, grid, st);
  else
    launch_shape<WHICH, 64, 4>(p, bf, score, grid, st);
}

// One launch, with one workgroup per sequence, up to this many logits per sequence
// (rows of fewer than 64 count as 64: they take the same lanes).  One CU takes about
// 0.14 ns for each, two launches the more the wider their sums are.  From Python, one
// launch and two (softmax): 64 tokens of 256 experts 5.4 us and 8.1, 128 of 256 7.0 and
// 8.4, 192 of 128 6.5 and 7.1, 256 of 128 7.3 and 7.3, 256 of 64 5.7 and 6.9, 384 of 64
// 7.0 and 6.9, 512 of 64 8.2 and 6.9, 1024 of 16 14.2 and 8.1.  Sigmoids cost one launch
// more than two (192 of 128 7.4 and 7.5, 384 of 64 8.0 and 7.2).
int one_values(int E) { return E <= 128 ? 24576 : 32768; }
// The starts are on the device: four sequences' share at the most for all tokens, which
// could be one sequence's (1024 tokens of 64 in 8 sequences 4.8 us and 7.6, in one of
// them 14 and 8).
constexpr int kOneShares = 4;

// Tokens per chunk at the least: a block of the kernel.  16384 tokens of 256 experts in
// one sequence and in 8: 17.3 and 13.5 us with 64, 25.9 and 16.6 with 32, 18.2 and 16.4
// with 128; 64 tokens of 1024 10.4 with 16, 13.3 with 32, 19.6 with 64.
int least_chunk(int E) { return E <= 256 ? 64 : E <= 512 ? 32 : 16; }

// Tokens per workgroup: a multiple of 16, at most `most` workgroups
int chunk_for(int T, int most, int least) {
  const long long c = ((long long)T + most - 1) / most;
  return (int)((c < least ? least : c) + 15) / 16 * 16;
}

int check_balance(const void* logits, int logits_type, const int32_t* starts, const void* counts, int T, int E,
                  int top_k, int S, int score) {
  if (logits_type != DG_F32 && logits_type != DG_BF16)
    return fail(DG_ERR_INVALID_ARG, "logits_type=%d is neither DG_F32 nor DG_BF16", logits_type);
  if (score != DG_SCORE_SOFTMAX && score != DG_SCORE_SIGMOID)
    return fail(DG_ERR_INVALID_ARG, "score=%d is neither DG_SCORE_SOFTMAX nor DG_SCORE_SIGMOID", score);
  if (T < 0 || S < 0) return fail(DG_ERR_INVALID_ARG, "negative size (T=%d num_seqs=%d)", T, S);
  if (E < 1 || top_k < 1 || top_k > E)
    return fail(DG_ERR_INVALID_ARG, "top_k=%d must lie in [1, E=%d]", top_k, E);
  if (E > kMaxExperts || top_k > kMaxTopK)
    return fail(DG_ERR_UNSUPPORTED, "E=%d or top_k=%d exceeds %d experts and %d choices", E, top_k, kMaxExperts,
                kMaxTopK);
  if ((long long)T * top_k > kMaxChoices)
    return fail(DG_ERR_UNSUPPORTED, "T * top_k = %lld choices exceed 2^30", (long long)T * top_k);
  if (!starts && S != 1) return fail(DG_ERR_INVALID_ARG, "num_seqs=%d needs seq_starts (NULL means one sequence)", S);
  if (T > 0 && !logits) return fail(DG_ERR_INVALID_ARG, "logits must not be NULL");
  if (S > 0 && !counts) return fail(DG_ERR_INVALID_ARG, "counts must not be NULL");
  if (!aligned(logits, logits_type == DG_F32 ? 4 : 2) || !aligned(starts, 4) || !aligned(counts, 4))
    return fail(DG_ERR_INVALID_ARG, "logits, seq_starts and counts must be aligned to their types");
  return DG_OK;
}

int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" int dg_route_balance(const void* logits, int logits_type, const int32_t* topk_ids,
                                const int32_t* seq_starts, float* loss, int32_t* counts, int T, int E, int top_k,
                                int num_seqs, int score, float scale, void* stream) {
  int s = check_balance(logits, logits_type, seq_starts, counts, T, E, top_k, num_seqs, score);
  if (s != DG_OK) return s;
  if (T > 0 && !topk_ids) return fail(DG_ERR_INVALID_ARG, "topk_ids must not be NULL");
  if (num_seqs > 0 && !loss) return fail(DG_ERR_INVALID_ARG, "loss must not be NULL");
  if (!aligned(topk_ids, 4) || !aligned(loss, 4))
    return fail(DG_ERR_INVALID_ARG, "topk_ids and loss must be 4-byte aligned");
  if (num_seqs == 0) return DG_OK;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  BalanceParams p{};
  p.logits = logits;
  p.ids = topk_ids;
  p.starts = seq_starts;
  p.loss = loss;
  p.counts = counts;
  p.T = T;
  p.E = E;
  p.top_k = top_k;
  p.S = num_seqs;
  p.row = (E + 3) / 4 * 4;
  p.scale = scale;
  if ((long long)T * std::max(p.row, 64) <= (long long)one_values(E) * std::min(num_seqs, kOneShares) &&
      num_seqs <= kSequencesPerLaunch) {
    launch_kernel<kOne>(p, logits_type == DG_BF16, score, num_seqs, st);
    return launched();
  }
  Scratch sc;
  s = call_scratch(st, &sc);
  if (s != DG_OK) return s;
  const size_t slot = (size_t)p.row * 8;
  if (sc.bytes / slot < 2)
    return fail(DG_ERR_UNSUPPORTED, "a workspace of %zu bytes has no room for the sums of %d experts", sc.bytes, E);
  // half of the room at most for the chunks, two workgroups per CU where that is enough
  const size_t slots = sc.bytes / slot;
  const int most = (size_t)(2 * sc.num_cus) > slots / 2 ? (int)(slots / 2) : 2 * sc.num_cus;
  p.chunk = chunk_for(T, most, least_chunk(E));
  const int chunks = T > 0 ? (T - 1) / p.chunk + 1 : 0;
  // as many sequences at a time as there is room for, usually all
  size_t per = slots - chunks;
  if (per > (size_t)kSequencesPerLaunch) per = kSequencesPerLaunch;
  if (per > (size_t)num_seqs) per = num_seqs;
  p.part_sums = reinterpret_cast<float*>(sc.ptr);
  p.part_counts = reinterpret_cast<int32_t*>(sc.ptr) + (chunks + per) * p.row;
  for (size_t first = 0; first < (size_t)num_seqs; first += per) {
    p.first = (int)first;
    p.last = (int)(first + per < (size_t)num_seqs ? first + per : num_seqs);
    const int n = p.last - p.first;
    if (chunks > 0) launch_kernel<kSums>(p, logits_type == DG_BF16, score, chunks, st);
    if (chunks / n >= 16)
      balance_loss_kernel<1024><<<n, 1024, 0, st>>>(p);
    else
      balance_loss_kernel<256><<<n, 256, 0, st>>>(p);
    s = launched();
    if (s != DG_OK) return s;
  }
  return DG_OK;
}

extern "C" int dg_route_balance_backward(const void* logits, int logits_type, const int32_t* counts,
                                         const int32_t* seq_starts, const float* grad_loss, const void* c,
                                         void* grad_logits, int T, int E, int top_k, int num_seqs, int score,
                                         float scale, void* stream) {
  int s = check_balance(logits, logits_type, seq_starts, counts, T, E, top_k, num_seqs, score);
  if (s != DG_OK) return s;
  if (T > 0 && !grad_logits) return fail(DG_ERR_INVALID_ARG, "grad_logits must not be NULL");
  const size_t size = logits_type == DG_F32 ? 4 : 2;
  if (!aligned(grad_loss, 4) || !aligned(c, size) || !aligned(grad_logits, size))
    return fail(DG_ERR_INVALID_ARG, "grad_loss, c and grad_logits must be aligned to their types");
  if (T == 0) return DG_OK;
  BalanceParams p{};
  p.logits = logits;
  p.counts = const_cast<int32_t*>(counts);
  p.starts = seq_starts;
  p.grad_loss = grad_loss;
  p.c = c;
  p.grad_logits = grad_logits;
  p.T = T;
  p.E = E;
  p.top_k = top_k;
  p.S = num_seqs;
  p.scale = scale;
  p.chunk = chunk_for(T, 2048, 16);
  launch_kernel<kBackward>(p, logits_type == DG_BF16, score, (T - 1) / p.chunk + 1, static_cast<hipStream_t>(stream));
  return launched();
}

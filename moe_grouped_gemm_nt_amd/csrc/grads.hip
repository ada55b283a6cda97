// The norm of many gradients together, and the gradients scaled to it (include/dg.h):
//   norm = sqrt(sum over all tensors of x^2),  out = x * min(1, max_norm / (norm + 1e-6))
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>
#include <vector>

#include "../../include/dg.h"
#include "dg_host.h"

namespace dg {
namespace {

constexpr int THREADS = 256;
// Tensors per launch: their addresses and sizes travel in the launch's arguments
// (4 KB), so that nothing is copied ahead of it and a captured graph replays with
// the tensors of the captured call.
constexpr int kTensors = 120;
constexpr int kChunk = 16384;            // bytes of a tensor per step of a workgroup

struct Grads {
  const void* in[kTensors];
  void* out[kTensors];
  long long size[kTensors];
  int start[kTensors + 1];               // chunks before each tensor's
  uint32_t half[(kTensors + 31) / 32];   // bf16
  int n;
  double* partial;                       // one per workgroup
  const float* norm;
  float max_norm;
};
static_assert(sizeof(Grads) <= 4096, "a launch's arguments");

template <int NE>
struct Piece16 {
  typedef uint16_t V __attribute__((ext_vector_type(NE)));
  typedef V U __attribute__((aligned(2)));
};
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_u __attribute__((aligned(4)));
typedef Piece16<8>::U u16x8_u;

__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// The tensor that chunk c belongs to
__device__ __forceinline__ int tensor_of(const Grads& g, int c) {
  int lo = 0, hi = g.n;                  // start[lo] <= c < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (g.start[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

constexpr int DEPTH = kChunk / (THREADS * 16);                   // 16-byte pieces per thread and chunk

// Calls f(tensor, its chunk) for this workgroup's chunks
template <typename F>
__device__ __forceinline__ void each_chunk(const Grads& g, F f) {
  int i = -1;
  for (int c = blockIdx.x; c < g.start[g.n]; c += gridDim.x) {
    if (i < 0) i = tensor_of(g, c);
    while (c >= g.start[i + 1]) ++i;
    f(i, c - g.start[i]);
  }
}

// Elements of a 16-byte piece
template <bool HALF>
struct Piece {
  typedef f32x4 V;
  typedef f32x4_u U;
  typedef float E;
  static constexpr int N = 4;
};
template <>
struct Piece<true> {
  typedef Piece16<8>::V V;
  typedef u16x8_u U;
  typedef uint16_t E;
  static constexpr int N = 8;
};

__device__ __forceinline__ double square(double sum, float v) { return fma((double)v, (double)v, sum); }
__device__ __forceinline__ double square(double sum, uint16_t v) { return square(sum, widen(v)); }

template <bool HALF>
__device__ __forceinline__ double chunk_squares(const Grads& g, int i, int chunk, double sum) {
  typedef Piece<HALF> P;
  const long long at = (long long)chunk * (kChunk / sizeof(typename P::E));
  const typename P::E* x = static_cast<const typename P::E*>(g.in[i]) + at;
  const long long n = g.size[i] - at;
  if (n >= (long long)(kChunk / sizeof(typename P::E))) {
    typename P::V v[DEPTH];
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) v[j] = *reinterpret_cast<const typename P::U*>(x + (j * THREADS + threadIdx.x) * P::N);
    __builtin_amdgcn_sched_barrier(0);                           // no sum before the last load is under way
#pragma unroll
    for (int j = 0; j < DEPTH; ++j)
#pragma unroll
      for (int e = 0; e < P::N; ++e) sum = square(sum, v[j][e]);
    return sum;
  }
  const int whole = (int)n / P::N * P::N;
  for (int e = threadIdx.x * P::N; e < whole; e += THREADS * P::N) {
    const typename P::V v = *reinterpret_cast<const typename P::U*>(x + e);
#pragma unroll
    for (int j = 0; j < P::N; ++j) sum = square(sum, v[j]);
  }
  return whole + (int)threadIdx.x < n ? square(sum, x[whole + threadIdx.x]) : sum;
}

// Bound by memory: 940 MB in 160 us (5.9 TB/s).  Streaming loads take 142, but leave
// nothing in the last-level cache for the clipping: together 441 us against 424.
//
// Squares are summed in fp64, where those of the largest and the smallest fp32
// values still differ from infinity and zero; one partial sum per workgroup, added
// up in their order by the second kernel.
__global__ __launch_bounds__(THREADS) void grad_squares_kernel(Grads g) {
  double sum = 0.0;
  each_chunk(g, [&](int i, int chunk) {
    if (g.half[i / 32] >> (i % 32) & 1)
      sum = chunk_squares<true>(g, i, chunk, sum);
    else
      sum = chunk_squares<false>(g, i, chunk, sum);
  });
  __shared__ double sums[THREADS / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int w = 0; w < THREADS / 64; ++w) sum += sums[w];
    g.partial[blockIdx.x] = sum;
  }
}

__global__ __launch_bounds__(THREADS) void grad_norm_kernel(const double* partial, int n, float* norm) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += THREADS) sum += partial[i];
  __shared__ double sums[THREADS / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int w = 0; w < THREADS / 64; ++w) sum += sums[w];
    *norm = (float)sqrt(sum);
  }
}

__device__ __forceinline__ float scaled(float v, float factor) { return v * factor; }
__device__ __forceinline__ uint16_t scaled(uint16_t v, float factor) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(widen(v) * factor));
}

template <bool HALF>
__device__ __forceinline__ void chunk_scale(const Grads& g, int i, int chunk, float factor) {
  typedef Piece<HALF> P;
  const long long at = (long long)chunk * (kChunk / sizeof(typename P::E));
  const typename P::E* x = static_cast<const typename P::E*>(g.in[i]) + at;
  typename P::E* y = static_cast<typename P::E*>(g.out[i]) + at;
  const long long n = g.size[i] - at;
  if (n >= (long long)(kChunk / sizeof(typename P::E))) {
    typename P::V v[DEPTH];                                      // all loads first: y may be x
#pragma unroll
    for (int j = 0; j < DEPTH; ++j)
      v[j] = __builtin_nontemporal_load(reinterpret_cast<const typename P::U*>(x + (j * THREADS + threadIdx.x) * P::N));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) {
#pragma unroll
      for (int e = 0; e < P::N; ++e) v[j][e] = scaled(v[j][e], factor);
      __builtin_nontemporal_store(v[j], reinterpret_cast<typename P::U*>(y + (j * THREADS + threadIdx.x) * P::N));
    }
    return;
  }
  const int whole = (int)n / P::N * P::N;
  for (int e = threadIdx.x * P::N; e < whole; e += THREADS * P::N) {
    typename P::V v = *reinterpret_cast<const typename P::U*>(x + e);
#pragma unroll
    for (int j = 0; j < P::N; ++j) v[j] = scaled(v[j], factor);
    *reinterpret_cast<typename P::U*>(y + e) = v;
  }
  if (whole + (int)threadIdx.x < n) y[whole + threadIdx.x] = scaled(x[whole + threadIdx.x], factor);
}

// Bound by memory: 940 MB read and written in 300 us (6.3 TB/s; a device copy reaches
// 5.1), with streaming loads and stores; 264 behind the norm, whose reads it finds in the
// last-level cache for a part.
__global__ __launch_bounds__(THREADS) void grad_clip_kernel(Grads g) {
  const float norm = *g.norm;
  const float q = g.max_norm / (norm + 1e-6f);
  const float factor = q > 1.0f ? 1.0f : q;                      // a NaN stays one
  each_chunk(g, [&](int i, int chunk) {
    if (factor == 1.0f && g.in[i] == g.out[i]) return;           // as it is
    if (g.half[i / 32] >> (i % 32) & 1)
      chunk_scale<true>(g, i, chunk, factor);
    else
      chunk_scale<false>(g, i, chunk, factor);
  });
}

// Workgroups per CU: few for the norm, each of which leaves a partial sum (940 MB in
// 160 us, with 256 per CU in 226), as good as one per chunk for the clipping (norm and
// clipping together 424 us, with 64 437, with 8 and chunks of twice the size 460).
constexpr int kNormGroups = 8, kClipGroups = 256;
constexpr long long kMaxBytes = 1LL << 45;
constexpr int kMaxTensors = 1 << 20;

size_t size_of(int type) { return type == DG_F32 ? 4 : 2; }

int check_grads(const void* const* grads, const int* types, const long long* sizes, int n) {
  if (n < 0) return fail(DG_ERR_INVALID_ARG, "num_tensors=%d must not be negative", n);
  if (n > kMaxTensors) return fail(DG_ERR_UNSUPPORTED, "num_tensors=%d exceeds 2^20", n);
  if (n > 0 && (!grads || !types || !sizes)) return fail(DG_ERR_INVALID_ARG, "grads, types and sizes must not be NULL");
  for (int i = 0; i < n; ++i) {
    if (types[i] != DG_F32 && types[i] != DG_BF16)
      return fail(DG_ERR_INVALID_ARG, "types[%d]=%d is neither DG_F32 nor DG_BF16", i, types[i]);
    if (sizes[i] < 0) return fail(DG_ERR_INVALID_ARG, "sizes[%d]=%lld must not be negative", i, sizes[i]);
    if (sizes[i] > kMaxBytes / 4) return fail(DG_ERR_UNSUPPORTED, "sizes[%d]=%lld exceeds 2^43", i, sizes[i]);
    if (sizes[i] > 0 && !grads[i]) return fail(DG_ERR_INVALID_ARG, "grads[%d] must not be NULL", i);
    if (!aligned(grads[i], size_of(types[i])))
      return fail(DG_ERR_INVALID_ARG, "grads[%d] must be aligned to its type", i);
  }
  return DG_OK;
}

// Calls f with the arguments of each launch: up to kTensors tensors with something
// in them, and no more chunks than an int counts (a larger tensor goes out in parts).
template <typename F>
int each_launch(const void* const* grads, void* const* out, const int* types, const long long* sizes, int n, F f) {
  constexpr int kMostChunks = 1 << 30;
  Grads g{};
  int s = DG_OK;
  auto flush = [&] {
    if (g.n > 0 && s == DG_OK) s = f(g);
    g = Grads{};
  };
  for (int i = 0; i < n && s == DG_OK; ++i) {
    const long long per = kChunk / (long long)size_of(types[i]);
    for (long long at = 0; at < sizes[i] && s == DG_OK;) {
      if (g.n == kTensors || g.start[g.n] == kMostChunks) flush();
      const long long room = (long long)(kMostChunks - g.start[g.n]) * per;
      const long long size = sizes[i] - at < room ? sizes[i] - at : room;
      const size_t bytes = (size_t)at * size_of(types[i]);
      g.in[g.n] = static_cast<const uint8_t*>(grads[i]) + bytes;
      g.out[g.n] = out ? static_cast<uint8_t*>(out[i]) + bytes : nullptr;
      g.size[g.n] = size;
      if (types[i] == DG_BF16) g.half[g.n / 32] |= 1u << (g.n % 32);
      g.start[g.n + 1] = g.start[g.n] + (int)((size + per - 1) / per);
      ++g.n;
      at += size;
    }
  }
  flush();
  return s;
}

int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

// A tensor of out may be that of grads in the same place, and has nothing in common
// with any other of either: such elements would be scaled twice, or while others
// read them.
int check_apart(const void* const* grads, void* const* out, const int* types, const long long* sizes, int n,
                const float* norm) {
  struct Span {
    uintptr_t from, to;
    bool written;
  };
  std::vector<Span> spans;
  spans.reserve(2 * (size_t)n + 1);
  spans.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm + 1), false});
  for (int i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    const size_t bytes = (size_t)sizes[i] * size_of(types[i]);
    const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]), b = reinterpret_cast<uintptr_t>(out[i]);
    if (a != b) spans.push_back({a, a + bytes, false});
    spans.push_back({b, b + bytes, true});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.from < b.from; });
  uintptr_t end = 0, written_end = 0;                            // of all spans so far, of those written
  for (const Span& s : spans) {
    if (s.from < (s.written ? end : written_end))
      return fail(DG_ERR_INVALID_ARG, "out may only be grads itself or apart from every tensor and norm (at %p)",
                  reinterpret_cast<void*>(s.from));
    end = std::max(end, s.to);
    if (s.written) written_end = std::max(written_end, s.to);
  }
  return DG_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" int dg_grad_norm(const void* const* grads, const int* types, const long long* sizes, int num_tensors,
                            float* norm, void* stream) {
  int s = check_grads(grads, types, sizes, num_tensors);
  if (s != DG_OK) return s;
  if (!norm || !aligned(norm, 4)) return fail(DG_ERR_INVALID_ARG, "norm must be a 4-byte aligned address");
  const hipStream_t st = static_cast<hipStream_t>(stream);
  Scratch sc;
  s = call_scratch(st, &sc);
  if (s != DG_OK) return s;
  // every launch has partial sums of its own: with little room fewer workgroups each
  long long launches = 0;
  s = each_launch(grads, nullptr, types, sizes, num_tensors, [&](const Grads&) {
    ++launches;
    return DG_OK;
  });
  const long long slots = (long long)(sc.bytes / sizeof(double));
  if (launches > slots)
    return fail(DG_ERR_UNSUPPORTED, "a workspace of %zu bytes has no room for the sums of %d tensors", sc.bytes,
                num_tensors);
  const long long most = std::min(launches ? slots / launches : 0, kNormGroups * (long long)sc.num_cus);
  double* partial = reinterpret_cast<double*>(sc.ptr);
  int used = 0;
  s = each_launch(grads, nullptr, types, sizes, num_tensors, [&](Grads& g) {
    const int grid = (int)std::min((long long)g.start[g.n], most);
    g.partial = partial + used;
    used += grid;
    grad_squares_kernel<<<grid, THREADS, 0, st>>>(g);
    return launched();
  });
  if (s != DG_OK) return s;
  grad_norm_kernel<<<1, THREADS, 0, st>>>(partial, used, norm);
  return launched();
}

extern "C" int dg_grad_clip(const void* const* grads, void* const* out, const int* types, const long long* sizes,
                            int num_tensors, const float* norm, float max_norm, void* stream) {
  int s = check_grads(grads, types, sizes, num_tensors);
  if (s != DG_OK) return s;
  if (num_tensors > 0 && !out) return fail(DG_ERR_INVALID_ARG, "out must not be NULL");
  if (!norm || !aligned(norm, 4)) return fail(DG_ERR_INVALID_ARG, "norm must be a 4-byte aligned address");
  if (!(max_norm >= 0.0f)) return fail(DG_ERR_INVALID_ARG, "max_norm=%g must not be negative", max_norm);
  for (int i = 0; i < num_tensors; ++i) {
    if (sizes[i] > 0 && !out[i]) return fail(DG_ERR_INVALID_ARG, "out[%d] must not be NULL", i);
    if (!aligned(out[i], size_of(types[i]))) return fail(DG_ERR_INVALID_ARG, "out[%d] must be aligned to its type", i);
  }
  try {
    s = check_apart(grads, out, types, sizes, num_tensors, norm);
  } catch (const std::bad_alloc&) {
    return fail(DG_ERR_INVALID_ARG, "no host memory for %d tensors", num_tensors);
  }
  if (s != DG_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  Scratch sc;
  s = call_scratch(st, &sc);
  if (s != DG_OK) return s;
  return each_launch(grads, out, types, sizes, num_tensors, [&](Grads& g) {
    g.norm = norm;
    g.max_norm = max_norm;
    const int grid = (int)std::min((long long)g.start[g.n], kClipGroups * (long long)sc.num_cus);
    grad_clip_kernel<<<grid, THREADS, 0, st>>>(g);
    return launched();
  });
}

// Low-rank adapters of many requests beside a shared projection (include/dg.h):
//   d[t] = c[t] + scales[i] * B[i] . (A[i] . x[t]),   i = adapter_ids[t]
#include <hip/hip_runtime.h>

#include "../../include/dg.h"
#include "dg_host.h"
#include "expert_rows.h"

namespace dg {
namespace {

constexpr int kMaxRank = 256;
constexpr int THREADS = 256;
constexpr int WAVES = THREADS / 64;
constexpr int kInlineTokens = 256;       // up to here every workgroup finds its tile's tokens itself

struct LoraParams {
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const float* scales;
  const int32_t* ids;
  const uint16_t* c;
  uint16_t* d;
  long long ldx, ldc, ldd;
  int T, N, K, R, L;
  float* partial;          // [k_splits][T][R]: A . x of each K range
  int k_splits;
  int kb_per_split;        // K blocks of 128 per range
  const int32_t* layout;   // tile lists (many tokens): group of each row, L = tokens without an adapter
  const int32_t* slot_of;  // token of each row, -1 where a tile is not full
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ uint16_t f32_bf16(float x) {
  __bf16 h = static_cast<__bf16>(x);
  return __builtin_bit_cast(uint16_t, h);
}

// The tokens of this workgroup's tile into rows[16 * MT] (-1 where there is none)
// and their adapter into *id (-1: none).  Returns false for a workgroup without a
// tile.  Ends with a barrier.
//
// INLINE: the workgroup of token t has a tile if the tokens before t hold a
// multiple of 16 * MT tokens of t's adapter; its tile is t and the next ones of
// that adapter.  Every wave counts for itself (at most kInlineTokens / 64
// ballots), so that no workgroup waits for a list.
template <int MT, bool INLINE>
__device__ __forceinline__ bool find_tile(const LoraParams& p, int tile, int* rows, int* id) {
  const int lane = threadIdx.x & 63;
  if constexpr (INLINE) {
    auto key = [&](int v) { return v >= 0 && v < p.L ? v : -1; };
    int ids[kInlineTokens / 64];
#pragma unroll
    for (int i = 0; i < kInlineTokens / 64; ++i)
      ids[i] = i * 64 + lane < p.T ? key(p.ids[i * 64 + lane]) : -2;
    const int mine = key(p.ids[tile]);
    if (threadIdx.x < 16 * MT) rows[threadIdx.x] = -1;
    __syncthreads();
    int before = 0, after = 0;
#pragma unroll
    for (int i = 0; i < kInlineTokens / 64; ++i) {
      const int s = i * 64 + lane;
      before += __popcll(__ballot(ids[i] == mine && s < tile));
      const uint64_t m = __ballot(ids[i] == mine && s >= tile);
      const int at = after + __popcll(m & ((1ull << lane) - 1));
      if (ids[i] == mine && s >= tile && at < 16 * MT && threadIdx.x < 64) rows[at] = s;
      after += __popcll(m);
    }
    *id = mine;
    if (before % (16 * MT) != 0) return false;
  } else {
    const int g = p.layout[(size_t)tile * 16 * MT];
    if (g < 0) return false;
    *id = g < p.L ? g : -1;
    if (threadIdx.x < 16 * MT) rows[threadIdx.x] = p.slot_of[(size_t)tile * 16 * MT + threadIdx.x];
  }
  __syncthreads();
  return true;
}

// h = A . x over one K range of one tile of 16 * MT tokens, as h^T: the ranks
// are the MFMA's rows and the tokens its columns, so that a lane ends with four
// neighbouring ranks of one token.  The waves take the 32-K quarters of each
// 128-K block (a row's 256 bytes go to the four waves together) and add up
// through LDS.  Operands come straight from global memory: each element is used
// once per tile.
template <int MT, int RT, bool INLINE>
__global__ __launch_bounds__(THREADS) void lora_shrink_kernel(LoraParams p) {
  constexpr int U = MT + RT <= 2 ? 8 : (MT + RT <= 5 ? 4 : 2);     // K blocks in flight
  __shared__ int rows[16 * MT];
  __shared__ f32x4 sums[2][MT * RT][64];
  int id;
  if (!find_tile<MT, INLINE>(p, blockIdx.x, rows, &id) || id < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g16 = lane >> 4;
  const int KB = p.K / 128;
  const int kb0 = blockIdx.y * p.kb_per_split, kb1 = min(KB, kb0 + p.kb_per_split);
  const int koff = wave * 32 + g16 * 8;
  const uint16_t* xp[MT];
  const uint16_t* ap[RT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = rows[m * 16 + r16];
    // a column without a token repeats the tile's first: MFMA columns are
    // independent, and this one is not stored
    xp[m] = p.x + (size_t)(t >= 0 ? t : rows[0]) * p.ldx + koff;
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
    ap[r] = p.a + ((size_t)id * p.R + min(r * 16 + r16, p.R - 1)) * p.K + koff;   // rows beyond R: not stored
  f32x4 acc[MT][RT] = {};
  for (int kb = kb0; kb < kb1; kb += U) {
    bf16x8 xf[U][MT], af[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t k = (size_t)min(kb + u, kb1 - 1) * 128;
#pragma unroll
      for (int r = 0; r < RT; ++r) af[u][r] = *reinterpret_cast<const bf16x8*>(ap[r] + k);
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[u][m] = *reinterpret_cast<const bf16x8*>(xp[m] + k);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + u >= kb1) break;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r)
          acc[m][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[u][r], xf[u][m], acc[m][r], 0, 0, 0);
    }
  }
  if (wave >= 2)
#pragma unroll
    for (int i = 0; i < MT * RT; ++i) sums[wave - 2][i][lane] = acc[i / RT][i % RT];
  __syncthreads();
  if (wave < 2)
#pragma unroll
    for (int i = 0; i < MT * RT; ++i) acc[i / RT][i % RT] += sums[wave][i][lane];
  __syncthreads();
  if (wave == 1)
#pragma unroll
    for (int i = 0; i < MT * RT; ++i) sums[0][i][lane] = acc[i / RT][i % RT];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = rows[m * 16 + r16];
    if (t < 0) continue;
    float* out = p.partial + ((size_t)blockIdx.y * p.T + t) * p.R;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int at = r * 16 + g16 * 4;
      if (at < p.R) *reinterpret_cast<f32x4*>(out + at) = acc[m][r] + sums[0][m * RT + r][lane];
    }
  }
}

// NE neighbouring bf16 of a row, at any 2-byte address.
template <int NE>
struct Piece {
  typedef uint16_t V __attribute__((ext_vector_type(NE)));
  typedef V U __attribute__((aligned(2)));
};

// d = c + B . h for one tile of tokens and 16 * NT * WAVES columns, again
// transposed: MFMA rows are columns of d.  h (the K ranges' sum times the
// adapter's scale) is split into two bf16, h = hi + lo to 16 bits, and both
// halves are multiplied: the products with B are then exact to 2^-17.
// MFMA row r of sub-tile j stands for column 4 * NT * (r / 4) + 4 * j + r % 4, so
// that a lane's 4 * NT results are neighbours in d.
template <int MT, int RK, int NT, bool INLINE>
__global__ __launch_bounds__(THREADS) void lora_expand_kernel(LoraParams p) {
  constexpr int RP = RK * 32;             // ranks padded to whole MFMA steps
  constexpr int LD = RP + 8;              // LDS row: 16 bytes on, so that 16 rows start in different banks
  constexpr int NE = 4 * NT;
  __shared__ int rows[16 * MT];
  __shared__ __attribute__((aligned(16))) uint16_t hs[2][16 * MT][LD];
  int id;
  if (!find_tile<MT, INLINE>(p, blockIdx.x, rows, &id)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g16 = lane >> 4;
  const int col0 = (blockIdx.y * WAVES + wave) * 16 * NT;      // this wave's first column
  f32x4 acc[MT][NT] = {};
  if (id >= 0) {
    const float scale = p.scales ? p.scales[id] : 1.0f;
    bf16x8 bf[NT][RK];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = min(col0 + 4 * NT * (r16 >> 2) + 4 * j + (r16 & 3), p.N - 1);    // beyond N: not stored
      const uint16_t* b = p.b + ((size_t)id * p.N + n) * p.R + g16 * 8;
#pragma unroll
      for (int k = 0; k < RK; ++k) {
        bf[j][k] = bf16x8{};
        if (k * 32 + g16 * 8 < p.R) bf[j][k] = *reinterpret_cast<const bf16x8*>(b + k * 32);
      }
    }
    for (int i = threadIdx.x; i < 16 * MT * (RP / 4); i += THREADS) {
      const int row = i / (RP / 4), r = i % (RP / 4) * 4;
      const int t = rows[row];
      f32x4 h = {};
      if (t >= 0 && r < p.R)
        for (int s = 0; s < p.k_splits; ++s)
          h += *reinterpret_cast<const f32x4*>(p.partial + ((size_t)s * p.T + t) * p.R + r);
      u16x4 hi, lo;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = h[e] * scale;
        hi[e] = f32_bf16(v);
        const float back = bf16_f32(hi[e]);
        lo[e] = fabsf(back) < INFINITY ? f32_bf16(v - back) : 0;
      }
      *reinterpret_cast<u16x4*>(&hs[0][row][r]) = hi;
      *reinterpret_cast<u16x4*>(&hs[1][row][r]) = lo;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int k = 0; k < RK; ++k)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const bf16x8 h = *reinterpret_cast<const bf16x8*>(&hs[q][m * 16 + r16][k * 32 + g16 * 8]);
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j][k], h, acc[m][j], 0, 0, 0);
        }
  }
  typedef typename Piece<NE>::U U;
  const int n = col0 + NE * g16;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = rows[m * 16 + r16];
    if (t < 0 || n >= p.N) continue;
    const uint16_t* c = p.c ? p.c + (size_t)t * p.ldc + n : nullptr;
    uint16_t* d = p.d + (size_t)t * p.ldd + n;
    if (n + NE <= p.N) {
      U v = {};
      if (c) v = *reinterpret_cast<const U*>(c);
#pragma unroll
      for (int e = 0; e < NE; ++e)
        if (id >= 0) v[e] = f32_bf16(bf16_f32(v[e]) + acc[m][e >> 2][e & 3]);
      *reinterpret_cast<U*>(d) = v;
    } else {
#pragma unroll
      for (int e = 0; e < NE; ++e)
        if (n + e < p.N) {
          const uint16_t v = c ? c[e] : 0;
          d[e] = id >= 0 ? f32_bf16(bf16_f32(v) + acc[m][e >> 2][e & 3]) : v;
        }
    }
  }
}

template <int MT, bool INLINE>
void launch_shrink(const LoraParams& p, int tiles, hipStream_t st) {
  const dim3 grid(tiles, p.k_splits);
  if (p.R <= 16)
    lora_shrink_kernel<MT, 1, INLINE><<<grid, THREADS, 0, st>>>(p);
  else if (p.R <= 32)
    lora_shrink_kernel<MT, 2, INLINE><<<grid, THREADS, 0, st>>>(p);
  else if (p.R <= 64)
    lora_shrink_kernel<MT, 4, INLINE><<<grid, THREADS, 0, st>>>(p);
  else if (p.R <= 128)
    lora_shrink_kernel<MT, 8, INLINE><<<grid, THREADS, 0, st>>>(p);
  else if constexpr (MT == 1)
    lora_shrink_kernel<MT, 16, INLINE><<<grid, THREADS, 0, st>>>(p);
}

template <int MT, int NT, bool INLINE>
void launch_expand(const LoraParams& p, int tiles, hipStream_t st) {
  const dim3 grid(tiles, (p.N + 16 * NT * WAVES - 1) / (16 * NT * WAVES));
  if (p.R <= 32)
    lora_expand_kernel<MT, 1, NT, INLINE><<<grid, THREADS, 0, st>>>(p);
  else if (p.R <= 64)
    lora_expand_kernel<MT, 2, NT, INLINE><<<grid, THREADS, 0, st>>>(p);
  else if (p.R <= 128)
    lora_expand_kernel<MT, 4, NT, INLINE><<<grid, THREADS, 0, st>>>(p);
  else if constexpr (MT == 1)
    lora_expand_kernel<MT, 8, NT, INLINE><<<grid, THREADS, 0, st>>>(p);
}

// K ranges: enough workgroups to fill the chip twice, at least one block each.
int k_splits_for(long long tiles, int KB, int num_cus) {
  const long long want = (2LL * num_cus + tiles - 1) / tiles;
  return (int)(want < 1 ? 1 : (want > KB ? KB : want));
}

constexpr int kNoRoom = 1;               // not a dg_status: the scratch memory is too small for so many tokens

int lora_tokens(LoraParams p, const Scratch& sc, hipStream_t st) {
  const int KB = p.K / 128;
  const bool terms = p.L > 0;
  const bool listed = p.T > kInlineTokens;
  // tokens per tile: 16 where every workgroup finds its own tokens and for the
  // largest ranks (their accumulators fill the registers), 64 otherwise
  const int bt = listed && p.R <= 128 ? 64 : 16;
  const int groups = p.L + 1;
  long long rows = p.T;
  size_t list_bytes = 0;
  if (listed) {
    const long long most = groups < p.T ? groups : p.T;
    rows = (p.T + (bt - 1) * most) / bt * bt;
    list_bytes = (size_t)(2 * rows + 64) / 64 * 64 * sizeof(int32_t);
  }
  const long long tiles = listed ? rows / bt : p.T;
  p.k_splits = 1;
  p.kb_per_split = KB;
  if (terms) {
    const size_t one = (size_t)p.T * p.R * sizeof(float);
    if (list_bytes + one > sc.bytes) return kNoRoom;
    int splits = k_splits_for(listed ? tiles : (p.T < p.L ? p.T : p.L), KB, sc.num_cus);
    const size_t room = (sc.bytes - list_bytes) / one;
    if ((size_t)splits > room) splits = (int)room;
    p.kb_per_split = (KB + splits - 1) / splits;
    p.k_splits = (KB + p.kb_per_split - 1) / p.kb_per_split;
    p.partial = reinterpret_cast<float*>(sc.ptr + list_bytes);
  } else if (list_bytes > sc.bytes) {
    return kNoRoom;
  }
  if (listed) {
    int32_t* layout = reinterpret_cast<int32_t*>(sc.ptr);
    LayoutParams lp{p.ids, p.T, 0, groups, bt, 0, (int)rows, layout, nullptr, layout + rows, nullptr};
    lp.others = 1;
    p.layout = layout;
    p.slot_of = layout + rows;
    // the lists' counts may stand where the partial sums come later
    const hipError_t e = launch_layout(lp, sc.ptr + list_bytes, sc.bytes - list_bytes, st);
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
  }
  // 64 columns per wave, or 16 where that would leave most of the chip without work
  const bool wide = tiles * ((p.N + 255) / 256) >= 2 * sc.num_cus;
  if (!listed) {
    if (terms) launch_shrink<1, true>(p, (int)tiles, st);
    if (wide) launch_expand<1, 4, true>(p, (int)tiles, st); else launch_expand<1, 1, true>(p, (int)tiles, st);
  } else if (bt == 64) {
    if (terms) launch_shrink<4, false>(p, (int)tiles, st);
    if (wide) launch_expand<4, 4, false>(p, (int)tiles, st); else launch_expand<4, 1, false>(p, (int)tiles, st);
  } else {
    if (terms) launch_shrink<1, false>(p, (int)tiles, st);
    if (wide) launch_expand<1, 4, false>(p, (int)tiles, st); else launch_expand<1, 1, false>(p, (int)tiles, st);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
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
  if (N > 65535 * 256) return fail(DG_ERR_UNSUPPORTED, "N=%d exceeds %d", N, 65535 * 256);
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
  Scratch sc;
  int s = call_scratch(static_cast<hipStream_t>(stream), &sc);
  if (s != DG_OK) return s;
  LoraParams p{};
  p.a = static_cast<const uint16_t*>(a);
  p.b = static_cast<const uint16_t*>(b);
  p.scales = scales;
  p.ldx = ldx;
  p.ldc = ldc;
  p.ldd = ldd;
  p.N = N;
  p.K = K;
  p.R = R;
  p.L = terms ? num_adapters : 0;
  // as many tokens at a time as the scratch memory has room for, usually all
  int step = T;
  for (int t = 0; t < T;) {
    const int n = T - t < step ? T - t : step;
    p.x = terms ? static_cast<const uint16_t*>(x) + (size_t)t * ldx : nullptr;
    p.ids = adapter_ids + t;
    p.c = c ? static_cast<const uint16_t*>(c) + (size_t)t * ldc : nullptr;
    p.d = static_cast<uint16_t*>(d) + (size_t)t * ldd;
    p.T = n;
    s = lora_tokens(p, sc, static_cast<hipStream_t>(stream));
    if (s == kNoRoom) {
      if (n <= 16)
        return fail(DG_ERR_UNSUPPORTED, "a workspace of %zu bytes has no room for %d tokens of rank %d", sc.bytes, n, R);
      step = (n + 1) / 2;
      continue;
    }
    if (s != DG_OK) return s;
    t += n;
  }
  return DG_OK;
}

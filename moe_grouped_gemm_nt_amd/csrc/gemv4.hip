// Products of a few tokens with 4-bit weights (include/dg.h), dense or with the
// experts of every choice:
//   d[i] = c[i] + sum_k x[row of i][k] * w[expert of i][n][k]
//   w = e2m1(code) * 2^(e - 127), one e per 32 values, or
//   w = (q - zero) * scale, one scale and zero point per group of 32, 64 or 128 values
#include "../../include/dg.h"
#include "dg_host.h"
#include "expert_rows.h"
#include "fp8_gemm_core.h"    // direct global->LDS loads, waits and the 128-byte row swizzle

namespace dg {
namespace {

constexpr int WAVES = 4;
constexpr int THREADS = WAVES * 64;
constexpr int kTile = 16;                // rows of d per workgroup: the columns of an MFMA
// Up to here every workgroup finds its tile's choices itself; beyond, layout kernels
// make lists.
constexpr int kInlineChoices = 512;

struct GemvParams {
  const uint16_t* x;
  const uint8_t* b;
  const int32_t* sfb;      // fp4: [G][K/128][N]
  const void* scales;      // int4: [G][K/group][N]
  const uint8_t* zeros;
  const int32_t* ids;      // expert of each choice, or nullptr: dense
  const uint16_t* c;
  uint16_t* d;
  long long ldx, ldc, ldd;
  int x_div;               // choices that share a row of x
  int i0;                  // first choice of this launch (ids begin there)
  int n;                   // choices, or rows of x
  int first, G;            // experts here: [first, first + G)
  int N, K;
  int tile0, tiles, parts;
  int scales_bf16;
  const int32_t* layout;   // lists (many choices): expert of each row, G = choices of other experts
  const int32_t* slot_of;  // choice of each row, -1 where a tile is not full
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The choices of this workgroup's tile into rows[kTile] (-1 where there is none) and
// their expert into *id (-1: none here).  Returns false for a workgroup without a
// tile.  Ends with a barrier.
//
// Without lists, the workgroup of choice t has a tile if the choices before t hold a
// multiple of 16 of t's expert; its tile is t and the next ones of that expert.
__device__ __forceinline__ bool find_tile(const GemvParams& p, int tile, int* rows, int* id) {
  if (!p.ids) {
    *id = 0;
    const int i = tile * kTile + (int)threadIdx.x;
    if (threadIdx.x < kTile) rows[threadIdx.x] = i < p.n ? i : -1;
  } else if (p.layout) {
    const int g = p.layout[(size_t)tile * kTile];
    if (g < 0) return false;
    *id = g < p.G ? g : -1;
    if (threadIdx.x < kTile) {
      const int i = p.slot_of[(size_t)tile * kTile + threadIdx.x];
      rows[threadIdx.x] = i < 0 ? -1 : p.i0 + i;
    }
  } else {
    const int lane = threadIdx.x & 63;
    auto key = [&](int v) { return v >= p.first && v - p.first < p.G ? v - p.first : -1; };
    int ids[kInlineChoices / 64];
#pragma unroll
    for (int i = 0; i < kInlineChoices / 64; ++i) ids[i] = i * 64 + lane < p.n ? key(p.ids[i * 64 + lane]) : -2;
    const int mine = key(p.ids[tile]);
    if (threadIdx.x < kTile) rows[threadIdx.x] = -1;
    __syncthreads();
    int before = 0, after = 0;
#pragma unroll
    for (int i = 0; i < kInlineChoices / 64; ++i) {
      if (i * 64 >= p.n) break;
      const int s = i * 64 + lane;
      before += __popcll(__ballot(ids[i] == mine && s < tile));
      const uint64_t m = __ballot(ids[i] == mine && s >= tile);
      const int at = after + __popcll(m & ((1ull << lane) - 1));
      if (ids[i] == mine && s >= tile && at < kTile && threadIdx.x < 64) rows[at] = p.i0 + s;
      after += __popcll(m);
    }
    *id = mine;
    if (before % kTile != 0) return false;
  }
  __syncthreads();
  return true;
}

// ---- weights as MFMA operands ------------------------------------------------
__device__ __forceinline__ float e8m0(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight E2M1 codes times 2^(e - 127): bf16 values in the order of K.
__device__ __forceinline__ bf16x8 widen_fp4(uint32_t w, float scale) {
  union {
    bf16x2 h[4];
    bf16x8 v;
  } u;
  u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return u.v;
}

// Eight integers of 0 to 15 as bf16, those of even K first.  A byte of that value
// is, read as e4m3, its value times 2^-9: subnormal up to 7, and of the first
// exponent, whose step is the same, from 8 on.
__device__ __forceinline__ bf16x8 widen_int4(uint32_t w) {
  const int even = (int)(w & 0x0F0F0F0Fu), odd = (int)((w >> 4) & 0x0F0F0F0Fu);
  union {
    bf16x2 h[4];
    bf16x8 v;
  } u;
  u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, false);
  u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, true);
  u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, false);
  u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, true);
  return u.v;
}
// Eight values of x in that order
__device__ __forceinline__ bf16x8 even_first(u32x4 x) {
  const u32x4 v = {__builtin_amdgcn_perm(x[1], x[0], 0x05040100), __builtin_amdgcn_perm(x[3], x[2], 0x05040100),
                   __builtin_amdgcn_perm(x[1], x[0], 0x07060302), __builtin_amdgcn_perm(x[3], x[2], 0x07060302)};
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ float load_scale(const GemvParams& p, size_t at) {
  return p.scales_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.scales)[at])
                       : static_cast<const float*>(p.scales)[at];
}

// GROUP 0: E2M1 codes.  16 columns of d per workgroup, as the MFMA's rows, and the
// tile's choices as its columns; the four waves take blocks of 128 K in turn.
template <int GROUP>
__global__ __launch_bounds__(THREADS) void gemv_kernel(GemvParams p) {
  __shared__ int rows[kTile];
  __shared__ f32x4 sums[WAVES][64];
  int id;
  const int tile = p.tile0 + (int)(blockIdx.x / p.parts), part = blockIdx.x % p.parts;
  if (!find_tile(p, tile, rows, &id)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g16 = lane >> 4;
  const int n0 = part * 16;
  f32x4 acc = {};
  if (id >= 0) {
    const int n = min(n0 + r16, p.N - 1);                        // beyond N: not stored
    const int i = rows[r16] >= 0 ? rows[r16] : rows[0];          // nor rows without a choice
    const uint16_t* x = p.x + (size_t)(i / p.x_div) * p.ldx;
    const uint8_t* b = p.b + ((size_t)id * p.N + n) * (p.K / 2);
    for (int kb = wave; kb < p.K / 128; kb += WAVES) {
      if constexpr (GROUP == 0) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(b + kb * 64 + g16 * 16);
        const uint32_t e = (uint32_t)p.sfb[((size_t)id * (p.K / 128) + kb) * p.N + n];
        const float scale = e8m0((e >> (8 * g16)) & 255);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 xf = *reinterpret_cast<const bf16x8*>(x + (size_t)kb * 128 + g16 * 32 + j * 8);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_fp4(w[j], scale), xf, acc, 0, 0, 0);
        }
      } else {
        const bf16x8 ones = {(__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f,
                             (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f};
        f32x4 q = {}, xsum = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(b + kb * 64 + j * 16 + g16 * 4);
          const bf16x8 xf = even_first(*reinterpret_cast<const u32x4*>(x + (size_t)kb * 128 + j * 32 + g16 * 8));
          q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_int4(w), xf, q, 0, 0, 0);
          xsum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xf, xsum, 0, 0, 0);
          if ((j + 1) * 32 % GROUP == 0) {
            const size_t at = ((size_t)id * (p.K / GROUP) + (kb * 128 + j * 32) / GROUP) * p.N;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int m = min(n0 + g16 * 4 + e, p.N - 1);
              const float zero = p.zeros ? (float)p.zeros[at + m] : 8.0f;
              acc[e] = fmaf(load_scale(p, at + m), fmaf(-zero, xsum[e], q[e]), acc[e]);
            }
            q = f32x4{};
            xsum = f32x4{};
          }
        }
      }
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  // thread: choice threadIdx.x / 16, column threadIdx.x % 16
  const int at = threadIdx.x >> 4, n = n0 + (threadIdx.x & 15);
  const int i = rows[at];
  if (i < 0 || n >= p.N) return;
  float v = p.c ? bf16_to_f32(p.c[(size_t)i * p.ldc + n]) : 0.0f;
  const int from = ((threadIdx.x & 15) >> 2) * 16 + at, e = threadIdx.x & 3;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) sum += sums[w][from][e];
  p.d[(size_t)i * p.ldd + n] = f32_to_bf16(v + sum);
}

constexpr long long kMaxChoices = 1LL << 30;
constexpr int kMaxColumns = 1 << 20;
constexpr int kMostGroups = 1 << 22;     // workgroups per launch: a grid has fewer than 2^32 threads

int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

int launch_tiles(GemvParams p, int group, long long tiles, hipStream_t st) {
  p.parts = (p.N + 15) / 16;
  const long long step = kMostGroups / p.parts;
  for (long long t = 0; t < tiles; t += step) {
    p.tile0 = (int)t;
    p.tiles = (int)(tiles - t < step ? tiles - t : step);
    const int grid = p.tiles * p.parts;
    if (group == 0)
      gemv_kernel<0><<<grid, THREADS, 0, st>>>(p);
    else if (group == 32)
      gemv_kernel<32><<<grid, THREADS, 0, st>>>(p);
    else if (group == 64)
      gemv_kernel<64><<<grid, THREADS, 0, st>>>(p);
    else
      gemv_kernel<128><<<grid, THREADS, 0, st>>>(p);
    const int s = launched();
    if (s != DG_OK) return s;
  }
  return DG_OK;
}

// By choice: as many choices at a time as the scratch memory has room to list,
// usually all, or kInlineChoices without lists.
int launch_choices(GemvParams p, int group, int n, const int32_t* ids, hipStream_t st) {
  Scratch sc;
  int s = call_scratch(st, &sc);
  if (s != DG_OK) return s;
  const long long groups = p.G + 1;
  for (int i = 0; i < n;) {
    int step = n - i;
    size_t list_bytes = 0;
    long long rows = 0;
    while (step > kInlineChoices) {
      rows = (step + (kTile - 1) * (groups < step ? groups : step)) / kTile * kTile;
      list_bytes = (size_t)(2 * rows + 64) / 64 * 64 * sizeof(int32_t);
      if (list_bytes <= sc.bytes && rows < (1LL << 30)) break;
      step = step / 2 > kInlineChoices ? step / 2 : kInlineChoices;
    }
    p.i0 = i;
    p.n = step;
    p.ids = ids + i;
    p.layout = nullptr;
    p.slot_of = nullptr;
    long long tiles = step;
    if (step > kInlineChoices) {
      int32_t* layout = reinterpret_cast<int32_t*>(sc.ptr);
      LayoutParams lp{p.ids, step, p.first, (int)groups, kTile, 0, (int)rows, layout, nullptr, layout + rows, nullptr};
      lp.others = 1;
      const hipError_t e = launch_layout(lp, sc.ptr + list_bytes, sc.bytes - list_bytes, st);
      if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
      p.layout = layout;
      p.slot_of = layout + rows;
      tiles = rows / kTile;
    }
    s = launch_tiles(p, group, tiles, st);
    if (s != DG_OK) return s;
    i += step;
  }
  return DG_OK;
}

// What the four calls share.  rows: rows of d; x_rows: rows of x.
int check_gemv(const GemvParams& p, long long rows, const void* scales, size_t scale_size, int ldx, int ldc, int ldd) {
  if (p.N < 0 || p.K < 0) return fail(DG_ERR_INVALID_ARG, "negative size (N=%d K=%d)", p.N, p.K);
  if (p.K % 128 != 0) return fail(DG_ERR_INVALID_ARG, "K=%d is not a multiple of 128", p.K);
  if (p.N > kMaxColumns) return fail(DG_ERR_UNSUPPORTED, "N=%d exceeds 2^20", p.N);
  if (rows == 0 || p.N == 0) return DG_OK;
  if (!p.d) return fail(DG_ERR_INVALID_ARG, "d must not be NULL");
  const bool terms = p.G > 0 && p.K > 0;                         // without them d = c
  if (terms && (!p.x || !p.b || !scales)) return fail(DG_ERR_INVALID_ARG, "x, b and its scales must not be NULL");
  if (terms && (!aligned(p.x, 16) || !aligned(p.b, 16)))
    return fail(DG_ERR_INVALID_ARG, "x and b must be 16-byte aligned");
  if (terms && !aligned(scales, scale_size))
    return fail(DG_ERR_INVALID_ARG, "the scales must be aligned to their type");
  if (terms && (ldx < p.K || ldx % 8 != 0))
    return fail(DG_ERR_INVALID_ARG, "ldx=%d must be a multiple of 8 and at least K=%d", ldx, p.K);
  if (ldd < p.N || (p.c && ldc < p.N))
    return fail(DG_ERR_INVALID_ARG, "ldc=%d and ldd=%d must be at least N=%d", ldc, ldd, p.N);
  if (p.c == p.d && ldc != ldd)
    return fail(DG_ERR_INVALID_ARG, "c may equal d only with ldc=%d equal to ldd=%d", ldc, ldd);
  if (!aligned(p.c, 2) || !aligned(p.d, 2)) return fail(DG_ERR_INVALID_ARG, "c and d must be 2-byte aligned");
  return DG_OK;
}

int check_int4(int group, int scales_type) {
  if (group != 32 && group != 64 && group != 128)
    return fail(DG_ERR_INVALID_ARG, "group_size=%d is neither 32, 64 nor 128", group);
  if (scales_type != DG_F32 && scales_type != DG_BF16)
    return fail(DG_ERR_INVALID_ARG, "scales_type=%d is neither DG_F32 nor DG_BF16", scales_type);
  return DG_OK;
}

int dense(GemvParams& p, int group, int M, const void* scales, size_t scale_size, int ldx, int ldc, int ldd,
          void* stream) {
  if (M < 0) return fail(DG_ERR_INVALID_ARG, "negative size (M=%d)", M);
  p.G = 1;
  p.x_div = 1;
  p.n = M;
  const int s = check_gemv(p, M, scales, scale_size, ldx, ldc, ldd);
  if (s != DG_OK || M == 0 || p.N == 0) return s;
  return launch_tiles(p, group, ((long long)M + kTile - 1) / kTile, static_cast<hipStream_t>(stream));
}

int by_choice(GemvParams& p, int group, int x_rows, const int32_t* ids, int T, int top_k, const void* scales,
              size_t scale_size, int ldx, int ldc, int ldd, void* stream) {
  if (T < 0 || top_k < 1) return fail(DG_ERR_INVALID_ARG, "T=%d must not be negative and top_k=%d at least 1", T, top_k);
  const long long n = (long long)T * top_k;
  if (n > kMaxChoices) return fail(DG_ERR_UNSUPPORTED, "T * top_k = %lld choices exceed 2^30", n);
  if (x_rows != T && x_rows != n)
    return fail(DG_ERR_INVALID_ARG, "x_rows=%d is neither T=%d nor T * top_k=%lld", x_rows, T, n);
  if (p.G < 0) return fail(DG_ERR_INVALID_ARG, "num_groups=%d must not be negative", p.G);
  if (p.G > kMaxLayoutGroups) return fail(DG_ERR_UNSUPPORTED, "num_groups=%d exceeds %d", p.G, kMaxLayoutGroups);
  if (p.first < 0) return fail(DG_ERR_INVALID_ARG, "first_expert=%d must not be negative", p.first);
  p.x_div = x_rows == n ? 1 : top_k;
  int s = check_gemv(p, n, scales, scale_size, ldx, ldc, ldd);
  if (s != DG_OK) return s;
  if (n > 0 && p.N > 0 && (!ids || !aligned(ids, 4)))
    return fail(DG_ERR_INVALID_ARG, "topk_ids must be a 4-byte aligned address");
  if (n == 0 || p.N == 0) return DG_OK;
  return launch_choices(p, group, (int)n, ids, static_cast<hipStream_t>(stream));
}

GemvParams operands(const void* x, int ldx, const void* b, const void* c, int ldc, void* d, int ldd, int N, int K) {
  GemvParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.b = static_cast<const uint8_t*>(b);
  p.c = static_cast<const uint16_t*>(c);
  p.d = static_cast<uint16_t*>(d);
  p.ldx = ldx;
  p.ldc = ldc;
  p.ldd = ldd;
  p.N = N;
  p.K = K;
  return p;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" int dg_bf16_fp4_gemv_nt(const void* x, int ldx, const void* b, const int32_t* sfb, const void* c, int ldc,
                                   void* d, int ldd, int M, int N, int K, void* stream) {
  GemvParams p = operands(x, ldx, b, c, ldc, d, ldd, N, K);
  p.sfb = sfb;
  return dense(p, 0, M, sfb, 4, ldx, ldc, ldd, stream);
}

extern "C" int dg_bf16_int4_gemv_nt(const void* x, int ldx, const void* b, const void* scales, int scales_type,
                                    const void* zeros, int group_size, const void* c, int ldc, void* d, int ldd, int M,
                                    int N, int K, void* stream) {
  const int s = check_int4(group_size, scales_type);
  if (s != DG_OK) return s;
  GemvParams p = operands(x, ldx, b, c, ldc, d, ldd, N, K);
  p.scales = scales;
  p.scales_bf16 = scales_type == DG_BF16;
  p.zeros = static_cast<const uint8_t*>(zeros);
  return dense(p, group_size, M, scales, scales_type == DG_F32 ? 4 : 2, ldx, ldc, ldd, stream);
}

extern "C" int dg_m_grouped_bf16_fp4_gemv_nt_topk(const void* x, int ldx, int x_rows, const int32_t* topk_ids,
                                                  const void* b, const int32_t* sfb, const void* c, int ldc, void* d,
                                                  int ldd, int T, int top_k, int first_expert, int num_groups, int N,
                                                  int K, void* stream) {
  GemvParams p = operands(x, ldx, b, c, ldc, d, ldd, N, K);
  p.sfb = sfb;
  p.first = first_expert;
  p.G = num_groups;
  return by_choice(p, 0, x_rows, topk_ids, T, top_k, sfb, 4, ldx, ldc, ldd, stream);
}

extern "C" int dg_m_grouped_bf16_int4_gemv_nt_topk(const void* x, int ldx, int x_rows, const int32_t* topk_ids,
                                                   const void* b, const void* scales, int scales_type,
                                                   const void* zeros, int group_size, const void* c, int ldc, void* d,
                                                   int ldd, int T, int top_k, int first_expert, int num_groups, int N,
                                                   int K, void* stream) {
  const int s = check_int4(group_size, scales_type);
  if (s != DG_OK) return s;
  GemvParams p = operands(x, ldx, b, c, ldc, d, ldd, N, K);
  p.scales = scales;
  p.scales_bf16 = scales_type == DG_BF16;
  p.zeros = static_cast<const uint8_t*>(zeros);
  p.first = first_expert;
  p.G = num_groups;
  return by_choice(p, group_size, x_rows, topk_ids, T, top_k, scales, scales_type == DG_F32 ? 4 : 2, ldx, ldc, ldd,
                   stream);
}

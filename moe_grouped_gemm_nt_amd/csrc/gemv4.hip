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

constexpr int kTile = 16;                // rows of d per workgroup: the columns of an MFMA
// Up to here every workgroup finds its tile's choices itself; beyond, layout kernels
// make lists.
constexpr int kInlineChoices = 2048;

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
  int tiles;               // tiles of choices, or the most there can be
  long long item0;         // of tiles * parts, in this launch
  int items;
  int scales_bf16;
  const int32_t* layout;   // lists (many choices): expert of each row, G = choices of other experts
  const int32_t* slot_of;  // choice of each row, -1 where a tile is not full
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef u16x4 u16x4_u __attribute__((aligned(2)));               // at any address of its elements

// The choices of tile `tile` into rows[kTile] (-1 where there is none) and their
// expert into *id (-1: none here).  Returns false where there is no such tile.  Ends
// with a barrier.
//
// Without lists every workgroup counts the experts' choices in LDS (`room`), so that
// the tiles are numbered by expert without gaps and few workgroups find none, and
// takes its sixteen in the order of the choices.
template <int THREADS>
__device__ __forceinline__ bool find_tile(const GemvParams& p, int tile, int* rows, int* id, int* room) {
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
    int* count = room;                                           // [G + 1], the last of choices that are not here
    int16_t* group = reinterpret_cast<int16_t*>(room + kMaxLayoutGroups + 1);            // [n]
    for (int g = threadIdx.x; g <= p.G; g += THREADS) count[g] = 0;
    if (threadIdx.x < kTile) rows[threadIdx.x] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += THREADS) {
      const long long e = (long long)p.ids[i] - p.first;
      const int g = e >= 0 && e < p.G ? (int)e : p.G;
      group[i] = (int16_t)g;
      atomicAdd(&count[g], 1);
    }
    __syncthreads();
    const int lane = threadIdx.x & 63;
    int before = 0, mine = -1, at = 0;                           // tiles of the groups so far; the tile's group and place
    for (int base = 0; base <= p.G && mine < 0; base += 64) {
      const int tiles = base + lane <= p.G ? (count[base + lane] + kTile - 1) / kTile : 0;
      int upto = tiles;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o);
        upto += lane >= o ? v : 0;
      }
      const uint64_t past = __ballot(before + upto > tile);
      if (past) {
        const int first = __ffsll((unsigned long long)past) - 1;
        mine = base + first;
        at = tile - before - __shfl(upto - tiles, first);
      }
      before += __shfl(upto, 63);
    }
    if (mine < 0) return false;
    *id = mine < p.G ? mine : -1;
    if (threadIdx.x < 64) {
      int seen = -at * kTile;
      for (int base = 0; base < p.n && seen < kTile; base += 64) {
        const bool is = base + lane < p.n && group[base + lane] == mine;
        const uint64_t m = __ballot(is);
        const int to = seen + __popcll(m & ((1ull << lane) - 1));
        if (is && to >= 0 && to < kTile) rows[to] = p.i0 + base + lane;
        seen += __popcll(m);
      }
    }
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

// ---- the kernel ----------------------------------------------------------------
// A workgroup has 16 * RT columns of d, as the MFMA's rows, for one tile of choices,
// the MFMA's columns; its W waves take pieces of 256 K in turn, each with LDS of its
// own (no barrier until the sums are joined).  Bound by reading the weights.
//
// A piece's rows of weights (one 128-byte line each) and of x come into LDS with
// direct loads of whole lines, as many pieces at a time as there is room for, and
// are read from there as MFMA operands.  (Operands loaded straight from memory,
// sixteen rows at a time, occupy the CU's memory pipe for one cycle per row and
// 16 bytes: 64 tokens of 8 of 128 experts, 32 of them here, of 4096 x 7168 took 307
// us.)  A row's 16-byte chunk c lies at c ^ swz(row) (weights) or c ^ row (x).
//
// FORM 0: E2M1 codes, scaled as they are widened, so that one sum runs over K.
// Otherwise the group size: a group's sum of q * x and its sum of x (a product with
// ones) are joined and scaled when it ends.
template <int FORM, int RT, int XL>
struct Slot {
  static constexpr int kWeights = RT * 2048;
  static constexpr int kX = XL * 1024;                           // two rows of 256 values per load
  static constexpr int kScales = FORM == 0 ? (RT < 2 ? 256 : RT * 128) : 256 / (FORM ? FORM : 1) * RT * 16 * 8;
  static constexpr int kBytes = kWeights + kX + kScales;
};

template <int FORM, int RT>
constexpr int kWaveBytes = (Slot<FORM, RT, 8>::kBytes + 255) / 256 * 256;

template <int FORM, int RT, int W, int XL>
__device__ __forceinline__ void sum_pieces(const GemvParams& p, const int* rows, int id, int n0, int wave, uint8_t* own,
                                           f32x4 (&acc)[RT]) {
  typedef Slot<FORM, RT, XL> S;
  constexpr int UP = kWaveBytes<FORM, RT> / S::kBytes < 4 ? kWaveBytes<FORM, RT> / S::kBytes : 4;
  constexpr int ITEMS = FORM ? (256 / (FORM ? FORM : 1) * RT * 16 + 63) / 64 : 1;        // scales per lane and piece
  const int lane = threadIdx.x & 63, r16 = lane & 15, g16 = lane >> 4;
  const int pieces = (p.K + 255) / 256;
  const bool odd = (p.K & 128) != 0;           // the last piece is half as long: its second half repeats the first
  const uint8_t* wsrc[2 * RT];
#pragma unroll
  for (int l = 0; l < 2 * RT; ++l)             // columns beyond N repeat the last: not stored
    wsrc[l] = p.b + ((size_t)id * p.N + min(n0 + l * 8 + (lane >> 3), p.N - 1)) * (p.K / 2);
  const uint16_t* xsrc[XL];
#pragma unroll
  for (int l = 0; l < XL; ++l) {
    const int i = rows[2 * l + (lane >> 5)];   // a row without a choice repeats the first: not stored
    xsrc[l] = p.x + (size_t)((i >= 0 ? i : rows[0]) / p.x_div) * p.ldx;
  }
  const uint32_t base = lds_u32(own);
  for (int i = wave; i < pieces; i += W * UP) {
    float sc[UP][ITEMS], zs[UP][ITEMS];
#pragma unroll
    for (int u = 0; u < UP; ++u) {
      const int piece = i + u * W;
      if (piece >= pieces) break;
      const bool half = odd && piece == pieces - 1;
      const uint32_t slot = __builtin_amdgcn_readfirstlane(base + u * S::kBytes);
      if constexpr (FORM != 0) {
        const size_t row0 = ((size_t)id * (p.K / FORM) + (size_t)piece * (256 / FORM)) * p.N;
#pragma unroll
        for (int t = 0; t < ITEMS; ++t) {
          const int item = t * 64 + lane;
          const int g = half ? (item / (16 * RT)) & (128 / FORM - 1) : (item / (16 * RT)) & (256 / FORM - 1);
          const size_t at = row0 + (size_t)g * p.N + min(n0 + item % (16 * RT), p.N - 1);
          sc[u][t] = p.scales_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.scales)[at])
                                   : static_cast<const float*>(p.scales)[at];
          zs[u][t] = p.zeros ? (float)p.zeros[at] : 8.0f;
        }
      } else {
        const int kb = piece * 2, row = lane % (16 * RT < 64 ? 16 * RT : 64);
        if constexpr (RT < 4) {
          const int h = half ? 0 : (lane / (16 * RT)) & 1;
          dma_4(p.sfb + ((size_t)id * (p.K / 128) + kb + h) * p.N + min(n0 + row, p.N - 1),
                __builtin_amdgcn_readfirstlane(slot + S::kWeights + S::kX));
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            dma_4(p.sfb + ((size_t)id * (p.K / 128) + kb + (half ? 0 : h)) * p.N + min(n0 + row, p.N - 1),
                  __builtin_amdgcn_readfirstlane(slot + S::kWeights + S::kX + h * 256));
        }
      }
#pragma unroll
      for (int l = 0; l < 2 * RT; ++l) {
        int chunk = (lane & 7) ^ swz(l * 8 + (lane >> 3));
        chunk = half ? chunk & 3 : chunk;
        dma_16_nt(wsrc[l] + (size_t)piece * 128 + chunk * 16, __builtin_amdgcn_readfirstlane(slot + l * 1024));
      }
#pragma unroll
      for (int l = 0; l < XL; ++l) {
        int chunk = (lane & 31) ^ (2 * l + (lane >> 5));
        chunk = half ? chunk & 15 : chunk;
        dma_16(xsrc[l] + (size_t)piece * 256 + chunk * 8,
               __builtin_amdgcn_readfirstlane(slot + S::kWeights + l * 1024));
      }
    }
    wait_vm_lgkm0<0>();
    asm volatile("" ::: "memory");
    if constexpr (FORM != 0) {
#pragma unroll
      for (int u = 0; u < UP; ++u) {
        if (i + u * W >= pieces) break;
        float2* to = reinterpret_cast<float2*>(own + u * S::kBytes + S::kWeights + S::kX);
#pragma unroll
        for (int t = 0; t < ITEMS; ++t)
          if (t * 64 + lane < 256 / FORM * RT * 16) to[t * 64 + lane] = make_float2(sc[u][t], -sc[u][t] * zs[u][t]);
      }
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int u = 0; u < UP; ++u) {
      const int piece = i + u * W;
      if (piece >= pieces) break;
      const uint8_t* slot = own + u * S::kBytes;
      const uint8_t* xs = slot + S::kWeights;
      const int xrow = r16 & (2 * XL - 1);     // columns from 2 * XL on repeat others: not stored
      f32x4 q[RT] = {}, xsum = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && odd && piece == pieces - 1) break;
        u32x4 w[RT];
        float scale[RT];
        if constexpr (FORM == 0) {
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int row = r * 16 + r16;
            w[r] = *reinterpret_cast<const u32x4*>(slot + row * 128 + (((h * 4 + g16) ^ swz(row)) << 4));
            const uint32_t e = reinterpret_cast<const uint32_t*>(xs + S::kX)[h * 16 * RT + row];
            scale[r] = e8m0((e >> (8 * g16)) & 255);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // K of lane group g: codes g * 32 + j * 8 of a block, integers j * 32 + g * 8
          const int chunk = FORM == 0 ? (h * 4 + g16) * 4 + j : (h * 4 + j) * 4 + g16;
          const u32x4 xv = *reinterpret_cast<const u32x4*>(xs + xrow * 512 + ((chunk ^ xrow) << 4));
          if constexpr (FORM == 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
              acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_fp4(w[r][j], scale[r]),
                                                               __builtin_bit_cast(bf16x8, xv), acc[r], 0, 0, 0);
          } else {
            const bf16x8 ones = {(__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f,
                                 (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f};
            const bf16x8 xf = even_first(xv);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const int row = r * 16 + r16;
              const uint32_t v = *reinterpret_cast<const uint32_t*>(slot + row * 128 + (((h * 4 + j) ^ swz(row)) << 4) +
                                                                    g16 * 4);
              q[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_int4(v), xf, q[r], 0, 0, 0);
            }
            xsum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xf, xsum, 0, 0, 0);
            constexpr int STEPS = FORM ? FORM / 32 : 1;
            if ((j + 1) % STEPS == 0) {
              const int g = (h * 4 + j) / STEPS;
#pragma unroll
              for (int r = 0; r < RT; ++r) {
                const f32x4* s = reinterpret_cast<const f32x4*>(xs + S::kX + (g * 16 * RT + r * 16 + g16 * 4) * 8);
                const f32x4 s0 = s[0], s1 = s[1];
                acc[r][0] = fmaf(s0[1], xsum[0], fmaf(s0[0], q[r][0], acc[r][0]));
                acc[r][1] = fmaf(s0[3], xsum[0], fmaf(s0[2], q[r][1], acc[r][1]));
                acc[r][2] = fmaf(s1[1], xsum[0], fmaf(s1[0], q[r][2], acc[r][2]));
                acc[r][3] = fmaf(s1[3], xsum[0], fmaf(s1[2], q[r][3], acc[r][3]));
                q[r] = f32x4{};
              }
              xsum = f32x4{};
            }
          }
        }
      }
    }
    wait_vm_lgkm0<0>();                        // the slots are read before the next round fills them
    asm volatile("" ::: "memory");
  }
}

template <int FORM, int RT, int W>
__global__ __launch_bounds__(W * 64) void gemv_kernel(GemvParams p) {
  __shared__ int rows[kTile];
  __shared__ __attribute__((aligned(128))) uint8_t lds[W][kWaveBytes<FORM, RT>];
  static_assert(sizeof(lds) >= (kMaxLayoutGroups + 1) * 4 + kInlineChoices * 2, "find_tile's room");
  // consecutive workgroups go to the 8 XCDs in turn: each takes a run of items, the
  // tiles of the same columns next to one another, for those that share an expert
  const int per = (p.items + 7) / 8;
  const int item = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || item >= p.items) return;
  const int part = (int)((p.item0 + item) / p.tiles), tile = (int)(p.item0 + item - (long long)part * p.tiles);
  int id;
  if (!find_tile<W * 64>(p, tile, rows, &id, reinterpret_cast<int*>(&lds[0][0]))) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g16 = lane >> 4;
  const int n0 = part * 16 * RT;
  f32x4 acc[RT] = {};
  if (id >= 0) {
    if (rows[8] >= 0)
      sum_pieces<FORM, RT, W, 8>(p, rows, id, n0, wave, lds[wave], acc);
    else if (rows[4] >= 0)
      sum_pieces<FORM, RT, W, 4>(p, rows, id, n0, wave, lds[wave], acc);
    else if (rows[2] >= 0)
      sum_pieces<FORM, RT, W, 2>(p, rows, id, n0, wave, lds[wave], acc);
    else
      sum_pieces<FORM, RT, W, 1>(p, rows, id, n0, wave, lds[wave], acc);
    f32x4* sums = reinterpret_cast<f32x4*>(lds[wave]);
#pragma unroll
    for (int r = 0; r < RT; ++r) sums[r * 64 + lane] = acc[r];
    __syncthreads();
  }
  const int i = rows[r16];
  if (i < 0) return;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (r % W != wave) continue;               // the waves share the sixteenths of the columns
    const int n = n0 + r * 16 + g16 * 4;
    if (n >= p.N) continue;
    f32x4 sum = {};
    if (id >= 0)
#pragma unroll
      for (int w = 0; w < W; ++w) sum += reinterpret_cast<const f32x4*>(lds[w])[r * 64 + lane];
    const uint16_t* c = p.c ? p.c + (size_t)i * p.ldc + n : nullptr;
    uint16_t* d = p.d + (size_t)i * p.ldd + n;
    if (n + 4 <= p.N) {
      u16x4 v = {};
      if (c) v = *reinterpret_cast<const u16x4_u*>(c);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = id >= 0 ? f32_to_bf16(bf16_to_f32(v[e]) + sum[e]) : v[e];
      *reinterpret_cast<u16x4_u*>(d) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (n + e < p.N) {
          const uint16_t v = c ? c[e] : 0;
          d[e] = id >= 0 ? f32_to_bf16(bf16_to_f32(v) + sum[e]) : v;
        }
    }
  }
}

constexpr long long kMaxChoices = 1LL << 30;
constexpr int kMaxColumns = 1 << 20;
constexpr int kMostGroups = 1 << 22;     // workgroups per launch: a grid has fewer than 2^32 threads

int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

template <int RT, int W>
int launch_items(GemvParams p, int group, hipStream_t st) {
  const long long items = (long long)p.tiles * ((p.N + 16 * RT - 1) / (16 * RT));
  for (long long at = 0; at < items; at += p.items) {
    p.item0 = at;
    p.items = (int)(items - at < kMostGroups ? items - at : kMostGroups);
    const int grid = (p.items + 7) / 8 * 8;
    if (group == 0)
      gemv_kernel<0, RT, W><<<grid, W * 64, 0, st>>>(p);
    else if (group == 32)
      gemv_kernel<32, RT, W><<<grid, W * 64, 0, st>>>(p);
    else if (group == 64)
      gemv_kernel<64, RT, W><<<grid, W * 64, 0, st>>>(p);
    else
      gemv_kernel<128, RT, W><<<grid, W * 64, 0, st>>>(p);
    const int s = launched();
    if (s != DG_OK) return s;
  }
  return DG_OK;
}

int launch_tiles(GemvParams p, int group, long long tiles, hipStream_t st) {
  p.tiles = (int)tiles;
  return launch_items<2, 4>(p, group, st);
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
    // an expert's last tile may not be full
    long long tiles = (groups < step ? groups : step) + step / kTile;
    tiles = tiles < step ? tiles : step;
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

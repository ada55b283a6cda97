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

// Up to here every workgroup finds its tile's choices itself, in four loads per thread
// at the most; beyond, layout kernels make lists, in launches of their own.  Inline and
// with lists, replayed from a graph: 64 tokens of 8 of 128 experts of 512 x 1024 13.1 us
// and 18.5, 128 14.7 and 19.3, of 4096 x 7168 with 32 experts here 64 tokens 92 and 94,
// 128 111 and 110; with the limit raised to 2048 (eight loads) 256 tokens of the small
// experts 23.3 and 24.1, of the large ones 151 and 145.
constexpr int kInlineChoices = 1024;

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
  int others;              // tiles before them that look after choices of experts that are not here
  int tile0, part0;        // first of this launch
  int items;               // tiles * parts of this launch
  int scales_bf16;
  int again;               // several tiles read the same weights
  const int32_t* layout;   // lists (many choices): expert of each row, G = choices of other experts
  const int32_t* slot_of;  // choice of each row, -1 where a tile is not full
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef u16x4 u16x4_u __attribute__((aligned(2)));               // at any address of its elements

// The local expert of an id, or -1
__device__ __forceinline__ int local_expert(const GemvParams& p, int id) {
  return id >= p.first && (unsigned)(id - p.first) < (unsigned)p.G ? id - p.first : -1;
}

__device__ __forceinline__ int wave_scan(int v) {                // sums over the lanes up to this one
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);          // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);          // row_bcast 15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);          // row_bcast 31 into rows 2 and 3
  return v;
}

// The choices of tile `tile` into rows[16] (-1 where there is none) and their expert
// into *id (-1: none here).  Returns false where there is no such tile.  Ends with a
// barrier.
//
// Without lists every workgroup counts the experts' choices in LDS (`room`), so that
// the tiles are numbered by expert without gaps and few workgroups find none.  An
// expert's only tile takes its choices in whatever order they were counted (no
// result depends on a choice's place in its tile), one of several its sixteen in
// the order of the choices, which all of its workgroups find alike.
template <int THREADS, int TILE>
__device__ __forceinline__ bool find_tile(const GemvParams& p, int tile, int* rows, int* id, int* room) {
  if (!p.ids) {
    *id = 0;
    const int i = tile * TILE + (int)threadIdx.x;
    if (threadIdx.x < 16) rows[threadIdx.x] = threadIdx.x < TILE && i < p.n ? i : -1;
  } else if (p.layout) {
    const int g = p.layout[(size_t)tile * TILE];
    if (g < 0) return false;
    *id = g < p.G ? g : -1;
    if (threadIdx.x < 16) {
      const int i = threadIdx.x < TILE ? p.slot_of[(size_t)tile * TILE + threadIdx.x] : -1;
      rows[threadIdx.x] = i < 0 ? -1 : p.i0 + i;
    }
  } else {
    constexpr int MOST = kInlineChoices / THREADS;
    int* count = room;                                           // [G]
    int e[MOST], place[MOST];
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      const int i = threadIdx.x + j * THREADS;
      e[j] = i < p.n ? p.ids[i] : -1;
    }
    for (int g = threadIdx.x; g < p.G; g += THREADS) count[g] = 0;
    if (threadIdx.x < 16) rows[threadIdx.x] = -1;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      if (j * THREADS >= p.n) break;
      e[j] = local_expert(p, e[j]);                              // (-1 stays it: first >= 0)
      if (e[j] >= 0) place[j] = atomicAdd(&count[e[j]], 1);
    }
    __syncthreads();
    const int lane = threadIdx.x & 63;
    int before = 0, mine = -1, at = 0;                           // tiles of the experts so far; the tile's expert and place
    for (int base = 0; base < p.G && mine < 0; base += 64) {
      const int tiles = base + lane < p.G ? (count[base + lane] + TILE - 1) / TILE : 0;
      const int upto = wave_scan(tiles);
      const uint64_t past = __ballot(before + upto > tile);
      if (past) {
        const int first = __ffsll((unsigned long long)past) - 1;
        mine = base + first;
        at = tile - before - __builtin_amdgcn_readlane(upto - tiles, first);
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (mine < 0) return false;
    *id = mine;
    if (count[mine] <= TILE) {
#pragma unroll
      for (int j = 0; j < MOST; ++j) {
        if (j * THREADS >= p.n) break;
        if (e[j] == mine) rows[place[j]] = p.i0 + (int)threadIdx.x + j * THREADS;
      }
    } else {
      // several tiles: in the order of the choices, by the numbers before each 64
      constexpr int WAVES = THREADS / 64;
      int* per = room + kMaxLayoutGroups;                        // [MOST * WAVES]
      const int wave = threadIdx.x / 64;
      uint64_t m[MOST];
#pragma unroll
      for (int j = 0; j < MOST; ++j) {
        m[j] = __ballot(e[j] == mine);
        if (lane == 0) per[j * WAVES + wave] = __popcll(m[j]);
      }
      __syncthreads();
      const int v = lane < MOST * WAVES ? per[lane] : 0, upto = wave_scan(v);
#pragma unroll
      for (int j = 0; j < MOST; ++j) {
        const int to = __shfl(upto - v, j * WAVES + wave) + __popcll(m[j] & ((1ull << lane) - 1)) - at * TILE;
        if (e[j] == mine && to >= 0 && to < TILE) rows[to] = p.i0 + (int)threadIdx.x + j * THREADS;
      }
    }
  }
  __syncthreads();
  return true;
}

// Columns n0 .. n0 + columns - 1 of the choices of experts that are not here, of 64
// choices from `first` on: c as it is, or zeros.
template <int THREADS>
__device__ __forceinline__ void write_others(const GemvParams& p, int first, int n0, int columns) {
  for (int at = threadIdx.x; at < 64 * (columns / 4); at += THREADS) {
    const int i = first + at / (columns / 4), n = n0 + at % (columns / 4) * 4;
    if (i >= p.n || n >= p.N || local_expert(p, p.ids[i]) >= 0) continue;
    const uint16_t* c = p.c ? p.c + (size_t)(p.i0 + i) * p.ldc + n : nullptr;
    uint16_t* d = p.d + (size_t)(p.i0 + i) * p.ldd + n;
    if (n + 4 <= p.N)
      *reinterpret_cast<u16x4_u*>(d) = c ? *reinterpret_cast<const u16x4_u*>(c) : u16x4{};
    else
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (n + e < p.N) d[e] = c ? c[e] : 0;
  }
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
// A workgroup has 16 * RT columns of d, as the MFMA's columns, for one tile of choices,
// the MFMA's rows; its W waves take pieces of 256 K in turn, each with LDS of its own
// (no barrier until the sums are joined).
//
// Bound by reading the weights where these are many: one token of 65536 x 7168 takes
// 36.7 us (6.8 TB/s of FP4; a device copy reaches 5.1), four of int4 45 (5.4 TB/s);
// 64 tokens of 8 of 128 experts, 32 of them here, of 4096 x 7168 92 (5.1 TB/s).
// 2112 x 7168 of one token is a launch and a chain of four loads: 6.0 us replayed from
// a graph, in which an empty kernel takes 2.3.  Integers run 10 to 20% behind E2M1:
// their scales pass through registers, so that one piece is under way at a time, not
// three.
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
  static constexpr int kScales = FORM != 0 ? 0 : RT < 2 ? 256 : RT * 128;            // E8M0 words of 16 * RT rows
  static constexpr int kBytes = kWeights + kX + kScales;
  static constexpr int kLoads = 2 * RT + XL + (FORM != 0 ? 0 : RT < 4 ? 1 : RT / 2);
};
// Integers: a table of a piece's pairs (scale, -scale * zero point): two sums that do
// not wait for one another, 5 to 15% of the time less than scale * (sum - zero * sum of x)
template <int FORM>
constexpr int kGroups = FORM ? 256 / (FORM ? FORM : 1) : 0;
template <int FORM, int RT>
constexpr int kTable = kGroups<FORM> * 16 * RT * 8;
// LDS of a wave: NS pieces of a full tile, more where it is not full
template <int FORM, int RT, int TILE, int NS>
constexpr int kWaveBytes = kTable<FORM, RT> + NS * Slot<FORM, RT, TILE / 2>::kBytes;

template <int FORM, int RT, int W, int BW, int XL>
__device__ __forceinline__ void sum_pieces(const GemvParams& p, const int* rows, int id, int n0, int wave, uint8_t* own,
                                           f32x4 (&acc)[RT]) {
  typedef Slot<FORM, RT, XL> S;
  constexpr int GROUPS = kGroups<FORM>, TABLE = kTable<FORM, RT>;
  constexpr int ITEMS = FORM ? (GROUPS * 16 * RT + 63) / 64 : 1; // scales per lane and piece
  constexpr int FIT = (BW - TABLE) / S::kBytes;
  constexpr int NS = FORM ? (FIT < 2 ? FIT : 2) : (FIT < 4 ? FIT : 4);
  static_assert(NS >= 1 && NS * S::kLoads < 64, "slots");
  const int lane = threadIdx.x & 63, r16 = lane & 15, g16 = lane >> 4;
  const int pieces = (p.K + 255) / 256;
  const int count = (pieces - wave + W - 1) / W;                 // this wave's: wave, wave + W, ...
  if (count <= 0) return;
  const bool odd = (p.K & 128) != 0;           // the last piece is half as long: its second half repeats the first
  const int last = p.N - 1 - n0;               // columns beyond N repeat the last: not stored
  const uint8_t* weights = p.b + ((size_t)id * p.N + n0) * (p.K / 2);
  uint32_t wrow[2 * RT];
#pragma unroll
  for (int l = 0; l < 2 * RT; ++l) wrow[l] = (uint32_t)min(l * 8 + (lane >> 3), last) * (uint32_t)(p.K / 2);
  const uint16_t* xsrc[XL];
#pragma unroll
  for (int l = 0; l < XL; ++l) {
    const int i = rows[2 * l + (lane >> 5)];   // a row without a choice repeats the first: not stored
    xsrc[l] = p.x + (size_t)((i >= 0 ? i : rows[0]) / p.x_div) * p.ldx;
  }
  const uint32_t base = lds_u32(own) + TABLE;
  auto issue = [&](int k) {
    const int piece = wave + k * W;
    const bool half = odd && piece == pieces - 1;
    const uint32_t slot = __builtin_amdgcn_readfirstlane(base + (k % NS) * S::kBytes);
    if constexpr (FORM == 0) {
      const int32_t* e = p.sfb + ((size_t)id * (p.K / 128) + piece * 2) * p.N + n0;
      const uint32_t to = slot + S::kWeights + S::kX;
      if constexpr (RT < 4) {                  // one load for both blocks
        const int h = half ? 0 : (lane / (16 * RT)) & 1;
        dma_4(e + (size_t)h * p.N + min(lane % (16 * RT), last), __builtin_amdgcn_readfirstlane(to));
      } else {
#pragma unroll
        for (int l = 0; l < RT / 2; ++l) {
          const int h = half ? 0 : l / (RT / 4), row = l % (RT / 4) * 64 + lane;
          dma_4(e + (size_t)h * p.N + min(row, last), __builtin_amdgcn_readfirstlane(to + l * 256));
        }
      }
    }
    const uint8_t* w = weights + (size_t)piece * 128;
#pragma unroll
    for (int l = 0; l < 2 * RT; ++l) {
      int chunk = (lane & 7) ^ swz(l * 8 + (lane >> 3));
      chunk = half ? chunk & 3 : chunk;
      if (p.again)
        dma_16s(w, wrow[l] + chunk * 16, __builtin_amdgcn_readfirstlane(slot + l * 1024));
      else
        dma_16s_nt(w, wrow[l] + chunk * 16, __builtin_amdgcn_readfirstlane(slot + l * 1024));
    }
#pragma unroll
    for (int l = 0; l < XL; ++l) {
      int chunk = (lane & 31) ^ (2 * l + (lane >> 5));
      chunk = half ? chunk & 15 : chunk;
      dma_16(xsrc[l] + (size_t)piece * 256 + chunk * 8,
             __builtin_amdgcn_readfirstlane(slot + S::kWeights + l * 1024));
    }
  };
  // integers: a piece's scales and zero points come through registers, as they are: a
  // conversion here would wait for each of them
  uint32_t sc[ITEMS], zs[ITEMS];
  auto load_scales = [&](int k) {
    if constexpr (FORM != 0) {
      const int piece = wave + k * W;
      const size_t at = ((size_t)id * (p.K / FORM) + (size_t)piece * GROUPS) * p.N + n0;
      const int mask = odd && piece == pieces - 1 ? GROUPS / 2 - 1 : GROUPS - 1;
#pragma unroll
      for (int t = 0; t < ITEMS; ++t) {
        const int item = t * 64 + lane;
        const uint32_t off = (uint32_t)((item / (16 * RT)) & mask) * (uint32_t)p.N + (uint32_t)min(item % (16 * RT), last);
        sc[t] = p.scales_bf16 ? (static_cast<const uint16_t*>(p.scales) + at)[off]
                              : (static_cast<const uint32_t*>(p.scales) + at)[off];
        zs[t] = p.zeros ? (p.zeros + at)[off] : 8;
      }
    }
  };
  if constexpr (FORM != 0) {
    load_scales(0);
    issue(0);
  } else {
    for (int k = 0; k < NS - 1 && k < count; ++k) issue(k);
  }
  for (int k = 0; k < count; ++k) {
    if constexpr (FORM != 0) {
      wait_vm_lgkm0<0>();
      asm volatile("" ::: "memory");
      float2* to = reinterpret_cast<float2*>(own);
#pragma unroll
      for (int t = 0; t < ITEMS; ++t) {
        const float s = __uint_as_float(p.scales_bf16 ? sc[t] << 16 : sc[t]);
        if (t * 64 + lane < GROUPS * 16 * RT) to[t * 64 + lane] = make_float2(s, -s * (float)zs[t]);
      }
      if (k + 1 < count) {
        load_scales(k + 1);
        if (NS > 1) issue(k + 1);
      }
    } else {
      if (k + NS - 1 < count) issue(k + NS - 1);
      // piece k is complete: only later ones may be under way
      wait_stages<S::kLoads, NS - 1>(min(NS - 1, count - 1 - k));
      asm volatile("" ::: "memory");
    }
    const uint8_t* slot = own + TABLE + (k % NS) * S::kBytes;
    const uint8_t* xs = slot + S::kWeights;
    const int xrow = r16 & (2 * XL - 1);       // rows of d from 2 * XL on repeat others: not stored
    f32x4 q[RT] = {}, xsum = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && odd && wave + k * W == pieces - 1) break;
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
            acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv), widen_fp4(w[r][j], scale[r]),
                                                             acc[r], 0, 0, 0);
        } else {
          const bf16x8 ones = {(__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f,
                               (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f};
          const bf16x8 xf = even_first(xv);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int row = r * 16 + r16;
            const uint32_t v = *reinterpret_cast<const uint32_t*>(slot + row * 128 + (((h * 4 + j) ^ swz(row)) << 4) +
                                                                  g16 * 4);
            q[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, widen_int4(v), q[r], 0, 0, 0);
          }
          xsum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, ones, xsum, 0, 0, 0);
          constexpr int STEPS = FORM ? FORM / 32 : 1;
          if ((j + 1) % STEPS == 0) {
            const int g = (h * 4 + j) / STEPS;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const float2 s = reinterpret_cast<const float2*>(own)[g * 16 * RT + r * 16 + r16];
#pragma unroll
              for (int e = 0; e < (XL == 1 ? 2 : 4); ++e)        // (a lane's rows of d from 2 * XL on are not stored)
                acc[r][e] = fmaf(s.y, xsum[e], fmaf(s.x, q[r][e], acc[r][e]));
              q[r] = f32x4{};
            }
            xsum = f32x4{};
          }
        }
      }
    }
    asm volatile("" ::: "memory");
    wait_vm_lgkm0<63>();                       // the slot is read before the next piece fills it
    if (FORM != 0 && NS == 1 && k + 1 < count) issue(k + 1);
  }
}

template <int FORM, int RT, int W, int TILE, int NS>
__global__ __launch_bounds__(W * 64) void gemv_kernel(GemvParams p) {
  constexpr int BW = kWaveBytes<FORM, RT, TILE, NS>;
  __shared__ int rows[16];
  __shared__ __attribute__((aligned(128))) uint8_t lds[W][BW];
  static_assert(sizeof(lds) >= (kMaxLayoutGroups + kInlineChoices / 64) * 4 && kInlineChoices <= 64 * 64, "find_tile's room");
  // consecutive workgroups go to the 8 XCDs in turn: each takes a run of items, the
  // tiles of the same columns next to one another, for those that share an expert
  const int per = (p.items + 7) / 8;
  const int item = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || item >= p.items) return;
  const int at = item / p.tiles, part = p.part0 + at, n0 = part * 16 * RT;
  int tile = p.tile0 + item - at * p.tiles;
  if (tile < p.others) {
    write_others<W * 64>(p, tile * 64, n0, 16 * RT);
    return;
  }
  tile -= p.others;
  int id;
  if (!find_tile<W * 64, TILE>(p, tile, rows, &id, reinterpret_cast<int*>(&lds[0][0]))) return;
  id = __builtin_amdgcn_readfirstlane(id);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g16 = lane >> 4;
  constexpr int OLD = 16 * RT + 4;             // a row of sums in LDS
  static_assert(TILE * OLD * 4 <= BW, "sums");
  f32x4 acc[RT] = {};
  if (id >= 0) {
    if (TILE > 8 && rows[8] >= 0) {
      if constexpr (TILE > 8) sum_pieces<FORM, RT, W, BW, 8>(p, rows, id, n0, wave, lds[wave], acc);
    } else if (TILE > 4 && rows[4] >= 0) {
      if constexpr (TILE > 4) sum_pieces<FORM, RT, W, BW, 4>(p, rows, id, n0, wave, lds[wave], acc);
    } else if (rows[2] >= 0) {
      sum_pieces<FORM, RT, W, BW, 2>(p, rows, id, n0, wave, lds[wave], acc);
    } else {
      sum_pieces<FORM, RT, W, BW, 1>(p, rows, id, n0, wave, lds[wave], acc);
    }
    // [row of d][column]
    float* sums = reinterpret_cast<float*>(lds[wave]);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (g16 * 4 + e < TILE) sums[(g16 * 4 + e) * OLD + r * 16 + r16] = acc[r][e];
    __syncthreads();
  }
  // thread: a row of d, four of its columns
  for (int at4 = threadIdx.x; at4 < TILE * RT * 4; at4 += W * 64) {
    const int row = at4 / (RT * 4), col = at4 % (RT * 4) * 4;
    const int i = rows[row], n = n0 + col;
    if (i < 0 || n >= p.N) continue;
    f32x4 sum = {};
    if (id >= 0)
#pragma unroll
      for (int w = 0; w < W; ++w) sum += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(lds[w]) + row * OLD + col);
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
constexpr int kMaxK = 1 << 24;           // a workgroup's rows of weights are addressed with 32 bits
constexpr int kMostGroups = 1 << 22;     // workgroups per launch: a grid has fewer than 2^32 threads

int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

template <int RT, int W, int TILE, int NS>
int launch_items(GemvParams p, int group, long long tiles, hipStream_t st) {
  const int parts = (p.N + 16 * RT - 1) / (16 * RT);
  for (long long t = 0; t < tiles; t += p.tiles) {
    p.tile0 = (int)t;
    p.tiles = (int)(tiles - t < kMostGroups ? tiles - t : kMostGroups);
    const int step = kMostGroups / p.tiles;
    for (p.part0 = 0; p.part0 < parts; p.part0 += step) {
      p.items = p.tiles * (parts - p.part0 < step ? parts - p.part0 : step);
      const int grid = (p.items + 7) / 8 * 8;
      if (group == 0)
        gemv_kernel<0, RT, W, TILE, NS><<<grid, W * 64, 0, st>>>(p);
      else if (group == 32) {
        if constexpr (RT * W < 32)                               // (launch_tile asks for no more: LDS has no room)
          gemv_kernel<32, RT, W, TILE, NS><<<grid, W * 64, 0, st>>>(p);
      } else if (group == 64)
        gemv_kernel<64, RT, W, TILE, NS><<<grid, W * 64, 0, st>>>(p);
      else
        gemv_kernel<128, RT, W, TILE, NS><<<grid, W * 64, 0, st>>>(p);
      const int s = launched();
      if (s != DG_OK) return s;
    }
  }
  return DG_OK;
}

// Columns per workgroup (16 * RT), its waves W and the pieces NS that a full tile's wave
// has room for: the widest with which there is more than one workgroup per CU.  Fewer
// leave CUs idle, more read x (and the choices) again for fewer columns.  Measured, as
// us of RT, W, NS (replayed from a graph, FP4 unless said):
//   tiles of 16   64 tokens of 4096 x 7168    4,8,1 11.2   2,4,1 12.8   4,4,1 15.0
//                 128 tokens of the same      4,4,1 16.6   4,8,1 18.6   2,4,1 22.2
//                 16 of 65536 x 7168          4,4,1 50     4,8,1 54     2,4,1 59
//                 16 of 7168 x 16384          2,8,1 19.3   4,8,1 23.8   1,8,1 26.8
//                 16 of 2112 x 7168           1,8,1 8.8    2,8,1 9.6
//   tiles of 4    one of 2112 x 7168          1,8,2 6.0    2,8,2 7.0    2,4,1 11.0
//                 one of 7168 x 16384         2,8,2 13.7   1,8,2 14.1   2,4,1 22.0
//                 the same of int4            2,8,2 16.0   1,8,2 16.8   2,4,1 27.9
//                 one of 65536 x 7168         2,4,2 36.6   2,4,1 38.8   2,8,2 49.4
// With K up to 4096 a wave of four has at most four pieces, and room for more only
// costs occupancy: one token of 57344 x 2048 of int4 2,4,1 17.0, 2,4,2 18.4, the 8
// experts of one token (7165 x 2048, int4) 19.6 and 21.7; so it does for tiles of 8 (8
// tokens of 8 of 64 experts of 2048 x 4096 36.5 and 42.1).  By choice the tiles are as
// many as there can be, copies of c for choices of other experts among them.
template <int TILE>
int launch_tile(const GemvParams& p, int group, long long tiles, int num_cus, hipStream_t st) {
  auto full = [&](int rt) { return tiles * ((p.N + 16 * rt - 1) / (16 * rt)) > num_cus; };
  if constexpr (TILE == 16) {
    if (full(4)) return launch_items<4, 4, TILE, 1>(p, group, tiles, st);
    if (full(2) && group != 32) return launch_items<4, 8, TILE, 1>(p, group, tiles, st);
    if (full(1)) return launch_items<2, 8, TILE, 1>(p, group, tiles, st);
    return launch_items<1, 8, TILE, 1>(p, group, tiles, st);
  } else {
    if (full(2)) {
      if (TILE == 4 && p.K > 4096) return launch_items<2, 4, TILE, 2>(p, group, tiles, st);
      return launch_items<2, 4, TILE, 1>(p, group, tiles, st);
    }
    if (full(1)) return launch_items<2, 8, TILE, 2>(p, group, tiles, st);
    return launch_items<1, 8, TILE, 2>(p, group, tiles, st);
  }
}

// Tokens per tile: those of a small batch (an expert has no more of them, unless a
// token's choices repeat it).  Tiles of 4 and 8 take 2 and 4 KB of LDS for x per piece
// against 8: one token of 7168 x 16384 13.8 us, 16 in their tile's best form 19.3.
int tile_of(int tokens) { return tokens <= 4 ? 4 : (tokens <= 8 ? 8 : 16); }

int launch_tiles(const GemvParams& p, int group, int tile, long long tiles, int num_cus, hipStream_t st) {
  if (tile == 4) return launch_tile<4>(p, group, tiles, num_cus, st);
  if (tile == 8) return launch_tile<8>(p, group, tiles, num_cus, st);
  return launch_tile<16>(p, group, tiles, num_cus, st);
}

// By choice: as many choices at a time as the scratch memory has room to list,
// usually all, or kInlineChoices without lists.
int launch_choices(GemvParams p, int group, int tile, int n, const int32_t* ids, const Scratch& sc, hipStream_t st) {
  const long long groups = p.G + 1;
  for (int i = 0; i < n;) {
    int step = n - i;
    size_t list_bytes = 0;
    long long rows = 0;
    while (step > kInlineChoices) {
      rows = (step + (tile - 1) * (groups < step ? groups : step)) / tile * tile;
      list_bytes = (size_t)(2 * rows + 64) / 64 * 64 * sizeof(int32_t);
      if (list_bytes <= sc.bytes && rows < (1LL << 30)) break;
      step = step / 2 > kInlineChoices ? step / 2 : kInlineChoices;
    }
    p.i0 = i;
    p.n = step;
    // experts with several tiles each, as for the dense product (256 tokens of 2 of 8
    // experts of 14336 x 4096 182 us against 191 with streaming loads, 256 and 512 of 8 of
    // 128, 32 here, of 4096 x 7168 146 against 152, 224 against 250); with about one tile
    // each streaming is better (64 and 128 tokens of the same 93 us against 100, 111
    // against 113).  The choices of all experts are counted: of 64 tokens with all of 32
    // experts here half of the experts have two tiles, and are streamed all the same (131
    // against 126)
    p.again = step > 2LL * tile * p.G;
    p.ids = ids + i;
    p.layout = nullptr;
    p.slot_of = nullptr;
    long long tiles;
    if (step > kInlineChoices) {
      int32_t* layout = reinterpret_cast<int32_t*>(sc.ptr);
      LayoutParams lp{p.ids, step, p.first, (int)groups, tile, 0, (int)rows, layout, nullptr, layout + rows, nullptr};
      lp.others = 1;
      const hipError_t e = launch_layout(lp, sc.ptr + list_bytes, sc.bytes - list_bytes, st);
      if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
      p.layout = layout;
      p.slot_of = layout + rows;
      p.others = 0;
      tiles = rows / tile;
    } else {
      // an expert's last tile may not be full
      tiles = (p.G < step ? p.G : step) + step / tile;
      p.others = (step + 63) / 64;
      tiles = p.others + (tiles < step ? tiles : step);
    }
    const int s = launch_tiles(p, group, tile, tiles, sc.num_cus, st);
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
  if (p.K > kMaxK) return fail(DG_ERR_UNSUPPORTED, "K=%d exceeds 2^24", p.K);
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
  const hipStream_t st = static_cast<hipStream_t>(stream);
  Scratch sc;
  const int e = call_scratch(st, &sc);
  if (e != DG_OK) return e;
  const int tile = tile_of(M);
  // more tiles than one read the weights again, from the caches if the first leaves them
  // there: 64 tokens of 4096 x 7168 11.0 us against 12.1 with streaming loads, 128 16.5
  // against 19.1
  p.again = M > tile;
  return launch_tiles(p, group, tile, ((long long)M + tile - 1) / tile, sc.num_cus, st);
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
  const hipStream_t st = static_cast<hipStream_t>(stream);
  Scratch sc;
  s = call_scratch(st, &sc);
  if (s != DG_OK) return s;
  return launch_choices(p, group, tile_of(T), (int)n, ids, sc, st);
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

// Low-rank adapters of many requests beside a shared projection (include/dg.h):
//   d[t] = c[t] + scales[i] * B[i] . (A[i] . x[t]),   i = adapter_ids[t]
#include "../../include/dg.h"
#include "dg_host.h"
#include "expert_rows.h"
#include "fp8_gemm_core.h"    // direct global->LDS loads, waits and the 128-byte row swizzle

namespace dg {
namespace {

constexpr int kMaxRank = 256;
constexpr int THREADS = 256;
constexpr int WAVES = THREADS / 64;
// Up to here every workgroup finds its tile's tokens itself; beyond, layout kernels
// make lists.  Measured beside a 2112 x 7168 projection at 256 tokens against 257:
// one adapter of rank 16 15.2 us against 17.2, 48 of them 15.4 against 18.4, 8 of
// rank 64 23.2 against 23.0; at 128 tokens 10.4, 11.4 and 15.8 us.
constexpr int kInlineTokens = 256;

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
  int pieces_per_split;    // 64-K pieces per range
  int tiles;
  int steps;               // column steps per workgroup of the product with B
  int parts;               // workgroups per tile of the product with B
  const int32_t* layout;   // tile lists (many tokens): group of each row, L = tokens without an adapter
  const int32_t* slot_of;  // token of each row, -1 where a tile is not full
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Two shapes of workgroup.  LISTED (many tokens): a tile of 64 tokens from the
// layout kernels' lists, 16 to a wave.  Otherwise (few tokens): a tile of 16, the
// four waves share its K range, or its columns.
template <bool LISTED>
constexpr int kTile = LISTED ? 64 : 16;

// The tokens of this workgroup's tile into rows[kTile] (-1 where there is none)
// and their adapter into *id (-1: none).  Returns false for a workgroup without a
// tile.  Ends with a barrier.
//
// Not LISTED: the workgroup of token t has a tile if the tokens before t hold a
// multiple of 16 tokens of t's adapter; its tile is t and the next ones of that
// adapter.  Every wave counts for itself (at most kInlineTokens / 64 ballots), so
// that no workgroup waits for a list.
template <bool LISTED>
__device__ __forceinline__ bool find_tile(const LoraParams& p, int tile, int* rows, int* id) {
  constexpr int BT = kTile<LISTED>;
  if constexpr (LISTED) {
    const int g = p.layout[(size_t)tile * BT];
    if (g < 0) return false;
    *id = g < p.L ? g : -1;
    if (threadIdx.x < BT) rows[threadIdx.x] = p.slot_of[(size_t)tile * BT + threadIdx.x];
  } else {
    const int lane = threadIdx.x & 63;
    auto key = [&](int v) { return v >= 0 && v < p.L ? v : -1; };
    int ids[kInlineTokens / 64];
#pragma unroll
    for (int i = 0; i < kInlineTokens / 64; ++i)
      ids[i] = i * 64 + lane < p.T ? key(p.ids[i * 64 + lane]) : -2;
    const int mine = key(p.ids[tile]);
    if (threadIdx.x < BT) rows[threadIdx.x] = -1;
    __syncthreads();
    int before = 0, after = 0;
#pragma unroll
    for (int i = 0; i < kInlineTokens / 64; ++i) {
      if (i * 64 >= p.T) break;
      const int s = i * 64 + lane;
      before += __popcll(__ballot(ids[i] == mine && s < tile));
      const uint64_t m = __ballot(ids[i] == mine && s >= tile);
      const int at = after + __popcll(m & ((1ull << lane) - 1));
      if (ids[i] == mine && s >= tile && at < BT && threadIdx.x < 64) rows[at] = s;
      after += __popcll(m);
    }
    *id = mine;
    if (before % BT != 0) return false;
  }
  __syncthreads();
  return true;
}

// The item of this workgroup, of `items` = tiles * parts: consecutive workgroups go
// to the 8 XCDs in turn, and with lists each XCD takes a run of tiles with all
// their parts, so that an adapter's weights are fetched into one L2.
template <bool LISTED>
__device__ __forceinline__ bool find_item(int items, int parts, int* tile, int* part) {
  int item = blockIdx.x;
  if (!LISTED && item >= items) return false;
  if (LISTED) {
    const int per = (items + 7) / 8;
    item = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || item >= items) return false;
  }
  *tile = item / parts;
  *part = item - *tile * parts;
  return true;
}

// ---- h = A . x ---------------------------------------------------------------
// One K range of one tile, as h^T: the ranks are the MFMA's rows and the tokens
// its columns, so that a lane ends with four neighbouring ranks of one token.
// Bound by x (many tokens) or A (few), each read from memory once.
//
// Rows of x and of A come into LDS in pieces of 64 K, one 128-byte line per row,
// with direct loads of eight whole lines each, and are read from there as MFMA
// operands.  (Operands loaded straight from memory, 64 bytes of sixteen rows at a
// time, took about 96 cycles of the CU's memory pipe per load: 97 us against 33
// for 8192 tokens of 7168 at rank 64.)  A row's 16-byte chunk c lies at
// c ^ swz(row).
__device__ __forceinline__ bf16x8 piece_operand(const uint8_t* rows, int row, int chunk) {
  return *reinterpret_cast<const bf16x8*>(rows + row * 128 + ((chunk ^ swz(row)) << 4));
}

// Many tokens: 64 to a tile, 16 to a wave; the waves load each piece together
// into a ring of slots, RING - 1 of them ahead of the products.  8192 tokens of
// 7168 with 8 adapters of rank 64: 34 us, 3.4 TB/s of x.
template <int RT>
__global__ __launch_bounds__(THREADS) void lora_shrink_listed_kernel(LoraParams p) {
  constexpr int BT = kTile<true>;
  constexpr int NR = BT + RT * 16;             // rows per piece: tokens, then ranks
  constexpr int RING = 3;
  constexpr int LPW = (NR / 8 + WAVES - 1) / WAVES;          // loads per wave and piece
  __shared__ int rows[BT];
  __shared__ __attribute__((aligned(128))) uint8_t ring[RING][NR * 128];
  int id, tile, split;
  if (!find_item<true>(p.tiles * p.k_splits, p.k_splits, &tile, &split)) return;
  if (!find_tile<true>(p, tile, rows, &id) || id < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g16 = lane >> 4;
  const int first = split * p.pieces_per_split;
  const int count = min(p.K / 64 - first, p.pieces_per_split);
  const uint16_t* src[LPW];
  uint32_t dst[LPW];                           // within a slot
#pragma unroll
  for (int l = 0; l < LPW; ++l) {
    const int at = min(wave + l * WAVES, NR / 8 - 1);        // the last load again where a wave has none left
    const int row = at * 8 + (lane >> 3), chunk = (lane & 7) ^ swz(row);
    dst[l] = at * 1024;
    if (row < BT)                              // a row without a token repeats the first: its column is not stored
      src[l] = p.x + (size_t)(rows[row] >= 0 ? rows[row] : rows[0]) * p.ldx + chunk * 8;
    else                                       // ranks beyond R repeat the last: not stored
      src[l] = p.a + ((size_t)id * p.R + min(row - BT, p.R - 1)) * p.K + chunk * 8;
  }
  const uint32_t ring0 = lds_u32(&ring[0][0]);
  auto load = [&](int i) {
    const int piece = first + i;
    const uint32_t slot = ring0 + (uint32_t)(i % RING) * (NR * 128);
#pragma unroll
    for (int l = 0; l < LPW; ++l) dma_16(src[l] + (size_t)piece * 64, __builtin_amdgcn_readfirstlane(slot + dst[l]));
  };
  f32x4 acc[RT] = {};
  for (int i = 0; i < RING - 1 && i < count; ++i) load(i);
  for (int i = 0; i < count; ++i) {
    // piece i is complete for this wave, then for all; they have also left the
    // slot of piece i - 1, which the next load fills
    wait_stages<LPW, RING - 2>(min(RING - 2, count - 1 - i));
    bare_barrier();
    if (i + RING - 1 < count) load(i + RING - 1);
    const uint8_t* slot = ring[i % RING];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bf16x8 xf = piece_operand(slot, wave * 16 + r16, h * 4 + g16);
#pragma unroll
      for (int r = 0; r < RT; ++r)
        acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(piece_operand(slot, BT + r * 16 + r16, h * 4 + g16), xf,
                                                         acc[r], 0, 0, 0);
    }
  }
  const int token = rows[wave * 16 + r16];
  if (token < 0) return;
  float* out = p.partial + ((size_t)split * p.T + token) * p.R;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int at = r * 16 + g16 * 4;
    if (at < p.R) *reinterpret_cast<f32x4*>(out + at) = acc[r];
  }
}

// Few tokens: a tile of 16, whose pieces the four waves take in turn, each with
// LDS of its own (no barrier), UP pieces at a time and all of them in flight.  64
// tokens of 48 adapters of rank 16, K 7168: 5.3 us (11 MB of A and x), of which a
// launch is about 2.3; the rest is the chain of ids, lines and sums.
template <int RT>
__global__ __launch_bounds__(THREADS) void lora_shrink_few_kernel(LoraParams p) {
  constexpr int UP = RT <= 1 ? 4 : (RT <= 4 ? 2 : 1);
  constexpr int NR = 16 + RT * 16;
  __shared__ int rows[16];
  __shared__ __attribute__((aligned(128))) uint8_t slots[WAVES][UP][NR * 128];
  int id, tile, split;
  if (!find_item<false>(p.tiles * p.k_splits, p.k_splits, &tile, &split)) return;
  if (!find_tile<false>(p, tile, rows, &id) || id < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g16 = lane >> 4;
  const int first = split * p.pieces_per_split;
  const int count = min(p.K / 64 - first, p.pieces_per_split);
  const int row8 = lane >> 3;
  const bool more = rows[8] >= 0;              // more than eight tokens: both halves of x
  const uint16_t *xs[2], *as[2 * RT];
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    const int row = l * 8 + row8;
    xs[l] = p.x + (size_t)(rows[row] >= 0 ? rows[row] : rows[0]) * p.ldx + ((lane & 7) ^ swz(row)) * 8;
  }
#pragma unroll
  for (int l = 0; l < 2 * RT; ++l) {
    const int row = l * 8 + row8;
    as[l] = p.a + ((size_t)id * p.R + min(row, p.R - 1)) * p.K + ((lane & 7) ^ swz(row)) * 8;
  }
  const uint32_t base = lds_u32(&slots[wave][0][0]);
  f32x4 acc[RT] = {};
  for (int i = wave; i < count; i += WAVES * UP) {
#pragma unroll
    for (int u = 0; u < UP; ++u) {
      if (i + u * WAVES >= count) break;
      const size_t k = (size_t)(first + i + u * WAVES) * 64;
      const uint32_t slot = base + u * (NR * 128);
#pragma unroll
      for (int l = 0; l < 2 * RT; ++l) dma_16_nt(as[l] + k, __builtin_amdgcn_readfirstlane(slot + 2048 + l * 1024));
      dma_16(xs[0] + k, __builtin_amdgcn_readfirstlane(slot));
      if (more) dma_16(xs[1] + k, __builtin_amdgcn_readfirstlane(slot + 1024));
    }
    wait_vm_lgkm0<0>();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < UP; ++u) {
      if (i + u * WAVES >= count) break;
      const uint8_t* slot = slots[wave][u];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // without more than eight tokens columns 8..15 repeat 0..7: not stored
        const bf16x8 xf = piece_operand(slot, more ? r16 : r16 & 7, h * 4 + g16);
#pragma unroll
        for (int r = 0; r < RT; ++r)
          acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(piece_operand(slot, 16 + r * 16 + r16, h * 4 + g16), xf,
                                                           acc[r], 0, 0, 0);
      }
    }
    wait_vm_lgkm0<0>();                        // the slots are read before the next round fills them
    asm volatile("" ::: "memory");
  }
  // the four waves' sums, in the waves' own LDS
  f32x4* sums = reinterpret_cast<f32x4*>(slots[wave][0]);
#pragma unroll
  for (int r = 0; r < RT; ++r) sums[r * 64 + lane] = acc[r];
  __syncthreads();
  // wave w adds up ranks w, w + 4, ... of the tile's sixteenths
  const int token = rows[r16];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if ((r & (WAVES - 1)) != wave) continue;
    f32x4 sum = {};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += reinterpret_cast<const f32x4*>(slots[w][0])[r * 64 + lane];
    const int at = r * 16 + g16 * 4;
    if (token >= 0 && at < p.R)
      *reinterpret_cast<f32x4*>(p.partial + ((size_t)split * p.T + token) * p.R + at) = sum;
  }
}

// NE neighbouring bf16 of a row, at any 2-byte address.
template <int NE>
struct Piece {
  typedef uint16_t V __attribute__((ext_vector_type(NE)));
  typedef V U __attribute__((aligned(2)));
};

// ---- d = c + B . h -----------------------------------------------------------
// Again transposed: MFMA rows are columns of d.  h (the K ranges' sum times the
// adapter's scale) stays fp32 in LDS and is multiplied as three bf16 that add up
// to it, so that differences of ranks in B keep its last bits.
template <int BT, int RP>
__device__ __forceinline__ void sum_h(const LoraParams& p, const int* rows, int id, float (*hs)[RP + 4]) {
  const float scale = p.scales ? p.scales[id] : 1.0f;
  for (int i = threadIdx.x; i < BT * (RP / 4); i += THREADS) {
    const int at = i / (RP / 4), r = i % (RP / 4) * 4;
    const int t = rows[at];
    f32x4 h = {};
    if (t >= 0 && r < p.R)
#pragma unroll 4
      for (int s = 0; s < p.k_splits; ++s)
        h += *reinterpret_cast<const f32x4*>(p.partial + ((size_t)s * p.T + t) * p.R + r);
    *reinterpret_cast<f32x4*>(&hs[at][r]) = h * scale;
  }
}

// Eight neighbouring values of h as MFMA operands, v = part[0] + part[1] + part[2]:
// its leading eight bits, the next and the last (cut off, not rounded: the largest
// values would round to infinity).  An infinity or a NaN is part[0] alone.
constexpr int kParts = 3;
__device__ __forceinline__ void split_h(const float* h, bf16x8 (&part)[kParts]) {
  const f32x4 h0 = *reinterpret_cast<const f32x4*>(h), h1 = *reinterpret_cast<const f32x4*>(h + 4);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float rest = e < 4 ? h0[e] : h1[e - 4];
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      const uint32_t head = __float_as_uint(rest) & 0xFFFF0000u;
      part[q][e] = __builtin_bit_cast(__bf16, (uint16_t)(head >> 16));
      rest = fabsf(rest) < INFINITY ? rest - __uint_as_float(head) : 0.0f;
    }
  }
}

// Few tokens: a tile of 16, the waves side by side on 16 * NT columns each (the
// same call's 2112 columns: 5.7 us at NT = 1, latency).
// MFMA row r of sub-tile j stands for column 4 * NT * (r / 4) + 4 * j + r % 4, so
// that a lane's 4 * NT results are neighbours in d.
template <int RK, int NT>
__global__ __launch_bounds__(THREADS) void lora_expand_few_kernel(LoraParams p) {
  constexpr int RP = RK * 32;             // ranks padded to whole MFMA steps
  constexpr int NE = 4 * NT;
  typedef typename Piece<NE>::U U;
  __shared__ int rows[16];
  __shared__ __attribute__((aligned(16))) float hs[16][RP + 4];
  int id, tile, part;
  if (!find_item<false>(p.tiles * p.parts, p.parts, &tile, &part)) return;
  if (!find_tile<false>(p, tile, rows, &id)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g16 = lane >> 4;
  const int col = (part * WAVES + wave) * 16 * NT;             // this wave's first column
  const int token = rows[r16];
  const int n = col + NE * g16;
  U v = {};                               // a column without a token reads the tile's first
  if (p.c && n + NE <= p.N) v = *reinterpret_cast<const U*>(p.c + (size_t)(token >= 0 ? token : rows[0]) * p.ldc + n);
  f32x4 acc[NT] = {};
  if (id >= 0) {
    bf16x8 bf[NT][RK];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int at = min(col + NE * (r16 >> 2) + 4 * j + (r16 & 3), p.N - 1);         // beyond N: not stored
      const uint16_t* b = p.b + ((size_t)id * p.N + at) * p.R + g16 * 8;
#pragma unroll
      for (int k = 0; k < RK; ++k) {
        bf[j][k] = bf16x8{};
        if (k * 32 + g16 * 8 < p.R) bf[j][k] = *reinterpret_cast<const bf16x8*>(b + k * 32);
      }
    }
    sum_h<16, RP>(p, rows, id, hs);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < RK; ++k) {
      bf16x8 h[kParts];
      split_h(&hs[r16][k * 32 + g16 * 8], h);
#pragma unroll
      for (int q = 0; q < kParts; ++q)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j][k], h[q], acc[j], 0, 0, 0);
    }
  }
  if (token < 0 || n >= p.N) return;
  uint16_t* d = p.d + (size_t)token * p.ldd + n;
  if (n + NE <= p.N) {
#pragma unroll
    for (int e = 0; e < NE; ++e)
      if (id >= 0) v[e] = f32_to_bf16(bf16_to_f32(v[e]) + acc[e >> 2][e & 3]);
    *reinterpret_cast<U*>(d) = v;
  } else {
    const uint16_t* c = p.c ? p.c + (size_t)token * p.ldc + n : nullptr;
#pragma unroll
    for (int e = 0; e < NE; ++e)
      if (n + e < p.N) {
        const uint16_t w = c ? c[e] : 0;
        d[e] = id >= 0 ? f32_to_bf16(bf16_to_f32(w) + acc[e >> 2][e & 3]) : w;
      }
  }
}

// Many tokens: 64 to a tile, 16 to a wave, `steps` times 64 columns.  B's 64 rows
// of a step are contiguous and come into LDS for the four waves with direct
// loads, a step ahead; results pass through LDS so that c and d are read and
// written in whole 128-byte lines (8 rows of 64 columns per instruction).  Bound
// by c and d: 8192 tokens, 4096 columns, rank 64 take 39 us (3.5 TB/s of c and d),
// 5 of them for the partial sums; with operands and results straight from and to
// memory, in 64-byte pieces of sixteen rows, it took 78.
template <int RK>
__global__ __launch_bounds__(THREADS) void lora_expand_listed_kernel(LoraParams p) {
  constexpr int BT = kTile<true>;
  constexpr int RP = RK * 32;
  constexpr int OLD = 68;                 // a row of results in LDS: 64 and 16 bytes on
  typedef typename Piece<8>::U U;
  union Shared {
    float hs[BT][RP + 4];
    float out[WAVES][16][OLD];
  };
  __shared__ int rows[BT];
  __shared__ __attribute__((aligned(16))) Shared sh;
  __shared__ __attribute__((aligned(128))) uint8_t ring[2][64 * RP * 2];
  int id, tile, part;
  if (!find_item<true>(p.tiles * p.parts, p.parts, &tile, &part)) return;
  if (!find_tile<true>(p, tile, rows, &id)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g16 = lane >> 4, row8 = lane >> 3, col8 = (lane & 7) * 8;
  const int first = part * p.steps;
  const int count = min(p.steps, (p.N + 63) / 64 - first);
  int token[2];                           // rows row8 and row8 + 8 of the wave's sixteen
  token[0] = rows[wave * 16 + row8];
  token[1] = rows[wave * 16 + 8 + row8];
  const bool both = rows[wave * 16 + 8] >= 0;                  // each half of the sixteen has a token: two stores a step
  const int some = rows[0];
  U cv[2] = {};
  auto load_c = [&](int step) {
    const int n = (first + step) * 64 + col8;
    if (p.c && n + 8 <= p.N)
#pragma unroll
      for (int h = 0; h < 2; ++h)         // a row without a token reads the tile's first
        cv[h] = *reinterpret_cast<const U*>(p.c + (size_t)(token[h] >= 0 ? token[h] : some) * p.ldc + n);
  };
  auto store = [&](int step, auto value) {                     // value(h, e): what is added to column e of half h
    const int n = (first + step) * 64 + col8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (token[h] < 0 || n >= p.N) continue;
      uint16_t* d = p.d + (size_t)token[h] * p.ldd + n;
      if (n + 8 <= p.N) {
        U v = cv[h];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = value(h, e, v[e]);
        *reinterpret_cast<U*>(d) = v;
      } else {
        const uint16_t* c = p.c ? p.c + (size_t)token[h] * p.ldc + n : nullptr;
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (n + e < p.N) d[e] = value(h, e, c ? c[e] : (uint16_t)0);
      }
    }
  };
  if (id < 0) {                           // no adapter: c as it is
    for (int step = 0; step < count; ++step) {
      load_c(step);
      store(step, [](int, int, uint16_t c) { return c; });
    }
    return;
  }
  // B: chunk q (16 bytes) of the step's 64 rows lies at q, its row's chunks turned by
  // the row where their number is a power of two
  const int row_chunks = p.R / 8;
  const int turn = (row_chunks & (row_chunks - 1)) == 0 ? row_chunks - 1 : 0;
  int bcol[RK], bchunk[RK];
  uint32_t bdst[RK];
#pragma unroll
  for (int l = 0; l < RK; ++l) {
    const int at = min(wave + l * WAVES, row_chunks - 1);      // the last load again where a wave has none left
    const int q = at * 64 + lane;
    bcol[l] = q / row_chunks;
    bchunk[l] = (q - bcol[l] * row_chunks) ^ (bcol[l] & turn);
    bdst[l] = at * 1024;
  }
  const uint32_t ring0 = lds_u32(&ring[0][0]);
  auto load_b = [&](int step) {
    const uint32_t slot = ring0 + (uint32_t)(step & 1) * (64 * RP * 2);
#pragma unroll
    for (int l = 0; l < RK; ++l) {
      const int n = min((first + step) * 64 + bcol[l], p.N - 1);             // beyond N: not stored
      dma_16(p.b + ((size_t)id * p.N + n) * p.R + bchunk[l] * 8, __builtin_amdgcn_readfirstlane(slot + bdst[l]));
    }
  };
  load_b(0);
  load_c(0);
  sum_h<BT, RP>(p, rows, id, sh.hs);
  __syncthreads();
  bf16x8 hf[RK][kParts];
#pragma unroll
  for (int k = 0; k < RK; ++k) split_h(&sh.hs[wave * 16 + r16][k * 32 + g16 * 8], hf[k]);
  for (int step = 0; step < count; ++step) {
    // this step's B is complete: only the last step's stores, issued after it, may
    // be under way; and every wave has left the other slot and, at first, hs
    if (step > 0 && both)
      wait_vm_lgkm0<2>();
    else
      wait_vm_lgkm0<0>();
    bare_barrier();
    const U now[2] = {cv[0], cv[1]};
    if (step + 1 < count) {
      load_b(step + 1);
      load_c(step + 1);
    }
    const U next[2] = {cv[0], cv[1]};
    const uint8_t* slot = ring[step & 1];
    f32x4 acc[4] = {};
#pragma unroll
    for (int k = 0; k < RK; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = j * 16 + r16, chunk = k * 4 + g16;
        bf16x8 bf = {};
        if (chunk < row_chunks)
          bf = *reinterpret_cast<const bf16x8*>(slot + (row * row_chunks + (chunk ^ (row & turn))) * 16);
#pragma unroll
        for (int q = 0; q < kParts; ++q) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf, hf[k][q], acc[j], 0, 0, 0);
      }
    // a wave's own rows: program order is enough
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4*>(&sh.out[wave][r16][j * 16 + g16 * 4]) = acc[j];
    __builtin_amdgcn_wave_barrier();
    f32x4 sum[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        sum[h][e] = *reinterpret_cast<const f32x4*>(&sh.out[wave][h * 8 + row8][col8 + e * 4]);
    __builtin_amdgcn_wave_barrier();
    cv[0] = now[0];
    cv[1] = now[1];
    store(step, [&](int h, int e, uint16_t c) { return f32_to_bf16(bf16_to_f32(c) + sum[h][e >> 2][e & 3]); });
    cv[0] = next[0];
    cv[1] = next[1];
  }
}

template <bool LISTED, int RT>
void launch_shrink_rt(const LoraParams& p, int grid, hipStream_t st) {
  if constexpr (LISTED)
    lora_shrink_listed_kernel<RT><<<grid, THREADS, 0, st>>>(p);
  else
    lora_shrink_few_kernel<RT><<<grid, THREADS, 0, st>>>(p);
}

template <bool LISTED>
void launch_shrink(const LoraParams& p, hipStream_t st) {
  const int grid = (p.tiles * p.k_splits + 7) / 8 * 8;
  if (p.R <= 16)
    launch_shrink_rt<LISTED, 1>(p, grid, st);
  else if (p.R <= 32)
    launch_shrink_rt<LISTED, 2>(p, grid, st);
  else if (p.R <= 64)
    launch_shrink_rt<LISTED, 4>(p, grid, st);
  else if (p.R <= 128)
    launch_shrink_rt<LISTED, 8>(p, grid, st);
  else
    launch_shrink_rt<LISTED, 16>(p, grid, st);
}

template <int NT>
void launch_expand_few(LoraParams p, hipStream_t st) {
  p.parts = (p.N + 16 * NT * WAVES - 1) / (16 * NT * WAVES);
  const int grid = p.tiles * p.parts;
  if (p.R <= 32)
    lora_expand_few_kernel<1, NT><<<grid, THREADS, 0, st>>>(p);
  else if (p.R <= 64)
    lora_expand_few_kernel<2, NT><<<grid, THREADS, 0, st>>>(p);
  else if (p.R <= 128)
    lora_expand_few_kernel<4, NT><<<grid, THREADS, 0, st>>>(p);
  else
    lora_expand_few_kernel<8, NT><<<grid, THREADS, 0, st>>>(p);
}

template <int RK, int SLOTS>
void launch_expand_listed(LoraParams p, int num_cus, hipStream_t st) {
  const int chunks = (p.N + 63) / 64;
  // as many workgroups as run at once (SLOTS per CU: what their LDS has room for,
  // and no more than four), so that no CU has a last one to itself (8192 tokens, rank
  // 64, 4096 columns, the whole call: 73 us against 78 with two per CU and a few
  // more); a workgroup's steps share one sum of h
  long long parts = (long long)SLOTS * num_cus / p.tiles;
  parts = parts < 1 ? 1 : (parts > chunks ? chunks : parts);
  p.steps = (int)((chunks + parts - 1) / parts);
  p.parts = (chunks + p.steps - 1) / p.steps;
  const int grid = (p.tiles * p.parts + 7) / 8 * 8;
  lora_expand_listed_kernel<RK><<<grid, THREADS, 0, st>>>(p);
}

// K ranges: three workgroups per CU with lists, as many as run at once at ranks 33
// to 64 (a further round for a few of them would cost as much as the others
// together), and two without; and at least a piece for each of the four waves.  The
// same at every rank, although the LDS has room for 5, 4, 3, 2 and 1 with lists up
// to ranks 16, 32, 64, 128 and 256, and for 2, 3, 1, 2 and 1 without: the other
// ranks' own numbers are not measured.
// Without lists every token has a workgroup per range, most of which may find that
// they have no tile: no more than four of those per CU (128 tokens of 8 adapters of
// rank 64: 15.8 us against 23.5 without this limit).
int k_splits_for(bool listed, int tokens, long long tiles, int pieces, int num_cus) {
  long long fit = (listed ? 3LL : 2LL) * num_cus / tiles;
  if (!listed && fit > 4LL * num_cus / tokens) fit = 4LL * num_cus / tokens;
  const long long most = pieces / WAVES;
  const long long n = fit < most ? fit : most;
  return (int)(n < 1 ? 1 : n);
}

constexpr int kTokensMost = 1 << 24;
constexpr int kNoRoom = 1;               // not a dg_status: the scratch memory is too small for so many tokens

int lora_tokens(LoraParams p, const Scratch& sc, hipStream_t st) {
  const int pieces = p.K / 64;
  const bool terms = p.L > 0;
  const bool listed = p.T > kInlineTokens;
  const int bt = listed ? kTile<true> : kTile<false>;
  const int groups = p.L + 1;
  long long rows = p.T;
  size_t list_bytes = 0;
  if (listed) {
    const long long most = groups < p.T ? groups : p.T;
    rows = (p.T + (bt - 1) * most) / bt * bt;
    list_bytes = (size_t)(2 * rows + 64) / 64 * 64 * sizeof(int32_t);
  }
  const long long tiles = listed ? rows / bt : p.T;
  p.tiles = (int)tiles;
  p.k_splits = 1;
  p.pieces_per_split = pieces;
  if (terms) {
    const size_t one = (size_t)p.T * p.R * sizeof(float);
    if (list_bytes + one > sc.bytes) return kNoRoom;
    int splits = k_splits_for(listed, p.T, listed ? tiles : (p.T < p.L ? p.T : p.L), pieces, sc.num_cus);
    const size_t room = (sc.bytes - list_bytes) / one;
    if ((size_t)splits > room) splits = (int)room;
    p.pieces_per_split = (pieces + splits - 1) / splits;
    p.k_splits = (pieces + p.pieces_per_split - 1) / p.pieces_per_split;
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
  if (listed) {
    if (terms) launch_shrink<true>(p, st);
    if (p.R <= 32)
      launch_expand_listed<1, 4>(p, sc.num_cus, st);
    else if (p.R <= 64)
      launch_expand_listed<2, 4>(p, sc.num_cus, st);
    else if (p.R <= 128)
      launch_expand_listed<4, 2>(p, sc.num_cus, st);
    else
      launch_expand_listed<8, 1>(p, sc.num_cus, st);
  } else {
    if (terms) launch_shrink<false>(p, st);
    // 64 columns per wave where that makes four workgroups per CU, 16 below (2112
    // columns, 8 adapters of rank 64: 64 tokens 13.3 us against 12.1, 128 tokens 15.8
    // against 15.9; 48 of rank 16: 9.9 against 9.8 and 11.4 against 13.3)
    if (tiles * ((p.N + 255) / 256) >= 4 * sc.num_cus)
      launch_expand_few<4>(p, st);
    else
      launch_expand_few<1>(p, st);
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
  // as many tokens at a time as the scratch memory has room for, usually all, and
  // no more than a grid's threads (fewer than 2^32) and the lists' indices cover
  int step = T < kTokensMost ? T : kTokensMost;
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

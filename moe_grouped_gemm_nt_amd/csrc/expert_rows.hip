// The tokens' rows out to the experts and back (include/dg.h): the layouts of
// the grouped products, the quantising scatter into their A operands, and the
// weighted gather of their results with the gradient of its weights.
#include "expert_rows.h"

#include <cfloat>
#include <climits>
#include <type_traits>

#include "../../include/dg.h"
#include "dg_host.h"

namespace dg {
namespace {

// ============================================================================
// layout
// ============================================================================
// A stable counting sort by group.  The choices are cut into chunks, one
// workgroup each, and a chunk into one run per wave.  A choice's row is
//   start[g] + (choices of g in earlier chunks) + (in earlier waves of the
//   chunk) + (earlier in the wave's run),
// the last from ballots over the bits of g, 64 choices at a time.  Bound by the
// chain of dependent loads and barriers, not by bytes.  Up to kOneLaunch choices
// every workgroup counts them all itself (8192 choices: 9.0 us against 11.3 in two
// launches); beyond, a first kernel leaves each chunk's counts in the workspace
// (65536 choices, 256 experts: 14.8 us against 49.6 in one launch).
constexpr int LT = 512;                  // threads per workgroup
constexpr int LW = LT / 64;
constexpr int LKEEP = 4;                 // choices of its run that a lane keeps in registers
constexpr int LCOUNT = 8;                // loads in flight while counting
constexpr int kOneLaunch = 8192;
constexpr int kShare = 1024;             // choices or rows per workgroup while there are workgroups to add
constexpr int kWorkgroupsMost = 64;
constexpr int kCopies = 2048;            // LDS words for copies of the counters
constexpr int kCopiesMost = 8;

__device__ __forceinline__ int group_of(const LayoutParams& p, int i) {
  const long long g = (long long)p.ids[i] - p.first;
  const int last = p.others ? p.groups - 1 : -1;
  return g >= 0 && g < p.groups - (p.others != 0) ? (int)g : last;
}

// add(i, g) for every choice i of [begin, end) that has a group, LCOUNT loads at a time.
template <typename F>
__device__ __forceinline__ void count_choices(const LayoutParams& p, int begin, int end, F add) {
  for (long long i0 = begin + (int)threadIdx.x; i0 < end; i0 += LT * LCOUNT) {
    int g[LCOUNT];
#pragma unroll
    for (int u = 0; u < LCOUNT; ++u) g[u] = group_of(p, (int)min(i0 + u * LT, (long long)end - 1));
#pragma unroll
    for (int u = 0; u < LCOUNT; ++u)
      if (i0 + u * LT < end && g[u] >= 0) add((int)i0 + u * LT, g[u]);
  }
}

// counts[chunk][g] of each chunk
__global__ __launch_bounds__(LT) void layout_count_kernel(LayoutParams p, int chunk, int copies, int32_t* counts) {
  extern __shared__ int32_t lds[];
  for (int i = threadIdx.x; i < copies * p.groups; i += LT) lds[i] = 0;
  __syncthreads();
  int32_t* own = lds + (threadIdx.x % copies) * p.groups;
  const int begin = (int)min((long long)p.n, (long long)blockIdx.x * chunk), end = min(p.n, begin + chunk);
  count_choices(p, begin, end, [&](int, int g) { atomicAdd(&own[g], 1); });
  __syncthreads();
  for (int g = threadIdx.x; g < p.groups; g += LT) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < kCopiesMost; ++c) n += c < copies ? lds[c * p.groups + g] : 0;
    counts[(size_t)blockIdx.x * p.groups + g] = n;
  }
}

// Places one chunk's choices; every workgroup also fills its share of the
// row-indexed outputs (layout, and slot_of where a row has no choice).
// The counters of the other chunks are kept in `copies` copies, by lane, so that
// the lanes of a wave seldom meet when there are few groups.
__global__ __launch_bounds__(LT) void layout_place_kernel(LayoutParams p, int chunk, int copies,
                                                          const int32_t* counts) {
  extern __shared__ int32_t lds[];
  const int G = p.groups;
  int32_t* base = lds;                   // [LW][G]: next row of group g in wave w's run, from start[g]
  int32_t* total = lds + LW * G;         // [G]: choices of group g
  int32_t* start = total + G;            // [G + 1]: first row of group g
  int32_t* early = start + G + 1;        // [copies][G]: choices of group g in earlier chunks
  int32_t* late = early + copies * G;    // [copies][G]: in later chunks
  __shared__ int wave_span[LW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int begin = (int)min((long long)p.n, (long long)blockIdx.x * chunk), end = min(p.n, begin + chunk);
  const int run = (end - begin + LW * 64 - 1) / (LW * 64) * 64;      // choices per wave
  const int wb = min(end, begin + wave * run), we = min(end, wb + run);
  int kept[LKEEP];                       // groups of this lane's first choices
#pragma unroll
  for (int j = 0; j < LKEEP; ++j) kept[j] = wb + 64 * j + lane < we ? group_of(p, wb + 64 * j + lane) : -1;
  for (int i = tid; i < LW * G; i += LT) base[i] = 0;
  for (int i = tid; i < 2 * copies * G; i += LT) early[i] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < LKEEP; ++j)
    if (kept[j] >= 0) atomicAdd(&base[wave * G + kept[j]], 1);
  for (int i = wb + 64 * LKEEP + lane; i < we; i += 64) {
    const int g = group_of(p, i);
    if (g >= 0) atomicAdd(&base[wave * G + g], 1);
  }
  int32_t* mine = early + (tid % copies) * G;
  if (counts) {                          // one thread per group and part of the chunks
    const int parts = G < LT ? LT / G : 1;
    for (int at = tid; at < parts * G; at += LT) {
      const int g = at % G;
      int before = 0, after = 0;
#pragma unroll 8
      for (int c = at / G; c < (int)gridDim.x; c += parts) {
        const int v = counts[(size_t)c * G + g];
        before += c < (int)blockIdx.x ? v : 0;
        after += c > (int)blockIdx.x ? v : 0;
      }
      if (before) atomicAdd(&mine[g], before);
      if (after) atomicAdd(&mine[copies * G + g], after);
    }
  } else {
    count_choices(p, 0, p.n, [&](int i, int g) {
      if (i < begin || i >= end) atomicAdd(&mine[(i < begin ? 0 : copies * G) + g], 1);
    });
  }
  __syncthreads();
  // per group: the runs' offsets, the total, and the segments' starts as an
  // exclusive scan (at most n + G * (align - 1) rows, or masked G * max_m: both fit an int)
  int carry = 0;
  for (int g0 = 0; g0 < G; g0 += LT) {
    const int g = g0 + tid;
    int span = 0;
    if (g < G) {
      int n = 0, rest = 0;
#pragma unroll
      for (int c = 0; c < kCopiesMost; ++c) {
        n += c < copies ? early[c * G + g] : 0;
        rest += c < copies ? late[c * G + g] : 0;
      }
#pragma unroll
      for (int w = 0; w < LW; ++w) {
        const int c = base[w * G + g];
        base[w * G + g] = n;
        n += c;
      }
      n += rest;
      total[g] = n;
      if (blockIdx.x == 0 && p.counts) p.counts[g] = p.align ? n : min(n, p.max_m);
      span = p.align ? (n + p.align - 1) / p.align * p.align : p.max_m;
    }
    int incl = span;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 63) wave_span[wave] = incl;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < LW; ++w) {
      if (w < wave) before += wave_span[w];
      carry += wave_span[w];
    }
    if (g < G) start[g] = before + incl - span;
    __syncthreads();
  }
  const int bits = 32 - __clz(G);        // ids 0..G-1, and G for a choice without a group
  for (int j = 0, i0 = wb; i0 < we; ++j, i0 += 64) {
    const int i = i0 + lane;
    int g;
    switch (j) {                         // kept[j] with a constant index
      case 0: g = kept[0]; break;
      case 1: g = kept[1]; break;
      case 2: g = kept[2]; break;
      case 3: g = kept[3]; break;
      default: g = i < we ? group_of(p, i) : -1;
    }
    const int key = g >= 0 ? g : G;
    uint64_t same = ~0ull;               // lanes with this lane's group
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? m : ~m;
    }
    int rank = 0;
    if (g >= 0) {
      const int at = wave * G + g;
      rank = base[at] + __popcll(same & ((1ull << lane) - 1));
      // the group's last lane moves the run's counter on; the reads above are of
      // the same wave and come first
      __builtin_amdgcn_wave_barrier();
      if ((same >> lane) == 1) base[at] = rank + 1;
    }
    __builtin_amdgcn_wave_barrier();
    if (i < we) {
      const bool in = g >= 0 && (p.align || rank < p.max_m);
      const int row = in ? start[g] + rank : -1;
      const bool fits = in && row < p.rows;
      if (p.row_of) p.row_of[i] = fits ? row : -1;
      if (fits) p.slot_of[row] = i;
    }
  }
  // row-indexed outputs
  for (long long r = (long long)blockIdx.x * LT + tid; r < p.rows; r += (long long)gridDim.x * LT) {
    int g, rank;
    if (p.align) {
      int lo = 0, hi = G;                // the last group that starts at or before r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= r) lo = mid; else hi = mid;
      }
      g = lo;
      rank = (int)(r - start[g]);
    } else {
      g = (int)r / p.max_m;
      rank = (int)r - g * p.max_m;
    }
    const bool used = rank < total[g];
    if (p.layout) p.layout[r] = used ? g : -1;
    if (!used) p.slot_of[r] = -1;
  }
}

}  // namespace

hipError_t launch_layout(const LayoutParams& p, void* scratch, size_t scratch_bytes, hipStream_t stream) {
  const long long most = p.n > p.rows ? p.n : p.rows;
  int grid = (int)((most + kShare - 1) / kShare);
  grid = grid < 1 ? 1 : (grid > kWorkgroupsMost ? kWorkgroupsMost : grid);
  int copies = kCopies / (2 * p.groups);
  copies = copies < 1 ? 1 : (copies > kCopiesMost ? kCopiesMost : copies);
  int32_t* counts = nullptr;
  if (p.n > kOneLaunch && (size_t)grid * p.groups * sizeof(int32_t) <= scratch_bytes)
    counts = static_cast<int32_t*>(scratch);
  const int chunk = (int)((p.n + (long long)grid - 1) / grid);
  if (counts) {
    layout_count_kernel<<<grid, LT, sizeof(int32_t) * copies * p.groups, stream>>>(p, chunk, copies, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const size_t lds = sizeof(int32_t) * ((LW + 2 + 2 * copies) * (size_t)p.groups + 1);
  layout_place_kernel<<<grid, LT, lds, stream>>>(p, chunk, copies, counts);
  return hipGetLastError();
}

namespace {

// ============================================================================
// scatter: quantise the tokens' rows into the products' A operands
// ============================================================================
constexpr float kE4m3Max = 448.0f;
constexpr float kLeastAmax = 0x1p-100f;

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf16_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// Scales and quotients are worked out in 64 bits: a product of a bf16 and an fp32
// value is exact there, and blocks of bf16 values often hold quotients that lie
// halfway between two codes, which fp32 roundings on the way would tip to either
// side.  The quotient is rounded to fp32 at the end, which takes the last fp64
// roundings out of such ties again, and then to a code.  The fp64 units run at the
// fp32 rate here, and the calls are bound by their bytes all the same.

// The scale of a block whose largest magnitude is amax (include/dg.h).
__device__ __forceinline__ float scale_of(double amax, bool pow2) {
  if (!(amax > 0.0)) return 1.0f;
  float sf = (float)(fmax(amax, (double)kLeastAmax) * (1.0 / 448.0));
  if (pow2) {
    const uint32_t u = __float_as_uint(sf);              // normal: at least 2^-100 / 448
    sf = u >= 0x7F800000u ? sf : __uint_as_float((u + 0x7FFFFFu) & 0x7F800000u);
  }
  return sf;
}
// What its values are multiplied by: 1 / sf before sf's rounding.
__device__ __forceinline__ double inverse_of(double amax, float sf, bool pow2) {
  if (!(amax > 0.0) || pow2) return 1.0 / (double)sf;
  return (double)kE4m3Max / fmax(amax, (double)kLeastAmax);
}

// Four e4m3 codes packed in an int, rounded to nearest even.  Products with a
// block's inverse need no clamp: they exceed 448 by less than 2^-22 of it, which
// rounds to 448 (the next step would begin at 464).  NaN, also from an infinity
// times 0, gives the NaN code.
__device__ __forceinline__ int pack_e4m3(float a, float b, float c, float d) {
  const int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

struct ScatterParams {
  const uint16_t* x;
  const float* weights;
  const int32_t* row_of;
  const int32_t* slot_of;
  uint8_t* a;
  float* sfa;
  int T, top_k;
  int rows;                // all rows: M, or G * max_m
  int rows_per_group;      // sfa is [rows / rows_per_group][K/128][rows_per_group]
  int K;
  int pow2;
};

// The block scales of many rows, row by row: sfa is laid out along the rows, and
// written from the tokens' side each line would be touched by some 16 workgroups
// (65536 rows of 7168: 24 us of 142).  The scatter leaves the blocks' maxima in
// table[T][ld], and here a wave writes 64 neighbouring rows' scales (10.8 us for
// 98048 rows of 56, of which 65536 are in use).
__global__ __launch_bounds__(256) void scatter_scales_kernel(ScatterParams p, const float* table, int ld) {
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= (size_t)p.rows) return;
  const int row = (int)at;
  const int slot = p.slot_of[row];
  if (slot < 0 || slot >= (long long)p.T * p.top_k) return;
  const int KB = p.K / 128;
  const float w = p.weights ? fabsf(p.weights[slot]) : 1.0f;
  const float* amax = table + (size_t)(slot / p.top_k) * ld;
  const int g = row / p.rows_per_group;
  float* sfa = p.sfa + (size_t)g * KB * p.rows_per_group + (row - g * p.rows_per_group);
  for (int kb = blockIdx.y * 4; kb < KB; kb += gridDim.y * 4) {
    const float4 m = *reinterpret_cast<const float4*>(amax + kb);
    const float v[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (kb + e < KB) sfa[(size_t)(kb + e) * p.rows_per_group] = scale_of((double)w * v[e], p.pow2);
  }
}

constexpr int SJ = 8;                    // rows a thread writes per turn; also lanes per block

// One thread per sixteen values of a token, eight threads per block of 128: the
// token is read and quantised once and stored to all its rows (without weights;
// with them the products are quantised per row).  In each group of eight lanes,
// lane i also works out and stores the scale of row i of the turn.  Bound by the
// bytes: 65536 rows of 7168 from 8192 tokens take 118 us without their scales
// (4.97 TB/s; with weights 120), 8192 rows from 4096 tokens 26.5 us with them (4.5
// TB/s); one workgroup per row, reading its token again for each, took 255 and 34.
template <bool WEIGHTED, bool MASKED, bool TABLE>
__global__ __launch_bounds__(256) void scatter_kernel(ScatterParams p, float* table, int ld) {
  const int per_token = p.K / 16;
  const size_t total = (size_t)p.T * per_token;        // a multiple of 8
  const int lane8 = threadIdx.x & 7;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
    const int t = (int)(i / per_token);
    const int k = (int)(i - (size_t)t * per_token) * 16;
    const u16x8* x = reinterpret_cast<const u16x8*>(p.x + (size_t)t * p.K + k);
    const u16x8 h0 = x[0], h1 = x[1];
    float v[16], amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = bf16_f32(h0[e]);
      v[8 + e] = bf16_f32(h1[e]);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    if (TABLE && lane8 == 0) table[(size_t)t * ld + k / 128] = amax;
    auto codes = [&](double f) {
      float u[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) u[e] = (float)((double)v[e] * f);
      return make_int4(pack_e4m3(u[0], u[1], u[2], u[3]), pack_e4m3(u[4], u[5], u[6], u[7]),
                       pack_e4m3(u[8], u[9], u[10], u[11]), pack_e4m3(u[12], u[13], u[14], u[15]));
    };
    int4 q;
    float sf = 1.0f;
    if constexpr (!WEIGHTED) {
      sf = scale_of(amax, p.pow2);
      q = codes(inverse_of(amax, sf, p.pow2));
    }
    for (int j0 = 0; j0 < p.top_k; j0 += SJ) {
      const int32_t* at = p.row_of + (size_t)t * p.top_k + j0;
      const float* wt = WEIGHTED ? p.weights + (size_t)t * p.top_k + j0 : nullptr;
      const int left = p.top_k - j0;
      int rows[SJ];
#pragma unroll
      for (int j = 0; j < SJ; ++j) rows[j] = at[j < left ? j : 0];
      const int mine = lane8 < left ? at[lane8] : -1;          // this lane's row of the scales
      double factor = 0.0;                                     // this lane's row: its weight times the inverse
      if constexpr (WEIGHTED) {
        const float w = wt[lane8 < left ? lane8 : 0];
        const double most = (double)fabsf(w) * amax;
        sf = scale_of(most, p.pow2);
        factor = w * inverse_of(most, sf, p.pow2);
      }
      if (!TABLE && mine >= 0 && mine < p.rows) {
        const int KB = p.K / 128, kb = k / 128;
        if constexpr (MASKED) {
          const int g = mine / p.rows_per_group;
          p.sfa[((size_t)g * KB + kb) * p.rows_per_group + (mine - g * p.rows_per_group)] = sf;
        } else {
          p.sfa[(size_t)kb * p.rows + mine] = sf;
        }
      }
#pragma unroll
      for (int j = 0; j < SJ; ++j) {
        if (j >= left) break;
        if constexpr (WEIGHTED) q = codes(__shfl(factor, j, 8));
        if (rows[j] >= 0 && rows[j] < p.rows) *reinterpret_cast<int4*>(p.a + (size_t)rows[j] * p.K + k) = q;
      }
    }
  }
}

// max(a, |b|), b's NaN left out; one instruction, without the quieting of signalling
// NaN (products are none) that the C function implies.
__device__ __forceinline__ double max_abs_f64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, |%2|" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

struct KScatterParams {
  const uint16_t* x;
  const float* weights;
  const int32_t* slot_of;
  uint8_t* a;
  float* sfa;
  int T, top_k;
  int K, N;                // K rows of N columns
  int pow2;
};

// One workgroup per 128 rows x 128 columns: 16 threads across (8 columns each)
// and KR rows per thread.  The rows stay in registers between the
// columns' maxima and the codes; one thread per column works out its scale.
// A value times its inverse comes from pairs of fp32 (a product and its exact
// remainder by FMA); the weighted maxima take fp64 instructions, and so do the
// codes of a block where a product is beyond fp32's range.  A row is read
// and written once; bound by the chain of map, row and maxima before the first
// store: 9088 rows of 4096 columns take 23.7 us weighted (3.05 TB/s) and 18.9
// unweighted in workgroups of 512 threads, 24.9 weighted in ones of 256 with 8 rows
// per thread.
constexpr int KT = 512;                  // threads per workgroup
constexpr int KR = 128 * 16 / KT;        // rows per thread
constexpr int kMaxGridY = 65535;         // a grid's second axis; what is beyond goes on the third

template <bool WEIGHTED>
__global__ __launch_bounds__(KT) void kscatter_kernel(KScatterParams p) {
  __shared__ double part[KT / 16][128];
  __shared__ float2 inverse[128];          // the sum of the two
  __shared__ int beyond[2];                // per wave: a column's maximum has no fp32 product
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const size_t block = (size_t)blockIdx.z * kMaxGridY + blockIdx.y;
  if (block >= (size_t)p.K / 128) return;
  const size_t row0 = block * 128;
  const int col = blockIdx.x * 128 + tx * 8;
  const bool in = col < p.N;               // N % 16 == 0: whole 8-column pieces
  int slot[KR];
#pragma unroll
  for (int i = 0; i < KR; ++i) slot[i] = p.slot_of[row0 + ty + KT / 16 * i];
  u16x8 h[KR];
  float w[KR];
  auto load = [&](int s, u16x8& hs, float& ws) {
    hs = u16x8{};
    ws = 0.0f;                             // a row without a choice: zeros
    if (in && s >= 0 && s < (long long)p.T * p.top_k) {
      hs = *reinterpret_cast<const u16x8*>(p.x + (size_t)(s / p.top_k) * p.N + col);
      if constexpr (WEIGHTED) ws = p.weights[s];
    }
  };
#pragma unroll
  for (int i = 0; i < KR; ++i) load(slot[i], h[i], w[i]);
  if constexpr (WEIGHTED) {
    double amax[8] = {};
#pragma unroll
    for (int i = 0; i < KR; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax[j] = max_abs_f64(amax[j], (double)w[i] * bf16_f32(h[i][j]));
#pragma unroll
    for (int j = 0; j < 8; ++j) part[ty][tx * 8 + j] = amax[j];
  } else {
    float amax[8] = {};
#pragma unroll
    for (int i = 0; i < KR; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax[j] = fmaxf(amax[j], fabsf(bf16_f32(h[i][j])));
#pragma unroll
    for (int j = 0; j < 8; ++j) part[ty][tx * 8 + j] = amax[j];
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    double m = 0.0;
#pragma unroll
    for (int r = 0; r < KT / 16; ++r) m = fmax(m, part[r][threadIdx.x]);
    const float sf = scale_of(m, p.pow2);
    const double inv = inverse_of(m, sf, p.pow2);
    const float hi = (float)inv;           // beyond fp32's range only where values below 2^-100 round to 0
    inverse[threadIdx.x] = make_float2(hi, (float)(inv - hi));
    if constexpr (WEIGHTED) {
      part[0][threadIdx.x] = inv;          // this thread has read its column
      const bool any = __any(m > (double)FLT_MAX);
      if ((threadIdx.x & 63) == 0) beyond[threadIdx.x >> 6] = any;
    }
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c < p.N) p.sfa[block * p.N + c] = sf;
  }
  __syncthreads();
  if (!in) return;
  if constexpr (WEIGHTED) {
    if (__builtin_expect(beyond[0] | beyond[1], 0)) {
      // the rows again, one at a time: kept for this, they cost the others registers
      // (weighted rows of 4096 columns: 27 us against 23)
#pragma unroll 1
      for (int i = 0; i < KR; ++i) {
        const size_t row = row0 + ty + KT / 16 * i;
        asm volatile("" ::: "memory");     // the inverses too: no register holds them from row to row
        load(p.slot_of[row], h[0], w[0]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)((double)w[0] * bf16_f32(h[0][j]) * part[0][tx * 8 + j]);
        int2 q;
        q.x = pack_e4m3(v[0], v[1], v[2], v[3]);
        q.y = pack_e4m3(v[4], v[5], v[6], v[7]);
        *reinterpret_cast<int2*>(p.a + row * p.N + col) = q;
      }
      return;
    }
  }
  float2 inv[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) inv[j] = inverse[tx * 8 + j];
#pragma unroll
  for (int i = 0; i < KR; ++i) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = bf16_f32(h[i][j]);
      if constexpr (WEIGHTED) {
        const float wx = __fmul_rn(w[i], x), rest = fmaf(w[i], x, -wx);
        v[j] = fmaf(wx, inv[j].x, fmaf(wx, inv[j].y, __fmul_rn(rest, inv[j].x)));
      } else {
        v[j] = fmaf(x, inv[j].x, __fmul_rn(x, inv[j].y));
      }
    }
    int2 q;
    q.x = pack_e4m3(v[0], v[1], v[2], v[3]);
    q.y = pack_e4m3(v[4], v[5], v[6], v[7]);
    *reinterpret_cast<int2*>(p.a + (row0 + ty + KT / 16 * i) * p.N + col) = q;
  }
}

// ============================================================================
// gather: the experts' rows back to the tokens
// ============================================================================
constexpr int kMaxTopK = 64;

struct GatherParams {
  const uint16_t* rows;
  const int32_t* row_of;
  const float* weights;
  const uint16_t* c;
  uint16_t* d;
  const uint16_t* grad_d;
  float* grad_weights;
  int T, top_k, M, N;
};

__device__ __forceinline__ uint16_t f32_bf16(float x) {
  __bf16 h = static_cast<__bf16>(x);
  return __builtin_bit_cast(uint16_t, h);
}

// Eight neighbouring bf16 at any 2-byte address (rows of an odd N start anywhere;
// the hardware's 16-byte loads and stores take any alignment).
typedef u16x8 u16x8_any __attribute__((aligned(2)));

constexpr int GJ = 8;                    // rows in flight per thread

// Columns n..n+7 of a row (WHOLE), or its columns from n up to N, then zeros.
template <bool WHOLE>
__device__ __forceinline__ u16x8 load_piece(const uint16_t* row, int n, int N) {
  if constexpr (WHOLE) return __builtin_nontemporal_load(reinterpret_cast<const u16x8_any*>(row + n));
  u16x8 v = {};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (n + e < N) v[e] = row[n + e];
  return v;
}

template <bool WHOLE>
__device__ __forceinline__ void gather_piece(const GatherParams& p, size_t t, int n) {
  float sum[8] = {};
  if (p.c) {
    const u16x8 c = load_piece<WHOLE>(p.c + t * p.N, n, p.N);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = bf16_f32(c[e]);
  }
  for (int j0 = 0; j0 < p.top_k; j0 += GJ) {
    // the same for the workgroup: scalar loads, in flight together
    int rs[GJ];
    float ws[GJ];
#pragma unroll
    for (int j = 0; j < GJ; ++j) {
      const bool in = j0 + j < p.top_k;
      const int r = p.row_of[t * p.top_k + (in ? j0 + j : 0)];
      rs[j] = in && r >= 0 && r < p.M ? r : -1;
      ws[j] = p.weights ? p.weights[t * p.top_k + (in ? j0 + j : 0)] : 1.0f;
    }
    int some = -1;                       // a slot without a row loads another's again: no branch between the loads
#pragma unroll
    for (int j = 0; j < GJ; ++j) some = rs[j] >= 0 ? rs[j] : some;
    if (some < 0) continue;
    u16x8 v[GJ];
#pragma unroll
    for (int j = 0; j < GJ; ++j)
      v[j] = load_piece<WHOLE>(p.rows + (size_t)(rs[j] >= 0 ? rs[j] : some) * p.N, n, p.N);
#pragma unroll
    for (int j = 0; j < GJ; ++j)
      if (rs[j] >= 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = fmaf(ws[j], bf16_f32(v[j][e]), sum[e]);
  }
  uint16_t* d = p.d + t * p.N + n;
  u16x8 o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = f32_bf16(sum[e]);
  if constexpr (WHOLE)
    *reinterpret_cast<u16x8_any*>(d) = o;
  else
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (n + e < p.N) d[e] = o[e];
}

// One thread per token and eight columns; the token's rows and weights are the
// same for the whole workgroup.  Bound by the rows' bytes: GJ 16-byte loads per
// thread are in flight before the first is summed, with the streaming policy
// (8192 tokens x 8 rows of 7168: 196 us against 201 with the default one), and
// a token's workgroups follow one another, so that its rows' pages are read whole
// (201 us against 206 with the tokens running fastest).
__global__ __launch_bounds__(256) void gather_kernel(GatherParams p) {
  const size_t t = (size_t)blockIdx.z * kMaxGridY + blockIdx.y;
  const int n = (blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (t >= (size_t)p.T) return;
  if (n + 8 <= p.N)
    gather_piece<true>(p, t, n);
  else if (n < p.N)
    gather_piece<false>(p, t, n);
}

// One workgroup per token and JG of its choices: a piece of grad_d is read once
// for them all.  Bound by the rows' bytes: 4095 tokens x 2 rows of 7165 take 36.7
// us, 4.6 TB/s.
template <int JG>
__global__ __launch_bounds__(256) void gather_weight_grad_kernel(GatherParams p) {
  __shared__ float part[4][JG];
  const int parts = (p.top_k + JG - 1) / JG;
  for (size_t i = blockIdx.x; i < (size_t)p.T * parts; i += gridDim.x) {
    const size_t t = i / parts;
    const int j0 = (int)(i - t * parts) * JG;
    const uint16_t* g = p.grad_d + t * p.N;
    int rs[JG], some = -1;
#pragma unroll
    for (int j = 0; j < JG; ++j) {
      const bool in = j0 + j < p.top_k;
      const int r = p.row_of[t * p.top_k + (in ? j0 + j : j0)];
      rs[j] = in && r >= 0 && r < p.M ? r : -1;
      some = rs[j] >= 0 ? rs[j] : some;
    }
    const uint16_t* row[JG];               // a slot without a row reads another's again and keeps 0
#pragma unroll
    for (int j = 0; j < JG; ++j) row[j] = p.rows + (size_t)(rs[j] >= 0 ? rs[j] : some) * p.N;
    float sum[JG] = {};
    auto add = [&](auto whole, int n) {
      const u16x8 gv = load_piece<whole.value>(g, n, p.N);
      u16x8 v[JG];
#pragma unroll
      for (int j = 0; j < JG; ++j) v[j] = load_piece<whole.value>(row[j], n, p.N);
#pragma unroll
      for (int j = 0; j < JG; ++j)
        if (rs[j] >= 0)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[j] = fmaf(bf16_f32(gv[e]), bf16_f32(v[j][e]), sum[j]);
    };
    int n = some >= 0 ? threadIdx.x * 8 : p.N;
#pragma unroll 2
    for (; n + 8 <= p.N; n += 256 * 8) add(std::true_type{}, n);
    if (n < p.N) add(std::false_type{}, n);
#pragma unroll
    for (int j = 0; j < JG; ++j) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum[j] += __shfl_xor(sum[j], o);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][j] = sum[j];
    }
    __syncthreads();
    const int j = threadIdx.x;
    if (j < JG && j0 + j < p.top_k)
      p.grad_weights[t * p.top_k + j0 + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
    __syncthreads();                     // part is written again for the next item
  }
}

int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

// ---- argument checks shared by the entry points ------------------------------
constexpr long long kMaxChoices = 1LL << 30;
// Scales row by row from here on, by the rows that there are: with 65536 of 98048
// rows of 7168 in use the two kernels take 130 us against 142 in one, with 32768 of
// 65280 56 against 75, with 16384 of 48896 29 against 31, with 8192 of 40704 the
// same.  Below 32768 rows few can be in use (8192: the scales' scattered words cost
// 1.5 us of 27, less than a second launch).  Buffers of more rows that are nearly
// empty pay for the second launch: 512 choices in 256 x 128 masked rows take 7.0
// us against 4.4.
constexpr long long kScaleRows = 32768;
constexpr long long kMaxGrid = 1 << 23;  // workgroups: a grid's thread count has 32 bits

int check_choices(int T, int top_k) {
  if (T < 0 || top_k < 1) return fail(DG_ERR_INVALID_ARG, "T=%d must not be negative and top_k=%d at least 1", T, top_k);
  if ((long long)T * top_k > kMaxChoices)
    return fail(DG_ERR_UNSUPPORTED, "T * top_k = %lld choices exceed 2^30", (long long)T * top_k);
  return DG_OK;
}

int check_layout_call(const int32_t* ids, int T, int top_k, int num_groups, const int32_t* row_of,
                      const int32_t* slot_of, long long rows) {
  int s = check_choices(T, top_k);
  if (s != DG_OK) return s;
  if (num_groups < 1) return fail(DG_ERR_INVALID_ARG, "num_groups=%d must be at least 1", num_groups);
  if (num_groups > kMaxLayoutGroups)
    return fail(DG_ERR_UNSUPPORTED, "num_groups=%d exceeds %d", num_groups, kMaxLayoutGroups);
  if (rows > INT_MAX) return fail(DG_ERR_UNSUPPORTED, "%lld rows exceed 2^31 - 1", rows);
  if (T > 0 && (!ids || !row_of)) return fail(DG_ERR_INVALID_ARG, "topk_ids and row_of must not be NULL");
  if (rows > 0 && !slot_of) return fail(DG_ERR_INVALID_ARG, "slot_of must not be NULL");
  if (!aligned(ids, 4) || !aligned(row_of, 4) || !aligned(slot_of, 4))
    return fail(DG_ERR_INVALID_ARG, "topk_ids, row_of and slot_of must be 4-byte aligned");
  return DG_OK;
}

int run_layout(LayoutParams& p, void* stream) {
  Scratch sc;
  const int s = call_scratch(static_cast<hipStream_t>(stream), &sc);
  if (s != DG_OK) return s;
  const hipError_t e = launch_layout(p, sc.ptr, sc.bytes, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? DG_OK : fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

int scatter(const void* x, const float* weights, const int32_t* row_of, const int32_t* slot_of, void* a, float* sfa,
            int T, int top_k, long long rows, int rows_per_group, int K, int pow2, void* stream) {
  int s = check_choices(T, top_k);
  if (s != DG_OK) return s;
  if (K < 0) return fail(DG_ERR_INVALID_ARG, "negative size (K=%d)", K);
  if (K % 128 != 0) return fail(DG_ERR_INVALID_ARG, "K=%d is not a multiple of 128", K);
  if (rows > INT_MAX) return fail(DG_ERR_UNSUPPORTED, "%lld rows exceed 2^31 - 1", rows);
  if (T == 0 || rows == 0 || K == 0) return DG_OK;
  if (!x || !row_of || !slot_of || !a || !sfa)
    return fail(DG_ERR_INVALID_ARG, "x, row_of, slot_of, a and sfa must not be NULL");
  if (!aligned(x, 16) || !aligned(a, 16)) return fail(DG_ERR_INVALID_ARG, "x and a must be 16-byte aligned");
  if (!aligned(sfa, 4) || !aligned(weights, 4) || !aligned(row_of, 4) || !aligned(slot_of, 4))
    return fail(DG_ERR_INVALID_ARG, "sfa, weights, row_of and slot_of must be 4-byte aligned");
  ScatterParams p{static_cast<const uint16_t*>(x), weights, row_of, slot_of, static_cast<uint8_t*>(a), sfa, T, top_k,
                  (int)rows, rows_per_group, K, pow2 != 0};
  const long long wgs = ((long long)T * (K / 16) + 255) / 256;
  const int grid = (int)(wgs < kMaxGrid ? wgs : kMaxGrid);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // the scales row by row from kScaleRows rows on, if the workspace has room for the maxima
  const int ld = (K / 128 + 3) / 4 * 4;
  float* table = nullptr;
  if (rows >= kScaleRows) {
    Scratch sc;
    s = call_scratch(st, &sc);
    if (s != DG_OK) return s;
    if ((size_t)T * ld * sizeof(float) <= sc.bytes) table = reinterpret_cast<float*>(sc.ptr);
  }
  if (table) {
    weights ? scatter_kernel<true, false, true><<<grid, 256, 0, st>>>(p, table, ld)
            : scatter_kernel<false, false, true><<<grid, 256, 0, st>>>(p, table, ld);
    const int parts = ld / 4 < 16 ? ld / 4 : 16;
    scatter_scales_kernel<<<dim3((int)((rows + 255) / 256), parts), 256, 0, st>>>(p, table, ld);
  } else if (rows_per_group != rows) {
    weights ? scatter_kernel<true, true, false><<<grid, 256, 0, st>>>(p, nullptr, 0)
            : scatter_kernel<false, true, false><<<grid, 256, 0, st>>>(p, nullptr, 0);
  } else {
    weights ? scatter_kernel<true, false, false><<<grid, 256, 0, st>>>(p, nullptr, 0)
            : scatter_kernel<false, false, false><<<grid, 256, 0, st>>>(p, nullptr, 0);
  }
  return launched();
}

int check_gather(const void* rows, const int32_t* row_of, int T, int top_k, int M, int N) {
  int s = check_choices(T, top_k);
  if (s != DG_OK) return s;
  if (M < 0 || N < 0) return fail(DG_ERR_INVALID_ARG, "negative size (M=%d N=%d)", M, N);
  if (top_k > kMaxTopK) return fail(DG_ERR_UNSUPPORTED, "top_k=%d exceeds %d", top_k, kMaxTopK);
  if (N > 1 << 30) return fail(DG_ERR_UNSUPPORTED, "N=%d exceeds 2^30", N);
  if (T > 0 && !row_of) return fail(DG_ERR_INVALID_ARG, "row_of must not be NULL");
  if (T > 0 && M > 0 && N > 0 && !rows) return fail(DG_ERR_INVALID_ARG, "rows must not be NULL");
  if (!aligned(rows, 2) || !aligned(row_of, 4))
    return fail(DG_ERR_INVALID_ARG, "rows must be 2-byte and row_of 4-byte aligned");
  return DG_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" int dg_m_grouped_rows_bound(long long choices, int num_groups) {
  if (choices < 0 || num_groups < 0) return -1;
  const long long used = choices < num_groups ? choices : num_groups;
  if (choices > INT_MAX) return -1;
  const long long rows = (choices + 127 * used) / 128 * 128;
  return rows > INT_MAX ? -1 : (int)rows;
}

extern "C" int dg_m_grouped_layout_contiguous(const int32_t* topk_ids, int T, int top_k, int first_expert,
                                              int num_groups, int M, int32_t* grouped_layout, int32_t* row_of,
                                              int32_t* slot_of, int32_t* counts, void* stream) {
  int s = check_layout_call(topk_ids, T, top_k, num_groups, row_of, slot_of, M);
  if (s != DG_OK) return s;
  if (M < 0 || M % 128 != 0) return fail(DG_ERR_INVALID_ARG, "M=%d is not a non-negative multiple of 128", M);
  if (M > 0 && !grouped_layout) return fail(DG_ERR_INVALID_ARG, "grouped_layout must not be NULL");
  if (!aligned(grouped_layout, 4) || !aligned(counts, 4))
    return fail(DG_ERR_INVALID_ARG, "grouped_layout and counts must be 4-byte aligned");
  LayoutParams p{topk_ids, T * top_k, first_expert, num_groups, 128, 0, M, grouped_layout, row_of, slot_of, counts, 0};
  return run_layout(p, stream);
}

extern "C" int dg_m_grouped_layout_masked(const int32_t* topk_ids, int T, int top_k, int first_expert, int num_groups,
                                          int max_m, int32_t* masked_m, int32_t* row_of, int32_t* slot_of,
                                          void* stream) {
  if (max_m < 0) return fail(DG_ERR_INVALID_ARG, "negative size (max_m=%d)", max_m);
  int s = check_layout_call(topk_ids, T, top_k, num_groups, row_of, slot_of, (long long)num_groups * max_m);
  if (s != DG_OK) return s;
  if (!masked_m) return fail(DG_ERR_INVALID_ARG, "masked_m must not be NULL");
  if (!aligned(masked_m, 4)) return fail(DG_ERR_INVALID_ARG, "masked_m must be 4-byte aligned");
  LayoutParams p{topk_ids, T * top_k, first_expert, num_groups, 0, max_m, num_groups * max_m, nullptr, row_of,
                 slot_of, masked_m, 0};
  return run_layout(p, stream);
}

extern "C" int dg_m_grouped_scatter_fp8_contiguous(const void* x, const float* weights, const int32_t* row_of,
                                                   const int32_t* slot_of, void* a, float* sfa, int T, int top_k,
                                                   int M, int K, int pow2_scales, void* stream) {
  if (M < 0) return fail(DG_ERR_INVALID_ARG, "negative size (M=%d)", M);
  return scatter(x, weights, row_of, slot_of, a, sfa, T, top_k, M, M, K, pow2_scales, stream);
}

extern "C" int dg_m_grouped_scatter_fp8_masked(const void* x, const float* weights, const int32_t* row_of,
                                               const int32_t* slot_of, void* a, float* sfa, int T, int top_k,
                                               int num_groups, int max_m, int K, int pow2_scales, void* stream) {
  if (num_groups < 1) return fail(DG_ERR_INVALID_ARG, "num_groups=%d must be at least 1", num_groups);
  if (max_m < 0) return fail(DG_ERR_INVALID_ARG, "negative size (max_m=%d)", max_m);
  return scatter(x, weights, row_of, slot_of, a, sfa, T, top_k, (long long)num_groups * max_m, max_m, K, pow2_scales,
                 stream);
}

extern "C" int dg_k_grouped_scatter_fp8(const void* x, const float* weights, const int32_t* slot_of, void* a,
                                        float* sfa, int T, int top_k, int K, int N, int pow2_scales, void* stream) {
  int s = check_choices(T, top_k);
  if (s != DG_OK) return s;
  if (K < 0 || N < 0) return fail(DG_ERR_INVALID_ARG, "negative size (K=%d N=%d)", K, N);
  if (K % 128 != 0) return fail(DG_ERR_INVALID_ARG, "K=%d is not a multiple of 128", K);
  if (N % 16 != 0) return fail(DG_ERR_UNSUPPORTED, "the K-grouped product needs N a multiple of 16 (N=%d)", N);
  if (N >= 1 << 30) return fail(DG_ERR_UNSUPPORTED, "N=%d must be below 2^30", N);     // 4 threads per column: a grid has 2^32
  if (K == 0 || N == 0) return DG_OK;
  if ((T > 0 && !x) || !slot_of || !a || !sfa)
    return fail(DG_ERR_INVALID_ARG, "x, slot_of, a and sfa must not be NULL");
  if (!aligned(x, 16) || !aligned(a, 16)) return fail(DG_ERR_INVALID_ARG, "x and a must be 16-byte aligned");
  if (!aligned(sfa, 4) || !aligned(weights, 4) || !aligned(slot_of, 4))
    return fail(DG_ERR_INVALID_ARG, "sfa, weights and slot_of must be 4-byte aligned");
  KScatterParams p{static_cast<const uint16_t*>(x), weights, slot_of, static_cast<uint8_t*>(a), sfa, T, top_k, K, N,
                   pow2_scales != 0};
  const int blocks = K / 128;
  const dim3 grid((N + 127) / 128, blocks < kMaxGridY ? blocks : kMaxGridY, (blocks + kMaxGridY - 1) / kMaxGridY);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (weights)
    kscatter_kernel<true><<<grid, KT, 0, st>>>(p);
  else
    kscatter_kernel<false><<<grid, KT, 0, st>>>(p);
  return launched();
}

extern "C" int dg_m_grouped_gather(const void* rows, const int32_t* row_of, const float* weights, const void* c,
                                   void* d, int T, int top_k, int M, int N, void* stream) {
  int s = check_gather(rows, row_of, T, top_k, M, N);
  if (s != DG_OK) return s;
  if (T == 0 || N == 0) return DG_OK;
  if (!d) return fail(DG_ERR_INVALID_ARG, "d must not be NULL");
  if (!aligned(d, 2) || !aligned(c, 2) || !aligned(weights, 4))
    return fail(DG_ERR_INVALID_ARG, "c and d must be 2-byte and weights 4-byte aligned");
  GatherParams p{};
  p.rows = static_cast<const uint16_t*>(rows);
  p.row_of = row_of;
  p.weights = weights;
  p.c = static_cast<const uint16_t*>(c);
  p.d = static_cast<uint16_t*>(d);
  p.T = T;
  p.top_k = top_k;
  p.M = M;
  p.N = N;
  // 2048 columns per workgroup, or 512 where that would leave CUs without one
  // (16 tokens of 8 rows of 7168: 2.8 us against 2.9)
  const int pieces = (int)((N + 7LL) / 8);
  const int threads = (long long)T * ((pieces + 255) / 256) >= 512 ? 256 : 64;
  const dim3 grid((pieces + threads - 1) / threads, T < kMaxGridY ? T : kMaxGridY, (T + kMaxGridY - 1) / kMaxGridY);
  gather_kernel<<<grid, threads, 0, static_cast<hipStream_t>(stream)>>>(p);
  return launched();
}

extern "C" int dg_m_grouped_gather_weight_grad(const void* rows, const int32_t* row_of, const void* grad_d,
                                               float* grad_weights, int T, int top_k, int M, int N, void* stream) {
  int s = check_gather(rows, row_of, T, top_k, M, N);
  if (s != DG_OK) return s;
  if (T == 0) return DG_OK;
  if ((N > 0 && !grad_d) || !grad_weights)
    return fail(DG_ERR_INVALID_ARG, "grad_d and grad_weights must not be NULL");
  if (!aligned(grad_d, 2) || !aligned(grad_weights, 4))
    return fail(DG_ERR_INVALID_ARG, "grad_d must be 2-byte and grad_weights 4-byte aligned");
  GatherParams p{};
  p.rows = static_cast<const uint16_t*>(rows);
  p.row_of = row_of;
  p.grad_d = static_cast<const uint16_t*>(grad_d);
  p.grad_weights = grad_weights;
  p.T = T;
  p.top_k = top_k;
  p.M = M;
  p.N = N;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // two choices per workgroup where eight would leave CUs idle (64 tokens of 8 rows
  // of 7168: 4.1 us against 7.3), eight to read grad_d once (1024 tokens: the same)
  const int jg = top_k <= 2 || T < 512 ? 2 : 8;
  const long long items = (long long)T * ((top_k + jg - 1) / jg);
  const int grid = (int)(items < kMaxGrid ? items : kMaxGrid);
  if (jg == 2)
    gather_weight_grad_kernel<2><<<grid, 256, 0, st>>>(p);
  else
    gather_weight_grad_kernel<8><<<grid, 256, 0, st>>>(p);
  return launched();
}

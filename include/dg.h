/*
 * dg.h -- FP8 (OCP e4m3) GEMM with fine-grained block scaling for AMD MI355X (gfx950).
 *
 * What the calls compute (DeepGEMM pages: likun.im/craft/deepgemm.html, section
 * 一 "the GEMM family", D = C + A @ B in the NT layout, and section 二, the
 * register_apis listing of the dense call and the two M-grouped MoE calls;
 * aitangshan.cn/news/1491278, "4. FP8 精度优化的核心": each block's GEMM result is
 * multiplied by that block's scale factors):
 *
 *   D[m,n] = bf16_rne( C[m,n] + sum_kb sa[kb][m] * sb[n/128][kb]
 *                                      * sum_{k in block kb} A[m,k] * B[n,k] )
 *
 * with kb running over the K/128 blocks of 128 consecutive K indices.  A and B
 * hold e4m3 codes; every product is summed in fp32 on the GPU ("fp32
 * accumulation"); each block's partial sum is multiplied by its A scale (one
 * per row per block, "1x128") and its B scale (one per 128x128 block) and added
 * to an fp32 total; C is added and the total is rounded once to bf16 (round to
 * nearest, ties to even).
 *
 * Layouts (every array row-major, every pointer a device pointer on the
 * current HIP device, owned by the caller; the library keeps no pointer after
 * the call returns):
 *   a    uint8  [M][K]            e4m3 codes, K contiguous            (16-byte aligned)
 *   sfa  float  [K/128][M]        A scales, M contiguous ("MN-major") (4-byte aligned)
 *   b    uint8  [N][K]            e4m3 codes, K contiguous ("NT")     (16-byte aligned)
 *   sfb  float  [ceil(N/128)][K/128]  B scales                        (4-byte aligned)
 *   c    bf16   [M][N]            bit patterns; NULL means C = 0; may equal d
 *   d    bf16   [M][N]            output                              (2-byte aligned)
 * K must be a multiple of 128.  The grouped forms add a leading group axis to
 * B and sfb: b [G][N][K], sfb [G][ceil(N/128)][K/128].
 *
 * Calls are asynchronous: they validate their arguments on the host, enqueue
 * one or more kernels on `stream` (a hipStream_t; NULL = the null stream) and
 * return without waiting.  Device-resident control data (grouped_layout,
 * masked_m) is read only by the kernels, so no call synchronises with the
 * device and every call may be captured in a HIP graph once dg_init() has run
 * on the device.  Faults inside a kernel surface at the caller's next
 * synchronisation, as for any HIP kernel.
 *
 * All calls on one device share its workspace (split-K partial tiles, and the
 * scratch of the operators around the products) and its scale-check results,
 * unless their stream has a workspace of its own
 * (dg_bind_stream_workspace).  Calls enqueued on one stream, or ordered across
 * streams by events, are safe; calls that may run at the same time on
 * different streams of one device race on the shared memory and must be
 * ordered by the caller, or given per-stream workspaces.
 *
 * Errors: an invalid argument returns DG_ERR_INVALID_ARG and launches nothing;
 * a shape the kernels do not handle returns DG_ERR_UNSUPPORTED; a failing HIP
 * call returns DG_ERR_HIP.  dg_last_error() then describes the failure (per
 * host thread).  No C++ exception crosses this interface.
 */
#ifndef DG_H
#define DG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DG_OK = 0,
  DG_ERR_INVALID_ARG = -1,
  DG_ERR_UNSUPPORTED = -2,
  DG_ERR_HIP = -3
} dg_status;

/* Dense FP8 GEMM, NT layout: D[M][N] = C + A[M][K] . B[N][K]^T with 1x128 A
 * scales and 128x128 B scales (likun.im section 一 naming: "fp8_gemm_nt";
 * aitangshan.cn usage example: a, a's scales, b, b's scales, c, out).
 * M == 0 or N == 0 is a successful no-op; K == 0 gives D = C.
 * Returns a dg_status. */
int dg_fp8_gemm_nt(const void* a, const float* sfa, const void* b, const float* sfb,
                   const void* c, void* d, int M, int N, int K, void* stream);

/* Dense FP8 GEMM with K-major operands (likun.im section 一: the family
 * fp8_gemm_{nt,nn,tn,tt}; the first letter gives A's storage, the second B's,
 * "n" for A meaning [M][K] and "t" [K][M], "t" for B meaning [N][K] and "n"
 * [K][N]).  Same arithmetic, scales (sfa [K/128][M], sfb [ceil(N/128)][K/128],
 * indexed by the logical row, column and K block whatever the storage), C and
 * D as dg_fp8_gemm_nt:
 *   nn: a [M][K] (K contiguous), b [K][N] (N contiguous)
 *   tn: a [K][M] (M contiguous), b [K][N] (N contiguous)
 *   tt: a [K][M] (M contiguous), b [N][K] (K contiguous)
 * An operand stored [K][M] needs M % 16 == 0, one stored [K][N] needs
 * N % 16 == 0; other sizes return DG_ERR_UNSUPPORTED.  Returns a dg_status. */
int dg_fp8_gemm_nn(const void* a, const float* sfa, const void* b, const float* sfb,
                   const void* c, void* d, int M, int N, int K, void* stream);
int dg_fp8_gemm_tn(const void* a, const float* sfa, const void* b, const float* sfb,
                   const void* c, void* d, int M, int N, int K, void* stream);
int dg_fp8_gemm_tt(const void* a, const float* sfa, const void* b, const float* sfb,
                   const void* c, void* d, int M, int N, int K, void* stream);

/* Dense FP8 x FP4 GEMM, NT layout (likun.im section 一: "fp8_fp4_gemm_nt";
 * section 五: packed UE8M0 scale factors, four to an int; lqnn.cn: the FP8 x
 * FP4 GEMM release):
 *   D[m,n] = bf16_rne( C[m,n] + sum_kb sa[kb][m]
 *            * sum_{k in block kb} A[m,k] * B[n,k] * 2^(e[n][k/32] - 127) )
 *   a    uint8  [M][K]       e4m3 codes (16-byte aligned); sfa float [K/128][M] as in dg_fp8_gemm_nt
 *   b    uint8  [N][K/2]     OCP E2M1 (FP4) codes, two per byte, element 2i in the
 *                            low nibble, K contiguous (16-byte aligned)
 *   sfb  int32  [K/128][N]   E8M0 scale exponents e (value 2^(e-127)), one byte per
 *                            32 K values: byte j of sfb[kb][n] scales K values
 *                            128*kb + 32*j .. +31 of row n (4-byte aligned)
 *   c, d bf16   [M][N]       as in dg_fp8_gemm_nt
 * K must be a multiple of 128.  Runs on the tile kernels (no split-K variant).
 * Returns a dg_status. */
int dg_fp8_fp4_gemm_nt(const void* a, const float* sfa, const void* b, const int32_t* sfb,
                       const void* c, void* d, int M, int N, int K, void* stream);

/* M-grouped GEMM, contiguous layout (likun.im section 二:
 * "m_grouped_..._gemm_nt_contiguous" taking grouped_layout): the rows of every
 * expert are concatenated along M.  grouped_layout is a device int32 array of
 * M entries; row m is computed with expert grouped_layout[m]'s B and sfb.
 * Rows come in aligned blocks of 128 (rows 128*i .. 128*i+127); within one
 * block every row whose id lies in [0, num_groups) must carry the same id.
 * Rows whose id lies outside [0, num_groups) (for example -1 on padding) are
 * not written.  a [M][K], sfa [K/128][M], b [num_groups][N][K],
 * sfb [num_groups][ceil(N/128)][K/128], c and d [M][N].
 * Returns a dg_status. */
int dg_m_grouped_fp8_gemm_nt_contiguous(const void* a, const float* sfa, const void* b,
                                        const float* sfb, const void* c, void* d, int M, int N,
                                        int K, int num_groups, const int32_t* grouped_layout,
                                        void* stream);

/* M-grouped GEMM, masked layout (likun.im section 二:
 * "m_grouped_..._gemm_nt_masked" taking masked_m and expected_m; zwt0204
 * DeepGEMM deep dive: the masked layout serves inference decoding).  Every
 * group g owns max_m rows; only its first min(max(masked_m[g], 0), max_m)
 * rows are computed and written, the others are left untouched.  masked_m is a
 * device int32 array of num_groups entries, read only by the kernel.
 * expected_m is a host-side hint of the typical masked_m; it only steers the
 * launch configuration and never changes which rows are computed.
 * a [G][max_m][K], sfa [G][K/128][max_m], b [G][N][K], sfb [G][ceil(N/128)][K/128],
 * c and d [G][max_m][N].  Returns a dg_status. */
int dg_m_grouped_fp8_gemm_nt_masked(const void* a, const float* sfa, const void* b,
                                    const float* sfb, const void* c, void* d, int max_m, int N,
                                    int K, int num_groups, const int32_t* masked_m,
                                    int expected_m, void* stream);

/* M-grouped FP8 x FP4 GEMMs (likun.im section 二: "m_grouped_fp8_fp4_gemm_nt_contiguous"
 * and "..._masked"): as dg_m_grouped_fp8_gemm_nt_contiguous / _masked with the
 * FP4 B of dg_fp8_fp4_gemm_nt per group: b uint8 [G][N][K/2] (packed E2M1),
 * sfb int32 [G][K/128][N] (four E8M0 exponents per int).  A, sfa, C, D,
 * grouped_layout, masked_m and expected_m exactly as in the FP8 forms.
 * Returns a dg_status. */
int dg_m_grouped_fp8_fp4_gemm_nt_contiguous(const void* a, const float* sfa, const void* b,
                                            const int32_t* sfb, const void* c, void* d, int M, int N,
                                            int K, int num_groups, const int32_t* grouped_layout,
                                            void* stream);
int dg_m_grouped_fp8_fp4_gemm_nt_masked(const void* a, const float* sfa, const void* b,
                                        const int32_t* sfb, const void* c, void* d, int max_m, int N,
                                        int K, int num_groups, const int32_t* masked_m,
                                        int expected_m, void* stream);

/* K-grouped GEMM, TN layout, for MoE weight gradients (likun.im section 一:
 * "k_grouped_fp8_gemm_tn", grouped along K for the MoE backward pass; section
 * 二: the call takes the per-group K sizes ks and the (1, 1, 128) scale
 * recipe).  Group g owns K rows k_start[g] .. k_start[g] + ks[g] - 1 of both
 * operands (k_start = running sum of ks), i.e. its tokens, and
 *   D[g][m][n] = C[g][m][n] + sum_kb sfa[kb][m] * sfb[kb][n]
 *                             * sum_{k in block kb} A[k][m] * B[k][n]
 * over the group's 128-row K blocks, accumulated in fp32 and stored in fp32.
 *   a    uint8  [K][M]   e4m3 codes, M contiguous (16-byte aligned)
 *   sfa  float  [K/128][M]   one scale per column per 128 K rows
 *   b    uint8  [K][N]   e4m3 codes, N contiguous (16-byte aligned)
 *   sfb  float  [K/128][N]   one scale per column per 128 K rows
 *   c    float  [G][M][N] or NULL (C = 0); may equal d (accumulation)
 *   d    float  [G][M][N] output (a group with ks[g] == 0 gets C, or zeros)
 *   ks   int32  [num_groups] on the HOST: each a non-negative multiple of 128
 *        (pad a group's tokens with zero rows); K = sum of ks.
 * M and N must be multiples of 16 and num_groups at most 256
 * (DG_ERR_UNSUPPORTED otherwise).  The K offsets travel in the launch's
 * arguments, so a captured graph replays the call with the ks it was captured
 * with.  Returns a dg_status. */
int dg_k_grouped_fp8_gemm_tn_contiguous(const void* a, const float* sfa, const void* b,
                                        const float* sfb, const float* c, float* d, int M, int N,
                                        int num_groups, const int32_t* ks, void* stream);

/* dg_fp8_gemm_nt without any device allocation, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation.  Same arguments, arithmetic, layouts and
 * errors as dg_fp8_gemm_nt.  Its kernels' scratch (split-K partial tiles and
 * scale-check verdicts) is a fixed 8 MiB device array per GPU, part of the
 * library's code object and held until the process ends; the call allocates
 * nothing, neither on its first use on a device nor later.  The kernel
 * configuration is chosen so that its partials fit the array; one forced
 * beyond it (DG_FORCE_SPLITS) returns DG_ERR_UNSUPPORTED.  Every call on a GPU
 * shares that GPU's array, and nothing in it needs clearing between calls
 * (every call writes what it reads; the one-launch decode configuration's
 * per-tile counters in it start at zero with the array and every call leaves
 * them at zero), but calls that may overlap on one GPU (different streams not
 * ordered by events) race on it and must be ordered by the caller.  Returns a
 * dg_status. */
int dg_fp8_gemm_nt_noalloc(const void* a, const float* sfa, const void* b, const float* sfb,
                           const void* c, void* d, int M, int N, int K, void* stream);

/* The kernel configuration the calls above would choose, as a host-side query
 * that touches no device (for tests and for callers that want to know what
 * runs).  form: 0 dense (any operand storage), 1 contiguous, 2 masked.  rows:
 * M for dense and contiguous calls, expected_m for masked ones.  ab_layout:
 * 0 nt, 1 tt (A stored [K][M]), 2 nn (B stored [K][N]), 3 tn, 4 FP4 B.
 * num_cus: the device's compute units (256 on MI355X).  has_c: nonzero when
 * the call passes a C.  Writes the configuration id to *cfg (0 128x128 tile,
 * 1 decode kernel with K split over workgroups, 2 128x64, 3 64x128, 4 128x128
 * two per CU, 5 256x128, 6 128x256, 7 and 8 128x256 and 10 256x256 with
 * power-of-two scales in the MFMA, 9 narrow 16x48 whole-K, 11 256x256, 12 the
 * decode kernel with its splits summed inside the same launch) and
 * the decode kernel's K splits to *splits (1 otherwise).  DG_FORCE_CONFIG and
 * DG_FORCE_SPLITS act as they do on the calls.  Returns DG_ERR_INVALID_ARG
 * for NULL outputs, a form outside 0-2, rows or N below 1, K negative or not
 * a multiple of 128, num_groups below 1, num_cus below 8 or ab_layout
 * outside 0-4; DG_OK otherwise. */
int dg_choose_config(int form, int rows, int N, int K, int num_groups, int num_cus, int ab_layout,
                     int has_c, int* cfg, int* splits);

/* Binds a caller-owned device workspace to a stream of the current device:
 * every later call of this library enqueued on that stream uses it in place of
 * the device's shared workspace (split-K partial tiles and scale-check
 * verdicts; and what the operators around the products put there: the layouts'
 * counts, the scatters' block maxima, the adapters' lists and partial sums, the
 * lists of the 4-bit products by choice, the balance loss's and the norm's partial
 * sums), so that calls running at the same time on different streams no longer share
 * scratch memory. workspace: device memory on the current device, 256-byte
 * aligned, at least 256 bytes (the verdicts). A workspace of at least 256 +
 * 4096 bytes also holds, after the verdicts, the 4096 bytes of counters of the
 * one-launch decode configuration, which this call clears (synchronously) and
 * every later call leaves at zero; the rest holds partials, and the
 * configuration is chosen so that they fit (a bound workspace of a few hundred
 * bytes simply means no split-K, and one launch for a layout or a scatter; the
 * adapters refuse one without room for 16 tokens). The caller keeps the memory
 * alive, and unused by anything else, while the binding lasts and while calls
 * enqueued with it run. workspace NULL (or bytes 0) removes the stream's
 * binding. The allocation-free call (dg_fp8_gemm_nt_noalloc) always uses its
 * own fixed array. Returns DG_ERR_INVALID_ARG for a misaligned or too small
 * workspace, DG_ERR_HIP if the current device cannot be queried or the counters
 * cannot be cleared. */
int dg_bind_stream_workspace(void* stream, void* workspace, size_t bytes);

/* Host-side check of a contiguous grouped_layout held in HOST memory (M int32
 * entries) against the contract of the contiguous calls: within every aligned
 * block of 128 rows, all rows whose id lies in [0, num_groups) carry the same
 * id.  Returns DG_OK, or DG_ERR_INVALID_ARG with dg_last_error() naming the
 * first offending block.  Touches no device.
 *
 * Debug mode: with the environment variable DG_VALIDATE=1, the M-grouped calls
 * copy their device-resident grouped_layout (or masked_m) to the host on the
 * call's stream, wait for it, and apply this check (masked: every masked_m[g]
 * within [0, max_m], which the kernels would otherwise clamp) before launching
 * anything; a violation returns DG_ERR_INVALID_ARG.  It synchronises, so it is
 * for debugging only, and it is skipped while the stream is being captured. */
int dg_check_grouped_layout(const int32_t* grouped_layout, int M, int num_groups);

/* ---- The operators around the products --------------------------------------
 *
 * A router chooses each token's experts, the layout calls give every choice a
 * row of the M-grouped (or K-grouped) products, the scatter calls move and
 * quantise the tokens' rows there, the gather call sums the experts' results
 * back per token, and the adapter call adds low-rank terms to (or ahead of) a
 * dense projection.  Beside them stand the router's balance loss, products of a
 * few tokens with 4-bit weights, and the norm and clipping of the gradients.  They
 * follow the rules above: device pointers owned by the
 * caller, checks on the host, no synchronisation, capturable in a HIP graph
 * after dg_init(), and the device's (or the stream's bound) workspace as
 * scratch where a call says so.  An array of no elements may be NULL.  T * top_k
 * at most 2^30 in all calls but the router's.
 *
 * Sums, softmax statistics and scales are fp32; bf16 results are rounded once
 * (to nearest, ties to even).  No result depends on the order of atomics. */

typedef enum { DG_F32 = 0, DG_BF16 = 1 } dg_dtype;
typedef enum { DG_SCORE_SOFTMAX = 0, DG_SCORE_SIGMOID = 1 } dg_score;

/* Routing: for every token the top_k of num_experts by
 *   key[e] = s[e] + bias[e],   s = softmax(logits) over the experts or sigmoid(logits),
 * and their weights scale * s[e], divided by the sum of the chosen s if
 * renormalize is nonzero (bias steers the choice only).  With num_groups > 1 the
 * experts are num_groups equal runs; a group's score is the sum of its
 * group_top (1 or 2) highest keys, and only the topk_groups highest groups'
 * experts can be chosen.  Equal keys, and equal group scores, go to the lowest
 * index; chosen experts come in falling order of key.
 *   logits  logits_type [T][E]   DG_F32 or DG_BF16
 *   bias    float [E] or NULL
 *   topk_ids int32 [T][top_k], topk_weights float [T][top_k]   outputs
 * An expert whose logit or key is -inf or NaN is masked: it is never chosen (a
 * masked logit adds nothing to the softmax either, and masked experts add
 * nothing to a group's score).  A token with fewer than top_k experts left gets
 * id -1 and weight 0 in its last slots.  A logit of +inf counts as the largest
 * finite value.  Scores are fp32 values down to the subnormal ones: those below
 * 2^-149 (a sigmoid's from a logit of about -104 down) are 0, and chosen scores
 * that sum to zero give weights of zero under renormalize.  E at most 1024,
 * top_k at most 64, num_groups at most 64 (DG_ERR_UNSUPPORTED otherwise); top_k
 * <= topk_groups * E / num_groups.
 * Returns a dg_status. */
int dg_route_topk(const void* logits, int logits_type, const float* bias, int32_t* topk_ids, float* topk_weights,
                  int T, int E, int top_k, int score, int num_groups, int topk_groups, int group_top,
                  int renormalize, float scale, void* stream);

/* Gradient of the routing weights with respect to the logits, for the choice
 * made in the forward pass (ids are constants; a token's ids are distinct, and
 * one outside [0, E) takes no part):
 *   grad_logits[t][i] = sum_j grad_weights[t][j] * d topk_weights[t][j] / d logits[t][i]
 *   logits, grad_logits  logits_type [T][E]; topk_ids int32 [T][top_k];
 *   grad_weights float [T][top_k]
 * A masked expert's gradient is 0.  Returns a dg_status. */
int dg_route_topk_backward(const void* logits, int logits_type, const int32_t* topk_ids, const float* grad_weights,
                           void* grad_logits, int T, int E, int top_k, int score, int renormalize, float scale,
                           void* stream);

/* The most rows that the contiguous layout of `choices` = T * top_k choices can
 * need over num_groups experts: every expert's rows rounded up to 128.  Host
 * only.  Returns -1 for a negative argument or a result beyond 2^31 - 1. */
int dg_m_grouped_rows_bound(long long choices, int num_groups);

/* Rows for the contiguous products.  The choices topk_ids [T][top_k] whose
 * expert lies in [first_expert, first_expert + num_groups) are this GPU's; choice
 * i = t * top_k + j of local expert g gets the next row of g's segment, in the
 * order of i, and the segments follow one another by g, each starting at a
 * multiple of 128.
 *   grouped_layout int32 [M]   local expert of each row, -1 for rows without one
 *   row_of   int32 [T][top_k]  each choice's row, -1 without one
 *   slot_of  int32 [M]         each row's choice i, -1 without one
 *   counts   int32 [num_groups]  choices per local expert, or NULL
 * M (a multiple of 128) is the room there is: dg_m_grouped_rows_bound() rows
 * always suffice; choices whose row would lie beyond M have none (row_of -1),
 * and counts still counts them.  num_groups at most 1024.  Scratch: workspace
 * (a small one costs speed only).  Returns a dg_status. */
int dg_m_grouped_layout_contiguous(const int32_t* topk_ids, int T, int top_k, int first_expert, int num_groups, int M,
                                   int32_t* grouped_layout, int32_t* row_of, int32_t* slot_of, int32_t* counts,
                                   void* stream);

/* Rows for the masked products: choice i of local expert g gets row
 * g * max_m + r with r counting g's choices in the order of i; choices beyond
 * max_m have none.
 *   masked_m int32 [num_groups]  min(choices, max_m) per local expert
 *   row_of   int32 [T][top_k], slot_of int32 [num_groups][max_m]   as above
 * num_groups at most 1024.  Scratch: workspace (a small one costs speed only).
 * Returns a dg_status. */
int dg_m_grouped_layout_masked(const int32_t* topk_ids, int T, int top_k, int first_expert, int num_groups, int max_m,
                               int32_t* masked_m, int32_t* row_of, int32_t* slot_of, void* stream);

/* Moves the tokens' rows to the experts' rows, quantised to e4m3 with one scale
 * per row per 128 values: for every choice i = t * top_k + j with row r = row_of[i],
 *   v = weights[i] * x[t] (x[t] without weights),  sf = max(amax, 2^-100) / 448
 *   with amax = max |v| over the block (sf = 1 if amax = 0; with pow2_scales
 *   rounded up to a power of two),  a[r] = e4m3_rne(v / sf),
 * worked out to more than fp32 precision; sf is then rounded to fp32 (an infinity
 * beyond its range) and the quotient to fp32 and from there to e4m3, both to
 * nearest even: a quotient within 2^-25 of itself of a value halfway between two
 * codes counts as that value.
 *   x        bf16  [T][K] (16-byte aligned)
 *   weights  float [T][top_k] or NULL
 *   row_of, slot_of   the maps of the layout call; entries outside the range of
 *            rows or choices are skipped
 *   contiguous: a uint8 [M][K], sfa float [K/128][M], slot_of [M]
 *   masked:     a uint8 [G][max_m][K], sfa float [G][K/128][max_m], slot_of [G][max_m]
 * Rows without a choice are left as they are.  A NaN in v gives a NaN code and
 * does not count for amax; an infinity gives its block an infinite scale and a
 * NaN code in its own place.  K must be a multiple of 128.  Scratch: workspace.
 * Returns a dg_status. */
int dg_m_grouped_scatter_fp8_contiguous(const void* x, const float* weights, const int32_t* row_of,
                                        const int32_t* slot_of, void* a, float* sfa, int T, int top_k, int M, int K,
                                        int pow2_scales, void* stream);
int dg_m_grouped_scatter_fp8_masked(const void* x, const float* weights, const int32_t* row_of,
                                    const int32_t* slot_of, void* a, float* sfa, int T, int top_k, int num_groups,
                                    int max_m, int K, int pow2_scales, void* stream);

/* The same rows as an operand of the K-grouped product: one scale per column per
 * 128 rows, and rows without a choice are zeros (128 such rows have scale 1).
 *   x bf16 [T][N] (16-byte aligned), weights float [T][top_k] or NULL,
 *   slot_of int32 [K], a uint8 [K][N] (16-byte aligned), sfa float [K/128][N]
 * K (the rows, a multiple of 128) may be less than the layout's M: the segments
 * used.  N must be a multiple of 16 and N below 2^30 (DG_ERR_UNSUPPORTED
 * otherwise).  Returns a dg_status. */
int dg_k_grouped_scatter_fp8(const void* x, const float* weights, const int32_t* slot_of, void* a, float* sfa, int T,
                             int top_k, int K, int N, int pow2_scales, void* stream);

/* The experts' rows back to the tokens:
 *   d[t] = bf16_rne( c[t] + sum_j weights[t][j] * rows[row_of[t][j]] )
 * summed in fp32 from j = 0 on, weights NULL meaning 1; a row_of outside [0, M)
 * adds nothing, whatever its weight.  Without weights it is also the gradient
 * of the scatter, and the scatter with weights is the gradient of this with
 * respect to rows.
 *   rows bf16 [M][N] (the masked form's [G][max_m][N] with M = G * max_m),
 *   row_of int32 [T][top_k], weights float [T][top_k] or NULL,
 *   c bf16 [T][N] or NULL (may equal d), d bf16 [T][N]
 * N at most 2^30, odd ones too; top_k at most 64 (DG_ERR_UNSUPPORTED otherwise).
 * Returns a dg_status. */
int dg_m_grouped_gather(const void* rows, const int32_t* row_of, const float* weights, const void* c, void* d, int T,
                        int top_k, int M, int N, void* stream);

/* Gradient of the gather with respect to its weights:
 *   grad_weights[t][j] = sum_n grad_d[t][n] * rows[row_of[t][j]][n]   (0 without a row)
 *   rows bf16 [M][N], grad_d bf16 [T][N], grad_weights float [T][top_k]
 * N at most 2^30, top_k at most 64.  Returns a dg_status. */
int dg_m_grouped_gather_weight_grad(const void* rows, const int32_t* row_of, const void* grad_d, float* grad_weights,
                                    int T, int top_k, int M, int N, void* stream);

/* Low-rank adapters of many requests beside a shared projection:
 *   d[t] = bf16_rne( c[t] + scales[i] * B[i] . (A[i] . x[t]) ),   i = adapter_ids[t]
 * A token whose id lies outside [0, num_adapters) has no adapter: d[t] = c[t].
 * With c the projection's result it completes it; with c NULL its d is the C of
 * the dense call.
 *   x  bf16 [T] rows of K values, ldx apart (16-byte aligned, ldx % 8 == 0)
 *   a  bf16 [num_adapters][R][K], b bf16 [num_adapters][N][R] (16-byte aligned)
 *   scales float [num_adapters] or NULL (1), adapter_ids int32 [T]
 *   c  bf16 [T] rows of N values, ldc apart, or NULL (0); may equal d
 *   d  bf16 [T] rows of N values, ldd apart
 * A . x is summed, scaled and multiplied with B in fp32.  K must be a
 * multiple of 128, R a multiple of 8 and at most 256 (adapters of lower rank are
 * filled up with zeros), N at most 16776960, odd ones too, num_adapters at most
 * 1024 (DG_ERR_UNSUPPORTED otherwise).  Scratch: workspace (DG_ERR_UNSUPPORTED if
 * a bound one has no room for 16 tokens).  Returns a dg_status. */
int dg_lora_bf16_nt(const void* x, int ldx, const void* a, const void* b, const float* scales,
                    const int32_t* adapter_ids, const void* c, int ldc, void* d, int ldd, int T, int N, int K, int R,
                    int num_adapters, void* stream);

/* The router's balance loss and the experts' counts.  The tokens are num_seqs
 * sequences, one behind the other: sequence s has the n_s tokens from
 * seq_starts[s] to seq_starts[s+1] - 1, and with p[t] = softmax(logits[t]) or
 * sigmoid(logits[t]) divided by the sum of the token's sigmoids
 *   counts[s][e] = choices of e among the sequence's topk_ids
 *   loss[s] = scale * E / (top_k * n_s^2) * sum_e counts[s][e] * sum_{t in s} p[t][e]
 * which is scale where every expert has the same share (0 for a sequence of no
 * tokens).
 *   logits  logits_type [T][E]; topk_ids int32 [T][top_k], ids outside [0, E) are
 *           not counted
 *   seq_starts int32 [num_seqs + 1], rising (not necessarily strictly), or NULL
 *           with num_seqs 1: all tokens.  Tokens before seq_starts[0] and from
 *           seq_starts[num_seqs] on (padding) take no part.  Entries outside
 *           [0, T] count as 0 or T
 *   loss float [num_seqs], counts int32 [num_seqs][E]   outputs
 * A logit of -inf or NaN is a masked expert's: its share is 0.  A token of masked
 * experts only has no shares, but counts in n_s.  +inf counts as the largest
 * finite value.  Sigmoids keep their shares however far below zero all of a
 * token's logits lie; shares below 2^-126 are 0.  Shares are fp32 and summed in
 * fp32 over stretches of tokens, two per CU (a small bound workspace makes them
 * longer), and those sums and the loss in fp64: with 256 CUs and the device's
 * workspace a loss is off by less than (E + 160 + T / 4096) * 2^-24 of itself.
 * E at most 1024, top_k at most 64, T * top_k at most 2^30 (DG_ERR_UNSUPPORTED
 * otherwise).  Scratch: workspace (DG_ERR_UNSUPPORTED if a bound one has no room
 * for 16 bytes per expert, their number rounded up to a multiple of 4).  Returns a
 * dg_status. */
int dg_route_balance(const void* logits, int logits_type, const int32_t* topk_ids, const int32_t* seq_starts,
                     float* loss, int32_t* counts, int T, int E, int top_k, int num_seqs, int score, float scale,
                     void* stream);

/* Gradient of the balance loss with respect to the logits, for the forward call's
 * counts (constants: a choice has no gradient):
 *   grad_logits[t][i] = c[t][i] + grad_loss[s] * d loss[s] / d logits[t][i]
 *   logits, c, grad_logits  logits_type [T][E]; c NULL means 0 and may equal
 *           grad_logits: the gradient of the routing weights, to which this is added
 *   grad_loss float [num_seqs] or NULL (ones); counts, seq_starts as above
 * A masked expert and a token of no sequence get c.  One rounding to logits_type.
 * Returns a dg_status. */
int dg_route_balance_backward(const void* logits, int logits_type, const int32_t* counts, const int32_t* seq_starts,
                              const float* grad_loss, const void* c, void* grad_logits, int T, int E, int top_k,
                              int num_seqs, int score, float scale, void* stream);

/* Products of a few tokens with 4-bit weights and unquantised activations:
 *   d[m][n] = bf16_rne( c[m][n] + sum_k x[m][k] * w[n][k] )
 * for the tokens of a decoding step, where reading the weights is all the time.
 * The FP4 form takes the weights of dg_fp8_fp4_gemm_nt as they are stored:
 *   w[n][k] = e2m1(b[n][k]) * 2^(e[n][k/32] - 127), as a bf16 value: exact, but
 *           an infinity from 2^128 on; a NaN where e = 255
 *   b uint8 [N][K/2] (16-byte aligned), sfb int32 [K/128][N] (4-byte aligned)
 * the integer form groups of group_size (32, 64 or 128) values along K:
 *   w[n][k] = (q[n][k] - zeros[k/group_size][n]) * scales[k/group_size][n]
 *   b uint8 [N][K/2], two q of 0 to 15 per byte, element 2i in the low nibble
 *           (16-byte aligned)
 *   scales scales_type [K/group_size][N]  DG_F32 or DG_BF16
 *   zeros uint8 [K/group_size][N] or NULL: 8
 * A group's sum of x * q and its sum of x are fp32 sums, scaled and joined in fp32:
 * both sums, and a scale times its zero point, have to stay within fp32's range
 * (the sums do where x is below 2^117 in magnitude), and the result's error is
 * measured by magnitudes of (q + zero) * scale * x.
 *   x  bf16 [M] rows of K values, ldx apart (16-byte aligned, ldx % 8 == 0)
 *   c  bf16 [M] rows of N values, ldc apart, or NULL (0); may equal d
 *   d  bf16 [M] rows of N values, ldd apart
 * x is finite in the integer form (an infinity makes its token's results NaN).  K
 * must be a multiple of 128 and at most 2^24, N at most 2^20, odd ones too
 * (DG_ERR_UNSUPPORTED otherwise).  Any M, in tiles of 4, 8 or 16 tokens (up to 4, up
 * to 8 and more in all) that each read the weights: many tokens take less time in the
 * FP8 products.  Returns a dg_status. */
int dg_bf16_fp4_gemv_nt(const void* x, int ldx, const void* b, const int32_t* sfb, const void* c, int ldc, void* d,
                        int ldd, int M, int N, int K, void* stream);
int dg_bf16_int4_gemv_nt(const void* x, int ldx, const void* b, const void* scales, int scales_type, const void* zeros,
                         int group_size, const void* c, int ldc, void* d, int ldd, int M, int N, int K, void* stream);

/* The same with the experts of every choice, straight from the router's ids: no
 * layout, no rows moved, an expert's weights read once for its choices (4, 8 or 16
 * at a time, by T as by M above).  Choice i = t * top_k + j of expert e = topk_ids[t][j], local expert
 * g = e - first_expert in [0, num_groups):
 *   d[i][n] = bf16_rne( c[i][n] + sum_k x[row][k] * w[g][n][k] )
 *   x  rows of K values as above: x_rows = T, a token's choices sharing row t, or
 *      x_rows = T * top_k, row i each (the experts' way back down)
 *   b, sfb, scales, zeros  as above with a leading axis [num_groups]
 *   c, d  rows of N values for T * top_k choices, as above
 * A choice whose expert is not here gets c (zeros without one), so that a gather
 * with row_of[t][j] = t * top_k + j sums what this GPU's experts give.  num_groups
 * at most 1024, T * top_k at most 2^30.  Scratch: workspace (lists, from 1025
 * choices on; a small one costs speed only).  Returns a dg_status. */
int dg_m_grouped_bf16_fp4_gemv_nt_topk(const void* x, int ldx, int x_rows, const int32_t* topk_ids, const void* b,
                                       const int32_t* sfb, const void* c, int ldc, void* d, int ldd, int T, int top_k,
                                       int first_expert, int num_groups, int N, int K, void* stream);
int dg_m_grouped_bf16_int4_gemv_nt_topk(const void* x, int ldx, int x_rows, const int32_t* topk_ids, const void* b,
                                        const void* scales, int scales_type, const void* zeros, int group_size,
                                        const void* c, int ldc, void* d, int ldd, int T, int top_k, int first_expert,
                                        int num_groups, int N, int K, void* stream);

/* The norm of all gradients together, such as the K-grouped product's and the
 * others of a training step:
 *   norm[0] = sqrt( sum over all tensors and elements of grads[i][j]^2 )
 * Squares and sums are fp64; the result is rounded to fp32.
 *   grads  num_tensors addresses, types their dg_dtypes, sizes their elements:
 *          arrays on the HOST, read during the call (they travel in the launches'
 *          arguments: a captured graph replays with the tensors of the captured
 *          call).  Each tensor is contiguous and aligned to its type; one of size
 *          0 may be NULL
 *   norm float [1]   output
 * No tensors have a norm of 0.  num_tensors at most 2^20, a tensor at most 2^43
 * elements (DG_ERR_UNSUPPORTED otherwise).  Scratch: workspace (8 bytes per 120
 * tensors at the least, DG_ERR_UNSUPPORTED if a bound one has less).  Returns a
 * dg_status. */
int dg_grad_norm(const void* const* grads, const int* types, const long long* sizes, int num_tensors, float* norm,
                 void* stream);

/* The gradients scaled so that their norm is at most max_norm:
 *   out[i][j] = grads[i][j] * f,   f = min(1, max_norm / (norm[0] + 1e-6))
 * f and the products in fp32, those of bf16 tensors rounded once more to bf16.  norm
 * is read by the kernels only, so that a job may sum the squares of several GPUs in
 * between.  A NaN norm makes f NaN, an infinite one 0.
 *   grads, types, sizes as above; out num_tensors addresses on the HOST: each may
 *   equal grads[i], and otherwise shares no memory with any tensor or with norm
 *   (DG_ERR_INVALID_ARG otherwise).  max_norm must not be negative.
 * Returns a dg_status. */
int dg_grad_clip(const void* const* grads, void* const* out, const int* types, const long long* sizes,
                 int num_tensors, const float* norm, float max_norm, void* stream);

/* Prepares per-device state for the current HIP device (device properties and
 * the split-K workspace, allocated once and kept until the process ends).
 * Calls above do this lazily on first use; call dg_init() first when the
 * first call would otherwise happen inside HIP graph capture.
 * Returns a dg_status. */
int dg_init(void);

/* Message describing the last non-DG_OK status returned on this host thread
 * (empty string if none).  The pointer stays valid until the next call on
 * this thread. */
const char* dg_last_error(void);

/* Library version as major*10000 + minor*100 + patch. */
int dg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DG_H */

/*
 * fp8bs.h -- C ABI of the MI355X (gfx950) block-scaled FP8 W8A8 GEMM library.
 *
 * The method: activations are quantized per token in 1x128 groups to OCP e4m3
 * with power-of-two (UE8M0) scales packed four to a 32-bit word; weights are
 * e4m3 with one scale per 128x128 block; the GEMM accumulates in fp32, applying
 * the two scales to each 128-wide K-block before adding it, and writes bf16.
 * Sources: vLLM DeepGEMM FP8 block GEMM benchmark post (sections 4.1-4.2:
 * quantization layouts, the three dense GEMM calls and their preconditions);
 * vLLM PR #29546 "Deepgemm fused layout kernel for activations" (quant with the
 * uint32 scale pack fused in); vLLM PR #19885 "Optimize the little operations
 * in the DeepGEMM + DeepEP low latency case" (fused SiLU-mul-quant that skips
 * padded tokens); vLLM PR #19111 "Integrate batched/masked deepgemm kernel"
 * (masked grouped GEMM over [experts, max_tokens, K] with per-expert counts).
 *
 * Conventions shared by every entry point
 *   - Data pointers are DEVICE pointers owned by the caller.  bf16 is passed as
 *     its 16-bit pattern, e4m3 as bytes (OCP E4M3FN, max 448).
 *   - stream is a hipStream_t passed as void* (NULL = the default stream).  Every
 *     call is asynchronous and stream-ordered; nothing reads device data on the
 *     host, so masked counts never leave the device.  Several host threads may call on
 *     one stream: the launches of a call that uses the stream's workspace stay together.
 *   - Return value: FP8BS_OK (0) or a negative status; on error nothing is
 *     launched.  fp8bs_status_string() names a status; after FP8BS_ERR_LAUNCH,
 *     fp8bs_last_hip_error() gives the hipError_t of the failed call (per thread).
 *   - Sizes of zero are a successful no-op, except K (see each call).
 *   - Outputs must not overlap inputs.
 *   - Alignment: every data pointer and every row of an e4m3/bf16 tensor must be
 *     16-byte aligned (FP8BS_ERR_ALIGN otherwise); scale pointers 4-byte aligned.
 *   - The device must be gfx950 (FP8BS_ERR_DEVICE otherwise).
 *
 * Packed activation-scale layout ("sf"): for K columns there are G = K/128 groups
 * per row and W = ceil(G/4) words per row.  Group g's exponent byte (e + 127,
 * where the group's scale is 2^e) sits in bits 8*(g%4)..8*(g%4)+7 of word g/4;
 * bytes of groups past G are zero.  Words are stored M-major: word w of row r is
 * sf[w*ld_sf + r] (the column-major, padded layout the benchmark post's section
 * 4.1 describes for DeepGEMM; ld_sf = round_up(M, 4) gives 16-byte columns).
 * Weight block scales ("sfb") are fp32 [ceil(N/128)][K/128], row-major: the
 * UE8M0 values the weight block quant produces (powers of two).  Every UE8M0 entry
 * point, whatever kernel it picks, reads only each scale's exponent field, i.e.
 * uses 2^floor(log2 |s|): a power of two is used as it is, any other finite scale
 * is taken as the power of two at or below its magnitude (sign and mantissa bits
 * ignored).  The float-scale entry points (fp8_block_gemm_nt_float_scales...) use
 * the whole fp32 value.
 */
#ifndef FP8BS_H
#define FP8BS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  FP8BS_OK = 0,
  FP8BS_ERR_NULL = -1,   /* a required pointer is NULL                              */
  FP8BS_ERR_SHAPE = -2,  /* a size or leading dimension is out of its allowed range */
  FP8BS_ERR_ALIGN = -3,  /* a pointer or row stride breaks the alignment rule       */
  FP8BS_ERR_DEVICE = -4, /* the current device is not gfx950                        */
  FP8BS_ERR_LAUNCH = -5, /* a HIP call failed; see fp8bs_last_hip_error()           */
  FP8BS_ERR_ALLOC = -6,  /* the split-K workspace could not be allocated            */
  FP8BS_ERR_SCRATCH = -7 /* a ..._noalloc entry point: scratch too small             */
};

/*
 * Per-token 1x128 group quant with the UE8M0 scale pack in the same pass
 * (PR #29546, Purpose; benchmark post section 4.1, per_token_group_quant with
 * column-major, aligned scales).  For every row r < M and group g:
 *   e = smallest integer with 448 * 2^e >= max(amax of the group, 1e-10),
 *   q[r][k] = e4m3_rne_saturating(x[r][k] * 2^-e),  byte e + 127 into sf.
 *   x   : bf16 [M][ldx], ldx >= K
 *   q   : e4m3 [M][ldq], ldq >= K, ldq % 16 == 0
 *   sf  : uint32 [ceil(K/512)][ld_sf], ld_sf >= M; entries of rows >= M untouched
 *   K % 128 == 0.
 */
int fp8_quant_group_pack(const void* x, int64_t ldx, int64_t M, int64_t K,
                         void* q, int64_t ldq, uint32_t* sf, int64_t ld_sf, void* stream);

/*
 * Fused SiLU-and-mul + the quant/pack above over a masked expert batch
 * (PR #19885, Summary item 2: outputs in the GEMM's layout, padded tokens
 * neither loaded nor computed).  For e < E and r < clamp(masked_m[e], 0, M_max):
 *   y = silu(gate) * up = gate / (1 + exp(-gate)) * up, in fp32, with gate =
 *   x[e][r][0:H] and up = x[e][r][H:2H]; then 1x128 quant/pack of y.
 *   x        : bf16 [E][M_max][2H] contiguous
 *   masked_m : int32 [E] on the device (clamped to [0, M_max] in the kernel)
 *   q        : e4m3 [E][M_max][H] contiguous
 *   sf       : uint32 [E][ceil(H/512)][M_max] contiguous
 *   H % 128 == 0.  Rows r >= count of q and sf are left untouched.
 */
int silu_mul_quant_group_pack(const void* x, const int32_t* masked_m, int64_t E, int64_t M_max,
                              int64_t H, void* q, uint32_t* sf, void* stream);

/*
 * Float-scale (non-UE8M0) format (benchmark post section 4.1: the scale of a
 * group or block is amax / fp8_max, rounded up to a power of two only when UE8M0
 * is asked for).  In IEEE fp32 with correctly rounded division:
 *   s = max(amax, 1e-10f) / 448,  q = e4m3_rne(clamp(x / s, -448, 448)).
 * fp8_quant_group_float: 1x128 groups of bf16 x [M][ldx] (ldx >= K, ldx % 8 == 0)
 *   -> q e4m3 [M][ldq] (ldq % 16 == 0), sf fp32 [K/128][ld_sf], ld_sf >= M
 *   (one float per group, M-major; entries of rows >= M untouched).
 * fp8_block_quant_128x128_float: 128x128 blocks of bf16 w [N][K] -> q e4m3 [N][K],
 *   sfb fp32 [ceil(N/128)][K/128].
 * fp8_block_gemm_nt_float_scales: C[m][n] = bf16( sum over K-blocks kb of
 *   sfa[kb][m] * sfb[n/128][kb] * (e4m3 dot product of the block) ), fp32
 *   accumulation; sfa fp32 [K/128][ld_sfa], ld_sfa >= M; other arguments and
 *   preconditions as fp8_block_gemm_nt (the scales may be any finite fp32).
 */
int fp8_quant_group_float(const void* x, int64_t ldx, int64_t M, int64_t K, void* q, int64_t ldq,
                          float* sf, int64_t ld_sf, void* stream);
int fp8_block_quant_128x128_float(const void* w, int64_t N, int64_t K, void* q, float* sfb,
                                  void* stream);
/*
 * fp8_block_gemm_nt_float_scales with the weights b in the layout of
 * fp8_weight_preshuffle (rows = N); every other argument and the result are those of
 * fp8_block_gemm_nt_float_scales.  Runs the float-scale decode kernel at every M:
 * meant for decode-sized M (M <= 64).
 */
int fp8_block_gemm_nt_float_scales_preshuffled(const void* a, const float* sfa, int64_t ld_sfa,
                                                const void* b, const float* sfb, void* c, int64_t ldc,
                                                int64_t M, int64_t N, int64_t K, void* stream);
int fp8_block_gemm_nt_float_scales(const void* a, const float* sfa, int64_t ld_sfa, const void* b,
                                   const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N,
                                   int64_t K, void* stream);

/*
 * Per-token group quant written into the masked expert layout of the routed
 * tokens: the quantization half of FP8 dispatch on one GPU (PR #19885, Summary
 * item 1: DeepEP quantizes and puts the scales in DeepGEMM's layout; PR #19111
 * review: the TODO asking for a batched quant).  Token t's choice j routes pair
 * p = t * topk + j to expert topk_ids[p]; its slot is the number of earlier pairs
 * (in p order) routed to the same expert.  Pairs whose id is outside [0, E) or
 * whose slot reaches M_max get slot -1 and are not written.  Every token is
 * quantized once, exactly as fp8_quant_group_pack quantizes a row, and its e4m3
 * row and scale words are written to row `slot` of its expert.
 *   x        : bf16 [T][ldx], ldx >= K, ldx % 8 == 0;  K % 128 == 0
 *   topk_ids : int32 [T][topk] on the device, 1 <= topk <= 64
 *   q        : e4m3 [E][M_max][K];   sf : uint32 [E][ceil(K/512)][M_max]
 *   masked_m : int32 [E] out: min(pairs routed to e, M_max)
 *   slot_of  : int32 [T][topk] out: the slot of every pair, or -1
 *   1 <= E <= 1024.  Rows at or past masked_m[e] of q and sf are left untouched.
 * Two launches on `stream`: one workgroup per 1024 pairs ranks the pairs, then the
 * quantization resolves the slots (deterministic) and reads every token once.  The
 * ranks and per-chunk counts (4 * (T * topk + ceil(T * topk / 1024) * E) bytes) go
 * to the library's per-(device, stream) workspace, allocated on the first call
 * that needs it (FP8BS_ERR_ALLOC during HIP graph capture, as for the GEMMs).
 */
int fp8_quant_group_pack_to_experts(const void* x, int64_t ldx, int64_t T, int64_t K,
                                    const int32_t* topk_ids, int32_t topk, int64_t E, int64_t M_max,
                                    void* q, uint32_t* sf, int32_t* masked_m, int32_t* slot_of,
                                    void* stream);

/*
 * 128x128 weight block quant (benchmark post section 4.1, per_block_cast with
 * UE8M0: scale = block amax / 448 rounded up to a power of two).
 *   w   : bf16 [N][K] contiguous;  q : e4m3 [N][K] contiguous
 *   sfb : fp32 [ceil(N/128)][K/128]; the last row block may be partial.
 *   K % 128 == 0.
 */
int fp8_block_quant_128x128(const void* w, int64_t N, int64_t K, void* q, float* sfb, void* stream);

/*
 * Dense block-scaled GEMM, NT form (benchmark post section 4.2, fp8_gemm_nt
 * writing into a preallocated output; preconditions there: bf16 output,
 * N % 64 == 0, K % 128 == 0):
 *   C[m][n] = bf16_rne( sum_kb 2^ea[m][kb] * sfb[n/128][kb]
 *                       * sum_{k in block kb} a[m][k] * b[n][k] )
 *   a   : e4m3 [M][K] contiguous;    sfa : packed scales [ceil(K/512)][ld_sfa], ld_sfa >= M
 *   b   : e4m3 [N][K] contiguous;    sfb : fp32 [ceil(N/128)][K/128]
 *   c   : bf16 [M][ldc], ldc >= N, ldc % 8 == 0
 *   K >= 128, K % 128 == 0, N % 64 == 0.
 * Decode-sized M splits K across workgroups; the split partials live in a
 * library-owned device workspace kept per (device, stream), allocated on the
 * first call that needs it (make that call outside HIP graph capture: during
 * capture an allocation is refused with FP8BS_ERR_ALLOC).  Calls on different
 * streams never share a workspace.  A workspace that a larger call outgrows is
 * replaced but never freed, so graphs captured earlier stay valid.  A captured
 * graph keeps the workspace of the stream it was captured on: replay it in
 * stream order with the other calls on that stream (a replay running at the same
 * time as calls on the capture stream would share the split-K partials with them,
 * and for the entries that reduce inside the kernel also the arrival counters).
 */
int fp8_block_gemm_nt(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                      const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                      void* stream);

/*
 * Offline weight layout for the decode GEMM.  The weights of a block-scaled GEMM
 * are prepared once, outside the timed step (benchmark post section 4.1 quantizes
 * B before timing); this library's own pre-shuffled layout is a byte permutation
 * of the e4m3 weights [rows][K] (same size) in which every 16-byte load of the
 * decode kernel reads one contiguous kilobyte:
 *   out[((g * KB + kb) * 4 + q) * 1024 + l * 16 + i]
 *     = w[32 g + (l & 31)][128 kb + 64 (q >> 1) + 32 (l >> 5) + 16 (q & 1) + i]
 * for g < rows/32, kb < KB = K/128, q < 4, l < 64, i < 16.  The block scales are
 * unchanged.  Expert weights [E][N][K] are shuffled as rows = E*N.
 *   w, out : device, 16-byte aligned, not overlapping;  rows % 32 == 0, K % 128 == 0.
 */
int fp8_weight_preshuffle(const void* w, int64_t rows, int64_t K, void* out, void* stream);

/*
 * fp8_block_gemm_nt with the weights b in the layout of fp8_weight_preshuffle
 * (rows = N); every other argument, the result and the workspace rules are those
 * of fp8_block_gemm_nt.  M <= 64 runs the weight-streaming kernel, whose loads this
 * layout makes contiguous; larger M the ring tiles of fp8_block_gemm_nt, each weight
 * DMA instruction then moving one contiguous kilobyte (bit-identical results; at
 * prefill sizes 1-6% shorter than fp8_block_gemm_nt on the plain layout).
 */
int fp8_block_gemm_nt_preshuffled(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                  const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N,
                                  int64_t K, void* stream);

/*
 * fp8_block_gemm_nt_preshuffled for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Arguments, kernels and result are those of
 * fp8_block_gemm_nt_preshuffled (bit-identical output); the split-K scratch
 * (arrival counters and fp32 partials) is a static device array of 8 MiB per GPU
 * instead of the per-stream workspace, so this call never allocates or frees.  For
 * M <= 64 and K <= 143360 (the weight-streaming kernel) the automatic configuration
 * needs at most 64 KiB + 224 * 64 * 128 * 4 bytes (7.4 MB), for larger M none where the
 * tiles fill the GPU (else K is split there too); a problem needing more than 8 MiB
 * returns FP8BS_ERR_SCRATCH without launching.  Every call on one GPU shares that array:
 * calls that overlap on one GPU (different streams, or a graph replay running
 * beside another call) race and give undefined results.  The first call on a device
 * clears the counters with a fill kernel on its stream; every call leaves them clear.
 */
int fp8_block_gemm_nt_preshuffled_noalloc(const void* a, const uint32_t* sfa, int64_t ld_sfa,
                                          const void* b, const float* sfb, void* c, int64_t ldc,
                                          int64_t M, int64_t N, int64_t K, void* stream);

/*
 * Masked grouped GEMM (PR #19111: m_grouped GEMM, masked, over [E, max_tokens, K]
 * with per-expert valid counts; 128x128 blocks).  For each expert e and row
 * r < clamp(masked_m[e], 0, M_max), row r of C[e] is the dense NT result of
 * a[e], sfa[e], b[e], sfb[e].  Rows at or past the count are not written, and
 * workgroup tiles that start past the count issue no loads and no MFMA.
 *   a        : e4m3 [E][M_max][K];      sfa : uint32 [E][ceil(K/512)][M_max]
 *   b        : e4m3 [E][N][K];          sfb : fp32 [E][ceil(N/128)][K/128]
 *   c        : bf16 [E][M_max][N];      masked_m : int32 [E] on the device
 *   K >= 128, K % 128 == 0, N % 64 == 0.
 */
int fp8_block_gemm_grouped_masked(const void* a, const uint32_t* sfa, const void* b,
                                  const float* sfb, void* c, const int32_t* masked_m, int64_t E,
                                  int64_t M_max, int64_t N, int64_t K, void* stream);

/*
 * fp8_block_gemm_grouped_masked with the expert weights b in the layout of
 * fp8_weight_preshuffle (rows = E*N, so each expert's [N][K] block is shuffled on
 * its own); every other argument and the result are those of
 * fp8_block_gemm_grouped_masked.  K <= 20480 (a masked group never splits K, and the
 * kernels reading this layout hold the scales of at most 160 K-blocks); larger K
 * returns FP8BS_ERR_SHAPE.
 */
int fp8_block_gemm_grouped_masked_preshuffled(const void* a, const uint32_t* sfa, const void* b,
                                              const float* sfb, void* c, const int32_t* masked_m,
                                              int64_t E, int64_t M_max, int64_t N, int64_t K,
                                              void* stream);

/*
 * Contiguous grouped GEMM, the layout of the high-throughput MoE path (PR #19111
 * page, changelog: the "High-Throughput" DeepEP + DeepGEMM test).  The pages name
 * that path only; the layout is read plainly: the rows of A and C are grouped by
 * expert in runs aligned to 128 rows, and m_indices[m] names the expert of row m
 * (-1 for padding).  Every aligned 128-row block holds rows of one expert followed
 * by padding rows, or padding only.  For every row m with 0 <= m_indices[m] < E,
 * row m of C is the dense NT result of a[m], sfa, b[m_indices[m]],
 * sfb[m_indices[m]].  A block whose first row is padding or names no expert in
 * [0, E) is skipped (no loads, no MFMA, C untouched); padding rows inside a block
 * of an expert are written with that expert's result (unspecified values).
 *   a         : e4m3 [M][K];            sfa : uint32 [ceil(K/512)][ld_sfa], ld_sfa >= M
 *   b         : e4m3 [E][N][K];         sfb : fp32 [E][ceil(N/128)][K/128]
 *   c         : bf16 [M][ldc], ldc >= N, ldc % 8 == 0
 *   m_indices : int32 [M] on the device (values outside [0, E) mean padding)
 *   K >= 128, K % 128 == 0, N % 64 == 0.
 */
int fp8_block_gemm_grouped_contiguous(const void* a, const uint32_t* sfa, int64_t ld_sfa,
                                      const void* b, const float* sfb, void* c, int64_t ldc,
                                      const int32_t* m_indices, int64_t E, int64_t M, int64_t N,
                                      int64_t K, void* stream);

/*
 * Tile-table access, for tuning and for tests that cover every compiled tile
 * shape.  fp8bs_gemm_config reports what the automatic choice would be for a
 * dense (masked = 0), masked (masked = 1), contiguous grouped (masked = 2),
 * dense float-scale (masked = 3), dense pre-shuffled-weight (masked = 4),
 * masked pre-shuffled-weight (masked = 5) or dense float-scale pre-shuffled-weight
 * (masked = 6) problem: kernel index into the tile
 * table, workgroup tile bm x bn, and the number of K splits.  The _cfg variants
 * run the same GEMMs with an explicit kernel index and split count (splits is
 * clamped to [1, K/128]; the masked and contiguous forms use splits == 1 only, and
 * the contiguous form only tiles of at most 128 rows).
 */
int fp8bs_gemm_config_count(void);
int fp8bs_gemm_config(int masked, int64_t M, int64_t N, int64_t K, int32_t* kernel, int32_t* bm,
                      int32_t* bn, int32_t* splits);
/* Whether table entry `kernel` accepts a dense (masked = 0), masked (masked = 1),
 * contiguous grouped (masked = 2), dense float-scale (masked = 3), dense
 * pre-shuffled-weight (masked = 4), masked pre-shuffled-weight (masked = 5) or dense
 * float-scale pre-shuffled-weight (masked = 6) problem of this
 * shape with `splits` K splits: FP8BS_OK with its workgroup tile and the split count
 * it would use, FP8BS_ERR_SHAPE if it does not (for instance K past the entry's scale
 * tables, a masked problem that would need K splits, or a scale format the entry does
 * not read).  Host-only; launches nothing. */
int fp8bs_gemm_config_of(int32_t kernel, int masked, int64_t M, int64_t N, int64_t K, int32_t splits,
                         int32_t* bm, int32_t* bn, int32_t* splits_out);
int fp8_block_gemm_nt_cfg(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                          const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                          int32_t kernel, int32_t splits, void* stream);
int fp8_block_gemm_grouped_masked_cfg(const void* a, const uint32_t* sfa, const void* b,
                                      const float* sfb, void* c, const int32_t* masked_m, int64_t E,
                                      int64_t M_max, int64_t N, int64_t K, int32_t kernel,
                                      void* stream);
int fp8_block_gemm_grouped_contiguous_cfg(const void* a, const uint32_t* sfa, int64_t ld_sfa,
                                          const void* b, const float* sfb, void* c, int64_t ldc,
                                          const int32_t* m_indices, int64_t E, int64_t M,
                                          int64_t N, int64_t K, int32_t kernel, void* stream);
int fp8_block_gemm_nt_float_scales_cfg(const void* a, const float* sfa, int64_t ld_sfa, const void* b,
                                       const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N,
                                       int64_t K, int32_t kernel, int32_t splits, void* stream);
int fp8_block_gemm_nt_preshuffled_cfg(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                      const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N,
                                      int64_t K, int32_t kernel, int32_t splits, void* stream);
int fp8_block_gemm_nt_float_scales_preshuffled_cfg(const void* a, const float* sfa, int64_t ld_sfa,
                                                    const void* b, const float* sfb, void* c, int64_t ldc,
                                                    int64_t M, int64_t N, int64_t K, int32_t kernel,
                                                    int32_t splits, void* stream);
int fp8_block_gemm_grouped_masked_preshuffled_cfg(const void* a, const uint32_t* sfa, const void* b,
                                                  const float* sfb, void* c, const int32_t* masked_m,
                                                  int64_t E, int64_t M_max, int64_t N, int64_t K,
                                                  int32_t kernel, void* stream);

/*
 * The operators around the experts' products: routing, combine, the norms of the
 * residual stream, and an 8-bit checkpoint of the gated activation, each with its
 * backward pass.  The conventions at the top of this file hold; rows that a call
 * leaves out (padding, pairs without a slot) are neither read nor written.  Where a call
 * quantizes "as fp8_quant_group_pack", finite values get the same codes and scales; a value
 * that is not finite gets the NaN code.
 */
enum { FP8BS_SIGMOID = 0, FP8BS_SOFTMAX = 1 };

/*
 * Routing.  For the logits l of a token over E experts:
 *   scores s = sigmoid(l) or softmax(l) (scoring);
 *   ranks  r = s + bias if bias is given, else l;
 *   groups of E / groups consecutive experts are scored by their best rank
 *   (group_top = 1) or by the sum of the two best (group_top = 2; without a bias the sum
 *   of the two best s); the topk_groups best groups take part, ties to the lowest group;
 *   the topk best ranks in them are chosen in descending order, ties to the lowest expert;
 *   weights w = scale * s, divided by the sum of the chosen s if renormalize is not 0
 *   (0 where that sum is 0; the softmax's is formed over the chosen logits).
 * An expert whose logit is NaN or -infinity, or whose rank is (a NaN bias), is not
 * available; where fewer than topk are, the ids that are left are -1 with weight 0, which
 * every other entry point takes as a pair that goes nowhere.  +infinity counts as the
 * largest finite logit.  All arithmetic is fp32; in ranks, sigmoid scores of logits under
 * -87 (below 2e-38) count as one.
 *   logits   : fp32 (logits_f32 = 1) or bf16 [T][ld], ld >= E; aligned to their type only
 *   bias     : fp32 [E] or NULL
 *   topk_ids : int32 [T][topk] out;  weights : fp32 [T][topk] out
 *   T <= 2^22, 1 <= E <= 1024, 1 <= topk <= 64, groups divides E, groups <= 64,
 *   1 <= topk_groups <= groups, topk <= topk_groups * E / groups, group_top <= E / groups.
 * Backward: the choice is held fixed and the bias gets no gradient.  d_logits [T][ld_d]
 * has the type of the logits and is written whole, zeros included.  logits, topk_ids and
 * the options are the forward's; an id of -1 takes no part; no id may stand twice in a row.
 */
int moe_route_topk(const void* logits, int32_t logits_f32, int64_t ld, int64_t T, int64_t E, const float* bias,
                   int32_t scoring, int32_t groups, int32_t topk_groups, int32_t group_top, int32_t topk,
                   int32_t renormalize, float scale, int32_t* topk_ids, float* weights, void* stream);
int moe_route_topk_backward(const void* logits, int32_t logits_f32, int64_t ld, int64_t T, int64_t E,
                            const int32_t* topk_ids, const float* d_weights, int32_t scoring, int32_t topk,
                            int32_t renormalize, float scale, void* d_logits, int64_t ld_d, void* stream);

/*
 * Combine: the experts' rows back to their tokens.
 *   out[t] = base[t] + sum_j weights[t][j] * y[topk_ids[t][j]][slot_of[t][j]]
 * in fp32, j ascending, rounded once.  A pair whose id is outside [0, E) or whose slot is
 * outside [0, M_max) is left out.  With weights = NULL (ones) this is also the gradient of
 * fp8_quant_group_pack_to_experts' dispatch.
 *   y         : bf16 [E][M_max][N] (what the masked GEMM wrote)
 *   topk_ids, slot_of : int32 [T][topk];  weights : fp32 [T][topk] or NULL
 *   base      : bf16 [T][ld_base] or NULL;  out : bf16 [T][ld_out]
 *   T <= 2^22, N % 8 == 0, N <= 2^20, T * ceil(N/2048) <= 2^24, 1 <= topk <= 64,
 *   ld_base and ld_out >= N and % 8 == 0.
 * Backward, for every pair that has a row: d_y[e][s] = weights[t][j] * d_out[t], in bf16
 * (d_y [E][M_max][N]) or, with d_y = NULL, as q e4m3 [E][M_max][N] and sf uint32
 * [E][ceil(N/512)][M_max] quantized as fp8_quant_group_pack quantizes the fp32 values
 * (N % 128 == 0), ready for the masked GEMM that takes the gradient on; and d_weights[t][j] =
 * <d_out[t], y[e][s]> (0 for a pair without a row, or with N == 0; NULL: not wanted, and y is not read).
 * No two pairs may name the same row.
 */
int moe_combine(const void* y, const int32_t* topk_ids, const int32_t* slot_of, const float* weights, const void* base,
                int64_t ld_base, int64_t T, int32_t topk, int64_t E, int64_t M_max, int64_t N, void* out,
                int64_t ld_out, void* stream);
int moe_combine_backward(const void* d_out, int64_t ld_d, const void* y, const int32_t* topk_ids,
                         const int32_t* slot_of, const float* weights, int64_t T, int32_t topk, int64_t E,
                         int64_t M_max, int64_t N, void* d_y, void* q, uint32_t* sf, float* d_weights, void* stream);

/*
 * Norms before and after a block, with the block's gate and the residual's scale:
 *   b = y * rsqrt(mean(y^2) + eps) * (w_post + weight_offset)    (b = y if w_post is NULL)
 *   h = residual_scale * x + gate * b                            (no gate: 1; y NULL: b = 0)
 *   z = h * rsqrt(mean(h^2) + eps) * (w_pre + weight_offset)
 * in fp32; z comes from the unrounded h.  Any of h, z and (q, sf) may be NULL.
 *   x, h   : bf16, or fp32 if residual_f32 = 1, [T][ldx], [T][ldh]
 *   y      : bf16 [T][ldy] or NULL;  w_post : bf16 [N] or NULL (needs y);  w_pre : bf16 [N]
 *   gate   : bf16 [N] with ld_gate = 0, or [T][ld_gate], or NULL (needs y)
 *   z      : bf16 [T][ldz];  q : e4m3 [T][ldq], sf : uint32 [ceil(N/512)][ld_sf], quantized as
 *            fp8_quant_group_pack quantizes the fp32 values (N % 128 == 0, ldq % 16 == 0)
 *   N % 8 == 0, N <= 16384, leading dimensions >= N and % 8 == 0, ld_sf >= T.
 * Backward: from d_z (bf16) and the gradient d_h of h that the residual stream brings (its
 * type; NULL: none), with h as the forward wrote it, the gradients d_x (type of x), d_y (bf16),
 * d_w_pre and d_w_post (fp32 [N]) and d_gate (fp32 [N] if ld_gate = 0, else bf16
 * [T][ld_dgate]).  Those of parts that the forward has not are NULL.  The sums over the tokens
 * are taken in a fixed order: equal calls give equal bits.  Their partial sums (at most
 * 52 MB) go to the library's per-(device, stream) workspace (FP8BS_ERR_ALLOC if
 * it has to grow during HIP graph capture).  T == 0 sets the weights' gradients to zero.
 * residual_rms_norm_backward_noalloc takes the partial sums' memory from the caller
 * instead: at least residual_rms_norm_backward_scratch_bytes(T, N) bytes (0 for one
 * row: scratch is not looked at), 16-byte aligned, free again for other work of the stream
 * once the call's own is done; FP8BS_ERR_SCRATCH if it is less.  It allocates nothing and
 * shares nothing with other calls, so a captured call replays on any stream.
 */
int residual_rms_norm(const void* x, int64_t ldx, int32_t residual_f32, const void* y, int64_t ldy, const void* w_post,
                      const void* gate, int64_t ld_gate, const void* w_pre, float residual_scale, float eps,
                      float weight_offset, int64_t T, int64_t N, void* h, int64_t ldh, void* z, int64_t ldz, void* q,
                      int64_t ldq, uint32_t* sf, int64_t ld_sf, void* stream);
int residual_rms_norm_backward(const void* d_z, int64_t ld_dz, const void* d_h, int64_t ld_dh, const void* h,
                               int64_t ldh, int32_t residual_f32, const void* y, int64_t ldy, const void* w_post,
                               const void* gate, int64_t ld_gate, const void* w_pre, float residual_scale, float eps,
                               float weight_offset, int64_t T, int64_t N, void* d_x, int64_t ld_dx, void* d_y,
                               int64_t ld_dy, float* d_w_pre, float* d_w_post, void* d_gate, int64_t ld_dgate,
                               void* stream);
int64_t residual_rms_norm_backward_scratch_bytes(int64_t T, int64_t N);
int residual_rms_norm_backward_noalloc(const void* d_z, int64_t ld_dz, const void* d_h, int64_t ld_dh, const void* h,
                                       int64_t ldh, int32_t residual_f32, const void* y, int64_t ldy,
                                       const void* w_post, const void* gate, int64_t ld_gate, const void* w_pre,
                                       float residual_scale, float eps, float weight_offset, int64_t T, int64_t N,
                                       void* d_x, int64_t ld_dx, void* d_y, int64_t ld_dy, float* d_w_pre,
                                       float* d_w_post, void* d_gate, int64_t ld_dgate, void* scratch,
                                       int64_t scratch_bytes, void* stream);

/*
 * silu_mul_quant_group_pack that also keeps gate and up for the backward pass in 8 bits:
 *   cq  : e4m3 [E][M_max][2H], gate then up, quantized as fp8_quant_group_pack does
 *   csf : uint32 [E][2 * ceil(H/512)][M_max]: the words of gate, then the words of up
 * x, masked_m, q and sf as there; q and sf are the same bits.  E <= 1024.
 * Backward from the checkpoint: with s = sigmoid(gate) of the decoded values, for the valid rows
 *   d_gate = d_y * up * s * (1 + gate * (1 - s)),   d_up = d_y * gate * s
 *   d_y : bf16 [E][M_max][H];  d_x : bf16 [E][M_max][2H] out, or, with d_x = NULL, q e4m3
 *   [E][M_max][2H] and sf uint32 [E][ceil(2H/512)][M_max] (the masked GEMM's layout for K = 2H).
 */
int silu_mul_quant_group_pack_checkpoint(const void* x, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                                         void* q, uint32_t* sf, void* cq, uint32_t* csf, void* stream);
int silu_mul_backward_from_checkpoint(const void* d_y, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                                      const void* cq, const uint32_t* csf, void* d_x, void* q, uint32_t* sf,
                                      void* stream);

/*
 * A mixture-of-experts layer for a few tokens (a decode step), from the router's choice to
 * the layer's output, in two launches.  For token t and choice j with e = topk_ids[t][j] in
 * [0, E), and v the values that codes stand for under their scales:
 *   g, u   = v(q[t]) v(w13[e])^T            the first H rows of w13[e] and the last H, in fp32
 *   y      = quantized(g / (1 + exp(-g)) * u)   1x128 groups, as fp8_quant_group_pack
 *   out[t] = base[t] + sum_j weights[t][j] * (v(y) v(w2[e])^T)     fp32, bf16 at the end
 * Pairs whose id is outside [0, E) are left out (a token without any gets base, or zeros); a
 * token may name an expert twice.  It is what the dispatch quantization, the masked products,
 * silu_mul_quant_group_pack and moe_combine compute, without their roundings of the products
 * to bf16.  Values that are not finite stay with their token.
 * The products take the values v in bf16, which holds them exactly under block scales and scale
 * bytes of 2^-124 to 2^119 (e2m1: bytes 1 to 252); past those, values of 2^128 and more are
 * infinite, and what of a value is under 2^-133 is lost.
 *   q        : e4m3 [T][ldq], 1 <= T <= 64;  sf : uint32 [ceil(K/512)][ld_sf], ld_sf >= T
 *   topk_ids : int32 [T][topk];  weights : fp32 [T][topk];  1 <= topk <= 64
 *   w13, s13 : e4m3 [E][2H][K], fp32 [E][2H/128][K/128];  w2, s2 : e4m3 [E][K][H], fp32
 *              [E][K/128][H/128];  as the masked GEMMs take them.  1 <= E <= 1024
 *   base     : bf16 [T][ld_base] or NULL;  out : bf16 [T][ld_out]
 *   scratch  : moe_decode_layer_scratch_bytes(T, topk, H) bytes, 16-byte aligned, that no other
 *              call uses until this one's work on the stream is done
 *   K % 128 == 0 and H % 128 == 0, both at most 65536; the rows of q and of sf span less than 2 GiB.
 * moe_decode_layer_preshuffled takes w13 and w2 in the layout of fp8_weight_preshuffle (rows = 2H
 * and K of each expert), moe_decode_layer_w4 in e2m1 as w4_preshuffle lays them out.  More than
 * 64 tokens go through the masked GEMMs; those take no e2m1 weights, so on these they go in
 * pieces of 64, each of which reads its experts again.
 * Equal calls give equal bits.
 */
int64_t moe_decode_layer_scratch_bytes(int64_t T, int32_t topk, int64_t H);
int moe_decode_layer(const void* q, int64_t ldq, const uint32_t* sf, int64_t ld_sf, const int32_t* topk_ids,
                     const float* weights, const void* w13, const float* s13, const void* w2, const float* s2,
                     const void* base, int64_t ld_base, int64_t T, int32_t topk, int64_t E, int64_t K, int64_t H,
                     void* out, int64_t ld_out, void* scratch, int64_t scratch_bytes, void* stream);
int moe_decode_layer_preshuffled(const void* q, int64_t ldq, const uint32_t* sf, int64_t ld_sf,
                                 const int32_t* topk_ids, const float* weights, const void* w13, const float* s13,
                                 const void* w2, const float* s2, const void* base, int64_t ld_base, int64_t T,
                                 int32_t topk, int64_t E, int64_t K, int64_t H, void* out, int64_t ld_out,
                                 void* scratch, int64_t scratch_bytes, void* stream);
int moe_decode_layer_w4(const void* q, int64_t ldq, const uint32_t* sf, int64_t ld_sf, const int32_t* topk_ids,
                        const float* weights, const void* w13, const void* s13, const void* w2, const void* s2,
                        const void* base, int64_t ld_base, int64_t T, int32_t topk, int64_t E, int64_t K, int64_t H,
                        void* out, int64_t ld_out, void* scratch, int64_t scratch_bytes, void* stream);

/*
 * Weights of 4 bits under group scales.  Two formats:
 *   FP8BS_E2M1  codes of 1 + 2 + 1 bits (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), a UE8M0
 *               byte b for every 32 columns: value = code * 2^(b - 127), b from 1 to 254; values of
 *               2^128 and more (codes from 4 on with b = 253, from 2 on with 254) are infinite
 *   FP8BS_INT4  codes c = 0..15, a bf16 scale s for every 32, 64 or 128 columns, and a zero point z
 *               (uint8) beside it, or 8 without one: value = s * (c - z)
 * K % 128 == 0, K <= 65536.
 *
 * w4_group_quant: bf16 w [rows][K] (contiguous, finite) -> codes [rows][K/2] (even column in the low
 *   half of a byte), scales [rows][K/group], zeros [rows][K/group] or NULL (FP8BS_INT4 only).
 *     FP8BS_E2M1: the smallest 2^e with 6 * 2^e >= amax (e >= -126), codes to nearest even (a w from
 *     3.5 * 2^126 on is rounded to 2^128, which is infinite as above).
 *     FP8BS_INT4: s = bf16(amax / 7), c = clamp(rint(w / s) + 8, 0, 15); with zeros s = bf16((max - min) / 15)
 *     over the group's values and 0, z = min(rint(-min / s), 15), c = clamp(rint(w / s) + z, 0, 15), in
 *     fp32 (max - min also where it passes fp32's range); where s is 0, c = z (0 with zeros).
 * w4_preshuffle: codes [E][N][K/2], scales and zeros [E][N][K/group] in row order -> the layout that the
 *   products read, rows past N and columns past K zero, with tiles = ceil(N/16), units = ceil(K/512):
 *     codes_out  [E][tiles][K/128][64][16 bytes]   entry 16 c + r of a tile is row r:
 *       FP8BS_E2M1  columns 32 c .. 32 c + 31;  FP8BS_INT4  in 32-bit word i the columns 32 i + 8 c +
 *       0, 2, 4, 6, 1, 3, 5, 7, from the low bits up
 *     scales_out, zeros_out   FP8BS_E2M1  [E][tiles][units][64][4]: byte b of entry 16 c + r is group
 *       4 b + c of row r;  FP8BS_INT4  [E][tiles][units][16][512/group]
 * w4_group_gemv_nt: out[t][n] = bf16( sum over k of x[t][k] * w[n][k] ), w in that layout (E = 1), sums in
 *   fp32.  Made for few rows of x: every 64 of them read the weights once.  zeros may be NULL.  A value of x that
 *   is not finite, or (FP8BS_INT4, whose codes are taken as 16 + c first) whose 32-fold sums, or z-fold ones if a zero
 *   point is larger, pass fp32's range, makes its own row not finite, and no other.
 *   x : bf16 [T][ldx];  out : bf16 [T][ld_out], ld_out >= N, rows 2-byte aligned;  T <= 2^21, N <= 2^27,
 *   64 rows of x span less than 2 GiB.
 */
enum { FP8BS_E2M1 = 0, FP8BS_INT4 = 1 };
int w4_group_quant(const void* w, int64_t rows, int64_t K, int32_t format, int32_t group, void* codes, void* scales,
                   void* zeros, void* stream);
int w4_preshuffle(const void* codes, const void* scales, const void* zeros, int64_t E, int64_t N, int64_t K,
                  int32_t format, int32_t group, void* codes_out, void* scales_out, void* zeros_out, void* stream);
int w4_group_gemv_nt(const void* x, int64_t ldx, const void* codes, const void* scales, const void* zeros, int64_t T,
                     int64_t N, int64_t K, int32_t format, int32_t group, void* out, int64_t ld_out, void* stream);

/* Status helpers. */
const char* fp8bs_status_string(int status);
int fp8bs_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_H */

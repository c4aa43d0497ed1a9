/*
 * vca.h -- C ABI of the VC-Attention hot path on GB300 (sm_103a).
 *
 * VC-Attention ("VC-Attention: Value Smoothing and Softmax Casting for Low-bit
 * Attention", agihunt.info/papers/2609.15810, section "method") changes two steps
 * of a FlashAttention-style FP8 kernel:
 *   V-Smooth   -- per (batch, head), k-means on the Value tokens; K and V are
 *                 permuted together by cluster label; every 128-token block
 *                 subtracts its mean (a 16-bit vector), only the residual is
 *                 quantised (per-channel E4M3 or NVFP4) and the mean is added
 *                 back through the row sums online softmax already keeps.
 *   ExpCast-FP8 -- one FMA writes the E4M3 byte of the softmax probability
 *                 straight from the log2-domain score:
 *                 byte = rne(8 log2 p + 56 + beta), beta = -0.35, clipped to the
 *                 normal range (codes below 8 flush to 0).
 *
 * The library computes on the device only; there is no CPU fallback.  Every
 * entry point is asynchronous on the caller's CUDA stream (`stream` is a
 * cudaStream_t; NULL is the legacy default stream).  The library allocates no
 * device memory: the caller owns every buffer (inputs, outputs and the scratch
 * workspace sized by vca_workspace_bytes).  Device pointers must be 16-byte
 * aligned.  No C++ exception crosses this boundary.
 *
 * Layouts (all contiguous, row-major, little-endian; BH = B*H, nb = N/128):
 *   Q, K, V       bf16 (uint16 bit patterns) [B][H][N][d], d = 128
 *   labels, perm  int32 [BH][N]; perm[i] = source token placed in slot i
 *   counts        int32 [BH][k];  centroids fp32 [BH][k][d]
 *   q8, k8        E4M3 bytes [BH][N][d] (q8 in original order, k8 permuted)
 *   sq, sk        fp32 [BH][nb]  (one dequantisation scale per 128-token block)
 *   v_mean        bf16 [BH][nb][d] (block means of the permuted V)
 *   E4M3 mode:  v_res E4M3 [BH][nb][d][128] (residual, channel-major per block),
 *               v_scale fp32 [BH][d] (one scale per channel), v_sf unused (NULL)
 *   NVFP4 mode: v_res [BH][nb][d][64] packed E2M1 (token 2i in the low nibble),
 *               v_sf E4M3 [BH][nb][d][8] (one scale per 16 tokens of a channel),
 *               v_scale fp32 [BH] (the per-(b,h) scale above the E4M3 scales)
 *   O             bf16 [B][H][N][d], rows in the original query order
 *
 * Sizes accepted by every entry point: B >= 1, H >= 1, B*H <= 65,535 (one grid
 * row of CTAs per head), N a positive multiple of 128, B*H*N <= 2^31 - 1
 * tokens, d = 128.  Anything else is VCA_ERR_INVALID_ARG.
 *
 * Return value: a vca_status.  Invalid arguments are reported synchronously and
 * launch nothing.  Device-side failures (a bounded wait that ran out) are
 * written to the optional `dev_status` word, which the caller reads after the
 * stream has synchronised.
 */
#ifndef VCA_H
#define VCA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    VCA_OK = 0,
    VCA_ERR_INVALID_ARG = 1,   /* bad size, null or misaligned pointer */
    VCA_ERR_UNSUPPORTED = 2,   /* a combination the method does not define */
    VCA_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
    VCA_ERR_TIMEOUT = 4,       /* a bounded device wait ran out (dev_status) */
    VCA_ERR_WORKSPACE = 5,     /* workspace missing or smaller than required */
    VCA_ERR_FULL = 6           /* too few free pages (dev_status of the cache's planning) */
} vca_status;

typedef enum { VCA_V_E4M3 = 0, VCA_V_NVFP4 = 1 } vca_vmode;
/* VCA_OP_PREP_KSMOOTH: the prep's workspace when VCA_PREP_K_SMOOTH is set. */
typedef enum {
    VCA_OP_GROUP = 0, VCA_OP_PREP = 1, VCA_OP_ATTENTION = 2, VCA_OP_PREP_KSMOOTH = 3,
    VCA_OP_CACHE_ATTENTION = 4, VCA_OP_CACHE_WEIGH = 5   /* vca_cache_workspace_bytes */
} vca_op;

/* Human-readable name of a vca_status value (static string, never NULL). */
const char *vca_status_string(int status);

/* Library version: major * 10000 + minor * 100 + patch. */
int vca_version(void);

/* Scratch bytes the caller must pass as `ws` for `op` at this problem size
 * (0 if none).  Returns 0 as well for invalid sizes. */
size_t vca_workspace_bytes(int op, int B, int H, int N, int d, int k, int vmode);

/*
 * vca_group -- V-Smooth "Group" step (paper page, "method"; news page,
 * "V-Smooth" bullet "Group"): per (b,h), Lloyd k-means on the N Value tokens
 * (d = 128 channels), then a stable counting sort of the tokens by label.
 *   init     centroid c = V row floor((c + 1/2) N / k)
 *   assign   label = argmin_c |v - C_c|^2, ties to the lowest c
 *   update   C_c = mean of its tokens (fp32); an empty cluster keeps C_c
 *   `iters` rounds of (assign, update); labels are those of the last assign.
 * Outputs: labels [BH][N], perm [BH][N] (tokens ordered by (label, index)),
 * counts [BH][k] (tokens per label), centroids [BH][k][d] (may be NULL).
 * The distances are taken on the tensor core from bf16 V and the centroids
 * split into bf16 hi + lo parts (fp32 accumulation): labels equal those of an
 * exact computation except where two centroids are within ~2^-16 relative of
 * each other.
 * Requires 1 <= k <= min(N, 128), 1 <= iters <= 1000,
 * ws_bytes >= vca_workspace_bytes(VCA_OP_GROUP, ...).
 * dev_status (optional, device int32): set to VCA_ERR_TIMEOUT if a bounded
 * wait inside the kernels ran out; left untouched otherwise.
 */
int vca_group(const uint16_t *V, int B, int H, int N, int d, int k, int iters,
              int32_t *labels, int32_t *perm, int32_t *counts, float *centroids,
              void *ws, size_t ws_bytes, int32_t *dev_status, void *stream);

/*
 * vca_prep_quant -- the fused V-Smooth prep (paper page, "method": demean each
 * 128-token hardware block, quantise only the residual, 16-bit mean per block;
 * Q/K to FP8; no high-precision intermediate is written to device memory):
 *   K and V are gathered by perm (perm may be reused across calls);
 *   v_mean[b] = bf16(fp32(sum of the block's 128 tokens) / 128);
 *   residual R = fp32(v) - fp32(v_mean);
 *   E4M3:  a_c = max |R[:, c]| over the sequence, v_scale[c] = a_c / 448,
 *          v_res = E4M3_rne_sat(R * (448 / a_c));
 *   NVFP4: g = max |R| / (6 * 448) per (b,h) (v_scale), per 16 tokens of a
 *          channel sf = E4M3(amax16 / (6 g)) (v_sf),
 *          v_res = E2M1_rne_sat(R * (1 / (sf * g)));
 *   Q (original order) and K (permuted) per 128-token block:
 *          s = amax / 448, x8 = E4M3_rne_sat(x * (448 / amax)).
 * An all-zero block or channel gets scale 1.
 */
int vca_prep_quant(const uint16_t *Q, const uint16_t *K, const uint16_t *V, const int32_t *perm,
                   int B, int H, int N, int d, int vmode,
                   uint8_t *q8, float *sq, uint8_t *k8, float *sk,
                   uint8_t *v_res, uint8_t *v_sf, float *v_scale, uint16_t *v_mean,
                   void *ws, size_t ws_bytes, void *stream);

/*
 * vca_prep_quant_ex -- vca_prep_quant with option flags (flags = 0 is exactly
 * vca_prep_quant; unknown bits return VCA_ERR_INVALID_ARG):
 *   VCA_PREP_QK_HADAMARD  rotate every Q and K row by the unnormalised 128-point
 *          Walsh-Hadamard transform H before the FP8 quantisation (the QK
 *          Hadamard of the Q/K prior art the insight page discusses, which
 *          spreads outlier channels over all channels).  H is symmetric with
 *          H H = 128 I, so (H q) . (H k) = 128 q . k: sk carries the factor
 *          1/128 (exact) and vca_attention needs no change.  The transform is
 *          defined as fp32 butterflies in a fixed order -- for bit k = 0..6 of
 *          the channel index, every pair (c, c + 2^k) with bit k of c clear
 *          becomes (a + b, a - b) -- so its rounding is reproducible; then
 *          s = amax / 448 and x8 = E4M3_rne_sat(x * (448 / amax)) as usual.
 *   VCA_PREP_K_SMOOTH  subtract the keys' channel mean over the sequence of
 *          each (b,h) before the FP8 quantisation (SageAttention's treatment
 *          of the keys' channel bias, the handling of Q/K outliers the paper
 *          page's motivation and the insight page's section "Value Is the
 *          Error Source Earlier Methods Underestimated" refer to).  Every score
 *          of a query row moves by the same amount, so softmax attention is
 *          unchanged and vca_attention needs no change.  The mean is fp32 in a
 *          fixed order, so it is reproducible: per permuted 128-token block a
 *          halving tree (token i plus token i + 64 for i < 64, then i + 32, ...,
 *          i + 1), the block sums added in block order, divided by N; each key
 *          value becomes fp32(k) - mean (one rounding), before the Hadamard
 *          rotation when both flags are set.  Needs ws_bytes >=
 *          vca_workspace_bytes(VCA_OP_PREP_KSMOOTH, ...).
 */
#define VCA_PREP_QK_HADAMARD 1u
#define VCA_PREP_K_SMOOTH 2u
int vca_prep_quant_ex(const uint16_t *Q, const uint16_t *K, const uint16_t *V, const int32_t *perm,
                      int B, int H, int N, int d, int vmode, uint32_t flags,
                      uint8_t *q8, float *sq, uint8_t *k8, float *sk,
                      uint8_t *v_res, uint8_t *v_sf, float *v_scale, uint16_t *v_mean,
                      void *ws, size_t ws_bytes, void *stream);

/*
 * vca_prep_quant_noalloc -- the same computation and outputs as vca_prep_quant,
 * for callers that cannot pass the library any scratch device memory (a host
 * program that owns all device memory and gives an operator only its tensors,
 * or a code path where a cudaMalloc and its possible device synchronisation are
 * not allowed).  The paper has no counterpart to this entry point.
 * Scratch: a buffer of VCA_NOALLOC_SCRATCH_BYTES built into the library, which
 * every GPU that loads the library holds until the process exits.  Problems
 * whose prep workspace (vca_workspace_bytes(VCA_OP_PREP, ...)) exceeds it return
 * VCA_ERR_WORKSPACE and launch nothing.  That workspace is 512 bytes per
 * 128-token block plus 512 bytes per head, so 16 MiB covers exactly the
 * problems with B*H*(N/128) + B*H <= 32,768 (B=1, H=40, N=70,656 needs 22,120
 * of those units, 11.3 MB).  The first call on a device looks
 * up the buffer's device address (make it before any stream capture).  Every
 * call shares the one buffer: calls that overlap on the GPU race and must be
 * ordered by the caller.  Nothing in the buffer needs clearing between calls.
 * This entry point allocates no device memory.
 */
#define VCA_NOALLOC_SCRATCH_BYTES (16u << 20)
int vca_prep_quant_noalloc(const uint16_t *Q, const uint16_t *K, const uint16_t *V, const int32_t *perm,
                           int B, int H, int N, int d, int vmode,
                           uint8_t *q8, float *sq, uint8_t *k8, float *sk,
                           uint8_t *v_res, uint8_t *v_sf, float *v_scale, uint16_t *v_mean,
                           void *stream);

/*
 * vca_attention -- non-causal FP8 attention over the prepared operands (paper
 * page, "method": online softmax; ExpCast; the block means come back as one
 * outer product rowsum_b x mean_b per key block, no second pass).  For every
 * query row, key blocks are visited in increasing (permuted) order; with
 * c = (sq * sk_b) * (softmax_scale * log2 e), S the raw FP8 product q8 . k8
 * and m the reference max (log2 units), which moves to the block's max
 * max_j(S_j * c) only when that exceeds m + 8 (the first block always sets it):
 *   expcast = 1:  P = E4M3 byte rne(fma(S, 8c, 55.65 - 8m)), flushed below 8
 *   expcast = 0:  P = E4M3_rne_sat(exp2(fma(S, c, -m)))
 *   NVFP4 mode (expcast must be 0): per 16 keys p = exp2(fma(S, c, -m)),
 *                 sf = E4M3(amax16 / 6), P = E2M1(p * (1 / sf)) * sf; the V
 *                 residual decodes to E2M1 * its 16-token E4M3 scale
 *   rowsum_b = sum of the decoded P of block b; l = sum_b rowsum_b
 *   O = (sum_b P_b . v_res_b * v_scale + sum_b rowsum_b (x) v_mean_b) / l
 * with accumulators rescaled by 2^(m_old - m_new) whenever m moves.
 * softmax_scale <= 0 selects 1/sqrt(d).  expcast = 1 with VCA_V_NVFP4 returns
 * VCA_ERR_UNSUPPORTED (NVFP4 has no single affine log-to-code map).
 * dev_status (optional, device int32): set to VCA_ERR_TIMEOUT if a bounded
 * wait inside the kernel ran out; left untouched otherwise.
 */
int vca_attention(const uint8_t *q8, const float *sq, const uint8_t *k8, const float *sk,
                  const uint8_t *v_res, const uint8_t *v_sf, const float *v_scale,
                  const uint16_t *v_mean, int B, int H, int N, int d,
                  float softmax_scale, int expcast, int vmode,
                  uint16_t *O, int32_t *dev_status, void *stream);

/*
 * vca_expcast_codes -- the device ExpCast map on its own (the same inline
 * function the attention kernel uses), for bit-exact testing:
 *   out[i] = clip(rne(fma(s_raw[i], 8 c[i], 55.65 - 8 m[i]))), codes < 8 -> 0,
 *   codes > 126 -> 126.  Device arrays of n elements.
 */
int vca_expcast_codes(const float *s_raw, const float *c, const float *m, int64_t n,
                      uint8_t *out, void *stream);

/*
 * vca_e4m3_encode_bits -- the device's E4M3 conversion (round to nearest even,
 * saturating to +-448) applied to the fp32 bit patterns start .. start+n-1;
 * out is a device array of n bytes.  Used to compare the hardware conversion
 * with a software one over every fp32 input.
 */
int vca_e4m3_encode_bits(uint32_t start, int64_t n, uint8_t *out, void *stream);

/*
 * vca_selftest_timeout -- launches one bounded wait on a barrier that nothing
 * completes, with the given limit in nanoseconds (1e3 .. 1e10); the kernel gives
 * up, writes VCA_ERR_TIMEOUT to dev_status and returns, leaving the context
 * usable.  Exercises the failure path every kernel wait uses.
 */
int vca_selftest_timeout(int32_t *dev_status, uint64_t limit_ns, void *stream);

/* Upper bound on every bounded device wait, in nanoseconds (default 2e9). */
void vca_set_wait_limit_ns(uint64_t limit_ns);

/*
 * The 8-bit cache: keys and values of a growing sequence kept as E4M3 in pages
 * of 128 tokens (the method's hardware block) with one scale per page and head,
 * for models that produce a video chunk by chunk, or a sequence token by token,
 * and attend to what came before.  The paper has no counterpart to it.
 *
 *   k8, v8   E4M3 bytes [pages][H][128][d]
 *   sk, sv   fp32 [pages][H], powers of two >= 2^-120: a value is code * scale
 *   table    int32 [B][cols]: the page of tokens 128 j .. 128 j + 127 of
 *            sequence b; entries behind its last page are never read
 *   len      int32 [B]: the tokens each sequence holds, the new ones of the
 *            current call included
 *
 * The struct lies in host memory and is read during the call; every pointer in
 * it is a device pointer (k8 and v8 16-byte aligned, the others 4-byte).
 * Sizes: d = 128, pages, H, B, cols >= 1, B*H <= 65,535, pages*H*128 <= 2^31 - 1,
 * cols*128 <= 2^31 - 1; codes are addressed with 64 bits.  Sequences may share
 * pages that no call writes.
 *
 * A call's rows (K, V, Q) are bf16 [T][heads][d]: `start`, int32 [B + 1] on the
 * device, cuts them: rows start[b] .. start[b+1] - 1, n of them (0 allowed),
 * are sequence b's newest tokens, row i at slot len - n + i.  Rows behind
 * start[B] belong to nobody and their outputs are left as they are.  The
 * distance from token to token and from head to head is given in elements
 * (multiples of 8; the d channels lie together), so views of a fused
 * projection need no copy.  T = 0 returns VCA_OK and launches nothing.
 *
 * What lies on the device is checked there: a sequence whose len is out of
 * range (above cols*128 or negative) counts as having no rows, and so do a
 * sequence whose start is (not rising within 0 .. T) and all sequences behind it;
 * a page outside 0 .. pages - 1 counts as holding no tokens; and dev_status
 * (optional, device int32) is set to VCA_ERR_INVALID_ARG, or to VCA_ERR_TIMEOUT if
 * a bounded wait ran out; it is left untouched otherwise.  Scales are trusted to
 * be powers of two.
 * Calls keep nothing between them: a workspace may be used by any call that
 * does not overlap with this one, and the calls can be captured into a graph.
 * Outputs and workspace must not overlap the inputs.
 */
typedef struct {
    uint8_t *k8, *v8;
    float *sk, *sv;
    const int32_t *table, *len;
    int pages, H, d, B, cols;
} vca_cache;

/* Scratch bytes for VCA_OP_CACHE_ATTENTION or VCA_OP_CACHE_WEIGH of T rows with
 * Hq query heads over H KV heads, B sequences and `cols` table columns (0 for
 * invalid sizes).  The workspace is 16-byte aligned; nothing has to be in it. */
size_t vca_cache_workspace_bytes(int op, int T, int Hq, int H, int B, int cols);

/*
 * vca_cache_append -- quantises new K and V rows [T][H][d] into the cache.  Per
 * page and head with new rows X: s = the smallest power of two >= 2^-120 with
 * max |X| <= 448 s, or the page's scale if that is larger and the page already
 * held tokens; sk (sv) = s; code = E4M3_rne(x / s).  x / s is exact.  Where s
 * grew, the codes already there become E4M3_rne(value / s): only values that
 * turn subnormal lose bits.  NaN and infinities become the NaN code and do not
 * enter the maximum.  Slots that are not new and not rescaled stay as they are.
 * A sequence with n > len is invalid.  No page may be written twice in a call.
 */
int vca_cache_append(const vca_cache *cache, const uint16_t *K, int64_t k_token, int64_t k_head, const uint16_t *V,
                     int64_t v_token, int64_t v_head, const int32_t *start, int T, int32_t *dev_status, void *stream);

/*
 * vca_cache_append_ex -- vca_cache_append that also clears the weights of the new
 * tokens: weight[page][h][slot] = 0 (vca_cache_weigh's, 16-byte aligned; NULL clears
 * nothing).  Who weighs and evicts in a pool whose pages are used again appends
 * with it, or clears a page's weights before its first token (before
 * vca_cache_evict, those of the pages it writes): else a new token starts with the
 * weight of the token that its slot held before.
 */
int vca_cache_append_ex(const vca_cache *cache, const uint16_t *K, int64_t k_token, int64_t k_head, const uint16_t *V,
                        int64_t v_token, int64_t v_head, const int32_t *start, int T, float *weight, int32_t *dev_status,
                        void *stream);

/*
 * vca_cache_attention -- attention of the rows Q [T][Hq][d] over the cache;
 * query heads h*G .. h*G + G - 1 read KV head h, G = Hq / H:
 *   s_ij = softmax_scale q_i . (k_j sk);  with softcap > 0: softcap tanh(s_ij / softcap)
 *   j visible to row i: j < len, and with causal = 1: j <= len - n + i
 *   O_i = sum_j softmax_j(s_ij) v_j sv,  lse_i = ln sum_j exp(s_ij)
 * A row that sees nothing gets O = 0 and lse = -inf.  softmax_scale <= 0 selects
 * 1/sqrt(d); softcap = 0 caps nothing, and softmax_scale, softcap and softmax_scale
 * / softcap have to be below 8.5e37.  A cap of 2^40 or more counts as none (scores
 * below 2^28 change by less than an fp32 rounding), one below 2^-40 as 2^-40.  O is
 * bf16 [T][Hq][d] and lse fp32 [T][Hq] (may be NULL), both contiguous.  The products
 * are exact but for query elements far below the largest of their row (2^-30 of it)
 * or of their 32 channels (2^-15, off by 2^-22 of the largest, where a sequence has
 * many rows); sums and statistics are fp32, the probabilities enter the second
 * product as fp16 (2^-12 relative, nothing below 2^-25 of the row's largest); where
 * a sequence has many rows, values of pages whose sv is below 2^-95 of the
 * sequence's largest lose bits and count as 0 below 2^-104.  A slot behind len may
 * hold any bytes; a NaN among the values of a sequence may reach every row of that
 * sequence, one in a query row, or an infinity, only that row.  Equal calls give
 * equal bits.
 * The kernel is chosen on the host for the whole call, by its average of
 * T (Hq / H) / B rows a sequence and KV head (vca_cache_weigh's too): a batch that
 * mixes single tokens with prompts, or has many sequences without rows, is
 * right, and faster as calls of their own for those with one row and with many.
 */
int vca_cache_attention(const vca_cache *cache, const uint16_t *Q, int64_t q_token, int64_t q_head,
                        const int32_t *start, int T, int Hq, int causal, float softmax_scale, float softcap,
                        uint16_t *O, float *lse, void *ws, size_t ws_bytes, int32_t *dev_status, void *stream);

/*
 * vca_cache_weigh -- adds to weight, fp32 [pages][H][128], what each cached token
 * received from the rows Q: weight[page][h][slot] += sum over the rows i and the
 * G query heads of KV head h, where the token is visible, of exp(s_ij - lse_i),
 * with s, visibility and lse [T][Hq] those of vca_cache_attention.  A key's sum
 * over the rows of one sequence has a fixed order and is added once (weight is
 * 16-byte aligned); sequences that share a page add to it in any order.  A token's
 * weight starts at what its slot holds: vca_cache_append_ex makes that 0.
 */
int vca_cache_weigh(const vca_cache *cache, const uint16_t *Q, int64_t q_token, int64_t q_head, const int32_t *start,
                    int T, int Hq, int causal, float softmax_scale, float softcap, const float *lse, float *weight,
                    void *ws, size_t ws_bytes, int32_t *dev_status, void *stream);

/*
 * vca_cache_evict -- cuts every sequence to its min(len, budget) most useful
 * tokens, for each KV head on its own, into fresh pages.  The newest
 * min(recent, len) tokens stay; of the others those with the largest weight
 * (NaN counts as -inf, ties go to the lower slot).  What stays keeps its order;
 * kept int32 [B][H][budget] names the slots (entries behind the last one are
 * left as they are), new_len int32 [B] their number.  dst_table [B][dst_cols]
 * names the pages to write, in the same pool: ceil(new_len / 128) of each row
 * are read, each named once and none a page that `table` names (the cached
 * pages are only read, so they may be shared with other sequences).  A written
 * page gets the scale of its own values, as in vca_cache_append; weights move
 * with their tokens, and those of the slots behind the last one stay as they are.
 * Requires budget >= 1, 0 <= recent <= budget, dst_cols*128 >= budget; new_len and
 * dst_table are not the cache's own len and table (refused).  `len` is the cache's
 * as always; afterwards the sequence is the cache with dst_table and new_len.
 */
int vca_cache_evict(const vca_cache *cache, float *weight, const int32_t *dst_table, int dst_cols, int budget,
                    int recent, int32_t *new_len, int32_t *kept, int32_t *dev_status, void *stream);

/*
 * vca_cache_plan -- places for the new tokens of the cache's next call, from the
 * sequences' lengths: `held` int32 [B], the tokens of each sequence before (may be
 * `len` itself), and `news` int32 [B], how many arrive.
 *   table   the columns ceil(held / 128) .. ceil((held + news) / 128) - 1 of each
 *           sequence get pages, the lowest free ones in the order of the
 *           sequences and columns; other entries stay as they are
 *   len     held + news
 *   start   int32 [B + 1], the sums of news: it cuts the call's rows
 *   slot, position (int32 [T], each may be NULL): row t = start[b] + i is token
 *           position = held + i of its sequence, in slot = page * 128 + position
 *           % 128 of the pool (-1 where the page does not exist); those of rows
 *           behind start[B] stay as they are
 * Free is a page that no live table entry names, live being the columns below
 * ceil(held / 128): no list is kept, a length of 0 gives a sequence's pages back, and
 * a page that sequences share is free when the last of them is gone.  Only full
 * pages may be shared by sequences with news: new tokens of two that share a partly
 * filled last page get the same slots, which is not looked for (no page may be
 * written twice in a call); copy such a page first.  A live
 * entry outside 0 .. pages - 1 names none; it is reported where pages are given out.
 * A plan is made whole or not at all: if held or news is negative or their sum
 * above cols*128 anywhere, or the news sum up to more than T (dev_status =
 * VCA_ERR_INVALID_ARG), or the free pages are too few (VCA_ERR_FULL), start becomes
 * 0 throughout, so that its rows belong to nobody, and all else stays as it was.
 * Sizes: B <= 65,535, pages*128 and cols*128 <= 2^31 - 1, T >= 0.  news is not len, and
 * start none of len, held and news (refused);
 * no two of the arrays overlap but held and len.
 */
int vca_cache_plan(int32_t *table, int32_t *len, int pages, int B, int cols, const int32_t *held, const int32_t *news,
                   int32_t *start, int32_t *slot, int32_t *position, int T, int32_t *dev_status, void *stream);

/*
 * vca_cache_fresh -- the pages that vca_cache_evict writes: columns 0 ..
 * ceil(min(len, budget) / 128) - 1 of every row of dst_table int32 [B][dst_cols] get
 * free pages, as in vca_cache_plan with held = len; other entries stay as they
 * are.  Whole or not at all, likewise: dst_table is left as it was where a length
 * is out of range or the free pages are too few.  Requires budget >= 1 and
 * dst_cols*128 >= budget; dst_table is neither table nor len (refused).
 */
int vca_cache_fresh(const int32_t *table, const int32_t *len, int pages, int B, int cols, int budget, int32_t *dst_table,
                    int dst_cols, int32_t *dev_status, void *stream);

/*
 * vca_prompt_attention -- attention of packed prompts over their own keys and
 * values as they are, bf16, before they are quantised into the cache: Q [T][Hq][d],
 * K and V [T][H][d], d = 128, all three cut by start[B + 1]; query heads h*G .. h*G + G - 1
 * read KV head h, G = Hq / H.  Row i of a sequence's n:
 *   s_ij = softmax_scale q_i . k_j;  with softcap > 0: softcap tanh(s_ij / softcap)
 *   j visible to row i: j < n, and with causal = 1: j <= i
 *   O_i = sum_j softmax_j(s_ij) v_j,  lse_i = ln sum_j exp(s_ij)
 * With `prior` bf16 [T][Hq][d] and prior_lse fp32 [T][Hq], both contiguous (NULL:
 * none), the result is joined with an attention of the same rows over other tokens,
 * such as vca_cache_attention's over what the sequence held before the chunk:
 *   lse_i = ln(sum_j exp(s_ij) + exp(prior_lse_i)),
 *   O_i = (sum_j exp(s_ij) v_j + exp(prior_lse_i) prior_i) / exp(lse_i)
 * in fp32 with one rounding of O; where prior_lse is -inf, prior is not read.  O may be
 * prior, and lse prior_lse; other outputs must not overlap the inputs.
 * Scale, cap, start, rows behind start[B], O, lse, T = 0 and dev_status as in
 * vca_cache_attention.  Distances are multiples of 8 elements, above 0 and below 2^39,
 * between tokens where T > 1 and between heads where there are several; 0 between
 * the heads of K or V makes all of them one.  B*H <= 65,535, T*Hq <= 2^31 - 1.
 * The products of bf16 values are exact, sums and statistics fp32; the
 * probabilities enter the second product as bf16 (2^-8 relative); the magnitudes of a
 * sequence's values have to sum up to less than 2^128 a channel.  A NaN or an infinity
 * among the values of a sequence may reach every row of that sequence, one in a
 * key or query only the rows that see it.  A cap up to 64 adds an error of up to 2^-20 of
 * the cap to a score; a larger one, and any in vca_cache_attention, 2^-20 of the score.
 * Equal calls give equal bits.  No workspace.
 * The kernel's form is chosen on the host for the whole call, by T / B: with many
 * sequences without rows, or room for many more rows than there are, it is right and
 * up to a few percent slower (a prompt of 32,768 tokens: 5 and 2 %).
 */
int vca_prompt_attention(const uint16_t *Q, int64_t q_token, int64_t q_head, const uint16_t *K, int64_t k_token,
                         int64_t k_head, const uint16_t *V, int64_t v_token, int64_t v_head, const int32_t *start, int B,
                         int T, int Hq, int H, int d, int causal, float softmax_scale, float softcap,
                         const uint16_t *prior, const float *prior_lse, uint16_t *O, float *lse, int32_t *dev_status,
                         void *stream);

#ifdef __cplusplus
}
#endif

#endif /* VCA_H */

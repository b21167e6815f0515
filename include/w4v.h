/*
 * w4v.h -- C ABI of libw4v, the GB300 (sm_103a) speculative-decoding verify
 * step for a W4A16 target with an int8 lm_head.
 *
 * The operations follow the statement of the problem in "Efficient LLM
 * Challenge Results" (AdaptFM @ ICML 2026):
 *   - section 3 "Speculative decoding did the heavy lifting": a drafter
 *     proposes K tokens, the target runs all K+1 positions in one forward
 *     pass, and greedy verification keeps the longest draft prefix equal to
 *     the target's own tokens; drafts may be padded to a constant K with -1
 *     sentinels, which are never accepted (runner-up paragraph);
 *   - sections 3 and 5 "Quantization was common, but not the deciding lever":
 *     the target's projections are 4-bit W4A16 GPTQ with group size 128 and
 *     fp16 activations, and its untied lm_head is quantized to 8 bits;
 *   - section 2 "Where the time goes": decode is bound by reading the weights
 *     from HBM, so the K+1 positions share one weight read.
 * The pages give no interface; this one is the plainest that carries those
 * operations.
 *
 * Conventions (all entry points):
 *   - fp16 data is passed as uint16_t holding IEEE-754 binary16 bit patterns.
 *   - Matrices are dense row-major with the leading dimension equal to the
 *     row length given.  Device pointers must be 16-byte aligned.
 *   - The caller owns every buffer, including the workspace; no entry point
 *     allocates device memory.  A workspace must be zero-filled once before
 *     its first use; every call that returns W4V_OK leaves the parts that
 *     must start at zero (arrival counters, best-key slots) at zero again,
 *     so it can be reused by the next call on the same stream (scratch
 *     parts such as fp32 partial tiles keep whatever the last call wrote and
 *     are always written before they are read).
 *   - Calls are asynchronous on `stream` (NULL = legacy default stream).
 *     Argument, shape and alignment errors are returned before anything is
 *     launched.  A launch failure returns W4V_ERR_CUDA.  A kernel that gives
 *     up on an internal wait (bounded at about two seconds) records
 *     W4V_ERR_TIMEOUT in a device status word read by w4v_get_status(); after
 *     that the workspace must be zero-filled again.
 *   - Nothing here is thread-safe against concurrent use of the same
 *     workspace; distinct workspaces may be used concurrently.
 */
#ifndef W4V_H
#define W4V_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
/* A cudaStream_t. */
typedef struct CUstream_st *w4v_stream_t;

typedef enum {
    W4V_OK = 0,
    W4V_ERR_ARG = 1,        /* null pointer or invalid enum/flag            */
    W4V_ERR_SHAPE = 2,      /* unsupported sizes (see each entry point)     */
    W4V_ERR_ALIGN = 3,      /* pointer not 16-byte aligned                  */
    W4V_ERR_WORKSPACE = 4,  /* workspace missing or smaller than required   */
    W4V_ERR_ARCH = 5,       /* current device is not sm_103 (GB300)         */
    W4V_ERR_CUDA = 6,       /* CUDA runtime / launch error                  */
    W4V_ERR_TIMEOUT = 7     /* a kernel abandoned a bounded wait            */
} w4v_status;

/* Short English text for a status code (static storage, never NULL). */
const char *w4v_status_string(w4v_status status);

/* Checks that the current device is compute capability 10.3 and runs one
 * tiny kernel, so that a library built for another architecture fails here
 * rather than at the first real launch ("DFlash K=15 for Qwen3.5-4B on a
 * single A10G", section "What transfers": build for the card you run on).
 * Idempotent per device; every entry point calls it implicitly.  What it
 * finds (the SM count, the device status word's address) is kept per device
 * for the life of the process, so a process that resets a device
 * (cudaDeviceReset) must be restarted before it calls the library again. */
w4v_status w4v_init(void);

/* Synchronizes `stream`, then returns and clears the device status word of
 * the current device: W4V_OK, or what happened since the last call:
 * W4V_ERR_TIMEOUT if a kernel gave up a wait, else W4V_ERR_SHAPE if the arrays
 * that paged_attn (or _sinks, _shared) found on the device ask for more than its
 * arguments allow. */
w4v_status w4v_get_status(w4v_stream_t stream);

/* ------------------------------------------------------- int4 weight packing
 * The logical W4A16 weight is q[N][K], one 4-bit code (0..15) per byte, with
 * w[n][k] = s[k/G][n] * (q[n][k] - z) (z = 8, or a per-group zero table).
 * The device format is this library's own tile layout: N is split into tiles
 * of 128 rows (the last one zero-padded), K into groups of 128; every
 * (tile, group) block is 8192 contiguous bytes, blocks ordered tile-major.
 * Inside a block, 16-byte chunk j (j = 0..3, k = 32j..32j+31 of the group)
 * of row r sits at byte (j*128 + r)*16 and holds four little-endian 32-bit
 * words; word w covers k = 32j+8w .. +7 with nibble i holding the code of
 * k offset {0,2,4,6,1,3,5,7}[i].
 * Sizes: K % 128 == 0, N % 8 == 0, N, K > 0.  Host memory only. */
size_t w4v_packed_bytes(int N, int K);
w4v_status w4v_pack_int4(const uint8_t *q_host, int N, int K, void *packed_host_out);
/* Inverse of w4v_pack_int4 (rows >= N of the padded tile are dropped). */
w4v_status w4v_unpack_int4(const void *packed_host, int N, int K, uint8_t *q_host_out);

/* ------------------------------------------------------------- w4a16_gemm
 * C[M][N] = A[M][K] * W^T, W[n][k] = scales[k/G][n] * (q[n][k] - z[k/G][n]),
 * z = 8 when zeros == NULL (symmetric GPTQ) else the uint8 table
 * zeros[K/G][N] (values 0..15, AWQ style).  A, scales, C are fp16; products
 * are accumulated in fp32.  For M <= 32 (verify sizes, HBM-bound) with
 * G = 128 each group's fp32 sum is multiplied by its scale in fp32; for
 * M > 32 (prefill, tensor-bound), and for G = 32 at any M, the dequantized
 * weight s*(q-z) is rounded to fp16 once.  The whole K is accumulated in
 * fp32, and for M <= 32 the per-element arithmetic does not depend on M.
 * C is rounded to fp16 (round to nearest even).  G = 128 is the GPTQ
 * target of "Efficient LLM Challenge Results" sections 3 and 5; G = 32 is
 * the group size of the compressed-tensors W4A16 target listed there.
 *   A        device, fp16 [M][K]
 *   Bq       device, packed int4 from w4v_pack_int4 (w4v_packed_bytes(N,K);
 *            the packed layout does not depend on G)
 *   scales   device, fp16 [K/G][N]
 *   zeros    device, uint8 [K/G][N] or NULL (requires N % 16 == 0)
 *   group    G: 128 or 32
 *   C        device, fp16 [M][N] (written, never read)
 * Sizes: M >= 0 (M == 0 is a no-op), N % 8 == 0, K % 128 == 0.
 * Workspace: w4a16_workspace_bytes(M, N, K) bytes, zero-filled before first
 * use: fp32 partial sums of output tiles whose k range is split between
 * CTAs, and one arrival counter per tile.  About 1 MB for M <= 16 and 2 MB
 * for M <= 32; for M > 32, the larger of the 32-row size and 256 KB per
 * 128 x 256 output tile when there are at most 1024 tiles (the prefill
 * kernel may then split tiles in two k halves), plus 4 bytes per tile. */
size_t w4a16_workspace_bytes(int M, int N, int K);
w4v_status w4a16_gemm(const uint16_t *A, const void *Bq, const uint16_t *scales,
                      const uint8_t *zeros, int group, uint16_t *C, int M, int N, int K,
                      void *workspace, size_t workspace_bytes, w4v_stream_t stream);

/* w4a16_gemm with flags (w4a16_gemm is w4a16_gemm_ex with flags == 0).
 *   W4V_STATIC_WEIGHTS: Bq, scales and zeros are not written by any GPU
 *     work that may still be running when this call's kernel starts (the
 *     weights of a model during inference).  The verify-sized kernel then
 *     loads and dequantizes its first weight stages while the previous
 *     kernel of the stream is still finishing; A is still read, and C and
 *     the workspace still written, only after that kernel has completed.
 *     Without the flag the weights are only prefetched into L2 early.  The
 *     pages have no counterpart: it is a scheduling promise of the caller,
 *     the result is the same either way.
 *   W4V_BATCH_INVARIANT: for M > 32, run the rows in blocks of 32 through
 *     the verify-sized kernel (one launch per block, the weights read once
 *     per block) instead of the prefill kernel, so that every row of C is
 *     bit for bit the row a call with that row alone would give.  Greedy
 *     speculative decoding then emits exactly the tokens of plain greedy
 *     decoding also when several sequences' verify blocks share one call
 *     ("Efficient LLM Challenge Results", section 3: verification leaves the
 *     output unchanged whatever the drafts).  No effect for M <= 32, which
 *     is batch-invariant anyway.
 * Unknown flag bits: W4V_ERR_ARG. */
#define W4V_STATIC_WEIGHTS 1u
#define W4V_BATCH_INVARIANT 2u
w4v_status w4a16_gemm_ex(const uint16_t *A, const void *Bq, const uint16_t *scales,
                         const uint8_t *zeros, int group, uint16_t *C, int M, int N, int K,
                         void *workspace, size_t workspace_bytes, unsigned flags, w4v_stream_t stream);

/* ----------------------------------------------------- w4a16_gemm_grouped
 * Several independent W4A16 products C_i = A_i * W_i^T (each exactly as
 * w4a16_gemm defines it) in one launch.  Decode and verify read every weight
 * from HBM once per step ("Efficient LLM Challenge Results", section 2
 * "Where the time goes"), and a decoder layer's projections are a few MB
 * each: one launch per projection pays a start-up and a drain of the weight
 * stream that are comparable to its transfer time.  A grouped launch streams
 * the weights of every problem through one pipeline, with one start-up.
 * All problems share M (1..32, the verify-sized kernel), the group size and
 * whether they carry zero points.  Each output element is computed by the
 * same arithmetic for every M in 1..32 (batch invariance), but a grouped
 * launch splits the k ranges differently from a one-problem launch, so its
 * results may differ from w4a16_gemm in the last fp32 bits before the fp16
 * rounding; both are within the same error bound of the exact product.
 *
 * Use: w4a16_grouped_plan once for a fixed set of buffers (it encodes the
 * problems into `plan`, device memory of w4a16_grouped_plan_bytes(n) bytes,
 * 64-byte aligned, and fills the host handle), then w4a16_gemm_grouped per
 * step.  The plan holds the buffers' addresses: it stays valid while they
 * do, and must be rebuilt if any of them moves.
 *   problems[i].A       device, fp16 [M][K_i]
 *   problems[i].Bq      device, packed int4 of q_i [N_i][K_i] (w4v_pack_int4)
 *   problems[i].scales  device, fp16 [K_i/G][N_i]
 *   problems[i].zeros   device, uint8 [K_i/G][N_i] or NULL (all NULL or none;
 *                       with zero points N_i % 16 == 0)
 *   problems[i].C       device, fp16 [M][N_i] (written, never read)
 * Sizes: 1 <= n_problems <= 4096, 1 <= M <= 32, G = 128 or 32,
 * N_i % 8 == 0, K_i % 128 == 0, N_i, K_i > 0.
 * w4a16_grouped_plan copies the table to the device and waits for the copy
 * (it synchronizes `stream`), so it must not be called while `stream` is
 * being captured into a graph (W4V_ERR_ARG); w4a16_gemm_grouped only
 * launches and may be captured.  A handle not written by w4a16_grouped_plan,
 * or changed since, is refused with W4V_ERR_ARG.
 * Workspace: w4a16_grouped_workspace_bytes(handle) bytes, zero-filled before
 * first use (fp32 partial tiles and one arrival counter per output tile).
 * Flags: W4V_STATIC_WEIGHTS as for w4a16_gemm_ex. */
typedef struct {
    const uint16_t *A;
    const void *Bq;
    const uint16_t *scales;
    const uint8_t *zeros;
    uint16_t *C;
    int N, K;
} w4a16_problem;

/* Filled by w4a16_grouped_plan; read-only for the caller. */
typedef struct {
    const void *plan;       /* the device table this handle describes */
    long long units;        /* work units of one launch */
    int n_problems, M, group, has_zeros, tiles;
    unsigned check;         /* consistency tag */
} w4a16_grouped_t;

size_t w4a16_grouped_plan_bytes(int n_problems);
w4v_status w4a16_grouped_plan(const w4a16_problem *problems, int n_problems, int M, int group, void *plan,
                              size_t plan_bytes, w4a16_grouped_t *handle, w4v_stream_t stream);
size_t w4a16_grouped_workspace_bytes(const w4a16_grouped_t *handle);
w4v_status w4a16_gemm_grouped(const w4a16_grouped_t *handle, void *workspace, size_t workspace_bytes,
                              unsigned flags, w4v_stream_t stream);

/* ------------------------------------------------------- w8_lmhead_argmax
 * Greedy token per row: argmax_out[r] = argmax_v scale[v] * sum_k X[r][k]*W[v][k],
 * int8 weights, one fp16 scale per vocabulary row, fp32 accumulation with
 * the scale applied to the finished sum.  Ties go to the lowest v; a NaN
 * logit counts as -inf; -0 equals +0.  Full logits are never written unless
 * logits_debug is given.
 *   X              device, fp16 [M][K]
 *   W              device, int8 [V][K]
 *   scale          device, fp16 [V]
 *   argmax_out     device, int32 [M]
 *   maxlogit       device, float [M] or NULL: the winning logit
 *   logits_debug   device, float [M][V] or NULL: every logit (testing aid)
 * Sizes: 0 <= M <= 128, K % 128 == 0, V % 8 == 0, V > 0.
 * Workspace: w8_lmhead_argmax_workspace_bytes(M, V) bytes, zero-filled
 * before first use (one best key per row and an arrival counter). */
size_t w8_lmhead_argmax_workspace_bytes(int M, int V);
w4v_status w8_lmhead_argmax(const uint16_t *X, const int8_t *W, const uint16_t *scale,
                            int M, int K, int V, int32_t *argmax_out, float *maxlogit,
                            float *logits_debug, void *workspace, size_t workspace_bytes,
                            w4v_stream_t stream);

/* w8_lmhead_argmax with flags (w8_lmhead_argmax is this with flags == 0).
 *   W4V_BATCH_INVARIANT: for M > 32, run the rows in blocks of 32 (one launch
 *     each, the weights read once per block), so that every row's logits and
 *     token are bit for bit those of a call with that row alone.  Up to 32
 *     rows every logit comes from the same arithmetic whatever M is; a
 *     single launch over more rows sums each logit in another order (within
 *     the same fp32 error bound), which may flip a token between two logits
 *     that close.  Several sequences' verify blocks in one call then accept
 *     exactly the tokens each would accept alone ("Efficient LLM Challenge
 *     Results", section 3: greedy verification leaves the output unchanged).
 * Unknown flag bits: W4V_ERR_ARG.  Other arguments as w8_lmhead_argmax. */
w4v_status w8_lmhead_argmax_ex(const uint16_t *X, const int8_t *W, const uint16_t *scale,
                               int M, int K, int V, int32_t *argmax_out, float *maxlogit,
                               float *logits_debug, void *workspace, size_t workspace_bytes,
                               unsigned flags, w4v_stream_t stream);

/* ---------------------------------------------- w8_lmhead_argmax_noalloc
 * The paper has no counterpart to this entry point; it exists for callers
 * that cannot allocate device memory for a workspace -- for example a plugin
 * running inside another inference engine whose execute step may not
 * allocate, or a serving loop whose device memory is already handed out by
 * its own allocator (cudaMalloc would also synchronize the device in the
 * middle of a decode step).  It computes exactly what w8_lmhead_argmax
 * computes, with the same arguments minus the workspace: the scratch lives
 * in a 4 KB device array inside this library, which every GPU that loads the
 * library keeps until the process exits.
 *   - Allocates nothing: no cudaMalloc, no cudaFree, no allocating library
 *     call.  It clears the scratch with an asynchronous memset on `stream`
 *     before each launch.  That memset sits between the previous kernel on
 *     the stream and the lm_head, so the lm_head's programmatic launch no
 *     longer overlaps its set-up with the previous kernel's end (the
 *     workspace entry keeps that overlap; the kernel itself leaves the
 *     scratch cleared on success, and the memset covers a call that gave
 *     up a bounded wait).
 *   - The first call on a device looks up that device's address of the
 *     array (cudaGetSymbolAddress with the device current) and keeps it for
 *     the life of the process; make that first call outside any stream
 *     capture.  After cudaDeviceReset (or anything else that unloads the
 *     library's module from a device) the kept address is stale: restart
 *     the process before calling this entry point again, as for the
 *     library's other per-device state (w4v_init).
 *   - Every call on a device shares the one array: calls that overlap on the
 *     GPU (different streams without ordering between them) race and give
 *     wrong tokens.  Serialize them, or use w8_lmhead_argmax with a
 *     workspace per stream.
 *   - Sizes: 0 <= M <= 128 (the array holds the keys of at most 128 rows);
 *     larger M returns W4V_ERR_SHAPE.  Other sizes as w8_lmhead_argmax. */
w4v_status w8_lmhead_argmax_noalloc(const uint16_t *X, const int8_t *W, const uint16_t *scale,
                                    int M, int K, int V, int32_t *argmax_out, float *maxlogit,
                                    float *logits_debug, w4v_stream_t stream);

/* --------------------------------------------------------- token_logprobs
 * What the target thinks of given tokens, from its logits (for instance those
 * that w8_lmhead_argmax writes): drafts and prompts are scored, continuations
 * ranked by it.  With z_v = x_v / temperature over a row of V logits x and
 * lse = ln sum_v exp(z_v),
 *     logprobs[r][i]     = z_t - lse, t = tokens[r][i] (-inf for a token
 *                          outside [0, V), such as the -1 of a padded draft);
 *     entropy[r]         = lse - sum_v p_v z_v, p_v = exp(z_v - lse);
 *     top_ids[r][j],     = the j-th largest logit's token and its log
 *     top_logprobs[r][j]   probability, of equal logits the lower token first.
 * Arithmetic is fp32, and the sums' error does not grow with V.  Logits of -inf
 * are tokens that cannot follow (p = 0); a row of nothing else gives logprobs of
 * -inf and an entropy of 0.  A row that holds a NaN or +inf gives NaN for every
 * token in [0, V) and for the entropy; its top_ids count NaN as -inf, as the
 * argmax does.  Logits further apart than fp32's largest number count as
 * infinitely far, whatever the temperature.
 *   logits        device, float rows of V logits (fp16 with W4V_LOGITS_FP16),
 *                 row_stride >= V elements apart; any address that is a
 *                 multiple of the element's size
 *   tokens        device, int32 [M][n] (may be NULL when n == 0)
 *   logprobs      device, float [M][n] (may be NULL when n == 0)
 *   entropy       device, float [M] or NULL
 *   top_ids       device, int32 [M][top] (may be NULL when top == 0)
 *   top_logprobs  device, float [M][top] (may be NULL when top == 0)
 * Sizes: 0 <= M <= 2^24 (0 is a no-op), 1 <= V <= 2^28, 0 <= n <= 2^20,
 * 0 <= top <= 32 and at most V, temperature > 0 and finite (as is its
 * reciprocal times log2 e).  No workspace. */
#define W4V_LOGITS_FP16 16u
w4v_status token_logprobs(const void *logits, long long row_stride, int M, int V, const int32_t *tokens, int n,
                          float temperature, float *logprobs, float *entropy, int top, int32_t *top_ids,
                          float *top_logprobs, unsigned flags, w4v_stream_t stream);

/* ----------------------------------------------------------- spec_accept
 * Longest-prefix greedy acceptance for B sequences:
 *   n[b] = the largest j <= K with draft[b][i] == target[b][i] for all i < j,
 * where a negative draft (the -1 padding sentinel) never matches.  The
 * emitted tokens are target[b][0..n[b]] (= drafts 0..n-1 then the target's
 * own next token); out_tokens[b][j] = target[b][j] for j <= n[b], else -1.
 *   target      device, int32 [B][K+1]: the target's greedy token after
 *               each verify position (row b*(K+1)+j of the verify block)
 *   draft       device, int32 [B][K] (may be NULL when K == 0)
 *   n_accepted  device, int32 [B]
 *   out_tokens  device, int32 [B][K+1] or NULL
 * Sizes: B >= 0 (0 is a no-op), 0 <= K <= 1024. */
w4v_status spec_accept(const int32_t *target, const int32_t *draft, int B, int K,
                       int32_t *n_accepted, int32_t *out_tokens, w4v_stream_t stream);

/* ----------------------------------------------- w8_lmhead_argmax_accept
 * The last two operations of a verify step in one launch: the int8 lm_head
 * argmax of w8_lmhead_argmax over M = B*(n_draft+1) rows, then the greedy
 * acceptance of spec_accept with target = those tokens viewed as
 * [B][n_draft+1] (row b*(n_draft+1)+j is position j of verify block b).
 * Results are identical to w8_lmhead_argmax followed by spec_accept; the
 * acceptance runs in the lm_head's last CTA, on the tokens it has just
 * written, so no second launch or dependency is needed.
 *   X, W, scale, argmax_out, maxlogit, workspace: as w8_lmhead_argmax
 *   draft       device, int32 [B][n_draft] (may be NULL when n_draft == 0)
 *   n_accepted  device, int32 [B]
 *   out_tokens  device, int32 [B][n_draft+1] or NULL (as spec_accept)
 * Sizes: B >= 0 (0 is a no-op), n_draft >= 0, B*(n_draft+1) <= 128,
 * K % 128 == 0, V % 8 == 0, V > 0.  Workspace: w8_lmhead_argmax_workspace_bytes
 * for M = B*(n_draft+1). */
w4v_status w8_lmhead_argmax_accept(const uint16_t *X, const int8_t *W, const uint16_t *scale,
                                   int B, int n_draft, int K, int V, const int32_t *draft,
                                   int32_t *argmax_out, int32_t *n_accepted, int32_t *out_tokens,
                                   float *maxlogit, void *workspace, size_t workspace_bytes,
                                   w4v_stream_t stream);

/* w8_lmhead_argmax_accept with flags (the plain entry point is this with
 * flags == 0).  W4V_BATCH_INVARIANT: for M = B*(n_draft+1) > 32, the argmax
 * runs as in w8_lmhead_argmax_ex with that flag (blocks of 32 rows) and the
 * acceptance follows in one more launch; the results are those of
 * w8_lmhead_argmax_ex followed by spec_accept.  Unknown flag bits:
 * W4V_ERR_ARG. */
w4v_status w8_lmhead_argmax_accept_ex(const uint16_t *X, const int8_t *W, const uint16_t *scale,
                                      int B, int n_draft, int K, int V, const int32_t *draft,
                                      int32_t *argmax_out, int32_t *n_accepted, int32_t *out_tokens,
                                      float *maxlogit, void *workspace, size_t workspace_bytes,
                                      unsigned flags, w4v_stream_t stream);

/* ------------------------------------------------------------ ngram_draft
 * Model-free drafts by prompt lookup ("Efficient LLM Challenge Results",
 * section 3, table of drafting methods: n-gram / prompt-lookup drafting
 * copies spans from the prompt; the runner-up pads drafts to a constant K
 * with -1).  For row b of `context`, c[0..L-1] with L = lengths[b] (values
 * outside [0, ld] are clamped to it): for n from n_max down to n_min, the
 * n-gram is c[L-n..L-1]; its latest earlier occurrence is the largest p with
 * p + n <= L - 1 and c[p+i] == c[L-n+i] for i < n.  The first n with an
 * occurrence gives drafts[b][i] = c[p+n+i] while p+n+i < L, else -1, and
 * match_len[b] = n; with none, every draft is -1 and match_len[b] = 0.
 *   context    device, int32 [B][ld] (tokens past a row's length are ignored)
 *   lengths    device, int32 [B]
 *   drafts     device, int32 [B][K] (may be NULL when K == 0)
 *   match_len  device, int32 [B] or NULL
 * Sizes: 0 <= B <= 65535 (0 is a no-op), ld >= 1, 1 <= n_min <= n_max <= 64,
 * 0 <= K <= 1024.  Workspace: ngram_draft_workspace_bytes(B) bytes,
 * zero-filled before first use (one best key and one arrival counter per
 * row). */
size_t ngram_draft_workspace_bytes(int B);
w4v_status ngram_draft(const int32_t *context, const int32_t *lengths, int B, int ld, int n_min,
                       int n_max, int K, int32_t *drafts, int32_t *match_len,
                       void *workspace, size_t workspace_bytes, w4v_stream_t stream);

/* --------------------------------------------------- gdn_verify / gdn_commit
 * The Gated DeltaNet recurrent state across a verify block, rolled back
 * under rejection.  Most of the target's layers are Gated DeltaNet, and a
 * rejected draft must not leave its update in their state ("Efficient LLM
 * Challenge Results", section 3, runner-up paragraph; "DFlash K=15 for
 * Qwen3.5-4B on a single A10G", "What transfers").  Per sequence b and head
 * h, with the recurrence of the first page's reference [12]:
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
 *     o_t = S_t q_t,
 * S the state [dv][dk] (row i = value index, column j = key index).
 * gdn_verify runs the T positions of a verify block from the committed state
 * and writes o_t for every t; it never writes the state.  gdn_commit then
 * advances the committed state in place by positions 0..n_accepted[b] of the
 * block (the last context token and the accepted drafts; n is clamped to
 * [0, T-1]), so the rejected positions leave no trace.  Keys and queries are
 * used as given (Gated DeltaNet normalises them to unit length upstream).
 *   state       device, fp32 [B][H][dv][dk] (read by gdn_verify, read and
 *               written by gdn_commit)
 *   q, k        device, fp16 [B][T][H][dk]  (gdn_commit takes no q)
 *   v           device, fp16 [B][T][H][dv]
 *   alpha, beta device, fp32 [B][T][H]
 *   o           device, fp16 [B][T][H][dv] (written; fp32 arithmetic inside)
 *   n_accepted  device, int32 [B] (as written by spec_accept or
 *               w8_lmhead_argmax_accept)
 * Sizes: 0 <= B <= 65535 (0 is a no-op), 1 <= T <= 64, 1 <= H <= 65535,
 * dk == 128, dv a multiple of 32 up to 4096.  No workspace. */
w4v_status gdn_verify(const float *state, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                      const float *alpha, const float *beta, int B, int T, int H, int dk, int dv,
                      uint16_t *o, w4v_stream_t stream);
w4v_status gdn_commit(float *state, const uint16_t *k, const uint16_t *v, const float *alpha,
                      const float *beta, const int32_t *n_accepted, int B, int T, int H, int dk,
                      int dv, w4v_stream_t stream);

/* gdn_step: the commit of the previous block and the verify of the next one
 * in one launch, reading and writing the state once: the state is advanced
 * by positions 0..n_prev[b] of the previous block (k_prev, v_prev,
 * alpha_prev, beta_prev over T_prev positions; n clamped as in gdn_commit)
 * and written back, then o_t of the current block is produced from it, with
 * the same arithmetic as gdn_commit followed by gdn_verify (bit for bit).
 * T_prev = 0 means no previous block (the *_prev pointers and n_prev are
 * then ignored and the state is not written).  Arrays, layouts and limits as
 * above, 0 <= T_prev <= 64. */
w4v_status gdn_step(float *state, const uint16_t *k_prev, const uint16_t *v_prev,
                    const float *alpha_prev, const float *beta_prev, const int32_t *n_prev, int T_prev,
                    const uint16_t *q, const uint16_t *k, const uint16_t *v, const float *alpha,
                    const float *beta, int B, int T, int H, int dk, int dv, uint16_t *o,
                    w4v_stream_t stream);

/* ------------------------------------------------- paged key/value cache --
 * What follows serves the target's softmax-attention layers, which a hybrid
 * target has next to its recurrent ones.  The pages give no layout; this is
 * the library's own.
 *
 * One layer's cache is two device arrays of pages, k and v, each fp16
 * [n_pages][kv_heads][page][head_dim]; a page holds `page` consecutive tokens
 * of one sequence.  Row b of `table` lists sequence b's pages in token order
 * (token p lies in page table[b][p / page], slot p % page); entries past the
 * sequence's last page are never read.  lengths[b] counts the sequence's
 * cached tokens INCLUDING the new ones of the call, and offsets[b] ..
 * offsets[b+1]-1 are the rows of q, k, v that hold its new tokens (none when
 * the two are equal), so new row offsets[b] + i of n sits at position
 * lengths[b] - n + i.  A block of K+1 verified positions, one decoded token
 * and a chunk of a prompt are all this one form, mixed freely in a batch.
 *   - head_dim 64, 128 or 256; page a power of two, 8 to 256; kv_heads >= 1;
 *     table_width * page < 2^31; n_pages * kv_heads * page < 2^34.
 *   - The device arrays are read as they are: a length is clamped to
 *     [0, table_width * page], an offset to [0, n_tokens], and a page id
 *     outside [0, n_pages) is never followed (a read gives zeros, a write is
 *     dropped).  Offsets should not decrease: a row that several sequences
 *     name gets the result of one of them.
 *   - table, lengths and offsets are int32 on the device, so a captured
 *     graph can be replayed while they change. */
typedef struct {
    uint16_t *k, *v;
    const int32_t *table;      /* [B][table_width] */
    const int32_t *lengths;    /* [B]              */
    const int32_t *offsets;    /* [B+1]            */
    int B, table_width, n_pages, kv_heads, page, head_dim;
} w4v_kv_t;

/* ------------------------------------------------------------ rope_append
 * Rotary positions, and the new tokens' keys and values into the cache.
 * With phi_i = p f_i at position p, pair i of the first `rot` elements of
 * every query and key head becomes
 *     (x_a, x_b) -> mul (x_a cos phi_i - x_b sin phi_i,
 *                        x_b cos phi_i + x_a sin phi_i),
 * (a, b) = (i, i + rot/2), or (2i, 2i+1) with W4V_ROPE_INTERLEAVED; elements
 * from rot on and the values are copied.  Arithmetic is fp32, rounded to
 * fp16 once.  Rotated queries go to q_out, keys and values to their pages.
 *   q, k, v     device, fp16 rows of q_heads / kv_heads / kv_heads heads of
 *               head_dim elements; *_stride elements from row to row (a
 *               multiple of 8, so the three may be slices of one projection's
 *               output)
 *   positions   device, int32 [n_tokens] or NULL: the rotation's position of
 *               each row where it is not the cache position
 *   phases      device, uint64 [rot/2]: the fraction of a full turn that one
 *               position adds to pair i, times 2^64 (rope_phases).  p * phase
 *               mod 2^64 is exact, so no position is too long.
 *   q_out       device, fp16 [n_tokens][q_heads][head_dim]; may be q itself
 *               where q is dense
 * A row that no sequence's offsets cover is left alone.
 * Sizes: n_tokens >= 0 (0 is a no-op), q_heads >= 1, rot even,
 * 0 <= rot <= head_dim. */
#define W4V_ROPE_INTERLEAVED 4u
w4v_status rope_append(const w4v_kv_t *kv, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                       long long q_stride, long long k_stride, long long v_stride, int n_tokens, int q_heads,
                       const int32_t *positions, const uint64_t *phases, int rot, float mul, unsigned flags,
                       uint16_t *q_out, w4v_stream_t stream);

/* rope_append for targets that norm their queries and keys: every query and
 * key head x (all head_dim elements) first becomes
 *     x / sqrt(mean(x^2) + eps) * (w + c),
 * w = q_weight or k_weight (device, fp16 [head_dim]; NULL: all factors 1),
 * c = 0, or 1 with W4V_NORM_ZERO_CENTRED (weights kept around zero; no
 * meaning where the weights are NULL), and is then rotated and written as
 * above; nothing is rounded in between.  eps >= 0 and finite; with eps = 0 a
 * head of zeros gives NaN.  Values are not normed.  A row's results do not
 * depend on the call's other rows, bit for bit.  Everything else as
 * rope_append. */
#define W4V_NORM_ZERO_CENTRED 8u
w4v_status norm_rope_append(const w4v_kv_t *kv, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                            long long q_stride, long long k_stride, long long v_stride, int n_tokens, int q_heads,
                            const uint16_t *q_weight, const uint16_t *k_weight, float eps,
                            const int32_t *positions, const uint64_t *phases, int rot, float mul, unsigned flags,
                            uint16_t *q_out, w4v_stream_t stream);

/* Host only: phases and mul of a base and a scaling for long contexts.
 * f_i = base^(-2i/rot), then
 *   W4V_ROPE_PLAIN    as it is;
 *   W4V_ROPE_LINEAR   f_i / factor                       params = {factor}
 *   W4V_ROPE_NTK      base * factor^(rot/(rot-2)) for base       {factor}
 *   W4V_ROPE_YARN     f_i / factor for slow pairs, f_i for fast ones, a ramp
 *                     over the pair index between the pairs that turn
 *                     `slow` and `fast` times in `context` tokens;
 *                     mul = 0.1 ln(factor) + 1      {factor, context, fast, slow}
 *   W4V_ROPE_BANDED   the same by a ramp over the turns themselves, from
 *                     `low` to `high`               {factor, low, high, context}
 * mul is 1 where not stated.  params holds 4 doubles (NULL for PLAIN). */
typedef enum {
    W4V_ROPE_PLAIN = 0, W4V_ROPE_LINEAR = 1, W4V_ROPE_NTK = 2, W4V_ROPE_YARN = 3, W4V_ROPE_BANDED = 4
} w4v_rope_scaling;
w4v_status rope_phases(int rot, double base, int scaling, const double *params, uint64_t *phases_out,
                       float *mul_out);

/* ------------------------------------------------------------- paged_attn
 * Causal attention of the new tokens over the cache that holds them:
 *     o_t = sum_j softmax_j(scale q_t . k_j) v_j   over p_t - window < j <= p_t
 * (window 0: every j <= p_t), p_t the row's position, query head h reading
 * key/value head h / (q_heads / kv_heads).  Scores, softmax statistics and
 * sums are fp32; the weights enter the product with v as fp16, scaled by 2^8
 * or more: each is off by at most 2^-11 of itself (from 2^-22 of the largest
 * on) or 2^-33 of the largest.  A row that sees no token gives zeros and
 * lse = -inf; a row that no sequence's offsets cover is left alone, in out and
 * in lse.  What the cache holds past a sequence's length is never used.
 *   q      device, fp16 rows of q_heads heads, q_stride elements apart
 *   out    device, fp16 [n_tokens][q_heads][head_dim] (written, never read)
 *   lse    device, float [n_tokens][q_heads] or NULL:
 *          ln sum_j exp(scale q_t . k_j)
 * Sizes: n_tokens >= 0 (0 is a no-op), q_heads a multiple of kv_heads and at
 * most 128 times as many, scale > 0 and finite, window >= 0, and
 * (n_tokens / tok + min(B, n_tokens)) * kv_heads * (table_width * page / 128
 * + 5) < 2^31 with tok = 128 / (q_heads / kv_heads).  Offsets on the device
 * that name rows again and again, for more work than that or than the workspace
 * holds: nothing is written, and w4v_get_status returns W4V_ERR_SHAPE.
 * W4V_BATCH_INVARIANT: each row's result is bit for bit the same whatever
 * rows and sequences share the call and however many new tokens come with
 * it, so verified positions equal the one-token steps they stand for.  The
 * table's size does count: a context is summed in parts of 512 tokens where
 * table_width * page is at most 16,384, of 1024 up to 32,768, and so on in
 * doublings.  Calls that are to agree need tables of one such class: keep one
 * width rather than trimming it to each batch.
 * Without it the contexts are cut where that balances the GPU.
 * Workspace: paged_attn_workspace_bytes(...) with the call's own n_tokens and
 * B or larger ones, max_context = table_width * page; zero-filled before
 * first use.  With W4V_BATCH_INVARIANT it grows with the number of rows times
 * up to 32 pieces of the context, so a long prompt goes through in chunks. */
size_t paged_attn_workspace_bytes(int n_tokens, int B, int q_heads, int kv_heads, int head_dim, int max_context,
                                  unsigned flags);
w4v_status paged_attn(const w4v_kv_t *kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads,
                      float scale, int window, uint16_t *out, float *lse, void *workspace,
                      size_t workspace_bytes, unsigned flags, w4v_stream_t stream);

/* paged_attn with a window and a few first tokens of every sequence that
 * stay visible (the system's prompt, or the tokens that a model lets idle
 * attention rest on): row t sees the keys j <= p_t with
 *     j > p_t - window  or  j < sinks.
 * What lies between is not read.  Keys are attended as they lie in the cache,
 * so positions are those that rope_append wrote them with.  sinks >= 0; with
 * sinks == 0 or window == 0 (every token visible) this is paged_attn.  All
 * else, W4V_BATCH_INVARIANT and the workspace among it, as paged_attn. */
w4v_status paged_attn_sinks(const w4v_kv_t *kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads,
                            float scale, int window, int sinks, uint16_t *out, float *lse, void *workspace,
                            size_t workspace_bytes, unsigned flags, w4v_stream_t stream);

/* paged_attn (without a window) for sequences that share a prefix, whose keys
 * and values are then read once for all of them: continuations of one prompt,
 * as kv_fork leaves them, requests behind one system prompt.  Group g is the
 * batch's sequences groups[g] .. groups[g+1]-1, and the first prefix[g] tokens
 * of each are the same; they are read from the pages of the group's first
 * sequence, in whole pages and in the partly filled one behind them (which
 * kv_fork copies).  The rows' results are those of paged_attn up to the order
 * of the sums.
 *   groups  device, int32 [n_groups + 1], not decreasing; sequences outside
 *           [groups[0], groups[n_groups]) share nothing
 *   prefix  device, int32 [n_groups]
 * The device arrays are read as they are: a group whose first sequence holds
 * fewer than prefix[g] tokens shares nothing (so when a group's first sequence
 * ends, begin the group behind it), and neither does a sequence with fewer
 * than prefix[g] tokens before its new ones; those attend over their own pages.
 * Sequences without new tokens may lie anywhere in a group.
 * A row that several sequences name gets no meaningful result.
 * When to use it: where several sequences of a group bring few rows each (well
 * under tok = 128 / (q_heads / kv_heads)) and the prefix is long.  On this GPU it
 * is faster than paged_attn from about 16 one-token sequences over a prefix of
 * 2000 tokens, 8 over 8000 or 4 over 32,000 on (64 over 32,000: seven times),
 * slower by up to 5 us below, and slower by half for prompt chunks, whose rows
 * fill tiles by themselves: those belong in paged_attn.
 * flags must be 0 (how a row's sum is cut depends on the batch).  Sizes as
 * paged_attn, 0 <= n_groups <= B (a group may be empty), and (2 (n_tokens / tok) + min(B,
 * n_tokens) + min(n_groups, n_tokens)) * kv_heads * (table_width * page / 128
 * + 5) < 2^31.
 * Workspace: paged_attn_shared_workspace_bytes(...) with the call's own
 * n_tokens or a larger one, zero-filled before first use; it holds two results
 * of each row in 32 bits. */
size_t paged_attn_shared_workspace_bytes(int n_tokens, int B, int n_groups, int q_heads, int kv_heads, int head_dim);
w4v_status paged_attn_shared(const w4v_kv_t *kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads,
                             float scale, const int32_t *groups, const int32_t *prefix, int n_groups, uint16_t *out,
                             float *lse, void *workspace, size_t workspace_bytes, unsigned flags, w4v_stream_t stream);

/* ------------------------------------------------------------ kv_* pages --
 * Bookkeeping of the pages, on the device (the accepted lengths that drive
 * it are there).  A page id stands for that page of every plane: pool is
 * [planes][n_pages][page_bytes], for instance layer l's k in plane 2l and v
 * in plane 2l+1.  refs[p] counts the sequences that hold page p (0: free).
 * Free pages are handed out lowest id first, to sequences in ascending order.
 *   pool     device, page_bytes a multiple of 16 (only what copies needs it)
 *   refs     device, int32 [n_pages]
 *   table    device, int32 [S][table_width]; entries past a row's last page
 *            are -1 once one of these calls has dropped or forked the row
 *   lengths  device, int32 [S]
 * Sizes: 1 <= n_pages <= 2^24, 0 <= S <= 65535 (0 is a no-op),
 * table_width >= 1, page a power of two, 8 to 256, table_width * page < 2^31.
 * Workspace: kv_workspace_bytes(n_pages, S), or more; it needs no clearing, and
 * one may serve pools and batches of different sizes in turn. */
typedef struct {
    void *pool;
    int32_t *refs, *table, *lengths;
    size_t page_bytes;
    int planes, n_pages, S, table_width, page;
} w4v_pages_t;
size_t kv_workspace_bytes(int n_pages, int S);

/* Pages for new_lengths[s] >= lengths[s] tokens (a smaller one changes
 * nothing).  A last page that is partly filled and shared is first replaced
 * by a copy of its own, so that appending never touches another sequence.
 * All or nothing: *short_out (device) is 0, or the number of pages that are
 * missing, or -1 if a new length does not fit its table row; then nothing is
 * changed. */
w4v_status kv_extend(const w4v_pages_t *pages, const int32_t *new_lengths, int32_t *short_out, void *workspace,
                     size_t workspace_bytes, w4v_stream_t stream);

/* Lengths down to new_lengths[s] (a larger one changes nothing, a negative
 * one counts as 0); pages that are no longer needed lose one reference, and
 * are free when none is left.  Rolls back rejected drafts; 0 ends a sequence.
 * No workspace; pool is not used. */
w4v_status kv_truncate(const w4v_pages_t *pages, const int32_t *new_lengths, w4v_stream_t stream);

/* Sequence children[i] becomes a copy of parents[i]: full pages are shared,
 * a partly filled last page is copied.  Children must be empty, named once
 * and no parents.  *short_out: 0, the number of pages that are missing, or -1
 * for an index outside [0, S) or such a child; then nothing is changed.
 * 0 <= n <= S. */
w4v_status kv_fork(const w4v_pages_t *pages, const int32_t *parents, const int32_t *children, int n,
                   int32_t *short_out, void *workspace, size_t workspace_bytes, w4v_stream_t stream);

/* Live pages at or above their count move, in ascending order, to the free
 * pages below it, in ascending order, so that all live pages come first.
 * refs_out / table_out get the new counts and tables; they may be the old
 * arrays.  Moved pages keep their old contents until they are handed out
 * again, so a step in flight may finish on the old tables. */
w4v_status kv_compact(const w4v_pages_t *pages, int32_t *refs_out, int32_t *table_out, void *workspace,
                      size_t workspace_bytes, w4v_stream_t stream);

/* Contents of page src[i] to page dst[i] in every plane, i < n (device int32;
 * a pair with an id outside [0, n_pages) is skipped).  No page of dst may be
 * named twice or be in src. */
w4v_status kv_copy(void *pool, int planes, int n_pages, size_t page_bytes, const int32_t *src,
                   const int32_t *dst, int n, w4v_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* W4V_H */

/*
 * w4a16.h - C ABI of the GB300 (sm_103a) int4 weight-only affine linear layer.
 *
 * The operation: a linear layer Y = X * W^T whose weight W[N][K] is stored as
 * 4-bit codes q in 0..15 with one binary16 scale and one binary16 bias per
 * group of G consecutive k (G = 64 by default), so that
 *     w[n][k] = scale[n][k/G]*q[n][k] + bias[n][k/G]          (affine), or,
 *     w[n][k] = scale[n][k/G]*(q[n][k] - 8)                   (symmetric),
 * when the weight has no biases.  Sources (page title, section):
 *   "The inference engine - Mojo 1.0 on Metal", "Crossing Mojo 1.0": decode
 *     is a weight-streaming multi-row GEMV plus on-device token selection;
 *     prefill dequantises each weight once into a transposed half-precision
 *     scratch and runs a half-precision GEMM.
 *   same page, "What's inside the engine today": int4 projections and LM
 *     head; greedy and top-k selection on the device.
 *   "engine-mlx", "Tech details": MLX 4-bit quantised format.
 *   "Engineering investigation ... 10x faster?", "Selective quantization":
 *     affine quantisation with group size 64.
 *   "The inference engine - Mojo 1.0 on Metal", "What's inside the engine
 *     today" and the appendix on porting MLX's kernels: that engine's own
 *     weights are symmetric int4 with group 128 (scale only).
 *
 * Storage format (shared by every call):
 *   qweight  uint32 [N][K/8], row-major.  Word j of row n holds q[n][8j+i]
 *            in bits 4i..4i+3 (lowest nibble = lowest k).
 *   scales   binary16 [N][K/G], row-major.
 *   biases   binary16 [N][K/G], row-major; NULL selects symmetric codes.
 *   group    G, a power of two with 32 <= G <= K and K % G == 0 (every call
 *            that takes `group`; 64 is the affine format above, 128 with
 *            NULL biases the symmetric group-128 format).
 *   Activations and outputs are binary16 (IEEE half, passed as uint16_t bit
 *   patterns), row-major.
 *
 * Conventions:
 *   - Every pointer is a DEVICE pointer on the current CUDA device, owned by
 *     the caller.  The library allocates no device memory and keeps no
 *     per-call state.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call
 *     only enqueues work and returns before it completes.
 *   - The return value is a status code (W4A16_OK = 0).  All argument checks
 *     happen on the host before anything is enqueued; a failing check
 *     enqueues nothing.  W4_ERR_LAUNCH reports a launch error from the CUDA
 *     runtime.  No kernel traps.
 *   - Pointers must be 16-byte aligned.
 */
#ifndef W4A16_H
#define W4A16_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define W4A16_API __attribute__((visibility("default")))
#else
#define W4A16_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define W4A16_OK          0
#define W4_ERR_NULL       1  /* a required pointer is NULL */
#define W4_ERR_SHAPE      2  /* a dimension is out of the supported range */
#define W4_ERR_ALIGN      3  /* a pointer or row stride is not 16-byte aligned */
#define W4_ERR_GROUP      4  /* group not a power of two in 32..K dividing K */
#define W4_ERR_LAUNCH     5  /* the CUDA runtime rejected a launch */
#define W4_ERR_WORKSPACE  6  /* workspace missing or smaller than required */
#define W4_ERR_DEVICE     7  /* current device is not sm_103 or lacks a needed driver entry point */
#define W4_ERR_TIMEOUT    8  /* a device-side bounded wait expired (reported by w4a16_device_status) */
#define W4_ERR_INDEX      9  /* a kernel met a page, length, offset or other index out of range (reported by w4a16_device_status) */

/*
 * Launch flag of the *_ex calls.  W4A16_OVERLAP_PREVIOUS lets the call's
 * kernel start while the previous kernel on the same stream is still running
 * (programmatic dependent launch): it streams its weights (qweight, scales,
 * biases) at once and waits for the previous kernel only before it reads its
 * activations and writes its outputs.  Use it when the weights are not
 * written by the preceding kernel on the stream (the usual case: weights are
 * loaded once).  Without the flag the call follows ordinary stream order.
 */
#define W4A16_OVERLAP_PREVIOUS 1u

/*
 * w4_gemv - decode GEMV, y[m][n] = sum_k w[n][k] * x[m][k].
 *   ("The inference engine - Mojo 1.0 on Metal", "Crossing Mojo 1.0": the
 *   multi-row weight-streaming GEMV.)
 *   x       binary16 [M][K]          activations
 *   qweight, scales, biases          int4 weight in the format above
 *   y       binary16 [M][N]          output; fp32 accumulation, rounded to
 *                                     nearest even once at the end
 *   M       1..16 activation rows, all sharing one pass over the weights
 *   N       >= 1 output features;  K  multiple of 64, >= 64;
 *   group   quantisation group (see the format); biases may be NULL
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_GROUP, W4_ERR_ALIGN, W4_ERR_LAUNCH.
 */
W4A16_API int w4_gemv(const uint16_t *x, const uint32_t *qweight, const uint16_t *scales,
            const uint16_t *biases, uint16_t *y, int M, int N, int K, int group,
            void *stream);

/* w4_gemv with launch flags (W4A16_OVERLAP_PREVIOUS or 0); otherwise identical. */
W4A16_API int w4_gemv_ex(const uint16_t *x, const uint32_t *qweight, const uint16_t *scales,
            const uint16_t *biases, uint16_t *y, int M, int N, int K, int group,
            unsigned flags, void *stream);

/*
 * w4_gemv_seq - a list of GEMVs in one persistent launch (decode projection
 * list).
 *   ("The inference engine - Mojo 1.0 on Metal", "Appendix: the remaining
 *   gap": the per-token floor of some 250 small launches binds decode.)
 *   Runs ops[0..nops) in order, each exactly as w4_gemv would (same format,
 *   same results).  An operation with wait_prev != 0 reads activations that
 *   earlier operations of the list write: it starts only after they are
 *   complete and visible.  Weights are streamed without waiting, so they
 *   must not be written by the operations of the list.
 *   M       1..16 activation rows, shared by all operations.
 *   Each operation: N >= 1, K a multiple of 256, group (0 means 64) and
 *   biases (NULL: symmetric) as for w4_gemv, pointers 16-byte aligned.
 *   workspace  device buffer, 16-byte aligned, ZERO-FILLED before its first
 *              use and then passed unchanged to every later call (the library
 *              keeps its counters consistent: the last CTA of each launch
 *              resets them and advances an epoch).  With at least
 *              w4_gemv_seq_workspace_bytes_ex(ops, nops, M) bytes, an operation
 *              whose x lies inside the output of the latest earlier operation
 *              that writes any of x reads a tagged copy of that output (each
 *              word carries a 16-bit (epoch, operation) tag and the reader
 *              polls the words themselves); other waits, and every wait when
 *              the workspace holds only w4_gemv_seq_workspace_bytes() bytes,
 *              use a completion counter.  A workspace is used by one call at
 *              a time.  After an expired wait its contents are undefined:
 *              zero it again.
 *   flags   0.
 *   Long lists run as several launches of up to 96 operations; a launch is
 *   cooperative (one CTA per SM) and waits inside it are bounded (2 s; an
 *   expiry is reported by w4a16_device_status).
 * Errors: as w4_gemv, plus W4_ERR_WORKSPACE.
 */
typedef struct {
    const uint16_t *x;        /* binary16 [M][K] */
    const uint32_t *qweight;  /* [N][K/8] */
    const uint16_t *scales;   /* binary16 [N][K/G] */
    const uint16_t *biases;   /* binary16 [N][K/G], or NULL: symmetric codes */
    uint16_t *y;              /* binary16 [M][N] */
    int N, K;
    int wait_prev;            /* nonzero: x is written by an earlier operation */
    int group;                /* G of this operation's weight; 0 means 64 */
} w4_gemv_op;

/* Minimum workspace (completion counters only). */
W4A16_API size_t w4_gemv_seq_workspace_bytes(void);

/* Workspace for the tagged activation exchange of this operation list:
 * the counters plus, per launch of up to 96 operations, one uint32 word per
 * output element of every operation whose output a later one reads. */
W4A16_API size_t w4_gemv_seq_workspace_bytes_ex(const w4_gemv_op *ops, int nops, int M);

W4A16_API int w4_gemv_seq(const w4_gemv_op *ops, int nops, int M, void *workspace,
            size_t workspace_bytes, unsigned flags, void *stream);

/*
 * lm_head_argmax_topk - LM-head GEMV fused with token selection.
 *   ("The inference engine - Mojo 1.0 on Metal", "Crossing Mojo 1.0" and
 *   "What's inside the engine today": greedy / top-k selection on the GPU so
 *   that no logits vector crosses to the host.)
 *   Computes the fp32 logits l[m][n] = sum_k w[n][k] * x[m][k] for every
 *   n < N and returns, for each activation row m, the k largest:
 *   idx int32 [M][k] and val float32 [M][k], ordered by value descending,
 *   ties broken by the lowest index (k == 1 is greedy argmax).  No logits
 *   tensor is written: a first pass leaves per-block candidates in
 *   `workspace`, a second pass merges them.
 *   M 1..16;  N >= k;  K multiple of 64;  group and biases as for w4_gemv;
 *   1 <= k <= 64;
 *   N * k must not exceed 16,777,216.
 *   workspace  device buffer of at least lm_head_workspace_bytes(M, N, k)
 *              bytes, 16-byte aligned; contents on entry are ignored.
 * Errors: as w4_gemv, plus W4_ERR_WORKSPACE.
 */
W4A16_API int lm_head_argmax_topk(const uint16_t *x, const uint32_t *qweight,
                        const uint16_t *scales, const uint16_t *biases,
                        int M, int N, int K, int group, int k,
                        int32_t *idx, float *val,
                        void *workspace, size_t workspace_bytes, void *stream);

/* lm_head_argmax_topk with launch flags (W4A16_OVERLAP_PREVIOUS or 0). */
W4A16_API int lm_head_argmax_topk_ex(const uint16_t *x, const uint32_t *qweight,
                        const uint16_t *scales, const uint16_t *biases,
                        int M, int N, int K, int group, int k,
                        int32_t *idx, float *val,
                        void *workspace, size_t workspace_bytes, unsigned flags, void *stream);

/*
 * lm_head_argmax_topk_noalloc - lm_head_argmax_topk without a workspace
 * argument, for callers that cannot allocate device memory where they call it
 * (inside an allocator or memory-pool callback, under a fixed memory budget,
 * or in an embedding with no allocator of its own).  None of the pages has a
 * counterpart; it is a packaging variant of the call above.
 *   Arguments, results and limits are those of lm_head_argmax_topk; the
 *   candidate buffer is a 2 MiB array inside this library's device image,
 *   which covers every size lm_head_argmax_topk accepts (M <= 16, k * blocks
 *   <= 16384 keys per row).  Every GPU that loads the library holds the array
 *   until the process exits.  This call allocates nothing (no cudaMalloc, no
 *   library allocator).
 *   Set-up: the first call on a device looks up the array's device address on
 *   that device (cudaGetSymbolAddress) and caches it with the id of the CUDA
 *   context it belongs to; the first call in a new context (e.g. after
 *   cudaDeviceReset) looks it up again.  Make the first call on a device, and
 *   in each new context, before any stream capture on it.
 *   Sharing: all calls use the same array and it keeps the last call's
 *   contents.  Nothing in it has to start at zero: pass 1 writes every slot
 *   pass 2 reads, so a smaller call after a larger one never sees the
 *   larger call's leftovers.  Calls whose kernels overlap on the GPU (other
 *   streams, other host threads) race on the array: order them on one
 *   stream.
 * Errors: as lm_head_argmax_topk; W4_ERR_WORKSPACE if a size would need more
 * than the built-in 2 MiB; W4_ERR_DEVICE if the address lookup fails.
 */
W4A16_API int lm_head_argmax_topk_noalloc(const uint16_t *x, const uint32_t *qweight,
                        const uint16_t *scales, const uint16_t *biases,
                        int M, int N, int K, int group, int k,
                        int32_t *idx, float *val, void *stream);

/*
 * Rules of a selection: penalties of tokens that a request has seen, biases of
 * listed tokens and a mask, applied to the fp32 logit z of token n in row m,
 * in this order, each step one fp32 operation:
 *   counts   c = counts[slot[m]][n]: bit 15 "in the prompt", the low 15 bits the
 *            times t in the output (w4_token_counts keeps them):
 *              c != 0:  z = z > 0 ? z / repetition[m] : z * repetition[m]
 *              t != 0:  z = (z - frequency[m] * t) - presence[m]
 *            a negative slot: no penalties for the row
 *   biases   row m has the entries bias_offsets[m] <= i < bias_offsets[m + 1]:
 *              z = z + bias_values[i]  where bias_tokens[i] == n
 *            (entries of one token one after the other, in the list's order; negative
 *            tokens are skipped)
 *   allowed  bit n % 32 of word n / 32 of row m: 0 = n cannot be selected
 * Parts whose first pointer is NULL are left out.  The arrays are read on the
 * device, so that a captured graph can be replayed with other contents; a slot,
 * an offset or a token out of range is skipped (a list of biases as a whole) and
 * reported by w4a16_device_status as W4_ERR_INDEX.
 */
typedef struct {
    const uint16_t *counts;     /* [slots][counts_stride], or NULL */
    int64_t counts_stride;      /* >= N */
    const int32_t *slot;        /* [M] */
    const float *repetition;    /* [M], NULL: 1 */
    const float *presence;      /* [M], NULL: 0 */
    const float *frequency;     /* [M], NULL: 0 */
    const int32_t *bias_offsets; /* [M + 1], or NULL */
    const int32_t *bias_tokens; /* [bias_entries] */
    const float *bias_values;   /* [bias_entries] */
    const uint32_t *allowed;    /* [M][allowed_stride], or NULL */
    int64_t allowed_stride;     /* words, >= ceil(N / 32) */
    int32_t slots;              /* >= 1 */
    int32_t bias_entries;       /* 0 .. 2^30 */
} w4_logit_rules;

/*
 * lm_head_argmax_topk_rules - lm_head_argmax_topk_ex with rules (NULL: none).
 *   Of a row with fewer than k tokens that its mask allows, idx is -1 and val
 *   -infinity past these (greedy selection of a row with none: -1).  val is the
 *   logit after the rules.  The rules are applied to each block's logits in shared
 *   memory before it selects, so a call reads 2 bytes of counts and one bit of
 *   mask a logit more than without; index arrays need their natural alignment
 *   only (rows of counts that start on 16 bytes are read fastest).
 * Errors: as lm_head_argmax_topk.
 */
W4A16_API int lm_head_argmax_topk_rules(const uint16_t *x, const uint32_t *qweight,
                        const uint16_t *scales, const uint16_t *biases,
                        int M, int N, int K, int group, int k,
                        int32_t *idx, float *val, const w4_logit_rules *rules,
                        void *workspace, size_t workspace_bytes, unsigned flags, void *stream);

/*
 * w4_token_counts - count tokens in their requests' rows of `counts`.
 *   counts   uint16 [slots][counts_stride], N tokens used: see w4_logit_rules
 *   slot     int32 [batch]: the slot of each sequence (negative: none)
 *   tokens   int32 [total]; negative ones are skipped
 *   offsets  int32 [batch + 1], ascending: sequence b has the tokens
 *            offsets[b] .. offsets[b + 1] - 1; NULL: token b alone (total = batch)
 *   flags    W4_COUNTS_PROMPT: tokens of a prompt (bit 15 is set); without it
 *            tokens of the output (the count goes up, and stays at 32767)
 *            W4_COUNTS_RESET: the sequences' rows are cleared first (a request
 *            takes its slot); of sequences with one slot the last takes it
 *   batch 0..65535;  total >= 0;  a token past N, a slot past the last, the tokens
 *   of a sequence whose offsets are out of order or past total, and slots taken
 *   again are skipped (a row is cleared all the same) and reported by
 *   w4a16_device_status as W4_ERR_INDEX.  Tokens that such offsets give to several
 *   sequences may count for any of them; rows that no sequence names stay as they are.
 * Pointers need their natural alignment only.  Results do not depend on the
 * order in which tokens are counted.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_DEVICE, W4_ERR_LAUNCH.
 */
#define W4_COUNTS_PROMPT 1u
#define W4_COUNTS_RESET  2u
W4A16_API int w4_token_counts(uint16_t *counts, int64_t counts_stride, int slots, int N, const int32_t *slot,
                              const int32_t *tokens, const int32_t *offsets, int batch, int total, unsigned flags,
                              void *stream);

/* Bytes of workspace lm_head_argmax_topk needs for these sizes (0 if the
 * sizes are invalid).  Depends only on its arguments. */
W4A16_API size_t lm_head_workspace_bytes(int M, int N, int k);

/*
 * w4_dequant_f16 - dequantise once into the transposed half scratch.
 *   ("The inference engine - Mojo 1.0 on Metal", "Crossing Mojo 1.0": each
 *   weight is dequantised once per prefill into a transposed half-precision
 *   scratch.)
 *   w16  binary16 [K][N] (= W transposed), w16[k][n] = the correctly rounded
 *        (nearest, ties to even) binary16 of the exact scale*q + bias, or of
 *        scale*(q - 8) when biases is NULL (a zero keeps the sign of the
 *        IEEE product scale*(q - 8)).
 *   N >= 1;  K multiple of 64;  group as for w4_gemv.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_GROUP, W4_ERR_ALIGN, W4_ERR_LAUNCH.
 */
W4A16_API int w4_dequant_f16(const uint32_t *qweight, const uint16_t *scales,
                   const uint16_t *biases, uint16_t *w16, int N, int K, int group,
                   void *stream);

/* w4_dequant_f16_ex - w4_dequant_f16 with flags (0 or W4A16_OVERLAP_PREVIOUS).
 * For this call W4A16_OVERLAP_PREVIOUS states more than for the GEMVs: the
 * call reads nothing the previous kernel on the stream writes and writes
 * nothing it reads or writes (e.g. one of many dequantisations of distinct
 * weights into distinct scratch buffers).  The kernel is then launched as a
 * programmatic dependent without any wait and may run concurrently with the
 * previous kernel. */
W4A16_API int w4_dequant_f16_ex(const uint32_t *qweight, const uint16_t *scales,
                                const uint16_t *biases, uint16_t *w16, int N, int K,
                                int group, unsigned flags, void *stream);

/*
 * w4_gemm - int4 GEMM with the dequantisation fused into the tensor-core
 * pipeline, for prefill with few activation rows:
 *   y[m][n] = sum_k w[n][k] * x[m][k],  w[n][k] = RNE_binary16(scale*q + bias)
 *   (or of scale*(q - 8) without biases): the weight values of
 *   w4_dequant_f16, multiplied without writing a scratch.
 *   ("The inference engine - Mojo 1.0 on Metal", "Crossing Mojo 1.0": the
 *   prefill GEMM over dequantised weights; here the weights are dequantised
 *   tile by tile into tensor memory and read from HBM only as 4-bit codes.)
 *   x        binary16 [M][K]   activations
 *   qweight, scales, biases, group    the int4 weight (format above)
 *   y        binary16 [M][N]   output; fp32 accumulation, one rounding
 *   M 1..128;  N >= 8, N % 8 == 0;  K >= 64, K % 64 == 0.
 *   workspace  device buffer of at least w4_gemm_workspace_bytes(M, N, K)
 *              bytes, 16-byte aligned, ZERO-FILLED before its first use and
 *              then passed unchanged to later calls (its grid-barrier
 *              counters are left ready for the next call).  Calls ordered on
 *              one stream may share it, also with W4A16_OVERLAP_PREVIOUS (a
 *              call touches it only after its dependency wait); calls that
 *              may run concurrently need separate workspaces.
 *              It holds the fp32 partial sums of the 128-row weight tiles
 *              whose k steps are shared by several blocks (the tiles left
 *              over after every block has taken whole tiles).
 *   The products are those of f16_gemm on the w4_dequant_f16 scratch (the
 *   same binary16 weight values); the 64-k steps of a tile are accumulated
 *   in fp32 starting from a per-tile rotation, and a tile shared by several
 *   blocks adds their partial sums in ascending k.  Results are
 *   deterministic.  For M <= 32 the last block to bring a shared tile's
 *   partial sums adds them all.  For M > 32 the launch is cooperative
 *   (every block resident): the blocks sharing a tile wait for each other's
 *   partial sums and each adds a slice (bounded: on expiry the call leaves
 *   that tile unwritten and w4a16_device_status reports W4_ERR_TIMEOUT).
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_GROUP, W4_ERR_ALIGN,
 * W4_ERR_WORKSPACE, W4_ERR_DEVICE, W4_ERR_LAUNCH.
 */
W4A16_API int w4_gemm(const uint16_t *x, const uint32_t *qweight, const uint16_t *scales,
                      const uint16_t *biases, uint16_t *y, int M, int N, int K, int group,
                      void *workspace, size_t workspace_bytes, void *stream);

/* w4_gemm with launch flags (W4A16_OVERLAP_PREVIOUS: the weights are not
 * written by the previous kernel; their first tiles are fetched and
 * converted before it finishes). */
W4A16_API int w4_gemm_ex(const uint16_t *x, const uint32_t *qweight, const uint16_t *scales,
                         const uint16_t *biases, uint16_t *y, int M, int N, int K, int group,
                         void *workspace, size_t workspace_bytes, unsigned flags, void *stream);

/* Workspace bytes for w4_gemm (0 if the sizes are invalid): 3328 bytes of
 * counters and flags and 2 x min(256, ceil(N / 128) x K / 64) fp32 tiles of
 * M x 128.  Depends only on its arguments. */
W4A16_API size_t w4_gemm_workspace_bytes(int M, int N, int K);

/*
 * f16_gemm - dense half GEMM for prefill, y = x16 * w16.
 *   ("The inference engine - Mojo 1.0 on Metal", "Crossing Mojo 1.0": the
 *   half-precision GEMM that follows the dequantise-once step.)
 *   x16  binary16 [M][K] row-major;  w16  binary16 [K][N] row-major;
 *   y    binary16 [M][N] row-major; fp32 accumulation on the tensor cores,
 *        rounded to nearest even once at the end.
 *   M >= 1;  N >= 8 and a multiple of 8;  K >= 8 and a multiple of 8
 *   (row strides must be 16-byte multiples for the tensor-memory copies).
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_DEVICE, W4_ERR_LAUNCH.
 */
W4A16_API int f16_gemm(const uint16_t *x16, const uint16_t *w16, uint16_t *y,
             int M, int N, int K, void *stream);

/* f16_gemm_ex - f16_gemm with flags (0 or W4A16_OVERLAP_PREVIOUS).  With the
 * flag the kernel is a programmatic dependent of the previous kernel on the
 * stream: it sets up and copies the w16 tiles of its first stages at once and
 * waits for the previous kernel before it reads x16 or writes y.  w16 must
 * therefore be complete when the call is issued (not written by the previous
 * kernel, nor by any kernel still running beside it). */
W4A16_API int f16_gemm_ex(const uint16_t *x16, const uint16_t *w16, uint16_t *y, int M, int N,
                          int K, unsigned flags, void *stream);

/*
 * Low-rank adapters of a projection: N x K updates B_a A_a of a shared weight.
 * The columns may be cut into up to four slices, each with an A of its own (the
 * q | k | v or gate | up blocks of one projection).
 */
typedef struct {
    const uint16_t *a;   /* binary16 [adapters][slices][rank][K], adapters a_adapter elements apart */
    const uint16_t *b;   /* binary16 [adapters][N][rank], adapters b_adapter elements apart */
    const float *scale;  /* [adapters], or NULL: 1 */
    int64_t a_adapter, b_adapter; /* multiples of 8 */
    int32_t adapters;    /* 1..4096 */
    int32_t rank;        /* a multiple of 8, 8..128 */
    int32_t K, N;        /* multiples of 8 */
    int32_t slices;      /* 1..4 */
    int32_t columns[4];  /* end of each slice, ascending multiples of 8; the last is N */
} f16_adapters;

/*
 * f16_lora - adapters of many requests at once, beside a projection of theirs
 * (w4_gemv, w4_gemm or f16_gemm, whose output is y):
 *     out[m] = y[m] + scale[a] * (x[m] A_a^T) B_a^T,   a = ids[m],
 *   the A being that of the column's slice; rows with a negative id get y[m].
 *   x        binary16 [M][K], y and out binary16 [M][N]: rows x_row, y_row and
 *            out_row elements apart (multiples of 8; out_row >= N); out may be y,
 *            else they must not overlap
 *   ids      int32 [M], in any order and mix (read on the device: a captured graph
 *            can be replayed with others); an id past the last adapter counts as
 *            negative and is reported by w4a16_device_status as W4_ERR_INDEX.
 *            Many rows of one adapter are fastest where they lie near each other
 *            (rows are gathered within blocks of up to 1024)
 *   M        >= 0
 *   workspace  device buffer of at least f16_lora_workspace_bytes bytes, 16-byte
 *              aligned; contents on entry are ignored.  Calls that may run
 *              concurrently need separate ones.
 *   Sums are fp32 over exact products; x A^T is carried on in two binary16 numbers
 *   a value (2^-22 of the row's largest finite one), and out is rounded once.  Results are
 *   deterministic; a row is not touched by what the others hold (NaN and infinities
 *   included), but its sums may be taken in another order in another mix of rows.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_WORKSPACE,
 * W4_ERR_DEVICE, W4_ERR_LAUNCH.
 */
W4A16_API int f16_lora(const uint16_t *x, int64_t x_row, const uint16_t *y, int64_t y_row, uint16_t *out,
                       int64_t out_row, const f16_adapters *adapters, const int32_t *ids, int M, void *workspace,
                       size_t workspace_bytes, void *stream);

/* Workspace bytes for f16_lora (0 if the sizes are invalid).  Depends only on the
 * adapters' sizes and M, and grows with M: a workspace for the most rows serves
 * all calls with fewer. */
W4A16_API size_t f16_lora_workspace_bytes(const f16_adapters *adapters, int M);

/*
 * Attention with a paged key/value cache: what a decoder layer does between
 * its q/k/v projections and its o projection.  The three calls share the
 * conventions above (binary16 tensors, fp32 arithmetic, host checks, one
 * stream).  Activations are [tokens][heads][head_dim] with strides in
 * elements: `*_token` from token to token, `*_head` from head to head, both
 * multiples of 8 (16 bytes), the head_dim elements of a head contiguous.
 * Index arrays (int32) need their natural alignment only.
 *
 * Sequences.  A call works on the tokens of `batch` sequences, whose new
 * tokens lie one after the other: sequence b has the tokens q_offsets[b] <= t
 * < q_offsets[b + 1], and kv_lens[b] tokens in the cache, these new ones
 * among them (they are its last).  Its token t therefore stands at position
 *     p = kv_lens[b] - (q_offsets[b + 1] - q_offsets[b]) + (t - q_offsets[b]).
 * Position p of sequence b is kept in token p % page_size of page
 * block_table[b][p / page_size].  Table entries that no visible position
 * needs may hold anything.  A sequence may bring no token, and may have
 * kv_lens[b] = 0 (a padded slot of a batch).  Lengths, offsets and pages are
 * read on the device, so that a captured graph can be replayed with others;
 * those out of range are clamped or skipped, never followed, and reported by
 * w4a16_device_status as W4_ERR_INDEX (with offsets out of order, f16_attention
 * writes nothing; of a sequence whose length or offsets are out of range,
 * f16_kv_append writes no keys or values).
 */
typedef struct {
    const int32_t *block_table; /* [batch][table_stride], the first max_pages of a row are used */
    const int32_t *q_offsets;   /* [batch + 1], ascending */
    const int32_t *kv_lens;     /* [batch], at most max_pages * page_size */
    int32_t batch;              /* >= 1 */
    int32_t max_pages;          /* >= 1 */
    int32_t table_stride;       /* >= max_pages */
    int32_t total_q;            /* tokens of the q, k, v tensors (rows past q_offsets[batch] are left alone) */
    int32_t max_q_len;          /* the most new tokens of one sequence: a kernel is chosen by it (results hold for any) */
} f16_kv_batch;

/*
 * A paged cache: binary16 k and v, num_pages pages of page_size tokens of
 * `heads` key/value heads, with strides in elements (multiples of 8), in any
 * order of page, token and head.  Filled in by f16_kv_cache_init, which also
 * encodes the tensor maps of its copies; plain data, copied and dropped freely.
 */
typedef struct {
    uint16_t *k, *v;
    int64_t k_page, k_token, k_head;
    int64_t v_page, v_token, v_head;
    int32_t num_pages, page_size, heads, head_dim;
    int32_t box_rows, reserved;
    uint64_t k_map[16], v_map[16];   /* copies of box_rows tokens x 64 elements */
    uint64_t k_wide[16], v_wide[16]; /* of whole heads (head_dim a multiple of 64 above 64) */
} f16_kv_cache;

/*
 * f16_kv_cache_init - describe a cache (host only, nothing is enqueued).
 *   strides   {page, token, head} in elements
 *   num_pages >= 1;  page_size a multiple of 8;  heads >= 1;
 *   head_dim  a multiple of 8, 8..256
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_DEVICE.
 */
W4A16_API int f16_kv_cache_init(f16_kv_cache *cache, uint16_t *k, uint16_t *v, const int64_t k_strides[3],
                                const int64_t v_strides[3], int num_pages, int page_size, int heads, int head_dim);

/*
 * A rotation of positions.  Pair i < rot / 2 of a head is turned by
 * p * turns[i] / 2^64 of a full turn at position p, and scaled by factor:
 *     (a, b) -> factor * (a cos - b sin, a sin + b cos).
 * turns[i] = round(2^64 * theta_i / (2 pi)) for an angle of theta_i per
 * position; p * turns[i] wraps modulo 2^64, which is the reduction of the
 * angle to one turn, exact at every position.  Negative positions turn back.
 * Pairs are (2i, 2i + 1) when interleaved, else (i, i + rot / 2); the
 * elements from rot on are copied.
 */
typedef struct {
    const uint64_t *turns; /* [rot / 2], device memory */
    int32_t rot;           /* a multiple of 8, 8..head_dim */
    int32_t interleaved;   /* 0 or 1 */
    float factor;          /* 1, or the scale of a stretched context */
} f16_rotation;

/*
 * f16_rope - rotate the heads of a tensor: y[t][h] = R(positions[t]) x[t][h].
 *   positions  int32 [tokens], any value; NULL: token t is at position t
 *   x, y       strided as above; y may be x (in place), else they must not overlap
 *   tokens >= 0;  heads >= 1;  head_dim a multiple of 8, 8..256
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_DEVICE, W4_ERR_LAUNCH.
 */
W4A16_API int f16_rope(const uint16_t *x, int64_t x_token, int64_t x_head, uint16_t *y, int64_t y_token,
                       int64_t y_head, const int32_t *positions, const f16_rotation *rotation, int tokens, int heads,
                       int head_dim, void *stream);

/*
 * A norm of heads, applied before their rotation:
 *     z_i = x_i * weight[i] / sqrt(mean_j x_j^2 + eps),  over the head_dim
 * elements of a head.  Squares, sum, root and products are fp32, and the result
 * is rounded to binary16 once, after the rotation.
 */
typedef struct {
    const float *weight; /* [head_dim], device memory, 16-byte aligned */
    float eps;           /* >= 0, finite (with 0, a head of zeros gives NaN) */
} f16_head_norm;

/* f16_rope_ex - f16_rope with a norm of each head before its rotation (NULL:
 * none); with a norm, rotation may be NULL (nothing is turned). */
W4A16_API int f16_rope_ex(const uint16_t *x, int64_t x_token, int64_t x_head, uint16_t *y, int64_t y_token,
                          int64_t y_head, const int32_t *positions, const f16_rotation *rotation,
                          const f16_head_norm *norm, int tokens, int heads, int head_dim, void *stream);

/*
 * f16_kv_append - write the new tokens' keys and values into the cache, the
 * keys rotated on the way, and rotate the queries in the same launch.
 *   k, v       [total_q][cache heads][head_dim], strided
 *   rotation   NULL: nothing is rotated
 *   positions  int32 [total_q], the rotation's positions where they are not
 *              the cache's (NULL: they are)
 *   q, y       [total_q][q_heads][head_dim], strided: y = R q (y may be q).
 *              q NULL: keys and values only
 * Cache slots of other positions keep their contents.  A token whose position
 * is negative (a padded slot) is not written to the cache.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_DEVICE, W4_ERR_LAUNCH.
 */
W4A16_API int f16_kv_append(const uint16_t *k, int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token,
                            int64_t v_head, const f16_kv_cache *cache, const f16_kv_batch *batch,
                            const f16_rotation *rotation, const int32_t *positions, const uint16_t *q,
                            int64_t q_token, int64_t q_head, uint16_t *y, int64_t y_token, int64_t y_head,
                            int q_heads, void *stream);

/* f16_kv_append_ex - f16_kv_append with a norm of each query head and of each
 * key head before its rotation (NULL: none for these heads).  Values are
 * written as they are. */
W4A16_API int f16_kv_append_ex(const uint16_t *k, int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token,
                               int64_t v_head, const f16_kv_cache *cache, const f16_kv_batch *batch,
                               const f16_rotation *rotation, const int32_t *positions, const f16_head_norm *q_norm,
                               const f16_head_norm *k_norm, const uint16_t *q, int64_t q_token, int64_t q_head,
                               uint16_t *y, int64_t y_token, int64_t y_head, int q_heads, void *stream);

/*
 * f16_attention - attention of the new tokens over the cache:
 *     y[t][h] = sum_j softmax_j(scale * q[t][h] . k_j) v_j,
 * over the positions j of t's sequence that it sees: j < kv_lens[b], with
 * causal != 0 also j <= p, with window > 0 also j > p - window (p is t's
 * position, above).  Query head h reads key/value head h / (q_heads / heads).
 *   q, y    [total_q][q_heads][head_dim], strided (y may be q)
 *   lse     float [total_q][q_heads]: log of the sum of exp(scale q . k_j), or NULL
 *   scale   > 0, finite;  causal 0 or 1;  window >= 0 (0: none)
 *   total_q x q_heads x max_pages x page_size up to about 2^42 (W4_ERR_SHAPE)
 *   q_heads a multiple of the cache's heads, at most 1024 for each
 *   (head_dim above 128: every call reads K and V once per 16 rows of a
 *   sequence and key/value head, so long prompts are several times slower)
 *   workspace  device buffer of at least f16_attention_workspace_bytes bytes,
 *              16-byte aligned, ZERO-FILLED before its first use and then
 *              passed unchanged to later calls (its counters are left ready for
 *              the next one).  Calls ordered on one stream may share it; calls
 *              that may run concurrently need separate ones.
 * Blocks that share a sequence wait for each other's partial results, once
 * every block of the call has begun (bounded: on expiry, which a workspace
 * that was not zeroed brings about, the rows concerned stay unwritten,
 * w4a16_device_status reports W4_ERR_TIMEOUT and the workspace has to be
 * zeroed again).
 * Products are binary16 with fp32 sums; the softmax's statistics and the
 * output's sum are fp32, the probabilities are rounded to binary16 for the
 * product with v, and y is rounded once.  A token that sees no position gets
 * y = 0 and lse = -infinity.  What the cache holds at positions that no token
 * of the call sees, and past a sequence's end, does not matter, NaN and
 * infinities included; keys and values that some token of a sequence sees are
 * taken to be finite (a value that is not may show in the sequence's earlier
 * tokens too).  Results are deterministic.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_WORKSPACE,
 * W4_ERR_DEVICE, W4_ERR_LAUNCH.
 */
W4A16_API int f16_attention(const uint16_t *q, int64_t q_token, int64_t q_head, uint16_t *y, int64_t y_token,
                            int64_t y_head, float *lse, int q_heads, float scale, int causal, int window,
                            const f16_kv_cache *cache, const f16_kv_batch *batch, void *workspace,
                            size_t workspace_bytes, void *stream);

/* Workspace bytes for f16_attention (0 if the sizes are invalid).  Depends
 * only on its arguments, and does not grow with the batch or the context. */
W4A16_API size_t f16_attention_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q_len);

/* Human-readable name of a status code (static string). */
W4A16_API const char *w4a16_status_string(int status);

/*
 * Synchronises the current device and reports whether any kernel of this
 * library gave up a bounded device-side wait since the last call
 * (W4_ERR_TIMEOUT) or met an index out of range (W4_ERR_INDEX), then clears
 * the record.  W4A16_OK otherwise.
 */
W4A16_API int w4a16_device_status(void);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H */

/*
 * fd.h — C ABI of the B200 (sm_100a) split-KV decode attention library
 * (libfd.so).
 *
 * The operation is Flash-Decoding ("What is Flash-Decoding, and when does it
 * speed up LLMs?", slavadubrov.com: the opening paragraph and the section
 * "Why decode needs a different schedule"). One new query token per
 * sequence attends over that sequence's long cached K/V history. The history
 * is split into chunks. Each chunk gives a partial output and a log-sum-exp,
 * and a reduction merges the partials into the exact attention over the
 * whole history:
 *
 *     out[b, h, :] = softmax_j(scale * q[b, h, :] . K[b, kv, j, :]) @ V[b, kv, j, :]
 *     lse[b, h]    = ln sum_j exp(scale * q[b, h, :] . K[b, kv, j, :])
 *
 * Here kv = h / (Hq / Hkv), which covers grouped-query attention, and j runs
 * over the seqlens[b] valid cached tokens.
 *
 * Conventions shared by every entry point:
 *  - Tensor pointers are DEVICE pointers owned by the caller. The library
 *    keeps no pointer and allocates nothing; the workspace is caller-supplied.
 *  - Element types: q and out are bf16; K and V are bf16, fp8 E4M3 codes or
 *    4-bit codes (fd_problem.kv_dtype); lse, the workspace and scale are fp32;
 *    seqlens and block_table are int32.
 *  - Errors are return codes. No entry point aborts, throws or prints.
 *    Argument checks run on the host before anything is launched; an invalid
 *    call launches nothing.
 *  - Work is asynchronous on the caller's stream. A fault inside a kernel
 *    surfaces at the caller's next synchronisation.
 *  - There is no CPU fallback. The kernels are built for sm_100a only.
 */
#ifndef FD_H_
#define FD_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FD_API __attribute__((visibility("default")))
#else
#define FD_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t (struct CUstream_st*); NULL is the legacy default
 * stream. */
typedef struct CUstream_st* fd_stream_t;

typedef enum fd_status {
  FD_OK = 0,
  /* Null pointer, non-positive size, Hq % Hkv != 0, a tensor pointer not
   * 16-byte aligned (lse: 4-byte), num_splits outside [1, 1024], scale not
   * finite and positive, unknown kv_layout, shape limits exceeded. */
  FD_ERR_INVALID_ARGUMENT = -1,
  /* Head dim D not in {64, 128}, group size Hq/Hkv not in {1, 2, 4, 8, 16},
   * block_size not a power of two in [8, 256], or the device is not sm_100. */
  FD_ERR_UNSUPPORTED = -2,
  /* The chosen split count needs a workspace, and the one passed is NULL or
   * smaller than fd_workspace_bytes() reports. */
  FD_ERR_WORKSPACE = -3,
  /* A CUDA runtime or driver call failed (launch error, tensor-map encode). */
  FD_ERR_CUDA = -4,
  /* A kernel gave up on a bounded wait. Its outputs are not valid. */
  FD_ERR_DEVICE_TIMEOUT = -5
} fd_status;

/* Order of the cache dimensions (see fd_decode for the full shapes). */
typedef enum fd_kv_layout {
  /* heads outside tokens: [B, Hkv, max_len, D] or [num_blocks, Hkv, block_size, D] */
  FD_LAYOUT_HND = 0,
  /* tokens outside heads: [B, max_len, Hkv, D] or [num_blocks, block_size, Hkv, D] */
  FD_LAYOUT_NHD = 1
} fd_kv_layout;

/* Element type of the K/V cache. */
typedef enum fd_kv_dtype {
  FD_KV_BF16 = 0,     /* bf16 */
  FD_KV_FP8_E4M3 = 1, /* OCP fp8 e4m3 (bias 7, max 448, no inf); value = scale * code */
  FD_KV_INT4 = 2      /* 4-bit codes with a scale and a bias per half row; for the entry points
                       * named fd_*_int4 (see fd_append_int4 for the format) and
                       * fd_plan_problem */
} fd_kv_dtype;

/* Tensor-core path of an fp8 cache.
 *   FD_FP8_MMA_SYNC     the default: e4m3 codes converted to f16 in registers,
 *                       both contractions on mma.sync with fp32 accumulation.
 *   FD_FP8_MMA_TCGEN05  kind::f8f6f4 tcgen05 MMAs on the codes as the TMA left
 *                       them in shared memory, accumulators in tensor memory;
 *                       q and the softmax weights enter as sums of e4m3 codes
 *                       (q exactly, the weights to 12 significant bits). Taken
 *                       where G is 2, 4 or 8 and the grid has at most one CTA
 *                       per SM; other calls run the default path. Measured
 *                       slower on B200 (CodeLlama-34B heads, 64K tokens:
 *                       40.8 against 24.2 us per call). */
typedef enum fd_fp8_mma {
  FD_FP8_MMA_SYNC = 0,
  FD_FP8_MMA_TCGEN05 = 1
} fd_fp8_mma;

/* Shape of one decode-attention call.
 *   B           sequences in the batch (1 .. 65535)
 *   Hq, Hkv     query heads and KV heads (Hkv .. 65535, Hq % Hkv == 0)
 *   D           head dimension (64 or 128)
 *   max_len     contiguous cache: rows held per (sequence, KV head);
 *               paged cache: the longest sequence the block table can hold
 *               (<= max_blocks_per_seq * block_size)
 *   block_size  0 for a contiguous cache; otherwise tokens per page
 *   num_blocks  paged cache: pages in the pool (ignored when contiguous)
 *   max_blocks_per_seq  paged cache: row length of block_table
 *   kv_layout   an fd_kv_layout value (FD_LAYOUT_HND when zero-initialised)
 *   kv_dtype    an fd_kv_dtype value (FD_KV_BF16 when zero-initialised)
 *   k_scale, v_scale
 *               fp8 caches: the real K and V are k_scale * code and
 *               v_scale * code (finite, > 0). Ignored for other caches.
 *               An fp8 cache needs D = 128; on the default path the
 *               contraction runs on f16 tensor cores, so q must be finite
 *               in f16 (|q| < 65504).
 *   fp8_mma     an fd_fp8_mma value (FD_FP8_MMA_SYNC when zero-initialised);
 *               ignored for bf16 caches. */
typedef struct fd_problem {
  int32_t B;
  int32_t Hq;
  int32_t Hkv;
  int32_t D;
  int32_t max_len;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_blocks_per_seq;
  int32_t kv_layout;
  int32_t kv_dtype;
  float k_scale;
  float v_scale;
  int32_t fp8_mma;
} fd_problem;

/* Split-count planner.
 * Follows the same page's section "Why decode needs a different schedule".
 * Splitting the history creates extra work units when the batch supplies too
 * few. For a short history the partials and the reduction can cost more than
 * they save, and a large batch already supplies the work.
 * Returns S >= 1 for fd_decode's num_splits, chosen for the current device's
 * SM count. Returns 1 when B*Hkv already fills the device or the history is
 * short. Returns a negative fd_status for invalid or unsupported shapes.
 * Host only and deterministic. It reads the SM count of the current device
 * once per device and caches it. */
FD_API int fd_plan(int B, int Hq, int Hkv, int D, int max_len, int block_size);

/* The same planner with the SM count given explicitly. Pure function: no
 * CUDA call. */
FD_API int fd_plan_sm(int num_sms, int B, int Hq, int Hkv, int D, int max_len,
               int block_size);

/* Split-count planner that also sees the sequence lengths of the batch.
 * Same rule as fd_plan, with one difference. When the lengths differ,
 * splitting also evens out the work per CTA: one long sequence would
 * otherwise decide the end of the call. This planner therefore models the
 * actual per-sequence lengths instead of assuming max_len for every sequence.
 *   num_sms   SM count to plan for; <= 0 means the current device's
 *   seqlens   HOST array [B] of valid tokens per sequence, clamped to
 *             [0, max_len] as in fd_decode
 * Returns S >= 1, or a negative fd_status (a NULL seqlens is
 * FD_ERR_INVALID_ARGUMENT). Host only and deterministic. It costs O(B)
 * per candidate split count. */
FD_API int fd_plan_seqlens(int num_sms, int B, int Hq, int Hkv, int D, int max_len,
                           int block_size, const int32_t* seqlens);

/* The planner for a whole problem description: the same cost model, with
 * the cache's element type (an fp8 CTA moves half the bytes of a bf16 one
 * at the same token rate, so fp8 caches want more CTAs in flight) and, when
 * given, the lengths. For a 4-bit cache it gives 1 where one cluster per row serves
 * best, and otherwise the least count whose workspace lets fd_decode_int4 use
 * every SM. fd_plan and fd_plan_seqlens plan for bf16 caches.
 *   num_sms   SM count to plan for; <= 0 means the current device's
 *   p         HOST pointer to the problem as passed to fd_decode (pointers
 *             and scales are not read)
 *   seqlens   HOST array [B] of valid tokens per sequence, or NULL when
 *             every sequence holds max_len
 * Returns S >= 1, or a negative fd_status: FD_ERR_INVALID_ARGUMENT for a
 * NULL p, a bad shape or an unknown kv_dtype; FD_ERR_UNSUPPORTED for an fp8
 * cache with D != 128. Host only and deterministic. */
FD_API int fd_plan_problem(int num_sms, const fd_problem* p, const int32_t* seqlens);

/* How a call cuts the history. With T = ceil(max_len / 64) tiles of 64
 * tokens, the effective split count is S = min(num_splits, T) (1 when
 * max_len is 0), and split s covers the tiles [floor(s*T/S),
 * floor((s+1)*T/S)) of every sequence: tokens [64*floor(s*T/S),
 * 64*floor((s+1)*T/S)), cut at the sequence's length. The splits differ by
 * at most one tile, so any split count up to T gives CTAs of balanced size.
 * Splits past a sequence's end are empty.
 * fd_split_chunk returns the largest split's tokens, 64*ceil(T/S) (64 when
 * max_len is 0); fd_effective_splits returns S. Both return a negative
 * fd_status for invalid arguments. */
FD_API int fd_split_chunk(int max_len, int num_splits);
FD_API int fd_effective_splits(int max_len, int num_splits);

/* Workspace bytes that fd_decode needs for num_splits splits. This is 0
 * when num_splits == 1. Otherwise it is the fp32 partial outputs
 * [B, Hq, S, D] followed by the fp32 partial log-sum-exps [B, Hq, S], each
 * part rounded up to 256 bytes, with S = num_splits. The effective split
 * count (fd_effective_splits) never exceeds num_splits, so this size is
 * always enough for the call.
 * Returns 0 for invalid arguments. */
FD_API size_t fd_workspace_bytes(int B, int Hq, int D, int num_splits);

/* Decode attention for one query token per sequence.
 *   p            shape (see fd_problem)
 *   q            [B, Hq, D] bf16, 16-byte aligned
 *   k_cache, v_cache
 *                (elements bf16, or fp8 e4m3 bytes when kv_dtype says so)
 *                FD_LAYOUT_HND contiguous: [B, Hkv, max_len, D];
 *                FD_LAYOUT_HND paged:      [num_blocks, Hkv, block_size, D];
 *                FD_LAYOUT_NHD contiguous: [B, max_len, Hkv, D];
 *                FD_LAYOUT_NHD paged:      [num_blocks, block_size, Hkv, D];
 *                row-major, 16-byte aligned
 *   seqlens      [B] int32 valid tokens per sequence, or NULL (all max_len).
 *                Values are clamped to [0, max_len]. Rows at or past a
 *                sequence's length are never summed; they may hold anything,
 *                NaN included. A length of 0 gives out = 0 and lse = -inf.
 *   block_table  paged only: [B, max_blocks_per_seq] int32; token t of
 *                sequence b sits in page block_table[b, t / block_size], row
 *                t % block_size. Entries are read only for pages that hold
 *                valid tokens. A page id outside [0, num_blocks) reads zeros.
 *                NULL selects the contiguous layout and needs block_size == 0.
 *   scale        softmax scale (finite, > 0), typically 1/sqrt(D)
 *   num_splits   requested split count in [1, 1024], normally fd_plan's
 *                result. The effective count is min(num_splits,
 *                ceil(max_len / 64)); see fd_split_chunk for the cut.
 *   out          [B, Hq, D] bf16, round-to-nearest-even, 16-byte aligned
 *   lse          [B, Hq] fp32 natural-log log-sum-exp of the scaled logits,
 *                or NULL to skip it
 *   workspace    fp32 scratch of at least fd_workspace_bytes(B, Hq, D, S)
 *                bytes for the effective split count S (the num_splits
 *                passed is always enough), 16-byte aligned. It may be NULL
 *                when S == 1. Its
 *                contents on entry do not matter, and it must not be shared
 *                by calls that overlap on the GPU.
 *   stream       the stream to run on
 * Results are bit-identical across repeated calls with the same inputs and
 * the same num_splits. The paged and contiguous layouts of the same logical
 * cache also give bit-identical results. */
FD_API fd_status fd_decode(const fd_problem* p, const void* q, const void* k_cache,
                    const void* v_cache, const int32_t* seqlens,
                    const int32_t* block_table, float scale, int num_splits,
                    void* out, float* lse, void* workspace,
                    size_t workspace_bytes, fd_stream_t stream);

/* Partial decode over a shard of each sequence's history, for merging
 * across GPUs (sequence-parallel decode).
 * When each GPU holds a contiguous slice of every sequence's cached tokens,
 * each GPU calls this on its own slice. The call returns the exact attention
 * over that slice: a normalised fp32 output and its log-sum-exp. After the
 * R results are gathered in one place (for example with an NCCL all-gather),
 * fd_combine merges them into the attention over the whole history. This is
 * the same log-sum-exp reduction that merges the splits of one GPU (page
 * "What is Flash-Decoding, and when does it speed up LLMs?", section "Why
 * decode needs a different schedule").
 * Arguments are those of fd_decode, except two outputs:
 *   out_f32  [B, Hq, D] fp32, 16-byte aligned (required)
 *   lse      [B, Hq] fp32 (required)
 * An empty slice gives out_f32 = 0 and lse = -inf, which weighs nothing in
 * fd_combine. */
FD_API fd_status fd_decode_partial(const fd_problem* p, const void* q, const void* k_cache,
                                   const void* v_cache, const int32_t* seqlens,
                                   const int32_t* block_table, float scale, int num_splits,
                                   float* out_f32, float* lse, void* workspace,
                                   size_t workspace_bytes, fd_stream_t stream);

/* Merges R partial results into the final output. Each part covers a
 * disjoint slice of the history, for example one per GPU from
 * fd_decode_partial:
 *   m = max_r lse_r,  out = sum_r e^(lse_r - m) O_r / sum_r e^(lse_r - m),
 *   lse = m + ln sum_r e^(lse_r - m).
 *   part_o    [R, B, Hq, D] fp32, 16-byte aligned (parts outermost, as an
 *             all-gather along a new leading dimension lays them out)
 *   part_lse  [R, B, Hq] fp32
 *   out       [B, Hq, D] bf16, round-to-nearest-even, 16-byte aligned
 *   lse       [B, Hq] fp32 or NULL
 * R is in [1, 1024] and D is 64 or 128. A row whose parts are all empty gives
 * out = 0 and lse = -inf. Parts are summed in index order, so the result is
 * deterministic. It runs asynchronously on `stream`. */
FD_API fd_status fd_combine(int R, int B, int Hq, int D, const float* part_o,
                            const float* part_lse, void* out, float* lse, fd_stream_t stream);

/* fd_combine over parts placed at any stride, so that a gathered buffer is
 * merged where it lies, with no copy. Part r of row i (i = b * Hq + h) is the
 * D floats at part_o + r * o_stride + i * D and the lse at
 * part_lse[r * lse_stride + i]; fd_combine is the case o_stride = B*Hq*D,
 * lse_stride = B*Hq. One packed buffer per part, for example
 *   [O: B*Hq*D floats][lse: B*Hq floats][padding]
 * all-gathered into R consecutive buffers of P floats, is merged with
 *   part_o = buf, part_lse = buf + B*Hq*D, o_stride = lse_stride = P.
 * Strides count floats. o_stride must be a multiple of 4 and at least
 * B*Hq*D; lse_stride at least B*Hq; otherwise FD_ERR_INVALID_ARGUMENT. The
 * rest is as fd_combine. */
FD_API fd_status fd_combine_strided(int R, int B, int Hq, int D, const float* part_o,
                                    size_t o_stride, const float* part_lse, size_t lse_stride,
                                    void* out, float* lse, fd_stream_t stream);

/* Low-bit key codes for fd_decode_sparse ("Faster Than Flash: Exploiting
 * Attention Sparsity for Efficient Long-Context Decoding", abstract: a scan
 * over low-bit keys replaces metadata indices). Call it when the cache
 * changes (in a decode loop, for the blocks that tokens were appended to).
 * For every 64-token block of every (sequence, KV head):
 *   k8_scale = max |K| over the block's valid rows / 127 (1 for an all-zero
 *              block), fp32;
 *   k8       = rint(K / k8_scale) in [-127, 127], int8; rows at or past the
 *              sequence's length get 0.
 *   p         contiguous head-major bf16 cache (block_size 0, FD_LAYOUT_HND,
 *             FD_KV_BF16), D 64 or 128
 *   k_cache   [B, Hkv, max_len, D] bf16, 16-byte aligned
 *   seqlens   [B] int32 or NULL (all max_len)
 *   k8        [B, Hkv, max_len, D] int8 out, 16-byte aligned
 *   k8_scale  [B, Hkv, ceil(max_len / 64)] fp32 out
 * Returns FD_ERR_UNSUPPORTED for a paged, token-major, fp8 or 4-bit cache. */
FD_API fd_status fd_quantize_keys(const fd_problem* p, const void* k_cache,
                                  const int32_t* seqlens, int8_t* k8, float* k8_scale,
                                  fd_stream_t stream);

/* Sparse decode: fd_decode over the blocks a low-bit scan selects (same page,
 * abstract: a top-delta rule that filters blocks adaptively with no global
 * synchronisation, selector and computation fused in one kernel). Inside the
 * split kernel, before any K/V tile is loaded, each CTA (one split of one
 * KV head of one sequence):
 *   1. turns each query head of the group into int8: sq = max |q| / 127,
 *      q8 = rint(q / sq);
 *   2. computes for every 64-token block of its split, and every head, the
 *      largest approximate logit ((scale * sq) * k8_scale) * (q8 . k8), with
 *      the dot product exact in integers and each product rounded to fp32 in
 *      that order;
 *   3. keeps a block when some head's block maximum is >= M - delta, M being
 *      that head's largest block maximum in the split;
 *   4. runs the exact bf16 attention of fd_decode over the kept blocks only.
 * The splits then merge as in fd_decode. The result is the exact attention
 * over the union of the kept blocks. delta = +inf keeps every block and gives
 * fd_decode's result bit for bit.
 *   k8, k8_scale  from fd_quantize_keys on the same cache and lengths
 *   delta         >= 0, natural-log units (NaN is invalid)
 *   kept          [B, Hkv, ceil(max_len / 64)] uint8 out (1 = kept), or NULL.
 *                 Blocks at or past a sequence's length are not written.
 * Other arguments are those of fd_decode with a contiguous head-major bf16
 * cache and D = 128 (FD_ERR_UNSUPPORTED otherwise). The split count must make
 * the largest split (fd_split_chunk) at most 16,384 tokens
 * (FD_ERR_INVALID_ARGUMENT otherwise). The
 * codes stream through the split kernel's tile pipeline (TMA, 256 tokens per
 * stage) and the dot products run on int8 tensor cores. Results are
 * deterministic. */
FD_API fd_status fd_decode_sparse(const fd_problem* p, const void* q, const void* k_cache,
                                  const void* v_cache, const int8_t* k8,
                                  const float* k8_scale, const int32_t* seqlens, float scale,
                                  float delta, int num_splits, void* out, float* lse,
                                  uint8_t* kept, void* workspace, size_t workspace_bytes,
                                  fd_stream_t stream);

/* ---- a KV cache held in 4 bits ----------------------------------------------
 *
 * A row of the cache is one token of one KV head: D entries (64 or 128) in two
 * groups of D / 2. An entry of a group is held as a code c in 0..15, the group
 * has a bf16 scale s and a bf16 bias b, and the entry stands for s (c - 8) + b.
 *   k4, v4   uint8, D / 2 bytes per row, entry 2j in the low nibble of byte j,
 *            in the orders of fd_decode's caches with D / 2 for D:
 *            [B, Hkv, max_len, D/2], [num_blocks, Hkv, block_size, D/2],
 *            [B, max_len, Hkv, D/2] or [num_blocks, block_size, Hkv, D/2]
 *   params   bf16, one record of 8 per row, the same orders with 8 for D / 2:
 *            ks0 kb0 ks1 kb1 vs0 vb0 vs1 vb1 (scale and bias of K's groups,
 *            then of V's)
 * All three are 16-byte aligned and row-major. A row takes D + 16 bytes for K
 * and V together: 4.5 bits an entry at D = 128, 5 at D = 64 (bf16: 16).
 * fd_problem describes the cache as for fd_decode, with kv_dtype = FD_KV_INT4;
 * k_scale, v_scale and fp8_mma are ignored. The entry points below return
 * FD_ERR_INVALID_ARGUMENT for another kv_dtype. For FD_KV_INT4 fd_decode,
 * fd_decode_partial, fd_decode_sparse and fd_decode_static_workspace return it too,
 * and fd_quantize_keys returns FD_ERR_UNSUPPORTED, as for every cache that is not
 * bf16. */

/* Quantises new K and V rows and writes them into a 4-bit cache. Per group of
 * a row, with mn and mx its smallest and largest entry:
 *   s = bf16((mx - mn) / 15)     b = bf16(mn + 8 s)
 *   c = clamp(rint((x - b) / s), -8, 7) + 8
 * in fp32, rounding to nearest, ties to even ((mx - mn) / 15 is rounded to fp32
 * before bf16; mn + 8 s is rounded once to fp32, then to bf16). A group whose
 * entries are all equal gets s = 0, c = 8. A group that holds a NaN or an
 * infinity gets s = b = NaN, so that attention over it gives NaN, as it does
 * over a bf16 cache. s and b are rounded, so that a code may stand for a value
 * beyond mn .. mx by about 2^-7 of the larger of |mn| and |mx|; next to the largest bf16
 * that is an infinity once it is rounded to bf16.
 *   p         the cache (max_blocks_per_seq and max_len are checked, not used,
 *             when it is paged; Hq only as Hq % Hkv)
 *   n_tokens  rows of k_new and v_new, >= 0; 0 launches nothing. n_tokens * Hkv
 *             is below 2^31.
 *   k_new, v_new
 *             bf16, 16-byte aligned: token i, head h starts at element
 *             i * k_stride + h * D (v_stride for V), so that slices of a fused
 *             projection's output are read where they lie. Strides count
 *             elements, are multiples of 8 and at least Hkv * D.
 *   slots     [n_tokens] int64, 8-byte aligned: the place of each token,
 *             page * block_size + row in a paged cache and b * max_len + t in
 *             a contiguous one. A token whose slot is negative or outside the
 *             cache is skipped. A slot may appear once; of two tokens with the
 *             same slot either one's codes or records may be found there.
 * Rows of other slots are left as they were. */
FD_API fd_status fd_append_int4(const fd_problem* p, int n_tokens, const void* k_new,
                                int64_t k_stride, const void* v_new, int64_t v_stride,
                                const int64_t* slots, void* k4, void* v4, void* params,
                                fd_stream_t stream);

/* The rows of a 4-bit cache as a contiguous bf16 cache: s (c - 8) + b, rounded
 * once. The result is a cache for fd_decode and the entry points beside it, and
 * what the attention of a prompt reads when it is to see the same K and V as the
 * later steps.
 *   k4, v4, params, seqlens, block_table   as for fd_decode_int4
 *   k_out, v_out   bf16, 16-byte aligned: [B, Hkv, max_len, D]
 *                  (FD_LAYOUT_HND) or [B, max_len, Hkv, D] (FD_LAYOUT_NHD),
 *                  with p's max_len for a paged cache too. Rows at or past a
 *                  sequence's length are left as they were. A page id outside
 *                  [0, num_blocks) gives zeros. */
FD_API fd_status fd_expand_int4(const fd_problem* p, const void* k4, const void* v4,
                                const void* params, const int32_t* seqlens,
                                const int32_t* block_table, void* k_out, void* v_out,
                                fd_stream_t stream);

/* Decode attention over a 4-bit cache: fd_decode over the values that the
 * codes stand for. D is 64 or 128; G, layouts, pages, lengths, scale, out and lse
 * are as for fd_decode, and rows at or past a sequence's length may hold
 * anything. A page id outside [0, num_blocks) reads zeros. max_len is at most
 * 0x7fffff00, and B * Hkv * (max_len / 32 + 2) below 2^31
 * (FD_ERR_INVALID_ARGUMENT otherwise).
 *   num_splits  1: one thread-block cluster per (sequence, KV head), of one to
 *               eight CTAs by the sizes in p, and no workspace. Above 1 the
 *               tokens of the whole batch are dealt evenly to the SMs, whatever
 *               the lengths, and a second kernel merges what a row's CTAs have;
 *               the count only says how large a workspace there is: with fewer
 *               than fd_plan_problem's, fewer CTAs may share the work. At most
 *               1024.
 *   workspace   fd_workspace_bytes(B, Hq, D, num_splits) bytes for num_splits
 *               above 1 (FD_ERR_WORKSPACE if it is smaller); nothing is kept in it
 *               between calls.
 * Scores and sums are taken in fp32. A softmax weight enters the product with V's
 * codes as weight * scale in f16 (11 significant bits), relative to a power of
 * two above the largest V scale (and 2^-64 of the largest V bias) that its warp has
 * seen, and counts to 2^-15 of the largest among the 16 tokens beside it; entries of
 * q count in the same way among 16 channels. V may be of any finite size: no sum on the way is larger than the result.
 * q, K and scale may be of any size whose scores are finite: scale * max|q| *
 * max|K| * D below 2^126, with the maxima over the G heads of q and the rows of K
 * that meet. The result of a call is the same bits every time; how a sequence's sum
 * is split over CTAs, and with it the last bits of its result, depends on the other
 * sequences' lengths when num_splits is above 1, but not on the order of the cache's
 * dimensions or pages. */
FD_API fd_status fd_decode_int4(const fd_problem* p, const void* q, const void* k4,
                                const void* v4, const void* params, const int32_t* seqlens,
                                const int32_t* block_table, float scale, int num_splits,
                                void* out, float* lse, void* workspace, size_t workspace_bytes,
                                fd_stream_t stream);

/* ---- pages of a paged cache, kept on the device -------------------------------
 *
 * The pool's free pages are a stack: free_pages[0 .. free_count - 1], with
 * free_pages of num_pages entries. Both calls are functions of device memory
 * alone, with no wait on the host, so that a decode loop can be captured. The
 * new lengths and the new count may be written over the old ones
 * (seqlens_out == seqlens, free_count_out == free_count) or elsewhere; no other
 * output may share memory with an input or with another output.
 * B is in [1, 65535], block_size a power of two in [8, 256]
 * (FD_ERR_UNSUPPORTED otherwise). Lengths are clamped to [0,
 * max_blocks_per_seq * block_size], free_count to [0, num_pages]. */

/* Pages and slots for the new tokens of a batch. Request b holds seqlens[b]
 * tokens and gets new_lens[b] more (negative: 0): in the order of the requests
 * each takes from the top of the stack the pages that its new tokens need
 * beyond those it has, and they are written into its row of block_table (other
 * entries are left as they were). The new tokens of all requests are listed
 * one request after another:
 *   cu_new     [B + 1] int32: request b's are cu_new[b] .. cu_new[b + 1] - 1;
 *              the list ends at max_tokens, and what is beyond it is not
 *              listed and not counted
 *   slots      [max_tokens] int64, 8-byte aligned: page * block_size + row of
 *              each new token, as fd_append_int4 takes them; -1 where the
 *              request's table row or the pool is exhausted, and behind the
 *              last token
 *   positions  [max_tokens] int32 or NULL: the token's index in its sequence;
 *              0 behind the last token
 *   seqlens_out     [B] int32: tokens that have a place. Less than seqlens[b] +
 *                   new_lens[b] when the request could not be served in full.
 *   free_count_out  [1] int32: pages still free
 * max_tokens is >= 0 (slots may be NULL when it is 0). */
FD_API fd_status fd_alloc_pages(int B, int block_size, int max_blocks_per_seq, int max_tokens,
                                int num_pages, const int32_t* seqlens, const int32_t* new_lens,
                                const int32_t* free_pages, const int32_t* free_count,
                                int32_t* block_table, int32_t* seqlens_out, int32_t* cu_new,
                                int64_t* slots, int32_t* positions, int32_t* free_count_out,
                                fd_stream_t stream);

/* Gives the pages of finished requests back. Request b is finished when
 * done[b] is not 0: the ceil(seqlens[b] / block_size) pages of its table row go
 * on top of the stack, in the order of the requests, and its length becomes 0.
 * Pages that do not fit num_pages are dropped.
 *   done            [B] uint8
 *   seqlens_out     [B] int32: 0 for a finished request, its length otherwise
 *   free_count_out  [1] int32 */
FD_API fd_status fd_release_pages(int B, int block_size, int max_blocks_per_seq, int num_pages,
                                  const int32_t* seqlens, const uint8_t* done,
                                  const int32_t* block_table, int32_t* free_pages,
                                  const int32_t* free_count, int32_t* seqlens_out,
                                  int32_t* free_count_out, fd_stream_t stream);

/* Largest workspace, in bytes, that fd_decode_static_workspace can use. */
#define FD_STATIC_WORKSPACE_BYTES (8u << 20)

/* fd_decode for callers that cannot allocate device memory.
 * The Flash-Decoding pages have no counterpart to this entry point; it is an
 * addition of this library. Some callers cannot call cudaMalloc at all. Examples: a plain C
 * host program that links only this library and has no device allocator of
 * its own; code inside a framework whose memory pool owns all device memory
 * and forbids raw allocations; a decode loop that must not call cudaMalloc
 * mid-step, because it can block on the device and can fail when memory runs
 * short.
 * Such callers still pass q, the caches, seqlens, block_table, out and lse,
 * exactly as for fd_decode. The workspace comes from a file-scope static
 * __device__ array of FD_STATIC_WORKSPACE_BYTES bytes, which every GPU that
 * loads this library holds until the process exits. This entry point calls
 * no cudaMalloc, cudaFree or other allocating routine.
 *  - Set-up: the first call on a device looks up the array's device address
 *    with the device current (cudaGetSymbolAddress) and caches it with the
 *    id of the device's context. Make that first call before any stream
 *    capture on that device. After a device reset (cudaDeviceReset) the
 *    device has a new context, in which the array may sit elsewhere: the
 *    next call sees the new context id and looks the address up again, so
 *    make that call, too, outside a capture.
 *  - Size limit: when the effective split count needs more than
 *    FD_STATIC_WORKSPACE_BYTES (see fd_workspace_bytes), the call returns
 *    FD_ERR_WORKSPACE and launches nothing. Pass a smaller num_splits, or use
 *    fd_decode with your own workspace.
 *  - Sharing: every call on a device uses the same array, which keeps the
 *    last call's contents. Nothing in it has to start at zero, because each
 *    call writes every partial result before reading it. Calls that overlap
 *    on the GPU, such as calls on two streams, race on the array and give
 *    wrong results: serialise them.
 * Returns the same codes as fd_decode. */
FD_API fd_status fd_decode_static_workspace(const fd_problem* p, const void* q,
                                            const void* k_cache, const void* v_cache,
                                            const int32_t* seqlens,
                                            const int32_t* block_table, float scale,
                                            int num_splits, void* out, float* lse,
                                            fd_stream_t stream);

/* Waits for `stream`, then reads and clears the current device's error word.
 * A kernel sets that word when one of its bounded waits runs out. Returns
 * FD_OK, FD_ERR_DEVICE_TIMEOUT, or FD_ERR_CUDA. */
FD_API fd_status fd_check_device_error(fd_stream_t stream);

/* Diagnostic of the failure path. Launches one warp that waits, with the
 * same bounded wait the kernels use, on an mbarrier that nothing ever
 * completes. After limit_us microseconds the wait gives up, and the kernel
 * sets the device error word the way a stalled split kernel would. The next
 * fd_check_device_error(stream) then returns FD_ERR_DEVICE_TIMEOUT and
 * clears the word. Nothing faults or hangs, and the context stays usable.
 * limit_us must be in [1, 5,000,000]. Returns FD_OK once launched. */
FD_API fd_status fd_selftest_device_timeout(unsigned int limit_us, fd_stream_t stream);

/* Static, human-readable name of a status code. */
FD_API const char* fd_status_string(fd_status status);

#ifdef __cplusplus
}
#endif

#endif /* FD_H_ */

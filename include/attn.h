/*
 * attn.h -- C ABI of the GB300 (sm_103a) exact tiled attention library.
 *
 * The library computes exact scaled-dot-product attention in the
 * FlashAttention style: blockwise Q K^T, an FP32 online softmax (running
 * row max and row sum, rescaling of the partial output) and blockwise P V,
 * forward and backward.  The operation is the "Baseline Attention" of
 * "Is Flash Attention Stable?" (abstract): O = softmax(scale * Q K^T) V, with
 * an optional causal mask; its tiled evaluation follows the block division
 * of "Why Low-Precision Transformer Training Fails", Algorithm 1 (Q split
 * into row blocks, K and V into column blocks).  The backward pass uses
 * delta = rowsum(dO o O) as defined in that paper (Figures 3 and 5).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors Q, K, V, O, dO, dQ, dK, dV are [B, H, N, d], contiguous,
 *    d fastest, in DEVICE memory (device or managed allocations), 16-byte
 *    aligned.  LSE is FP32 [B, H, N] (natural log): LSE_i = ln sum_j
 *    exp(scale * q_i . k_j) over the visible keys.
 *  - causal != 0 hides key j from query i when j > i (square, top-left).
 *  - dt selects the element type of Q, K, V, O, dO, dQ, dK, dV:
 *      ATTN_DTYPE_BF16 -- tensor-core path (TMA + tcgen05/TMEM), FP32
 *                         softmax and accumulation, BF16 results;
 *      ATTN_DTYPE_FP32 -- reference mode: the same tiled online softmax in
 *                         FP32 CUDA-core arithmetic (no tensor cores).
 *  - Supported: d in {64, 128}; N >= 1; B*H*N*d < 2^31; scale finite > 0.
 *  - Ownership: the caller allocates every buffer and owns the stream; the
 *    library makes no allocation calls and keeps no per-call state (its one
 *    fixed device array is described at attn_bwd_noalloc).
 *  - Asynchrony: kernels are enqueued on `stream` and the call returns
 *    without synchronizing.  Argument errors are reported synchronously,
 *    before anything is enqueued; launch failures map to ATTN_ERR_CUDA.
 *  - Every wait inside a kernel is bounded (about 2 s).  A wait that gives
 *    up records ATTN_ERR_TIMEOUT on the device and the kernel returns;
 *    attn_check_status() reports it.
 *  - The device is the one current on the calling thread; all pointers
 *    must belong to it.
 */
#ifndef ATTN_H_
#define ATTN_H_

#include <stddef.h>

#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1, /* bad pointer, shape, scale or workspace size */
  ATTN_ERR_UNSUPPORTED = 2, /* valid request outside the supported set     */
  ATTN_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed           */
  ATTN_ERR_TIMEOUT = 4      /* a bounded in-kernel wait gave up            */
} attn_status;

typedef enum { ATTN_DTYPE_BF16 = 0, ATTN_DTYPE_FP32 = 1 } attn_dtype;

/* Library version, major * 10000 + minor * 100 + patch. */
ATTN_API int attn_version(void);

/* Static description of a status code. */
ATTN_API const char* attn_status_string(attn_status s);

/* Human-readable detail of the last error returned on the calling thread
 * (empty string when none).  The pointer stays valid until the next call on
 * the same thread. */
ATTN_API const char* attn_last_error(void);

/*
 * Forward pass ("Is Flash Attention Stable?", abstract: Baseline Attention;
 * tiled as in "Why Low-Precision Transformer Training Fails", Algorithm 1).
 *   q, k, v : [B,H,N,d] inputs (dt).
 *   o       : [B,H,N,d] output (dt), O = softmax(scale Q K^T [+mask]) V.
 *   lse     : [B,H,N] FP32 output, natural-log log-sum-exp of each row of
 *             scale Q K^T over the visible keys.
 * Returns ATTN_OK once the kernel is enqueued.
 */
ATTN_API attn_status attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                              int B, int H, int N, int d, float scale, int causal, attn_dtype dt,
                              cudaStream_t stream);

/*
 * Forward pass with the stabilised normaliser of "Why Low-Precision Transformer
 * Training Fails" (Figure 7 and Algorithm 1): while a row's running maximum
 * r_m of scale * q.k is attained by two or more keys, the exponentials are
 * taken relative to m = beta * r_m if r_m > 0 and m = 0 if r_m <= 0, so that
 * no unnormalised probability exp(S - m) is exactly 1.  Mathematically O and
 * LSE are those of attn_fwd (LSE is formed with the normaliser actually
 * used); only the rounding differs.  attn_bwd accepts its outputs unchanged.
 * BF16 only; beta must be finite and > 1.  With c = scale * log2(e), m is
 * then kept within [r_m + 2^-8 / c, r_m + 64 / c]:
 *   - the floor makes the row's largest exponent "sufficiently negative" (the
 *     paper's words) once rounded: 2^(c (r_m - m)) <= 2^(-2^-8) rounds to at
 *     most 1 - 2^-8 in BF16, also for repeated maxima that are 0, tiny, or
 *     tiny and negative, where beta * r_m or 0 alone would leave the BF16
 *     operand of the P V product at exactly 1;
 *   - the cap keeps the largest exponential at or above 2^-64, so a very
 *     large repeated maximum cannot underflow the whole row.
 */
ATTN_API attn_status attn_fwd_stable(const void* q, const void* k, const void* v, void* o,
                                     float* lse, int B, int H, int N, int d, float scale,
                                     int causal, float beta, attn_dtype dt, cudaStream_t stream);

/*
 * Per-token symmetric INT8 quantization ("INT-FlashAttention: Enabling Flash
 * Attention for INT8 Quantization", abstract; the page fixes no scheme, the
 * one here is a reading): for every row r of every head of the BF16 tensor
 * x [B,H,N,d], scales[r] = max_j |x_rj| / 127 (FP32) and codes[r][j] =
 * rint(x_rj / scales[r]) clamped to [-127, 127], rint rounding half to even;
 * a row of zeros gets scale 0 and codes 0.
 *   x      : [B,H,N,d] BF16, device.
 *   codes  : [B,H,N,d] int8, device, written.
 *   scales : [B,H,N] FP32, device, written.
 * d in {64, 128}; all pointers 16-byte aligned.
 */
ATTN_API attn_status attn_quantize_int8(const void* x, void* codes, float* scales, int B, int H,
                                        int N, int d, cudaStream_t stream);

/*
 * Forward on per-token INT8 Q and K (as written by attn_quantize_int8) and
 * BF16 V: S_ij = scale * q_scale[i] * k_scale[j] * (q8_i . k8_j) with the
 * integer dot product exact, then the FP32 online softmax and P V (P rounded
 * to BF16), O = softmax(S [+mask]) V and LSE = ln sum_j exp(S_ij) as in
 * attn_fwd.  sm_103a has no INT8 tcgen05 MMA, so this path runs on the
 * warp-level mma.sync tensor-core instructions and is several times slower
 * than attn_fwd; attn_fwd_int8_as_bf16 computes the same scores on the
 * tcgen05 path from codes held in BF16.
 *   q8, k8  : [B,H,N,d] int8, device.   q_scale, k_scale : [B,H,N] FP32.
 *   v       : [B,H,N,d] BF16.           o : [B,H,N,d] BF16.   lse : [B,H,N] FP32.
 * d in {64, 128}; all pointers 16-byte aligned, device memory.
 */
ATTN_API attn_status attn_fwd_int8(const void* q8, const float* q_scale, const void* k8,
                                   const float* k_scale, const void* v, void* o, float* lse,
                                   int B, int H, int N, int d, float scale, int causal,
                                   cudaStream_t stream);

/*
 * The quantization of attn_quantize_int8 with the codes held in BF16: every
 * code is an integer in [-127, 127], which BF16 represents exactly, so these
 * are the same codes in a 2-byte type.  The scales are laid out per head with
 * the row count padded: scales[(b*H + h) * N_pad + n], N_pad = N rounded up
 * to a multiple of 128; the padded entries are written as 0.
 *   x      : [B,H,N,d] BF16, device.
 *   codes  : [B,H,N,d] BF16, device, written.
 *   scales : B*H*N_pad FP32, device, written.
 * d in {64, 128}; all pointers 16-byte aligned.
 */
ATTN_API attn_status attn_quantize_int8_as_bf16(const void* x, void* codes, float* scales, int B,
                                                int H, int N, int d, cudaStream_t stream);

/*
 * attn_fwd_int8 on codes held in BF16 (attn_quantize_int8_as_bf16): the same
 * scores S_ij = scale * q_scale[i] * k_scale[j] * (q8_i . k8_j), the integer
 * dot product exact, evaluated on the BF16 tcgen05 path of attn_fwd -- every
 * product of two codes (|c| <= 127) and every partial sum over d <= 128
 * terms (< 2^24) is exact in the FP32 accumulator, whatever the order.  The
 * row scale is clamped below at 1e-20 (a row of zero codes has zero scores
 * either way).  Compared with attn_fwd_int8, Q and K take two bytes per code
 * and the path runs at the speed of the BF16 forward.
 *   q_codes, k_codes : [B,H,N,d] BF16 holding integer codes, device.
 *   q_scale, k_scale : B*H*N_pad FP32 (layout of attn_quantize_int8_as_bf16).
 *   v : [B,H,N,d] BF16.   o : [B,H,N,d] BF16.   lse : [B,H,N] FP32.
 * d in {64, 128}; all pointers 16-byte aligned, device memory.
 */
ATTN_API attn_status attn_fwd_int8_as_bf16(const void* q_codes, const float* q_scale,
                                           const void* k_codes, const float* k_scale,
                                           const void* v, void* o, float* lse, int B, int H,
                                           int N, int d, float scale, int causal,
                                           cudaStream_t stream);

/*
 * Bytes of device workspace attn_bwd needs for this problem (0 on invalid
 * arguments).  Layout (internal): -LSE*log2(e) and delta, FP32 [B*H][Npad]
 * each, and the FP32 dQ accumulator [B*H][Npad][d], Npad = N rounded up to
 * 128.  The workspace needs no initialisation; attn_bwd overwrites it.
 */
ATTN_API size_t attn_bwd_workspace_bytes(int B, int H, int N, int d, attn_dtype dt);

/*
 * Backward pass from the saved LSE: dQ, dK, dV of L = sum(dO o O).
 * The gradient of the attention definition, with delta = rowsum(dO o O)
 * ("Why Low-Precision Transformer Training Fails", Figures 3 and 5),
 * dS = P o (dO V^T - delta), dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO.
 *   q, k, v, o, dout : [B,H,N,d] inputs (dt); o is the forward output.
 *   lse              : [B,H,N] FP32, the forward's LSE.
 *   dq, dk, dv       : [B,H,N,d] outputs (dt).
 *   workspace        : device buffer of at least
 *                      attn_bwd_workspace_bytes(...) bytes, 256-byte aligned,
 *                      not shared with a concurrently running call.
 * Enqueues three kernels on `stream`: preprocess (delta, -LSE*log2(e), zero
 * the dQ accumulator), the main kernel (dK, dV, dQ accumulation), and the
 * dQ conversion (scale and round).  The three phases are also exported
 * below so that each can be timed on its own.
 */
ATTN_API attn_status attn_bwd(const void* q, const void* k, const void* v, const void* o,
                              const float* lse, const void* dout, void* dq, void* dk, void* dv,
                              int B, int H, int N, int d, float scale, int causal, attn_dtype dt,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Phase 1 of attn_bwd (BF16 only): delta_i = rowsum(dO o O)_i in FP32 from
 * the stored O, -LSE*log2(e), and a zeroed dQ accumulator, into `workspace`. */
ATTN_API attn_status attn_bwd_preprocess(const void* o, const float* lse, const void* dout, int B,
                                         int H, int N, int d, attn_dtype dt, void* workspace,
                                         size_t workspace_bytes, cudaStream_t stream);

/* Phase 2 of attn_bwd (BF16 only): dK and dV (written to dk, dv) and the FP32
 * dQ accumulation into `workspace`; needs phase 1 to have run on it. */
ATTN_API attn_status attn_bwd_main(const void* q, const void* k, const void* v, const void* dout,
                                   void* dk, void* dv, int B, int H, int N, int d, float scale,
                                   int causal, attn_dtype dt, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/* Phase 3 of attn_bwd (BF16 only): dQ = bf16(scale * accumulator). */
ATTN_API attn_status attn_bwd_dq_convert(void* dq, int B, int H, int N, int d, float scale,
                                         attn_dtype dt, void* workspace, size_t workspace_bytes,
                                         cudaStream_t stream);

/*
 * Synchronizes `stream`, then reads and clears the device-side status words
 * of the library on the current device.  Returns ATTN_ERR_TIMEOUT if any
 * kernel gave up on a bounded wait since the last check, ATTN_ERR_CUDA if
 * the stream reports an error, else ATTN_OK.
 *
 * The status words are per device and per process, not per stream or per
 * call: a timeout recorded by any of this library's kernels on the current
 * device, launched from any stream or host thread, is reported by the next
 * attn_check_status on that device, whatever stream it is given, and that
 * check clears it.  `stream` only selects what is synchronized first; a
 * caller that needs to attribute a timeout to one call must check after that
 * call with no other call of the library in flight on the device.
 */
ATTN_API attn_status attn_check_status(cudaStream_t stream);

/*
 * Self-test of the bounded-wait path: enqueues a one-block kernel that waits
 * on a shared-memory barrier nothing ever arrives at, for at most limit_ns
 * nanoseconds (1 <= limit_ns <= 10^9), then records ATTN_ERR_TIMEOUT and
 * returns.  attn_check_status() afterwards must report ATTN_ERR_TIMEOUT.
 */
ATTN_API attn_status attn_selftest_wait_timeout(unsigned long long limit_ns, cudaStream_t stream);

/*
 * attn_bwd without a caller workspace, for callers that must not allocate
 * device memory (no counterpart in the pages: this is a library-usage entry
 * point, not part of the method).  Typical such callers run inside a host
 * framework that owns the whole device-memory budget, or in latency-critical
 * loops where cudaMalloc/cudaFree and their implicit synchronization are not
 * acceptable.  Same arguments and results as attn_bwd with dt = BF16; the
 * scratch (-LSE*log2(e), delta, FP32 dQ accumulator) lives in a fixed 32 MiB
 * device array inside the library instead of `workspace`.
 *   - Limit: attn_bwd_workspace_bytes(B, H, N, d, BF16) must be at most
 *     33554432 bytes (e.g. B8 H12 N1024 d64 fits); larger problems return
 *     ATTN_ERR_INVALID_ARG before anything is launched.
 *   - The array occupies 32 MiB on each GPU where the library's module is
 *     loaded (at the latest from this entry point's first call there) until
 *     the process exits.  No call allocates memory.
 *   - All calls share the array: calls that can overlap on the GPU (other
 *     streams, unordered host threads) race and give wrong results.  Each call
 *     rewrites what it reads (the dQ accumulator is zeroed every call).
 *   - The first call on a device looks up the array's device address; make
 *     that first call before any stream capture.  The address is kept with
 *     the id of the CUDA context it belongs to; after cudaDeviceReset the next
 *     call looks it up again, so that call too belongs before any capture.
 *   - Shape errors are those of attn_bwd (ATTN_ERR_UNSUPPORTED for a head size
 *     outside {64, 128}, ATTN_ERR_INVALID_ARG for a bad N, B*H or scale).
 */
ATTN_API attn_status attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                                      const float* lse, const void* dout, void* dq, void* dk,
                                      void* dv, int B, int H, int N, int d, float scale,
                                      int causal, cudaStream_t stream);

/*
 * Serving: prompts of different lengths, and a paged INT8 cache
 * ---------------------------------------------------------------
 * These entry points work on PACKED sequences with GROUPED heads: a batch of B
 * sequences lies one behind the other in tensors of T tokens, sequence b in
 * tokens [cu_seqlens[b], cu_seqlens[b+1]); H query heads share H_kv key heads
 * (H a multiple of H_kv, at most 64 times it), query head h using key head
 * h / (H / H_kv).  d in {64, 128}, BF16 inputs.  Rows have d contiguous elements;
 * token and head strides (in elements, multiples of 8) are given, so q, k and v
 * may be views of one projection's output.
 *
 * Lengths, page numbers and plans lie in device memory and are read by the
 * kernels, so a call can be captured in a CUDA graph and replayed on new ones.
 * They cannot be checked before the launch: a value out of range never leads
 * outside the tensors, and attn_check_status() reports ATTN_ERR_INVALID_ARG.  Pages
 * whose number is out of range are neither written nor seen; appending leaves out
 * a sequence whose length or start is, and the other calls cut lengths to
 * what the tensors hold.  A sequence may have no token at all.
 *
 * The cache: codes k_cache, v_cache int8 [num_pages, H_kv, page_size, d],
 * contiguous, and scales k_scale, v_scale FP32 [num_pages, H_kv]; a code c stands
 * for c * scale.  Position t of sequence b is row t % page_size of page
 * block_table[b * max_blocks + t / page_size].  page_size in {16, 32, 64, 128};
 * num_pages * H_kv * page_size < 2^31.  Entries of the table behind a sequence's
 * last page are never used.
 */

/* Bytes of the plan of attn_varlen_plan (0 on invalid arguments). */
ATTN_API size_t attn_varlen_plan_bytes(int B, int T, int H, int H_kv);

/*
 * Lists the work of attn_varlen_fwd on a packed batch, heaviest first, from the
 * sequences' lengths.  One plan serves any number of calls with the same
 * cu_seqlens, T, H, H_kv and causal flag (every layer of a model, say).
 *   cu_seqlens : int32 [B+1], device: 0 <= cu_seqlens[b] <= cu_seqlens[b+1] <= T.
 *                Tokens from cu_seqlens[B] on belong to no sequence.
 *   plan       : device buffer of attn_varlen_plan_bytes(...) bytes, 16-byte
 *                aligned, written.
 */
ATTN_API attn_status attn_varlen_plan(const int* cu_seqlens, int B, int T, int H, int H_kv, int causal,
                                      void* plan, size_t plan_bytes, cudaStream_t stream);

/*
 * Attention over whole prompts: for every token i of a sequence and head h,
 * O = sum_j softmax_j(scale q_i . k_j) v_j over the sequence's own tokens j
 * (causal != 0: j <= i), and the natural-log LSE.
 *   q    : [T,H,d] BF16;  k, v : [T,H_kv,d] BF16, with the given strides.
 *   plan : of attn_varlen_plan for the same B, T, H, H_kv and causal; a plan made
 *          for another T, group size, H_kv or causal flag is reported by
 *          attn_check_status() and nothing is computed.
 *   o    : [T,H,d] BF16, contiguous.   lse : [T,H] FP32.
 * Rows of o and lse that belong to no sequence are left as they were.  What lies
 * in other sequences' rows (a NaN, say) does not reach a sequence; a NaN or an
 * infinity in v at token j of a sequence may reach the rows of earlier tokens in
 * j's block of 128 keys, and of up to 127 tokens before that block, although the
 * causal mask hides it from them.
 */
ATTN_API attn_status attn_varlen_fwd(const void* q, const void* k, const void* v,
                                     long long q_token_stride, long long q_head_stride,
                                     long long k_token_stride, long long k_head_stride,
                                     long long v_token_stride, long long v_head_stride,
                                     const void* plan, size_t plan_bytes, void* o, float* lse, int B,
                                     int T, int H, int H_kv, int d, float scale, int causal,
                                     cudaStream_t stream);

/*
 * Writes new rows into the cache: token cu_seqlens[b] + i goes to position
 * starts[b] + i of sequence b.  For every page and head the new rows fall into,
 * with a the largest |x| of their finite elements:
 *   a page whose first row is among them takes scale s = a / 127 (FP32);
 *   a page begun earlier takes s = max(its scale, a / 127), and where that is
 *   larger than before, the rows it holds become rint(c * s_old / s).
 * New codes are rint(x / s), all clamped to [-127, 127], with rint half to even
 * of the exact quotient (s = 0: codes 0; NaN: 0; an infinity: +-127).  Rows of a
 * page behind the new ones are left as they were.
 *   k, v   : [T,H_kv,d] BF16, with the given strides.
 *   starts : int32 [B], device: positions each sequence holds already.
 * The pages that one call writes must be distinct: a page shared by two
 * sequences is copied before either writes to it.
 */
ATTN_API attn_status attn_cache_append_int8(const void* k, const void* v, long long k_token_stride,
                                            long long k_head_stride, long long v_token_stride,
                                            long long v_head_stride, void* k_cache, void* v_cache,
                                            float* k_scale, float* v_scale, const int* block_table,
                                            const int* cu_seqlens, const int* starts, int B, int T,
                                            int H_kv, int d, int num_pages, int page_size,
                                            int max_blocks, cudaStream_t stream);

/*
 * attn_cache_append_int8 without the rows from position lens[b] on (int32 [B], device, 0 or more):
 * they are neither written nor counted into a scale, and their pages are not looked up.  With the
 * lens that attn_cache_reserve has written these are the rows of the requests that were not served,
 * which leave the cache as it was; nothing is reported for them.
 */
ATTN_API attn_status attn_cache_append_served_int8(
    const void* k, const void* v, long long k_token_stride, long long k_head_stride,
    long long v_token_stride, long long v_head_stride, void* k_cache, void* v_cache, float* k_scale,
    float* v_scale, const int* block_table, const int* cu_seqlens, const int* starts, const int* lens,
    int B, int T, int H_kv, int d, int num_pages, int page_size, int max_blocks, cudaStream_t stream);

/*
 * Reads ranges of positions back as values code * scale: packed token
 * cu_seqlens[b] + i of the outputs is position starts[b] + i of sequence b.
 *   k, v : [T,H_kv,d] of type dt (the product in FP32, or that rounded to BF16),
 *          contiguous, written; 0 = cu_seqlens[0] <= cu_seqlens[b] <= cu_seqlens[b+1],
 *          cu_seqlens[B] = T.  Other lengths are reported by attn_check_status();
 *          tokens outside the sequences or without a valid page become 0 and are
 *          reported as well.
 */
ATTN_API attn_status attn_cache_read_int8(const void* k_cache, const void* v_cache,
                                          const float* k_scale, const float* v_scale,
                                          const int* block_table, const int* cu_seqlens,
                                          const int* starts, void* k, void* v, int B, int T, int H_kv,
                                          int d, int num_pages, int page_size, int max_blocks,
                                          attn_dtype dt, cudaStream_t stream);

/* Bytes of device workspace attn_decode_int8 needs (0 also on invalid arguments). */
ATTN_API size_t attn_decode_int8_workspace_bytes(int B, int n_q, int H, int H_kv, int d,
                                                 int page_size, int max_blocks);

/*
 * Attention of the newest n_q tokens of every sequence over the cache: token i of
 * them sees positions j <= seqlens[b] - n_q + i.  With ck, cv the codes and ks, vs
 * the scales of position j's page and the query head's key head,
 * O = sum_j softmax_j(scale q . (ck_j ks_j)) (cv_j vs_j), LSE = ln sum_j exp.
 * A row that sees no position (seqlens[b] < n_q - i) gets O = 0, LSE = -inf.
 *   q       : [B,n_q,H,d] BF16, with the given strides; 1 <= n_q <= 256.
 *   seqlens : int32 [B], device: positions each sequence holds, the newest n_q
 *             tokens' among them; at most max_blocks * page_size.
 *   o       : [B,n_q,H,d] BF16, contiguous.   lse : [B,n_q,H] FP32.
 *   max_blocks : the room per sequence in the block table.  How the work is split over
 *             the SMs follows from it and B: a table far wider than the histories
 *             gives the same result, short ones a few microseconds later.
 *   workspace : device buffer, 256-byte aligned, that no concurrently running call
 *             uses (also not the replay of another graph); needs no initialisation.
 * The weights p_j vs_j of the codes (p the softmax) keep 11 bits down to 2^-20 of the
 * row's largest weight; below that they are off by at most 2^-31 of it, whatever the
 * scales of pages that the row does not see or barely weighs.  A p below 2^-126
 * counts as 0 or loses bits.
 * Scales must be >= 0 and finite.  A position whose page number is out of range
 * is not seen.
 */
ATTN_API attn_status attn_decode_int8(const void* q, long long q_batch_stride,
                                      long long q_token_stride, long long q_head_stride,
                                      const void* k_cache, const void* v_cache, const float* k_scale,
                                      const float* v_scale, const int* block_table,
                                      const int* seqlens, void* o, float* lse, int B, int n_q, int H,
                                      int H_kv, int d, int num_pages, int page_size, int max_blocks,
                                      float scale, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream);

/* Bytes of device workspace attn_decode_shared_int8 needs (0 also on invalid arguments). */
ATTN_API size_t attn_decode_shared_int8_workspace_bytes(int B, int n_q, int H, int H_kv, int d,
                                                        int page_size, int prefix_blocks,
                                                        int max_blocks);

/*
 * attn_decode_int8 for a batch whose sequences all begin with the same prefix_len
 * positions, which the cache holds once: token i of a sequence's newest n_q sees the
 * whole prefix and its own positions j <= seqlens[b] - n_q + i.  The prefix's codes are
 * read once for up to 256 of a key head's B * n_q * H / H_kv query rows, or once a
 * sequence, in one launch, where the prefix is short or the sequences are few.
 *   prefix_table  : int32 [prefix_blocks], device: the prefix's pages; position t is
 *                   row t % page_size of page prefix_table[t / page_size].  How the
 *                   prefix is read follows from prefix_blocks and the shape: a table far
 *                   wider than the prefix gives O within the same bounds, but not always the same
 *                   bits, and a short prefix takes up to twice as long (8 key heads of 128: 8 sequences
 *                   behind 400 positions 8.3 us, in a table for 32768 14.9; 64 behind 100 16 and 30).
 *   prefix_len    : int32 [1], device: 0 to prefix_blocks * page_size.
 *   block_table   : int32 [B, max_blocks]: the pages of each sequence's own positions,
 *                   which are counted from 0 behind the prefix (the first of them begins a
 *                   page, also where the prefix ends inside one).
 *   seqlens       : int32 [B]: own positions, the newest n_q tokens' among them.  A sequence
 *                   may have fewer than n_q, or none: its tokens then see the prefix alone.
 *   workspace     : device buffer, 256-byte aligned, that no concurrently running call
 *                   uses (also not the replay of another graph); needs no initialisation.
 * q, o, lse and the cache as for attn_decode_int8, and so is the weights' precision, with
 * 11 bits down to 2^-20 of a row's largest weight in the prefix, or in the own positions.  A
 * row that sees no position gets O = 0, LSE = -inf.  The same call gives the same bits.
 */
ATTN_API attn_status attn_decode_shared_int8(
    const void* q, long long q_batch_stride, long long q_token_stride, long long q_head_stride,
    const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    const int* prefix_table, int prefix_blocks, const int* prefix_len, const int* block_table,
    const int* seqlens, void* o, float* lse, int B, int n_q, int H, int H_kv, int d, int num_pages,
    int page_size, int max_blocks, float scale, void* workspace, size_t workspace_bytes,
    cudaStream_t stream);

/*
 * Block tables, offsets and slots of a step from the requests' lengths.  Sequence b holds
 * held[b] positions, whose pages are the first ceil(held[b] / page_size) of its row of the
 * table, and is to hold wanted[b]: more (new tokens), fewer (rejected drafts), none (it has
 * ended).  Pages that are held no longer go to the stack of free pages, then those that are
 * needed are taken from it, both in the order of the sequences and of their positions:
 *   - released pages are put at free_pages[n_free], free_pages[n_free + 1], ..., and their
 *     entries in the table become -1;
 *   - requests are served in their order for as long as the stack has the pages they need
 *     together; one that needs none is always served.  Those that are served take the topmost
 *     pages, the last one the topmost.  The entries that a request which is not served would
 *     have needed become -1, and it holds what it held.
 * So the reverse call (held = lens, wanted = the old held) takes a step back, table and stack
 * and all.
 *   block_table : int32 [B, max_blocks], device, updated.
 *   held, wanted: int32 [B], device, 0 to max_blocks * page_size.  A sequence with another
 *                 value is left as it is (lens = held, no tokens) and reported.
 *   free_pages  : int32 [num_pages], device, updated; entries from n_free on are free room.
 *   n_free      : int32 [1], device, updated.  Pages that the stack has no room for (more than
 *                 num_pages: some were given back twice) are dropped and reported; a number
 *                 out of range, in a table or in the stack, becomes -1 and is reported.
 *   lens        : int32 [B], written: wanted[b], or held[b] where the request was not served.
 *   cu_seqlens  : int32 [B+1], written: offsets of the packed new tokens, max(wanted - held, 0)
 *                 of every sequence, served or not.
 *   slots       : int32 [T], written: row block_table[..] * page_size + position % page_size of
 *                 the pool for each new token; -1 where its request was not served, and behind
 *                 the last token.
 *   positions   : int32 [T], written: each new token's position in its sequence; -1 behind the
 *                 last token.  More new tokens than T are reported, and the first T written.
 * num_pages * page_size < 2^31.  lens, cu_seqlens, slots and positions, and what is updated, overlap
 * nothing.  attn_cache_append_served_int8 takes cu_seqlens, held (as starts) and lens for the new
 * rows, and attn_decode_int8 takes lens.  (attn_cache_append_int8, which has no lens, is for steps whose
 * requests are all served: it would put the rows of one that was not into the room that its last page has, count
 * them into that page's scales, and report the pages that they lack.)  What attention gives for the new
 * tokens of a request that was not served is of no use: their positions are not there.
 */
ATTN_API attn_status attn_cache_reserve(int* block_table, const int* held, const int* wanted,
                                        int* free_pages, int* n_free, int* lens, int* cu_seqlens,
                                        int* slots, int* positions, int B, int T, int num_pages,
                                        int page_size, int max_blocks, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H_ */

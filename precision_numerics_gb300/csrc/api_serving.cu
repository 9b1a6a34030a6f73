// C-ABI entry points of the serving operators: argument validation and
// dispatch for attention over packed sequences, the paged INT8 cache and its
// block tables, and attention over that cache.
#include <limits.h>
#include <math.h>

#include "attn_internal.h"

namespace attn {
namespace {

attn_status check_heads(int H, int H_kv, int d) {
  if (H < 1 || H_kv < 1) return fail(ATTN_ERR_INVALID_ARG, "H and H_kv must be >= 1 (got H=%d H_kv=%d)", H, H_kv);
  if (H % H_kv != 0) return fail(ATTN_ERR_INVALID_ARG, "H=%d is not a multiple of H_kv=%d", H, H_kv);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d is not supported (64 or 128)", d);
  if (H / H_kv > 64) return fail(ATTN_ERR_UNSUPPORTED, "H / H_kv = %d is not supported (up to 64)", H / H_kv);
  if (H_kv > 65535) return fail(ATTN_ERR_UNSUPPORTED, "H_kv = %d is not supported (up to 65535)", H_kv);
  return ATTN_OK;
}

attn_status check_scale(float scale) {
  if (!(isfinite(scale) && scale > 0.f))
    return fail(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0 (got %g)", (double)scale);
  return ATTN_OK;
}

// A stride in elements of a 16-bit tensor whose rows are read 16 bytes at a time.
attn_status check_stride(long long s, const char* name) {
  if (s < 0 || s % 8 != 0 || s >= (1ll << 39))
    return fail(ATTN_ERR_INVALID_ARG, "%s = %lld must be a multiple of 8 elements in [0, 2^39)", name, s);
  return ATTN_OK;
}

// Packed input: B sequences of T tokens together.
attn_status check_packed(int B, int T) {
  if (B < 1 || T < 0) return fail(ATTN_ERR_INVALID_ARG, "B must be >= 1 and T >= 0 (got B=%d T=%d)", B, T);
  // The kernels go over the sequences in strides of up to 1024 in 32 bits.
  if (B > INT_MAX - 1024) return fail(ATTN_ERR_INVALID_ARG, "B = %d is too large", B);
  return ATTN_OK;
}

attn_status check_varlen(int B, int T, int H, int H_kv, int d, VarlenProblem* p) {
  ATTN_CHECK(check_packed(B, T));
  ATTN_CHECK(check_heads(H, H_kv, d));
  const long long tq = kBlockM / (H / H_kv);
  if (((long long)T / tq + B) * H_kv > INT_MAX)
    return fail(ATTN_ERR_INVALID_ARG, "B=%d, T=%d and H_kv=%d make more than 2^31 - 1 work items", B, T, H_kv);
  p->B = B, p->T = T, p->H = H, p->Hkv = H_kv, p->d = d, p->causal = 0, p->scale = 1.f;
  return ATTN_OK;
}

attn_status check_pages(int H_kv, int d, int num_pages, int page_size, int max_blocks) {
  ATTN_CHECK(check_heads(H_kv, H_kv, d));
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return fail(ATTN_ERR_UNSUPPORTED, "page_size = %d is not supported (16, 32, 64 or 128)", page_size);
  if (num_pages < 1 || max_blocks < 1)
    return fail(ATTN_ERR_INVALID_ARG, "num_pages and max_blocks must be >= 1 (got %d and %d)", num_pages, max_blocks);
  if ((long long)num_pages * H_kv > INT_MAX / page_size)
    return fail(ATTN_ERR_UNSUPPORTED, "num_pages * H_kv * page_size exceeds 2^31 - 1 rows");
  if (max_blocks > (INT_MAX - 4096) / page_size)
    return fail(ATTN_ERR_UNSUPPORTED, "max_blocks * page_size exceeds 2^31 positions");
  return ATTN_OK;
}

attn_status check_cache(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                        const int* block_table, int B, int H_kv, int d, int num_pages, int page_size, int max_blocks,
                        PtrCheck& ptr, PagedCache* c) {
  ATTN_CHECK(check_pages(H_kv, d, num_pages, page_size, max_blocks));
  ATTN_CHECK(ptr(k_cache, "k_cache"));
  ATTN_CHECK(ptr(v_cache, "v_cache"));
  ATTN_CHECK(ptr(k_scale, "k_scale", 4));
  ATTN_CHECK(ptr(v_scale, "v_scale", 4));
  ATTN_CHECK(ptr(block_table, "block_table", 4));
  *c = PagedCache{k_cache, v_cache, k_scale, v_scale, block_table, B, H_kv, d, num_pages, page_size, max_blocks};
  return ATTN_OK;
}

attn_status check_decode(int B, int n_q, int H, int H_kv, int d) {
  ATTN_CHECK(check_packed(B, 0));
  ATTN_CHECK(check_heads(H, H_kv, d));
  if (n_q < 1 || n_q > 256)
    return fail(n_q < 1 ? ATTN_ERR_INVALID_ARG : ATTN_ERR_UNSUPPORTED, "n_q = %d is not supported (1 to 256)", n_q);
  if ((long long)B * n_q * H > INT_MAX)
    return fail(ATTN_ERR_INVALID_ARG, "B * n_q * H = %lld exceeds 2^31 - 1", (long long)B * n_q * H);
  return ATTN_OK;
}

attn_status check_shared(int B, int n_q, int H, int H_kv, int d, int page_size, int prefix_blocks, int max_blocks) {
  ATTN_CHECK(check_decode(B, n_q, H, H_kv, d));
  ATTN_CHECK(check_pages(H_kv, d, 1, page_size, max_blocks));
  if ((long long)B * n_q * H > INT_MAX - 1024)
    return fail(ATTN_ERR_UNSUPPORTED, "B * n_q * H = %lld is not supported", (long long)B * n_q * H);
  if (prefix_blocks < 1) return fail(ATTN_ERR_INVALID_ARG, "prefix_blocks must be >= 1 (got %d)", prefix_blocks);
  if (prefix_blocks > (INT_MAX - 4096) / page_size)
    return fail(ATTN_ERR_UNSUPPORTED, "prefix_blocks * page_size exceeds 2^31 positions");
  // Tiles of 256 rows and 128 positions are counted in 32 bits.
  const long long units = (((long long)B * n_q * (H / H_kv) - 1) / 256 + 1) * H_kv;
  if (units * (((long long)prefix_blocks * page_size - 1) / 128 + 1) > INT_MAX - 1024)
    return fail(ATTN_ERR_UNSUPPORTED, "B * n_q * H = %lld rows over %d blocks of prefix are not supported",
                (long long)B * n_q * H, prefix_blocks);
  return ATTN_OK;
}

// An int32 array of one call.
struct Ints {
  const char* name;
  const int* p;
  long long n;
};
// attn_cache_append_int8, with the lengths at which rows end where there are any.
attn_status append(const void* k, const void* v, long long k_token_stride, long long k_head_stride,
                   long long v_token_stride, long long v_head_stride, void* k_cache, void* v_cache, float* k_scale,
                   float* v_scale, const int* block_table, const int* cu_seqlens, const int* starts, const int* lens,
                   bool with_lens, int B, int T, int H_kv, int d, int num_pages, int page_size, int max_blocks,
                   cudaStream_t stream, const char* what) {
  PagedCache c;
  PtrCheck ptr;
  ATTN_CHECK(check_packed(B, T));
  const long long strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  const char* names[4] = {"k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride"};
  for (int i = 0; i < 4; ++i) ATTN_CHECK(check_stride(strides[i], names[i]));
  ATTN_CHECK(check_cache(k_cache, v_cache, k_scale, v_scale, block_table, B, H_kv, d, num_pages, page_size,
                         max_blocks, ptr, &c));
  ATTN_CHECK(ptr(cu_seqlens, "cu_seqlens", 4));
  ATTN_CHECK(ptr(starts, "starts", 4));
  if (with_lens) ATTN_CHECK(ptr(lens, "lens", 4));
  if (T == 0) return launched(cudaSuccess, what);
  ATTN_CHECK(ptr(k, "k"));
  ATTN_CHECK(ptr(v, "v"));
  return launched(launch_cache_append_int8(c, k, v, strides, cu_seqlens, starts, lens, T, stream), what);
}

attn_status check_apart(const Ints& x, const Ints& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  if (a != 0 && b != 0 && x.n > 0 && y.n > 0 && a < b + 4 * (uintptr_t)y.n && b < a + 4 * (uintptr_t)x.n)
    return fail(ATTN_ERR_INVALID_ARG, "%s and %s overlap", x.name, y.name);
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

size_t attn_varlen_plan_bytes(int B, int T, int H, int H_kv) {
  VarlenProblem p;
  if (check_varlen(B, T, H, H_kv, 64, &p) != ATTN_OK) return 0;
  return varlen_plan_bytes(B, T, H, H_kv);
}

attn_status attn_varlen_plan(const int* cu_seqlens, int B, int T, int H, int H_kv, int causal, void* plan,
                             size_t plan_bytes, cudaStream_t stream) {
  VarlenProblem p;
  PtrCheck ptr;
  ATTN_CHECK(check_varlen(B, T, H, H_kv, 64, &p));
  p.causal = causal != 0;
  if (plan_bytes < varlen_plan_bytes(B, T, H, H_kv))
    return fail(ATTN_ERR_INVALID_ARG, "plan has %zu bytes, %zu needed", plan_bytes, varlen_plan_bytes(B, T, H, H_kv));
  ATTN_CHECK(ptr(cu_seqlens, "cu_seqlens", 4));
  ATTN_CHECK(ptr(plan, "plan"));
  return launched(launch_varlen_plan(p, cu_seqlens, plan, stream), "attn_varlen_plan");
}

attn_status attn_varlen_fwd(const void* q, const void* k, const void* v, long long q_token_stride,
                            long long q_head_stride, long long k_token_stride, long long k_head_stride,
                            long long v_token_stride, long long v_head_stride, const void* plan, size_t plan_bytes,
                            void* o, float* lse, int B, int T, int H, int H_kv, int d, float scale, int causal,
                            cudaStream_t stream) {
  VarlenProblem p;
  PtrCheck ptr;
  ATTN_CHECK(check_varlen(B, T, H, H_kv, d, &p));
  ATTN_CHECK(check_scale(scale));
  p.causal = causal != 0;
  p.scale = scale;
  const long long strides[6] = {q_token_stride, q_head_stride, k_token_stride,
                                k_head_stride,  v_token_stride, v_head_stride};
  const char* names[6] = {"q_token_stride", "q_head_stride", "k_token_stride",
                          "k_head_stride",  "v_token_stride", "v_head_stride"};
  for (int i = 0; i < 6; ++i) ATTN_CHECK(check_stride(strides[i], names[i]));
  if (plan_bytes < varlen_plan_bytes(B, T, H, H_kv))
    return fail(ATTN_ERR_INVALID_ARG, "plan has %zu bytes, %zu needed", plan_bytes, varlen_plan_bytes(B, T, H, H_kv));
  if (T == 0) return launched(cudaSuccess, "attn_varlen_fwd");
  ATTN_CHECK(ptr(q, "q"));
  ATTN_CHECK(ptr(k, "k"));
  ATTN_CHECK(ptr(v, "v"));
  ATTN_CHECK(ptr(plan, "plan"));
  ATTN_CHECK(ptr(o, "o"));
  ATTN_CHECK(ptr(lse, "lse", 4));
  if (encode_tiled_fn() == nullptr)
    return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  return launched(launch_varlen_fwd(p, q, k, v, plan, o, lse, strides, stream), "attn_varlen_fwd");
}

attn_status attn_cache_append_int8(const void* k, const void* v, long long k_token_stride, long long k_head_stride,
                                   long long v_token_stride, long long v_head_stride, void* k_cache, void* v_cache,
                                   float* k_scale, float* v_scale, const int* block_table, const int* cu_seqlens,
                                   const int* starts, int B, int T, int H_kv, int d, int num_pages, int page_size,
                                   int max_blocks, cudaStream_t stream) {
  return append(k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, k_cache, v_cache, k_scale, v_scale,
                block_table, cu_seqlens, starts, nullptr, false, B, T, H_kv, d, num_pages, page_size, max_blocks, stream,
                "attn_cache_append_int8");
}

attn_status attn_cache_append_served_int8(const void* k, const void* v, long long k_token_stride,
                                          long long k_head_stride, long long v_token_stride, long long v_head_stride,
                                          void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                          const int* block_table, const int* cu_seqlens, const int* starts,
                                          const int* lens, int B, int T, int H_kv, int d, int num_pages, int page_size,
                                          int max_blocks, cudaStream_t stream) {
  return append(k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, k_cache, v_cache, k_scale, v_scale,
                block_table, cu_seqlens, starts, lens, true, B, T, H_kv, d, num_pages, page_size, max_blocks, stream,
                "attn_cache_append_served_int8");
}

attn_status attn_cache_read_int8(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                                 const int* block_table, const int* cu_seqlens, const int* starts, void* k, void* v,
                                 int B, int T, int H_kv, int d, int num_pages, int page_size, int max_blocks,
                                 attn_dtype dt, cudaStream_t stream) {
  PagedCache c;
  PtrCheck ptr;
  if (dt != ATTN_DTYPE_BF16 && dt != ATTN_DTYPE_FP32)
    return fail(ATTN_ERR_INVALID_ARG, "dt must be ATTN_DTYPE_BF16 or ATTN_DTYPE_FP32 (got %d)", (int)dt);
  ATTN_CHECK(check_packed(B, T));
  ATTN_CHECK(check_cache(k_cache, v_cache, k_scale, v_scale, block_table, B, H_kv, d, num_pages, page_size,
                         max_blocks, ptr, &c));
  if ((long long)H_kv * d * 16 > INT_MAX) return fail(ATTN_ERR_UNSUPPORTED, "H_kv * d is too large");
  ATTN_CHECK(ptr(cu_seqlens, "cu_seqlens", 4));
  ATTN_CHECK(ptr(starts, "starts", 4));
  if (T == 0) return launched(cudaSuccess, "attn_cache_read_int8");
  ATTN_CHECK(ptr(k, "k"));
  ATTN_CHECK(ptr(v, "v"));
  return launched(launch_cache_read_int8(c, cu_seqlens, starts, k, v, T, dt == ATTN_DTYPE_FP32, stream),
                  "attn_cache_read_int8");
}

size_t attn_decode_int8_workspace_bytes(int B, int n_q, int H, int H_kv, int d, int page_size, int max_blocks) {
  if (check_decode(B, n_q, H, H_kv, d) != ATTN_OK || check_pages(H_kv, d, 1, page_size, max_blocks) != ATTN_OK) return 0;
  PagedCache c = {nullptr, nullptr, nullptr, nullptr, nullptr, B, H_kv, d, 1, page_size, max_blocks};
  return decode_workspace_bytes(c, n_q, H);
}

attn_status attn_decode_int8(const void* q, long long q_batch_stride, long long q_token_stride,
                             long long q_head_stride, const void* k_cache, const void* v_cache, const float* k_scale,
                             const float* v_scale, const int* block_table, const int* seqlens, void* o, float* lse,
                             int B, int n_q, int H, int H_kv, int d, int num_pages, int page_size, int max_blocks,
                             float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  PagedCache c;
  PtrCheck ptr;
  ATTN_CHECK(check_decode(B, n_q, H, H_kv, d));
  ATTN_CHECK(check_scale(scale));
  ATTN_CHECK(check_stride(q_batch_stride, "q_batch_stride"));
  ATTN_CHECK(check_stride(q_token_stride, "q_token_stride"));
  ATTN_CHECK(check_stride(q_head_stride, "q_head_stride"));
  ATTN_CHECK(check_cache(k_cache, v_cache, k_scale, v_scale, block_table, B, H_kv, d, num_pages, page_size,
                         max_blocks, ptr, &c));
  ATTN_CHECK(ptr(q, "q"));
  ATTN_CHECK(ptr(seqlens, "seqlens", 4));
  ATTN_CHECK(ptr(o, "o"));
  ATTN_CHECK(ptr(lse, "lse", 4));
  const size_t need = decode_workspace_bytes(c, n_q, H);
  if (need > 0) {
    if (workspace_bytes < need)
      return fail(ATTN_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    ATTN_CHECK(ptr(workspace, "workspace", 256));
  }
  if (encode_tiled_fn() == nullptr)
    return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  const long long strides[3] = {q_batch_stride, q_token_stride, q_head_stride};
  return launched(launch_decode_int8(c, q, strides, seqlens, o, lse, n_q, H, scale, workspace, stream),
                  "attn_decode_int8");
}

size_t attn_decode_shared_int8_workspace_bytes(int B, int n_q, int H, int H_kv, int d, int page_size,
                                               int prefix_blocks, int max_blocks) {
  if (check_shared(B, n_q, H, H_kv, d, page_size, prefix_blocks, max_blocks) != ATTN_OK) return 0;
  PagedCache c = {nullptr, nullptr, nullptr, nullptr, nullptr, B, H_kv, d, 1, page_size, max_blocks};
  return decode_shared_workspace_bytes(c, n_q, H, prefix_blocks);
}

attn_status attn_decode_shared_int8(const void* q, long long q_batch_stride, long long q_token_stride,
                                    long long q_head_stride, const void* k_cache, const void* v_cache,
                                    const float* k_scale, const float* v_scale, const int* prefix_table,
                                    int prefix_blocks, const int* prefix_len, const int* block_table,
                                    const int* seqlens, void* o, float* lse, int B, int n_q, int H, int H_kv, int d,
                                    int num_pages, int page_size, int max_blocks, float scale, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  PagedCache c;
  PtrCheck ptr;
  ATTN_CHECK(check_shared(B, n_q, H, H_kv, d, page_size, prefix_blocks, max_blocks));
  ATTN_CHECK(check_scale(scale));
  ATTN_CHECK(check_stride(q_batch_stride, "q_batch_stride"));
  ATTN_CHECK(check_stride(q_token_stride, "q_token_stride"));
  ATTN_CHECK(check_stride(q_head_stride, "q_head_stride"));
  ATTN_CHECK(check_cache(k_cache, v_cache, k_scale, v_scale, block_table, B, H_kv, d, num_pages, page_size,
                         max_blocks, ptr, &c));
  ATTN_CHECK(ptr(q, "q"));
  ATTN_CHECK(ptr(prefix_table, "prefix_table", 4));
  ATTN_CHECK(ptr(prefix_len, "prefix_len", 4));
  ATTN_CHECK(ptr(seqlens, "seqlens", 4));
  ATTN_CHECK(ptr(o, "o"));
  ATTN_CHECK(ptr(lse, "lse", 4));
  const size_t need = decode_shared_workspace_bytes(c, n_q, H, prefix_blocks);
  if (need > 0) {
    if (workspace_bytes < need)
      return fail(ATTN_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    ATTN_CHECK(ptr(workspace, "workspace", 256));
  }
  if (encode_tiled_fn() == nullptr)
    return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  const long long strides[3] = {q_batch_stride, q_token_stride, q_head_stride};
  return launched(launch_decode_shared_int8(c, q, strides, prefix_table, prefix_blocks, prefix_len, seqlens, o, lse,
                                            n_q, H, scale, workspace, stream),
                  "attn_decode_shared_int8");
}

attn_status attn_cache_reserve(int* block_table, const int* held, const int* wanted, int* free_pages, int* n_free,
                               int* lens, int* cu_seqlens, int* slots, int* positions, int B, int T, int num_pages,
                               int page_size, int max_blocks, cudaStream_t stream) {
  PtrCheck ptr;
  ATTN_CHECK(check_packed(B, T));
  ATTN_CHECK(check_pages(1, 64, num_pages, page_size, max_blocks));
  if (T > INT_MAX - 4096) return fail(ATTN_ERR_INVALID_ARG, "T = %d is too large", T);
  const Ints ins[5] = {{"block_table", block_table, (long long)B * max_blocks}, {"free_pages", free_pages, num_pages},
                       {"n_free", n_free, 1},                                   {"held", held, B},
                       {"wanted", wanted, B}};
  const Ints outs[4] = {{"lens", lens, B}, {"cu_seqlens", cu_seqlens, B + 1ll}, {"slots", slots, T},
                        {"positions", positions, T}};
  // Every array that is written is apart from all others.
  for (int i = 0; i < 4; ++i) {
    for (const Ints& y : ins) ATTN_CHECK(check_apart(outs[i], y));
    for (int j = 0; j < i; ++j) ATTN_CHECK(check_apart(outs[i], outs[j]));
  }
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 5; ++j) ATTN_CHECK(check_apart(ins[i], ins[j]));
  for (const Ints& x : ins) ATTN_CHECK(ptr(x.p, x.name, 4));
  for (const Ints& x : outs)
    if (x.n > 0) ATTN_CHECK(ptr(x.p, x.name, 4));
  const Tables t = {block_table, held,       wanted, free_pages, n_free,    lens,
                    cu_seqlens,  slots,      positions, B,       T,         num_pages,
                    page_shift(page_size), max_blocks};
  return launched(launch_cache_reserve(t, stream), "attn_cache_reserve");
}

}  // extern "C"

// Internal launch interface shared by the C-ABI layer and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "attn.h"

namespace attn {

// Problem description after validation.  Tensors are [B, H, N, d],
// contiguous, d fastest; LSE is [B, H, N].
struct Problem {
  int B, H, N, d;
  float scale;
  int causal;
};

// Tile geometry of the BF16 tensor-core path.
constexpr int kBlockM = 128;  // query rows per tile (one TMEM lane per row)
constexpr int kBlockN = 128;  // key rows per tile

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
inline int n_pad(int N) { return ceil_div(N, kBlockN) * kBlockN; }

// Launch with programmatic stream serialization: the kernel may be scheduled
// before the previous kernel in the stream has completed (its set-up then
// overlaps that kernel's tail), so it must call griddep_wait() before its
// first global-memory access, in every thread that makes one.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// The same in clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                      cudaStream_t stream, unsigned cluster, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {cluster, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Allows `kernel` so much dynamic shared memory, once per device (`done`: a bit for each
// of the first 64): asking the runtime takes 0.2 us, a tenth of a small call.
template <typename... KArgs>
inline cudaError_t allow_smem(void (*kernel)(KArgs...), int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (err != cudaSuccess || (done.load(std::memory_order_relaxed) & bit)) return err;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

// Backward workspace layout (all offsets 256-byte aligned):
//   neg_lse2 FP32 [B*H][Npad] -(LSE * log2(e)); -inf for padded rows
//   delta FP32 [B*H][Npad]    rowsum(dO o O); 0 for padded rows
//   dqacc FP32 [B*H][Npad][d] unscaled dQ accumulator
struct BwdWorkspace {
  float* neg_lse2;
  float* delta;
  float* dqacc;
};
size_t bwd_workspace_bytes(const Problem& p);
BwdWorkspace bwd_workspace_carve(void* base, const Problem& p);

// Kernel launchers.  Return cudaSuccess or the launch error.
// beta > 0 selects the stabilised normaliser (beta * repeated row max).
cudaError_t launch_fwd_bf16(const Problem& p, const void* q, const void* k, const void* v, void* o,
                            float* lse, cudaStream_t stream, float beta = 0.f);
cudaError_t launch_bwd_preprocess_bf16(const Problem& p, const void* o, const void* dout,
                                       const float* lse, const BwdWorkspace& ws,
                                       cudaStream_t stream);
cudaError_t launch_bwd_main_bf16(const Problem& p, const void* q, const void* k, const void* v,
                                 const void* dout, void* dk, void* dv, const BwdWorkspace& ws,
                                 cudaStream_t stream);
cudaError_t launch_bwd_dq_convert_bf16(const Problem& p, const BwdWorkspace& ws, void* dq,
                                       cudaStream_t stream);

cudaError_t launch_fwd_fp32(const Problem& p, const float* q, const float* k, const float* v,
                            float* o, float* lse, cudaStream_t stream);
cudaError_t launch_bwd_fp32(const Problem& p, const float* q, const float* k, const float* v,
                            const float* o, const float* lse, const float* dout, float* dq,
                            float* dk, float* dv, const BwdWorkspace& ws, cudaStream_t stream);

cudaError_t launch_wait_selftest(unsigned long long limit_ns, cudaStream_t stream);

// INT8-input forward: per-token quantization of a BF16 [B,H,N,d] tensor, and
// the forward on INT8 Q, K (with their per-row scales) and BF16 V.
cudaError_t launch_quantize_int8(const Problem& p, const void* x, void* codes, float* scales,
                                 cudaStream_t stream);
cudaError_t launch_fwd_int8(const Problem& p, const void* q8, const float* qs, const void* k8,
                            const float* ks, const void* v, void* o, float* lse,
                            cudaStream_t stream);
// The same on INT8 codes held in BF16, with scales in the padded per-head
// layout [B*H][n_pad(N)], on the tcgen05 forward kernel.
cudaError_t launch_quantize_int8_as_bf16(const Problem& p, const void* x, void* codes,
                                         float* scales, cudaStream_t stream);
cudaError_t launch_fwd_int8_as_bf16(const Problem& p, const void* qc, const float* qs,
                                    const void* kc, const float* ks, const void* v, void* o,
                                    float* lse, cudaStream_t stream);

// Paged INT8 cache: codes [P, Hkv, page, d], one FP32 scale per page and head
// [P, Hkv], and the pages of B sequences [B, max_blocks].
struct PagedCache {
  const void *k, *v;
  const float *k_scale, *v_scale;
  const int* table;
  int B, Hkv, d, P, page, max_blocks;
};
// Base-2 logarithm of a page size (16, 32, 64 or 128).
inline int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// strides: token and head stride of the K rows, then of the V rows (elements).
cudaError_t launch_cache_append_int8(const PagedCache& c, const void* k, const void* v,
                                     const long long* strides, const int* cu, const int* starts,
                                     int T, cudaStream_t stream);
cudaError_t launch_cache_read_int8(const PagedCache& c, const int* cu, const int* starts, void* k,
                                   void* v, int T, bool fp32, cudaStream_t stream);
// strides: batch, token and head stride of q (elements).
size_t decode_workspace_bytes(const PagedCache& c, int n_q, int H);
cudaError_t launch_decode_int8(const PagedCache& c, const void* q, const long long* strides,
                               const int* lens, void* o, float* lse, int n_q, int H, float scale,
                               void* workspace, cudaStream_t stream);

// Attention over packed sequences (csrc/fwd_varlen.cu).
struct VarlenProblem {
  int B, T, H, Hkv, d, causal;
  float scale;
};
size_t varlen_plan_bytes(int B, int T, int H, int Hkv);
cudaError_t launch_varlen_plan(const VarlenProblem& p, const int* cu, void* plan, cudaStream_t stream);
// strides: token and head stride of q, k, v and o (elements).
cudaError_t launch_varlen_fwd(const VarlenProblem& p, const void* q, const void* k, const void* v,
                              const void* plan, void* o, float* lse, const long long* strides,
                              cudaStream_t stream);

// Addresses of the device status words (one per kernel translation unit) on the current device.
cudaError_t status_word_fwd(void** word);
cudaError_t status_word_bwd(void** word);
cudaError_t status_word_misc(void** word);
cudaError_t status_word_varlen(void** word);
cudaError_t status_word_cache(void** word);
cudaError_t status_word_decode(void** word);

// Shape and scalar checks shared by every entry point (d, N, B*H*N*d, dtype,
// and the scale when need_scale); fills *out and records the error detail.
attn_status check_problem(int B, int H, int N, int d, attn_dtype dt, float scale, bool need_scale,
                          Problem* out);

// Helpers of the entry points.  fail() records the detail text and returns its
// status; check_ptr() refuses a pointer that is NULL, not `align`-byte aligned or
// not device memory of the current device; launched() maps a launch's result.
attn_status fail(attn_status s, const char* fmt, ...);
attn_status check_ptr(const void* p, const char* name, unsigned align = 16);
attn_status launched(cudaError_t err, const char* what);

// check_ptr() for the pointers of one call: those that lie in an allocation that an
// earlier one of the call was found in need no query (10 pointers took 0.7 us of a call's
// host time, 0.2 us if they share an allocation).
class PtrCheck {
 public:
  attn_status operator()(const void* p, const char* name, unsigned align = 16);

 private:
  uintptr_t begin_ = 0, end_ = 0;
  int device_ = -1;
};
size_t align256(size_t x);

#define ATTN_CHECK(expr)          \
  do {                            \
    attn_status _s = (expr);      \
    if (_s != ATTN_OK) return _s; \
  } while (0)

// Record the detail text returned by attn_last_error() on this thread.
void set_last_error(const char* msg);

// Number of SMs of the current device (cached per device); 0 if the query fails.
int device_sm_count();

// Driver entry point for cuTensorMapEncodeTiled (resolved once, no -lcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled_fn();

// 3-D BF16 tensor map over a [B*H, N, d] tensor with a (64 x box_rows x 1) box
// and 128-byte swizzle.  Returns false when the driver rejects it.
bool make_tmap_bhnd(CUtensorMap* map, const void* base, int BH, int N, int d, int box_rows = 128);

}  // namespace attn

// Paged INT8 cache of keys and values: writing new rows into the pages of
// their sequences, and reading ranges of positions back as values.
//
// A cache holds, for keys and for values, codes int8 [P][Hkv][page][d] and one
// FP32 scale per page and head; code c stands for c * scale.  A sequence's
// position t lies in row t % page of page block_table[b][t / page].
//
// Append.  For every page that new rows of a sequence fall into and every
// head, with a = max|x| over the new rows' finite elements:
//   page begun by these rows:  s = a / 127 (FP32)
//   page begun earlier:        s = max(s_old, a / 127); where s > s_old the rows
//                              it holds become rint(c s_old / s)
//   new rows:                  rint(x / s)
// clamped to +-127, with rint half to even on the exact quotient.  Exactness
// matters: x = a / 2 lies next to the border between 63 and 64 for every a, and
// there an FP32 quotient's own rounding would decide the code.
//
// One CTA per (page, head, K or V), found from the sequences' lengths by a
// scan over the batch; the new rows stay in registers between the maximum and
// the codes, so every byte moves once.
#include <math.h>
#include <stdint.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {

static __device__ unsigned int g_status_cache;

namespace {

constexpr int kAppendThreads = 128;

__device__ __forceinline__ void set_fail(unsigned int code) { atomicOr(&g_status_cache, code); }

// rint(x / s) of the exact quotient (x = xh + xl, |xl| below xh's last bit;
// s > 0), half to even.  k starts as the rounded approximate quotient, which
// is off by at most one next to a border; the remainder x - k s is exact there
// (it is below s and a multiple of the operands' last bits), and its double
// against s decides.
__device__ __forceinline__ float rint_quotient(float xh, float xl, float s) {
  float k = rintf(fminf(fmaxf(xh / s, -128.f), 128.f));
  const float e = fmaf(-k, s, xh) + xl;
  const float e2 = 2.f * fabsf(e);
  if (e2 > s || (e2 == s && (static_cast<int>(k) & 1))) k += copysignf(1.f, e);
  return k;
}

__device__ __forceinline__ int code_of(float xh, float xl, float s) {
  // NaN becomes 0, an infinity +-127.
  if (!(s > 0.f) || isnan(xh)) return 0;
  if (isinf(xh)) return xh > 0.f ? 127 : -127;
  return static_cast<int>(fminf(fmaxf(rint_quotient(xh, xl, s), -127.f), 127.f));
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Sequence b's new rows: `first` is its first row of the packed input, n their
// number (clamped to the rows there are, whatever cu_seqlens holds).
__device__ __forceinline__ void new_rows(const int* cu, int b, int T, int& first, int& n) {
  first = min(max(__ldcg(cu + b), 0), T);
  n = min(max(__ldcg(cu + b + 1), first), T) - first;
}

struct AppendArgs {
  const uint16_t* x[2];            // K, V rows (BF16)
  long long token_stride[2], head_stride[2];
  int8_t* codes[2];
  float* scales[2];
  const int *table, *cu, *starts;
  int B, T, Hkv, P, page, page_shift, max_blocks;
};

// D head dims; kUnits: 16-byte units of new rows a thread holds at most
// (page * D / 8 units over 128 threads).
template <int D, int kUnits>
__global__ void __launch_bounds__(kAppendThreads) append_int8_kernel(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ int s_warp[kAppendThreads / 32];
  __shared__ int s_found[4];  // sequence, page number in it, first row, rows
  __shared__ float s_max[kAppendThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x, head = blockIdx.y, kv = blockIdx.z;

  // Which page of which sequence is number `item` of the touched ones?
  if (tid == 0) s_found[0] = -1;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kAppendThreads) {
    const int b = b0 + tid;
    int first = 0, n = 0, start = 0, count = 0;
    if (b < a.B) {
      new_rows(a.cu, b, a.T, first, n);
      start = max(__ldcg(a.starts + b), 0);
      if (n > 0) count = ((n - 1 + (start & (a.page - 1))) >> a.page_shift) + 1;
    }
    int upto = count;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int chunk = 0;
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) {
      if (w < warp) upto += s_warp[w];
      chunk += s_warp[w];
    }
    const int at = item - before - (upto - count);
    if (at >= 0 && at < count) {
      s_found[0] = b;
      s_found[1] = at;
      s_found[2] = first;
      s_found[3] = n;
    }
    before += chunk;
    if (before > item) break;
  }
  __syncthreads();
  const int b = s_found[0];
  if (b < 0) return;  // fewer pages are touched than the launch allows for
  const int start = max(__ldcg(a.starts + b), 0);
  const long long blk = (long long)(start >> a.page_shift) + s_found[1];
  const int page_id = blk < a.max_blocks ? __ldcg(a.table + (size_t)b * a.max_blocks + blk) : -1;
  if (page_id < 0 || page_id >= a.P) {
    if (tid == 0) set_fail(ATTN_ERR_INVALID_ARG);
    return;
  }
  // Rows [r0, r1) of the page take the packed rows from `row0` on.
  const int r0 = s_found[1] == 0 ? (start & (a.page - 1)) : 0;
  const int done = s_found[1] == 0 ? 0 : s_found[1] * a.page - (start & (a.page - 1));
  const int r1 = min(a.page, r0 + s_found[3] - done);
  const long long row0 = (long long)s_found[2] + done;
  const uint16_t* x = a.x[kv] + row0 * a.token_stride[kv] + head * a.head_stride[kv];
  const size_t slot = (size_t)page_id * a.Hkv + head;
  int8_t* codes = a.codes[kv] + slot * a.page * D;
  float* scale = a.scales[kv] + slot;

  constexpr int kPerRow = D / 8;
  const int units = (r1 - r0) * kPerRow;
  uint4 w[kUnits];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = tid + i * kAppendThreads;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (u < units)
      w[i] = __ldcg(reinterpret_cast<const uint4*>(x + (u / kPerRow) * a.token_stride[kv] + (u % kPerRow) * 8));
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = fabsf(bf16_lo(v[e])), hi = fabsf(bf16_hi(v[e]));
      if (lo < INFINITY) m = fmaxf(m, lo);
      if (hi < INFINITY) m = fmaxf(m, hi);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) s_max[warp] = m;
  const float s_old = r0 > 0 ? __ldcg(scale) : 0.f;
  __syncthreads();  // the maxima, and everyone has read the old scale
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) m = fmaxf(m, s_max[i]);
  const float s = fmaxf(s_old, m / 127.f);
  if (tid == 0) *scale = s;

  if (s > s_old) {
    // Rows the page holds already, on the coarser scale.
    for (int u = tid; u < r0 * (D / 4); u += kAppendThreads) {
      uint32_t* p = reinterpret_cast<uint32_t*>(codes) + u;
      const uint32_t c4 = __ldcg(p);
      uint32_t out = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = static_cast<float>(static_cast<int8_t>(c4 >> (8 * e)));
        const float hi = c * s_old;
        out |= (static_cast<uint32_t>(code_of(hi, fmaf(c, s_old, -hi), s)) & 255u) << (8 * e);
      }
      *p = out;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = tid + i * kAppendThreads;
    if (u >= units) continue;
    const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = (e & 1) ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]);
      out[e >> 2] |= (static_cast<uint32_t>(code_of(f, 0.f, s)) & 255u) << (8 * (e & 3));
    }
    *reinterpret_cast<uint2*>(codes + (size_t)r0 * D + (size_t)u * 8) = make_uint2(out[0], out[1]);
  }
}

// ------------------------------------------------------------------- read
struct ReadArgs {
  const int8_t* codes[2];
  const float* scales[2];
  void* out[2];
  const int *table, *cu, *starts;
  int B, T, Hkv, P, page, page_shift, max_blocks;
};

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 16;  // packed tokens per CTA

// A CTA reads kReadTokens packed tokens' rows of every head, 16 codes at a
// time.  Positions without a valid page read as zeros.
template <int D, bool FP32>
__global__ void __launch_bounds__(kReadThreads) read_int8_kernel(const ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ long long s_row[kReadTokens];  // page * Hkv * page_size + row in page, or -1
  const int tid = threadIdx.x, kv = blockIdx.y;
  const int t0 = blockIdx.x * kReadTokens;
  if (tid < kReadTokens && t0 + tid < a.T) {
    const int t = t0 + tid;
    int lo = 0, hi = a.B;  // the last sequence that begins at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(a.cu + mid) <= t) lo = mid; else hi = mid;
    }
    long long row = -1;
    const int first = __ldcg(a.cu + lo);
    if (t >= first && t < __ldcg(a.cu + lo + 1)) {
      const long long pos = (long long)max(__ldcg(a.starts + lo), 0) + (t - first);
      const long long blk = pos >> a.page_shift;
      const int id = blk < a.max_blocks ? __ldcg(a.table + (size_t)lo * a.max_blocks + blk) : -1;
      if (id >= 0 && id < a.P)
        row = ((long long)id * a.Hkv << a.page_shift) + (pos & (a.page - 1));
      else
        set_fail(ATTN_ERR_INVALID_ARG);
    } else {
      set_fail(ATTN_ERR_INVALID_ARG);
    }
    s_row[tid] = row;
  }
  __syncthreads();
  constexpr int kPerRow = D / 16;
  const int per_token = a.Hkv * kPerRow;
  const int n = min(kReadTokens, a.T - t0) * per_token;
  for (int u = tid; u < n; u += kReadThreads) {
    const int t = u / per_token, rest = u - t * per_token;
    const int head = rest / kPerRow, col = rest % kPerRow;
    uint4 c4 = make_uint4(0u, 0u, 0u, 0u);
    float s = 0.f;
    if (s_row[t] >= 0) {
      const long long row = s_row[t] + ((long long)head << a.page_shift);
      c4 = __ldcg(reinterpret_cast<const uint4*>(a.codes[kv] + row * D + col * 16));
      s = __ldcg(a.scales[kv] + (row >> a.page_shift));
    }
    const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      f[e] = static_cast<float>(static_cast<int8_t>(c[e >> 2] >> (8 * (e & 3)))) * s;
    const size_t o = ((size_t)(t0 + t) * a.Hkv + head) * D + col * 16;
    if (FP32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out[kv]) + o);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
    } else {
      uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[kv]) + o);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        p[e] = make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]), pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                          pack_bf16x2(f[8 * e + 4], f[8 * e + 5]), pack_bf16x2(f[8 * e + 6], f[8 * e + 7]));
    }
  }
}

}  // namespace

cudaError_t launch_cache_append_int8(const PagedCache& c, const void* k, const void* v,
                                     const long long* strides, const int* cu, const int* starts,
                                     int T, cudaStream_t stream) {
  AppendArgs a;
  a.x[0] = static_cast<const uint16_t*>(k);
  a.x[1] = static_cast<const uint16_t*>(v);
  for (int i = 0; i < 2; ++i) {
    a.token_stride[i] = strides[2 * i];
    a.head_stride[i] = strides[2 * i + 1];
    a.codes[i] = static_cast<int8_t*>(const_cast<void*>(i ? c.v : c.k));
    a.scales[i] = const_cast<float*>(i ? c.v_scale : c.k_scale);
  }
  a.table = c.table;
  a.cu = cu;
  a.starts = starts;
  a.B = c.B, a.T = T, a.Hkv = c.Hkv, a.P = c.P, a.page = c.page, a.max_blocks = c.max_blocks;
  a.page_shift = page_shift(c.page);
  // A token touches one page at most, a sequence of n tokens (n - 1) / page + 2.
  const long long pages = (long long)T / c.page + 2ll * c.B;
  const dim3 grid((unsigned)(pages < T ? pages : T), c.Hkv, 2);
  const int units = ceil_div(c.page * c.d / 8, kAppendThreads);
#define ATTN_APPEND_CASE(DD, UU) \
  if (c.d == DD && units == UU)  \
    return launch_pdl(append_int8_kernel<DD, UU>, grid, dim3(kAppendThreads), 0, stream, a);
  ATTN_APPEND_CASE(64, 1)
  ATTN_APPEND_CASE(64, 2)
  ATTN_APPEND_CASE(64, 4)
  ATTN_APPEND_CASE(64, 8)
  ATTN_APPEND_CASE(128, 2)
  ATTN_APPEND_CASE(128, 4)
  ATTN_APPEND_CASE(128, 8)
  ATTN_APPEND_CASE(128, 16)
#undef ATTN_APPEND_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache_read_int8(const PagedCache& c, const int* cu, const int* starts, void* k,
                                   void* v, int T, bool fp32, cudaStream_t stream) {
  ReadArgs a;
  a.codes[0] = static_cast<const int8_t*>(c.k);
  a.codes[1] = static_cast<const int8_t*>(c.v);
  a.scales[0] = c.k_scale;
  a.scales[1] = c.v_scale;
  a.out[0] = k;
  a.out[1] = v;
  a.table = c.table;
  a.cu = cu;
  a.starts = starts;
  a.B = c.B, a.T = T, a.Hkv = c.Hkv, a.P = c.P, a.page = c.page, a.max_blocks = c.max_blocks;
  a.page_shift = page_shift(c.page);
  const dim3 grid(ceil_div(T, kReadTokens), 2);
  if (c.d == 128)
    return fp32 ? launch_pdl(read_int8_kernel<128, true>, grid, dim3(kReadThreads), 0, stream, a)
                : launch_pdl(read_int8_kernel<128, false>, grid, dim3(kReadThreads), 0, stream, a);
  return fp32 ? launch_pdl(read_int8_kernel<64, true>, grid, dim3(kReadThreads), 0, stream, a)
              : launch_pdl(read_int8_kernel<64, false>, grid, dim3(kReadThreads), 0, stream, a);
}

cudaError_t read_and_clear_status_cache(unsigned int* out, cudaStream_t stream) {
  static const unsigned int zero = 0;
  cudaError_t err = cudaMemcpyFromSymbolAsync(out, g_status_cache, sizeof(unsigned int), 0,
                                              cudaMemcpyDeviceToHost, stream);
  if (err != cudaSuccess) return err;
  err = cudaStreamSynchronize(stream);
  if (err != cudaSuccess) return err;
  err = cudaMemcpyToSymbolAsync(g_status_cache, &zero, sizeof(unsigned int), 0,
                                cudaMemcpyHostToDevice, stream);
  if (err != cudaSuccess) return err;
  return cudaStreamSynchronize(stream);
}

}  // namespace attn

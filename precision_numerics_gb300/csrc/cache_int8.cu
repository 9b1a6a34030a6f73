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
// Both directions move a byte or two per element and do little with it, so HBM
// bounds them for long inputs and the chain of dependent loads (lengths, page
// number, rows) for a decoding step.  For prompts one CTA takes a (page, head, K
// or V) and keeps the new rows in registers between the maximum and the codes, so
// every byte moves once; for a step's few rows a page a CTA takes a page of K or
// V and its warps the heads, so that the search for the page is done once.
// Measured (8 heads of 128, pages of 64): 16 prompts of 150 to 4096 tokens appended
// and read back as FP32 in 41.8 us, 23.5 of them the reading (5.7 TB/s); one token of each of 96
// sequences in 4.5 us.  Both while no begun page's scale grows.  Where scales grow the rows that
// are held are read and written again: the same prompts take 7 us more, the step 44 to 51 us
// (by up to page * d bytes a warp, 16 bytes a lane at a time, one after the other).  Which a
// decoding step meets depends on its values: a scale grows when a new row exceeds all before
// it in its page and head.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {

static __device__ unsigned int g_status_cache;

namespace {

// Up to so many rows a sequence are a step.  On average: one prompt of up to 8 B rows among
// B - 1 sequences with none takes a warp a page and head as well.
constexpr int kStepRows = 8;

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

__device__ __noinline__ int code_of(float xh, float xl, float s) {
  // NaN becomes 0, an infinity +-127.
  if (!(s > 0.f) || isnan(xh)) return 0;
  if (isinf(xh)) return xh > 0.f ? 127 : -127;
  return static_cast<int>(fminf(fmaxf(rint_quotient(xh, xl, s), -127.f), 127.f));
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Largest of |a|, |b|, |c|; NaN where one is.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A scale and what its codes need: 1 / s, and the bound on |x - k s| below which
// the rounded x * (1 / s) is the code (0 where the scale is too small or large
// for that: every code then goes through code_of).
struct Quantizer {
  float s, inv, near;
  __device__ __forceinline__ explicit Quantizer(float scale) : s(scale) {
    const bool usual = s > 0x1p-100f && s < 0x1p100f;
    inv = usual ? 1.f / s : 0.f;
    near = usual ? s * 0.4999f : 0.f;
  }
  // Codes of 8 BF16 values.  x (1 / s) is off by less than 2^-22 of at most 127, so
  // k = rint of it (adding 1.5 * 2^23 rounds, half to even, and leaves k in the
  // sum's low byte) is the code unless x lies within 1e-4 s of a border between
  // two, where |x - k s|, which is exact, is not below 0.4999 s.  Then its double
  // against s decides, as in rint_quotient; what is no finite multiple of the scale
  // at all is done one by one.
  __device__ __forceinline__ uint2 codes(const uint4& w) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t q[8];
    float far = 0.f;  // NaN as well: an infinity's rest
    const uint64_t inv2 = f2_pack(inv, inv), up2 = f2_pack(12582912.f, 12582912.f),
                   down2 = f2_pack(-12582912.f, -12582912.f), minus_s2 = f2_pack(-s, -s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t x = f2_pack(bf16_lo(v[e]), bf16_hi(v[e]));
      const uint64_t y = fma2(x, inv2, up2);
      float r0, r1, y0, y1;
      f2_unpack(fma2(add2(y, down2), minus_s2, x), r0, r1);
      f2_unpack(y, y0, y1);
      far = max3_abs_nan(far, r0, r1);
      q[2 * e] = __float_as_uint(y0);
      q[2 * e + 1] = __float_as_uint(y1);
    }
    if (!(far < near)) {
      bool plain = near > 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = (e & 1) ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]);
        const float rest = fmaf(-(__uint_as_float(q[e]) - 12582912.f), s, x);
        const float twice = 2.f * fabsf(rest);
        plain = plain && twice < 1.001f * s;
        if (twice > s || (twice == s && (q[e] & 1u))) q[e] += rest > 0.f ? 1u : ~0u;
      }
      if (!plain) {
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          const uint32_t u = e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w;
          const uint32_t lo = code_of(bf16_lo(u), 0.f, s), hi = code_of(bf16_hi(u), 0.f, s);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i == e) q[2 * i] = lo, q[2 * i + 1] = hi;
        }
      }
    }
    return make_uint2(
        __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410),
        __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410));
  }
  // Four held codes on this scale instead of `old`; ratio = old / s.  As above: the
  // rounded c * ratio is the code unless it lies next to a border.
  __device__ __forceinline__ uint32_t again(uint32_t c4, float old, float ratio) const {
    const uint32_t u = c4 ^ 0x80808080u;
    float c[4];
    uint32_t q[4];
    bool fine = near > 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + e)) - 8388736.f;  // 2^23 + (c + 128)
      const float y = fmaf(c[e], ratio, 12582912.f);
      fine = fine && fabsf(fmaf(c[e], ratio, 12582912.f - y)) < 0.4999f;
      q[e] = __float_as_uint(fmaxf(y, 12582912.f - 127.f));  // a held -128 as well
    }
    if (!fine) {
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const float x = static_cast<float>(static_cast<int8_t>(c4 >> (8 * e)));
        const float hi = x * old;
        const uint32_t k = code_of(hi, fmaf(x, old, -hi), s);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i == e) q[i] = k;
      }
    }
    return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  }
};

// Rows of a page that were held on scale `old`, 16 codes at a time by threads
// first, first + step, ...
__device__ __forceinline__ void requantize(int8_t* codes, int units, const Quantizer& qz, float old, int first,
                                           int step) {
  const float ratio = old / qz.s;
  for (int u = first; u < units; u += step) {
    uint4* p = reinterpret_cast<uint4*>(codes) + u;
    uint4 c = __ldcg(p);
    c.x = qz.again(c.x, old, ratio);
    c.y = qz.again(c.y, old, ratio);
    c.z = qz.again(c.z, old, ratio);
    c.w = qz.again(c.w, old, ratio);
    *p = c;
  }
}

// Largest |x| of 8 BF16 values, as bits in both halves of the result, with `m`.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const uint4& w) {
  m = __vimax3_u16x2(m, w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu);
  return __vimax3_u16x2(m, w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu);
}
// The same over finite values only.
__device__ __forceinline__ uint32_t finite_bits(uint32_t m, const uint4& w) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t lo = v[e] & 0x7FFFu, hi = (v[e] >> 16) & 0x7FFFu;
    m = max(m, lo < 0x7F80u ? lo : 0u);
    m = max(m, hi < 0x7F80u ? hi : 0u);
  }
  return m;
}
__device__ __forceinline__ uint32_t one_half(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
__device__ __forceinline__ uint32_t warp_max(uint32_t m) { return __reduce_max_sync(0xffffffffu, m); }
// The scale that a page needs for new rows whose largest |x| has these bits.
__device__ __forceinline__ float scale_for(uint32_t bits) { return __uint_as_float(bits << 16) / 127.f; }

// Sequence b's new rows: `first` is its first row of the packed input, n their
// number, `start` the position of the first.  None where a length in memory is out of
// range: rows put elsewhere would overwrite what the pages hold.
__device__ __forceinline__ void new_rows(const int* cu, const int* starts, int b, int T, int& first, int& n,
                                         int& start) {
  const int x = __ldcg(cu + b), y = __ldcg(cu + b + 1), z = __ldcg(starts + b);
  const bool fine = x >= 0 && y >= x && y <= T && z >= 0;
  if (!fine) set_fail(ATTN_ERR_INVALID_ARG);
  first = fine ? x : 0;
  n = fine ? y - x : 0;
  start = fine ? z : 0;
}

struct AppendArgs {
  const uint16_t* x[2];            // K, V rows (BF16)
  long long token_stride[2], head_stride[2];
  int8_t* codes[2];
  float* scales[2];
  const int *table, *cu, *starts;
  int B, T, Hkv, P, page, page_shift, max_blocks;
};

// What a CTA writes: rows [r0, r1) of page `page` take the packed rows from row0 on.
struct Found {
  int page, r0, r1;
  long long row0;
};

// Number `item` of the pages that new rows fall into, over all sequences.  Every
// thread of the CTA calls it; page < 0: there is none, or it is out of range.
template <int kThreads>
__device__ __forceinline__ Found find_page(const AppendArgs& a, int item) {
  __shared__ int s_warp[kThreads / 32];
  __shared__ Found s_found;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s_found.page = -1;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int first = 0, n = 0, start = 0, count = 0;
    if (b < a.B) {
      new_rows(a.cu, a.starts, b, a.T, first, n, start);
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
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) upto += s_warp[w];
      chunk += s_warp[w];
    }
    const int at = item - before - (upto - count);
    if (at >= 0 && at < count) {
      const int in_page = start & (a.page - 1);
      const long long blk = (long long)(start >> a.page_shift) + at;
      int id = blk < a.max_blocks ? __ldcg(a.table + (size_t)b * a.max_blocks + blk) : -1;
      if (id < 0 || id >= a.P) {
        set_fail(ATTN_ERR_INVALID_ARG);
        id = -1;
      }
      const int done = at == 0 ? 0 : at * a.page - in_page;  // rows that go to earlier pages
      Found f;
      f.page = id;
      f.r0 = at == 0 ? in_page : 0;
      f.r1 = min(a.page, f.r0 + n - done);
      f.row0 = (long long)first + done;
      s_found = f;
    }
    before += chunk;
    if (before > item) break;
  }
  __syncthreads();
  return s_found;
}

// D head dims; kUnits: 16-byte units of new rows a thread holds at most
// (page * D / 8 units over its threads).
template <int D, int kUnits, int kThreads>
__global__ void __launch_bounds__(kThreads) append_int8_kernel(const __grid_constant__ AppendArgs a) {
  griddep_wait();
  __shared__ uint32_t s_max[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kv = blockIdx.z;
  const Found f = find_page<kThreads>(a, blockIdx.x);
  if (f.page < 0) return;
  for (int head = blockIdx.y; head < a.Hkv; head += gridDim.y) {
    const uint16_t* x = a.x[kv] + f.row0 * a.token_stride[kv] + head * a.head_stride[kv];
    const size_t slot = (size_t)f.page * a.Hkv + head;
    int8_t* codes = a.codes[kv] + slot * a.page * D;
    float* scale = a.scales[kv] + slot;

    constexpr int kPerRow = D / 8;
    const int units = (f.r1 - f.r0) * kPerRow;
    uint4 w[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = tid + i * kThreads;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (u < units)
        w[i] = __ldcg(reinterpret_cast<const uint4*>(x + (u / kPerRow) * a.token_stride[kv] + (u % kPerRow) * 8));
    }
    const float s_old = f.r0 > 0 ? __ldcg(scale) : 0.f;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) m = max_bits(m, w[i]);
    m = warp_max(one_half(m));
    if (m >= 0x7F80u) {  // an infinity or a NaN in this warp's values
      m = 0;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) m = finite_bits(m, w[i]);
      m = warp_max(m);
    }
    if (lane == 0) s_max[warp] = m;
    __syncthreads();  // the maxima, and everyone has read the old scale
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, s_max[i]);
    const Quantizer qz(fmaxf(s_old, scale_for(m)));
    if (tid == 0) *scale = qz.s;

    if (qz.s > s_old) {  // rows the page holds already, on the coarser scale
      requantize(codes, f.r0 * (D / 16), qz, s_old, tid, kThreads);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = tid + i * kThreads;
      if (u < units) *reinterpret_cast<uint2*>(codes + (size_t)f.r0 * D + (size_t)u * 8) = qz.codes(w[i]);
    }
    __syncthreads();  // before the next head's maxima
  }
}

// The same for few rows a page: a warp takes one head at a time and reads its
// rows twice.
constexpr int kStepThreads = 256;
template <int D>
__global__ void __launch_bounds__(kStepThreads) append_step_int8_kernel(const __grid_constant__ AppendArgs a) {
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kv = blockIdx.y;
  const Found f = find_page<kStepThreads>(a, blockIdx.x);
  if (f.page < 0) return;
  constexpr int kPerRow = D / 8;
  const int units = (f.r1 - f.r0) * kPerRow;
  for (int head = warp; head < a.Hkv; head += kStepThreads / 32) {
    const uint16_t* x = a.x[kv] + f.row0 * a.token_stride[kv] + head * a.head_stride[kv];
    const size_t slot = (size_t)f.page * a.Hkv + head;
    int8_t* codes = a.codes[kv] + slot * a.page * D;
    float* scale = a.scales[kv] + slot;
    const float s_old = f.r0 > 0 ? __ldcg(scale) : 0.f;
    auto unit = [&](int u) {
      return __ldcg(reinterpret_cast<const uint4*>(x + (u / kPerRow) * a.token_stride[kv] + (u % kPerRow) * 8));
    };
    uint32_t m = 0;
    for (int u = lane; u < units; u += 32) m = max_bits(m, unit(u));
    m = warp_max(one_half(m));
    if (m >= 0x7F80u) {
      m = 0;
      for (int u = lane; u < units; u += 32) m = finite_bits(m, unit(u));
      m = warp_max(m);
    }
    const Quantizer qz(fmaxf(s_old, scale_for(m)));
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = qz.s;
    if (qz.s > s_old) requantize(codes, f.r0 * (D / 16), qz, s_old, lane, 32);
    for (int u = lane; u < units; u += 32)
      *reinterpret_cast<uint2*>(codes + (size_t)f.r0 * D + (size_t)u * 8) = qz.codes(unit(u));
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

constexpr int kReadWarps = 8;
constexpr int kReadCu = 1024;

// A lane reads 4 codes for FP32 values, 8 for BF16, and writes 16 bytes; a row of
// a head is D / that many lanes, and a warp takes as many tokens at a time as it
// has rows' worth of lanes, head by head.  Positions without a valid page read as
// zeros.
template <int D, bool FP32>
struct ReadCfg {
  static constexpr int kCodes = FP32 ? 4 : 8;
  static constexpr int kLanes = D / kCodes;
  static constexpr int kAtOnce = 32 / kLanes;              // tokens of a warp at a time
  static constexpr int kTokens = kReadWarps * kAtOnce;      // of a CTA
};
template <int D, bool FP32>
__global__ void __launch_bounds__(32 * kReadWarps) read_int8_kernel(const __grid_constant__ ReadArgs a) {
  using C = ReadCfg<D, FP32>;
  griddep_wait();
  __shared__ long long s_row[C::kTokens];  // row of the pool's head 0 in the token's page, or -1
  __shared__ int s_cu[kReadCu];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kv = blockIdx.y;
  const int t0 = blockIdx.x * C::kTokens;
  // The search runs in shared memory where the sequences' ends fit it.
  const bool near_cu = a.B < kReadCu;
  if (near_cu) {
    for (int b = tid; b <= a.B; b += 32 * kReadWarps) s_cu[b] = __ldcg(a.cu + b);
    __syncthreads();
  }
  auto cu = [&](int b) { return near_cu ? s_cu[b] : __ldcg(a.cu + b); };
  if (tid < C::kTokens && t0 + tid < a.T) {
    const int t = t0 + tid;
    int lo = 0, hi = a.B;  // the last sequence that begins at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu(mid) <= t) lo = mid; else hi = mid;
    }
    long long row = -1;
    const int first = cu(lo);
    if (t >= first && t < cu(lo + 1)) {
      const long long pos = (long long)__ldcg(a.starts + lo) + (t - first);
      const long long blk = pos >> a.page_shift;
      const int id = pos >= 0 && blk < a.max_blocks ? __ldcg(a.table + (size_t)lo * a.max_blocks + blk) : -1;
      if (id >= 0 && id < a.P)
        row = ((long long)id * a.Hkv << a.page_shift) + (pos & (a.page - 1));
    }
    if (row < 0) set_fail(ATTN_ERR_INVALID_ARG);
    s_row[tid] = row;
  }
  // Sequences have to follow one another from 0 to T.  By warps that search nothing (write-step
  // 5.2 us a pass; 5.6 ahead of the search).
  static_assert(C::kTokens <= 32, "the first warp searches");
  if (blockIdx.x == 0 && kv == 0 && warp > 0)
    for (long long b = tid - 32; b <= a.B; b += 32 * (kReadWarps - 1)) {
      const int x = cu((int)b);
      if (b == 0 ? x != 0 : x < cu((int)b - 1)) set_fail(ATTN_ERR_INVALID_ARG);
      if (b == a.B && x != a.T) set_fail(ATTN_ERR_INVALID_ARG);
    }
  __syncthreads();
  const int col = lane % C::kLanes * C::kCodes;
  const int8_t* codes = a.codes[kv] + col;
  const float* scales = a.scales[kv];
  const int t = warp * C::kAtOnce + lane / C::kLanes;
  if (t0 + t >= a.T) return;
  const long long at = s_row[t];
  const bool have = at >= 0;
  const long long row = have ? at : 0;
  const size_t out = (size_t)(t0 + t) * a.Hkv * D + col;
#pragma unroll 4
  for (int h = 0; h < a.Hkv; ++h) {
    const long long r = row + ((long long)h << a.page_shift);
    const float s = have ? __ldcg(scales + (r >> a.page_shift)) : 0.f;
    uint32_t c[C::kCodes / 4];
    if constexpr (FP32) {
      c[0] = __ldcg(reinterpret_cast<const uint32_t*>(codes + r * D));
    } else {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(codes + r * D));
      c[0] = v.x, c[1] = v.y;
    }
    float f[C::kCodes];
#pragma unroll
    for (int e = 0; e < C::kCodes; ++e)
      f[e] = have ? static_cast<float>(static_cast<int8_t>(c[e >> 2] >> (8 * (e & 3)))) * s : 0.f;
    if constexpr (FP32)  // evicted first: four bytes a code would push everything else out of L2 (27 -> 24 us)
      __stcs(reinterpret_cast<float4*>(static_cast<float*>(a.out[kv]) + out + h * D),
             make_float4(f[0], f[1], f[2], f[3]));
    else
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[kv]) + out + h * D) =
          make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                     pack_bf16x2(f[6], f[7]));
  }
}

template <int D, bool FP32>
cudaError_t launch_read(const ReadArgs& a, cudaStream_t stream) {
  return launch_pdl(read_int8_kernel<D, FP32>, dim3(ceil_div(a.T, ReadCfg<D, FP32>::kTokens), 2),
                    dim3(32 * kReadWarps), 0, stream, a);
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
  const unsigned most = (unsigned)(pages < T ? pages : T);
  // A step appends a row or a few to every sequence.
  if ((long long)T <= (long long)kStepRows * c.B) {
    auto kernel = c.d == 128 ? append_step_int8_kernel<128> : append_step_int8_kernel<64>;
    return launch_pdl(kernel, dim3(most, 2), dim3(kStepThreads), 0, stream, a);
  }
  // As many heads a CTA as make three waves of 8 CTAs an SM: the search for the page
  // takes as long as a head's rows, and a single wave waits for the SMs that have a CTA
  // more (16 prompts 42.4 us with their read-back, 41.4 in three waves).
  const int sms = device_sm_count();
  const long long waves = sms > 0 ? ((long long)most * c.Hkv * 2 + sms * 24ll - 1) / (sms * 24ll) : 1;
  const dim3 grid(most, ceil_div(c.Hkv, (int)std::min<long long>(waves, c.Hkv)), 2);
  const int units = c.page * c.d / 8;
  // 128 threads with up to 8 units each; 16 would cost half the CTAs of an SM.
#define ATTN_APPEND_CASE(DD, UU, TT) \
  if (c.d == DD && units == UU * TT) \
    return launch_pdl(append_int8_kernel<DD, UU, TT>, grid, dim3(TT), 0, stream, a);
  ATTN_APPEND_CASE(64, 1, 128)
  ATTN_APPEND_CASE(64, 2, 128)
  ATTN_APPEND_CASE(64, 4, 128)
  ATTN_APPEND_CASE(64, 8, 128)
  ATTN_APPEND_CASE(128, 2, 128)
  ATTN_APPEND_CASE(128, 4, 128)
  ATTN_APPEND_CASE(128, 8, 128)
  ATTN_APPEND_CASE(128, 8, 256)
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
  if (c.d == 128) return fp32 ? launch_read<128, true>(a, stream) : launch_read<128, false>(a, stream);
  return fp32 ? launch_read<64, true>(a, stream) : launch_read<64, false>(a, stream);
}

cudaError_t status_word_cache(void** word) { return cudaGetSymbolAddress(word, g_status_cache); }

}  // namespace attn

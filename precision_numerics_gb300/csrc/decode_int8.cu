// Attention of each sequence's newest tokens over the paged INT8 cache.
//
// For query token i of n_q of a sequence of len cached positions (the newest
// n_q of them its own) and head h of group h / G:
//   s_j = scale * q . (ck_j * ks_j),  j <= len - n_q + i
//   O   = sum_j softmax(s)_j (cv_j * vs_j),  LSE = ln sum_j exp(s_j)
// with codes ck, cv and the scales ks, vs of position j's page and head.
//
// What bounds it: every code is read once and used for n_q * G rows, so the
// bytes of the cache (2 d per position and head) over HBM's rate.  The rows of
// one key head (16 at a time) form the M side of mma.sync m16n8k16: with so
// few rows the tensor work is a small part of the time the bytes take, and
// the accumulators stay in registers.  A 128-row tcgen05 tile would be mostly
// padding here.
//
// Codes become FP16 exactly (|c| <= 127): the byte c + 128 under the exponent
// of 1024 is the FP16 number 1152 + c.  Q becomes FP16 after division by a
// power of two of its row's maximum, so it is exact down to 2^-17 of that
// maximum, and what lies below is rounded by at most 2^-25 of it.  P is
// rounded to FP16 (relative 2^-11) as the P V operand, scaled by 2^15 so that
// probabilities down to 2^-29 of the largest keep all their bits; the row sum
// adds the FP32 values.  Value scales enter P relative to a running power of
// two R >= vs, which the accumulators carry.
//
// Each warp streams its own 32-position tiles of K and V by TMA through its own
// ring (no barrier is shared between warps), with its own running maximum,
// sum and accumulator; the four warps of a CTA take every fourth tile and are
// merged through shared memory once at the end of a segment, the tiles of one
// (sequence, key head, row block) that the CTA has.
//
// Where a sequence can be longer than kWholeTiles tiles, the tiles of all
// segments, one behind the other, are dealt to the CTAs in equal runs, so that
// ragged lengths and few sequences keep every SM busy alike.  A run that holds a
// whole segment writes its output; of a segment that runs on into the next
// CTAs' runs every part leaves (m, l, unnormalised O) in the workspace, two slots
// a CTA at most, and decode_join_kernel joins them in the order of the CTAs.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {

static __device__ unsigned int g_status_decode;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;   // positions per tile
constexpr int kRows = 16;   // query rows (token, head of the group) per pass over the keys
constexpr int kWholeTiles = 16;  // sequences up to this long are not split
constexpr int kLeastRun = 4;     // tiles a CTA takes at least: one a warp

__device__ __forceinline__ void set_fail(unsigned int code) { atomicOr(&g_status_decode, code); }

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kHalfBytes = kTile * D;          // K or V of a tile
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kOffMerge = kWarps * kRingBytes;  // FP32 [warp][16 rows][64 columns]
  static constexpr int kOffStat = kOffMerge + kWarps * kRows * 64 * 4;  // m, l: FP32 [2][warp][16]
  // Per warp and stage: ks, vs of the tile's two halves (16 positions each),
  // then one word of flags (bit per half that was loaded).
  static constexpr int kOffHead = kOffStat + 2 * kWarps * kRows * 4;
  static constexpr int kHeadBytes = 32;
  static constexpr int kOffBar = kOffHead + kWarps * kStages * kHeadBytes;
  static constexpr int kSmemBytes = kOffBar + kWarps * kStages * 8;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// Copy 4 bytes to shared memory; `bar` counts one arrival when they landed.
__device__ __forceinline__ void copy4_arrive(uint32_t dst, const float* src, uint64_t* bar) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two bytes of `u` (codes + 128), picked by `sel`, as a pair of FP16 codes.
__device__ __forceinline__ uint32_t codes_f16(uint32_t u, uint32_t sel) {
  const uint32_t x = __byte_perm(u, 0x64646464u, sel);  // 1024 + (c + 128)
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64806480u));
  return r;
}

// Byte offset of 16-byte unit u of row r, as TMA's 128-byte (D = 128) or 64-byte
// (D = 64) swizzle places it: eight consecutive rows' units u cover all banks.
template <int D>
__device__ __forceinline__ uint32_t unit_offset(uint32_t r, uint32_t u) {
  return D == 128 ? r * 128u + ((u ^ (r & 7u)) << 4) : r * 64u + ((u ^ ((r >> 1) & 3u)) << 4);
}

// Natural-log LSE from the base-2 maximum and the row sum, which carries 2^15.
__device__ __forceinline__ float lse_of(float M, float L) {
  return L > 0.f ? (M + log2f(L) - 15.f) * 0.69314718055994531f : -INFINITY;
}

struct Args {
  const uint16_t* q;
  long long q_batch, q_token, q_head;
  const float *k_scale, *v_scale;
  const int *table, *lens;
  uint16_t* o;
  float* lse;
  int B, n_q, H, Hkv, G, P, page, page_shift, max_blocks, row_blocks;
  float scale_log2;
  // Split mode (else null): parts [CTA][2], and what each CTA's last segment is.
  float* parts;
  int4* chains;
};

// A part in the workspace: O [16][D], m [16], l [16], FP32.
template <int D>
constexpr int part_floats() { return kRows * (D + 2); }

__device__ __forceinline__ int length_of(const Args& a, int b) {
  const long long cap = (long long)a.max_blocks << a.page_shift;
  const int len = __ldcg(a.lens + b);
  if (len < 0 || len > cap) {
    set_fail(ATTN_ERR_INVALID_ARG);
    return len < 0 ? 0 : (int)cap;
  }
  return len;
}

__device__ __forceinline__ int tiles_of(int len) { return (int)(((unsigned)len + kTile - 1) / kTile); }

// A position in a CTA's run of tiles: tiles [ta, tb) of (sequence b, key head h,
// row block rb), `left` tiles behind them.
struct Walk {
  int b, h, rb, len, ta, tb;
  long long left;
  __device__ __forceinline__ int count(int warp) const {  // tiles of warp `warp`: ta + warp + kWarps * k
    return tb > ta + warp ? (tb - ta - warp + kWarps - 1) / kWarps : 0;
  }
  __device__ __forceinline__ bool next(const Args& a) {
    if (left <= 0) return false;
    if (++rb == a.row_blocks) {
      rb = 0;
      if (++h == a.Hkv) {
        h = 0;
        do {
          if (++b >= a.B) return false;
          len = length_of(a, b);
        } while (len == 0);
      }
    }
    ta = 0;
    tb = (int)min((long long)tiles_of(len), left);
    left -= tb;
    return true;
  }
};

// Sum over the CTA's threads before this one, and over all of them.
__device__ __forceinline__ long long scan_before(long long x, long long* s_warp, long long& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long upto = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_warp[w];
    all += s_warp[w];
  }
  return upto - x;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    decode_int8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::kStages;
  const uint32_t ring = smem_u32(smem) + warp * C::kRingBytes;
  const uint32_t heads = smem_u32(smem + C::kOffHead) + warp * C::kStages * C::kHeadBytes;
  float* s_merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float* s_m = reinterpret_cast<float*>(smem + C::kOffStat);
  float* s_l = s_m + kWarps * kRows;

  griddep_launch_dependents();
  bool ok = (smem_u32(smem) & 1023u) == 0;
  if (lane == 0) {
    // Five arrivals per tile: lane 0's, with the bytes of K and V, and the four
    // scales'.
    for (int s = 0; s < C::kStages; ++s) mbar_init(&bars[s], 5);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  griddep_wait();
  if (!ok && threadIdx.x == 0) set_fail(ATTN_ERR_INVALID_ARG);

  Walk sg;
  long long per = 0, begin = 0, run = 0;  // tiles of a run; where this CTA's begins, its length
  if (a.parts == nullptr) {
    const int x = blockIdx.x;
    sg.rb = x % a.row_blocks;
    sg.h = (x / a.row_blocks) % a.Hkv;
    sg.b = x / a.row_blocks / a.Hkv;
    sg.len = length_of(a, sg.b);
    sg.ta = 0;
    sg.tb = tiles_of(sg.len);
    sg.left = 0;
  } else {
    // All tiles, and the sequence in which this CTA's run begins.
    long long* s_warp = reinterpret_cast<long long*>(s_merge);
    const long long copies = (long long)a.Hkv * a.row_blocks;
    long long total = 0, sum;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      scan_before(b < a.B ? tiles_of(length_of(a, b)) : 0, s_warp, sum);
      total += sum;
    }
    total *= copies;
    per = max((total + gridDim.x - 1) / gridDim.x, (long long)kLeastRun);
    begin = per * blockIdx.x;
    int4* s_start = reinterpret_cast<int4*>(s_m);
    if (threadIdx.x == 0) s_start[0].x = -1;
    long long before = 0;
    for (int b0 = 0; b0 < a.B && before <= begin; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      const int len = b < a.B ? length_of(a, b) : 0;
      const int tiles = tiles_of(len);
      const long long at = before + copies * scan_before(tiles, s_warp, sum);
      if (begin >= at && begin < at + copies * tiles) {
        const long long rest = begin - at;
        s_start[0] = make_int4(b, len, (int)(rest / tiles), (int)(rest % tiles));
      }
      before += copies * sum;
    }
    __syncthreads();
    const int4 st = s_start[0];
    __syncthreads();
    if (threadIdx.x == 0) a.chains[blockIdx.x] = make_int4(0, 0, 0, 0);
    // Sequences without a position have no tile: their rows are empty.
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      if (length_of(a, b) > 0) continue;
      const size_t row = (size_t)b * a.n_q * a.H;
      for (int i = threadIdx.x; i < a.n_q * a.H * (D / 8); i += kThreads)
        reinterpret_cast<uint4*>(a.o + row * D)[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int i = threadIdx.x; i < a.n_q * a.H; i += kThreads) a.lse[row + i] = -INFINITY;
    }
    if (st.x < 0) return;  // more CTAs than runs
    run = min(per, total - begin);
    sg.b = st.x;
    sg.len = st.y;
    sg.h = st.z / a.row_blocks;
    sg.rb = st.z % a.row_blocks;
    sg.ta = st.w;
    sg.left = run;
    sg.tb = (int)min((long long)tiles_of(sg.len), sg.ta + sg.left);
    sg.left -= sg.tb - sg.ta;
  }

  // ------------------------------------------------------------------ loads
  // The loads run kStages tiles ahead, into the next segments too.
  Walk lw = sg;
  int ld_n = lw.count(warp);     // this warp's tiles of lw
  int ld_k = 0;                  // those issued
  int ld_base = 0;               // first tile whose page ids the lanes hold
  int id0 = -1, id1 = -1;        // pages of the two halves of tile ld_base + lane
  uint32_t issued = 0;
  bool more = ok;
  auto look_up = [&]() {
    ld_base = ld_k;
    id0 = id1 = -1;
    const long long pos = ((long long)lw.ta + warp + (long long)kWarps * (ld_k + lane)) * kTile;
    if (ld_k + lane < ld_n) {
      const int* row = a.table + (size_t)lw.b * a.max_blocks;
      id0 = __ldcg(row + (pos >> a.page_shift));
      if (id0 < 0 || id0 >= a.P) {
        set_fail(ATTN_ERR_INVALID_ARG);
        id0 = -1;
      }
      if (a.page >= kTile) {
        id1 = id0;
      } else if (pos + 16 < lw.len) {
        id1 = __ldcg(row + ((pos + 16) >> a.page_shift));
        if (id1 < 0 || id1 >= a.P) {
          set_fail(ATTN_ERR_INVALID_ARG);
          id1 = -1;
        }
      }
    }
  };
  auto issue = [&]() {
    if (!more) return;
    if (ld_k == ld_n) {
      do {
        more = lw.next(a);
        ld_n = more ? lw.count(warp) : 0;
      } while (more && ld_n == 0);
      if (!more) return;
      ld_k = 0;
      look_up();
    } else if (ld_k - ld_base == 32) {
      look_up();
    }
    const int p0 = __shfl_sync(0xffffffffu, id0, ld_k - ld_base);
    const int p1 = __shfl_sync(0xffffffffu, id1, ld_k - ld_base);
    const uint32_t st = issued % C::kStages;
    uint64_t* bar = &bars[st];
    const uint32_t head = heads + st * C::kHeadBytes;
    const uint32_t dst = ring + st * C::kStageBytes;
    if (lane == 0) {
      const uint32_t flags = (p0 >= 0 ? 1u : 0u) | (p1 >= 0 ? 2u : 0u);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(head + 16), "r"(flags) : "memory");
      if (a.page >= kTile) {
        mbar_arrive_expect_tx(bar, p0 >= 0 ? C::kStageBytes : 0);
        if (p0 >= 0) {
          const int in_page = ((lw.ta + warp + kWarps * ld_k) * kTile) & (a.page - 1);
          const int row = ((p0 * a.Hkv + lw.h) << a.page_shift) + in_page;
          tma_load_2d(dst, &tmK, bar, 0, row);
          tma_load_2d(dst + C::kHalfBytes, &tmV, bar, 0, row);
        }
      } else {
        mbar_arrive_expect_tx(bar, ((p0 >= 0) + (p1 >= 0)) * (C::kStageBytes / 2));
        if (p0 >= 0) {
          const int row = (p0 * a.Hkv + lw.h) << a.page_shift;
          tma_load_2d(dst, &tmK, bar, 0, row);
          tma_load_2d(dst + C::kHalfBytes, &tmV, bar, 0, row);
        }
        if (p1 >= 0) {
          const int row = (p1 * a.Hkv + lw.h) << a.page_shift;
          tma_load_2d(dst + 16 * D, &tmK, bar, 0, row);
          tma_load_2d(dst + C::kHalfBytes + 16 * D, &tmV, bar, 0, row);
        }
      }
    }
    if (lane < 4) {
      // ks, vs of half 0, ks, vs of half 1.  A half without a page takes any
      // valid scale: its flag hides it.
      const int p = max(lane < 2 ? p0 : p1, 0);
      copy4_arrive(head + 4 * lane, ((lane & 1) ? a.v_scale : a.k_scale) + (size_t)p * a.Hkv + lw.h, bar);
    }
    ++issued;
    ++ld_k;
  };
  if (more) look_up();
  for (int i = 0; i < C::kStages; ++i) issue();

  const int rows_total = a.n_q * a.G;
  uint32_t used = 0;
  bool last_segment = false;
  while (!last_segment) {
  // ------------------------------------------------------------------ Q rows
  // Row r of the block: token (rb * 16 + r) / G, head (rb * 16 + r) % G of the
  // group.  K step ks of the products covers head dims [16 ks, 16 ks + 16), of
  // which this thread holds 4 c + {0, 1} as k = 2c, 2c + 1 and 4 c + {2, 3} as
  // k = 2c + 8, 2c + 9 (the same assignment as the K operand's).
  int my_last[2];   // last visible position of rows g and g + 8 (-1: none)
  float f_row[2];   // factor of the scores, in base 2
  uint32_t qf[D / 16][4];
  const int tiles = sg.count(warp);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = sg.rb * kRows + g + 8 * i;
    const bool have = r < rows_total;
    const int t = r / a.G, hq = sg.h * a.G + r % a.G;
    const uint16_t* src = a.q + sg.b * a.q_batch + t * a.q_token + hq * a.q_head;
    uint2 w[D / 16];
    float m = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      w[ks] = have ? __ldcg(reinterpret_cast<const uint2*>(src + 16 * ks + 4 * c)) : make_uint2(0u, 0u);
      m = fmaxf(fmaxf(m, fmaxf(fabsf(__uint_as_float(w[ks].x << 16)), fabsf(__uint_as_float(w[ks].x & 0xFFFF0000u)))),
                fmaxf(fabsf(__uint_as_float(w[ks].y << 16)), fabsf(__uint_as_float(w[ks].y & 0xFFFF0000u))));
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // 2^e <= m < 2^(e+1), e within the range whose negative is a normal exponent.
    const int e = min(max((int)((__float_as_uint(m) >> 23) & 255u) - 127, -126), 126);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[ks][i] = pack_f16x2(__uint_as_float(w[ks].x << 16) * down, __uint_as_float(w[ks].x & 0xFFFF0000u) * down);
      qf[ks][2 + i] = pack_f16x2(__uint_as_float(w[ks].y << 16) * down, __uint_as_float(w[ks].y & 0xFFFF0000u) * down);
    }
    f_row[i] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
    my_last[i] = have ? sg.len - a.n_q + t : -1;
  }

  // ------------------------------------------------------------------ tiles
  float acc[D / 16][2][4];
#pragma unroll
  for (int u = 0; u < D / 16; ++u)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[u][e][x] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  float R = 0x1p-126f;  // power of two the accumulators' values are relative to

  for (int k = 0; k < tiles && ok; ++k) {
    const uint32_t st = used % C::kStages;
    ok = warp_wait(&bars[st], (used / C::kStages) & 1);
    if (!ok) break;
    ++used;
    const uint32_t tK = ring + st * C::kStageBytes, tV = tK + C::kHalfBytes;
    float ksc[2], vsc[2];
    uint32_t flags;
    {
      const uint32_t head = heads + st * C::kHeadBytes;
      asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(ksc[0]), "=f"(vsc[0]), "=f"(ksc[1]), "=f"(vsc[1])
                   : "r"(head)
                   : "memory");
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(flags) : "r"(head + 16) : "memory");
    }
    // S = Q K^T: 4 blocks of 8 positions.
    float s[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int u = 0; u < D / 16; u += 4) {
        uint32_t r[4];
        ldsm4(r, tK + unit_offset<D>(n * 8 + (lane & 7), u + (lane >> 3)));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t b = r[x] ^ 0x80808080u;
          mma_f16(s[n], qf[u + x], codes_f16(b, 0x4140u), codes_f16(b, 0x4342u));
        }
      }
    }
    // Scores in base 2; positions behind a row's last one are hidden.
    const int pos0 = (sg.ta + warp + kWarps * k) * kTile;
    const bool all = pos0 + kTile - 1 <= sg.len - a.n_q && flags == 3u;
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f0 = f_row[i] * ksc[0], f1 = f_row[i] * ksc[1];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = s[n][2 * i + x] * (n < 2 ? f0 : f1);
          if (!all && (pos0 + n * 8 + 2 * c + x > my_last[i] || !(flags & (n < 2 ? 1u : 2u)))) v = -INFINITY;
          s[n][2 * i + x] = v;
          mx[i] = fmaxf(mx[i], v);
        }
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
    }
    const float v_big = fmaxf((flags & 1u) ? vsc[0] : 0.f, (flags & 2u) ? vsc[1] : 0.f);
    float shrink = 1.f;
    if (v_big > R) {
      // The power of two at or above v_big (at most 2^126).
      const float r_new = __uint_as_float(min((__float_as_uint(v_big) + 0x7FFFFFu) & 0x7F800000u, 0x7E800000u));
      shrink = R / r_new;
      R = r_new;
    }
    const float inv_r = 1.f / R;
    const float vr[2] = {(flags & 1u) ? vsc[0] * inv_r : 0.f, (flags & 2u) ? vsc[1] * inv_r : 0.f};
    float alpha[2];
    uint32_t pf[2][4];  // P as the A operand: K step (16 positions), register
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float m_new = fmaxf(m_run[i], mx[i]);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      alpha[i] = ex2(m_run[i] - m_use);
      m_run[i] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float p0 = ex2(s[n][2 * i] - m_use + 15.f), p1 = ex2(s[n][2 * i + 1] - m_use + 15.f);
        sum += p0 + p1;
        const float w = vr[n >> 1];
        pf[n >> 1][(n & 1) * 2 + i] = pack_f16x2(p0 * w, p1 * w);
      }
      l_run[i] = l_run[i] * alpha[i] + sum;
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f || shrink != 1.f)) {
      const float s0 = alpha[0] * shrink, s1 = alpha[1] * shrink;
#pragma unroll
      for (int u = 0; u < D / 16; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          acc[u][e][0] *= s0;
          acc[u][e][1] *= s0;
          acc[u][e][2] *= s1;
          acc[u][e][3] *= s1;
        }
    }
    // O += P V.  A transposed load gives positions 2c, 2c + 1 of the columns
    // d = 16 u + 2 g (even bytes) and + 1 (odd bytes).
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int u = 0; u < D / 16; u += 2) {
        uint32_t r[4];  // positions 0-7 and 8-15 of unit u, then of unit u + 1
        ldsm4_trans(r, tV + unit_offset<D>(kk * 16 + (lane & 15), u + (lane >> 4)));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t b0 = r[2 * x] ^ 0x80808080u, b1 = r[2 * x + 1] ^ 0x80808080u;
          mma_f16(acc[u + x][0], pf[kk], codes_f16(b0, 0x4240u), codes_f16(b1, 0x4240u));
          mma_f16(acc[u + x][1], pf[kk], codes_f16(b0, 0x4341u), codes_f16(b1, 0x4341u));
        }
      }
    __syncwarp();
    issue();
  }

  // ------------------------------------------------------------------ merge
  const bool whole = sg.ta == 0 && sg.tb == tiles_of(sg.len);
  float* part = nullptr;
  if (!whole) {
    part = a.parts + (size_t)(2 * blockIdx.x + (sg.ta == 0)) * part_floats<D>();
    if (sg.ta == 0 && threadIdx.x == 0) {
      // The segment runs on into as many CTAs as hold the rest of its tiles.
      const long long end = begin + run - sg.tb + tiles_of(sg.len);
      a.chains[blockIdx.x] = make_int4((int)((end - 1) / per) - (int)blockIdx.x, sg.b, sg.h, sg.rb);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 1);
    l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 2);
    if (c == 0) {
      s_m[warp * kRows + g + 8 * i] = m_run[i];
      s_l[warp * kRows + g + 8 * i] = l_run[i];
    }
  }
  __syncthreads();
  float fac[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w * kRows + g + 8 * i]);
    const float M_use = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) L += s_l[w * kRows + g + 8 * i] * ex2(s_m[w * kRows + g + 8 * i] - M_use);
    fac[i] = ex2(m_run[i] - M_use) * R;
    const int r = sg.rb * kRows + g + 8 * i;
    if (whole) {
      fac[i] = L > 0.f ? fac[i] / L : 0.f;
      if (warp == 0 && c == 0 && r < rows_total) {
        const size_t row = ((size_t)sg.b * a.n_q + r / a.G) * a.H + sg.h * a.G + r % a.G;
        a.lse[row] = lse_of(M, L);
      }
    } else if (warp == 0 && c == 0) {
      part[kRows * D + g + 8 * i] = M;
      part[kRows * D + kRows + g + 8 * i] = L;
    }
  }
#pragma unroll
  for (int half = 0; half < D / 64; ++half) {
    if (half > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float(&x)[2][4] = acc[half * 4 + u];
        const float4 v = make_float4(x[0][2 * i] * fac[i], x[1][2 * i] * fac[i], x[0][2 * i + 1] * fac[i],
                                     x[1][2 * i + 1] * fac[i]);
        // Odd rows' units are moved by four, so a phase of eight lanes covers all banks.
        *reinterpret_cast<float4*>(s_merge + (warp * kRows + r) * 64 + (((u * 4 + c) ^ ((r & 1) << 2)) << 2)) = v;
      }
    }
    __syncthreads();
    // 16 rows x 64 columns over 128 threads: 8 columns each.
    const int r = threadIdx.x >> 3, part8 = threadIdx.x & 7;
    float v[8] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 x = *reinterpret_cast<const float4*>(
            s_merge + (w * kRows + r) * 64 + (((part8 * 2 + e) ^ ((r & 1) << 2)) << 2));
        v[4 * e] += x.x;
        v[4 * e + 1] += x.y;
        v[4 * e + 2] += x.z;
        v[4 * e + 3] += x.w;
      }
    const int rr = sg.rb * kRows + r;
    if (!whole) {
      float4* p = reinterpret_cast<float4*>(part + r * D + half * 64 + part8 * 8);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if (rr < rows_total) {
      const size_t row = ((size_t)sg.b * a.n_q + rr / a.G) * a.H + sg.h * a.G + rr % a.G;
      *reinterpret_cast<uint4*>(a.o + row * D + half * 64 + part8 * 8) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
    }
  }
  last_segment = !sg.next(a);
  }  // segments
  if (!ok) {
    if (lane == 0) set_fail(ATTN_ERR_TIMEOUT);
    // Do not leave while copies into this CTA's shared memory are in flight.
    for (; used < issued; ++used) mbar_wait(&bars[used % C::kStages], (used / C::kStages) & 1);
  }
}

// Joins the parts of the segments that begin in one CTA's run and end in
// another's: grid (CTAs of the main kernel, rows), one row per CTA, whose warps
// take every fourth part.  The order of the sums is that of the parts.
template <int D>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(const Args a) {
  __shared__ float s_o[kWarps][D], s_l[kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int4 ch = __ldcg(a.chains + blockIdx.x);
  const int rr = ch.w * kRows + blockIdx.y;
  if (ch.x == 0 || rr >= a.n_q * a.G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = ch.x + 1;
  auto part = [&](int i) {
    return a.parts + (size_t)(2 * (blockIdx.x + i) + (i == 0)) * part_floats<D>();
  };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(part(i) + kRows * D + blockIdx.y));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float M_use = M == -INFINITY ? 0.f : M;
  float L = 0.f, o[D / 32] = {};
#pragma unroll 4
  for (int i = warp; i < n; i += kWarps) {
    const float* p = part(i);
    const float f = ex2(__ldcg(p + kRows * D + blockIdx.y) - M_use);
    L += f * __ldcg(p + kRows * D + kRows + blockIdx.y);
    const float* x = p + blockIdx.y * D + lane * (D / 32);
    if constexpr (D == 128) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(x));
      o[0] += f * v.x, o[1] += f * v.y, o[2] += f * v.z, o[3] += f * v.w;
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(x));
      o[0] += f * v.x, o[1] += f * v.y;
    }
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) s_o[warp][lane * (D / 32) + e] = o[e];
  if (lane == 0) s_l[warp] = L;
  __syncthreads();
  const size_t row = ((size_t)ch.y * a.n_q + rr / a.G) * a.H + ch.z * a.G + rr % a.G;
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) L += s_l[w];
  if (threadIdx.x < D / 2) {
    const int d = threadIdx.x * 2;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += s_o[w][d], y += s_o[w][d + 1];
    const float inv = L > 0.f ? 1.f / L : 0.f;
    *reinterpret_cast<uint32_t*>(a.o + row * D + d) = pack_bf16x2(x * inv, y * inv);
  }
  if (threadIdx.x == 0) a.lse[row] = lse_of(M, L);
}

// Runs the tiles are dealt in: two CTAs fit an SM.  (The largest device's count
// where there is no device to ask, for workspace sizes.)
unsigned decode_runs() {
  const int sms = device_sm_count();
  return 2u * (sms > 0 ? sms : 152);
}

bool make_tmap_codes(CUtensorMap* map, const void* base, const PagedCache& c) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)c.d, (cuuint64_t)c.P * c.Hkv * c.page};
  const cuuint64_t strides[1] = {(cuuint64_t)c.d};
  const cuuint32_t box[2] = {(cuuint32_t)c.d, (cuuint32_t)std::min(c.page, kTile)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_decode_impl(const PagedCache& cache, const Args& a, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap mk, mv;
  if (!make_tmap_codes(&mk, cache.k, cache) || !make_tmap_codes(&mv, cache.v, cache))
    return cudaErrorInvalidValue;
  auto kernel = decode_int8_kernel<D>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (err != cudaSuccess) return err;
  if (a.parts == nullptr) {
    const unsigned grid = (unsigned)((long long)a.B * a.Hkv * a.row_blocks);
    return launch_pdl(kernel, dim3(grid), dim3(kThreads), C::kSmemBytes, stream, mk, mv, a);
  }
  const unsigned runs = decode_runs();
  err = launch_pdl(kernel, dim3(runs), dim3(kThreads), C::kSmemBytes, stream, mk, mv, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(decode_join_kernel<D>, dim3(runs, std::min(kRows, a.n_q * a.G)), dim3(kThreads), 0, stream, a);
}

bool splits(const PagedCache& c) { return (long long)c.max_blocks * c.page > (long long)kWholeTiles * kTile; }

}  // namespace

size_t decode_workspace_bytes(const PagedCache& c, int, int) {
  if (!splits(c)) return 0;
  const size_t part = (c.d == 128 ? part_floats<128>() : part_floats<64>()) * sizeof(float);
  return align256(decode_runs() * 2 * part) + align256(decode_runs() * sizeof(int4));
}

cudaError_t launch_decode_int8(const PagedCache& c, const void* q, const long long* strides, const int* lens,
                               void* o, float* lse, int n_q, int H, float scale, void* workspace,
                               cudaStream_t stream) {
  Args a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_batch = strides[0];
  a.q_token = strides[1];
  a.q_head = strides[2];
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.table = c.table;
  a.lens = lens;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.B = c.B, a.n_q = n_q, a.H = H, a.Hkv = c.Hkv, a.G = H / c.Hkv, a.P = c.P, a.page = c.page;
  a.page_shift = page_shift(c.page);
  a.max_blocks = c.max_blocks;
  a.row_blocks = ceil_div(n_q * a.G, kRows);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.parts = nullptr;
  a.chains = nullptr;
  if (splits(c)) {
    const size_t part = (c.d == 128 ? part_floats<128>() : part_floats<64>()) * sizeof(float);
    a.parts = static_cast<float*>(workspace);
    a.chains = reinterpret_cast<int4*>(static_cast<char*>(workspace) + align256(decode_runs() * 2 * part));
  }
  return c.d == 128 ? launch_decode_impl<128>(c, a, stream) : launch_decode_impl<64>(c, a, stream);
}

cudaError_t read_and_clear_status_decode(unsigned int* out, cudaStream_t stream) {
  static const unsigned int zero = 0;
  cudaError_t err = cudaMemcpyFromSymbolAsync(out, g_status_decode, sizeof(unsigned int), 0,
                                              cudaMemcpyDeviceToHost, stream);
  if (err != cudaSuccess) return err;
  err = cudaStreamSynchronize(stream);
  if (err != cudaSuccess) return err;
  err = cudaMemcpyToSymbolAsync(g_status_decode, &zero, sizeof(unsigned int), 0,
                                cudaMemcpyHostToDevice, stream);
  if (err != cudaSuccess) return err;
  return cudaStreamSynchronize(stream);
}

}  // namespace attn

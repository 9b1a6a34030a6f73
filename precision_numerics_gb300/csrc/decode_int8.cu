// Attention of each sequence's newest tokens over the paged INT8 cache.
//
// For query token i of n_q of a sequence of len cached positions (the newest
// n_q of them its own) and head h of group h / G:
//   s_j = scale * q . (ck_j * ks_j),  j <= len - n_q + i
//   O   = sum_j softmax(s)_j (cv_j * vs_j),  LSE = ln sum_j exp(s_j)
// with codes ck, cv and the scales ks, vs of position j's page and head.
//
// What bounds it: up to 32 rows of a key head (n_q * G) use every code that is
// read, so with few rows the bytes of the cache (2 d per position and head) over
// HBM's rate, which leave the tensor pipe mostly idle.  The products are mma.sync
// m16n8k16 with the codes on the 16-row side, S^T = K Q^T and O^T = V^T P^T, and the
// query rows of one key head on the 8-column side, NT blocks of 8: the conversion of
// a code, which costs the most instructions, serves all of them, and few rows leave
// little of a product empty.  From 17 rows on the accumulators' registers leave 8
// warps an SM, and the chain of a tile bounds it instead; tcgen05 with 128 positions
// of codes on its rows and the accumulators in TMEM would not have that limit, and is
// not built.  More than 32 rows take a pass over the keys for every 32.
//
// Codes become FP16 exactly (|c| <= 127): the byte c + 128 under the exponent
// of 1024 is the FP16 number 1152 + c.  Q becomes FP16 after division by a
// power of two of its row's maximum, so it is exact down to 2^-17 of that
// maximum, and what lies below is rounded by at most 2^-25 of it.  The weights
// of the values' codes, P vs, are rounded to FP16 (relative 2^-11) as the P V
// operand, times 2^15 / R with a running power of two R >= vs, which the
// accumulators carry.  While the scales that a warp meets lie within 2^8 of R, one
// R serves all rows, and a row's weights down to 2^-20 of its largest keep all their
// bits.  Scales further apart could take a row's bits by values that it does not see
// or barely weighs (a large V of a later token, say): the warp then goes on with an
// R of each row's own, the power of two at or above its largest 2^(s - m) vs.  On 64
// sequences of 500 to 16000 positions that takes 99 us in place of 102 with 4 rows a key
// head, 131 in place of 111 with 12, 159 in place of 142 with 20 (d = 128).  The row
// sum adds the FP32 values.  The 2^15 goes with the scale: taken into the exponent's
// maximum it would be lost in part where scores reach 2^24.
//
// Each warp streams its own 32-position tiles of K and V by TMA through its own
// ring (no barrier is shared between warps), with its own running maximum,
// sum and accumulator; the four warps of a CTA take every fourth tile and are
// merged through shared memory once at the end of a segment, the tiles of one
// (sequence, key head, row block) that the CTA has.
//
// Which way the work is split follows from the room in the block table, not from the
// lengths, which are device data: 77 positions take 4.2 us in a table that is as wide
// as they need and 6.9 in one of 2048 blocks.  In a table for short sequences a CTA
// takes every segment.  Where the segments are fewer than the CTAs that the SMs hold,
// and not too long, a cluster of CTAs shares one and joins its
// parts through their shared memory.  Else the tiles of all segments, one behind the
// other, are dealt to the CTAs in equal runs, so that ragged lengths and few sequences
// keep every SM busy alike.  A run that holds a whole segment writes its output; of a
// segment that runs on into the next CTAs' runs every part leaves (m, l, O / l) in the
// workspace, two slots a CTA at most, and decode_join_kernel joins them in the order of
// the CTAs.  Warps and parts are joined as means with weights of at most 1, so that
// values up to the largest that a scale allows do not overflow on the way.
//
// The kernel also serves attention behind a prefix that a batch shares.  Either (kWithPrefix) it goes over the prefix's
// pages ahead of each sequence's own: the prefix's positions, then none up to a whole tile, then the own ones.  Or
// decode_shared_int8.cu's kernel has the prefix, and this one leaves (m, l, O / l) of every row for the join with it
// (kBehind; an instance of its own: the choice at run time cost attn_decode_int8 2% with 20 rows).
//
// Measured (d = 128, 8 key heads, pages of 64): 64 sequences of 500 to 16000
// positions with 4 query rows a key head 102-105 us (5.9 TB/s, 86% of a copy's
// rate), one of 131000 positions 50 us (5.4 TB/s); d = 64: 58 us and 30 us; with 20
// rows 64 sequences 142 us, where the dependent conversions and products of a tile (2
// us a warp) set the pace; 8 sequences of 4000 positions with 256 rows 148 us.
#include <float.h>
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
constexpr int kWholeTiles = 16;  // sequences up to this long are not split
constexpr int kWholeMany = 2048;  // positions up to which many sequences are not split for another join
constexpr int kLeastRun = 4;     // tiles a CTA takes at least: one a warp
// Parts that the warps of a row's join have in flight together; a segment has hardly more
// (one sequence of 114589 positions, 1 key head of 64 and 6 rows: 14.8 us; 21.2 in runs of 4
// tiles, 600 parts, by half as many warps).
constexpr int kJoinBatch = 8, kJoinShared = 16;
constexpr int kPartsAtOnce = kJoinBatch * kJoinShared;
// A segment's start and end (its Q rows, the merge of the warps, its output) take
// as long as so many tiles: runs are measured in tiles plus this for each segment
// that begins in them.
constexpr int kSegmentCost = 8;
constexpr int kMaxCluster = 8;  // CTAs that can share a segment through their shared memory
constexpr int kClusterTiles = 16;  // tiles a CTA that the join is worth
constexpr int kLoneTiles = 8;      // sequences up to this long are not shared by a cluster

__device__ __forceinline__ void set_fail(unsigned int code) { atomicOr(&g_status_decode, code); }

// CTAs an SM for blocks of 8 rows of d columns: as many as the registers allow.
// More warps are worth more than deeper rings (d = 64, 8 rows: 4 CTAs with 2 stages
// 56.7 us on a ragged batch, 3 with 4 stages 62.6, 2 with 5 stages 75.8);
// 12 rows over 64 sequences: 3 CTAs with 3 stages 81 us, 2 with 5 stages 96; d = 128,
// 12 rows: 3 CTAs with 2 stages 114 us, 2 with 3 stages 121; d = 64, 20 rows: 3 CTAs
// with 3 stages 99 us, 2 with 4 stages 111 (one sequence and key head 17.3 and 15.8).
constexpr int ctas_per_sm(int d, int nt) {
  if (d == 64) return nt == 1 ? 4 : nt <= 3 ? 3 : 2;
  return nt <= 2 ? 3 : 2;
}

// NT blocks of 8 query rows (token, head of the group) per pass over the keys.
template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = ctas_per_sm(D, NT);
  static constexpr int kStages = D == 64 ? (NT == 1 ? 2 : NT == 4 ? 4 : 3) : 2;
  static constexpr int kHalfBytes = kTile * D;          // K or V of a tile
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  // Columns that are merged at a time, and the buffer, FP32 [warp][rows][columns].
  static constexpr int kMerge = D == 128 && NT == 2 ? 32 : 64;
  static constexpr int kOffMerge = kWarps * kRingBytes;
  static constexpr int kOffStat = kOffMerge + kWarps * kRows * kMerge * 4;  // m, l: FP32 [2][warp][rows]
  // Per warp and stage: ks, vs of the tile's two halves (16 positions each),
  // then one word of flags (bit per half that was loaded).
  static constexpr int kOffHead = kOffStat + 2 * kWarps * kRows * 4;
  static constexpr int kHeadBytes = 32;
  static constexpr int kOffBar = kOffHead + kWarps * kStages * kHeadBytes;
  static constexpr int kSmemBytes = kOffBar + kWarps * kStages * 8;
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of an SM");
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

template <int kOffset>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(kOffset)
               : "memory");
}
template <int kOffset>
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(kOffset)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8x8 matrix of 16-bit values held one row (two columns) per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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

// The same place in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(uint32_t saddr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float load_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// All threads of the cluster; what was written before is seen after.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Byte offset of 16-byte unit u of row r, as TMA's 128-byte (D = 128) or 64-byte
// (D = 64) swizzle places it: eight consecutive rows' units u cover all banks.
template <int D>
__device__ __forceinline__ uint32_t unit_offset(uint32_t r, uint32_t u) {
  return D == 128 ? r * 128u + ((u ^ (r & 7u)) << 4) : r * 64u + ((u ^ ((r >> 1) & 3u)) << 4);
}

// 1 / L (L < 2^32, off by 2 units of the last bit at most), or 0 where a row has seen
// nothing.  A NaN stays one.
__device__ __forceinline__ float inverse(float L) { return L == 0.f ? 0.f : __fdividef(1.f, L); }

// Natural-log LSE from the base-2 maximum and the row sum.
__device__ __forceinline__ float lse_of(float M, float L) {
  return L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// The whole number W >= w that is nearest w + 1/2, given w + 1/2 (|w| < 2^21), plus 1.5 * 2^23; its
// low byte and the bit above are W's.  And 2^(E - 127 + SIGN * W), of an exponent within 1 to 254.
__device__ __forceinline__ float whole(float w_half) { return w_half + 12582912.f; }
template <int E, int SIGN>
__device__ __forceinline__ float exp2_whole(float w_half) {
  const uint32_t W = __float_as_uint(whole(w_half)) << 23;
  return __uint_as_float(SIGN > 0 ? ((uint32_t)E << 23) + W : ((uint32_t)E << 23) - W);
}
// Largest ratio of R to a scale that one R for all rows serves.
constexpr float kNarrow = 0x1p8f;
// Least w + 1/2: codes of a scale below 2^-110 lose bits that are multiples of 2^-150.
constexpr float kLeastWeight = -110.f;

// A segment in several parts: those behind the first (0: nothing to join), its
// sequence, key head * row_blocks + row block, and the CTA it begins in.
struct Chain {
  int more, b, hr, cta;
};
static_assert(sizeof(Chain) == 16, "one 16-byte access");

struct Args {
  const uint16_t* q;
  long long q_batch, q_token, q_head;
  const float *k_scale, *v_scale;
  const int *table, *lens;
  uint16_t* o;
  float* lse;
  uint32_t by_G;  // ceil(2^32 / G)
  int B, n_q, H, Hkv, G, P, page, page_shift, max_blocks, row_blocks;
  float scale_log2;
  // Split mode (else null): parts [CTA][2], and the segments that are joined, by
  // the segment's number if by_segment, else by the CTA it begins in.
  float* parts;
  Chain* chains;
  int by_segment;
  unsigned cluster;  // without split mode: CTAs that share a segment
  // In place of o and lse (kBehind): O / l [rows][D], m [rows], l [rows], FP32, of all B n_q H
  // rows, for a caller that joins them with others.
  float* whole;
  size_t whole_rows;
  // With a prefix that all sequences begin with (kWithPrefix): its pages, its length, and their number.
  const int *pre_table, *pre_len;
  int pre_blocks;
};

// What a kernel does besides the sequences' own positions: nothing; it goes over the pages of a prefix ahead of them; or
// it runs behind the kernel that has the prefix.
enum Mode { kAlone, kWithPrefix, kBehind };

// The prefix as the sequences have it (kWithPrefix): `len` positions, then none up to a whole tile, from where on a
// sequence's own are counted.
struct Prefix {
  int len, end;
};
template <int MODE>
__device__ __forceinline__ Prefix prefix_of(const Args& a);

// A part in the workspace: O [rows][D] divided by l, m [rows], l [rows], FP32.
__host__ __device__ constexpr int part_floats(int d, int rows) { return rows * (d + 2); }

// Query token of row r (< 2^14) of a key head's rows, and its row of o and lse.
__device__ __forceinline__ int token_of(const Args& a, int r) {
  return a.G == 1 ? r : (int)__umulhi((uint32_t)r, a.by_G);
}
__device__ __forceinline__ size_t out_row(const Args& a, int b, int h, int r) {
  const int t = token_of(a, r);
  return ((size_t)b * a.n_q + t) * a.H + h * a.G + (r - t * a.G);
}

// Four columns of a row of the output, and its maximum and sum.
template <int D, int MODE>
__device__ __forceinline__ void put_columns(const Args& a, size_t row, int col, float x, float y, float z, float w) {
  if constexpr (MODE == kBehind)
    *reinterpret_cast<float4*>(a.whole + row * D + col) = make_float4(x, y, z, w);
  else
    *reinterpret_cast<uint2*>(a.o + row * D + col) = make_uint2(pack_bf16x2(x, y), pack_bf16x2(z, w));
}
template <int D, int MODE>
__device__ __forceinline__ void put_sums(const Args& a, size_t row, float M, float L) {
  if constexpr (MODE == kBehind) {
    a.whole[a.whole_rows * D + row] = M;
    a.whole[a.whole_rows * (D + 1) + row] = L;
  } else {
    a.lse[row] = lse_of(M, L);
  }
}

// A sequence's length as it is in memory, and what is made of it.  Separate, since
// the check waits for the value.
__device__ __forceinline__ int read_length(const Args& a, int b) { return b < a.B ? __ldcg(a.lens + b) : 0; }
__device__ __forceinline__ int checked(const Args& a, int len) {
  const long long cap = (long long)a.max_blocks << a.page_shift;
  if (len < 0 || len > cap) {
    set_fail(ATTN_ERR_INVALID_ARG);
    return len < 0 ? 0 : (int)cap;
  }
  return len;
}

template <int MODE>
__device__ __forceinline__ Prefix prefix_of(const Args& a) {
  if constexpr (MODE != kWithPrefix) return Prefix{0, 0};
  const int len = __ldcg(a.pre_len);
  const long long cap = (long long)a.pre_blocks << a.page_shift;
  const int cut = len < 0 ? 0 : (int)min((long long)len, cap);
  if (cut != len) set_fail(ATTN_ERR_INVALID_ARG);
  return Prefix{cut, (cut + kTile - 1) / kTile * kTile};
}

__device__ __forceinline__ int tiles_of(int len) { return (int)(((unsigned)len + kTile - 1) / kTile); }

// Cost of a segment: kSegmentCost, then one per tile.
__device__ __forceinline__ int cost_of(int len) { return len > 0 ? tiles_of(len) + kSegmentCost : 0; }

// A position in a CTA's run: tiles [ta, tb) of (sequence b, key head h, row block
// rb), cost `left` behind them.
struct Walk {
  int before;  // positions of a prefix, which lengths count in
  int b, h, rb, len, ta, tb;
  int len_next;  // of sequence b + 1, read ahead, not yet checked
  long long left;
  __device__ __forceinline__ int count(int warp) const {  // tiles of warp `warp`: ta + warp + kWarps * k
    return tb > ta + warp ? (tb - ta - warp + kWarps - 1) / kWarps : 0;
  }
  // The tiles that the run has of this segment, whose first `from` units of cost are before it.
  __device__ __forceinline__ void take(int from) {
    const int to = (int)min((long long)cost_of(len), from + left);
    left -= to - from;
    ta = max(from - kSegmentCost, 0);
    tb = max(to - kSegmentCost, 0);
  }
  __device__ __forceinline__ bool next(const Args& a) {
    if (left <= 0) return false;
    if (++rb == a.row_blocks) {
      rb = 0;
      if (++h == a.Hkv) {
        h = 0;
        do {
          if (++b >= a.B) return false;
          len = before + checked(a, len_next);
          len_next = read_length(a, b + 1);
        } while (len == 0);
      }
    }
    take(0);
    return tb > 0;  // a run may end before the first tile
  }
};

// x / y, in 32 bits where they suffice.
__device__ __forceinline__ long long divide(long long x, int y) {
  return x <= 0xffffffffll ? (long long)((unsigned)x / (unsigned)y) : x / y;
}

// Sequences without a position have no tile: their rows are empty.  The CTAs take
// them by turns; len_first is the unchecked length of sequence blockIdx.x.
template <int D, int MODE>
__device__ __forceinline__ void fill_empty(const Args& a, int len_first, int before) {
  if (MODE == kWithPrefix && before > 0) return;
  const int copies = a.Hkv * a.row_blocks;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (checked(a, b == blockIdx.x ? len_first : read_length(a, b)) > 0) continue;
    const size_t row = (size_t)b * a.n_q * a.H;
    if constexpr (MODE == kBehind) {
      for (int i = threadIdx.x; i < a.n_q * a.H * (D / 4); i += kThreads)
        reinterpret_cast<float4*>(a.whole + row * D)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int i = threadIdx.x; i < a.n_q * a.H * (D / 8); i += kThreads)
        reinterpret_cast<uint4*>(a.o + row * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    for (int i = threadIdx.x; i < a.n_q * a.H; i += kThreads) put_sums<D, MODE>(a, row + i, -INFINITY, 0.f);
    if (a.by_segment)
      for (int i = threadIdx.x; i < copies; i += kThreads) a.chains[(long long)b * copies + i] = Chain{0, 0, 0, 0};
  }
}

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

template <int D, int NT, int MODE>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas)
    decode_int8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const Args a) {
  using C = Cfg<D, NT>;
  constexpr int kRows = C::kRows;
  constexpr bool PRE = MODE == kWithPrefix, behind = MODE == kBehind;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::kStages;
  const uint32_t ring = smem_u32(smem) + warp * C::kRingBytes;
  const uint32_t heads = smem_u32(smem + C::kOffHead) + warp * C::kStages * C::kHeadBytes;
  float* s_merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float* s_m = reinterpret_cast<float*>(smem + C::kOffStat);
  float* s_l = s_m + kWarps * kRows;
  float* s_w = s_m + warp * kRows;  // per row while the warp has tiles: see `wide`
  // In the merge's buffer between merges: Q, then per row the factor of its scores
  // and its last visible position.
  uint2* s_q = reinterpret_cast<uint2*>(s_merge);
  float* s_f = reinterpret_cast<float*>(s_q + NT * (D / 16) * 32);
  int* s_last = reinterpret_cast<int*>(s_f + kRows);

  // The dependents (the join, or the next launch) are let in when a warp has no more
  // tiles to ask for, not here: they would fill the slots that free up first and the
  // CTAs of the next launch keep an uneven share of the SMs (one long sequence 54 us a
  // call, 72 with it).
  bool ok = (smem_u32(smem) & 1023u) == 0;
  if (lane == 0) {
    // Five arrivals per tile: lane 0's, with the bytes of K and V, and the four
    // scales'.
    for (int s = 0; s < C::kStages; ++s) mbar_init(&bars[s], 5);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  // Behind the prefix's kernel, which let this one in when all before it was complete, and of which
  // nothing is used here: its end is waited for by the time this one lets the join in, which reads both's parts.
  // (That q, tables and lengths are seen without a wait here is the assumption named in shared_prefix_kernel.)
  if (!behind) griddep_wait();
  if (!ok && threadIdx.x == 0) set_fail(ATTN_ERR_INVALID_ARG);

  const Prefix pre = prefix_of<MODE>(a);
  Walk sg;
  sg.before = pre.end;
  int len_first = 1;
  long long per = 0;  // cost of a run
  if (a.parts == nullptr) {
    unsigned x = blockIdx.x, rank = 0;
    if (a.cluster > 1) rank = x % a.cluster, x /= a.cluster;
    sg.rb = x % a.row_blocks;
    sg.h = (x / a.row_blocks) % a.Hkv;
    sg.b = x / a.row_blocks / a.Hkv;
    sg.len = pre.end + checked(a, read_length(a, sg.b));
    sg.len_next = 0;
    sg.ta = 0;
    sg.tb = tiles_of(sg.len);
    if (a.cluster > 1) {  // its share of the tiles (products below 2^26 * 8)
      sg.ta = sg.tb * rank / a.cluster;
      sg.tb = sg.tb * (rank + 1) / a.cluster;
    }
    sg.left = 0;
  } else {
    // All segments' cost, and the sequence in which this CTA's run begins.  The
    // first kThreads sequences are read and scanned once.
    long long* s_warp = reinterpret_cast<long long*>(s_merge);
    int* s_longest = reinterpret_cast<int*>(s_l);
    const long long copies = (long long)a.Hkv * a.row_blocks;
    // (Threads behind the last sequence have none, of a prefix neither.)
    auto len_at = [&](int b) { return PRE && b >= a.B ? 0 : pre.end + checked(a, read_length(a, b)); };
    const int len_mine = read_length(a, threadIdx.x);
    len_first = read_length(a, blockIdx.x);  // for fill_empty, after the first loads are under way
    int len = PRE && (int)threadIdx.x >= a.B ? 0 : pre.end + checked(a, len_mine);
    long long total, sum;
    long long ahead = scan_before(cost_of(len), s_warp, total);
    const long long first = total;
    int longest = len;
    for (int b0 = kThreads; b0 < a.B; b0 += kThreads) {
      const int more = len_at(b0 + threadIdx.x);
      longest = max(longest, more);
      scan_before(cost_of(more), s_warp, sum);
      total += sum;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) s_longest[warp] = longest;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) longest = max(longest, s_longest[w]);
    total *= copies;
    // One run for every CTA that the SMs hold at a time: more and shorter runs cost
    // more to start than they even out (ragged batch 106 us, with two to a slot 110).
    // Runs are not so short that a segment has more parts than a join takes at once.
    per = max(divide(total + gridDim.x - 1, gridDim.x), (long long)max(kLeastRun, tiles_of(longest) / kPartsAtOnce));
    const long long begin = per * blockIdx.x;
    int4* s_start = reinterpret_cast<int4*>(s_m);
    if (threadIdx.x == 0) s_start[0].x = -1;
    __syncthreads();
    long long before = 0;
    for (int b0 = 0; b0 < a.B && before <= begin; b0 += kThreads) {
      sum = first;
      if (b0 > 0) {
        len = len_at(b0 + threadIdx.x);
        ahead = scan_before(cost_of(len), s_warp, sum);
      }
      const int cost = cost_of(len);
      const long long rest = begin - before - copies * ahead;
      if (rest >= 0 && rest < copies * cost) {
        const long long copy = divide(rest, cost);
        s_start[0] = make_int4(b0 + threadIdx.x, len, (int)copy, (int)(rest - copy * cost));
      }
      before += copies * sum;
    }
    __syncthreads();
    const int4 st = s_start[0];
    __syncthreads();
    if (!a.by_segment && threadIdx.x == 0) a.chains[blockIdx.x] = Chain{0, 0, 0, 0};
    if (st.x < 0) {  // more CTAs than runs
      fill_empty<D, MODE>(a, len_first, pre.end);
      if (behind) griddep_wait();
      return;
    }
    sg.b = st.x;
    sg.len = st.y;
    sg.h = st.z / a.row_blocks;
    sg.rb = st.z % a.row_blocks;
    sg.left = min(per, total - begin);
    sg.len_next = read_length(a, sg.b + 1);
    sg.take(st.w);
    if (sg.tb == sg.ta) {  // the run ends before the segment's first tile
      fill_empty<D, MODE>(a, len_first, pre.end);
      if (behind) griddep_wait();
      return;
    }
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
  int ids_b = -1, ids_ta = 0, ids_n = 0;  // what they were read for
  auto look_up = [&]() {
    ld_base = ld_k;
    ids_b = lw.b, ids_ta = lw.ta, ids_n = ld_n;
    id0 = id1 = -1;
    const long long pos = ((long long)lw.ta + warp + (long long)kWarps * (ld_k + lane)) * kTile;
    if (ld_k + lane < ld_n) {
      const bool in_prefix = PRE && pos < pre.end;
      const int* row = in_prefix ? a.pre_table : a.table + (size_t)lw.b * a.max_blocks;
      const long long at = PRE && !in_prefix ? pos - pre.end : pos;
      const bool second = in_prefix ? pos + 16 < pre.len : pos + 16 < lw.len;
      id0 = __ldcg(row + (at >> a.page_shift));
      id1 = second ? __ldcg(row + ((at + 16) >> a.page_shift)) : -1;
      const bool fine0 = id0 >= 0 && id0 < a.P, fine1 = id1 >= 0 && id1 < a.P;
      if (!fine0 || (second && !fine1)) set_fail(ATTN_ERR_INVALID_ARG);
      if (!fine0) id0 = -1;
      if (!fine1) id1 = -1;
    }
  };
  auto issue = [&]() {
    if (!more) return;
    if (ld_k == ld_n) {
      do {
        more = lw.next(a);
        ld_n = more ? lw.count(warp) : 0;
      } while (more && ld_n == 0);
      if (!more) {
        if (!behind) griddep_launch_dependents();
        return;
      }
      ld_k = 0;
      // The next key head of a sequence has the same pages: the lanes may hold them.
      if (lw.b != ids_b || lw.ta != ids_ta || ld_base != 0 || ld_n > ids_n) look_up();
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
      // A page of 32 positions or more holds both halves.
      const uint32_t flags = a.page >= kTile ? (p0 >= 0 ? 3u : 0u) : (p0 >= 0 ? 1u : 0u) | (p1 >= 0 ? 2u : 0u);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(head + 16), "r"(flags) : "memory");
      if (a.page >= kTile) {
        mbar_arrive_expect_tx(bar, p0 >= 0 ? C::kStageBytes : 0);
        if (p0 >= 0) {
          const int pos = (lw.ta + warp + kWarps * ld_k) * kTile;
          const int in_page = (PRE && pos >= pre.end ? pos - pre.end : pos) & (a.page - 1);
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
      const int p = max(lane < 2 || a.page >= kTile ? p0 : p1, 0);
      copy4_arrive(head + 4 * lane, ((lane & 1) ? a.v_scale : a.k_scale) + (size_t)p * a.Hkv + lw.h, bar);
    }
    ++issued;
    ++ld_k;
  };
  const int rows_total = a.n_q * a.G;
  static_assert(NT <= kWarps, "a warp prepares one block of rows");
  uint2 w[D / 16];  // the segment's Q row 8 warp + g, as this lane prepares it
  auto load_q = [&]() {
    const int r = sg.rb * kRows + 8 * warp + g;
    const int t = token_of(a, r), hq = sg.h * a.G + (r - t * a.G);
    const uint16_t* src = a.q + sg.b * a.q_batch + t * a.q_token + hq * a.q_head;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      w[ks] = warp < NT && r < rows_total ? __ldcg(reinterpret_cast<const uint2*>(src + 16 * ks + 4 * c))
                                          : make_uint2(0u, 0u);
  };
  // Ahead of the first tiles: behind every CTA's these few bytes would wait for
  // tens of megabytes (3.5 us).  With 17 rows and more the registers are needed
  // elsewhere (64 sequences of 20 rows 153 us, 157 us with it).
  constexpr bool kAhead = NT <= 2;
  if (kAhead) load_q();
  if (more) look_up();
#pragma unroll 1
  for (int i = 0; i < C::kStages; ++i) issue();
  if (a.parts != nullptr) fill_empty<D, MODE>(a, len_first, pre.end);

  uint32_t used = 0;
  bool last_segment = false;
  while (!last_segment) {
    // ------------------------------------------------------------------ Q rows
    // Row r of the block: token (rb * rows + r) / G, head (rb * rows + r) % G of the
    // group.  K step ks of the products covers head dims [16 ks, 16 ks + 16), of
    // which a lane holds 4 c + {0, 1} as k = 2c, 2c + 1 and 4 c + {2, 3} as
    // k = 2c + 8, 2c + 9 (the same assignment as the codes') of rows 8 n + g.  Warp n
    // prepares block n for all; the merge's buffer holds the fragments meanwhile.
    if (!kAhead) load_q();
    if (warp < NT) {
      const int n = warp, r = sg.rb * kRows + 8 * n + g;
      const bool have = r < rows_total;
      const int t = token_of(a, r);
      float m = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        m = fmaxf(fmaxf(m, fmaxf(fabsf(__uint_as_float(w[ks].x << 16)), fabsf(__uint_as_float(w[ks].x & 0xFFFF0000u)))),
                  fmaxf(fabsf(__uint_as_float(w[ks].y << 16)), fabsf(__uint_as_float(w[ks].y & 0xFFFF0000u))));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // 2^e <= m < 2^(e+1), e within the range whose negative is a normal exponent.
      const int e = min(max((int)((__float_as_uint(m) >> 23) & 255u) - 127, -126), 126);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        s_q[(n * (D / 16) + ks) * 32 + lane] =
            make_uint2(pack_f16x2(__uint_as_float(w[ks].x << 16) * down, __uint_as_float(w[ks].x & 0xFFFF0000u) * down),
                       pack_f16x2(__uint_as_float(w[ks].y << 16) * down, __uint_as_float(w[ks].y & 0xFFFF0000u) * down));
      if (c == 0) {
        s_f[8 * n + g] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
        s_last[8 * n + g] = !have ? -1 : PRE ? max(sg.len - a.n_q + t, pre.end - 1) : sg.len - a.n_q + t;
      }
    }
    __syncthreads();
    // The scores and accumulators a lane holds are those of rows 8 n + 2 c + {0, 1}.
    // Factor of the scores of those, in base 2, and their last visible position (-1: none).
    auto f_row = [&](int n, int i) { return s_f[8 * n + 2 * c + i]; };
    auto my_last = [&](int n, int i) { return s_last[8 * n + 2 * c + i]; };
    const int tiles = sg.count(warp);

    // ------------------------------------------------------------------ tiles
    // Unit (lane / 16) of row lane % 16; unit u more is at this ^ (u << 4) for even u.
    const uint32_t lane_unit = unit_offset<D>(lane & 15, lane >> 4);
    float acc[D / 16][NT][4];  // head dims 16 u + 2 g + {0, 0, 1, 1}, rows 2 c + {0, 1, 0, 1}
#pragma unroll
    for (int u = 0; u < D / 16; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[u][n][x] = 0.f;
    float m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) m_run[n][i] = -INFINITY, l_run[n][i] = 0.f;
    // The accumulators' values times 2^-15 are relative to R, or, where wide, to 2^whole(s_w) of
    // their row (R is 2^15 then).  v_least: the smallest scale so far.
    float R = 0x1p-110f, v_least = FLT_MAX;
    bool wide = false;

    for (int k = 0; k < tiles && ok; ++k) {
      const uint32_t st = used % C::kStages;
      ok = warp_wait(&bars[st], (used / C::kStages) & 1);
      if (!ok) break;
      ++used;
      const uint32_t tile = ring + st * C::kStageBytes;
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
      // S^T = K Q^T for the tile's halves of 16 positions: of s[h][n], elements 0
      // and 1 are position g, 2 and 3 position g + 8.
      float s[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n) s[h][n][0] = s[h][n][1] = s[h][n][2] = s[h][n][3] = 0.f;
#pragma unroll
      for (int u = 0; u < D / 16; u += 2) {
        uint32_t r[2][4];  // positions 0-7 and 8-15 of unit u, then of unit u + 1
        ldsm4<0>(r[0], tile + (lane_unit ^ (u << 4)));
        ldsm4<16 * D>(r[1], tile + (lane_unit ^ (u << 4)));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint2 qf[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) qf[n] = s_q[(n * (D / 16) + u + x) * 32 + lane];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t b0 = r[h][2 * x] ^ 0x80808080u, b1 = r[h][2 * x + 1] ^ 0x80808080u;
            const uint32_t af[4] = {codes_f16(b0, 0x4140u), codes_f16(b1, 0x4140u), codes_f16(b0, 0x4342u),
                                    codes_f16(b1, 0x4342u)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(s[h][n], af, qf[n].x, qf[n].y);
          }
        }
      }
      // Scores in base 2; positions behind a row's last one are hidden.
      const int pos0 = (sg.ta + warp + kWarps * k) * kTile;
      const bool hide = pos0 + kTile - 1 > sg.len - a.n_q || flags != 3u ||
                        (PRE && pos0 < pre.end && pos0 + kTile > pre.len);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[h][n][x] *= f_row(n, x & 1) * ksc[h];
      if (hide) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
            {
              const int pos = pos0 + h * 16 + (x >> 1) * 8 + g;
              if (pos > my_last(n, x & 1) || !((flags >> h) & 1u) || (PRE && pos >= pre.len && pos < pre.end))
                s[h][n][x] = -INFINITY;
            }
        // A half that was not loaded has no weights: any scale will do.
        if (!(flags & 1u)) vsc[0] = flags != 0u ? vsc[1] : 0.f;
        if (!(flags & 2u)) vsc[1] = vsc[0];
      }
      // P in place of the scores.
      float back[NT][2];  // the accumulators' factors
      bool same = true;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = fmaxf(fmaxf(s[0][n][i], s[0][n][2 + i]), fmaxf(s[1][n][i], s[1][n][2 + i]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          mx = fmaxf(m_run[n][i], mx);
          const float m_use = mx == -INFINITY ? 0.f : mx;
          back[n][i] = ex2(m_run[n][i] - m_use);
          l_run[n][i] *= back[n][i];
          same = same && back[n][i] == 1.f;
          m_run[n][i] = mx;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              s[h][n][2 * y + i] = ex2(s[h][n][2 * y + i] - m_use);
              l_run[n][i] += s[h][n][2 * y + i];
            }
        }
      const float v_big = fmaxf(vsc[0], vsc[1]), v_small = fminf(vsc[0], vsc[1]);
      const bool other = v_big > R || v_small < v_least;  // always where wide
      if (!__all_sync(0xffffffffu, same && !other)) {
        float shrink = 1.f;
        if (other && !wide) {
          v_least = fminf(v_least, v_small);
          // The power of two at or above v_big.
          const float r_new = fmaxf(R, __uint_as_float((__float_as_uint(v_big) + 0x7FFFFFu) & 0x7F800000u));
          if (r_new > v_least * kNarrow || r_new > 0x1p126f) {
            wide = true;
            if (g == 0) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
                s_w[8 * n + 2 * c] = s_w[8 * n + 2 * c + 1] = (float)((int)(__float_as_uint(R) >> 23) - 127);
            }
            __syncwarp();
            R = 0x1p15f, v_least = INFINITY;
          } else {
            shrink = R / r_new;
            R = r_new;
          }
        }
        if (wide) {
          const float lv[2] = {__log2f(vsc[0]) + 0.5f, __log2f(vsc[1]) + 0.5f};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float w_old = s_w[8 * n + 2 * c + i];
              float w = fmaxf(w_old + __log2f(back[n][i]), kLeastWeight);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float p = fmaxf(s[h][n][i], s[h][n][2 + i]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) p = fmaxf(p, __shfl_xor_sync(0xffffffffu, p, off));
                w = fmaxf(w, __log2f(p) + lv[h]);
              }
              // At most 2^127 unless back is 0, and finite then too: a row that has seen nothing, or
              // nothing of a p above 2^-126, has no W to come from.
              back[n][i] *= ex2(fminf(whole(w_old) - whole(w), 127.f));
              const float up = exp2_whole<142, -1>(w);  // 2^(15 - W)
#pragma unroll
              for (int h = 0; h < 2; ++h) s[h][n][i] *= up, s[h][n][2 + i] *= up;
              __syncwarp();
              if (g == 0) s_w[8 * n + 2 * c + i] = w;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float s0 = back[n][0] * shrink, s1 = back[n][1] * shrink;
#pragma unroll
          for (int u = 0; u < D / 16; ++u) {
            acc[u][n][0] *= s0;
            acc[u][n][1] *= s1;
            acc[u][n][2] *= s0;
            acc[u][n][3] *= s1;
          }
        }
      }
      const float inv_r = __uint_as_float(0x86800000u - __float_as_uint(R));  // 2^15 / R
      const float vr[2] = {vsc[0] * inv_r, vsc[1] * inv_r};
      uint32_t pf[2][NT][2];  // P^T as the B operand of the halves
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            pf[h][n][y] = transpose8(pack_f16x2(s[h][n][2 * y] * vr[h], s[h][n][2 * y + 1] * vr[h]));
      // O^T += V^T P^T.  A transposed load gives positions 2c, 2c + 1 of the columns
      // d = 16 u + 2 g (even bytes) and + 1 (odd bytes), rows g and g + 8 of the
      // A operand.
#pragma unroll
      for (int u = 0; u < D / 16; u += 2) {
        uint32_t r[2][4];  // positions 0-7 and 8-15 of unit u, then of unit u + 1
        ldsm4_trans<C::kHalfBytes>(r[0], tile + (lane_unit ^ (u << 4)));
        ldsm4_trans<C::kHalfBytes + 16 * D>(r[1], tile + (lane_unit ^ (u << 4)));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t b0 = r[h][2 * x] ^ 0x80808080u, b1 = r[h][2 * x + 1] ^ 0x80808080u;
            const uint32_t af[4] = {codes_f16(b0, 0x4240u), codes_f16(b0, 0x4341u), codes_f16(b1, 0x4240u),
                                    codes_f16(b1, 0x4341u)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(acc[u + x][n], af, pf[h][n][0], pf[h][n][1]);
          }
      }
      __syncwarp();
      issue();
    }

    // ------------------------------------------------------------------ merge
    if (behind && !more) {
      griddep_wait();
      griddep_launch_dependents();
    }
    // In a cluster the part stays in shared memory, where the rings were.
    const bool whole = sg.ta == 0 && sg.tb == tiles_of(sg.len) && a.cluster <= 1;
    float* part = nullptr;
    if (a.cluster > 1)
      part = reinterpret_cast<float*>(smem);
    else if (!whole) part = a.parts + (size_t)(2 * blockIdx.x + (sg.ta == 0)) * part_floats(D, kRows);
    if (a.parts != nullptr && sg.ta == 0 && threadIdx.x == 0 && (a.by_segment || !whole)) {
      const int hr = sg.h * a.row_blocks + sg.rb;
      const long long slot = a.by_segment ? (long long)sg.b * a.Hkv * a.row_blocks + hr : blockIdx.x;
      // The segment runs on into as many CTAs as hold the rest of its tiles.
      const unsigned rest = tiles_of(sg.len) - sg.tb;
      const int more = rest == 0 ? 0 : 1 + (int)((rest - 1) / (unsigned)min(per, 0x7fffffffll));
      a.chains[slot] = Chain{more, sg.b, hr, (int)blockIdx.x};
    }
    float from[NT][2];  // what the accumulators are relative to
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) from[n][i] = wide ? exp2_whole<112, 1>(s_w[8 * n + 2 * c + i]) : R * 0x1p-15f;
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l_run[n][i] += __shfl_xor_sync(0xffffffffu, l_run[n][i], off);
        if (g == 0) {
          s_m[warp * kRows + 8 * n + 2 * c + i] = m_run[n][i];
          s_l[warp * kRows + 8 * n + 2 * c + i] = l_run[n][i];
        }
        l_run[n][i] = inverse(l_run[n][i]);
      }
#pragma unroll
    for (int at = 0; at < D; at += C::kMerge) {
      __syncthreads();  // the buffer holds Q, or the columns before, until here
      if (at == 0 && threadIdx.x < kRows) {  // the warps' shares of a row, in place of their sums
        const int r = threadIdx.x, rr = sg.rb * kRows + r;
        float M = -INFINITY, L = 0.f, share[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w * kRows + r]);
        const float M_use = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          share[w] = s_l[w * kRows + r] * ex2(s_m[w * kRows + r] - M_use);
          L += share[w];
        }
        const float inv = inverse(L);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s_l[w * kRows + r] = share[w] * inv;
        if (!whole) {
          part[kRows * D + r] = M;
          part[kRows * D + kRows + r] = L;
        } else if (rr < rows_total) {
          put_sums<D, MODE>(a, out_row(a, sg.b, sg.h, rr), M, L);
        }
      }
      // Pairs of columns, moved by four for every second row, so that the 16 lanes
      // of a phase cover all banks.
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * n + 2 * c + i;
#pragma unroll
          for (int u = 0; u < C::kMerge / 16; ++u)
            *reinterpret_cast<float2*>(s_merge + (warp * kRows + r) * C::kMerge + (((8 * u + g) ^ (c << 2)) << 1)) =
                make_float2(acc[at / 16 + u][n][i] * l_run[n][i] * from[n][i],
                            acc[at / 16 + u][n][2 + i] * l_run[n][i] * from[n][i]);
        }
      __syncthreads();
      // rows x columns over 128 threads, 4 columns at a time.
#pragma unroll 1
      for (int x = threadIdx.x; x < kRows * (C::kMerge / 4); x += kThreads) {
        const int r = x / (C::kMerge / 4), part4 = x % (C::kMerge / 4);
        float v[4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = s_l[w * kRows + r];
          const float4 y = *reinterpret_cast<const float4*>(
              s_merge + (w * kRows + r) * C::kMerge + (((2 * part4) ^ (((r >> 1) & 3) << 2)) << 1));
          v[0] += y.x * f, v[1] += y.y * f, v[2] += y.z * f, v[3] += y.w * f;
        }
        const int rr = sg.rb * kRows + r;
        if (!whole) {
          *reinterpret_cast<float4*>(part + r * D + at + part4 * 4) = make_float4(v[0], v[1], v[2], v[3]);
        } else if (rr < rows_total) {
          put_columns<D, MODE>(a, out_row(a, sg.b, sg.h, rr), at + part4 * 4, v[0], v[1], v[2], v[3]);
        }
      }
    }
    last_segment = !sg.next(a);
    if (kAhead && !last_segment) load_q();
    if (!last_segment) __syncthreads();  // before the next segment's Q
  }
  if (a.cluster > 1) {
    // Every CTA of the cluster joins the parts of its share of the rows and columns.
    const unsigned rank = blockIdx.x % a.cluster;
    const uint32_t mine = smem_u32(smem);
    cluster_sync();
    for (int x = rank * kThreads + threadIdx.x; x < kRows * (D / 4); x += a.cluster * kThreads) {
      const int r = x / (D / 4), col = x % (D / 4) * 4, rr = sg.rb * kRows + r;
      float m[kMaxCluster], l[kMaxCluster], M = -INFINITY, L = 0.f;
      float4 y[kMaxCluster], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (unsigned w = 0; w < kMaxCluster; ++w) {
        m[w] = -INFINITY, l[w] = 0.f, y[w] = v;
        if (w >= a.cluster) continue;
        const uint32_t at = peer(mine, w);
        m[w] = load_peer(at + 4 * (kRows * D + r));
        l[w] = load_peer(at + 4 * (kRows * D + kRows + r));
        y[w] = load_peer4(at + 4 * (r * D + col));
      }
#pragma unroll
      for (int w = 0; w < kMaxCluster; ++w) M = fmaxf(M, m[w]);
      const float M_use = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kMaxCluster; ++w) L += l[w] *= ex2(m[w] - M_use);
      const float inv = inverse(L);
#pragma unroll
      for (int w = 0; w < kMaxCluster; ++w) {
        const float f = l[w] * inv;
        v.x += f * y[w].x, v.y += f * y[w].y, v.z += f * y[w].z, v.w += f * y[w].w;
      }
      if (rr < rows_total) {
        const size_t row = out_row(a, sg.b, sg.h, rr);
        put_columns<D, MODE>(a, row, col, v.x, v.y, v.z, v.w);
        if (col == 0) put_sums<D, MODE>(a, row, M, L);
      }
    }
    cluster_sync();  // nobody leaves while its part is read
  }
  if (behind) griddep_wait();
  if (!ok) {
    if (lane == 0) set_fail(ATTN_ERR_TIMEOUT);
    // Do not leave while copies into this CTA's shared memory are in flight.
    for (; used < issued; ++used) mbar_wait(&bars[used % C::kStages], (used / C::kStages) & 1);
  }
}

// Joins the parts of the segments that begin in one CTA's run and end in
// another's: grid (chains, groups of rows).  Either a warp takes a row (SHARED false, where
// there are many chains of a few parts), or all of a CTA's warps share one and take its
// parts in turn (few chains of many).  The order of the sums is that of the parts.
template <int D, bool SHARED, int MODE>
__global__ void __launch_bounds__(32 * (SHARED ? kJoinShared : 8)) decode_join_kernel(const Args a, int rows) {
  constexpr int kJoinWarps = SHARED ? kJoinShared : 8, per_row = SHARED ? kJoinWarps : 1;
  __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int4 ch = __ldcg(reinterpret_cast<const int4*>(a.chains) + blockIdx.x);  // more, b, hr, cta
  if (ch.x == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * (kJoinWarps / per_row) + warp / per_row;
  const int rr = ch.z % a.row_blocks * rows + r;
  const bool have = r < rows && rr < a.n_q * a.G;
  const int n = have ? ch.x + 1 : 0;
  // O is kept as the mean of the parts so far, whose weights are at most 1.  kBatch parts
  // at a time, all their loads in flight together.
  constexpr int kBatch = kJoinBatch;
  float M = -INFINITY, L = 0.f, o[D / 32] = {};
  for (int i0 = warp % per_row; i0 < n; i0 += kBatch * per_row) {
    float m[kBatch], l[kBatch], x[kBatch][D / 32];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * per_row;
      m[k] = -INFINITY, l[k] = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) x[k][e] = 0.f;
      if (i < n) {
        const float* p = a.parts + (size_t)(2 * (ch.w + i) + (i == 0)) * part_floats(D, rows);
        m[k] = __ldcg(p + rows * D + r);
        l[k] = __ldcg(p + rows * D + rows + r);
        const float* q = p + r * D + lane * (D / 32);
        if constexpr (D == 128) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(q));
          x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(q));
          x[k][0] = v.x, x[k][1] = v.y;
        }
      }
    }
    float m_new = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) m_new = fmaxf(m_new, m[k]);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float before = L * ex2(M - m_use);
    M = m_new;
    L = before;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) L += l[k] *= ex2(m[k] - m_use);
    const float inv = inverse(L);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] *= before * inv;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] += l[k] * inv * x[k][e];
    }
  }
  if constexpr (SHARED) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e) s_o[warp][lane * (D / 32) + e] = o[e];
    if (lane == 0) s_m[warp] = M, s_l[warp] = L;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) M = fmaxf(M, s_m[w]);
    const float m_use = M == -INFINITY ? 0.f : M;
    L = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) L += s_l[w] * ex2(s_m[w] - m_use);
    const float inv = inverse(L);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = s_l[w] * ex2(s_m[w] - m_use) * inv;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] += f * s_o[w][lane * (D / 32) + e];
    }
  }
  if (!have) return;
  const size_t row = out_row(a, ch.y, ch.z / a.row_blocks, rr);
  const int col = lane * (D / 32);
  if constexpr (D == 128)
    put_columns<D, MODE>(a, row, col, o[0], o[1], o[2], o[3]);
  else if constexpr (MODE == kBehind)
    *reinterpret_cast<float2*>(a.whole + row * D + col) = make_float2(o[0], o[1]);
  else
    *reinterpret_cast<uint32_t*>(a.o + row * D + col) = pack_bf16x2(o[0], o[1]);
  if (lane == 0) put_sums<D, MODE>(a, row, M, L);
}

// Runs the tiles are dealt in: the CTAs that the SMs hold at a time.  (The full
// device's SM count where there is no device to ask, for workspace sizes.)
unsigned decode_runs(int d, int nt) {
  const int sms = device_sm_count();
  return (unsigned)(ctas_per_sm(d, nt) * (sms > 0 ? sms : 152));
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

template <int D, int NT, int MODE>
cudaError_t launch_impl(const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, unsigned runs,
                        cudaStream_t stream) {
  using C = Cfg<D, NT>;
  auto kernel = decode_int8_kernel<D, NT, MODE>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_smem(kernel, C::kSmemBytes, allowed);
  if (err != cudaSuccess) return err;
  const long long segments = (long long)a.B * a.Hkv * a.row_blocks;
  if (a.parts == nullptr)
    return launch_pdl_cluster(kernel, dim3((unsigned)(segments * a.cluster)), dim3(kThreads), C::kSmemBytes, stream,
                      a.cluster, mk, mv, a);
  err = launch_pdl(kernel, dim3(runs), dim3(kThreads), C::kSmemBytes, stream, mk, mv, a);
  if (err != cudaSuccess) return err;
  const bool shared = segments * 4 <= runs;
  const int rows = std::min(C::kRows, a.n_q * a.G);
  const unsigned chains = a.by_segment ? (unsigned)segments : runs;
  if (shared)
    return launch_pdl(decode_join_kernel<D, true, MODE>, dim3(chains, rows), dim3(32 * kJoinShared), 0, stream, a, C::kRows);
  return launch_pdl(decode_join_kernel<D, false, MODE>, dim3(chains, ceil_div(rows, 8)), dim3(256), 0, stream, a, C::kRows);
}


// Blocks of 8 rows a pass takes, and passes: as few passes as possible, then as
// few blocks.
int row_passes(int rows) { return ceil_div(rows, 32); }
int row_tiles(int rows) { return ceil_div(rows, 8 * row_passes(rows)); }

}  // namespace

// Clusters of `size` CTAs that the device holds at a time (the GPCs' SMs do not divide by
// every size).
template <int D, int NT, int MODE>
int clusters_held(int size) {
  using C = Cfg<D, NT>;
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];  // and one
  static std::atomic<uint64_t> allowed{0};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kDevices && (n = known[dev][size].load(std::memory_order_relaxed)) > 0) return n - 1;
  auto kernel = decode_int8_kernel<D, NT, MODE>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)size, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (allow_smem(kernel, C::kSmemBytes, allowed) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < kDevices) known[dev][size].store(n + 1, std::memory_order_relaxed);
  return n;
}

int clusters_held(int d, int nt, int size, Mode mode) {
#define ATTN_DECODE_CASE(DD, TT) \
  if (d == DD && nt == TT)                                               \
    return mode == kAlone        ? clusters_held<DD, TT, kAlone>(size)      \
           : mode == kWithPrefix ? clusters_held<DD, TT, kWithPrefix>(size) \
                                 : clusters_held<DD, TT, kBehind>(size);
  ATTN_DECODE_CASE(64, 1)
  ATTN_DECODE_CASE(64, 2)
  ATTN_DECODE_CASE(64, 3)
  ATTN_DECODE_CASE(64, 4)
  ATTN_DECODE_CASE(128, 1)
  ATTN_DECODE_CASE(128, 2)
  ATTN_DECODE_CASE(128, 3)
  ATTN_DECODE_CASE(128, 4)
#undef ATTN_DECODE_CASE
  return 0;
}

bool splits(const PagedCache& c) { return (long long)c.max_blocks * c.page > (long long)kWholeTiles * kTile; }

// CTAs that share a segment through their shared memory, or 0 where its tiles are dealt
// in runs instead.  The cluster saves the join (25 sequences of 1024 to 1850 positions, 4
// key heads of 128: 16.5 -> 13.4 us; one of 2000, 8 heads: 8.4 -> 7.3), the runs use all CTAs
// and even out ragged lengths.  By the longest sequences that the table has room for: a
// share against the run if the lengths were half of that.
int cluster_size(const PagedCache& c, int n_q, int H, Mode mode) {
  const int rows = n_q * (H / c.Hkv), nt = row_tiles(rows);
  const long long tiles = (long long)c.max_blocks * c.page / kTile;
  const long long segments = (long long)c.B * c.Hkv * row_passes(rows), runs = decode_runs(c.d, nt);
  if (tiles <= kLoneTiles) return 0;  // (250 positions 5.9 us, 6.5 in clusters; 500 7.8 and 5.9)
  for (long long size = std::min({runs / segments, (long long)kMaxCluster, tiles / 4}); size >= 2; --size) {
    if (tiles / size - tiles * segments / (2 * runs) > kClusterTiles) return 0;
    if (clusters_held(c.d, nt, (int)size, mode) >= segments) return (int)size;
  }
  return 0;
}

size_t decode_workspace_bytes(const PagedCache& c, int n_q, int H) {
  if (!splits(c)) return 0;
  const int rows = n_q * (H / c.Hkv), nt = row_tiles(rows);
  const size_t runs = decode_runs(c.d, nt);
  return align256(runs * 2 * part_floats(c.d, 8 * nt) * sizeof(float)) + runs * sizeof(Chain);
}

namespace {

// The cache as the choice of how to split the work has it: with room for the prefix in every row of the table.
PagedCache with_prefix(const PagedCache& c, int pre_blocks) {
  PagedCache room = c;
  room.max_blocks += pre_blocks;
  return room;
}

cudaError_t launch_any(const PagedCache& c, const void* q, const long long* strides, const int* pre_table,
                       int pre_blocks, const int* pre_len, const int* lens, void* o, float* lse, int n_q, int H,
                       float scale, void* workspace, cudaStream_t stream, float* whole) {
  const Mode mode = pre_blocks > 0 ? kWithPrefix : whole != nullptr ? kBehind : kAlone;
  const PagedCache room = with_prefix(c, pre_blocks);
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
  a.pre_table = pre_table, a.pre_len = pre_len, a.pre_blocks = pre_blocks;
  a.whole = whole;
  a.whole_rows = (size_t)c.B * n_q * H;
  a.B = c.B, a.n_q = n_q, a.H = H, a.Hkv = c.Hkv, a.G = H / c.Hkv, a.P = c.P, a.page = c.page;
  a.by_G = (uint32_t)(((1ull << 32) + a.G - 1) / a.G);
  a.page_shift = page_shift(c.page);
  a.max_blocks = c.max_blocks;
  a.row_blocks = row_passes(n_q * a.G);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.parts = nullptr;
  a.chains = nullptr;
  const int nt = row_tiles(n_q * a.G);
  a.by_segment = 0;
  unsigned runs = 0;
  a.cluster = cluster_size(room, n_q, H, mode);
  // Whole segments also where a join follows anyway and half of the slots or more have one, if they are not too long: a
  // launch less.  That is for calls made one by one, where the host's launches count; replayed as a graph, even runs are
  // worth up to 3% where the segments are ragged and more than the slots.  (48 sequences of 30 to 800 positions behind
  // 9001, 12 key heads of 64, in all: 27.0 us, split 28.0; 24 of 9 to 400, 20 rows, 34.3 and 34.4; 64 of 20 to 1500, 8 key
  // heads of 128, 512 segments for 456 slots: 50.6 and 54.7, as a graph 49.6 and 48.0; 256 of 50 to 1000 157 and 157.)
  const bool many = mode == kBehind && 2ll * a.B * a.Hkv * a.row_blocks >= decode_runs(c.d, nt) &&
                    (long long)c.max_blocks * c.page <= kWholeMany;
  if (a.cluster == 0 && (many || !splits(room))) a.cluster = 1;
  if (a.cluster == 0) {
    runs = decode_runs(c.d, nt);
    a.by_segment = (long long)a.B * a.Hkv * a.row_blocks <= runs;
    a.parts = static_cast<float*>(workspace);
    a.chains = reinterpret_cast<Chain*>(static_cast<char*>(workspace) +
                                        align256((size_t)runs * 2 * part_floats(c.d, 8 * nt) * sizeof(float)));
  }
  CUtensorMap mk, mv;
  if (!make_tmap_codes(&mk, c.k, c) || !make_tmap_codes(&mv, c.v, c)) return cudaErrorInvalidValue;
#define ATTN_DECODE_CASE(DD, TT)                                                       \
  if (c.d == DD && nt == TT)                                                            \
    return mode == kAlone        ? launch_impl<DD, TT, kAlone>(mk, mv, a, runs, stream)      \
           : mode == kWithPrefix ? launch_impl<DD, TT, kWithPrefix>(mk, mv, a, runs, stream) \
                                 : launch_impl<DD, TT, kBehind>(mk, mv, a, runs, stream);
  ATTN_DECODE_CASE(64, 1)
  ATTN_DECODE_CASE(64, 2)
  ATTN_DECODE_CASE(64, 3)
  ATTN_DECODE_CASE(64, 4)
  ATTN_DECODE_CASE(128, 1)
  ATTN_DECODE_CASE(128, 2)
  ATTN_DECODE_CASE(128, 3)
  ATTN_DECODE_CASE(128, 4)
#undef ATTN_DECODE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode_int8(const PagedCache& c, const void* q, const long long* strides, const int* lens,
                               void* o, float* lse, int n_q, int H, float scale, void* workspace,
                               cudaStream_t stream, float* whole) {
  return launch_any(c, q, strides, nullptr, 0, nullptr, lens, o, lse, n_q, H, scale, workspace, stream, whole);
}

size_t decode_prefix_workspace_bytes(const PagedCache& c, int n_q, int H, int pre_blocks) {
  return decode_workspace_bytes(with_prefix(c, pre_blocks), n_q, H);
}

cudaError_t launch_decode_prefix_int8(const PagedCache& c, const void* q, const long long* strides,
                                      const int* pre_table, int pre_blocks, const int* pre_len, const int* lens,
                                      void* o, float* lse, int n_q, int H, float scale, void* workspace,
                                      cudaStream_t stream) {
  return launch_any(c, q, strides, pre_table, pre_blocks, pre_len, lens, o, lse, n_q, H, scale, workspace, stream,
                    nullptr);
}

cudaError_t status_word_decode(void** word) { return cudaGetSymbolAddress(word, g_status_decode); }

}  // namespace attn

// Attention of each sequence's newest tokens over the paged INT8 cache, where all
// sequences of the batch share a prefix that is stored once.
//
// For query token i of n_q of sequence b and head h of group h / G, over the L positions
// of the prefix and the sequence's own positions j <= len - n_q + i:
//   s_j = scale * q . (ck_j * ks_j),   O = sum_j softmax(s)_j (cv_j * vs_j),   LSE = ln sum_j exp(s_j)
// with codes ck, cv and the scales ks, vs of position j's page and key head.  Prefix and own
// part are each reduced to (m, l, O / l), m the largest score, l the sum of exp(s - m), and joined as
//   m = max m_x,   l = sum_x l_x e^(m_x - m),   O = sum_x (l_x e^(m_x - m) / l) (O / l)_x,
// means with weights of at most 1.  Three launches: the prefix, the own positions, the join.  The own part is
// attn_decode_int8's kernel (decode_int8.cu), or with many new tokens this file's (own_by_units); a short prefix of
// few sequences is read once for each of them by attn_decode_int8's kernel, in one launch (reads_by_sequence).
//
// The rows of a key head over the prefix are those of all sequences, tokens and heads of
// the group, R = B n_q G, so the prefix's codes are read once for 256 of them instead of once a
// sequence, and the products have the rows of a tile of tcgen05.mma: S = Q K^T and O += P V of
// 128 rows by 128 positions, accumulators in TMEM.  A CTA (one per SM) has two row tiles that
// share each tile of keys; with up to 128 rows it has one, and its two halves take the
// even and the odd key tiles of it.  Roles of the warps:
//   copies (1 warp)    asks for the codes of the pages (bulk copies to a ring in shared memory) and
//                      for their scales
//   codes (8 warps)    codes of K and of V to FP16, from the ring to swizzled tiles
//   products (1 warp)  issues them
//   softmax (8 warps)  a thread for each row of the two tiles (or halves); also their Q rows and the
//                      results' way out
// What bounds it (d = 128).  A key tile of two row tiles takes 1.7 us (3450 clocks): the softmax of a row tile, 1850
// clocks of eight warps that fill the issue slots by turns, the P V and S that follow it, 1280, and 300 until the
// other side sees that they are done, while the tensor pipe needs 2048 for both row tiles' products, 2560 with their
// operands from shared memory.  1024 rows of 8 key heads over 32768 positions take 105 us, 1.31 PFLOP/s, 68% of what
// a library product reaches; 6400 rows over 12000 229 us, 1.37.  With one row tile the halves' chains run beside one
// another at 1.3 us a key tile: 16 rows of 8 key heads over 100003 positions 54 us, 3.8 TB/s, 56% of the copy rate.
// Shared memory alone asks for 0.87 us of those: the codes in and out, K and V in FP16 in and out, Q: 224 KB.
// Around the tiles are about 10 us: launch, Q and the first tile's chain of loads, the last tile's, the part of a run
// (133 KB, FP32); 256 rows over 16000 positions are 6.6 tiles a CTA and 21 us.
// Loads to registers are avoided where much is in flight: shared memory leaves L1 28 KB, and codes that
// were loaded through it kept the warps that ask for them waiting (a key tile took 3.9 us).
// The tiles of all (key head, row block) units, one behind the other, are dealt to the CTAs
// in equal runs; every run leaves a part (m, l, O / l) of each unit it meets in the workspace.
//
// Numerics, as in decode_int8.cu: codes are exact in FP16; Q becomes FP16 after division by a
// power of two of its row's maximum (exact down to 2^-17 of it); the weights p vs of the
// values' codes are FP16 relative to a row's own W, by which its largest weight so far is 2^6 or more
// (kTop), so that they keep 11 bits down to 2^-20 of it.  W and the maximum that the row sum is relative to
// follow the running maxima of s + log2(vs) and of s only when the weights would grow too large: the
// accumulators in TMEM are rescaled then, by the softmax's threads.  Sums and statistics are FP32.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {

static __device__ unsigned int g_status_shared;

namespace {

// Warps 0 to 7 softmax, 8 to 11 K's codes, 12 to 15 V's, 16 copies, 17 products (and two that have nothing
// to do: a warpgroup has four).
constexpr int kSoftmaxWarps = 8, kCodeWarps = 4, kCopyWarp = 16, kMmaWarp = 17;
constexpr int kThreads = 32 * 20;
// Registers a thread at launch (five warps a quarter of an SM), and of the warpgroups of each kind.
constexpr int kRegsLaunch = 96, kRegsSoftmax = 160, kRegsCodes = 48, kRegsMma = 64;
static_assert(2 * kRegsSoftmax + 2 * kRegsCodes + kRegsMma <= 5 * kRegsLaunch,
              "setmaxnreg split exceeds the launch pool");
static_assert(kRegsMma <= kRegsLaunch && kRegsCodes <= kRegsLaunch && kRegsSoftmax >= kRegsLaunch,
              "setmaxnreg directions");
constexpr int kUnitRows = 256;  // rows of a unit: two tiles
// Cost of a key tile where the unit has two row tiles, and where it has one.
constexpr int kCostTwo = 3, kCostOne = 2;
constexpr int kLeastRun = 2;  // key tiles of a run at least
// The largest weight of a row just after its reference W moved is 2^kTop, so the 128 weights of a tile sum to
// 2^(kTop + 7) or less; W moves again when a tile's could sum to more than kMost, which FP16 still holds.
constexpr float kTop = 6.f, kMost = 65000.f;
constexpr float kLeastScale = -104.f;  // log2 of the least value scale whose weights reach 2^kTop
constexpr float kMostSum = 0x1p40f;  // of a tile's weights relative to the row's m
// A row's m moves to its maximum less kLow.  Its W lies above s + log2(vs) - kTop of all positions, so 2^(m - W) vs stays
// below 2^(kTop + 126 - kLow), which FP32 holds, for every position whose weight in the row's sum, e^(s - max), is a
// normal number, whatever the ratio of the value scales.  (Those below count as 0.)  And W is at most that of the largest
// vs, so 2^(m - W) is above 2^(kTop - kLow - 128), which FP32 holds too.
constexpr float kLow = kTop - 2.f, kLowFactor = 1.f / 16;
static_assert(kLow == 4.f, "kLowFactor is 2^-kLow");
constexpr float kMostFloat = 0x1.fffffep127f;

__device__ __forceinline__ void set_fail(unsigned int code) { atomicOr(&g_status_shared, code); }

struct Args {
  const uint16_t* q;
  long long q_batch, q_token, q_head;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int *table, *len;  // of the prefix; or [B][blocks] and [B], of the own positions
  int B, n_q, H, Hkv, G, P, page_shift, blocks;
  int rows, row_blocks, runs;
  float scale_log2;
  int* starts;  // [runs + 1]: each run's first tile, and the key tiles of the prefix
  float* parts;
  float* own;  // O / l [B n_q H][D], m [B n_q H], l [B n_q H] of the own parts
  uint16_t* o;
  float* lse;
};

// A part: O / l as [D / 4][256 rows][4], m [256], l [256].
__host__ __device__ constexpr size_t part_floats(int d) { return (size_t)kUnitRows * (d + 2); }

// x / y, in 32 bits where they suffice.
__device__ __forceinline__ long long divide(long long x, int y) {
  return x <= 0xffffffffll ? (long long)((unsigned)x / (unsigned)y) : x / y;
}

// How the key tiles of all units (unit = key head * row_blocks + row block) are dealt to the runs.  Tiles of
// all units together are below 2^31 (the host's check), and cost kCostTwo, or kCostOne in a head's last
// unit where that has one row tile.  First tile (unit * tiles + key tile) of run c:
__device__ __forceinline__ int run_begin(const Args& a, int tiles, int c) {
  const int before = tiles * (a.row_blocks - 1);  // tiles of a head before its last unit
  const int last_cost = a.rows - (a.row_blocks - 1) * kUnitRows <= kBlockM ? kCostOne : kCostTwo;
  if (a.row_blocks == 1 || last_cost == kCostTwo) {  // all cost the same
    const int units = a.row_blocks * a.Hkv, all = tiles * units;
    int runs = min(a.runs, max(all / kLeastRun, 1));
    // As many for each unit where that makes no run longer by more than a tile: a run that meets two units pays
    // for their rows' way in and out twice (16 units of 40 tiles 23 us, 19 with 9 runs each).  No more of them than
    // the longest asks for: SMs without one take the own positions meanwhile (64 sequences behind 16000 positions
    // 53.3 us in all with 19 runs a unit, 50.3 with 18).
    const int each = runs / units;
    if (each > 0) {
      const int most = (tiles + each - 1) / each;
      if (most <= all / runs + 1) runs = max((tiles + most - 1) / max(most, 1), 1) * units;
    }
    return c >= runs ? all : (int)divide((long long)all * c, runs);
  }
  if (tiles == 0) return 0;
  const long long head_cost = (long long)before * kCostTwo + (long long)tiles * last_cost, all = head_cost * a.Hkv;
  // The same with two costs: the least most that a run takes for which there are runs enough (280 rows of two key heads
  // over 30000 positions 33.8 us in all, 32.9 so).
  if (a.row_blocks * a.Hkv <= a.runs && all <= INT_MAX) {
    const unsigned n = tiles, even = max((unsigned)all / a.runs + 1, (unsigned)(kLeastRun * kCostTwo));
#pragma unroll 1
    for (unsigned most = even; most <= even + kCostTwo; ++most) {
      const unsigned full = a.row_blocks - 1, of_full = (n - 1) / (most / kCostTwo) + 1;
      const unsigned of_head = full * of_full + (n - 1) / (most / kCostOne) + 1;
      if (of_head * a.Hkv > (unsigned)a.runs) continue;
      const unsigned h = c / of_head, x = c - h * of_head, u = min(x / of_full, full), i = x - u * of_full;
      if (h >= (unsigned)a.Hkv) return tiles * a.row_blocks * a.Hkv;
      return (h * a.row_blocks + u) * n + n * i / (u < full ? of_full : of_head - full * of_full);
    }
  }
  const int runs = (int)max(1ll, min((long long)a.runs, all / (kLeastRun * kCostTwo)));
  if (c >= runs) return tiles * a.row_blocks * a.Hkv;
  const long long x = divide(all * c, runs), h = x / head_cost, y = x - h * head_cost;
  const long long full = (long long)before * kCostTwo;
  return (int)(h * a.row_blocks * tiles + (y < full ? y / kCostTwo : before + (y - full) / last_cost));
}

// A length as it is used; one that the table has no room for is cut and reported.
__device__ __forceinline__ int checked_length(const Args& a, int len, bool report) {
  const long long cap = (long long)a.blocks << a.page_shift;
  if (len >= 0 && len <= cap) return len;
  if (report) set_fail(ATTN_ERR_INVALID_ARG);
  return len < 0 ? 0 : (int)cap;
}

// What a CTA does, as every role goes through it: key tiles [k0, k0 + nk) for rows of block rb of key head h.
// OWN false: its run over the prefix, `left` tiles behind these.  OWN true: every gridDim.x-th (sequence, key
// head, row block) over the sequence's own positions, of which there may be none.
template <bool OWN>
struct Walk {
  int b, h, rb, k0, nk, len, left, tiles, start;
  __device__ __forceinline__ Walk(const Args& a, bool none) : b(0), nk(0) {
    if constexpr (OWN) {
      k0 = tiles = start = len = 0;
      left = none ? INT_MAX : (int)blockIdx.x;
      return;
    }
    len = __shfl_sync(0xffffffffu, checked_length(a, __ldcg(a.len), threadIdx.x == 0 && blockIdx.x == 0), 0);
    tiles = none ? 0 : (len + kBlockN - 1) / kBlockN;
    // Lane 1 finds where the next run begins.
    const int at = run_begin(a, tiles, blockIdx.x + (threadIdx.x & 1));
    start = __shfl_sync(0xffffffffu, at, 0);
    left = __shfl_sync(0xffffffffu, at, 1) - start;
    const int unit = (unsigned)start / (unsigned)max(tiles, 1);
    h = a.row_blocks == 1 ? unit : unit / a.row_blocks;
    rb = unit - h * a.row_blocks;
    k0 = start - unit * tiles;
  }
  __device__ __forceinline__ bool next(const Args& a) {
    if constexpr (OWN) {
      const int copies = a.Hkv * a.row_blocks;
      b = left / copies;
      if (b >= a.B) return false;
      const int copy = left - b * copies;
      h = copy / a.row_blocks;
      rb = copy - h * a.row_blocks;
      len = __shfl_sync(0xffffffffu, checked_length(a, __ldcg(a.len + b), true), 0);
      nk = (len + kBlockN - 1) / kBlockN;
      left += gridDim.x;
      return true;
    }
    if (left == 0) return false;
    if (nk > 0) {
      k0 = 0;
      if (++rb == a.row_blocks) rb = 0, ++h;
    }
    nk = min(tiles - k0, left);
    left -= nk;
    return true;
  }
  // Two row tiles; else the key tiles alternate between the two halves of the CTA.
  __device__ __forceinline__ bool two(const Args& a) const { return OWN || a.rows - rb * kUnitRows > kBlockM; }
};

// Scales of a key tile in groups of 16 positions, and how many of each are seen.
struct Head {
  float ks[8], vs[8];
  float v_most;  // the largest of vs
  uint8_t seen[8];
  int hidden;  // not all are seen
};

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 2 : 3;  // of K and of V tiles
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kRawBytes = 128 * D;  // K or V codes of a key tile
  // Key tiles in the ring of codes; one more where all units have one row tile and the second
  // one's Q has no need of its place.
  static constexpr int kRawTiles = D == 128 ? 1 : 4;
  // Key tiles whose scales are held.  Those of tile g are overwritten when the codes of tile g + kHeads -
  // kRawTiles - 2 have been read from the ring; then S of the tile kStages + 1 before that one is complete, and
  // the softmax is past the tile two before that.
  static constexpr int kHeads = D == 128 ? 8 : 16;
  static_assert(kHeads - (kRawTiles + 2) - (kStages + 1) - 2 >= 0, "scales stay until the softmax has used them");
  static constexpr int kOffQ = 0;
  static constexpr int kOffRaw = 2 * kTileBytes;
  static constexpr int kOffK = kOffRaw + 2 * kRawTiles * kRawBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffHead = kOffV + kStages * kTileBytes;
  static constexpr int kOffE = kOffHead + kHeads * (int)sizeof(Head);  // int8 [2][128]: exponent of a row's power of two
  static constexpr int kOffBar = (kOffE + 2 * 128 + 15) / 16 * 16;
  static constexpr int kSlots = 2 * (kRawTiles + 1);
  // raw_full, raw_empty [slots], k_full, k_empty, v_full, v_empty [stages], q [2], s_full [2], p_full [2], o_done [2], final
  static constexpr int kNumBars = 2 * kSlots + 4 * kStages + 9;
  static constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 16;
  static_assert(kTileBytes == 2 * kRawBytes, "the place of a Q tile holds a key tile's codes");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
  static constexpr uint32_t kTmemCols = 512;
  static __device__ __forceinline__ uint32_t col_s(int t) { return 128u * t; }
  static __device__ __forceinline__ uint32_t col_o(int t) { return 256u + D * t; }
};

// Instruction descriptor for kind::f16 with FP16 A and B, FP32 D (fields as in idesc_bf16).
constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Codes 0 and 2 of four, or 1 and 3 of them shifted by a byte, as FP16: the byte c + 128 under the
// exponent of 1024 is 1152 + c.  (Q's elements are put in the same order, and O's come out of it.)
__device__ __forceinline__ uint32_t codes_f16(uint32_t u) {
  const uint32_t x = (u & 0x00FF00FFu) ^ 0x64806480u;
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64806480u));
  return r;
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 1 / L, or 0 where a row has seen nothing.  A NaN stays one.
__device__ __forceinline__ float inverse(float L) { return L == 0.f ? 0.f : 1.f / L; }
// l 2^x, x <= 0, of a part: m may lie far below its largest score where the value scales fall as the scores rise, and l be
// as much larger, so that 2^x alone could be 0 where the product counts.
__device__ __forceinline__ float share_of(float l, float x) {
  const float half = ex2(0.5f * x);
  return l * half * half;
}
// Sequence, token and head of row r of key head h's rows.
__device__ __forceinline__ void row_of(const Args& a, int r, int& b, int& t, int& g) {
  const int x = r / a.G;
  g = r - x * a.G;
  b = x / a.n_q;
  t = x - b * a.n_q;
}

// GROUP: positions that share a page's scales for certain (16, or 32 in pages of 32 and more).
template <int D, int GROUP, bool OWN>
__global__ void __launch_bounds__(kThreads, 1) shared_prefix_kernel(const Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // What decides where a warp goes comes from a shuffle, which tells the compiler that it is the same in
  // all lanes: the products' descriptors then stay in uniform registers.
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* bar_rfull = bars;
  uint64_t* bar_rempty = bar_rfull + C::kSlots;
  uint64_t* bar_kfull = bar_rempty + C::kSlots;
  uint64_t* bar_kempty = bar_kfull + C::kStages;
  uint64_t* bar_vfull = bar_kempty + C::kStages;
  uint64_t* bar_vempty = bar_vfull + C::kStages;
  uint64_t* bar_q = bar_vempty + C::kStages;
  uint64_t* bar_sfull = bar_q + 2;
  uint64_t* bar_pfull = bar_sfull + 2;
  uint64_t* bar_odone = bar_pfull + 2;
  uint64_t* bar_final = bar_odone + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  int8_t* s_e = reinterpret_cast<int8_t*>(smem + C::kOffE);
  Head* heads = reinterpret_cast<Head*>(smem + C::kOffHead);

  if (threadIdx.x == 0) {
    tmem_slot[1] = (smem_u32(smem) & 1023u) != 0;
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bar_rfull[s], 1);
      mbar_init(&bar_rempty[s], kCodeWarps);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar_kfull[s], kCodeWarps);
      mbar_init(&bar_kempty[s], 1);
      mbar_init(&bar_vfull[s], kCodeWarps);
      mbar_init(&bar_vempty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar_q[t], 4);
      mbar_init(&bar_sfull[t], 1);
      mbar_init(&bar_pfull[t], 4);
      mbar_init(&bar_odone[t], 1);
    }
    mbar_init(bar_final, 1);
    fence_mbar_init();
  }
  if (warp == kCopyWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // What comes before the call is complete when the prefix's kernel lets the own positions' in, which uses nothing of
  // it: that kernel waits for the prefix's when it lets the join in, which reads what both have left.
  // (PTX promises the grid that waits that it sees what came before.  That the grid which this one then lets in sees it
  // too, without a wait of its own, is an assumption: it was complete and in L2 before that grid began, which reads it from
  // there, by ld.cg and bulk copies.)
  if (!OWN) {
    griddep_wait();
    griddep_launch_dependents();
  }
  const bool abort_all = __any_sync(0xffffffffu, tmem_slot[1] != 0);
  if (threadIdx.x == 0 && abort_all) set_fail(ATTN_ERR_INVALID_ARG);
  Walk<OWN> sg(a, abort_all);
  if (!OWN && threadIdx.x == 32 * kCopyWarp) {
    a.starts[blockIdx.x] = sg.start;
    if (blockIdx.x == 0) a.starts[a.runs] = sg.tiles;
  }
  // All units have one row tile: one copy of Q, and a longer ring.
  const bool one = !OWN && a.rows <= kBlockM;
  const int slots = one ? 2 * (C::kRawTiles + 1) : 2 * C::kRawTiles;
  uint8_t* raw = smem + (one ? C::kTileBytes : C::kOffRaw);

  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;

  if (warp >= kCopyWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == kCopyWarp) {
      // ------------------------------------------------------------ copies
      // Key tiles by fours: lane x has the page of group x % 8 (16 positions) of the x / 8-th tile, and its
      // scales.  Pages are read two fours ahead, scales one: both take as long as a tile.
      const int group = lane & 7;
      const int page_mask = (1 << a.page_shift) - 1;
      bool ok = true;
      // The page of a group: one whose first position is seen, as a whole, or -1.
      auto first_at = [&](int tile) {
        return (((long long)tile + (lane >> 3)) * kBlockN + 16 * group) & ~(long long)page_mask;
      };
      auto pages_at = [&](int tile) {
        const long long pos = first_at(tile);
        return pos < sg.len ? __ldcg(a.table + (size_t)sg.b * a.blocks + (pos >> a.page_shift)) : -1;
      };
      auto checked = [&](int tile, int id) {
        if (first_at(tile) < sg.len && (id < 0 || id >= a.P)) {
          set_fail(ATTN_ERR_INVALID_ARG);
          return -1;
        }
        return id;
      };
      int g = 0, slot = 0;
      unsigned use = 0;  // rounds of the ring so far
      while (ok && sg.next(a)) {
        // (Where there is no page, page 0's, which is not used.)
        auto scale_at = [&](const float* scales, int id) { return __ldcg(scales + (max(id, 0) * a.Hkv + sg.h)); };
        int ids = checked(sg.k0, pages_at(sg.k0)), ids_next = pages_at(sg.k0 + 4);
        float ks = scale_at(a.k_scale, ids), vs = scale_at(a.v_scale, ids);
        for (int e0 = 0; e0 < sg.nk && ok; e0 += 4) {
          const int ids_after = pages_at(sg.k0 + e0 + 8);
          ids_next = checked(sg.k0 + e0 + 4, ids_next);
          const float ks_next = scale_at(a.k_scale, ids_next), vs_next = scale_at(a.v_scale, ids_next);
          for (int e = e0; e < min(e0 + 4, sg.nk); ++e, ++g) {
            const int lanes = (e - e0) * 8;  // those of the tile
            const int id = __shfl_sync(0xffffffffu, ids, lanes + group);
            const unsigned loaded = __ballot_sync(0xffffffffu, lane < 8 && id >= 0);
            const int seen = id >= 0 ? max(0, min(16, sg.len - ((sg.k0 + e) * kBlockN + 16 * group))) : 0;
            const bool hidden = __any_sync(0xffffffffu, seen < 16);
            // Positions without a page are hidden, and their scale is 0: another page's must decide nothing.
            float k = __shfl_sync(0xffffffffu, ks, lanes + group), v = __shfl_sync(0xffffffffu, vs, lanes + group);
            if (id < 0) k = v = 0.f;
            const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
            // The scales' slot: its last tile, kHeads before, has been through the softmax.  (The ring's place for
            // the tile before was free, so the products S of the tile that many tiles and stages ago are complete.)
            // Whoever waits for the codes, or for what follows from them, sees these.
            Head& hd = heads[g % C::kHeads];
            if (lane < 8) {
              hd.ks[group] = k;
              hd.vs[group] = v;
              hd.seen[group] = (uint8_t)seen;
            }
            if (lane == 0) hd.v_most = most, hd.hidden = hidden;
            __syncwarp();
            // K, then V: a copy a page.  Where there is none the ring's bytes are codes as well, of positions that
            // are hidden.  With two row tiles and a ring of one key tile K's codes are not taken before V's of the
            // tile before have been: the products want V first, and the two conversions slow each other (6400
            // rows of 8 key heads over 12000 positions: 229 us, 242 as they come, 1024 over 32768: 105 and 107.5; with
            // one row tile it is 56 and 54).
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              if (use > 0) ok = warp_wait(&bar_rempty[slot], (use - 1) & 1);
              if (x == 1 && !one && lane == 0) mbar_arrive(&bar_rfull[slot - 1]);
              if (!ok) break;
              if (lane == 0) {
                const uint32_t bytes = __popc(loaded) * 16 * D;
                if (x == 1 || one) mbar_arrive_expect_tx(&bar_rfull[slot], bytes);
                else mbar_expect_tx(&bar_rfull[slot], bytes);
              }
              __syncwarp();
              if (lane < 8 && id >= 0 && ((16 * group) & page_mask) == 0)
                bulk_load(raw + slot * C::kRawBytes + group * 16 * D,
                          (x == 0 ? a.k : a.v) + (size_t)((id * a.Hkv + sg.h) << a.page_shift) * D,
                          min(page_mask + 1, kBlockN) * D, &bar_rfull[slot]);
              if (++slot == slots) slot = 0, ++use;
            }
            if (!ok) break;
          }
          ids = ids_next, ids_next = ids_after;
          ks = ks_next, vs = vs_next;
        }
      }
      if (!ok && lane == 0) set_fail(ATTN_ERR_TIMEOUT);
      // Do not leave while copies into this CTA's shared memory are in flight.
      for (int x = 0; x < slots; ++x) {
        const unsigned uses = use + (x < slot ? 1 : 0);
        if (uses > 0) mbar_wait(&bar_rfull[x], (uses - 1) & 1);
      }
      if (OWN) {
        griddep_wait();
        griddep_launch_dependents();
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ products
      constexpr uint32_t idesc_qk = idesc_f16(128, 128, false);
      constexpr uint32_t idesc_pv = idesc_f16(128, D, true);
      const uint64_t descQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t descK = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t descV = sdesc_sw128(smem_u32(sV), C::kChunkBytes, 1024);
      auto issue_s = [&](int t, int st) {
        const uint64_t a0 = sdesc_add(descQ, one ? 0 : t * C::kTileBytes);
        const uint64_t b0 = sdesc_add(descK, st * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
          mma_ss_elect(tmem + C::col_s(t), sdesc_add(a0, off), sdesc_add(b0, off), idesc_qk, kk > 0 ? 1u : 0u);
        }
        mma_commit_elect(&bar_sfull[t]);
      };
      auto issue_pv = [&](int t, int st, bool acc) {
        const uint64_t b0 = sdesc_add(descV, st * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < kBlockN / 16; ++kk)
          mma_ts_elect(tmem + C::col_o(t), tmem + C::col_s(t) + kk * 8, sdesc_add(b0, kk * 2048),
                       idesc_pv, (acc || kk > 0) ? 1u : 0u);
      };
      bool ok = true;
      int g = 0, items = 0;
      unsigned pc = 0;  // bit t: phase of P_t
      while (ok && sg.next(a)) {
        if (OWN && sg.nk == 0) continue;
        const bool two = sg.two(a);
        // S_t's columns are free: the P V products issued before read them first.
        ok = warp_wait(&bar_q[0], items & 1) && (one || warp_wait(&bar_q[1], items & 1));
        ++items;
        // Step e: P V of key tile e - lag, then S of key tile e, of both halves, or of the half whose turn it is.
        const int lag = two ? 1 : 2;
#pragma unroll 1
        for (int e = 0; e < sg.nk + lag && ok; ++e) {
          const int i = e - lag;  // the tile of P V
          const bool pv = i >= 0, qk = e < sg.nk;
          const int sv = pv ? (g + i) % C::kStages : 0, sk = (g + e) % C::kStages;
#pragma unroll 1
          for (int t = two ? 0 : e & 1; t < (two ? 2 : (e & 1) + 1) && ok; ++t) {
            const bool first = !two || t == 0;
            if (pv) {
              if (first) ok = warp_wait(&bar_vfull[sv], ((g + i) / C::kStages) & 1);
              ok = ok && warp_wait(&bar_pfull[t], (pc >> t) & 1);
              if (!ok) break;
              pc ^= 1u << t;
              tc_fence_after();
              issue_pv(t, sv, i >= lag);
              if (!qk) mma_commit_elect(&bar_odone[t]);
            }
            if (qk) {
              if (first) {
                ok = warp_wait(&bar_kfull[sk], ((g + e) / C::kStages) & 1);
                if (!ok) break;
                tc_fence_after();
              }
              issue_s(t, sk);
            }
          }
          if (!ok) break;
          if (pv) mma_commit_elect(&bar_vempty[sv]);
          if (qk) mma_commit_elect(&bar_kempty[sk]);
        }
        // A half without a key tile is told too: it waits for the segment's end before the next.
        if (ok && !two && sg.nk == 1) mma_commit_elect(&bar_odone[1]);
        g += sg.nk;
      }
      if (!ok && lane == 0) set_fail(ATTN_ERR_TIMEOUT);
      // Every product that was issued completes before TMEM is released.
      mma_commit_elect(bar_final);
      mbar_wait(bar_final, 0);
    }
    __syncwarp();
  } else if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCodes));
    // --------------------------------------------------------------- codes
    // A thread has one 16-byte unit of a row, kPasses rows of a tile.  The eight lanes of a phase have
    // 128 bytes of codes that meet all banks, and so do the units that they become: those of two rows
    // with units 0, 2, 4, 6 each, which the swizzle of an odd row moves to the odd places (d = 128: units of
    // the first chunk of one row and of the second of the other).
    constexpr int kUnits = D / 16, kRows = 128 / kUnits, kPasses = 128 / kRows;
    const int unit = lane % kUnits, pair = lane >> 3;
    const int kv = (warp - kSoftmaxWarps) / kCodeWarps;  // K or V
    const int row = warp % kCodeWarps * (kRows / 4) +
                    (D == 128 ? (pair >> 1) * 2 + ((unit >> 2) ^ (pair & 1)) : lane / kUnits);
    bool ok = true;
    const uint32_t from = smem_u32(raw) + row * D + unit * 16;
    const uint32_t to0 = (unit >> 2) * C::kChunkBytes + sw128_offset(row, (unit & 3) * 2);
    const uint32_t to1 = to0 ^ 16u;  // the odd unit beside it
    // A slot of the ring to the tile at `to`, which is free when `empty` has completed its phase.
    auto convert = [&](int slot, unsigned round, uint32_t to, uint64_t* empty, int phase) {
      if (!warp_wait(&bar_rfull[slot], round & 1)) return false;
      constexpr int kBatch = 4;
#pragma unroll
      for (int p0 = 0; p0 < kPasses; p0 += kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                       : "r"(from + slot * C::kRawBytes + (p0 + i) * kRows * D)
                       : "memory");
        }
        if (p0 == 0 && phase >= 0 && !warp_wait(empty, phase & 1)) return false;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const uint32_t at = to + (p0 + i) * kRows * 128;
          st_shared_v4(at + to0, codes_f16(w[i].x), codes_f16(w[i].x >> 8), codes_f16(w[i].y), codes_f16(w[i].y >> 8));
          st_shared_v4(at + to1, codes_f16(w[i].z), codes_f16(w[i].z >> 8), codes_f16(w[i].w), codes_f16(w[i].w >> 8));
        }
      }
      return true;
    };
    uint64_t* bar_full = kv == 0 ? bar_kfull : bar_vfull;  // the empty ones are behind them
    const uint32_t tiles = smem_u32(kv == 0 ? sK : sV);
    int slot = kv, st = 0;  // places in the ring and among the tiles
    unsigned round = 0, st_round = 0;
    while (ok && sg.next(a)) {
      for (int e = 0; e < sg.nk; ++e) {
        ok = convert(slot, round, tiles + st * C::kTileBytes, bar_full + C::kStages + st, (int)st_round - 1);
        if (!ok) break;
        // Only now: what was read from the ring has arrived where it has been used.  (An arrival right behind
        // the loads let copies overwrite codes that were still to be read.)
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_rempty[slot]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_full + st);
        if ((slot += 2) >= slots) slot = kv, ++round;
        if (++st == C::kStages) st = 0, ++st_round;
      }
    }
    if (!ok && lane == 0) set_fail(ATTN_ERR_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // -------------------------------------------------------------- softmax
    // A thread has a row of tile (or half) t: m_ref, kLow below its maximum when that last moved it, the sum of the
    // weights relative to it, and the reference W (in base 2) of the weights that are multiplied with the codes, and
    // so of the accumulators.
    const int t = warp >> 2, w0 = (warp & 3) * 32;
    const int r = w0 + lane;  // row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)w0 << 16;
    const uint32_t tS = tmem + lane_off + C::col_s(t);
    const uint32_t tO = tmem + lane_off + C::col_o(t);
    bool ok = true;
    int sc = 0, oc = 0;  // S tiles consumed, segments completed
    int g = 0, items = 0;  // key tiles and number of the segments before
    while (ok && sg.next(a)) {
      const bool two = sg.two(a);
      const int first = sg.rb * kUnitRows + (two ? t * kBlockM : 0);  // the tile's first row
      const int have = min(kBlockM, a.rows - first);                  // and how many it has
      // This thread's row: its sequence, token and head of the group.
      int b, tok, gg;
      row_of(a, max(min(first + r, a.rows - 1), 0), b, tok, gg);
      if (OWN) b = sg.b;
      const size_t own_row = ((size_t)b * a.n_q + tok) * a.H + sg.h * a.G + gg, own_rows = (size_t)a.B * a.n_q * a.H;
      if (OWN && sg.nk == 0) {
        if (r < have) {
#pragma unroll 4
          for (int c = 0; c < D / 4; ++c)
            reinterpret_cast<float4*>(a.own + own_row * D)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          a.own[own_rows * D + own_row] = -INFINITY;
          a.own[own_rows * (D + 1) + own_row] = 0.f;
        }
        continue;
      }
      // -------------------------------------------------------- Q rows
      // This warp's 32 rows, kLanes lanes a row and kBatch loads of a lane in flight, divided by a power of two
      // and swizzled.  The products that read the rows before are complete: the softmax has had their results,
      // of both halves where they share them.
      if (!one || t == 0) {
        const unsigned long long mine = reinterpret_cast<unsigned long long>(
            a.q + b * a.q_batch + tok * a.q_token + (long long)(sg.h * a.G + gg) * a.q_head);
        if (one && items > 0) {
          ok = warp_wait(&bar_odone[1], (items - 1) & 1);
          if (!ok) break;
        }
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kBatch = 32 / kAtOnce;
        const int u = lane % kLanes;
        const uint32_t chunk = smem_u32(sQ) + t * C::kTileBytes + (u >> 3) * C::kChunkBytes;
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += kBatch * kAtOnce) {
          uint4 x[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            x[k] = __ldcg(reinterpret_cast<const uint4*>(
                              __shfl_sync(0xffffffffu, mine, i0 + k * kAtOnce + lane / kLanes)) + u);
          float m[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            m[k] = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y)
              m[k] = fmax3(m[k], fabsf(__uint_as_float(w[y] << 16)), fabsf(__uint_as_float(w[y] & 0xFFFF0000u)));
          }
#pragma unroll
          for (int off = kLanes / 2; off > 0; off >>= 1)
#pragma unroll
            for (int k = 0; k < kBatch; ++k) m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], off));
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int rr = w0 + i0 + k * kAtOnce + lane / kLanes;
            // 2^e <= m < 2^(e+1), e within the range whose negative is a normal exponent.
            const int e = min(max((int)((__float_as_uint(m[k]) >> 23) & 255u) - 127, -126), 126);
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            float y[8];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              y[2 * z] = __uint_as_float(w[z] << 16) * down;
              y[2 * z + 1] = __uint_as_float(w[z] & 0xFFFF0000u) * down;
            }
            // Elements in the codes' order.
            st_shared_v4(chunk + sw128_offset(rr, u & 7), pack_f16x2(y[0], y[2]), pack_f16x2(y[1], y[3]),
                         pack_f16x2(y[4], y[6]), pack_f16x2(y[5], y[7]));
            if (u == 0) s_e[t * 128 + rr] = (int8_t)e;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_q[t]);
      }
      ++items;
      float f = 0.f;  // factor of the row's scores, known when the first ones are: they waited for all of Q
      const int n = two ? sg.nk : (sg.nk + 1 - t) / 2;  // key tiles of this half
      const bool idle = w0 >= have;  // none of the warp's rows is one
      float m_ref = -INFINITY, W = -INFINITY, l_run = 0.f;
      float minus_m = 0.f, up = 1.f;  // -m_ref and 2^(m_ref - W), once the row has seen something
      bool any_large = false;         // of the warp's rows' maxima
      for (int j = 0; j < n; ++j) {
        // (The tile's scales are there as well: they were written before the codes were asked for.)
        ok = warp_wait(&bar_sfull[t], (sc + j) & 1);
        const int tile = g + (two ? j : 2 * j + t);
        if (!ok) break;
        tc_fence_after();
        if (!idle) {
          if (j == 0) f = a.scale_log2 * __uint_as_float((uint32_t)(127 + s_e[(one ? 0 : t * 128) + r]) << 23);
          const Head& hd = heads[tile % C::kHeads];
          // Changes scores where they lie, 16 at a time; for what is rare.
          auto change = [&](auto&& to) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              uint32_t s[16];
              tmem_ld16(tS + 16 * i, s);
              tmem_wait_ld();
              reg_fence(s);
              to(i, s);
              tmem_st16(tS + 16 * i, s);
            }
            tmem_wait_st();
          };
          // Own positions from `shown` on are those of later tokens.
          const int shown = OWN ? sg.len - a.n_q + tok + 1 - j * kBlockN : kBlockN;
          if (hd.hidden || (OWN && sg.len - a.n_q + 1 < (j + 1) * kBlockN)) {
            change([&](int i, uint32_t (&s)[16]) {
              const int seen = OWN ? min((int)hd.seen[i], shown - 16 * i) : hd.seen[i];
#pragma unroll
              for (int x = 0; x < 16; ++x)
                if (x >= seen) s[x] = __float_as_uint(-INFINITY);
            });
          }
          // Factor of the scores of group i of 16 (base 2); not 0, so that hidden ones stay -inf.
          bool rounded = false;  // the row's scores have been multiplied with it
          auto factor = [&](int i) { return rounded ? 1.f : fmaxf(f * hd.ks[i], 0x1p-126f); };
          // The weights are formed with the references of the tiles before, without a look at the maximum first.
          // Where they could be too large (which the tile's sum tells), and in the first tile, the row's
          // references move to the maximum, the accumulators with them, and the weights are formed again.
          // Other rows of the warp form the same ones again: no row's bits depend on another's.
          // The fma below leaves the rounding of the largest score's product, half its last bit, in the exponent.
          // From 2^24 on that could take a weight out of FP16: such a row's products are rounded first.
          auto round_large = [&]() {
            const bool large = !rounded && fabsf(minus_m) >= 0x1p24f;
            change([&](int i, uint32_t (&s)[16]) {
              const float k = large ? factor(i) : 1.f;
#pragma unroll
              for (int x = 0; x < 16; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) * k);
            });
            rounded = rounded || large;
          };
          if (any_large) round_large();
          bool moves = j == 0, again = j == 0;
          float sum;
          uint32_t pk[64];
          while (true) {
            if (again) {
              float mt = -INFINITY, mw = -INFINITY;  // largest score and largest log2 of a weight
#pragma unroll 1
              for (int i = 0; i < 8; ++i) {
                uint32_t s[16];
                tmem_ld16(tS + 16 * i, s);
                tmem_wait_ld();
                reg_fence(s);
                float m = __uint_as_float(s[0]);
#pragma unroll
                for (int x = 1; x < 15; x += 2) m = fmax3(m, __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
                m = fmaxf(m, __uint_as_float(s[15])) * factor(i);
                mt = fmaxf(mt, m);
                mw = fmaxf(mw, m + fmaxf(__log2f(hd.vs[i]), kLeastScale));
              }
              float f_o = 1.f;
              if (moves && mt > -INFINITY) {
                const float m_new = fmaxf(m_ref, mt - kLow), W_new = fmaxf(W, mw - kTop);
                l_run *= ex2(m_ref - m_new);
                f_o = ex2(W - W_new);
                m_ref = m_new;
                W = W_new;
                minus_m = -m_new;
                up = ex2(m_new - W_new);
              }
              if (j > 0) {
                const uint64_t f2 = f2_pack(f_o, f_o);
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t o[16];
                  tmem_ld16(tO + c * 16, o);
                  tmem_wait_ld();
                  reg_fence(o);
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    float lo, hi;
                    f2_unpack(mul2(f2_pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), f2), lo, hi);
                    o[2 * i] = __float_as_uint(lo);
                    o[2 * i + 1] = __float_as_uint(hi);
                  }
                  tmem_st16(tO + c * 16, o);
                }
              }
              any_large = __any_sync(0xffffffffu, fabsf(minus_m) >= 0x1p24f);
              if (any_large) round_large();
            }
            const uint64_t nm2 = f2_pack(minus_m, minus_m);
            uint64_t sums2[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sums2[i] = 0ull;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint64_t k2[32 / GROUP], v2[32 / GROUP];
#pragma unroll
              for (int i = 0; i < 32 / GROUP; ++i) {
                const int group = c * 2 + i;
                const float k = factor(group), v = fminf(hd.vs[group] * up, kMostFloat);
                k2[i] = f2_pack(k, k);
                v2[i] = f2_pack(v, v);
              }
              // (Nothing may come between the loads and the wait: the compiler takes the registers for loaded, and
              // could move them.)
              uint32_t s[32];
              tmem_ld32(tS + c * 32, s);
              tmem_wait_ld();
              reg_fence(s);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float x0, x1;
                f2_unpack(fma2(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), k2[2 * i / GROUP],
                               nm2), x0, x1);
                const uint64_t p2 = f2_pack(ex2(x0), ex2(x1));
                sums2[i & 3] = add2(sums2[i & 3], p2);
                f2_unpack(mul2(p2, v2[2 * i / GROUP]), x0, x1);
                pk[c * 16 + i] = pack_f16x2(x0, x1);
              }
            }
            float sums[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(sums2[i], sums[2 * i], sums[2 * i + 1]);
            sum = ((sums[0] + sums[1]) + (sums[2] + sums[3])) + ((sums[4] + sums[5]) + (sums[6] + sums[7]));
            if (again) break;
            // (So does a product that FP32 does not hold.)
            moves = m_ref == -INFINITY || !(sum * (hd.v_most * up) <= kMost && sum <= kMostSum);
            again = __any_sync(0xffffffffu, moves);
            if (!again) break;
          }
          l_run += sum;
          tmem_st32(tS, reinterpret_cast<uint32_t(&)[32]>(pk[0]));
          tmem_st32(tS + 32, reinterpret_cast<uint32_t(&)[32]>(pk[32]));
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_pfull[t]);
      }
      if (!ok) break;
      sc += n;
      g += sg.nk;
      // ------------------------------------------------------------- part
      ok = warp_wait(&bar_odone[t], oc & 1);
      if (!ok) break;
      ++oc;
      tc_fence_after();
      if (!idle) {
        // Columns c of a row are `step` floats apart by fours; the maximum and the sum `rows` apart.
        float* part = OWN ? a.own + own_row * D
                          : a.parts + (size_t)(blockIdx.x + sg.h * a.row_blocks + sg.rb) * part_floats(D) +
                                (t * kBlockM + r) * 4;
        constexpr int step = OWN ? 4 : kUnitRows * 4;
        float* sums = OWN ? a.own + own_rows * D + own_row
                          : a.parts + (size_t)(blockIdx.x + sg.h * a.row_blocks + sg.rb) * part_floats(D) +
                                D * kUnitRows + t * kBlockM + r;
        const size_t rows = OWN ? own_rows : kUnitRows;
        // (Relative to kLow above m_ref: 2^(W - m_ref) alone may pass what values next to FP32's end leave.)
        const float inv = inverse(l_run * kLowFactor), down = W == -INFINITY ? 0.f : ex2(W - m_ref - kLow);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
          if (n > 0) {
            tmem_ld32(tO + c * 32, o);
            tmem_wait_ld();
            reg_fence(o);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)  // columns in the codes' order
            if (!OWN || r < have)
              *reinterpret_cast<float4*>(part + (c * 8 + i) * step) =
                  make_float4(__uint_as_float(o[4 * i]) * inv * down, __uint_as_float(o[4 * i + 2]) * inv * down,
                              __uint_as_float(o[4 * i + 1]) * inv * down, __uint_as_float(o[4 * i + 3]) * inv * down);
        }
        if (!OWN || r < have) {
          // As the join and the sum's logarithm have them best, where adding is exact enough.
          const bool back = fabsf(m_ref) < 0x1p24f;
          sums[0] = back ? m_ref + kLow : m_ref;
          sums[rows] = back ? l_run * kLowFactor : l_run;
        }
      }
      // O_t has been read: the next segment's first P V, which overwrites it, waits for these warps' next P.
      tc_fence_before();
    }
    if (!ok && lane == 0) set_fail(ATTN_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kCopyWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// What bounds the join is the latency of its two rounds of loads (runs, then parts) and, with many units, the parts'
// bytes in L2: 152 parts (20 MB) 9.5 us, 351 of 6400 rows a key
// head (47 MB, and 27 MB of own parts) 34 us.
// Joins the parts of 32 rows of a unit and their own part, 4 columns a warp and turn; a lane has a row.  First every
// warp takes some of the parts' maxima and sums, then all of them their columns, whose loads wait for nothing
// else.  SPLIT warps share the parts of the same columns where there are many of them.  A CTA takes all columns in
// turns where there are enough rows to fill the SMs (then gridDim.x is one for each 32 rows).  The order of the
// sums is that of the runs.
constexpr int kJoinRows = 32, kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;
constexpr int kJoinBatch = 8;    // parts whose loads a thread has in flight together
constexpr int kJoinShares = kJoinBatch * kJoinWarps;  // parts whose shares of the rows are held
template <int D, int SPLIT>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const Args a, int turns) {
  __shared__ float s_m[kJoinWarps][32], s_l[kJoinWarps][32], s_share[kJoinShares][32];
  __shared__ float4 s_o[SPLIT > 1 ? kJoinWarps : 1][32];
  constexpr int kQuads = kJoinWarps / SPLIT;      // of columns at a time
  constexpr int kTurns = D / 4 / kQuads;
  griddep_launch_dependents();
  // The prefix's parts are there: every CTA of the kernel over the own positions has waited for them before it let this
  // one in.  (That they are seen without a wait here is the assumption named in shared_prefix_kernel.)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, share = warp % SPLIT;
  const int per = kTurns / turns;  // CTAs for the same rows
  int turn = blockIdx.x % per * turns;
  const unsigned x = blockIdx.x / per;
  const int rows0 = x % (kUnitRows / kJoinRows) * kJoinRows, unit = x / (kUnitRows / kJoinRows);
  const int h = unit / a.row_blocks, rb = unit - h * a.row_blocks;
  if (rb * kUnitRows + rows0 >= a.rows) return;
  const int begin = (int)threadIdx.x < a.runs ? __ldcg(a.starts + threadIdx.x) : INT_MAX;
  const int tiles = __ldcg(a.starts + a.runs);
  const int r = rows0 + lane, row = min(rb * kUnitRows + r, a.rows - 1);
  int b, tok, gg;
  row_of(a, row, b, tok, gg);
  const size_t out = ((size_t)b * a.n_q + tok) * a.H + h * a.G + gg;
  const size_t all = (size_t)a.B * a.n_q * a.H;
  // The runs that the unit's tiles are in.  (Runs without a tile begin where the tiles end.)
  const int from = unit * tiles, to = from + tiles;
  const int c0 = __syncthreads_count(begin <= from) - 1, c1 = __syncthreads_count(begin < to) - 1;
  // A unit with one row tile has two parts a run, beside one another.
  const int halves = a.rows - rb * kUnitRows > kBlockM ? 1 : 2;
  const int n = tiles == 0 ? 0 : (c1 - c0 + 1) * halves;
  const float* parts = a.parts + (size_t)(c0 + unit) * part_floats(D);
  // Part i, and the row's place in it.
  auto part = [&](int i) { return parts + (halves == 1 ? i : i >> 1) * part_floats(D); };
  auto place = [&](int i) { return halves == 1 ? r : r + (i & 1) * kBlockM; };
  auto max_of = [&](int i) { return __ldcg(part(i) + D * kUnitRows + place(i)); };
  auto sum_of = [&](int i) { return __ldcg(part(i) + (D + 1) * kUnitRows + place(i)); };

  // The first columns' parts are asked for before anything is waited for.
  const bool few = n <= kJoinShares;  // (kJoinBatch parts for each of kJoinWarps warps)
  const int col0 = (turn * kQuads + warp / SPLIT) * 4;
  auto columns = [&](int i, int col) {
    return __ldcg(reinterpret_cast<const float4*>(part(i)) + (col / 4) * kUnitRows + place(i));
  };
  float4 y[kJoinBatch];
  auto fetch = [&](int i0, int i, int some, int col) {
#pragma unroll
    for (int z = 0; z < kJoinBatch; ++z)
      if (i + z * SPLIT < some) y[z] = columns(i0 + i + z * SPLIT, col);
  };
  fetch(0, share, min(n, kJoinShares), col0);
  float M = -INFINITY, L = 0.f;
  float m[kJoinBatch], l[kJoinBatch];
  for (int i0 = warp; i0 < max(n, 1); i0 += kJoinBatch * kJoinWarps) {
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const int i = i0 + k * kJoinWarps;
      m[k] = i < n ? max_of(i) : -INFINITY;
      l[k] = i < n ? sum_of(i) : 0.f;
    }
    float m_new = M;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) m_new = fmaxf(m_new, m[k]);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    L *= ex2(M - m_use);
    M = m_new;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) L += l[k] * ex2(m[k] - m_use);
  }
  s_m[warp][lane] = M;
  s_l[warp][lane] = L;
  griddep_wait();
  const float own_m = __ldcg(a.own + all * D + out), own_l = __ldcg(a.own + all * (D + 1) + out);
  float4 own_o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (share == 0) own_o = __ldcg(reinterpret_cast<const float4*>(a.own + out * D + col0));
  __syncthreads();
  M = own_m;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_m[w][lane]);
  const float m_use = M == -INFINITY ? 0.f : M;
  const float own_share = share_of(own_l, own_m - m_use);
  L = own_share;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) L += s_l[w][lane] * ex2(s_m[w][lane] - m_use);
  // Values times 1 / L, then times their weight: the two factors' product could fall below FP32's range
  // where a small weight meets large values.
  const float inv = inverse(L);
  auto add = [&](float4& o, const float4& v, float l) {
    o.x += v.x * inv * l, o.y += v.y * inv * l, o.z += v.z * inv * l, o.w += v.w * inv * l;
  };
  if (few) {
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k)
      if (warp + k * kJoinWarps < n) s_share[warp + k * kJoinWarps][lane] = share_of(l[k], m[k] - m_use);
    __syncthreads();
  }
  for (int k = 0; k < turns; ++k, ++turn) {
    const int col = (turn * kQuads + warp / SPLIT) * 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (share == 0) {
      if (k > 0) own_o = __ldcg(reinterpret_cast<const float4*>(a.own + out * D + col));
      add(o, own_o, own_share);
    }
    for (int i0 = 0; i0 < n; i0 += kJoinShares) {
      const int some = min(kJoinShares, n - i0);
      if (!few) {
        __syncthreads();
        for (int i = warp; i < some; i += kJoinWarps) s_share[i][lane] = share_of(sum_of(i0 + i), max_of(i0 + i) - m_use);
        __syncthreads();
      }
      for (int i = share; i < some; i += kJoinBatch * SPLIT) {
        if (k > 0 || i0 > 0 || i > share) fetch(i0, i, some, col);
#pragma unroll
        for (int z = 0; z < kJoinBatch; ++z)
          if (i + z * SPLIT < some) add(o, y[z], s_share[i + z * SPLIT][lane]);
      }
    }
    if constexpr (SPLIT > 1) {
      if (k > 0) __syncthreads();
      s_o[warp][lane] = o;
      __syncthreads();
      if (share > 0) continue;
#pragma unroll
      for (int w = 1; w < SPLIT; ++w) {
        const float4 z = s_o[warp + w][lane];
        o.x += z.x, o.y += z.y, o.z += z.z, o.w += z.w;
      }
    }
    if (rb * kUnitRows + r < a.rows) {
      *reinterpret_cast<uint2*>(a.o + out * D + col) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
      if (col == 0) a.lse[out] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    }
  }
}

template <int D>
cudaError_t launch_join(const Args& a, cudaStream_t stream) {
  const unsigned units = (unsigned)(a.Hkv * a.row_blocks), groups = units * (kUnitRows / kJoinRows);
  // Four warps share a row's parts where a unit has many: 32 of two tiles of rows, 8 of one, whose tiles make two
  // parts each (19 parts of 16 rows: 38.1 us in all, 36.6 shared; 19 of 256 rows 53.5 and 56.8).
  if (units * (a.rows <= kBlockM ? 8 : 32) <= (unsigned)a.runs)
    return launch_pdl(shared_join_kernel<D, 4>, dim3(groups * (D / 8)), dim3(kJoinThreads), 0, stream, a, 1);
  const int all = D / 4 / kJoinWarps, turns = groups >= 4u * a.runs ? all : 1;
  return launch_pdl(shared_join_kernel<D, 1>, dim3(groups * (all / turns)), dim3(kJoinThreads), 0, stream, a, turns);
}

// Runs that the prefix's tiles are dealt in: one CTA an SM.  (The full device's count where
// there is no device to ask, for workspace sizes; a join's CTA has a thread for each.)
int shared_runs() {
  const int sms = device_sm_count();
  return std::min(sms > 0 ? sms : 152, kJoinThreads);
}

template <int D, int GROUP, bool OWN>
cudaError_t launch_prefix(const Args& a, unsigned grid, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kernel = shared_prefix_kernel<D, GROUP, OWN>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_smem(kernel, C::kSmemBytes, allowed);
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), C::kSmemBytes, stream, a);
}

template <bool OWN>
cudaError_t launch_prefix(const Args& a, int d, int page, unsigned grid, cudaStream_t stream) {
  if (d == 128)
    return page >= 32 ? launch_prefix<128, 32, OWN>(a, grid, stream) : launch_prefix<128, 16, OWN>(a, grid, stream);
  return page >= 32 ? launch_prefix<64, 32, OWN>(a, grid, stream) : launch_prefix<64, 16, OWN>(a, grid, stream);
}

// Rows of a sequence and key head from which on its own positions are this file's kernel's as well, where there are
// enough units to fill the SMs and, unless the rows fill a unit, the table has no room for more than rows^2 / kOwnRoom
// positions: attn_decode_int8's goes over the positions for every 32 rows, but deals long histories to all SMs, where a
// unit is one CTA's from its first key tile to its last.  (20 sequences behind 8000 positions, 8 key heads of 128, us so
// and by attn_decode_int8's kernel: all of a quarter of a length to it, and one of that length among those of 300 or
// less.  36 rows and 500: 56 and 51, 53 and 50; 64 rows and 500 73 and 67, 67 and 68, 1000 79 and 80, 74 and 70, 16000 317
// and 251, 250 and 90; 128 rows and 2048 129 and 168, 121 and 122, 4096 183 and 208, 146 and 120; 256 rows and 2048 219 and
// 264, 197 and 202, 16384 437 and 914, 374 and 270; 400 rows and 25600 1058 and 2413, 592 and 510.  d = 64: 48 rows and 500
// 46 and 43, 46 and 41, 128 and 2048 97 and 122, 93 and 91, 256 and 16384 366 and 649, 308 and 195.)
constexpr int kOwnRows = 64, kOwnRoom = 8;

struct Layout {
  size_t starts, parts, decode, bytes;  // byte offsets; the own part is at 0
};
Layout layout(const PagedCache& c, int n_q, int H) {
  const size_t all = (size_t)c.B * n_q * H, rows = all / c.Hkv;
  const size_t units = (size_t)c.Hkv * ((rows + kUnitRows - 1) / kUnitRows);
  Layout w;
  w.starts = align256(all * (c.d + 2) * sizeof(float));
  w.parts = w.starts + align256((shared_runs() + 1) * sizeof(int));
  w.decode = w.parts + align256((units + shared_runs()) * part_floats(c.d) * sizeof(float));
  w.bytes = w.decode + decode_workspace_bytes(c, n_q, H);
  return w;
}

// Whether the own positions are this file's kernel's too.
bool own_by_units(const PagedCache& c, int n_q, int H) {
  const long long rows = (long long)n_q * (H / c.Hkv);
  return rows >= kOwnRows && (rows >= kUnitRows || (long long)c.max_blocks * c.page <= rows * rows / kOwnRoom) &&
         c.B * c.Hkv * ((rows - 1) / kUnitRows + 1) >= shared_runs();
}

// Whether the prefix is read once a sequence, by attn_decode_int8's kernel in one launch with the own positions,
// instead of once for 256 rows.  That saves two launches and a join, which are worth some us, so it is for short
// prefixes and few sequences.  By the length that the prefix's table has room for, at these costs in ns for
// 1000 positions and key head: of a pass of up to 8, 16, 24 or 32 rows of a sequence, and of a unit of one row
// tile and of two; fitted to 1 to 64 sequences of 1 to 64 rows a key head behind 100 to 102400 positions, of whose 60 and
// 60 cases it chooses none worse than 1.07 and 1.03 times the better.  (Us, by sequence and by unit; 8 key heads
// of 128: 1 x 102400 42 and 70; 2 x 25600 24 and 31; 4 x 25600 36 and 31; 8 x 1600 11.3 and 16.6, 8 x 6400 23.5 and 19.7;
// 64 x 400 20 and 24, 64 x 1600 39 and 25.5; 16 x 400 with 20 rows 14 and 21, 16 x 1600 24.4 and 22.2; d = 64: 8 x 1600
// 9.4 and 13.4, 8 x 6400 16.4 and 14.0; 64 x 100 8.6 and 18.7, 64 x 400 16.2 and 14.8.)
bool reads_by_sequence(const PagedCache& c, int n_q, int H, int prefix_blocks) {
  const long long rows = (long long)n_q * (H / c.Hkv), all = rows * c.B;
  const double positions = 1e-3 * prefix_blocks * c.page * c.Hkv;
  if ((long long)(prefix_blocks + (long long)c.max_blocks) * c.page > INT_MAX - 4096 || own_by_units(c, n_q, H)) return false;
  const double pass[2][4] = {{22, 28, 36, 48}, {31, 40, 53, 69}}, unit[2][2] = {{44, 70}, {61, 90}};
  const int wide = c.d == 128;
  const long long passes = (rows + 31) / 32, units = (all - 1) / kUnitRows + 1, last = all - (units - 1) * kUnitRows;
  const double by_sequence = pass[wide][((rows + passes - 1) / passes - 1) / 8] * passes * c.B;
  const double by_unit = unit[wide][1] * (units - 1) + unit[wide][last > kBlockM];
  return (by_sequence - by_unit) * positions < (wide ? 8000 : 4700);
}

}  // namespace

size_t decode_shared_workspace_bytes(const PagedCache& c, int n_q, int H, int prefix_blocks) {
  if (reads_by_sequence(c, n_q, H, prefix_blocks)) return decode_prefix_workspace_bytes(c, n_q, H, prefix_blocks);
  return layout(c, n_q, H).bytes;
}

cudaError_t launch_decode_shared_int8(const PagedCache& c, const void* q, const long long* strides,
                                      const int* prefix_table, int prefix_blocks, const int* prefix_len,
                                      const int* lens, void* o, float* lse, int n_q, int H, float scale,
                                      void* workspace, cudaStream_t stream) {
  if (reads_by_sequence(c, n_q, H, prefix_blocks))
    return launch_decode_prefix_int8(c, q, strides, prefix_table, prefix_blocks, prefix_len, lens, o, lse, n_q, H,
                                     scale, workspace, stream);
  const Layout w = layout(c, n_q, H);
  Args a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_batch = strides[0], a.q_token = strides[1], a.q_head = strides[2];
  a.k = static_cast<const uint8_t*>(c.k), a.v = static_cast<const uint8_t*>(c.v);
  a.k_scale = c.k_scale, a.v_scale = c.v_scale;
  a.table = prefix_table, a.len = prefix_len;
  a.B = c.B, a.n_q = n_q, a.H = H, a.Hkv = c.Hkv, a.G = H / c.Hkv, a.P = c.P;
  a.page_shift = page_shift(c.page), a.blocks = prefix_blocks;
  a.rows = c.B * n_q * a.G;
  a.row_blocks = (a.rows - 1) / kUnitRows + 1;
  a.runs = shared_runs();
  a.scale_log2 = scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  a.starts = reinterpret_cast<int*>(ws + w.starts);
  a.parts = reinterpret_cast<float*>(ws + w.parts);
  a.own = reinterpret_cast<float*>(ws);
  a.o = static_cast<uint16_t*>(o), a.lse = lse;
  cudaError_t err = launch_prefix<false>(a, c.d, c.page, a.runs, stream);
  if (err != cudaSuccess) return err;
  Args own = a;
  own.table = c.table, own.len = lens, own.blocks = c.max_blocks;
  own.rows = n_q * a.G;
  own.row_blocks = (own.rows - 1) / kUnitRows + 1;
  if (own_by_units(c, n_q, H))
    err = launch_prefix<true>(own, c.d, c.page, a.runs, stream);
  else
    err = launch_decode_int8(c, q, strides, lens, nullptr, nullptr, n_q, H, scale, ws + w.decode, stream, a.own);
  if (err != cudaSuccess) return err;
  return c.d == 128 ? launch_join<128>(a, stream) : launch_join<64>(a, stream);
}

cudaError_t status_word_shared(void** word) { return cudaGetSymbolAddress(word, g_status_shared); }

}  // namespace attn

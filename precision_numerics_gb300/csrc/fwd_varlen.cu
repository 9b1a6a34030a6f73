// BF16 attention over packed sequences with grouped heads, for sm_103a.
//
// What is computed, for token i of a sequence, query head h and key head
// h / G (G = H / Hkv): O = sum_j softmax_j(scale q_i . k_j) v_j and the natural-
// log LSE, j over the sequence's own keys (causal: j <= i).  The softmax is the
// blockwise one of fwd_bf16.cu (FP32 statistics, P rounded to BF16 as the P V
// operand only), with the same roles of the warps, barriers and TMEM columns;
// that file's head gives them.  What differs:
//
//  - A 128-row query tile holds tq = 128 / G tokens of all G heads of one key
//    head: row r is token r / G, head r % G, which one TMA box of tq tokens x G
//    heads x 64 columns lays out directly.  The rows of a tile share their keys,
//    so short sequences fill a tile G times better than with a tile per head.
//    Where G does not divide 128 the last rows of a tile are idle.
//  - The work items (tq or 2 tq tokens of one sequence, for every key head) are listed
//    by a plan kernel, heaviest first, from the sequences' lengths in device
//    memory; the plan serves every call on the same packed batch.
//  - A key tile that runs past its sequence's end holds rows of the next
//    sequence.  Their scores are masked; their V rows, which P = 0 would turn
//    into NaN if they held an infinity or a NaN, are overwritten with zeros by
//    the MMA warp before the P V product reads the tile (only in such tiles).
//  - A tile's last tokens may belong to the next sequence's tile, so output rows
//    are written one by one, 8 lanes a 128-byte line, after a turn through shared
//    memory that gives each lane 16 bytes of it.
//
// Apart from fwd_bf16.cu so that what serves packed and grouped sequences (list of
// items, masks at both ends, row-wise output) takes no register or instruction from
// the forward over equal lengths.
//
// Where there are fewer items than SMs the two tiles of a CTA share the keys of one
// instead (split items, below).
//
// Bound, as in fwd_bf16.cu, by the softmax and its hand-over to the tensor pipe
// for long sequences (16384 tokens, 16 query and 2 key heads of 128: 730 us, 1500
// TFLOP/s), and by the ends of the items for short ones (12 sequences of 65 to 2048
// tokens, 32 and 8 heads of 128: 84 us, 925 TFLOP/s; 0.8 us of softmax a key tile,
// 0.85 us until the next scores, 2.2 us from an item's last key tile to the next
// item's first).
#include <math.h>

#include <algorithm>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {

static __device__ unsigned int g_status_varlen;

namespace {

constexpr int kThreads = 512;
constexpr int kRegsWG0 = 80, kRegsCorr = 80, kRegsSoftmax = 176;
static_assert(kRegsWG0 + kRegsCorr + 2 * kRegsSoftmax <= 512, "setmaxnreg split exceeds the launch pool");
static_assert(kRegsWG0 <= 128 && kRegsCorr <= 128 && kRegsSoftmax >= 128, "setmaxnreg directions");

__device__ __forceinline__ void set_fail(unsigned int code) { atomicOr(&g_status_varlen, code); }

// ---------------------------------------------------------------------------
// Plan: a header of 64 words, then one item per tile or two (tq or 2 tq tokens of
// a sequence).
// ---------------------------------------------------------------------------
constexpr int kPlanMagic = 0x564c504e;
constexpr int kPlanHeader = 64;  // words
struct PlanItem {
  int first, len, q0, end;  // sequence's first packed token and length; item's tokens in it: [q0, end)
};
static_assert(sizeof(PlanItem) == 16, "one 16-byte load per item");

inline int tile_tokens(int H, int Hkv) { return kBlockM / (H / Hkv); }
// Items at most, of one tile each.
inline long long plan_capacity(int B, int T, int H, int Hkv) { return (long long)T / tile_tokens(H, Hkv) + B; }

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 1024;

// One CTA: counts the items by their number of key tiles (kPlanBins classes,
// heaviest first), then writes each into its class's range.  The order within
// a class is that of the atomics; no result depends on it.  Where items of two
// tiles would not fill the SMs once, an item is one tile, for the other SMs to
// share the work (2048 tokens, 8 heads of 128: 36 -> 28 us).  Without a causal mask
// all items weigh the same, and the tiles have to fit the SMs in one round (one
// and a half rounds of tiles take longer than one of pairs: 30 -> 43 us).  With a
// causal mask and an odd number of tiles the first tile, not the longest, is the one
// without a partner (ungrouped heads of 200 to 1024 tokens: 20.5 -> 19.8 us).
__global__ void __launch_bounds__(kPlanThreads)
    varlen_plan_kernel(const int* __restrict__ cu, int* __restrict__ plan, int B, int T, int G, int Hkv, int tq,
                       int causal, int capacity, int sms, int split) {
  __shared__ int s_pairs;
  __shared__ int s_count[kPlanBins], s_warp[32], s_max;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  s_count[tid] = 0;
  if (tid == 0) s_max = 1, s_pairs = 0;
  __syncthreads();
  int longest = 0, pairs = 0;
  for (int b = tid; b < B; b += kPlanThreads) {
    const int x = __ldcg(cu + b), y = __ldcg(cu + b + 1);
    if (x < 0 || y < x || y > T) set_fail(ATTN_ERR_INVALID_ARG);
    const int first = min(max(x, 0), T);
    const int len = min(max(y, first), T) - first;
    longest = max(longest, len);
    pairs = min(pairs + (len + 2 * tq - 1) / (2 * tq), sms);
  }
  atomicMax(&s_max, (longest + kBlockN - 1) / kBlockN);
  if (pairs > 0) atomicAdd(&s_pairs, pairs);
  __syncthreads();
  const int most = s_max;
  const int tiles_per_item = split || (long long)s_pairs * Hkv * (causal ? 1 : 2) <= sms ? 1 : 2;
  const int per_item = tiles_per_item * tq;  // tokens
  auto each = [&](auto&& put) {
    for (int b = warp; b < B; b += kPlanThreads / 32) {
      const int first = min(max(__ldcg(cu + b), 0), T);
      const int len = min(max(__ldcg(cu + b + 1), first), T) - first;
      const int n = (len + per_item - 1) / per_item;
      const bool odd = causal && tiles_per_item == 2 && ((len + tq - 1) / tq & 1);
      for (int i = lane; i < n; i += 32) {
        const int q0 = max(i * per_item - (odd ? tq : 0), 0);
        const int end = min((i + 1) * per_item - (odd ? tq : 0), len);
        const int tiles = ((causal ? end : len) + kBlockN - 1) / kBlockN;
        put(kPlanBins - 1 - (int)((long long)(tiles - 1) * kPlanBins / most), first, len, q0, end);
      }
    }
  };
  each([&](int bin, int, int, int, int) { atomicAdd(&s_count[bin], 1); });
  __syncthreads();
  const int mine = s_count[tid];
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += y;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += s_warp[w];
  s_count[tid] = upto - mine;
  if (tid == kPlanThreads - 1) {
    plan[0] = kPlanMagic;
    plan[1] = T;
    plan[2] = G;
    plan[3] = Hkv;
    plan[4] = causal;
    // More than the capacity only for cu_seqlens that run backwards: what is dropped is reported.
    if (upto > capacity) set_fail(ATTN_ERR_INVALID_ARG);
    plan[5] = min(upto, capacity);
  }
  __syncthreads();
  PlanItem* items = reinterpret_cast<PlanItem*>(plan + kPlanHeader);
  each([&](int bin, int first, int len, int q0, int end) {
    const int at = atomicAdd(&s_count[bin], 1);
    if (at < capacity) items[at] = PlanItem{first, len, q0, end};
  });
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
template <int D>
struct Cfg {
  static constexpr int kStages = (D == 128) ? 2 : 3;
  static constexpr int kChunks = D / 64;          // 64-column (128-byte) chunks per row
  static constexpr int kChunkBytes = 128 * 128;   // 128 rows x 128 bytes
  static constexpr int kTileBytes = 128 * D * 2;  // 128 rows x d BF16
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  // Output staging: 32 rows x 128 bytes per softmax warp.
  static constexpr int kOffStage = kOffV + kStages * kTileBytes;
  static constexpr int kOffBar = kOffStage + 8 * 32 * 128;
  // q_full, q_empty, k_full[S], k_empty[S], v_full[S], v_empty[S],
  // s_full[2], p_full[2], o_done[2], mma_final, alpha[2][4], stat, o_read
  static constexpr int kNumBars = 2 + 4 * kStages + 17;
  static constexpr int kOffAlpha = kOffBar + kNumBars * 8 + 16;  // FP32 [2][128]
  static constexpr int kOffSum = kOffAlpha + 2 * 128 * 4;  // FP32 [2][128]
  static constexpr int kSmemBytes = kOffSum + 2 * 128 * 4;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
  static constexpr uint32_t kTmemCols = 512;
  static __device__ __forceinline__ uint32_t col_s(int t) { return 128u * t; }
  static __device__ __forceinline__ uint32_t col_o(int t) { return 256u + D * t; }
};

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t saddr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(saddr)
               : "memory");
  return v;
}

// Item of round r for this CTA: the list is dealt in snake order (CTA c takes
// item c of round 0, item G-1-c of round 1, ...), so that heavy and light items
// even out.  -1 once the list is done.
__device__ __forceinline__ int item_of(int r, int total) {
  const long long n = gridDim.x;
  const long long c = (r & 1) ? (n - 1 - (long long)blockIdx.x) : (long long)blockIdx.x;
  const long long idx = (long long)r * n + c;
  return idx < total ? (int)idx : -1;
}

// q0: first token (in the sequence) of tile 0; n: key tiles of the two tiles, nmax: of the
// item.  In a split item both tiles are the same queries; tile 0 takes the key tiles 0,
// 2, ..., tile 1 the others, and their results are joined.  That halves the chain of
// an item (one prompt of 2048 tokens, 8 heads of 128: 28.9 -> 20.2 us, 4096 tokens of 4 heads
// 49.6 -> 33.8); the join takes as long as a key tile, so short items are not split.
constexpr int kSplitTiles = 4;
struct Item {
  int first, len, head, q0, n[2], nmax;
  bool split;
};
// The plan's words of item L.  They take 0.6 us to come, so roles that would wait for
// them ask ahead (ragged prompts with 7 items a CTA: 87.1 -> 85.6 us).
__device__ __forceinline__ int4 item_words(const int* plan, int L, int Hkv) {
  return L >= 0 ? *(reinterpret_cast<const int4*>(plan + kPlanHeader) + L / Hkv) : make_int4(0, 0, 0, 0);
}
template <bool CAUSAL, bool SPLIT>
__device__ __forceinline__ Item make_item(const int4& p, int L, int Hkv, int tq) {
  Item it;
  it.first = p.x;
  it.len = p.y;
  it.q0 = p.z;
  it.head = L % Hkv;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int q = it.q0 + t * tq;
    const int keys = CAUSAL ? min(q + tq, it.len) : it.len;
    it.n[t] = q >= p.w ? 0 : (keys + kBlockN - 1) / kBlockN;
  }
  it.nmax = max(it.n[0], it.n[1]);
  it.split = SPLIT && it.n[1] == 0 && it.nmax >= kSplitTiles;
  if (it.split) it.n[0] = (it.nmax + 1) / 2, it.n[1] = it.nmax / 2;
  return it;
}
// Rows of key tile j that belong to the sequence.
__device__ __forceinline__ int tile_keys(const Item& it, int j) { return min(kBlockN, it.len - j * kBlockN); }

template <int D, bool CAUSAL, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    varlen_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const int* plan,
                      uint16_t* __restrict__ out, float* __restrict__ lse, int T, int H, int Hkv, int G, int tq,
                      int capacity, float scale, float scale_log2) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* bar_q = bars;
  uint64_t* bar_qempty = bars + 1;
  uint64_t* bar_kfull = bars + 2;
  uint64_t* bar_kempty = bar_kfull + C::kStages;
  uint64_t* bar_vfull = bar_kempty + C::kStages;
  uint64_t* bar_vempty = bar_vfull + C::kStages;
  uint64_t* bar_sfull = bar_vempty + C::kStages;
  uint64_t* bar_pfull = bar_sfull + 2;
  uint64_t* bar_odone = bar_pfull + 2;
  uint64_t* bar_final = bar_odone + 2;
  uint64_t* bar_alpha = bar_final + 1;
  uint64_t* bar_stat = bar_alpha + 8;
  uint64_t* bar_oread = bar_stat + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  float* s_alpha = reinterpret_cast<float*>(smem + C::kOffAlpha);
  float* s_sum = reinterpret_cast<float*>(smem + C::kOffSum);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    *s_abort = (smem_u32(smem) & 1023u) != 0;
    mbar_init(bar_q, 1);
    mbar_init(bar_qempty, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar_kfull[s], 1);
      mbar_init(&bar_kempty[s], 1);
      mbar_init(&bar_vfull[s], 1);
      mbar_init(&bar_vempty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar_sfull[t], 1);
      mbar_init(&bar_pfull[t], 256);  // softmax (P stored) + correction (O rescaled)
      for (int q = 0; q < 4; ++q) mbar_init(&bar_alpha[t * 4 + q], 32);
      mbar_init(&bar_odone[t], 1);
    }
    mbar_init(bar_final, 1);
    mbar_init(bar_stat, 256);   // both softmax warpgroups
    mbar_init(bar_oread, 256);
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Set-up above touches no global memory; from here on the previous kernel's
  // results must be complete and visible.
  griddep_wait();
  // The plan must be one for this call: anything else is reported and nothing
  // is computed, so that no item can reach outside the tensors.
  const int4 head0 = __ldcg(reinterpret_cast<const int4*>(plan));
  const int4 head1 = __ldcg(reinterpret_cast<const int4*>(plan) + 1);
  const bool plan_ok = head0.x == kPlanMagic && head0.y == T && head0.z == G && head0.w == Hkv &&
                       head1.x == (CAUSAL ? 1 : 0) && head1.y >= 0 && head1.y <= capacity;
  const bool abort_all = *s_abort != 0 || !plan_ok;
  const int total = plan_ok ? head1.y * Hkv : 0;
  if (threadIdx.x == 0 && abort_all) set_fail(ATTN_ERR_INVALID_ARG);

  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;

  // Barrier phases run on across items: every role counts the completions it
  // has consumed (K/V ring position g, items, S and P tiles per query tile).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWG0));
    if (warp == 0 && lane == 0 && !abort_all) {
      // ------------------------------------------------------------ producer
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      const uint32_t q_bytes = 128u * G * tq;  // one chunk of a query tile
      bool ok = true;
      int g = 0, items = 0, issued_k = 0, issued_v = 0;
      for (int r = 0; ok; ++r) {
        const int L = item_of(r, total);
        if (L < 0) break;
        const Item it = make_item<CAUSAL, SPLIT>(item_words(plan, L, Hkv), L, Hkv, tq);
        // The Q slots are free once the previous item's last S products have run.
        if (items > 0 && !mbar_wait(bar_qempty, (items - 1) & 1)) { ok = false; break; }
        mbar_arrive_expect_tx(bar_q, 2 * C::kChunks * q_bytes);
        for (int t = 0; t < 2; ++t)
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(sQ + t * C::kTileBytes + c * C::kChunkBytes, &tmQ, bar_q, c * 64, it.head * G,
                        it.first + it.q0 + (SPLIT && it.split ? 0 : t * tq));
        ++items;
        for (int j = 0; j < it.nmax; ++j, ++g) {
          const int st = g % C::kStages;
          const int use = g / C::kStages;
          if (use > 0 && !mbar_wait(&bar_kempty[st], (use - 1) & 1)) { ok = false; break; }
          mbar_arrive_expect_tx(&bar_kfull[st], C::kTileBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(sK + st * C::kTileBytes + c * C::kChunkBytes, &tmK, &bar_kfull[st], c * 64,
                        it.first + j * kBlockN, it.head);
          issued_k = g + 1;
          if (use > 0 && !mbar_wait(&bar_vempty[st], (use - 1) & 1)) { ok = false; break; }
          mbar_arrive_expect_tx(&bar_vfull[st], C::kTileBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(sV + st * C::kTileBytes + c * C::kChunkBytes, &tmV, &bar_vfull[st], c * 64,
                        it.first + j * kBlockN, it.head);
          issued_v = g + 1;
        }
      }
      if (!ok) set_fail(ATTN_ERR_TIMEOUT);
      // Do not leave while copies into this CTA's shared memory are in flight.
      if (items > 0) mbar_wait(bar_q, (items - 1) & 1);
      for (int x = max(0, issued_k - C::kStages); x < issued_k; ++x)
        mbar_wait(&bar_kfull[x % C::kStages], (x / C::kStages) & 1);
      for (int x = max(0, issued_v - C::kStages); x < issued_v; ++x)
        mbar_wait(&bar_vfull[x % C::kStages], (x / C::kStages) & 1);
    } else if (warp == 1 && !abort_all) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc_qk = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16(128, D, false, true);
      const uint64_t descQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t descK = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t descV = sdesc_sw128(smem_u32(sV), C::kChunkBytes, 1024);
      auto issue_s = [&](int t, int st) {
        const uint64_t a0 = sdesc_add(descQ, t * C::kTileBytes);
        const uint64_t b0 = sdesc_add(descK, st * C::kTileBytes);
        const uint32_t d = tmem + C::col_s(t);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
          mma_ss_elect(d, sdesc_add(a0, off), sdesc_add(b0, off), idesc_qk, kk > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int t, int st, bool acc) {
        const uint64_t b0 = sdesc_add(descV, st * C::kTileBytes);
        const uint32_t d = tmem + C::col_o(t), a = tmem + C::col_s(t);
#pragma unroll
        for (int kk = 0; kk < kBlockN / 16; ++kk)
          mma_ts_elect(d, a + kk * 8, sdesc_add(b0, kk * 2048), idesc_pv, (acc || kk > 0) ? 1u : 0u);
      };
      // Rows past the sequence's end become zero while the softmax works on the tile's
      // scores.  Rows are 128 bytes in every 64-column chunk; the swizzle moves units within
      // a row only.
      auto zero_behind = [&](const Item& it, int j, int st) {
        const int keys = tile_keys(it, j);
        if (keys >= kBlockN) return;
        for (int c = 0; c < C::kChunks; ++c)
          for (int i = keys * 8 + lane; i < kBlockN * 8; i += 32)
            st_shared_v4(smem_u32(sV + st * C::kTileBytes + c * C::kChunkBytes + i * 16), 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      };
      bool ok = true;
      int g = 0, items = 0;
      int pc[2] = {0, 0};   // P tiles consumed per query tile (p_full phases)
      int L = item_of(0, total);
      int4 words = item_words(plan, L, Hkv);
      for (int r = 1; ok && L >= 0; ++r) {
        const Item it = make_item<CAUSAL, SPLIT>(words, L, Hkv, tq);
        L = item_of(r, total);
        words = item_words(plan, L, Hkv);
        // S_t(0).  S_t's columns are free: the previous item's P_t V, issued
        // earlier on this thread, reads P_t before these products run.
        ok = warp_wait(bar_q, items & 1);
        if (SPLIT && it.split) {
          // Key tile e is tile t = e & 1's; the products of one tile run while the other's
          // softmax works.
          ++items;
          auto s_of = [&](int e) {
            const int ge = g + e;
            if (!warp_wait(&bar_kfull[ge % C::kStages], (ge / C::kStages) & 1)) return false;
            tc_fence_after();
            issue_s(e & 1, ge % C::kStages);
            mma_commit_elect(&bar_sfull[e & 1]);
            mma_commit_elect(&bar_kempty[ge % C::kStages]);
            if (e + 1 == it.nmax) mma_commit_elect(bar_qempty);
            return true;
          };
          ok = ok && s_of(0) && s_of(1);
          for (int e = 0; e < it.nmax && ok; ++e) {
            const int t = e & 1, st = (g + e) % C::kStages;
            ok = warp_wait(&bar_vfull[st], ((g + e) / C::kStages) & 1);
            if (!ok) break;
            zero_behind(it, e, st);
            ok = warp_wait(&bar_pfull[t], (pc[t] + (e >> 1)) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, st, e >= 2);
            mma_commit_elect(&bar_vempty[st]);
            if (e + 2 < it.nmax)
              ok = s_of(e + 2);
            else
              mma_commit_elect(&bar_odone[t]);
          }
          g += it.nmax;
          pc[0] += it.n[0];
          pc[1] += it.n[1];
          continue;
        }
        if (ok) ok = warp_wait(&bar_kfull[g % C::kStages], (g / C::kStages) & 1);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < 2; ++t) {
          if (it.n[t] == 0) continue;
          issue_s(t, g % C::kStages);
          mma_commit_elect(&bar_sfull[t]);
        }
        mma_commit_elect(&bar_kempty[g % C::kStages]);  // K is free once S(0) has completed
        if (it.nmax == 1) mma_commit_elect(bar_qempty);  // every S product of the item issued
        ++items;
        for (int j = 0; j < it.nmax && ok; ++j) {
          const int gj = g + j;
          const int st = gj % C::kStages;
          const int st1 = (gj + 1) % C::kStages;
          const bool has_next = j + 1 < it.nmax;
          if (!warp_wait(&bar_vfull[st], (gj / C::kStages) & 1)) { ok = false; break; }
          zero_behind(it, j, st);
          if (has_next && !warp_wait(&bar_kfull[st1], ((gj + 1) / C::kStages) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int t = 0; t < 2 && ok; ++t) {
            if (j >= it.n[t]) continue;
            if (!warp_wait(&bar_pfull[t], (pc[t] + j) & 1)) { ok = false; break; }
            tc_fence_after();
            issue_pv(t, st, j > 0);
            if (j + 1 < it.n[t]) {
              issue_s(t, st1);
              mma_commit_elect(&bar_sfull[t]);
            } else {
              mma_commit_elect(&bar_odone[t]);
            }
          }
          if (!ok) break;
          mma_commit_elect(&bar_vempty[st]);
          // Release K_{j+1} as soon as the S(j+1) products above have read it, so
          // the producer can start loading K_{j+1+S} a full iteration ahead.
          if (has_next) mma_commit_elect(&bar_kempty[st1]);
          // The item's last S products were issued above: Q may be replaced.
          if (j + 2 == it.nmax) mma_commit_elect(bar_qempty);
        }
        g += it.nmax;
        pc[0] += it.n[0];
        pc[1] += it.n[1];
      }
      if (!ok && lane == 0) set_fail(ATTN_ERR_TIMEOUT);
      // Every MMA this warp issued completes before TMEM is released.
      mma_commit_elect(bar_final);
      mbar_wait(bar_final, 0);
    }
    __syncwarp();
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCorr));
    // -------------------------------------------------------------- correction
    // O_t(j-1) has completed when the softmax of tile t publishes alpha(j):
    // that happens after S_t(j) completed, and the commit that signalled S_t(j)
    // covers every earlier MMA, PV_t(j-1) included.
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = !abort_all;
    int ac[2] = {0, 0};  // alpha phases consumed per query tile
    for (int rr = 0; ok; ++rr) {
      const int L = item_of(rr, total);
      if (L < 0) break;
      const Item it = make_item<CAUSAL, SPLIT>(item_words(plan, L, Hkv), L, Hkv, tq);
      const int steps = SPLIT ? max(it.n[0], it.n[1]) : it.nmax;
      for (int j = 0; j < steps && ok; ++j) {
        for (int t = 0; t < 2; ++t) {
          if (j >= it.n[t]) continue;
          // Only the softmax warp that owns the same 32 TMEM lanes is waited for.
          ok = __all_sync(0xffffffffu, mbar_wait(&bar_alpha[t * 4 + (warp & 3)], (ac[t] + j) & 1));
          if (!ok) break;
          const float alpha = s_alpha[t * 128 + r];
          if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            tc_fence_after();
            const uint32_t tO = tmem + lane_off + C::col_o(t);
            const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float lo, hi;
                f2_unpack(mul2(f2_pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), a2), lo, hi);
                o[2 * i] = __float_as_uint(lo);
                o[2 * i + 1] = __float_as_uint(hi);
              }
              tmem_st32(tO + c * 32, o);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          mbar_arrive(&bar_pfull[t]);
        }
      }
      ac[0] += it.n[0];
      ac[1] += it.n[1];
    }
    if (!ok && !abort_all) set_fail(ATTN_ERR_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // -------------------------------------------------------------- softmax
    const int t = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;  // query row within the tile = TMEM lane
    const int row_tok = r / G, row_head = r - row_tok * G;
    const bool row_used = row_tok < tq;
    const uint32_t by_G = (65536u + G - 1) / G;  // (x * by_G) >> 16 is x / G for x < 128, G <= 128
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::col_s(t);
    const uint32_t tO = tmem + lane_off + C::col_o(t);
    // The product m scale_log2 is rounded before the fma that takes it off, so that all weights of a
    // row are off by 2^(half its last bit) together.  From 2^28 on that would leave the type (from
    // 2^31), and any two scores lie 16 and more apart: a power of two in place of the scale, whose
    // products are exact, then gives the same weights, all but 2^-16 of them.
    const float scale_up = __uint_as_float((__float_as_uint(scale_log2) + 0x7FFFFFu) & 0x7F800000u);
    bool ok = !abort_all;
    int sc = 0;  // S_t tiles consumed so far (s_full phases)
    int oc = 0;  // items whose O_t was completed so far (o_done phases)
    int splits = 0;  // split items so far (stat and o_read phases)
    int L = item_of(0, total);
    int4 words = item_words(plan, L, Hkv);
    for (int round = 1; ok && L >= 0; ++round) {
      const Item it = make_item<CAUSAL, SPLIT>(words, L, Hkv, tq);
      const int n = it.n[t];
      const int q_first = it.q0 + (SPLIT && it.split ? 0 : t * tq);
      const int tok = q_first + (row_used ? row_tok : 0);  // token within the sequence
      const int limit = CAUSAL ? min(tok + 1, it.len) : it.len;
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_sfull[t], (sc + j) & 1));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence(s[c]);

        const int kv0 = (SPLIT && it.split ? 2 * j + t : j) * kBlockN;
        if (kv0 + kBlockN > it.len || (CAUSAL && kv0 + kBlockN - 1 > q_first)) {
          const int lim = limit - kv0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= lim) s[c >> 5][c & 31] = __float_as_uint(-INFINITY);
        }
        // Row max as four independent chains of three-input maxima.
        float mx4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float m = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
          for (int e = 2; e < 32; e += 2)
            m = fmax3(m, __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
          mx4[c] = m;
        }
        const float m_new = fmaxf(fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]), m_run);
        const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
        const float unit = fabsf(m_use * scale_log2) < 0x1p28f ? scale_log2 : scale_up;
        const float neg_ms = -m_use * unit;
        const float alpha = ex2((m_run - m_use) * scale_log2);
        s_alpha[t * 128 + r] = alpha;
        mbar_arrive(&bar_alpha[t * 4 + (warp & 3)]);  // the correction warp rescales O_t meanwhile
        uint64_t sums2[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) sums2[u] = 0ull;
        const uint64_t c2 = f2_pack(unit, unit);
        const uint64_t nm2 = f2_pack(neg_ms, neg_ms);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x0, x1;
            f2_unpack(fma2(f2_pack(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), c2, nm2), x0, x1);
            const float p0 = ex2(x0);
            const float p1 = ex2(x1);
            sums2[i & 3] = add2(sums2[i & 3], f2_pack(p0, p1));
            pk[i] = pack_bf16x2(p0, p1);
          }
          tmem_st16(tS + c * 16, pk);
        }
        float sums[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) f2_unpack(sums2[u], sums[2 * u], sums[2 * u + 1]);
        const float tile_sum = ((sums[0] + sums[1]) + (sums[2] + sums[3])) +
                               ((sums[4] + sums[5]) + (sums[6] + sums[7]));
        l_run = l_run * alpha + tile_sum;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar_pfull[t]);
        m_run = m_new;
      }
      sc += n;
      L = item_of(round, total);
      words = item_words(plan, L, Hkv);
      if (!ok || n == 0) continue;
      // ------------------------------------------------------------ epilogue
      // O = O_acc / l and LSE = m * scale + ln(l).  The next item's first P V
      // product, which overwrites O_t, waits for this warpgroup's next P, so it
      // cannot run before O_t has been read here.
      ok = __all_sync(0xffffffffu, mbar_wait(&bar_odone[t], oc & 1));
      if (!ok) break;
      ++oc;
      tc_fence_after();
      const bool have = row_used && tok < it.len;
      const size_t row_at = (size_t)(it.first + tok) * H + it.head * G + row_head;
      const uint32_t stage = smem_u32(smem + C::kOffStage) + (warp - 4) * 32 * 128;
      // 64 columns to memory; get(h, o) reads 32 of them, scaled, in pairs.
      auto write_chunk = [&](int c, auto&& get) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint64_t o2[16];
          get(h, o2);
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float lo, hi;
            f2_unpack(o2[i], lo, hi);
            pk[i] = pack_bf16x2(lo, hi);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            st_shared_v4(stage + sw128_offset(lane, h * 4 + u), pk[4 * u], pk[4 * u + 1], pk[4 * u + 2],
                         pk[4 * u + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + (lane >> 3);  // row of this warp's 32
          const int tile_row = (warp & 3) * 32 + rr;
          const int rt = (int)(((uint32_t)tile_row * by_G) >> 16), rh = tile_row - rt * G;
          if (rt < tq && q_first + rt < it.len) {
            const uint4 v = ld_shared_v4(stage + sw128_offset(rr, lane & 7));
            *reinterpret_cast<uint4*>(out + ((size_t)(it.first + q_first + rt) * H + it.head * G + rh) * D + c * 64 +
                                      (lane & 7) * 8) = v;
          }
        }
        __syncwarp();
      };
      auto load = [&](uint32_t from, uint32_t (&o)[32]) {
        tmem_ld32(from, o);
        tmem_wait_ld();
        reg_fence(o);
      };
      if (!SPLIT || !it.split) {
        const float inv_l = l_run > 0.f ? 1.f / l_run : 0.f;
        const uint64_t il2 = f2_pack(inv_l, inv_l);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          write_chunk(c, [&](int h, uint64_t (&o2)[16]) {
            uint32_t o[32];
            load(tO + c * 64 + h * 32, o);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o2[i] = mul2(f2_pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), il2);
          });
        if (have) lse[row_at] = m_run * scale + logf(l_run);
      } else {
        // Both halves of a row are in the same TMEM lane: with the other's maximum and
        // sum, every warpgroup joins 64 columns (d = 64: the first one does).
        s_alpha[t * 128 + r] = m_run;  // the correction has read the last factor: O_t is complete
        s_sum[t * 128 + r] = l_run;
        tc_fence_before();
        mbar_arrive(bar_stat);
        ok = __all_sync(0xffffffffu, mbar_wait(bar_stat, splits & 1));
        if (!ok) break;
        tc_fence_after();
        const float m_other = s_alpha[(t ^ 1) * 128 + r], l_other = s_sum[(t ^ 1) * 128 + r];
        const float m = fmaxf(m_run, m_other), m_use = m == -INFINITY ? 0.f : m;
        const float mine = ex2((m_run - m_use) * scale_log2), others = ex2((m_other - m_use) * scale_log2);
        const float l = l_run * mine + l_other * others;
        const float inv_l = l > 0.f ? 1.f / l : 0.f;
        const float f0 = mine * inv_l, f1 = others * inv_l;
        const uint64_t f02 = f2_pack(f0, f0), f12 = f2_pack(f1, f1);
        const uint32_t tOther = tmem + lane_off + C::col_o(t ^ 1);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          if (c == t)
            write_chunk(c, [&](int h, uint64_t (&o2)[16]) {
              uint32_t o[32];
              load(tO + c * 64 + h * 32, o);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o2[i] = mul2(f2_pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), f02);
              load(tOther + c * 64 + h * 32, o);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o2[i] = fma2(f2_pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), f12, o2[i]);
            });
        if (have && t == 0) lse[row_at] = m * scale + logf(l);
        // The next item's P V may overwrite O_t when both warpgroups have read it.
        tc_fence_before();
        mbar_arrive(bar_oread);
        ok = __all_sync(0xffffffffu, mbar_wait(bar_oread, splits & 1));
        if (!ok) break;
        ++splits;
      }
    }
    if (!ok && !abort_all) set_fail(ATTN_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// 3-D BF16 map of a [T, heads, d] tensor with strides in elements.  `rows`
// first: (d, T, heads) with a 64 x n x 1 box (keys), else (d, heads, T) with a
// 64 x G x n box (queries).
bool make_tmap_packed(CUtensorMap* map, const void* base, int T, int heads, int d, long long token_stride,
                      long long head_stride, bool keys, int G, int n) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return false;
  const cuuint64_t tok = (cuuint64_t)token_stride * 2, head = (cuuint64_t)head_stride * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)(keys ? T : heads), (cuuint64_t)(keys ? heads : T)};
  const cuuint64_t strides[2] = {keys ? tok : head, keys ? head : tok};
  const cuuint32_t box[3] = {64, (cuuint32_t)(keys ? n : G), (cuuint32_t)(keys ? 1 : n)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Items are of one tile, and long ones split, where items of two would not fill the SMs
// whatever the lengths of B sequences of T tokens are (at 1.5 to 3 times as many items the
// two halves of a pair are the better use of an SM: ragged d = 64 23.5 us, 19.3 in pairs).
bool splits_items(const VarlenProblem& p) {
  const int sms = device_sm_count();
  const long long pairs = (long long)p.T / (2 * tile_tokens(p.H, p.Hkv)) + p.B;
  return p.T > (kSplitTiles - 1) * kBlockN && pairs * p.Hkv * (p.causal ? 1 : 2) <= sms;
}

template <int D, bool CAUSAL, bool SPLIT>
cudaError_t launch_impl(const VarlenProblem& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                        const void* plan, void* o, float* lse, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kernel = varlen_fwd_kernel<D, CAUSAL, SPLIT>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_smem(kernel, C::kSmemBytes, allowed);
  if (err != cudaSuccess) return err;
  const long long capacity = plan_capacity(p.B, p.T, p.H, p.Hkv);
  // One CTA per SM (one fits); without an SM count, one per item.
  const int sms = device_sm_count();
  const long long most = capacity * p.Hkv;
  const unsigned grid = (unsigned)(sms > 0 ? std::min<long long>(most, sms) : most);
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), C::kSmemBytes, stream, mq, mk, mv,
                    static_cast<const int*>(plan), static_cast<uint16_t*>(o), lse, p.T, p.H, p.Hkv, p.H / p.Hkv,
                    tile_tokens(p.H, p.Hkv), (int)capacity, p.scale, p.scale * 1.4426950408889634f);
}

}  // namespace

size_t varlen_plan_bytes(int B, int T, int H, int Hkv) {
  return kPlanHeader * 4 + (size_t)plan_capacity(B, T, H, Hkv) * sizeof(PlanItem);
}

cudaError_t launch_varlen_plan(const VarlenProblem& p, const int* cu, void* plan, cudaStream_t stream) {
  return launch_pdl(varlen_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, cu, static_cast<int*>(plan), p.B, p.T,
                    p.H / p.Hkv, p.Hkv, tile_tokens(p.H, p.Hkv), p.causal,
                    (int)plan_capacity(p.B, p.T, p.H, p.Hkv), device_sm_count(), splits_items(p) ? 1 : 0);
}

cudaError_t launch_varlen_fwd(const VarlenProblem& p, const void* q, const void* k, const void* v, const void* plan,
                              void* o, float* lse, const long long* strides, cudaStream_t stream) {
  CUtensorMap mq, mk, mv;
  const int G = p.H / p.Hkv;
  if (!make_tmap_packed(&mq, q, p.T, p.H, p.d, strides[0], strides[1], false, G, tile_tokens(p.H, p.Hkv)) ||
      !make_tmap_packed(&mk, k, p.T, p.Hkv, p.d, strides[2], strides[3], true, G, kBlockN) ||
      !make_tmap_packed(&mv, v, p.T, p.Hkv, p.d, strides[4], strides[5], true, G, kBlockN))
    return cudaErrorInvalidValue;
  const bool split = splits_items(p);
#define ATTN_VARLEN_CASE(DD, CC, SS)                   \
  if (p.d == DD && (p.causal != 0) == CC && split == SS) \
    return launch_impl<DD, CC, SS>(p, mq, mk, mv, plan, o, lse, stream);
  ATTN_VARLEN_CASE(64, false, false)
  ATTN_VARLEN_CASE(64, false, true)
  ATTN_VARLEN_CASE(64, true, false)
  ATTN_VARLEN_CASE(64, true, true)
  ATTN_VARLEN_CASE(128, false, false)
  ATTN_VARLEN_CASE(128, false, true)
  ATTN_VARLEN_CASE(128, true, false)
  ATTN_VARLEN_CASE(128, true, true)
#undef ATTN_VARLEN_CASE
  return cudaErrorInvalidValue;
}

cudaError_t status_word_varlen(void** word) { return cudaGetSymbolAddress(word, g_status_varlen); }

}  // namespace attn

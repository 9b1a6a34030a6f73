// Block tables, offsets and slots of a step from the requests' lengths.
//
// With pages(x) = ceil(x / page), a sequence that goes from held to wanted positions gives the
// pages [pages(wanted), pages(held)) of its table back to the stack of free pages, or takes
// pages [pages(held), pages(wanted)) from it.  In the order of the sequences and, within one,
// of the positions:
//   released page i goes to stack[n + i], i < R;
//   a request is served if the pages needed up to and with it are n + R at most (or it needs none);
//   the N pages of those that are served are stack[n + R - N .. n + R).
// So a step that is taken back leaves table and stack as they were.  New token i of sequence b
// is packed token cu[b] + i, position held + i, row table[b][position / page] * page + position %
// page of the pool.
//
// Nothing is computed but sums, and the bytes are few: what bounds it is the chain of dependent loads
// (lengths, table entries, stack, slots) with their barriers.  So one launch does it all: a CTA, or a cluster of
// them that work in step where there are many pages or tokens.  Each scans all lengths, kThreads at a time, and
// takes its share of the pages and tokens, which it finds by bisection in the sums.  Tokens take their pages
// from where the table gets them, not from the table.  Slots of more tokens than a cluster writes quickly are
// a second kernel's (kSlotsInside).
//
// Measured, a call among others: 3 sequences of one new token 3.7 us, 256 5.8 (one CTA of 256 threads, for which
// __syncthreads and the scan's rounds cost half of what they do for 1024: 17 -> 7.9 us for two calls); 64 prompts of
// 150 to 4096 tokens 5.7 and 4.4 for their slots, 1000 of 10 to 6000 10.5 and 10.5 (1 M tokens, 8 MB).  With the
// table written first and the tokens' pages read back from it, behind another barrier, these took 35 and 59 us in
// place of 18 and 32 with the call that takes the step back.
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {

static __device__ unsigned int g_status_tables;

namespace {

// A small CTA for up to kFew sequences with up to kFew * kAtOnce tokens; else one of kThreads, or with more than
// kAlone tokens a cluster of kMany.  (A step and its reverse, us, 64 sequences: of a token each 6.5, 8.9 with 1024
// threads; of 16 7.8 and 9.2; of 64 10.5 by one CTA and 8.6 by the cluster, of 256 19.2 and 9.2; 500 sequences of a token
// 9.5 and 10.1.)
constexpr int kFew = 256, kThreads = 1024, kMany = 8, kAlone = 1024;
// The pages that a call gives back are not known here, but the table's room is: a cluster from 16384 on.  (4096 pages
// taken and given back 18.3 us by the small CTA and 9.6 by the cluster, 16384 59 and 10.8, 65536 222 and 18.9; 200
// sequences of a token 7.0 and 10.1.)
constexpr int kAlonePages = 16384;
// Tokens whose slots the cluster writes; with more of them a second kernel's CTAs do, which find their tokens' sequences
// in the offsets (32000 tokens 10.9 us inside and 12.0 so, 64000 15.0 and 12.7, 128000 22.4 and 14.3).
constexpr int kSlotsInside = 40960;
constexpr int kAtOnce = 4;           // pages or tokens of a thread with their loads in flight together

__device__ __forceinline__ void set_fail(unsigned int code) { atomicOr(&g_status_tables, code); }

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned n;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

// What a sequence does in this step.
struct Move {
  int held, wanted;
  int have, want;  // pages
  __device__ __forceinline__ Move(const Tables& t, int b, bool report) : held(0), wanted(0), have(0), want(0) {
    if (b >= t.B) return;
    held = __ldcg(t.held + b);
    wanted = __ldcg(t.wanted + b);
    const int room = t.max_blocks << t.page_shift;
    if (held < 0 || wanted < 0 || held > room || wanted > room) {  // left as it is
      if (report) set_fail(ATTN_ERR_INVALID_ARG);
      wanted = held;
      return;
    }
    const int up = (1 << t.page_shift) - 1;
    have = (held + up) >> t.page_shift;
    want = (wanted + up) >> t.page_shift;
  }
  __device__ __forceinline__ int need() const { return max(want - have, 0); }
  __device__ __forceinline__ int released() const { return max(have - want, 0); }
  __device__ __forceinline__ int tokens() const { return max(wanted - held, 0); }
};

// The last of the N starts that is i or less.
template <int N>
__device__ __forceinline__ int find(const long long* s_start, long long i) {
  int at = 0;
#pragma unroll
  for (int step = N / 2; step > 0; step >>= 1)
    if (s_start[at + step] <= i) at += step;
  return at;
}

// N sequences from b0 on: where each one's needed and released pages and its new tokens begin, and their ends.
template <int N>
struct Chunk {
  long long need[N + 1], released[N + 1], tokens[N + 1];
  int held[N], wanted[N];
  long long warp[3][N / 32];

  __device__ __forceinline__ void scan(const Move& m) {
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    long long x[3] = {m.need(), m.released(), m.tokens()};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const long long y = __shfl_up_sync(0xffffffffu, x[k], off);
        if (lane >= off) x[k] += y;
      }
    __syncthreads();  // what was here before has been read
    if (lane == 31)
#pragma unroll
      for (int k = 0; k < 3; ++k) warp[k][w] = x[k];
    __syncthreads();
    long long before[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      long long y = lane < N / 32 ? warp[k][lane] : 0;
#pragma unroll
      for (int off = 1; off < N / 32; off <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) y += z;
      }
      before[k] = w > 0 ? __shfl_sync(0xffffffffu, y, w - 1) : 0;
    }
    if (tid == 0) need[0] = released[0] = tokens[0] = 0;
    need[tid + 1] = before[0] + x[0];
    released[tid + 1] = before[1] + x[1];
    tokens[tid + 1] = before[2] + x[2];
    held[tid] = m.held;
    wanted[tid] = m.wanted;
    __syncthreads();
  }
};

template <int N>
__global__ void __launch_bounds__(N) cache_reserve_kernel(const Tables t, int slots_inside) {
  __shared__ Chunk<N> s;
  __shared__ long long s_sum[N / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  const bool first_cta = blockIdx.x == 0, single = t.B <= N;
  const unsigned threads = cluster_size() * N, gtid = blockIdx.x * N + tid;
  int n = __ldcg(t.n_free);
  const Move mine(t, tid, first_cta);  // of the first N sequences
  if (n < 0 || n > t.P) {
    if (first_cta && tid == 0) set_fail(ATTN_ERR_INVALID_ARG);
    n = min(max(n, 0), t.P);
  }
  const int up = (1 << t.page_shift) - 1;
  s.scan(mine);
  long long released = s.released[N];  // by all sequences
  if (!single) {
    long long x = 0;
    for (int b = tid; b < t.B; b += N) x += Move(t, b, b >= N && first_cta).released();
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if ((tid & 31) == 0) s_sum[tid >> 5] = x;
    __syncthreads();
    released = 0;
    for (int w = 0; w < N / 32; ++w) released += s_sum[w];
  }
  const long long full = n + released, top = min(full, (long long)t.P);
  if (full > t.P && first_cta && tid == 0) set_fail(ATTN_ERR_INVALID_ARG);

  // Released pages go on the stack, and the pages of all requests that are served are counted.
  long long before_released = 0, before_need = 0, served = 0;
  for (int b0 = 0; b0 < t.B; b0 += N) {
    if (b0 > 0) s.scan(Move(t, b0 + tid, false));
    for (long long i0 = gtid; i0 < s.released[N]; i0 += (long long)threads * kAtOnce) {
      int* from[kAtOnce];
      int page[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const long long i = i0 + (long long)k * threads;
        from[k] = nullptr;
        if (i < s.released[N]) {
          const int x = find<N>(s.released, i), keep = (s.wanted[x] + up) >> t.page_shift;
          from[k] = t.table + (size_t)(b0 + x) * t.max_blocks + keep + (i - s.released[x]);
          page[k] = __ldcg(from[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const long long to = n + before_released + i0 + (long long)k * threads;
        if (from[k] == nullptr) continue;
        if (page[k] < 0 || page[k] >= t.P) {
          set_fail(ATTN_ERR_INVALID_ARG);
          page[k] = -1;
        }
        *from[k] = -1;
        if (to < t.P) t.free_pages[to] = page[k];
      }
    }
    // The last end of a request's pages that the stack reaches.
    if (before_need <= top) {
      const long long left = top - before_need;
      served = before_need + (s.need[N] <= left ? s.need[N] : s.need[find<N>(s.need, left)]);
    }
    before_released += s.released[N];
    before_need += s.need[N];
  }
  // Every CTA has read the count and the lengths; what was put on the stack is seen.
  if (threads > N)
    cluster_sync();
  else
    __syncthreads();

  // Lengths and offsets, the pages that are needed, and the tokens' slots.
  const long long bottom = top - served;  // of those pages
  auto stack_at = [&](long long i) {
    const int page = __ldcg(t.free_pages + bottom + i);
    if (page >= 0 && page < t.P) return page;
    set_fail(ATTN_ERR_INVALID_ARG);
    return -1;
  };
  if (first_cta && tid == 0) *t.n_free = (int)bottom;
  before_need = 0;
  long long before_tokens = 0;
  for (int b0 = 0; b0 < t.B; b0 += N) {
    if (!single) s.scan(Move(t, b0 + tid, false));
    auto fits = [&](int x) { return s.need[x + 1] == s.need[x] || before_need + s.need[x + 1] <= served; };
    if (first_cta && b0 + tid < t.B) {
      const int b = b0 + tid;
      t.lens[b] = fits(tid) ? s.wanted[tid] : s.held[tid];
      t.cu[b] = (int)min(before_tokens + s.tokens[tid], (long long)INT_MAX);
      if (b == t.B - 1) {
        const long long all = before_tokens + s.tokens[tid + 1];
        t.cu[t.B] = (int)min(all, (long long)INT_MAX);
        if (all > t.T) set_fail(ATTN_ERR_INVALID_ARG);
      }
    }
    for (long long i0 = gtid; i0 < s.need[N]; i0 += (long long)threads * kAtOnce) {
      int* to[kAtOnce];
      int page[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const long long i = i0 + (long long)k * threads;
        to[k] = nullptr;
        page[k] = -1;
        if (i < s.need[N]) {
          const int x = find<N>(s.need, i), have = (s.held[x] + up) >> t.page_shift;
          to[k] = t.table + (size_t)(b0 + x) * t.max_blocks + have + (i - s.need[x]);
          if (before_need + i < served) page[k] = stack_at(before_need + i);
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (to[k] != nullptr) *to[k] = page[k];
    }
    if (slots_inside) {
      const long long some = min(s.tokens[N], t.T - before_tokens);
      for (long long i0 = gtid; i0 < some; i0 += (long long)threads * kAtOnce) {
        int slot[kAtOnce], pos[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const long long i = i0 + (long long)k * threads;
          slot[k] = pos[k] = -1;
          if (i >= some) continue;
          const int x = find<N>(s.tokens, i), have = (s.held[x] + up) >> t.page_shift;
          pos[k] = s.held[x] + (int)(i - s.tokens[x]);
          if (!fits(x)) continue;
          const int j = pos[k] >> t.page_shift;
          int page;
          if (j >= have) {
            page = stack_at(before_need + s.need[x] + (j - have));
          } else {
            page = __ldcg(t.table + (size_t)(b0 + x) * t.max_blocks + j);
            if (page < 0 || page >= t.P) {
              set_fail(ATTN_ERR_INVALID_ARG);
              page = -1;
            }
          }
          if (page >= 0) slot[k] = (page << t.page_shift) + (pos[k] & up);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const long long i = i0 + (long long)k * threads;
          if (i < some) t.slots[before_tokens + i] = slot[k], t.positions[before_tokens + i] = pos[k];
        }
      }
    }
    before_need += s.need[N];
    before_tokens += s.tokens[N];
  }
  if (slots_inside)
    for (long long i = before_tokens + gtid; i < t.T; i += threads) t.slots[i] = t.positions[i] = -1;
}

// Slots of many tokens, four a thread: a CTA finds the sequences that its tokens belong to, all threads looking at
// once, and takes their offsets and lengths into shared memory.
constexpr int kSlotThreads = 256, kPerCta = 4 * kSlotThreads, kHeld = 1024;
__global__ void __launch_bounds__(kSlotThreads) cache_slots_kernel(const Tables t) {
  __shared__ int s_cu[kHeld + 1], s_held[kHeld], s_lens[kHeld];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  const long long at = (long long)blockIdx.x * kPerCta;
  const int first = (int)at, total = min(__ldcg(t.cu + t.B), t.T);
  const int behind = (int)min(at + kPerCta, (long long)total);  // this CTA's tokens of a sequence: [first, behind)
  int lo = 0, count = 0;
  if (first < behind) {
    // The last sequences that begin at or before the first and the last of them, both at once.
    int from[2] = {0, 0}, n[2] = {t.B, t.B};
    while (n[0] > 1 || n[1] > 1) {
      int step[2];
      bool before[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        step[x] = (n[x] - 1) / kSlotThreads + 1;
        before[x] = tid * step[x] < n[x] && __ldcg(t.cu + from[x] + tid * step[x]) <= (x == 0 ? first : behind - 1);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int skip = (__syncthreads_count(before[x]) - 1) * step[x];
        from[x] += skip;
        n[x] = min(step[x], n[x] - skip);
      }
    }
    lo = from[0];
    count = from[1] - lo + 1;
  }
  const bool held = count <= kHeld;  // else there are many without a token among them
  if (held) {
    for (int i = tid; i < count; i += kSlotThreads) {
      s_cu[i] = __ldcg(t.cu + lo + i);
      s_held[i] = __ldcg(t.held + lo + i);
      s_lens[i] = __ldcg(t.lens + lo + i);
    }
    if (tid == 0 && count > 0) s_cu[count] = __ldcg(t.cu + lo + count);
    __syncthreads();
  }
  auto cu_at = [&](int i) { return held ? s_cu[i] : __ldcg(t.cu + lo + i); };
  const int up = (1 << t.page_shift) - 1;
  const int mine = first + 4 * tid;
  int slot[4], pos[4], x = 0;
  if (mine < behind) {
    int hi = count - 1;
    while (x < hi) {  // the first that ends behind `mine`
      const int mid = (x + hi) >> 1;
      if (cu_at(mid + 1) > mine)
        hi = mid;
      else
        x = mid + 1;
    }
  }
  // The pages of all four are asked for before any is used.
  const int* entry[4];
  int page[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    slot[i] = pos[i] = -1;
    entry[i] = nullptr;
    if (mine + i >= behind) continue;
    while (cu_at(x + 1) <= mine + i) ++x;
    const int before = held ? s_held[x] : __ldcg(t.held + lo + x);
    const int after = held ? s_lens[x] : __ldcg(t.lens + lo + x);
    pos[i] = mine + i - cu_at(x) + before;
    if (after > before)  // served
      entry[i] = t.table + (size_t)(lo + x) * t.max_blocks + (pos[i] >> t.page_shift);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (entry[i] != nullptr) page[i] = __ldcg(entry[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (entry[i] == nullptr) continue;
    if (page[i] >= 0 && page[i] < t.P)
      slot[i] = (page[i] << t.page_shift) + (pos[i] & up);
    else
      set_fail(ATTN_ERR_INVALID_ARG);
  }
  const bool aligned = ((reinterpret_cast<uintptr_t>(t.slots) | reinterpret_cast<uintptr_t>(t.positions)) & 15) == 0;
  if (aligned && at + 4 * tid + 3 < t.T) {
    *reinterpret_cast<int4*>(t.slots + mine) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    *reinterpret_cast<int4*>(t.positions + mine) = make_int4(pos[0], pos[1], pos[2], pos[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + 4 * tid + i < t.T) t.slots[mine + i] = slot[i], t.positions[mine + i] = pos[i];
  }
}

}  // namespace

cudaError_t launch_cache_reserve(const Tables& t, cudaStream_t stream) {
  const long long room = (long long)t.B * t.max_blocks;
  const bool inside = t.T <= kSlotsInside;
  cudaError_t err;
  if (t.B <= kFew && t.T <= kFew * kAtOnce && room <= kAlonePages)
    err = launch_pdl(cache_reserve_kernel<kFew>, dim3(1), dim3(kFew), 0, stream, t, 1);
  else {
    const unsigned ctas = t.T > kAlone || room > kAlonePages ? kMany : 1;
    err = launch_pdl_cluster(cache_reserve_kernel<kThreads>, dim3(ctas), dim3(kThreads), 0, stream, ctas, t,
                             inside ? 1 : 0);
  }
  if (err != cudaSuccess || inside) return err;
  const unsigned blocks = (unsigned)(((long long)t.T + kPerCta - 1) / kPerCta);
  return launch_pdl(cache_slots_kernel, dim3(blocks), dim3(kSlotThreads), 0, stream, t);
}

cudaError_t status_word_tables(void** word) { return cudaGetSymbolAddress(word, g_status_tables); }

}  // namespace attn

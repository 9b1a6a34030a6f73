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
// Nothing is computed but sums, and the bytes are few: what bounds it is the chain of dependent
// loads (lengths, their sums, table entries, stack, slots).  So one launch does it all: a CTA, or
// a cluster of them that work in step where there are many pages or tokens; each scans all
// lengths (1024 at a time) and then takes its share of the pages, found by bisection in the sums.
// Slots of more tokens than a cluster writes quickly are a second kernel's.
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {

static __device__ unsigned int g_status_tables;

namespace {

constexpr int kThreads = 1024;
constexpr int kMany = 8;             // CTAs of a cluster
constexpr int kAlone = 4096;         // tokens, or sequences' pages at most, that one CTA handles
constexpr int kSlotsInside = 65536;  // tokens whose slots the cluster writes
constexpr int kAtOnce = 4;           // pages a thread moves with their loads in flight together

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

// Sum over the CTA's threads before this one; all: over every thread.
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
  long long w = s_warp[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += y;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  return upto - x + (warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

// The last of the kThreads starts that is i or less.
__device__ __forceinline__ int find(const long long* s_start, long long i) {
  int at = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step >>= 1)
    if (s_start[at + step] <= i) at += step;
  return at;
}

// Slot and position of packed token tok, of sequence b.
__device__ __forceinline__ int2 slot_of(const Tables& t, int b, int tok) {
  const int held = __ldcg(t.held + b), pos = tok - __ldcg(t.cu + b) + held;
  int slot = -1;
  if (__ldcg(t.lens + b) > held) {  // served
    const int page = __ldcg(t.table + (size_t)b * t.max_blocks + (pos >> t.page_shift));
    if (page >= 0 && page < t.P)
      slot = (page << t.page_shift) + (pos & ((1 << t.page_shift) - 1));
    else
      set_fail(ATTN_ERR_INVALID_ARG);
  }
  return make_int2(slot, pos);
}
// The sequence of packed token tok < cu[B], among [lo, hi].
__device__ __forceinline__ int sequence_of(const Tables& t, int tok, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(t.cu + mid + 1) > tok)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}
// Four tokens of a lane from `first` on, of sequences [lo, hi].
__device__ __forceinline__ void put_slots(const Tables& t, int first, int total, int lo, int hi) {
  int slot[4], pos[4];
  int b = first < total ? sequence_of(t, first, lo, hi) : 0;
  int until = first < total ? __ldcg(t.cu + b + 1) : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    slot[i] = pos[i] = -1;
    if (first + i < total) {
      while (first + i >= until) until = __ldcg(t.cu + ++b + 1);
      const int2 x = slot_of(t, b, first + i);
      slot[i] = x.x, pos[i] = x.y;
    }
  }
  if (first + 3 < t.T && (reinterpret_cast<uintptr_t>(t.slots) & 15) == 0 &&
      (reinterpret_cast<uintptr_t>(t.positions) & 15) == 0) {
    *reinterpret_cast<int4*>(t.slots + first) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    *reinterpret_cast<int4*>(t.positions + first) = make_int4(pos[0], pos[1], pos[2], pos[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (first + i < t.T) t.slots[first + i] = slot[i], t.positions[first + i] = pos[i];
  }
}

__global__ void __launch_bounds__(kThreads) cache_reserve_kernel(const Tables t, int slots_inside) {
  __shared__ long long s_warp[32], s_start[kThreads];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  const bool first_cta = blockIdx.x == 0;
  const unsigned ctas = cluster_size(), threads = ctas * kThreads;
  const unsigned gtid = blockIdx.x * kThreads + tid;
  int n = __ldcg(t.n_free);
  const Move mine(t, tid, first_cta);  // of the first kThreads sequences
  if (n < 0 || n > t.P) {
    if (first_cta && tid == 0) set_fail(ATTN_ERR_INVALID_ARG);
    n = min(max(n, 0), t.P);
  }
  // Released pages, all of them.
  long long released = 0, sum;
  for (int b0 = 0; b0 < t.B; b0 += kThreads) {
    scan_before((b0 == 0 ? mine : Move(t, b0 + tid, false)).released(), s_warp, sum);
    released += sum;
  }
  const long long full = n + released, top = min(full, (long long)t.P);
  if (full > t.P && first_cta && tid == 0) set_fail(ATTN_ERR_INVALID_ARG);

  // They go on the stack; lengths and offsets.
  long long before_released = 0, before_need = 0, before_tokens = 0, served = 0;
  for (int b0 = 0; b0 < t.B; b0 += kThreads) {
    const Move m = b0 == 0 ? mine : Move(t, b0 + tid, first_cta);
    const long long need = before_need + scan_before(m.need(), s_warp, sum) + m.need();
    before_need += sum;
    const bool fits = m.need() == 0 || need <= top;
    long long upto = fits ? need : 0;
    if (m.need() == 0) upto = 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) upto = max(upto, __shfl_xor_sync(0xffffffffu, upto, off));
    __syncthreads();
    if ((tid & 31) == 0) s_start[tid >> 5] = upto;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) served = max(served, s_start[w]);
    if (first_cta) {
      const long long at = before_tokens + scan_before(m.tokens(), s_warp, sum);
      before_tokens += sum;
      if (b0 + tid < t.B) {
        t.lens[b0 + tid] = fits ? m.wanted : m.held;
        t.cu[b0 + tid] = (int)min(at, (long long)INT_MAX);
        if (b0 + tid == t.B - 1) {
          const long long all = at + m.tokens();
          t.cu[t.B] = (int)min(all, (long long)INT_MAX);
          if (all > t.T) set_fail(ATTN_ERR_INVALID_ARG);
        }
      }
    }
    const long long start = scan_before(m.released(), s_warp, sum);
    __syncthreads();
    s_start[tid] = start;
    __syncthreads();
    for (long long i0 = gtid; i0 < sum; i0 += (long long)threads * kAtOnce) {
      int* from[kAtOnce];
      int page[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const long long i = i0 + (long long)k * threads;
        from[k] = nullptr;
        if (i < sum) {
          const int x = find(s_start, i), b = b0 + x;
          const int keep = (__ldcg(t.wanted + b) + (1 << t.page_shift) - 1) >> t.page_shift;
          from[k] = t.table + (size_t)b * t.max_blocks + keep + (i - s_start[x]);
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
    before_released += sum;
  }
  cluster_sync();

  // The pages that are needed.
  before_need = 0;
  for (int b0 = 0; b0 < t.B; b0 += kThreads) {
    const Move m = b0 == 0 ? mine : Move(t, b0 + tid, false);
    const long long start = scan_before(m.need(), s_warp, sum);
    __syncthreads();
    s_start[tid] = start;
    __syncthreads();
    for (long long i0 = gtid; i0 < sum; i0 += (long long)threads * kAtOnce) {
      int* to[kAtOnce];
      int page[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const long long i = i0 + (long long)k * threads;
        to[k] = nullptr;
        page[k] = -1;
        if (i < sum) {
          const int x = find(s_start, i), b = b0 + x;
          const int have = (__ldcg(t.held + b) + (1 << t.page_shift) - 1) >> t.page_shift;
          to[k] = t.table + (size_t)b * t.max_blocks + have + (i - s_start[x]);
          // A request's pages are served if its last one is: those up to `served`.
          const long long at = before_need + i;
          if (at < served) {
            page[k] = __ldcg(t.free_pages + (top - served + at));
            if (page[k] < 0 || page[k] >= t.P) {
              set_fail(ATTN_ERR_INVALID_ARG);
              page[k] = -1;
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (to[k] != nullptr) *to[k] = page[k];
    }
    before_need += sum;
  }
  if (first_cta && tid == 0) *t.n_free = (int)(top - served);
  if (!slots_inside) return;
  cluster_sync();
  const int total = min(__ldcg(t.cu + t.B), t.T);
  for (unsigned i = gtid; i < ((unsigned)t.T + 3) / 4; i += threads) put_slots(t, 4 * i, total, 0, t.B - 1);
}

// Slots of many tokens: a warp takes kPerWarp of them, whose sequences it bounds first.
constexpr int kSlotThreads = 256, kPerWarp = 512;
__global__ void __launch_bounds__(kSlotThreads) cache_slots_kernel(const Tables t) {
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long at = ((long long)blockIdx.x * (kSlotThreads / 32) + warp) * kPerWarp;
  if (at >= t.T) return;
  const int first = (int)at, total = min(__ldcg(t.cu + t.B), t.T);
  int lo = 0, hi = t.B - 1;
  if (first < total) {
    // Lanes 0 and 1 find the sequences of the first and the last token.
    const int x = sequence_of(t, lane == 0 ? first : (int)min(at + kPerWarp, (long long)total) - 1, 0, t.B - 1);
    lo = __shfl_sync(0xffffffffu, x, 0);
    hi = __shfl_sync(0xffffffffu, x, 1);
  }
#pragma unroll 1
  for (int i = 4 * lane; i < kPerWarp; i += 128)
    if (at + i < t.T) put_slots(t, first + i, total, lo, hi);
}

}  // namespace

cudaError_t launch_cache_reserve(const Tables& t, cudaStream_t stream) {
  const bool many = t.T > kAlone || (long long)t.B * t.max_blocks > kAlone;
  const bool inside = t.T <= kSlotsInside;
  const unsigned ctas = many ? kMany : 1;
  cudaError_t err =
      launch_pdl_cluster(cache_reserve_kernel, dim3(ctas), dim3(kThreads), 0, stream, ctas, t, inside ? 1 : 0);
  if (err != cudaSuccess || inside) return err;
  const unsigned blocks = (unsigned)(((long long)t.T + kSlotThreads / 32 * kPerWarp - 1) / (kSlotThreads / 32 * kPerWarp));
  return launch_pdl(cache_slots_kernel, dim3(blocks), dim3(kSlotThreads), 0, stream, t);
}

cudaError_t status_word_tables(void** word) { return cudaGetSymbolAddress(word, g_status_tables); }

}  // namespace attn

// The pages of the paged cache: block tables and slots from the requests' lengths, on the GPU.
//
// Sequence b grows by new_lens[b] tokens (shrinks by them where negative).  The pages it needs come off a stack of
// free ones, the pages it gives back go onto it, in the order of the sequences, so that a call which takes back what
// the call before gave leaves the stack as it was.  Sums over the sequences before decide who takes what, so the result
// does not depend on the order in which threads run.
//
// Latency is all that counts: a step of a serving loop moves a few pages of a few hundred sequences.  One block, a
// thread a sequence, 1024 at a time: one scan over their pages, then every thread fetches its sequence's pages (a warp, where
// there are more than two) and slots, whose pages come from the stack or the table as it was, so that nothing waits
// for the table's new entries.  What is overwritten in place is the block's own, and barriers are enough.  (Measured: a cluster
// of up to eight blocks, three scans and slots from the new table took 4.8 us a call of 64 sequences, this 2.8.)  Slots of
// many tokens are a second kernel over all SMs.
#include "internal.h"
#include "ptx.cuh"

namespace fattn {
namespace {

constexpr int kThreads = 1024;
constexpr int kOwn = 2;                // pages of a sequence that its thread moves itself
constexpr long long kFewSlots = 4096;  // slots that the first kernel writes itself

static_assert(kThreads == 32 * 32, "a warp of warps");

// Inclusive sums of x and y over the block's threads; *all: over all of them.
__device__ __forceinline__ int2 block_scan(int2 v, int2* warps, int2* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) v.x += x, v.y += y;
  }
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  // (the warps' sums, added up by every warp for itself)
  int2 sum = warps[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, sum.x, o), y = __shfl_up_sync(0xffffffffu, sum.y, o);
    if (lane >= o) sum.x += x, sum.y += y;
  }
  int2 total, before;
  total.x = __shfl_sync(0xffffffffu, sum.x, 31);
  total.y = __shfl_sync(0xffffffffu, sum.y, 31);
  before.x = __shfl_sync(0xffffffffu, sum.x, warp - 1 & 31);
  before.y = __shfl_sync(0xffffffffu, sum.y, warp - 1 & 31);
  if (warp == 0) before = make_int2(0, 0);
  *all = total;
  return make_int2(before.x + v.x, before.y + v.y);
}

// A sequence's change: `had` pages of `len` tokens become `want` (if there is room in its table).
struct Change {
  int len = 0, more = 0, had = 0, want = 0;
  __device__ __forceinline__ Change() {}
  __device__ __forceinline__ Change(const PagesLaunch& a, int now, int change) {
    const int room = a.max_pages * a.page_size;  // (the host keeps it within an int)
    len = min(max(now, 0), room);
    more = max(change, -len);
    had = pages(len, a.page_size);
    if (static_cast<long long>(len) + more > room) more = 0;
    want = pages(len + more, a.page_size);
  }
  static __device__ __forceinline__ int pages(int n, int size) { return n / size + (n % size ? 1 : 0); }
};

__device__ __forceinline__ long long slot_of(const PagesLaunch& a, int id, int key) {
  return id >= 0 && id < a.num_pages ? static_cast<long long>(id) * a.page_size + key % a.page_size : -1;
}

template <bool SLOTS>
__global__ void __launch_bounds__(kThreads) pages_kernel(const PagesLaunch a) {
  __shared__ int2 warps[kThreads / 32];
  // of the chunk's sequences: length before, tokens granted, pages before; pages to move, the first's place in the
  // stack's order
  __shared__ int sh_len[kThreads], sh_granted[kThreads], sh_had[kThreads], sh_moved[kThreads], sh_start[kThreads];
  __shared__ int sh_got;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  grid_dep_launch();
  grid_dep_wait();
  const int n_free = a.n_free[0];
  int free = 0;
  long long wanted = 0;  // pages that the chunks before asked for
  int taken = 0, given = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid, end = min(kThreads, a.B - b0);
    const Change c = tid < end ? Change(a, a.seq_lens[b], a.new_lens[b]) : Change();
    const int take = max(c.want - c.had, 0);
    int2 all;
    if (tid == 0) sh_got = 0;
    const int2 last = block_scan(make_int2(take, max(c.had - c.want, 0)), warps, &all);
    free = min(max(n_free, 0), a.num_pages);
    const bool ok = wanted + last.x <= free;  // (false for every later one that wants pages, once it is)
    const int granted = take > 0 && !ok ? 0 : c.more, mine = ok ? take : 0;
    const int start = static_cast<int>(wanted) + last.x - take;
    int* const row = a.block_table + static_cast<long long>(b) * a.max_pages + c.had;
    sh_len[tid] = c.len;
    sh_granted[tid] = granted;
    sh_had[tid] = c.had;
    sh_moved[tid] = mine;
    sh_start[tid] = start;
    if (wanted + all.x > free && mine > 0) atomicMax(&sh_got, last.x);
    const bool more_pages = __syncthreads_or(mine > kOwn);
    const int got = wanted + all.x <= free ? all.x : sh_got;
    if (tid < end) a.granted[b] = granted;
    if (more_pages) {
      for (int i = warp; i < end; i += kThreads / 32) {
        const int n = sh_moved[i], top = free - 1 - sh_start[i];
        int* const to = a.block_table + static_cast<long long>(b0 + i) * a.max_pages + sh_had[i];
#pragma unroll 4
        for (int k = lane; k < n; k += 32) to[k] = a.free_pages[top - k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < kOwn; ++k)
        if (k < mine) row[k] = a.free_pages[free - 1 - start - k];
    }
    if constexpr (SLOTS) {
#pragma unroll 2
      for (int e = tid; e < end * a.N; e += kThreads) {
        const int i = e / a.N, t = e - i * a.N, key = sh_len[i] + t;
        long long slot = -1;
        if (t < sh_granted[i]) {
          const int p = key / a.page_size, extra = p - sh_had[i];
          slot = slot_of(a, extra >= 0 ? a.free_pages[free - 1 - sh_start[i] - extra]
                                       : a.block_table[static_cast<long long>(b0 + i) * a.max_pages + p], key);
        }
        a.slots[static_cast<long long>(b0) * a.N + e] = slot;
      }
    }
    wanted = min(wanted + all.x, static_cast<long long>(free) + 1);  // (beyond that nothing is served)
    taken += got;
    given += all.y;
    if (a.B > kThreads || given > 0) __syncthreads();  // the chunk's sums, the stack and the lengths have been read
    if (a.B <= kThreads && tid < end) a.seq_lens[b] = c.len + granted;
    if (a.B <= kThreads && given > 0) {  // (one chunk: its changes are at hand)
      sh_had[tid] = c.want;
      sh_moved[tid] = max(c.had - c.want, 0);
      sh_start[tid] = last.y - sh_moved[tid];
    }
  }
  // Pages given back: the first sequence's first lies on top at the end.
  if (given > 0 || a.B > kThreads) {
    const int top = free - taken + given - 1;
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int b = b0 + tid, end = min(kThreads, a.B - b0);
      if (a.B > kThreads) {
        const Change c = tid < end ? Change(a, a.seq_lens[b], a.new_lens[b]) : Change();
        const int give = max(c.had - c.want, 0);
        int2 all;
        const int2 last = block_scan(make_int2(give, 0), warps, &all);
        sh_had[tid] = c.want;
        sh_moved[tid] = give;
        sh_start[tid] = before + last.x - give;
        before += all.x;
        if (tid < end) a.seq_lens[b] = c.len + a.granted[b];
      }
      auto move = [&](int* from, int at, int k) {
        if (at - k < a.num_pages) a.free_pages[at - k] = from[k];  // (more than there are: a page given back twice)
        from[k] = -1;
      };
      const int mine = sh_moved[tid];
      const bool more_pages = __syncthreads_or(mine > kOwn);
      if (more_pages) {
        for (int i = warp; i < end; i += kThreads / 32) {
          const int n = sh_moved[i], at = top - sh_start[i];
          int* const from = a.block_table + static_cast<long long>(b0 + i) * a.max_pages + sh_had[i];
#pragma unroll 4
          for (int k = lane; k < n; k += 32) move(from, at, k);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
          if (k < mine) move(a.block_table + static_cast<long long>(b) * a.max_pages + sh_had[tid], top - sh_start[tid], k);
      }
      __syncthreads();
    }
  }
  if (tid == 0) a.n_free[0] = min(free - taken + given, a.num_pages);
}

// Slots of many tokens, after pages_kernel: blockIdx.x = sequence * blocks a sequence + block.
constexpr int kSlotThreads = 256, kSlotsPerThread = 4;

__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const PagesLaunch a, int per_seq) {
  const int b = static_cast<int>(blockIdx.x) / per_seq;
  const int t0 = (static_cast<int>(blockIdx.x) % per_seq) * (kSlotThreads * kSlotsPerThread) + static_cast<int>(threadIdx.x);
  grid_dep_wait();
  const int granted = a.granted[b], len = a.seq_lens[b] - max(granted, 0);  // (seq_lens: as they are now)
  const int* const row = a.block_table + static_cast<long long>(b) * a.max_pages;
  long long* const out = a.slots + static_cast<long long>(b) * a.N;
  long long s[kSlotsPerThread];
#pragma unroll
  for (int i = 0; i < kSlotsPerThread; ++i) {
    const int t = t0 + i * kSlotThreads;
    s[i] = t < granted ? slot_of(a, row[(len + t) / a.page_size], len + t) : -1;
  }
#pragma unroll
  for (int i = 0; i < kSlotsPerThread; ++i)
    if (t0 + i * kSlotThreads < a.N) out[t0 + i * kSlotThreads] = s[i];
}

}  // namespace

cudaError_t launch_pages(const PagesLaunch& a, cudaStream_t stream) {
  const bool few = a.slots && static_cast<long long>(a.B) * a.N <= kFewSlots;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, few ? pages_kernel<true> : pages_kernel<false>, a);
  if (e != cudaSuccess || !a.slots || few) return e;
  const int per_seq = (a.N + kSlotThreads * kSlotsPerThread - 1) / (kSlotThreads * kSlotsPerThread);
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * static_cast<unsigned>(per_seq));
  cfg.blockDim = dim3(kSlotThreads);
  return cudaLaunchKernelEx(&cfg, slots_kernel, a, per_seq);
}

}  // namespace fattn

// The pages of the paged cache: block tables and slots from the requests' lengths, on the GPU.
//
// Sequence b grows by new_lens[b] tokens (shrinks by them where negative).  The pages it needs come off a stack of
// free ones, the pages it gives back go onto it, in the order of the sequences, so that a call which takes back what
// the call before gave leaves the stack as it was.  Sums over the sequences before decide who takes what, so the result
// does not depend on the order in which threads run.
//
// Latency is all that counts: a step of a serving loop moves a few pages of a few hundred sequences.  One kernel, of
// one block, or of up to eight that are a thread-block cluster where there are more sequences: every block makes
// the sums over all sequences itself and writes every S-th sequence's entries, and cluster barriers keep what is
// overwritten in place (the stack, the lengths) until all have read it.  Slots of many tokens are a second kernel over
// all SMs.
#include "internal.h"
#include "ptx.cuh"

namespace fattn {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;
constexpr long long kFewSlots = 8192;  // slots that the first kernel writes itself

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The sum of v over the block's threads up to and with this one; *all: over all of them.
__device__ __forceinline__ int block_scan(int v, int* warps, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // (the sums of the call before have been read)
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    before += i < warp ? warps[i] : 0;
    total += warps[i];
  }
  *all = total;
  return before + v;
}

// A sequence's change: `had` pages of `len` tokens become `want` (if there is room in its table).
struct Change {
  int len, more, had, want;
  __device__ __forceinline__ Change(const PagesLaunch& a, int b) {
    const long long room = static_cast<long long>(a.max_pages) * a.page_size;
    len = static_cast<int>(min(static_cast<long long>(max(a.seq_lens[b], 0)), room));
    more = max(a.new_lens[b], -len);
    had = pages(len, a.page_size);
    if (static_cast<long long>(len) + more > room) more = 0;
    want = pages(len + more, a.page_size);
  }
  static __device__ __forceinline__ int pages(int n, int size) { return n / size + (n % size ? 1 : 0); }
};

// Token t of a sequence that had `len`: its row in the pools, or -1.
__device__ __forceinline__ long long slot_of(const PagesLaunch& a, long long b, int len, int t, int granted) {
  if (t >= granted) return -1;
  const int key = len + t, i = key / a.page_size;
  const int id = __ldcg(a.block_table + b * a.max_pages + i);  // (written by another block, perhaps)
  return id >= 0 && id < a.num_pages ? static_cast<long long>(id) * a.page_size + (key - i * a.page_size) : -1;
}

template <bool SLOTS>
__global__ void __launch_bounds__(kThreads) pages_kernel(const PagesLaunch a) {
  __shared__ int warps[kThreads / 32];
  __shared__ int sh_start[kThreads], sh_from[kThreads], sh_count[kThreads];
  const int S = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_launch();
  grid_dep_wait();
  const int free = min(max(a.n_free[0], 0), a.num_pages);
  // Pages handed out, from the top of the stack down.
  long long wanted = 0;
  int taken = 0, given = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int take = 0, give = 0, from = 0, more = 0;
    if (b < a.B) {
      const Change c(a, b);
      take = max(c.want - c.had, 0);
      give = max(c.had - c.want, 0);
      from = c.had;
      more = c.more;
    }
    int all;
    const int last = block_scan(take, warps, &all);
    const bool ok = wanted + last <= free;  // (false for every later one that wants pages, once it is)
    sh_start[threadIdx.x] = static_cast<int>(wanted) + last - take;
    sh_from[threadIdx.x] = from;
    sh_count[threadIdx.x] = ok ? take : 0;
    wanted += all;
    if (b < a.B && static_cast<int>(threadIdx.x) % S == rank) a.granted[b] = take > 0 && !ok ? 0 : more;
    int got, back;
    block_scan(ok ? take : 0, warps, &got);
    block_scan(give, warps, &back);
    taken += got;
    given += back;
    if (got > 0) {  // (the scans' barriers order sh_ before these reads)
      const int end = min(kThreads, a.B - b0);
      for (int i = rank + S * warp; i < end; i += S * (kThreads / 32)) {
        const int n = sh_count[i], top = free - 1 - sh_start[i];
        int* const row = a.block_table + static_cast<long long>(b0 + i) * a.max_pages + sh_from[i];
#pragma unroll 4
        for (int k = lane; k < n; k += 32) row[k] = a.free_pages[top - k];
      }
      __syncthreads();
    }
    if (wanted > free) wanted = static_cast<long long>(free) + 1;  // (no more: keep it from growing)
  }
  cluster_sync();  // the stack has been read, the table is filled, all that was granted is known
  if constexpr (SLOTS) {
    const long long total = static_cast<long long>(a.B) * a.N;
    for (long long e = rank * kThreads + threadIdx.x; e < total; e += S * kThreads) {
      const int b = static_cast<int>(e / a.N);
      const int room = static_cast<int>(min(static_cast<long long>(a.max_pages) * a.page_size, 0x7fffffffll));
      a.slots[e] = slot_of(a, b, min(max(a.seq_lens[b], 0), room), static_cast<int>(e - static_cast<long long>(b) * a.N),
                           __ldcg(a.granted + b));
    }
  }
  if (given > 0) {
    // Pages given back: the first sequence's first lies on top at the end.
    const int top = free - taken + given - 1;
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      int give = 0, from = 0;
      if (b < a.B) {
        const Change c(a, b);
        give = max(c.had - c.want, 0);
        from = c.want;
      }
      int all;
      const int last = block_scan(give, warps, &all);
      sh_start[threadIdx.x] = before + last - give;
      sh_from[threadIdx.x] = from;
      sh_count[threadIdx.x] = give;
      before += all;
      __syncthreads();
      const int end = min(kThreads, a.B - b0);
      for (int i = rank + S * warp; i < end; i += S * (kThreads / 32)) {
        const int n = sh_count[i], at = top - sh_start[i];
        int* const row = a.block_table + static_cast<long long>(b0 + i) * a.max_pages + sh_from[i];
#pragma unroll 4
        for (int k = lane; k < n; k += 32) {
          if (at - k < a.num_pages) a.free_pages[at - k] = row[k];  // (more than there are: a page given back twice)
          row[k] = -1;
        }
      }
      __syncthreads();
    }
  }
  cluster_sync();  // the lengths have been read
  for (int b = static_cast<int>(threadIdx.x); b < a.B; b += kThreads)
    if (b % kThreads % S == rank) a.seq_lens[b] = Change(a, b).len + a.granted[b];
  if (rank == 0 && threadIdx.x == 0) a.n_free[0] = min(free - taken + given, a.num_pages);
}

// Slots of many tokens, after pages_kernel: blockIdx.x = sequence * blocks a sequence + block.
constexpr int kSlotThreads = 256, kSlotsPerThread = 4;

__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const PagesLaunch a, int per_seq) {
  const int b = static_cast<int>(blockIdx.x) / per_seq;
  const int t0 = (static_cast<int>(blockIdx.x) % per_seq) * (kSlotThreads * kSlotsPerThread) + static_cast<int>(threadIdx.x);
  grid_dep_wait();
  const int granted = a.granted[b], len = a.seq_lens[b] - max(granted, 0);  // (seq_lens: as they are now)
  long long* const out = a.slots + static_cast<long long>(b) * a.N;
  long long s[kSlotsPerThread];
#pragma unroll
  for (int i = 0; i < kSlotsPerThread; ++i) s[i] = slot_of(a, b, len, t0 + i * kSlotThreads, granted);
#pragma unroll
  for (int i = 0; i < kSlotsPerThread; ++i)
    if (t0 + i * kSlotThreads < a.N) out[t0 + i * kSlotThreads] = s[i];
}

}  // namespace

cudaError_t launch_pages(const PagesLaunch& a, cudaStream_t stream) {
  const bool few = a.slots && static_cast<long long>(a.B) * a.N <= kFewSlots;
  int blocks = 1;
  while (blocks < kMaxCluster && blocks * 16 < a.B) blocks *= 2;  // 16 warps a block, a sequence each
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, few ? pages_kernel<true> : pages_kernel<false>, a);
  if (e != cudaSuccess || !a.slots || few) return e;
  const int per_seq = (a.N + kSlotThreads * kSlotsPerThread - 1) / (kSlotThreads * kSlotsPerThread);
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * static_cast<unsigned>(per_seq));
  cfg.blockDim = dim3(kSlotThreads);
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, slots_kernel, a, per_seq);
}

}  // namespace fattn

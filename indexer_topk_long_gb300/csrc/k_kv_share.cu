// k_kv_share.cu -- which pages the sequences of a group have in common.
//
// A group's sharing sequences are those whose page table begins like the lead's, the first of the
// group with a page to share; what they share is the shortest of these beginnings, cut to whole
// pages that every query of theirs sees (so the shared part needs no mask).  What comes out are the
// batches of the two steps of the attention: the shared part with all of a group's queries in the
// lead's place, and each sequence's rest.  Found here and not taken from the caller, so that the
// results are those of the plain attention whatever the tables hold.
//
// One CTA a sequence compares its row of the table; the last of them makes the batches.  Bound by
// latency: 128 sequences of 520 pages add 6.5 us to what follows, of which the loads' way to memory, the
// count of CTAs that are done and the last one's scan are three waits in turn.
#include "kv_internal.cuh"

namespace ltk {
namespace {

constexpr int kThreads = 256;

// Whole pages that every query of sequence b sees, 0 for one without queries or tokens.
__device__ __forceinline__ int pages_seen(const ShareParams& p, int b) {
  const KvSeq s = kv_seq(p.batch, p.cache, b);
  if (s.nq <= 0) return 0;
  return max(min(s.pos0, s.len - 1), 0) >> p.cache.page_log2;
}

// First sequence of group g (that of group num_groups: the number of sequences).
__device__ __forceinline__ int first_of(const ShareParams& p, int g) {
  return p.groups == nullptr ? (g == 0 ? 0 : p.batch.B) : kv_load(p.groups + g);
}

// Group of sequence b: the last g whose first sequence is not behind b.
__device__ __forceinline__ int group_of(const ShareParams& p, int b) {
  int lo = 0, hi = p.num_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_of(p, mid) <= b) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Whether this thread's groups rise from 0 to the number of sequences.
__device__ __forceinline__ bool groups_rise(const ShareParams& p, int g0, int step) {
  bool rises = true;
  for (int g = g0; g < p.num_groups; g += step) {
    const int at = first_of(p, g), to = first_of(p, g + 1);
    rises = rises && at >= 0 && at <= to && to <= p.batch.B && (g > 0 || at == 0) && (g + 1 < p.num_groups || to == p.batch.B);
  }
  return rises;
}

// Nothing but that, where all is attended to in one step.
__global__ void __launch_bounds__(kThreads) kv_groups_kernel(const ShareParams p) {
  begin_after_previous();
  const bool rises = groups_rise(p, threadIdx.x, kThreads);
  if (__syncthreads_or(rises ? 0 : 1) != 0 && threadIdx.x == 0) raise_status(p.status, kDevArg);
}

// One thread block's results for groups that its shared memory holds; beyond, in the workspace.
constexpr int kHeld = 1024;

__global__ void __launch_bounds__(kThreads) kv_share_kernel(const ShareParams p) {
  __shared__ int found;
  __shared__ int last;
  __shared__ int held[3][kHeld];
  const int tid = threadIdx.x, b = blockIdx.x, B = p.batch.B;
  begin_after_previous();
  {
    const int g = group_of(p, b);
    const int b0 = max(first_of(p, g), 0);
    const int seen = pages_seen(p, b);
    // the lead is b itself or before it
    if (tid == 0) found = b;
    __syncthreads();
    for (int x0 = b0; x0 < b; x0 += kThreads) {
      const bool on = x0 + tid < b && pages_seen(p, x0 + tid) > 0;
      if (on) atomicMin(&found, x0 + tid);
      if (__syncthreads_or(on ? 1 : 0)) break;
    }
    const int lead = found;
    int same = seen;
    if (lead != b && seen > 0) {
      const int most = min(seen, pages_seen(p, lead));
      const int* mine = p.batch.page_table + static_cast<size_t>(b) * p.batch.width;
      const int* its = p.batch.page_table + static_cast<size_t>(lead) * p.batch.width;
      int end = most;
      constexpr int kAhead = 8;          // a row's numbers in flight, for the latency
      for (int i0 = tid; i0 < end; i0 += kThreads * kAhead) {
        int x[kAhead], y[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int i = i0 + j * kThreads;
          x[j] = i < most ? kv_load(mine + i) : 0;
          y[j] = i < most ? kv_load(its + i) : 0;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (x[j] != y[j]) end = min(end, i0 + j * kThreads);
      }
      __syncthreads();
      if (tid == 0) found = most;
      __syncthreads();
      if (end < most) atomicMin(&found, end);
      __syncthreads();
      same = found;
    }
    if (tid == 0) {
      p.common[b] = same;
      __threadfence();
      last = atomicAdd(p.counter, 1) == B - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (tid == 0) *p.counter = 0;
  const bool few = p.num_groups <= kHeld;
  int* leads = few ? held[0] : p.lead;
  int* least = few ? held[1] : p.least;
  int* sharing = few ? held[2] : p.sharing;
  const bool rises = groups_rise(p, tid, kThreads);
  for (int g = tid; g < p.num_groups; g += kThreads) {
    leads[g] = B;
    least[g] = p.batch.width;
    sharing[g] = 0;
  }
  const bool wrong = __syncthreads_or(rises ? 0 : 1) != 0;
  if (wrong) {                           // nothing is shared
    if (tid == 0) raise_status(p.status, kDevArg);
    for (int x = tid; x <= B; x += kThreads) {
      p.cu[x] = 0;
      if (x < B) p.start[x] = p.lens[x] = 0;
    }
    return;
  }
  for (int x = tid; x < B; x += kThreads) {
    const int n = __ldcg(p.common + x);
    if (n == 0) continue;
    const int g = group_of(p, x);
    atomicMin(leads + g, x);
    atomicMin(least + g, n);
    atomicAdd(sharing + g, 1);
  }
  __threadfence_block();
  __syncthreads();
  for (int x = tid; x <= B; x += kThreads) {
    const int g = group_of(p, min(x, B - 1));
    const int b0 = first_of(p, g), b1 = first_of(p, g + 1);
    auto of = [&](int* of_group) { return *static_cast<volatile int*>(of_group + g); };
    const bool shares = of(sharing) > 1;
    const int lead = shares ? of(leads) : b0;
    const int tokens = shares ? of(least) << p.cache.page_log2 : 0;
    p.cu[x] = min(max(kv_load(p.batch.cu_q + (x <= lead ? b0 : b1)), 0), p.batch.N);
    if (x < B) {
      p.start[x] = __ldcg(p.common + x) > 0 ? tokens : 0;
      p.lens[x] = x == lead ? tokens : 0;
    }
  }
}

}  // namespace

cudaError_t launch_kv_groups(const ShareParams& p, cudaStream_t stream) {
  count_launches(1);
  return launch_overlapped(kv_groups_kernel, 1, kThreads, 0, stream, p);
}

cudaError_t launch_kv_share(const ShareParams& p, cudaStream_t stream) {
  count_launches(1);
  return launch_overlapped(kv_share_kernel, p.batch.B, kThreads, 0, stream, p);
}

}  // namespace ltk

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
// latency: 128 sequences of 520 pages take 4 us, 16 of 4128 pages 5.
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

__global__ void __launch_bounds__(kThreads) kv_share_kernel(const ShareParams p) {
  __shared__ int found;
  __shared__ int last;
  const int tid = threadIdx.x, b = blockIdx.x, B = p.batch.B;
  begin_after_previous();
  {
    const int g = group_of(p, b);
    const int b0 = max(first_of(p, g), 0);
    const int seen = pages_seen(p, b);
    // the lead is b itself or before it
    if (tid == 0) found = b;
    __syncthreads();
    for (int x = b0 + tid; x < b; x += kThreads)
      if (pages_seen(p, x) > 0) {
        atomicMin(&found, x);
        break;
      }
    __syncthreads();
    const int lead = found;
    __syncthreads();
    int same = seen;
    if (lead != b && seen > 0) {
      if (tid == 0) found = min(seen, pages_seen(p, lead));
      __syncthreads();
      const int most = found;
      const int* mine = p.batch.page_table + static_cast<size_t>(b) * p.batch.width;
      const int* its = p.batch.page_table + static_cast<size_t>(lead) * p.batch.width;
      int end = most;
      for (int i = tid; i < most; i += kThreads)
        if (kv_load(mine + i) != kv_load(its + i)) {
          end = i;
          break;
        }
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
  bool rises = true;
  for (int g = tid; g < p.num_groups; g += kThreads) {
    const int at = first_of(p, g), to = first_of(p, g + 1);
    rises = rises && at >= 0 && at <= to && to <= B && (g > 0 || at == 0) && (g + 1 < p.num_groups || to == B);
    p.lead[g] = B;
    p.least[g] = p.batch.width;
    p.sharing[g] = 0;
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
    atomicMin(p.lead + g, x);
    atomicMin(p.least + g, n);
    atomicAdd(p.sharing + g, 1);
  }
  __syncthreads();
  for (int x = tid; x <= B; x += kThreads) {
    const int g = group_of(p, min(x, B - 1));
    const int b0 = first_of(p, g), b1 = first_of(p, g + 1);
    const bool shares = __ldcg(p.sharing + g) > 1;
    const int lead = shares ? __ldcg(p.lead + g) : b0;
    const int tokens = shares ? __ldcg(p.least + g) << p.cache.page_log2 : 0;
    p.cu[x] = min(max(kv_load(p.batch.cu_q + (x <= lead ? b0 : b1)), 0), p.batch.N);
    if (x < B) {
      p.start[x] = __ldcg(p.common + x) > 0 ? tokens : 0;
      p.lens[x] = x == lead ? tokens : 0;
    }
  }
}

}  // namespace

cudaError_t launch_kv_share(const ShareParams& p, cudaStream_t stream) {
  count_launches(1);
  return launch_overlapped(kv_share_kernel, p.batch.B, kThreads, 0, stream, p);
}

}  // namespace ltk

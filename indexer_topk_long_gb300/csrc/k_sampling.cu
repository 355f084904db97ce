// k_sampling.cu -- a token for each row of logits, from a given random number.
//
//   w_i = 2^((x_i - max) log2(e) / T)        tokens ordered by (x descending, index ascending)
//   min-p: keep w_i >= min_p;  top-k: of these the first k;  top-p: of these the fewest first ones
//   whose weights reach p of their total;  token: the first kept one, in the order of the
//   vocabulary, at which the running sum of kept weights exceeds u * total.
//
// Which token that is depends on sums over a whole vocabulary being right to far better than one
// token's share, so weights are whole numbers in units of 2^-44 of the largest, right to 2^-32 of
// themselves, and every sum of them is exact in 64 bits, in any order: the result does not depend
// on how a row is split.  (fp32 weights would put one in a hundred draws from a flat vocabulary of
// 100000 on the neighbouring token.)
//
// A cluster of 1 to 8 CTAs holds a row in its shared memory, so that logits are read once; what has
// to be known of the whole row (maximum, counts, sums) goes from CTA to CTA through distributed
// shared memory.  Small top-k: each thread's largest element gives a bound that k elements reach,
// the few at or above it go to one CTA, which sorts them and finishes.  Else the cut is found by
// histograms over ever smaller ranges of x, of counts (top-k) or weights (top-p), until what is
// left can be sorted; the draw then takes one pass over the row.
#include <cooperative_groups.h>

#include <atomic>

#include "block_sort.cuh"
#include "kv_internal.cuh"
#include "sampling_internal.cuh"

namespace ltk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kBins = 1024;
constexpr int kList = 2048;              // elements that one CTA sorts
constexpr int kUnitBits = 44;            // weights are in units of 2^-44
constexpr uint32_t kNoCut = 0xFFFFFFFFu;

// 2^(j / 256) in units of 2^-30, rounded: by the exponential series in double, at compile time.
struct PowTable {
  uint32_t v[256];
};
constexpr PowTable make_pow_table() {
  PowTable t{};
  for (int j = 0; j < 256; ++j) {
    const double z = j * (0.693147180559945309417232 / 256.0);
    double term = 1.0, sum = 1.0;
    for (int i = 1; i < 30; ++i) {
      term *= z / i;
      sum += term;
    }
    t.v[j] = static_cast<uint32_t>(sum * 1073741824.0 + 0.5);
  }
  return t;
}
__device__ constexpr PowTable kPow = make_pow_table();

struct Shared {
  uint32_t pow[256];
  // what the CTAs of a cluster tell one another, by rank; two sets in turn where there is a next time
  float top[kMaxCtas], bound[2][kMaxCtas];
  int bad[kMaxCtas];
  unsigned long long mass[2][kMaxCtas];
  float lo[2][kMaxCtas], hi[2][kMaxCtas];
  uint32_t count[2][kMaxCtas];
  unsigned long long answer;
  // a CTA's own
  unsigned long long warp_sum[kWarps];
  float warp_a[kWarps], warp_b[kWarps];
  uint32_t warp_n[kWarps];
  uint32_t listed;
  uint32_t found;
  float reached[2];
  float min_hi, min_lo;                  // T ln(min_p)
  unsigned long long found_before;
  union {
    struct {
      uint32_t hist[3][kBins];           // counts, or weights in pieces of 15, 15 and 15 bits
      unsigned long long merged[kBins];
    };
    unsigned long long weights[kList];   // of a sorted list
  };
  unsigned long long list[kList];
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Elements of 16 bytes to fp32.
template <typename E>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[16 / sizeof(E)]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = kv_unpack16(w[i], std::is_same<E, __nv_bfloat16>::value);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// The largest of many elements, two at a time where they are of 16 bits; NaN if any is.
template <typename E>
struct Largest {
  uint32_t v = std::is_same<E, float>::value ? 0xFF800000u : std::is_same<E, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
  __device__ __forceinline__ void one(uint32_t w) {
    if constexpr (std::is_same<E, float>::value) {
      float m = __uint_as_float(v);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(__uint_as_float(w)));
      v = __float_as_uint(m);
    }
    else if constexpr (std::is_same<E, __half>::value) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(v) : "r"(w));
    else asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(w));
  }
  __device__ __forceinline__ void add(const uint4& w) {
    one(w.x);
    one(w.y);
    one(w.z);
    one(w.w);
  }
  __device__ __forceinline__ float get() const {
    if constexpr (std::is_same<E, float>::value) return __uint_as_float(v);
    const float2 f = kv_unpack16(v, std::is_same<E, __nv_bfloat16>::value);
    return f.x != f.x || f.y != f.y ? __int_as_float(0x7FC00000) : fmaxf(f.x, f.y);
  }
};

// Weights: w = 2^(x c - top), top the whole number next above max c, so that the largest is in (1/2, 1].
//
// x c is rounded to a multiple of 1/256, whose power comes from the table; what is left, below 2^-9, is
// fma(x, ch, -that) + x cl with one rounding of 2^-34, and three terms of its exponential series are within
// 2^-42.  This holds while |x c| < 2^14.  Where max c is beyond 2^13, weights above 0 belong to x within 1% of
// the maximum, whose difference from it is exact in fp32, and that takes the place of x.
struct Weigher {
  float ref, least;                      // subtracted from x; smaller x have no weight
  float ch, cl;                          // log2(e) / T in two fp32 numbers
  int top;
  const uint32_t* pow;

  __device__ __forceinline__ Weigher(float m, float T, const uint32_t* table) : pow(table) {
    constexpr float kLog2e = 1.44269502162933349609375f, kRest = 1.92596299112661746887e-8f;
    ch = kLog2e / T;
    cl = (fmaf(-ch, T, kLog2e) + kRest) / T;
    const bool far = !(fabsf(m * ch) < 8192.f);
    ref = far ? m : 0.f;
    top = far ? 0 : static_cast<int>(ceilf(m * ch));
    // x c >= top - kUnitBits and a little: what is below rounds to 0 in any case
    least = m - (kUnitBits + 1) / ch;
  }
  __device__ __forceinline__ unsigned long long operator()(float x) const {
    const float s = x - ref;
    const float t = fmaf(s, ch, 49152.f);                    // 1.5 * 2^15: its last bit is 1/256
    const int k = __float_as_int(t) - 0x47400000;
    const float r = fmaf(s, cl, fmaf(s, ch, 49152.f - t));
    // 2^30 (2^r - 1), at most 2^21.4
    const float q = r * fmaf(r, fmaf(r, 0x1p30f * 0.05550410866f, 0x1p30f * 0.2402265070f), 0x1p30f * 0.6931471806f);
    const uint32_t p = pow[k & 255];
    const float f = __uint_as_float((p >> 7) + 0x3F000000u); // p in units of 2^30, to 24 bits
    const uint32_t w = p + (__float_as_uint(fmaf(f, q, 12582912.f)) - 0x4B400000u);
    return x >= least ? (static_cast<unsigned long long>(w) << (kUnitBits - 30)) >> min(top - (k >> 8), 63) : 0ull;
  }
};

// Whether element i comes before or at the one with key `cut`: ckey(x, i) >= cut.
__device__ __forceinline__ bool not_before(float x, uint32_t i, unsigned long long cut) {
  const float at = ckey_score(cut);
  return x > at || (x == at && i <= static_cast<uint32_t>(ckey_idx(cut)));
}

__device__ __forceinline__ unsigned long long warp_total(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += shfl_xor_key(v, o);
  return v;
}
__device__ __forceinline__ unsigned long long warp_running(unsigned long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

template <typename E>
struct Row {
  static constexpr int VEC = 16 / sizeof(E);
  const SamplingParams& p;
  Shared& sh;
  const uint4* slice;
  cg::cluster_group cluster;
  int tid, lane, warp, rank, ctas;
  int begin, end;                        // this warp's 16-byte pieces of the slice
  int index0;                            // vocabulary index of the slice's first element
  int turn = 0;                          // which set of `mass`, `count`, `lo`, `hi` is next

  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int i = begin + lane; i < end; i += 32) {
      float x[VEC];
      unpack<E>(slice[i], x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f(x[e], static_cast<uint32_t>(index0 + i * VEC + e));
    }
  }

  // Sums of v over the CTA, at every thread.
  __device__ __forceinline__ unsigned long long block_total(unsigned long long v) {
    v = warp_total(v);
    __syncthreads();
    if (lane == 0) sh.warp_sum[warp] = v;
    __syncthreads();
    unsigned long long sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh.warp_sum[w];
    return sum;
  }
  // Sum of v over the threads before this one; *total over all.
  __device__ __forceinline__ unsigned long long block_before(unsigned long long v, unsigned long long* total) {
    const unsigned long long run = warp_running(v, lane);
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = run;
    __syncthreads();
    unsigned long long before = run - v, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.warp_sum[w];
      sum += sh.warp_sum[w];
    }
    *total = sum;
    return before;
  }

  // The first element, in the vocabulary's order, at which the running sum of f exceeds the target
  // that `target` makes of the total; `hit` is called by the one thread that holds it.  One
  // meeting of the cluster.
  template <typename F, typename T, typename H>
  __device__ void find(F f, T target, H hit) {
    unsigned long long mine = 0;
    each([&](float x, uint32_t i) { mine += f(x, i); });
    mine = warp_total(mine);
    __syncthreads();
    if (lane == 0) sh.warp_sum[warp] = mine;
    __syncthreads();
    unsigned long long sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh.warp_sum[w];
    const int set = turn++ & 1;
    if (tid < ctas) cluster.map_shared_rank(&sh, tid)->mass[set][rank] = sum;
    cluster.sync();
    unsigned long long total = 0, before = 0;
    for (int c = 0; c < ctas; ++c) {
      if (c < rank) before += sh.mass[set][c];
      total += sh.mass[set][c];
    }
    const unsigned long long t = target(total);
    if (t < before || t >= before + sum) return;
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
    if (t < before || t >= before + mine) return;
    for (int i0 = begin; i0 < end; i0 += 32) {
      const int i = i0 + lane;
      float x[VEC];
      unsigned long long own = 0;
      if (i < end) {
        unpack<E>(slice[i], x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) own += f(x[e], static_cast<uint32_t>(index0 + i * VEC + e));
      }
      const unsigned long long run = before + warp_running(own, lane);
      const uint32_t over = __ballot_sync(0xFFFFFFFFu, run > t);
      if (over != 0) {
        if (lane == __ffs(over) - 1) {
          unsigned long long at = run - own;
          bool done = false;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const uint32_t index = static_cast<uint32_t>(index0 + i * VEC + e);
            at += f(x[e], index);
            if (!done && at > t) {
              done = true;
              hit(x[e], index, total);
            }
          }
        }
        return;
      }
      before = __shfl_sync(0xFFFFFFFFu, run, 31);
    }
  }

  // Elements that `take` accepts into the first CTA's list (their keys), and how many there are; nothing
  // is listed when they are too many.  Meetings: one, and a second when they fit.
  template <typename F>
  __device__ uint32_t gather(bool scan, F take) {
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    if (scan)
      each([&](float x, uint32_t i) {
        if (take(x, i)) {
          const uint32_t at = atomicAdd(&sh.listed, 1u);
          if (at < kList) sh.list[at] = ckey(x, static_cast<int>(i));
        }
      });
    __syncthreads();
    const int set = turn++ & 1;
    if (tid < ctas) cluster.map_shared_rank(&sh, tid)->count[set][rank] = sh.listed;
    cluster.sync();
    uint32_t n = 0;
    for (int c = 0; c < ctas; ++c) n += sh.count[set][c];   // (of at most 2^20 elements)
    if (n > kList || ctas == 1) return n;
    if (rank == 0) {
      const uint32_t own = sh.count[set][0];
      for (uint32_t at = own + tid; at < n; at += kThreads) {
        uint32_t i = at - own;
        int c = 1;
        while (i >= sh.count[set][c]) i -= sh.count[set][c++];
        sh.list[at] = cluster.map_shared_rank(&sh, c)->list[i];
      }
    }
    cluster.sync();
    return n;
  }

  // The list's n keys, descending; thread t gets places [E t, E t + E).  The list's memory is used.
  template <int P>
  __device__ __forceinline__ void sort_list(uint32_t n, unsigned long long (&v)[P]) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = tid * P + e < n ? sh.list[tid * P + e] : 0;
    __syncthreads();
    block_sort_regs<P, true>(v, sh.list);
  }

  // The key of the list's element at which the running sum (of ones or weights, in the keys'
  // descending order, from `above`) reaches `target`.  First CTA only; result at sh.answer.
  template <int P, typename F>
  __device__ void cut_list(uint32_t n, unsigned long long above, unsigned long long target, F f) {
    unsigned long long v[P], w[P], own = 0, total;
    sort_list<P>(n, v);
#pragma unroll
    for (int e = 0; e < P; ++e) own += w[e] = tid * P + e < n ? f(ckey_score(v[e])) : 0;
    unsigned long long run = above + block_before(own, &total);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      if (run < target && run + w[e] >= target) sh.answer = v[e];
      run += w[e];
    }
    __syncthreads();
  }

  // Of the elements with ckey >= cut and lo <= x <= hi, in descending order: the key of the one at which the
  // running sum of f reaches `target` (the sum over all of them does).  MASS: f are weights, else ones.
  template <bool MASS, typename F>
  __device__ unsigned long long select(float lo, float hi, unsigned long long cut, unsigned long long target, F f) {
    unsigned long long above = 0;
    while (true) {
      // equal bins from hi down to lo; halves where the range passes fp32's, and a range too small to
      // divide by is scaled up (so the largest is always in the first bin, the smallest in the last)
      const float half = hi - lo < __int_as_float(0x7F800000) ? 1.f : 0.5f, range = half * hi - half * lo;
      const float up = range < 1e-30f ? 0x1p100f : 1.f, by = static_cast<float>(kBins) / (range * up);
      auto bin_at = [&](float x) { return min(__float2int_rz((half * hi - half * x) * up * by), kBins - 1); };
      auto inside = [&](float x, uint32_t i) { return x >= lo && x <= hi && not_before(x, i, cut); };
      int bin = 0;
      if (lo < hi) {
        for (int i = tid; i < 3 * kBins; i += kThreads) sh.hist[i / kBins][i % kBins] = 0;
        __syncthreads();
        each([&](float x, uint32_t i) {
          if (!inside(x, i)) return;
          const int b = bin_at(x);
          if constexpr (MASS) {
            const unsigned long long w = f(x);
            const uint32_t w0 = static_cast<uint32_t>(w) & 0x7FFFu, w1 = static_cast<uint32_t>(w >> 15) & 0x7FFFu;
            atomicAdd(&sh.hist[0][b], w0);
            atomicAdd(&sh.hist[1][b], w1);
            const uint32_t w2 = static_cast<uint32_t>(w >> 30);
            if (w2 != 0) atomicAdd(&sh.hist[2][b], w2);
          } else {
            atomicAdd(&sh.hist[0][b], 1u);
          }
        });
        cluster.sync();
        const int share = kBins / ctas;
        for (int b = rank * share + tid; b < (rank + 1) * share; b += kThreads) {
          unsigned long long sum = 0;
          for (int c = 0; c < ctas; ++c) {
            const Shared* o = cluster.map_shared_rank(&sh, c);
            sum += o->hist[0][b];
            if (MASS) sum += (static_cast<unsigned long long>(o->hist[1][b]) << 15) + (static_cast<unsigned long long>(o->hist[2][b]) << 30);
          }
          for (int c = 0; c < ctas; ++c) cluster.map_shared_rank(&sh, c)->merged[b] = sum;
        }
        cluster.sync();
        // the first bin, from the top, at which the running sum reaches the target
        constexpr int kEach = kBins / kThreads;
        unsigned long long own = 0, total;
#pragma unroll
        for (int e = 0; e < kEach; ++e) own += sh.merged[tid * kEach + e];
        unsigned long long run = above + block_before(own, &total);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const unsigned long long w = sh.merged[tid * kEach + e];
          if (run < target && run + w >= target) {
            sh.found = tid * kEach + e;
            sh.found_before = run;
          }
          run += w;
        }
        __syncthreads();
        bin = sh.found;
        above = sh.found_before;
      }
      auto there = [&](float x, uint32_t i) { return inside(x, i) && (!(lo < hi) || bin_at(x) == bin); };
      const uint32_t n = gather(true, there);
      if (n <= kList) {
        if (rank == 0) {
          if (n <= kThreads) cut_list<1>(n, above, target, f); else cut_list<kList / kThreads>(n, above, target, f);
          if (tid > 0 && tid < ctas) cluster.map_shared_rank(&sh, tid)->answer = sh.answer;
        }
        cluster.sync();
        return sh.answer;
      }
      if (!(lo < hi)) {
        // equal values, more than a list holds: the last one is found by its index
        const unsigned long long one = f(lo), need = (target - above + one - 1) / one;
        find([&](float x, uint32_t i) { return inside(x, i) ? 1ull : 0ull; },
             [&](unsigned long long) { return need - 1; },
             [&](float x, uint32_t i, unsigned long long) {
               for (int c = 0; c < ctas; ++c) cluster.map_shared_rank(&sh, c)->answer = ckey(x, static_cast<int>(i));
             });
        cluster.sync();
        return sh.answer;
      }
      // the bin's own range is the next one
      float least = hi, most = lo;
      each([&](float x, uint32_t i) {
        if (there(x, i)) {
          least = fminf(least, x);
          most = fmaxf(most, x);
        }
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      }
      if (lane == 0) {
        sh.warp_a[warp] = least;
        sh.warp_b[warp] = most;
      }
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) {
        least = fminf(least, sh.warp_a[w]);
        most = fmaxf(most, sh.warp_b[w]);
      }
      const int set = turn++ & 1;
      if (tid < ctas) {
        cluster.map_shared_rank(&sh, tid)->lo[set][rank] = least;
        cluster.map_shared_rank(&sh, tid)->hi[set][rank] = most;
      }
      cluster.sync();
      for (int c = 0; c < ctas; ++c) {
        least = fminf(least, sh.lo[set][c]);
        most = fmaxf(most, sh.hi[set][c]);
      }
      lo = least;
      hi = most;
    }
  }

  // Bounds that at least need[0] and need[1] of this CTA's elements reach, by their threads' largest, at
  // sh.reached; -inf: none.  Warps 0 and 1 look for them bit by bit, from the first in which they differ.
  __device__ void reached_by(int need0, int need1, float most) {
    uint32_t* keys = &sh.hist[0][0];
    keys[tid] = ord_f32(most) >> 12;
    __syncthreads();
    if (warp < 2) {
      const int need = warp == 0 ? need0 : need1;
      uint32_t key[kThreads / 32], hi = 0, lo = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) {
        key[i] = keys[i * 32 + lane];
        hi = max(hi, key[i]);
        lo = min(lo, key[i]);
      }
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
      const int bits = 32 - __clz(hi ^ lo);
      uint32_t at = hi >> bits << bits;
#pragma unroll 1
      for (int bit = bits - 1; bit >= 0; --bit) {
        const uint32_t next = at | (1u << bit);
        int n = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) n += key[i] >= next ? 1 : 0;
        if (__reduce_add_sync(0xFFFFFFFFu, n) >= need) at = next;
      }
      if (lane == 0)
        sh.reached[warp] = at <= (ord_f32(-__int_as_float(0x7F800000)) >> 12) ? -__int_as_float(0x7F800000) : unord_f32(at << 12);
    }
    __syncthreads();
  }
};

// floor(u * total), 0 <= u < 1, in whole numbers (u is 24 bits times a power of two; the few double
// units of an SM would hold up 512 threads); *exact: whether that is u * total.
__device__ __forceinline__ unsigned long long part_of(float u, unsigned long long total, bool* exact) {
  const uint32_t bits = __float_as_uint(u), e = bits >> 23;
  const unsigned long long mantissa = (bits & 0x7FFFFFu) | (e > 0 ? 0x800000u : 0u);
  const int shift = 150 - static_cast<int>(e > 0 ? e : 1);  // u = mantissa * 2^-shift, shift >= 24
  const unsigned long long lo = mantissa * total, hi = __umul64hi(mantissa, total);
  if (shift >= 64) {
    const unsigned long long up = shift - 64 < 64 ? hi >> (shift - 64) : 0;
    *exact = lo == 0 && (shift - 64 < 64 ? (hi & ((1ull << (shift - 64)) - 1)) == 0 : hi == 0);
    return up;
  }
  *exact = (lo & ((1ull << shift) - 1)) == 0;
  return (lo >> shift) | (hi << (64 - shift));
}
// The random number's place among `total` units of weight.
__device__ __forceinline__ unsigned long long place_of(float u, unsigned long long total) {
  bool exact;
  return part_of(u, total, &exact);
}
// The weight that a share p < 1 of `total` has to reach, at least 1.
__device__ __forceinline__ unsigned long long share_of(float p, unsigned long long total) {
  bool exact;
  const unsigned long long t = part_of(p, total, &exact) + (exact ? 0 : 1);
  return t < 1 ? 1 : t;
}

// All that is kept is in the first CTA's list: filters, draw and results, by that CTA.
template <int P, typename E, typename W, typename H>
__device__ void finish_list(Row<E>& row, uint32_t n, int k, float top_p, float u, const W& weigh, H hit) {
  Shared& sh = row.sh;
  const int tid = row.tid;
  unsigned long long v[P], w[P], own = 0, total;
  row.template sort_list<P>(n, v);
  const uint32_t most = k > 0 ? min(n, static_cast<uint32_t>(k)) : n;
#pragma unroll
  for (int e = 0; e < P; ++e) own += w[e] = tid * P + e < most ? weigh(ckey_score(v[e])) : 0;
  unsigned long long run = row.block_before(own, &total);
  const unsigned long long enough = top_p < 1.f ? share_of(top_p, total) : total;
  own = 0;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    const unsigned long long x = w[e];
    if (run >= enough) w[e] = 0;
    run += x;
    own += w[e];
    // the kept ones' order in the vocabulary: the list's places, by index
    sh.weights[tid * P + e] = w[e];
    v[e] = w[e] != 0 ? (v[e] << 32) | static_cast<uint32_t>(tid * P + e) : 0;
  }
  if constexpr (P == 1) {
    // few: each finds its own place, from the others' indices
    constexpr int kFew = 64;
    const int left = __syncthreads_count(w[0] != 0);         // (they are the first of the sorted)
    if (left <= kFew) {
      if (tid < left) sh.list[tid] = v[0];
      const unsigned long long sum = row.block_total(w[0]), at = place_of(u, sum);
      if (tid < left) {
        unsigned long long before = 0;
        for (int j = 0; j < left; ++j)
          if (sh.list[j] > v[0]) before += sh.weights[j];    // (larger keys: smaller indices)
        if (before <= at && at < before + w[0]) hit(0xFFFFFFFFu - static_cast<uint32_t>(v[0] >> 32), sum);
      }
      return;
    }
  }
  __syncthreads();
  block_sort_regs<P, true>(v, sh.list);
  // (the low half of a key is 2^32 - 1 - index, so descending keys are ascending indices)
  own = 0;
#pragma unroll
  for (int e = 0; e < P; ++e) own += w[e] = v[e] != 0 ? sh.weights[static_cast<uint32_t>(v[e])] : 0;
  run = row.block_before(own, &total);
  const unsigned long long at = place_of(u, total);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    if (run <= at && at < run + w[e]) hit(0xFFFFFFFFu - static_cast<uint32_t>(v[e] >> 32), total);
    run += w[e];
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 2) sample_tokens_kernel(const __grid_constant__ SamplingParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  uint4* slice = reinterpret_cast<uint4*>(raw + (sizeof(Shared) + 15) / 16 * 16);
  constexpr int VEC = 16 / sizeof(E);
  const float inf = __int_as_float(0x7F800000);
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = p.ctas, rank = static_cast<int>(blockIdx.x) % ctas, b = static_cast<int>(blockIdx.x) / ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 256) sh.pow[tid] = kPow.v[tid];
  if (tid == 0) sh.found = kNoCut;

  begin_after_previous();
  const float T = p.temperature != nullptr ? kv_load(p.temperature + b) : p.temperature_all;
  int k = p.top_k != nullptr ? kv_load(p.top_k + b) : p.top_k_all;
  const float top_p = p.top_p != nullptr ? kv_load(p.top_p + b) : p.top_p_all;
  const float min_p = p.min_p != nullptr ? kv_load(p.min_p + b) : p.min_p_all;
  const float given = kv_load(p.u + b), u = fminf(fmaxf(given, 0.f), 1.f - 0x1p-24f);
  const bool settings = T >= 0.f && T < inf && top_p >= 0.f && min_p >= 0.f && min_p <= 1.f && given == given;
  if (k < 0 || k >= p.V) k = 0;
  if (tid == kThreads - 1 && min_p > 0.f) {
    const double by = log(static_cast<double>(min_p)) * static_cast<double>(T);
    sh.min_hi = static_cast<float>(by);
    sh.min_lo = static_cast<float>(by - static_cast<double>(sh.min_hi));
  }

  // --- the row's slice, and its largest ---------------------------------------------------
  // Pieces of 16 aligned bytes; elements before the row and behind it are -inf.
  const E* logits = reinterpret_cast<const E*>(p.logits) + static_cast<size_t>(b) * p.stride;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(logits) & 15u) / sizeof(E));
  const int pieces = (p.V + shift + VEC - 1) / VEC;
  const int first = min(rank * p.per, pieces), mine = min(p.per, pieces - first);
  const int per_warp = (mine + kWarps - 1) / kWarps;
  Row<E> row{p, sh, slice, cluster, tid, lane, warp, rank, ctas, min(warp * per_warp, mine), min((warp + 1) * per_warp, mine),
             first * VEC - shift};
  Largest<E> largest;
  {
    constexpr int kUnroll = 4;
    const E* from = logits + row.index0;
#pragma unroll 1
    for (int i0 = row.begin + lane; i0 < row.end; i0 += 32 * kUnroll) {
      uint4 v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int i = i0 + 32 * j, at = row.index0 + i * VEC;
        if (i >= row.end) continue;
        if (at >= 0 && at + VEC <= p.V) {
          v[j] = kv_load(reinterpret_cast<const uint4*>(from + i * VEC));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = sizeof(E) == 4 ? 0xFF800000u : std::is_same<E, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if (at + e < 0 || at + e >= p.V) continue;
            if constexpr (sizeof(E) == 4) {
              w[e] = kv_load(reinterpret_cast<const uint32_t*>(logits) + at + e);
            } else {
              const uint32_t x = kv_load(reinterpret_cast<const uint16_t*>(logits) + at + e);
              w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xFFFFu) | (x << 16) : (w[e >> 1] & 0xFFFF0000u) | x;
            }
          }
          v[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int i = i0 + 32 * j;
        if (i >= row.end) continue;
        slice[i] = v[j];
        largest.add(v[j]);
      }
    }
  }
  const float most = largest.get();      // NaN if any element is
  bool bad = __syncthreads_or(most < inf ? 0 : 1) != 0;
  // Few enough are kept to be sorted by one CTA: all of a small vocabulary, or a small top-k.  For that each
  // CTA finds what its share of k elements reach, and what k of them do: k elements of the row reach the least of
  // the CTAs' former bounds, and any of the latter.
  const bool all_listed = p.V <= kList, few = k > 0 && k <= kThreads / 2;
  if (few && !all_listed) row.reached_by((k + ctas - 1) / ctas, k, bad ? -inf : most);
  float cta_most = most;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) cta_most = fmaxf(cta_most, __shfl_xor_sync(0xFFFFFFFFu, cta_most, o));
  if (lane == 0) sh.warp_a[warp] = cta_most;
  __syncthreads();
  if (warp == 0) {
    cta_most = lane < kWarps ? sh.warp_a[lane] : -inf;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) cta_most = fmaxf(cta_most, __shfl_xor_sync(0xFFFFFFFFu, cta_most, o));
    if (lane < ctas) {
      Shared* o = cluster.map_shared_rank(&sh, lane);
      o->top[rank] = cta_most;
      o->bound[0][rank] = few && !all_listed ? sh.reached[0] : -inf;
      o->bound[1][rank] = few && !all_listed ? sh.reached[1] : -inf;
      o->bad[rank] = bad;
    }
  }
  cluster.sync();
  float m = -inf, floor_x = inf, by_one = -inf;
  for (int c = 0; c < ctas; ++c) {
    m = fmaxf(m, sh.top[c]);
    floor_x = fminf(floor_x, sh.bound[0][c]);
    by_one = fmaxf(by_one, sh.bound[1][c]);
    bad = bad || sh.bad[c] != 0;
  }
  floor_x = fmaxf(floor_x, by_one);
  int* token = p.token + b;
  float* logp = p.logp + b;
  if (!settings || bad || m == -inf) {
    if (rank == 0 && tid == 0) {
      *token = -1;
      *logp = settings && !bad ? -inf : __int_as_float(0x7FC00000);
    }
    return;
  }
  if (T < 0x1p-127f) {                   // (1 / T would pass fp32) the largest, the first of equal ones
    uint32_t at = kNoCut;
    if (most == m) row.each([&](float x, uint32_t i) { at = x == m && i < at ? i : at; });
    if (at != kNoCut) atomicMin(cluster.map_shared_rank(&sh.found, 0), at);
    cluster.sync();
    if (rank == 0 && tid == 0) {
      *token = static_cast<int>(sh.found);
      *logp = 0.f;
    }
    return;
  }
  const Weigher weigh(m, T, sh.pow);
  // the result: its logarithm from x itself, which small weights hold to a few bits only
  auto hit = [&](uint32_t i, unsigned long long total) {
    const double x = static_cast<double>(as_float(kv_load(logits + i))) - static_cast<double>(weigh.ref);
    *token = static_cast<int>(i);
    *logp = static_cast<float>(x / static_cast<double>(T) - log(static_cast<double>(total)) - (weigh.top - kUnitBits) * 0.69314718055994530942);
  };
  // min-p is a bound on x; -inf is never kept
  float least = -__int_as_float(0x7F7FFFFF);
  if (min_p > 0.f) {
    // max + T ln(min_p), rounded up: from two fp32 numbers by an exact sum
    const float by = sh.min_hi, s = m + by, z = s - m, rest = ((m - (s - z)) + (by - z)) + sh.min_lo;
    const float up = rest > 0.f ? nextafterf(s, inf) : s;
    least = fmaxf(least, fminf(m, up));
  }
  if (all_listed || few) {
    const float from = fmaxf(floor_x, least);
    const uint32_t n = row.gather(most >= from, [&](float x, uint32_t) { return x >= from; });
    if (n <= kList) {
      if (rank == 0) {
        if (n <= kThreads) finish_list<1>(row, n, k, top_p, u, weigh, hit);
        else finish_list<kList / kThreads>(row, n, k, top_p, u, weigh, hit);
      }
      return;
    }
  }
  unsigned long long cut = ckey(least, -1);                  // (index 2^32 - 1: all of equal value)
  auto kept = [&](float x, uint32_t i) { return not_before(x, i, cut); };
  if (k > 0) {
    // how many there are, and the smallest
    uint32_t n = 0;
    float lo = m;
    row.each([&](float x, uint32_t) {
      if (x >= least) {
        ++n;
        lo = fminf(lo, x);
      }
    });
    n = __reduce_add_sync(0xFFFFFFFFu, n);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    if (lane == 0) {
      sh.warp_n[warp] = n;
      sh.warp_a[warp] = lo;
    }
    __syncthreads();
    n = 0;
    for (int w = 0; w < kWarps; ++w) {
      n += sh.warp_n[w];
      lo = fminf(lo, sh.warp_a[w]);
    }
    const int set = row.turn++ & 1;
    if (tid < ctas) {
      Shared* o = cluster.map_shared_rank(&sh, tid);
      o->count[set][rank] = n;
      o->lo[set][rank] = lo;
    }
    cluster.sync();
    n = 0;
    for (int x = 0; x < ctas; ++x) {
      n += sh.count[set][x];
      lo = fminf(lo, sh.lo[set][x]);
    }
    if (n > static_cast<uint32_t>(k)) cut = row.template select<false>(lo, m, cut, k, [](float) { return 1ull; });
  }
  if (top_p < 1.f) {
    unsigned long long own = 0;
    uint32_t n = 0;
    row.each([&](float x, uint32_t i) {
      if (kept(x, i)) {
        own += weigh(x);
        ++n;
      }
    });
    own = row.block_total(own);
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) sh.warp_n[warp] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kWarps; ++w) n += sh.warp_n[w];
    const int set = row.turn++ & 1;
    if (tid < ctas) {
      Shared* o = cluster.map_shared_rank(&sh, tid);
      o->mass[set][rank] = own;
      o->count[set][rank] = n;
    }
    cluster.sync();
    unsigned long long total = 0;
    n = 0;
    for (int x = 0; x < ctas; ++x) {
      total += sh.mass[set][x];
      n += sh.count[set][x];
    }
    const unsigned long long target = share_of(top_p, total);
    // n elements of less than (total - target) / n each cannot hold the rest, so the cut is above that
    // (fp32 logarithms and products here are right to 2^-20, the bound is taken 2^-7 lower)
    float lo = fmaxf(least, ckey_score(cut));
    const float rest = static_cast<float>(total - target) / n;
    if (rest > 1.f) lo = fmaxf(lo, fminf(m, weigh.ref + (weigh.top + log2f(rest) - kUnitBits - 0x1p-7f) / weigh.ch - 0x1p-20f * fabsf(weigh.ref)));
    cut = row.template select<true>(lo, m, cut, target, weigh);
  }
  row.find([&](float x, uint32_t i) { return kept(x, i) ? weigh(x) : 0ull; },
           [&](unsigned long long total) { return place_of(u, total); },
           [&](float, uint32_t i, unsigned long long total) { hit(i, total); });
}

template <typename E>
cudaError_t launch_sampling(const SamplingParams& p, int device, cudaStream_t stream) {
  static std::atomic<unsigned long long> ready{0};           // devices whose kernel may use all its shared memory
  const int smem = static_cast<int>((sizeof(Shared) + 15) / 16 * 16) + p.per * 16;
  if (device > 63 || (ready.load() >> device & 1) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(sample_tokens_kernel<E>),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSamplingSmem);
    if (e != cudaSuccess) return e;
    if (device <= 63) ready.fetch_or(1ull << device);
  }
  cudaLaunchAttribute attrs[2] = {};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = p.ctas;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.B * p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, sample_tokens_kernel<E>, p);
}

}  // namespace

bool sampling_plan(SamplingParams& p, int num_sms) {
  const long long size = p.dtype == LTK_F32 ? 4 : 2, vec = 16 / size;
  const long long pieces = (p.V + 2 * vec - 2) / vec;        // wherever the row begins
  // CTAs of a row: as few as hold it in 64 KB each (two fit an SM), more where SMs would be idle and
  // a CTA still has 8 KB to read.
  int ctas = 1;
  while (ctas < kMaxCtas && (pieces * 16 > ctas * 65536ll ||
                             (static_cast<long long>(p.B) * ctas * 2 <= num_sms && pieces * 16 > ctas * 8192ll)))
    ctas *= 2;
  p.ctas = ctas;
  p.per = static_cast<int>((pieces + ctas - 1) / ctas);
  return (sizeof(Shared) + 15) / 16 * 16 + p.per * 16ull <= kSamplingSmem && static_cast<long long>(p.B) * ctas <= 0x7FFFFFFF;
}

cudaError_t launch_sampling(const SamplingParams& p, int device, cudaStream_t stream) {
  switch (p.dtype) {
    case LTK_F32: return launch_sampling<float>(p, device, stream);
    case LTK_F16: return launch_sampling<__half>(p, device, stream);
    default: return launch_sampling<__nv_bfloat16>(p, device, stream);
  }
}

}  // namespace ltk

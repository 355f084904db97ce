// k_sampling.cu -- a token for each row of logits, from a given random number.
//
//   w_i = 2^((x_i - max) log2(e) / T)        tokens ordered by (x descending, index ascending)
//   min-p: keep w_i >= min_p;  top-k: of these the first k;  top-p: of these the fewest first ones
//   whose weights reach p of their total;  token: the first kept one, in the order of the
//   vocabulary, at which the running sum of kept weights exceeds u * total.
//
// Which token that is depends on sums over a whole vocabulary being right to far better than one
// token's share, so weights are whole numbers in units of 2^-44 of (about) the largest, right to
// 2^-30.5 of themselves (those below 2^-42 are nothing), and every sum of them is exact in 64 bits, in
// any order: the result does not depend on how a row is split.  (fp32 weights would put one in a
// hundred draws from a flat vocabulary of 100000 on the neighbouring token.)
//
// A cluster of 1 to 8 CTAs takes a row, each a slice of it; what has to be known of the whole row
// (maximum, counts, sums) goes from CTA to CTA through distributed shared memory.  Slices are read
// from memory once, for the maximum, and from L2 in later passes:
//   no filter, min-p:  one more pass for the weights; the draw goes down to a warp's part of a slice;
//   top-k up to 256:   the threads' first elements give a bound that k elements reach, and what is
//                      above it is listed while the rest is read; the few that pass a better bound, by
//                      all threads' largest, go to one CTA, which compares them with one another;
//   larger top-k:      a histogram of x; up to 1024 elements are then listed and finished by one CTA,
//                      else the cut is looked for among those of one bin;
//   top-p:             a histogram of rough weights, and a pass with exact ones (select_share).
//
// With 192 rows of 131071 in bf16 (50 MB, 7.5 us to read): greedy 17 us, no filter 52, min-p 54, top-k
// of 50 34, of 1000 98, of 20000 131, top-p of 0.95 120.  No one thing bounds it: an exact weight takes some
// 20 instructions (27 an element in all, 22 us of full issue without filters), a histogram's atomic with its bin as much
// time; but half of the issue slots are empty, as a thread has one piece's load in flight (the largest stall) and
// CTAs end unevenly.
// One row of 32000 in fp32, top-k of 50: 8 us, of which the cluster's three meetings and the lists
// they pass on are latency.
#include <cooperative_groups.h>

#include <cmath>

#include "block_sort.cuh"
#include "kv_tensor.cuh"
#include "sampling_internal.cuh"

namespace ltk {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kBins = 1024, kFineBins = 2048;  // (the latter of rough weights)
constexpr int kList = 1024;              // elements that one CTA takes
constexpr int kPairs = 256;              // of them, that are all compared with one another
constexpr int kUnitBits = 44;            // weights are in units of 2^-44
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr int kRun = 8;                  // 16-byte pieces that a thread reads at a time at first
constexpr int kMostElements = 131072;    // of a slice: a bin's sum of 15-bit pieces of weights stays below 2^32, a thread's sum of
                                         // weights within 2^53
constexpr int kEarly = 2048;             // elements listed while a slice is first read

// (1 - h) 2^(j / 512) in units of 2^-31, rounded, where 1 / (1 - h) = 1 + kWholeBits / 2^32 (see Weigher): by the
// exponential series in double, at compile time.
constexpr uint32_t kWholeBits = 0x4B400000u;                 // 1.5 * 2^23 in fp32, whose last bit is 1
struct PowTable {
  uint32_t v[512];
};
constexpr PowTable make_pow_table() {
  PowTable t{};
  for (int j = 0; j < 512; ++j) {
    const double z = j * (0.693147180559945309417232 / 512.0);
    double term = 1.0, sum = 1.0;
    for (int i = 1; i < 30; ++i) {
      term *= z / i;
      sum += term;
    }
    t.v[j] = static_cast<uint32_t>(sum * (2147483648.0 / (1.0 + kWholeBits / 4294967296.0)) + 0.5);
  }
  return t;
}
__device__ constexpr PowTable kPow = make_pow_table();

struct Shared {
  uint32_t pow[512];
  // what the CTAs of a cluster tell one another, by rank; two sets in turn where there is a next time
  uint32_t top[kMaxCtas], bound[2][kMaxCtas];
  u64 mass[2][kMaxCtas];
  uint32_t count[2][kMaxCtas], lo[2][kMaxCtas], hi[2][kMaxCtas];
  u64 all[kMaxCtas];
  uint32_t least[kMaxCtas];
  u64 answer;
  // a CTA's own
  u64 warp_sum[2][kWarps], listed_sum[kWarps];
  uint32_t listed, early;
  uint32_t found;
  u64 found_before;
  float min_hi, min_lo;                  // T ln(min_p)
  uint32_t reached[2];
  int reached_bin[2];
  float edge[2];
  union {
    struct {
      uint32_t hist[3][kBins];           // counts, or weights in pieces of 15, 15 and 15 bits
      u64 merged[kBins];
    };
    struct {
      uint32_t fine[kFineBins];          // rough weights
      u64 merged_fine[kFineBins];
    };
    struct {                             // while the largest are looked for
      uint32_t first_hist[kBins];
      float early_x[kEarly];             // elements at or above a first bound, and their indices
      uint32_t early_i[kEarly];
    };
    struct {
      u64 weights[kList];                // the list's
      u64 part_mass[kThreads];
      uint32_t part_rank[kThreads];
    };
  };
  u64 list[kList];                       // keys (ckey)
};

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
    } else if constexpr (std::is_same<E, __half>::value) {
      asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(v) : "r"(w));
    } else {
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(w));
    }
  }
  __device__ __forceinline__ void add(const uint4& w) {
    one(w.x);
    one(w.y);
    one(w.z);
    one(w.w);
  }
  __device__ __forceinline__ void with(const Largest& o) { one(o.v); }
  __device__ __forceinline__ float get() const {
    if constexpr (std::is_same<E, float>::value) return __uint_as_float(v);
    const float2 f = kv_unpack16(v, std::is_same<E, __nv_bfloat16>::value);
    return f.x != f.x || f.y != f.y ? __int_as_float(0x7FC00000) : fmaxf(f.x, f.y);
  }
};

// Weights: w = 2^(x c - top), top the whole number next above max c, so that the largest is in (1/2, 1].
//
// x c is rounded to a multiple of 1/512, whose power comes from the table; what is left is
// r = fma(x, ch, -that) + x cl, |r| <= 2^-10 + |x cl|, with one rounding of 2^-35, and three terms of its exponential series
// are within 2^-46.  They are a whole number of units of 2^-32 only while (1 + h') 2^32 |2^r - 1| is below 2^22, which is
// |r| < 1.114 * 2^-10, and |cl| is up to 2^-23.7 of ch: so |x c| has to stay below 1534.  Where max c is beyond 2^10,
// weights above 0 belong to x within 5% of the maximum, whose difference from it is exact in fp32, and that takes
// the place of x.  (A bound of 2^12 left weights off by up to 2^-13 with temperatures like 5 and logits near -10000.)
struct Weigher {
  float ref, least;                      // subtracted from x; smaller x weigh nothing
  float ch, cl;                          // log2(e) / T in two fp32 numbers
  int top;
  const uint32_t* pow;
  static constexpr float kRound = 24576.f;                   // 1.5 * 2^14: its last bit is 1/512
  static constexpr int kRoundBits = 0x46C00000;

  __device__ __forceinline__ Weigher(float m, float T, const uint32_t* table) : pow(table) {
    constexpr float kLog2e = 1.44269502162933349609375f, kRest = 1.92596299112661746887e-8f;
    ch = kLog2e / T;
    cl = (fmaf(-ch, T, kLog2e) + kRest) / T;
    const bool far = !(fabsf(m * ch) < 1024.f);
    ref = far ? m : 0.f;
    top = far ? 0 : static_cast<int>(ceilf(m * ch));
    least = m - (kUnitBits - 2) / ch;    // x c >= top - kUnitBits + 1
    if ((least - m) * ch < 1.5f - kUnitBits) least = nextafterf(least, __int_as_float(0x7F800000));   // (rounded too far down)
  }
  // The weight of an element not below `least`: bits is what x c was rounded to, v = kWhole + (1 + h') 2^32 (2^r - 1),
  // of which r is what that leaves and 1 + h' = 1 + kWholeBits / 2^32.  With p the table's entry,
  // p (2^32 + bits of v) = 2^32 2^(31 + j / 512) 2^r: one wide product.
  __device__ __forceinline__ u64 weight(int bits, float v) const {
    const uint32_t p = pow[bits & 511];
    const u64 w = (static_cast<u64>(p) << 32) + static_cast<u64>(p) * __float_as_uint(v);
    return w >> (top + (kRoundBits >> 9) + (63 - kUnitBits) - (bits >> 9));
  }
  static constexpr float kWhole = 12582912.f, kH = 1.f + kWholeBits / 4294967296.f;
  // (1 + h') 2^32 (2^r - 1) is at most 2^21.95: |x c| is at most 2^10 + 42 here, |r| 1.08 * 2^-10
  static constexpr float kA = 0x1p32f * kH * 0.6931471806f, kB = 0x1p32f * kH * 0.2402265070f, kC = 0x1p32f * kH * 0.05550410866f;
  __device__ __forceinline__ u64 operator()(float x) const {
    const float s = x - ref, t = fmaf(s, ch, kRound);
    const float r = fmaf(s, cl, fmaf(s, ch, kRound - t));
    const float v = fmaf(r, fmaf(r, fmaf(r, kC, kB), kA), kWhole);
    return x >= least ? weight(__float_as_int(t), v) : 0ull;
  }
  // Two elements' weights, of those not below `from` (>= least), onto a sum: the same numbers, with the arithmetic
  // two at a time.
  __device__ __forceinline__ void add2_to(u64& sum, float from, float x0, float x1) const {
    u64 w0, w1;
    two(x0, x1, w0, w1);
    if (x0 >= from) sum += w0;
    if (x1 >= from) sum += w1;
  }
  // The same, and those of elements above `over` (>= from) onto another.
  __device__ __forceinline__ void add2_to(u64& sum, u64& above, float from, float over, float x0, float x1) const {
    u64 w0, w1;
    two(x0, x1, w0, w1);
    if (x0 >= from) sum += w0;
    if (x1 >= from) sum += w1;
    if (x0 > over) above += w0;
    if (x1 > over) above += w1;
  }
  __device__ __forceinline__ void two(float x0, float x1, u64& w0, u64& w1) const {
    const uint64_t c = pack2(ch, ch), s = add2(pack2(x0, x1), pack2(-ref, -ref));
    const uint64_t t = fma2(s, c, pack2(kRound, kRound));
    const uint64_t d = fma2(t, pack2(-1.f, -1.f), pack2(kRound, kRound));
    const uint64_t r = fma2(s, pack2(cl, cl), fma2(s, c, d));
    const float2 v = unpack2(fma2(r, fma2(r, fma2(r, pack2(kC, kC), pack2(kB, kB)), pack2(kA, kA)), pack2(kWhole, kWhole)));
    const float2 tt = unpack2(t);
    w0 = weight(__float_as_int(tt.x), v.x);
    w1 = weight(__float_as_int(tt.y), v.y);
  }
  // ln of the share of x (with a weight) in `total`, right to 2^-24 of itself + 2^-30: x c and log2(total) are each
  // split into a multiple of 1/512, exact, and a rest.
  __device__ float log_share(float x, u64 total) const {
    const float s = x - ref, t = fmaf(s, ch, kRound);
    const float r = fmaf(s, cl, fmaf(s, ch, kRound - t));
    const int e = 63 - __clzll(total);
    const u64 z = total << (63 - e);     // [1, 2) in units of 2^-63
    const int j = min(max(__float2int_rn(log2f(__ull2float_rz(z >> 40) * 0x1p-23f) * 512.f), 0), 511);
    const u64 p = (static_cast<u64>(pow[j]) << 32) + static_cast<u64>(pow[j]) * kWholeBits;      // in units of 2^-63
    const float by = static_cast<float>(static_cast<long long>(z - p)) / static_cast<float>(p);
    const float l = by * fmaf(by, fmaf(by, 0.4808983470f, -0.7213475204f), 1.442695041f);
    const float a = (t - kRound) - static_cast<float>(top - kUnitBits + e) - static_cast<float>(j) * (1.f / 512.f);
    return fmaf(a, 0.693147182464599609375f, fmaf(a, -1.904654299957768e-9f, (r - l) * 0.6931471806f));
  }
};

// What is kept: elements before or at one in the order (x descending, index ascending).
struct Cut {
  float x;
  uint32_t i;                            // kNone: all elements of that x
  __device__ __forceinline__ bool operator()(float y, uint32_t j) const { return y > x || (y == x && j <= i); }
};
__device__ __forceinline__ Cut cut_at(u64 key) { return Cut{ckey_score(key), static_cast<uint32_t>(ckey_idx(key))}; }

// Equal bins from hi down to lo < hi: halves where the range passes fp32's, and all scaled up where it is too
// small to divide by, so that hi is always in the first bin and lo in the last.  (lo == hi: there is only one bin.)
template <int N>
struct BinsOf {
  float minus, from, by;
  __device__ __forceinline__ BinsOf(float lo, float hi) {
    const float range = hi - lo;         // (below 1e-30 but not 0: hi and lo are below 1e-22)
    const float scale = range > 0.f && range < 1e-30f ? 0x1p100f : range < __int_as_float(0x7F800000) ? 1.f : 0.5f;
    minus = -scale;
    from = scale * hi;
    by = range > 0.f ? static_cast<float>(N) / (from - scale * lo) : 0.f;
  }
  // Where x <= hi lies, in bins from hi; of what lies below lo, the end of the last bin.
  __device__ __forceinline__ float place(float x) const { return fminf(fmaf(minus, x, from) * by, N - 0x1p-10f); }
  // A place's bin, from the place rounded down in a sum with 2^23.
  static __device__ __forceinline__ int number(float whole) { return __float_as_int(whole) & (N - 1); }
  __device__ __forceinline__ int operator()(float x) const { return number(__fadd_rd(place(x), 0x1p23f)); }
};
using Bins = BinsOf<kBins>;

// Sum over the warp of numbers below 2^53.
__device__ __forceinline__ u64 warp_total(u64 v) {
  const uint32_t lo = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(v) & 0x7FFFFFFu);
  return lo + (static_cast<u64>(__reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(v >> 27))) << 27);
}
__device__ __forceinline__ u64 warp_running(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// floor(u * total), 0 <= u < 1, in whole numbers (u is 24 bits times a power of two; the few double
// units of an SM would hold up 512 threads); *exact: whether that is u * total.
__device__ __forceinline__ u64 part_of(float u, u64 total, bool* exact) {
  const uint32_t bits = __float_as_uint(u), e = bits >> 23;
  const u64 mantissa = (bits & 0x7FFFFFu) | (e > 0 ? 0x800000u : 0u);
  const int shift = 150 - static_cast<int>(e > 0 ? e : 1);  // u = mantissa * 2^-shift, shift >= 24
  const u64 lo = mantissa * total, hi = __umul64hi(mantissa, total);
  if (shift >= 64) {
    const int rest = shift - 64;
    *exact = lo == 0 && (rest < 64 ? (hi & ((1ull << rest) - 1)) == 0 : hi == 0);
    return rest < 64 ? hi >> rest : 0;
  }
  *exact = (lo & ((1ull << shift) - 1)) == 0;
  return (lo >> shift) | (hi << (64 - shift));
}
// The random number's place among `total` units of weight.
__device__ __forceinline__ u64 place_of(float u, u64 total) {
  bool exact;
  return part_of(u, total, &exact);
}
// The weight that a share p < 1 of `total` has to reach, at least 1.
__device__ __forceinline__ u64 share_of(float p, u64 total) {
  bool exact;
  u64 t = part_of(p, total, &exact);
  if (!exact) ++t;
  return t < 1 ? 1 : t;
}

template <typename E>
struct Row {
  static constexpr int VEC = 16 / sizeof(E);
  Shared& sh;
  const E* logits;                       // the row
  int V;
  cg::cluster_group cluster;
  int tid, lane, warp, rank, ctas;
  int slice, longest;                    // pieces (16 aligned bytes) of this CTA's slice, and of the longest one
  int begin, end;                        // this warp's of them
  int index0;                            // vocabulary index of the slice's first element
  int sums = 0;                          // which of warp_sum was used last
  int turn = 0;                          // which set of `mass`, `count`, `lo`, `hi` is next

  __device__ __forceinline__ Shared* at(int c) const { return cluster.map_shared_rank(&sh, c); }

  __device__ __forceinline__ float element(int i) const {
    if constexpr (sizeof(E) == 4) return kv_load(logits + i);
    const uint32_t x = kv_load(reinterpret_cast<const uint16_t*>(logits) + i);
    return kv_unpack16(x, std::is_same<E, __nv_bfloat16>::value).x;
  }
  static __device__ __forceinline__ uint4 nothing() {
    const uint32_t w = sizeof(E) == 4 ? 0xFF800000u : std::is_same<E, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
    return make_uint4(w, w, w, w);
  }
  // A piece; elements before the row and behind it are -inf.
  __device__ __forceinline__ uint4 piece(int i) const {
    const int from = index0 + i * VEC;
    if (from >= 0 && from + VEC <= V) return kv_load(reinterpret_cast<const uint4*>(logits + from));
    uint32_t w[4] = {nothing().x, nothing().x, nothing().x, nothing().x};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (from + e < 0 || from + e >= V) continue;
      if constexpr (sizeof(E) == 4) {
        w[e] = kv_load(reinterpret_cast<const uint32_t*>(logits) + from + e);
      } else {
        const uint32_t x = kv_load(reinterpret_cast<const uint16_t*>(logits) + from + e);
        w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xFFFFu) | (x << 16) : (w[e >> 1] & 0xFFFF0000u) | x;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // f(piece, its number) for this thread's pieces, the next one's load ahead of it.  (Two pieces a round make loops
  // that pass what an SM holds of instructions close by: a seventh of the warps' time, without filters.)
  template <typename F>
  __device__ __forceinline__ void each_piece(F f) const {
    uint4 next = nothing();
    if (begin + lane < end) next = piece(begin + lane);
#pragma unroll 1
    for (int i = begin + lane; i < end; i += 32) {
      const uint4 v = next;
      if (i + 32 < end) next = piece(i + 32);
      f(v, i);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each_piece([&](const uint4& v, int i) {
      float x[VEC];
      unpack<E>(v, x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f(x[e], static_cast<uint32_t>(index0 + i * VEC + e));
    });
  }
  // The weight of what is kept of this thread's elements.
  __device__ __forceinline__ u64 mass_of(const Weigher& weigh, const Cut& kept) const {
    u64 sum = 0;
    const float from = fmaxf(kept.x, weigh.least);
    each_piece([&](const uint4& v, int i) {
      float x[VEC];
      unpack<E>(v, x);
      if (kept.i == kNone) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) weigh.add2_to(sum, from, x[e], x[e + 1]);
      } else {
        const uint32_t index = static_cast<uint32_t>(index0 + i * VEC);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          u64 w[2];
          weigh.two(x[e], x[e + 1], w[0], w[1]);
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (x[e + y] >= from && kept(x[e + y], index + e + y)) sum += w[y];
        }
      }
    });
    return sum;
  }

  // Sums of v (below 2^53 each) over the CTA, at every thread, and over the warps, at warp_sums().  Two places in
  // turn: a call's numbers are read before the next one's barrier.
  __device__ __forceinline__ u64* warp_sums() const { return sh.warp_sum[sums & 1]; }
  __device__ __forceinline__ u64 block_total(u64 v) {
    v = warp_total(v);
    ++sums;
    if (lane == 0) warp_sums()[warp] = v;
    __syncthreads();
    u64 sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += warp_sums()[w];
    return sum;
  }
  // Sum of v over the threads before this one; *total over all.
  __device__ __forceinline__ u64 block_before(u64 v, u64* total) {
    const u64 run = warp_running(v, lane);
    ++sums;
    if (lane == 31) warp_sums()[warp] = run;
    __syncthreads();
    u64 before = run - v, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const u64 x = warp_sums()[w];
      sum += x;
      if (w < warp) before += x;
    }
    *total = sum;
    return before;
  }
  // The smallest a and the largest b over the CTA, at every thread.
  __device__ __forceinline__ void block_range(uint32_t& a, uint32_t& b) {
    a = __reduce_min_sync(0xFFFFFFFFu, a);
    b = __reduce_max_sync(0xFFFFFFFFu, b);
    ++sums;
    uint2* place = reinterpret_cast<uint2*>(warp_sums());
    if (lane == 0) place[warp] = make_uint2(a, b);
    __syncthreads();
    const uint2 x = place[lane % kWarps];
    a = __reduce_min_sync(0xFFFFFFFFu, x.x);
    b = __reduce_max_sync(0xFFFFFFFFu, x.y);
  }

  // The first element, in the vocabulary's order, at which the running sum of f exceeds the target that
  // `target` makes of the total; `hit` is called by the one thread that holds it.  mine, summed over a warp: f of
  // its elements.  One meeting of the cluster.
  template <typename F, typename T, typename H>
  __device__ __forceinline__ void find(u64 mine, F f, T target, H hit) {
    u64 before, total;
    const u64 sum = block_total(mine), t = place_in_row(sum, target, &before, &total);
    if (t < before || t >= before + sum) return;
    // All warps take a part of the one's that has it, a second time of that part's.
    int from = 0, to = 0;
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      int w = 0;
      for (; w < kWarps - 1 && t >= before + warp_sums()[w]; ++w) before += warp_sums()[w];
      if (level == 0) {
        const int each_warp = (slice + kWarps - 1) / kWarps;
        from = min(w * each_warp, slice);
        to = min(from + each_warp, slice);
      } else {
        const int part = (to - from + kWarps - 1) / kWarps;
        from = min(from + w * part, to);
        to = min(from + part, to);
      }
      if (to - from <= 32) break;
      const int part = (to - from + kWarps - 1) / kWarps;
      const int a = min(from + warp * part, to), b = min(a + part, to);
      u64 own = 0;
#pragma unroll 1
      for (int i = a + lane; i < b; i += 32) {
        float x[VEC];
        unpack<E>(piece(i), x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) own += f(x[e], static_cast<uint32_t>(index0 + i * VEC + e));
      }
      block_total(own);
    }
    if (warp != 0) return;
#pragma unroll 1
    for (int i0 = from; i0 < to; i0 += 32) {
      const int i = i0 + lane;
      u64 own = 0;
      if (i < to) {
        float x[VEC];
        unpack<E>(piece(i), x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) own += f(x[e], static_cast<uint32_t>(index0 + i * VEC + e));
      }
      const u64 run = before + warp_running(own, lane);
      const uint32_t over = __ballot_sync(0xFFFFFFFFu, run > t);
      if (over != 0) {
        if (lane == __ffs(over) - 1) {
          u64 upto = run - own;
#pragma unroll 1
          for (int e = 0; e < VEC; ++e) {
            const int index = index0 + i * VEC + e;
            if (index < 0 || index >= V) continue;
            const float x = element(index);
            upto += f(x, static_cast<uint32_t>(index));
            if (upto > t) {
              hit(x, static_cast<uint32_t>(index), total);
              break;
            }
          }
        }
        return;
      }
      before = __shfl_sync(0xFFFFFFFFu, run, 31);
    }
  }
  // What `target` makes of the total over the CTAs, that total, and the sum over the CTAs before this one.  One
  // meeting of the cluster.
  template <typename T>
  __device__ __forceinline__ u64 place_in_row(u64 sum, T target, u64* before, u64* total) {
    const int set = turn++ & 1;
    if (tid < ctas) at(tid)->mass[set][rank] = sum;
    cluster.sync();
    *total = *before = 0;
    for (int c = 0; c < ctas; ++c) {
      if (c < rank) *before += sh.mass[set][c];
      *total += sh.mass[set][c];
    }
    return target(*total);
  }

  // Elements that `take` accepts into the first CTA's list, and how many there are; nothing is listed when they are
  // too many.  Meetings: one, and a second when they fit.
  template <typename F>
  __device__ __forceinline__ uint32_t gather(F take) {
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    each([&](float x, uint32_t i) {
      if (take(x, i)) enlist(x, i);
    });
    __syncthreads();
    const int set = turn++ & 1;
    if (tid < ctas) at(tid)->count[set][rank] = sh.listed;
    cluster.sync();
    return lists_to_first(set);
  }
  __device__ __forceinline__ void enlist(float x, uint32_t i) {
    const uint32_t to = atomicAdd(&sh.listed, 1u);
    if (to < kList) sh.list[to] = ckey(x, static_cast<int>(i));
  }
  // The CTAs' lists, of sh.count[set] elements, to the first one's; how many they are.
  __device__ __forceinline__ uint32_t lists_to_first(int set) {
    uint32_t n = 0;
    for (int c = 0; c < ctas; ++c) n += sh.count[set][c];   // (of at most 2^20 elements)
    if (n > kList || ctas == 1) return n;
    if (rank == 0) {
      const uint32_t own = sh.count[set][0];
      for (uint32_t to = own + tid; to < n; to += kThreads) {
        uint32_t i = to - own;
        int c = 1;
        while (i >= sh.count[set][c]) i -= sh.count[set][c++];
        sh.list[to] = at(c)->list[i];
      }
    }
    cluster.sync();
    return n;
  }
  // The smallest and largest element that `take` accepts (by ord_f32), over the row.  One meeting.
  template <typename F>
  __device__ __forceinline__ void range_of(F take, uint32_t* least, uint32_t* most) {
    uint32_t a = kNone, b = 0;
    each([&](float x, uint32_t i) {
      if (take(x, i)) {
        a = min(a, ord_f32(x));
        b = max(b, ord_f32(x));
      }
    });
    block_range(a, b);
    const int set = turn++ & 1;
    if (tid < ctas) {
      at(tid)->lo[set][rank] = a;
      at(tid)->hi[set][rank] = b;
    }
    cluster.sync();
    for (int c = 0; c < ctas; ++c) {
      a = min(a, sh.lo[set][c]);
      b = max(b, sh.hi[set][c]);
    }
    *least = a;
    *most = b;
  }
  // The cut that the first CTA finds in its list of n.  One meeting.
  template <bool MASS, typename F>
  __device__ __forceinline__ Cut cut_of_list(uint32_t n, u64 above, u64 target, F f) {
    if (rank == 0) {
      cut_list<MASS>(n, above, target, [&](u64 key) { return f(ckey_score(key)); });
      if (tid > 0 && tid < ctas) at(tid)->answer = sh.answer;
    }
    cluster.sync();
    return cut_at(sh.answer);
  }

  // Of each of the list's n <= kPairs elements, by thread i < n: how many of the others come before it and what
  // they weigh; before: by key, or by index.
  __device__ __forceinline__ void pair_sums(uint32_t n, bool by_index, uint32_t* rank_of, u64* before) {
    const int log = n <= 32 ? 5 : n <= 64 ? 6 : n <= 128 ? 7 : 8, parts = kThreads >> log;
    const uint32_t i = tid & ((1 << log) - 1), part = tid >> log;
    __syncthreads();
    u64 sum = 0;
    uint32_t count = 0;
    if (i < n) {
      const u64 mask = by_index ? 0xFFFFFFFFull : ~0ull, key = sh.list[i] & mask;
#pragma unroll 4
      for (uint32_t j = part; j < n; j += parts) {
        const u64 other = sh.list[j] & mask, w = sh.weights[j];
        const bool first = other > key;              // (a larger key: a larger value, or a smaller index)
        sum += first ? w : 0;
        count += first ? 1 : 0;
      }
    }
    sh.part_mass[tid] = sum;
    sh.part_rank[tid] = count;
    __syncthreads();
    if (tid < (1 << log)) {
#pragma unroll 4
      for (int x = 1; x < parts; ++x) {
        sum += sh.part_mass[tid + (x << log)];
        count += sh.part_rank[tid + (x << log)];
      }
    }
    *rank_of = count;
    *before = sum;
  }

  // The list's n keys, descending; thread t gets places [P t, P t + P).  The list's memory is used.
  static constexpr int P = kList / kThreads;
  __device__ __forceinline__ void sort_list(uint32_t n, u64 (&v)[P]) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = tid * P + e < n ? sh.list[tid * P + e] : 0;
    __syncthreads();
    block_sort_regs<P, true>(v, sh.list);
  }

  // The key of the list's element at which the running sum of f (of keys), in descending order and from `above`, reaches
  // `target`, to sh.answer.  First CTA only.  Long lists are cut by a histogram first.
  template <bool MASS, typename F>
  __device__ void cut_list(uint32_t n, u64 above, u64 target, F f) {
    u64 v[P];
    __syncthreads();
#pragma unroll 1
    while (n > kPairs) {
      uint32_t a = kNone, b = 0;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        v[e] = tid + e * kThreads < n ? sh.list[tid + e * kThreads] : 0;
        if (v[e] != 0) {
          a = min(a, static_cast<uint32_t>(v[e] >> 32));
          b = max(b, static_cast<uint32_t>(v[e] >> 32));
        }
      }
      block_range(a, b);
      if (a == b) break;
      const Bins bins(unord_f32(a), unord_f32(b));
      if (tid == 0) sh.listed = 0;
      clear_bins();
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (v[e] != 0) add_to_bin<MASS>(bins(ckey_score(v[e])), f(v[e]));
      __syncthreads();
      for (int i = tid; i < kBins; i += kThreads) sh.merged[i] = bin_sum<MASS>(sh, i);
      above = find_bin(above, target);
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (v[e] != 0 && bins(ckey_score(v[e])) == static_cast<int>(sh.found)) sh.list[atomicAdd(&sh.listed, 1u)] = v[e];
      __syncthreads();
      n = sh.listed;
      __syncthreads();
    }
    if (n > kPairs) {                    // equal values
      sort_list(n, v);
      u64 w[P], own = 0;
#pragma unroll
      for (int e = 0; e < P; ++e) own += w[e] = tid * P + e < n ? f(v[e]) : 0;
      u64 all, run = above + block_before(own, &all);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        if (run < target && run + w[e] >= target) sh.answer = v[e];
        run += w[e];
      }
    } else {
      uint32_t ignored;
      u64 before = 0, own = 0;
      if (tid < n) own = sh.weights[tid] = f(sh.list[tid]);
      pair_sums(n, false, &ignored, &before);
      before += above;
      if (tid < n && before < target && before + own >= target) sh.answer = sh.list[tid];
    }
    __syncthreads();
  }

  __device__ __forceinline__ void clear_bins() {
    for (int i = tid; i < 3 * kBins; i += kThreads) sh.hist[i / kBins][i % kBins] = 0;
    __syncthreads();
  }
  template <bool MASS>
  __device__ __forceinline__ void add_to_bin(int b, u64 w) {
    if constexpr (MASS) {
      const uint32_t w0 = static_cast<uint32_t>(w) & 0x7FFFu, w1 = static_cast<uint32_t>(w >> 15) & 0x7FFFu;
      const uint32_t w2 = static_cast<uint32_t>(w >> 30);
      atomicAdd(&sh.hist[0][b], w0);
      atomicAdd(&sh.hist[1][b], w1);
      if (w2 != 0) atomicAdd(&sh.hist[2][b], w2);
    } else {
      atomicAdd(&sh.hist[0][b], 1u);
    }
  }
  template <bool MASS>
  __device__ __forceinline__ u64 bin_sum(const Shared& of, int b) const {
    u64 sum = of.hist[0][b];
    if (MASS) sum += (static_cast<u64>(of.hist[1][b]) << 15) + (static_cast<u64>(of.hist[2][b]) << 30);
    return sum;
  }
  // The first of the merged bins, from the top, at which the running sum from `above` reaches the target: at
  // sh.found; returns the sum before it.
  __device__ __forceinline__ u64 find_bin(u64 above, u64 target) {
    constexpr int kEach = kBins / kThreads;
    __syncthreads();
    u64 own = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) own += sh.merged[tid * kEach + e];
    u64 all, run = above + block_before(own, &all);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const u64 w = sh.merged[tid * kEach + e];
      if (run < target && run + w >= target) {
        sh.found = tid * kEach + e;
        sh.found_before = run;
      }
      run += w;
    }
    __syncthreads();
    return sh.found_before;
  }

  // The CTAs' histograms, summed into every CTA's `merged`.  Two meetings.
  template <bool MASS>
  __device__ __forceinline__ void merge_bins() {
    cluster.sync();
    const int part = (kBins + ctas - 1) / ctas;
    for (int b = rank * part + tid; b < min((rank + 1) * part, kBins); b += kThreads) {
      u64 sum = 0;
      for (int c = 0; c < ctas; ++c) sum += bin_sum<MASS>(*at(c), b);
      for (int c = 0; c < ctas; ++c) at(c)->merged[b] = sum;
    }
    cluster.sync();
  }
  // Of the kept elements with lo <= x <= hi, in descending order: where the running sum of f, from `above`, reaches
  // `target` (with all of them it does).  MASS: f are weights, else ones.
  template <bool MASS, typename F>
  __device__ Cut select(float lo, float hi, const Cut kept, u64 above, u64 target, F f) {
#pragma unroll 1
    while (true) {
      const Bins bins(lo, hi);
      auto inside = [&](float x, uint32_t i) { return x >= lo && x <= hi && kept(x, i); };
      int bin = 0;
      if (lo < hi) {
        clear_bins();
        each([&](float x, uint32_t i) {
          if (inside(x, i)) add_to_bin<MASS>(bins(x), f(x));
        });
        merge_bins<MASS>();
        above = find_bin(above, target);
        bin = sh.found;
      }
      auto there = [&](float x, uint32_t i) { return inside(x, i) && (!(lo < hi) || bins(x) == bin); };
      const uint32_t n = gather(there);
      if (n <= kList) return cut_of_list<MASS>(n, above, target, f);
      if (!(lo < hi)) {
        // equal values, more than a list holds: the last one is found by its index
        const u64 one = f(lo), need = (target - above + one - 1) / one;
        u64 mine = 0;
        each([&](float x, uint32_t i) { mine += inside(x, i) ? 1 : 0; });
        find(mine, [&](float x, uint32_t i) { return inside(x, i) ? 1ull : 0ull; }, [&](u64) { return need - 1; },
             [&](float x, uint32_t i, u64) {
               for (int c = 0; c < ctas; ++c) at(c)->answer = ckey(x, static_cast<int>(i));
             });
        cluster.sync();
        return cut_at(sh.answer);
      }
      // the bin's own range is the next one
      uint32_t a, b;
      range_of(there, &a, &b);
      lo = unord_f32(a);
      hi = unord_f32(b);
    }
  }

  // The first k of the elements with lo <= x <= hi, in descending order; nothing below lo that *kept lets through weighs
  // anything.  True: they and few others, n in all and none smaller, are in the first CTA's list.  Else *kept is cut, where
  // there are more than k.  About all are above guess >= lo.
  __device__ bool first_k(float lo, float guess, float hi, int k, Cut* kept, uint32_t* n) {
    const Bins bins(guess, hi);
    clear_bins();
    each([&](float x, uint32_t) {
      if (x >= lo) atomicAdd(&sh.hist[0][bins(x)], 1u);
    });
    merge_bins<false>();
    u64 own = 0;
    for (int i = tid; i < kBins; i += kThreads) own += sh.merged[i];
    if (block_total(own) <= static_cast<u64>(k)) return false;
    const u64 above = find_bin(0, k), there = sh.merged[sh.found];
    const int bin = static_cast<int>(sh.found);
    if (above + there <= kList) {
      *n = gather([&](float x, uint32_t) { return x >= lo && bins(x) <= bin; });
      return true;
    }
    auto one = [](float) { return 1ull; };
    auto in_bin = [&](float x, uint32_t) { return x >= lo && bins(x) == bin; };
    if (there <= kList) {
      *kept = cut_of_list<false>(gather(in_bin), above, k, one);
      return false;
    }
    uint32_t a, b;
    range_of(in_bin, &a, &b);
    *kept = select<false>(unord_f32(a), unord_f32(b), *kept, above, k, one);
    return false;
  }

  // The end of what `bins` puts into bins from `bin` on (up: or into those up to `bin`): the largest x (smallest x) of
  // those, by ord_f32, between lo and hi, of which one is there at least.  By a whole warp.
  template <typename B>
  __device__ __forceinline__ float edge_of(const B& bins, uint32_t lo, uint32_t hi, int bin, bool up) const {
    while (lo < hi) {
      // 32 places up to the other end; those that are in come first
      const uint32_t step = static_cast<uint32_t>((static_cast<u64>(hi - lo) * (lane + 1) + 31) / 32);
      const uint32_t x = up ? hi - step : lo + step;
      const int n = __popc(__ballot_sync(0xFFFFFFFFu, up ? bins(unord_f32(x)) <= bin : bins(unord_f32(x)) >= bin));
      const uint32_t last = __shfl_sync(0xFFFFFFFFu, x, max(n - 1, 0)), next = __shfl_sync(0xFFFFFFFFu, x, min(n, 31));
      if (up) {
        if (n > 0) hi = last;
        if (n < 32) lo = next + 1;
      } else {
        if (n > 0) lo = last;
        if (n < 32) hi = next - 1;
      }
    }
    return unord_f32(up ? hi : lo);
  }

  // Where the weights of the kept elements, in descending order, reach the share p of their sum.  *mine, summed
  // over a warp: what is kept then of its elements weighs.
  //
  // A histogram of rough weights shows in which few bins the cut can be; one pass with exact weights then sums what lies
  // above them and all, and lists what is in them.  A rough weight is that of the bin's upper edge, times a share of it
  // for the place within the bin, by two terms of a series: no exponential, no conversion, and no sum needed first to
  // scale them.  (With exponentials scaled by the row's sum, a pass of its own, top-p of 192 rows of 131071 took 162 us.)
  __device__ Cut select_share(float hi, const Cut kept, float p, const Weigher& weigh, u64* mine) {
    const bool simple = kept.i == kNone; // no cut among equal elements so far
    const float least = fmaxf(kept.x, fmaxf(weigh.least, -__int_as_float(0x7F7FFFFF)));
    // V elements of less than (1 - p) / V of the largest cannot hold what is left out, so the cut is above that; and
    // of less than 2^-15 / V they do not count here
    const float lo = fmaxf(least, fminf(hi, hi + (log2f(fminf(1.f - p, 0x1p-15f) / V) - 0x1p-5f) / weigh.ch - 0x1p-20f * fabsf(hi)));
    const BinsOf<kFineBins> bins(lo, hi);
    const float width = weigh.ch * (hi / kFineBins - lo / kFineBins);        // of a bin, in powers of two: 42 / 2048 at most
    // a bin's sum in units of 2^-bits of its edge's weight stays below 2^32
    const int bits = min(__clz(longest * VEC) - 1, 20);
    const float one = __int_as_float((127 + bits) << 23), a1 = one * -0.6931471806f * width, a2 = one * 0.2402265070f * width * width;
    for (int i = tid; i < kFineBins; i += kThreads) sh.fine[i] = 0;
    __syncthreads();
    each([&](float x, uint32_t i) {
      if (x >= lo && (simple || kept(x, i))) {
        const float t = bins.place(x), whole = __fadd_rd(t, 0x1p23f), rest = t - (whole - 0x1p23f);
        const float w = fmaf(rest, fmaf(rest, a2, a1), one) + 0x1p23f;
        atomicAdd(&sh.fine[bins.number(whole)], __float_as_uint(w) & 0x7FFFFFu);
      }
    });
    cluster.sync();
    {
      const int part = (kFineBins + ctas - 1) / ctas;
      for (int b = rank * part + tid; b < min((rank + 1) * part, kFineBins); b += kThreads) {
        u64 sum = 0;
        for (int c = 0; c < ctas; ++c) sum += at(c)->fine[b];
        // (all together below 2^34 units of 2^-bits of the largest weight, in 2^-16 of those)
        const u64 w = __float2ull_rz(static_cast<float>(sum) * (0x1p16f * exp2_approx(-width * b)));
        for (int c = 0; c < ctas; ++c) at(c)->merged_fine[b] = w;
      }
    }
    cluster.sync();
    {
      constexpr int kEach = kFineBins / kThreads;
      u64 w[kEach], own = 0, total;
#pragma unroll
      for (int e = 0; e < kEach; ++e) own += w[e] = sh.merged_fine[tid * kEach + e];
      u64 run = block_before(own, &total);
      // weights, and so their sum, are off by less than 2^-15 of themselves (the series 2^-21, places rounded three times
      // 2^-16.5, the edges' weights 2^-18), and by their unit; 2^-15 of the sum may be missing
      const float sum = static_cast<float>(total), off = sum * (0x1p-14f + 1.f / one);
      const u64 at_least = __float2ull_rz(fmaxf(sum * p - off, 0.f)), at_most = __float2ull_ru(sum * p + off);
      if (tid == 0) {
        sh.reached_bin[0] = kFineBins - 1;
        sh.reached_bin[1] = kFineBins - 1;
        sh.listed = 0;
      }
      if (tid < kWarps) sh.listed_sum[tid] = 0;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const u64 before = run;
        run += w[e];
        if (before < at_least && run >= at_least) sh.reached_bin[0] = tid * kEach + e;
        if (before < at_most && run >= at_most) sh.reached_bin[1] = tid * kEach + e;
      }
      if (tid == 0 && at_least == 0) sh.reached_bin[0] = 0;
      __syncthreads();
      // those bins as a range of x: above it is what lies in bins before them
      if (warp < 2) {
        const float x = edge_of(bins, ord_f32(lo), ord_f32(hi), sh.reached_bin[warp], warp == 1);
        if (lane == 0) sh.edge[warp] = x;
      }
      __syncthreads();
    }
    // (a first bin without any x: the edge is that of the bins after it)
    const float from = sh.edge[1], upto = sh.edge[0];
    u64 all = 0, above = 0;
    each_piece([&](const uint4& v, int i) {
      float x[VEC];
      unpack<E>(v, x);
      const uint32_t index = static_cast<uint32_t>(index0 + i * VEC);
      if (simple) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) weigh.add2_to(all, above, least, upto, x[e], x[e + 1]);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (x[e] >= from && x[e] <= upto) enlist(x[e], index + e);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          u64 w[2];
          weigh.two(x[e], x[e + 1], w[0], w[1]);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (!(x[e + y] >= least && kept(x[e + y], index + e + y))) continue;
            all += w[y];
            if (x[e + y] > upto) above += w[y];
            else if (x[e + y] >= from) enlist(x[e + y], index + e + y);
          }
        }
      }
    });
    *mine = above;
    const u64 cta_above = block_total(above), cta_all = block_total(all);
    const int set = turn++ & 1;
    if (tid < ctas) {
      at(tid)->mass[set][rank] = cta_above;
      at(tid)->all[rank] = cta_all;
      at(tid)->count[set][rank] = sh.listed;
    }
    u64 own[P];                          // this CTA's listed ones (the first one's list is used up)
    const uint32_t listed = sh.listed;
#pragma unroll
    for (int e = 0; e < P; ++e) own[e] = tid + e * kThreads < listed ? sh.list[tid + e * kThreads] : 0;
    cluster.sync();
    above = 0;
    u64 total = 0;
    for (int c = 0; c < ctas; ++c) {
      above += sh.mass[set][c];
      total += sh.all[c];
    }
    const u64 target = share_of(p, total);
    const uint32_t n = lists_to_first(set);
    Cut end;
    if (n <= kList) {
      end = cut_of_list<true>(n, above, target, weigh);
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (own[e] != 0 && end(ckey_score(own[e]), static_cast<uint32_t>(ckey_idx(own[e]))))
          atomicAdd(&sh.listed_sum[(ckey_idx(own[e]) - index0) / VEC / ((slice + kWarps - 1) / kWarps)], weigh(ckey_score(own[e])));
      __syncthreads();
      if (lane == 0) *mine += sh.listed_sum[warp];
    } else {
      end = select<true>(from, upto, kept, above, target, weigh);
      each([&](float x, uint32_t i) {
        if (x >= from && x <= upto && x >= least && kept(x, i) && end(x, i)) *mine += weigh(x);
      });
    }
    return end;
  }

  // For need[0] and need[1]: a bound that at least so many of the threads' largest elements reach (keys by ord_f32; on:
  // this thread's counts, they lie in [lo, hi]), to sh.reached; 0 where there are not so many.  By a histogram
  // of them; sh.hist[0] is zero before and after.
  __device__ __forceinline__ void reached_by(const int (&need)[2], bool on, uint32_t key, uint32_t lo, uint32_t hi) {
    const Bins bins(unord_f32(lo), unord_f32(hi));           // (all in the first bin where lo == hi)
    const int bin = on ? bins(unord_f32(key)) : -2;
    if (tid < 2) {
      sh.reached[tid] = 0;
      sh.reached_bin[tid] = -1;
    }
    if (on) atomicAdd(&sh.hist[0][bin], 1u);
    __syncthreads();
    constexpr int kEach = kBins / kThreads;
    uint32_t mine[kEach], run = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      run += mine[e] = sh.hist[0][tid * kEach + e];
      sh.hist[0][tid * kEach + e] = 0;
    }
    uint32_t upto = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += x;
    }
    ++sums;
    if (lane == 31) warp_sums()[warp] = upto;
    __syncthreads();
    upto -= run;
    for (int w = 0; w < warp; ++w) upto += static_cast<uint32_t>(warp_sums()[w]);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (upto < static_cast<uint32_t>(need[x]) && upto + mine[e] >= static_cast<uint32_t>(need[x])) {
          sh.reached_bin[x] = tid * kEach + e;
          sh.reached[x] = kNone;
        }
      upto += mine[e];
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (bin == sh.reached_bin[x]) atomicMin(&sh.reached[x], key);
    __syncthreads();
  }

  // All that is kept is in the list: filters and draw, by the first CTA.
  template <typename H>
  __device__ void finish(uint32_t n, int k, float top_p, float u, const Weigher& weigh, H hit) {
    if (n <= kPairs) {
      uint32_t place = 0;
      u64 before = 0, w = 0, key = 0;
      if (tid < n) {
        key = sh.list[tid];
        w = sh.weights[tid] = weigh(ckey_score(key));
      }
      pair_sums(n, false, &place, &before);
      bool kept = tid < n && (k == 0 || place < static_cast<uint32_t>(k));
      if (top_p < 1.f) {
        const u64 enough = share_of(top_p, block_total(kept ? w : 0));
        kept = kept && before < enough;
      }
      w = kept ? w : 0;
      const u64 total = block_total(w), to = place_of(u, total);
      // the kept ones come first in the order: they take the first places of the list
      const uint32_t left = __syncthreads_count(kept);
      if (kept) {
        sh.list[place] = key;
        sh.weights[place] = w;
      }
      __syncthreads();
      if (tid < left) {
        key = sh.list[tid];
        w = sh.weights[tid];
      } else {
        w = 0;
      }
      pair_sums(left, true, &place, &before);
      if (before <= to && to < before + w) hit(ckey_score(key), static_cast<uint32_t>(ckey_idx(key)), total);
      return;
    }
    // each thread keeps its keys, as the cuts use up the list
    u64 v[P];
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = tid + e * kThreads < n ? sh.list[tid + e * kThreads] : 0;
    auto total_of = [&]() {
      u64 own = 0;
#pragma unroll
      for (int e = 0; e < P; ++e) own += v[e] != 0 ? weigh(ckey_score(v[e])) : 0;
      return block_total(own);
    };
    auto list_again = [&](auto key_of) {
      __syncthreads();
      if (tid == 0) sh.listed = 0;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (v[e] != 0) sh.list[atomicAdd(&sh.listed, 1u)] = key_of(v[e]);
      __syncthreads();
      return sh.listed;
    };
    auto cut = [&]() {
      const Cut c = cut_at(sh.answer);
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (v[e] != 0 && !c(ckey_score(v[e]), static_cast<uint32_t>(ckey_idx(v[e])))) v[e] = 0;
    };
    if (k > 0 && static_cast<uint32_t>(k) < n) {
      cut_list<false>(n, 0, k, [](u64) { return 1ull; });
      cut();
    }
    u64 total = total_of();
    if (top_p < 1.f) {
      cut_list<true>(list_again([](u64 key) { return key; }), 0, share_of(top_p, total), [&](u64 key) { return weigh(ckey_score(key)); });
      cut();
      total = total_of();
    }
    // in the vocabulary's order: (-index, x) takes the place of (x, index); an index is exact in fp32
    cut_list<true>(list_again([](u64 key) {
                     return (static_cast<u64>(ord_f32(-static_cast<float>(ckey_idx(key)))) << 32) | (key >> 32);
                   }), 0, place_of(u, total) + 1, [&](u64 key) { return weigh(unord_f32(static_cast<uint32_t>(key))); });
    if (tid == 0) hit(unord_f32(static_cast<uint32_t>(sh.answer)), static_cast<uint32_t>(-ckey_score(sh.answer)), total);
  }
};

template <typename E>
__global__ void __launch_bounds__(kThreads, 4) sample_tokens_kernel(const __grid_constant__ SamplingParams p) {
  __shared__ Shared sh;
  constexpr int VEC = 16 / sizeof(E);
  const float inf = __int_as_float(0x7F800000);
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = p.ctas, rank = static_cast<int>(blockIdx.x) % ctas, b = static_cast<int>(blockIdx.x) / ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 512; i += kThreads) sh.pow[i] = kPow.v[i];
  for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = 0;
  if (tid == 0) {
    sh.found = kNone;
    sh.listed = 0;
    sh.early = 0;
  }
  cluster.barrier_arrive();

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

  const E* logits = reinterpret_cast<const E*>(p.logits) + static_cast<size_t>(b) * p.stride;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(logits) & 15u) / sizeof(E));
  const int pieces = (p.V + shift + VEC - 1) / VEC;
  const int first = min(rank * p.per, pieces), mine = min(p.per, pieces - first);
  const int per_warp = (mine + kWarps - 1) / kWarps;
  Row<E> row{sh, logits, p.V, cluster, tid, lane, warp, rank, ctas, mine, p.per, min(warp * per_warp, mine), min((warp + 1) * per_warp, mine),
             first * VEC - shift};
  Largest<E> largest;
  // A small top-k: what k threads' first elements reach is a bound that the cut is not below, and elements at or above it
  // are listed while the slice is read, or what is kept would have to be looked for again (256 rows of 131072: 51 us, not 38).
  const bool all_listed = p.V <= kList, few = k > 0 && k <= kThreads / 4 * ctas && k <= kPairs;
  const bool early = few && !all_listed;
  const int needs[2] = {(k + ctas - 1) / ctas, k};
  float bound = inf;
  auto run_at = [&](int i0, uint4 (&v)[kRun]) {
#pragma unroll
    for (int j = 0; j < kRun; ++j) v[j] = i0 + 32 * j < row.end ? row.piece(i0 + 32 * j) : row.nothing();
  };
  {
    uint4 v[kRun];
    run_at(row.begin + lane, v);
    cluster.barrier_wait();              // the others have begun, and their shared memory can be written
    if (k > 0 && !few) {
      // about the smallest
      uint32_t lo = kNone, ignored = 0;
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        float x[VEC];
        unpack<E>(v[j], x);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (x[e] > -inf) lo = min(lo, ord_f32(x[e]));
      }
      row.block_range(lo, ignored);
      if (tid < ctas) row.at(tid)->least[rank] = lo;
    }
    if (early) {
      Largest<E> first;
#pragma unroll
      for (int j = 0; j < kRun; ++j) first.add(v[j]);
      const float first_most = first.get();
      const uint32_t key = first_most == first_most ? ord_f32(first_most) : kNone;
      const bool some = key > ord_f32(-inf);
      uint32_t lo = some ? key : kNone, hi = key;
      row.block_range(lo, hi);
      if (hi < ord_f32(inf) && hi > ord_f32(-inf)) {
        row.reached_by(needs, some, key, lo, hi);
        if (sh.reached[1] != 0) bound = unord_f32(sh.reached[1]);
      }
    }
#pragma unroll 1
    for (int i0 = row.begin + lane;;) {
      if (!early) {
#pragma unroll
        for (int j = 0; j < kRun; ++j) largest.add(v[j]);
      }
#pragma unroll
      for (int j = 0; j < kRun && early; ++j) {
        Largest<E> of_piece;
        of_piece.add(v[j]);
        largest.with(of_piece);
        if (!(of_piece.get() >= bound)) continue;
        float x[VEC];
        unpack<E>(v[j], x);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (x[e] >= bound) {
            const uint32_t to = atomicAdd(&sh.early, 1u);
            if (to < kEarly) {
              sh.early_x[to] = x[e];
              sh.early_i[to] = static_cast<uint32_t>(row.index0 + (i0 + 32 * j) * VEC + e);
            }
          }
      }
      i0 += 32 * kRun;
      if (i0 >= row.end) break;
      run_at(i0, v);
    }
  }
  const float most = largest.get();      // NaN if any element is
  // Few enough are kept for one CTA: all of a small vocabulary, or a small top-k.  For that each CTA finds
  // what its share of k elements reach, and what k of them do, by its threads' largest: k elements of the row reach
  // the least of the CTAs' former bounds, and any of the latter.
  {
    const uint32_t key = most == most ? ord_f32(most) : kNone;   // (above +inf)
    const bool some = key > ord_f32(-inf);
    uint32_t lo = some ? key : kNone, hi = key;
    row.block_range(lo, hi);
    const bool look = few && !all_listed && hi < ord_f32(inf) && hi > ord_f32(-inf);
    if (look && per_warp > 32 * kRun) row.reached_by(needs, some, key, lo, hi);   // (else those are all elements)
    if (tid < ctas) {
      Shared* o = row.at(tid);
      o->top[rank] = hi;
      o->bound[0][rank] = look ? sh.reached[0] : 0;
      o->bound[1][rank] = look ? sh.reached[1] : 0;
    }
  }
  cluster.sync();
  uint32_t m_key = 0, floor_key = kNone, by_one = 0;
  for (int c = 0; c < ctas; ++c) {
    m_key = max(m_key, sh.top[c]);
    floor_key = min(floor_key, sh.bound[0][c]);
    by_one = max(by_one, sh.bound[1][c]);
  }
  floor_key = max(floor_key, by_one);
  const bool bad = m_key >= ord_f32(inf);
  int* token = p.token + b;
  float* logp = p.logp + b;
  if (!settings || bad || m_key == ord_f32(-inf)) {
    if (rank == 0 && tid == 0) {
      *token = -1;
      *logp = settings && !bad ? -inf : __int_as_float(0x7FC00000);
    }
    return;
  }
  const float m = unord_f32(m_key);
  if (T < 0x1p-127f) {                   // (1 / T would pass fp32) the largest, the first of equal ones
    uint32_t at = kNone;
    if (most == m) row.each([&](float x, uint32_t i) { at = x == m && i < at ? i : at; });
    if (at != kNone) atomicMin(cluster.map_shared_rank(&sh.found, 0), at);
    cluster.sync();
    if (rank == 0 && tid == 0) {
      *token = static_cast<int>(sh.found);
      *logp = 0.f;
    }
    return;
  }
  const Weigher weigh(m, T, sh.pow);
  auto hit = [&](float x, uint32_t i, u64 total) {
    *token = static_cast<int>(i);
    // what is (nearly) certain by what is left, of which the weights know as many bits (nothing, for the only one kept)
    const u64 rest = total - weigh(x);
    *logp = rest < total >> 7 ? log1pf(-__ull2float_rn(rest) / __ull2float_rn(total)) + 0.f : weigh.log_share(x, total);
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
    // each CTA's straight into its part of the first one's list
    const float from = fmaxf(unord_f32(floor_key), least);
    const uint32_t room = kList / ctas;
    u64* list = row.at(0)->list + rank * room;
    auto push = [&](float x, uint32_t i) {
      const uint32_t to = atomicAdd(&sh.listed, 1u);
      if (to < room) list[to] = ckey(x, static_cast<int>(i));
    };
    auto push_piece = [&](const uint4& v, int i) {
      float x[VEC];
      unpack<E>(v, x);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (x[e] >= from) push(x[e], static_cast<uint32_t>(row.index0 + i * VEC + e));
    };
    const bool again = bound == inf || sh.early > kEarly;    // (the same for all threads)
    if (again) {
      if (most >= from) row.each_piece(push_piece);
    } else {
      for (uint32_t j = tid; j < sh.early; j += kThreads)
        if (sh.early_x[j] >= from) push(sh.early_x[j], sh.early_i[j]);
    }
    __syncthreads();
    const int set = row.turn++ & 1;
    if (tid < ctas) row.at(tid)->count[set][rank] = sh.listed;
    cluster.sync();
    uint32_t n = 0;
    bool fits = true;
    for (int c = 0; c < ctas; ++c) {
      n += sh.count[set][c];
      fits = fits && sh.count[set][c] <= room;
    }
    if (fits) {
      if (rank == 0) {
        if (ctas > 1) {                  // close the gaps
          u64 v[kList / kThreads];
#pragma unroll
          for (int e = 0; e < kList / kThreads; ++e) {
            uint32_t i = tid + e * kThreads;
            if (i >= n) continue;
            int c = 0;
            while (i >= sh.count[set][c]) i -= sh.count[set][c++];
            v[e] = sh.list[c * room + i];
          }
          __syncthreads();
#pragma unroll
          for (int e = 0; e < kList / kThreads; ++e)
            if (tid + e * kThreads < n) sh.list[tid + e * kThreads] = v[e];
          __syncthreads();
        }
        row.finish(n, k, top_p, u, weigh, hit);
      }
      return;
    }
  }
  Cut kept{least, kNone};
  if (k > 0) {
    // (what weighs nothing need not be counted)
    float lo = fmaxf(least, weigh.least), guess;
    if (few) {
      // k elements reach that; where no more do, others with weights lie below it, and nothing else cuts them off
      kept.x = guess = lo = fmaxf(lo, unord_f32(floor_key));
    } else {
      uint32_t smallest = m_key;
      for (int c = 0; c < ctas; ++c) smallest = min(smallest, sh.least[c]);
      guess = fmaxf(lo, unord_f32(smallest));
    }
    uint32_t n = 0;
    if (row.first_k(lo, fminf(guess, m), m, k, &kept, &n)) {
      if (rank == 0) row.finish(n, k, top_p, u, weigh, hit);
      return;
    }
  }
  u64 mass;
  if (top_p < 1.f) kept = row.select_share(m, kept, top_p, weigh, &mass);
  else mass = row.mass_of(weigh, kept);
  row.find(mass, [&](float x, uint32_t i) { return kept(x, i) ? weigh(x) : 0ull; },
           [&](u64 total) { return place_of(u, total); }, hit);
}

template <typename E>
cudaError_t launch_rows(const SamplingParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attrs[2] = {};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = p.ctas;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.B * p.ctas);
  cfg.blockDim = dim3(kThreads);
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
  // CTAs of a row: as many as are estimated to be the fastest.  An SM's CTAs (in rounds of four; clusters leave some places
  // empty, those of no power of two more) share its issue slots for what each does whatever its slice, 1.5 us, and for 0.06 us
  // a KB; a round waits 0.1 us a KB of a slice.  A small top-k has little to do but to read, and each CTA its bounds to
  // find: 2 us, nothing, and 0.1 us a KB.  Over 180 batches (1 to 432 rows of 2000 to 262144) this is 3% behind the best
  // number of CTAs, with a small top-k as without filters or with top-p.  In us with 1, 2, 4 and 8 CTAs a row: 2 rows of
  // 145224 in fp32, top-k of 50, 35, 22, 15, 12; 52 of 7508 in bf16 9.0, 8.8, 9.7, 13.5; 228 of 146675 39, 32, 41, 56; 192 of
  // 131071 without filters 64, 56, 53, 55.
  const bool small_k = p.top_k == nullptr && p.top_k_all > 0 && p.top_k_all <= kPairs;
  const double own = small_k ? 2.0 : 1.5, shared = small_k ? 0.0 : 0.06;
  int ctas = 1;
  double best = 0;
  for (int c = 1; c <= kMaxCtas; ++c) {
    if ((pieces + c - 1) / c * vec > kMostElements) continue;
    const double n = p.B * static_cast<double>(c), sm = std::ceil(1.05 * n / num_sms), rounds = std::ceil(n / (3.8 * num_sms));
    const double time = (own * sm + pieces / 64.0 / c * (0.1 * rounds + shared * sm)) * ((c & (c - 1)) != 0 ? 1.1 : 1.0);
    if (best == 0 || time < best) {
      best = time;
      ctas = c;
    }
  }
  p.ctas = ctas;
  p.per = static_cast<int>((pieces + ctas - 1) / ctas);
  return static_cast<long long>(p.B) * ctas <= 0x7FFFFFFF;
}

cudaError_t launch_sampling(const SamplingParams& p, cudaStream_t stream) {
  switch (p.dtype) {
    case LTK_F32: return launch_rows<float>(p, stream);
    case LTK_F16: return launch_rows<__half>(p, stream);
    default: return launch_rows<__nv_bfloat16>(p, stream);
  }
}

}  // namespace ltk

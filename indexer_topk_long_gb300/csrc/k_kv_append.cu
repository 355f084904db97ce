// k_kv_append.cu -- new tokens' keys and values into the paged e4m3 cache, keys
// (and the step's queries) rotated by their positions on the way.
//
//   k'[i] = k[i] cos - k[j] sin,  k'[j] = k[j] cos + k[i] sin   for each rotated pair (i, j)
//   e     = smallest exponent >= -40 with max |x| <= 448 * 2^e over the block's tokens
//   code  = e4m3(x * 2^-e), nearest even; scale = 2^e
//
// A block is one page and head.  The scale is a power of two: e4m3's relative
// precision is the same at every exponent, so nothing is lost against 448 / max,
// x * 2^-e is exact, and when a later token raises a partly filled page's
// exponent its held codes are re-rounded by a power of two (exact but for
// subnormal codes).  A page that was filled by others under a scale that is no
// power of two gets the next one above, its codes rounded once more.  Products and sums are rounded one by one in fp32 (no
// fused multiply-add), so codes do not depend on the compiler's contraction.
//
// A token whose key or value row holds a NaN, an infinity or a value beyond
// 448 * 2^40 is held as a NaN key row and a zero value row: every query that
// sees it gets NaN, and no other query does (a NaN value code would reach every
// row of a matrix product through 0 * NaN).  So is a token whose position lies
// past the rotation table.
//
// Bound by latency: of decode steps by that of one token, of chunks by the loads' with a third of
// the warps resident and 61% of the issue slots used (DRAM is at 38%).  A page's rows are read
// twice, for its largest and for its codes (the second time from L2), since rows held in
// registers left still fewer warps: 8192 tokens of 8 KV and 32 query heads of 128 take 42 us, 189
// MB at 4.5 TB/s, 66% of the copy rate; one token of each of 256 sequences 4.3 us, one token 3.0
// (calls back to back).
#include "kv_internal.cuh"

namespace ltk {
namespace {

// Head rows per lane group in a rotation unit: few for a decode step (latency), more for
// chunks (bytes in flight; a unit's look at its token's position is paid once).
constexpr int kQPassesFew = 4, kQPassesMany = 8;

struct Chunk {                           // 8 consecutive elements of one row, fp32
  float x[8];
};

__device__ __forceinline__ Chunk unpack(const uint4& r, bool bf16) {
  Chunk c;
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = kv_unpack16(w[i], bf16);
    c.x[2 * i] = f.x;
    c.x[2 * i + 1] = f.y;
  }
  return c;
}

// cos/sin of a chunk's pairs: 8 of each for split halves, 4 (in [0..3]) for adjacent pairs.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(Turn& t, const AppendParams& p, int pos, int j, int h) {
  const int half = p.rot >> 1;
  const int at = p.interleaved ? j * 4 : (j < h ? j : j - h) * 8;
  const float4* c = reinterpret_cast<const float4*>(p.cos + static_cast<size_t>(pos) * half + at);
  const float4* s = reinterpret_cast<const float4*>(p.sin + static_cast<size_t>(pos) * half + at);
  const float4 c0 = kv_load(c), s0 = kv_load(s);
  t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w;
  t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w;
  if (!p.interleaved) {
    const float4 c1 = kv_load(c + 1), s1 = kv_load(s + 1);
    t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
    t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
  }
}

// Rotate chunk j of a row held 8 elements per lane (all lanes of the warp call).
// h = rot / 16 chunks in each half.  `on`: this lane holds a live, rotated chunk.
template <int LPR>
__device__ __forceinline__ void rotate(Chunk& c, const Turn& t, int j, int h, bool interleaved, bool on) {
  if (interleaved) {
    if (!on) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = c.x[2 * i], b = c.x[2 * i + 1];
      c.x[2 * i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
      c.x[2 * i + 1] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
    }
    return;
  }
  const int lane = threadIdx.x & 31;
  const int other = j < h ? j + h : (j < 2 * h ? j - h : j);
  const int src = (lane & ~(LPR - 1)) + other;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = __shfl_sync(0xFFFFFFFFu, c.x[i], src);
    if (on) {
      const float own = __fmul_rn(c.x[i], t.c[i]), turned = __fmul_rn(o, t.s[i]);
      c.x[i] = j < h ? __fsub_rn(own, turned) : __fadd_rn(own, turned);
    }
  }
}

// Smallest e in [kKvMinExp, kKvMaxExp] with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kKvMinExp), kKvMaxExp);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Smallest e >= kKvMinExp with s <= 2^e, for the scale of what a page holds (by append a power of two).
__device__ __forceinline__ int exp_above(float s) {
  const uint32_t b = __float_as_uint(fmaxf(s, 0.f));
  return min(max(static_cast<int>(b >> 23) - 127 + ((b & 0x7FFFFFu) != 0 ? 1 : 0), kKvMinExp), 126);
}

__device__ __forceinline__ uint2 encode(const Chunk& c, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(c.x[2 * i] * inv, c.x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ uint2 rescale_codes(uint2 w, float by) {
  uint32_t in[2] = {w.x, w.y}, out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2];
    e4m3x4_to_f16(in[i], h[0], h[1]);
    out[i] = 0;
#pragma unroll
    for (int hlf = 0; hlf < 2; ++hlf) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[hlf]));
      out[i] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f.x * by, f.y * by), __NV_SATFINITE, __NV_E4M3))
                << (16 * hlf);
    }
  }
  return make_uint2(out[0], out[1]);
}

// Queries: one warp rotates kQPasses * (32 / LPR) head rows of one token, the
// table's row read once for all of them.
template <int D, int kQPasses>
__device__ __forceinline__ void rotate_queries(const AppendParams& p, long long unit) {
  constexpr int LPR = D / 8, RPP = 32 / LPR;
  const int lane = threadIdx.x & 31, j = lane % LPR, sub = lane / LPR;
  const int per_token = (p.q_heads + kQPasses * RPP - 1) / (kQPasses * RPP);
  if (unit >= static_cast<long long>(p.batch.N) * per_token) return;
  const int n = static_cast<int>(unit / per_token), h0 = static_cast<int>(unit % per_token) * kQPasses * RPP;
  const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + n * p.q_stride;
  uint16_t* dst = reinterpret_cast<uint16_t*>(p.q_out) + static_cast<size_t>(n) * p.q_heads * D;
  uint4 raw[kQPasses];
#pragma unroll
  for (int i = 0; i < kQPasses; ++i) {
    const int head = h0 + i * RPP + sub;
    raw[i] = head < p.q_heads ? __ldcs(reinterpret_cast<const uint4*>(src + static_cast<size_t>(head) * D) + j)
                              : make_uint4(0, 0, 0, 0);
  }
  const int h = p.rot >> 4;
  bool on = false;
  Turn t;
  if (p.cos != nullptr) {
    const int b = kv_seq_of_query(p.batch, n);
    const KvSeq s = kv_seq(p.batch, p.cache, b);
    const int pos = s.pos0 + n - s.q0;
    const bool known = n >= s.q0 && n < s.q0 + s.nq && pos >= 0 && pos < p.table_rows;
    if (!known && lane == 0) raise_status(p.status, kDevArg);
    on = known && j < 2 * h;
    if (on) load_turn(t, p, pos, j, h);
  }
#pragma unroll
  for (int i = 0; i < kQPasses; ++i) {
    Chunk c = unpack(raw[i], p.bf16);
    if (p.cos != nullptr) rotate<LPR>(c, t, j, h, p.interleaved, on);
    const int head = h0 + i * RPP + sub;
    if (head < p.q_heads) {
      uint4 o;
      o.x = kv_pack16(c.x[0], c.x[1], p.bf16);
      o.y = kv_pack16(c.x[2], c.x[3], p.bf16);
      o.z = kv_pack16(c.x[4], c.x[5], p.bf16);
      o.w = kv_pack16(c.x[6], c.x[7], p.bf16);
      reinterpret_cast<uint4*>(dst + static_cast<size_t>(head) * D)[j] = o;
    }
  }
}

// Few new tokens for each sequence (a decode step): one warp for each token and head.
// The first token of a page in the step answers for the page's other new tokens too
// (rare: a step of several tokens), the others do nothing.  Against a block of
// page / 16 warps for each page that might be touched: 45 -> 6.3 us for 256 sequences
// of one token and 8 heads.
template <int D>
__global__ void __launch_bounds__(128) kv_append_few_kernel(const AppendParams p, long long kv_blocks) {
  constexpr int LPR = D / 8, RPP = 32 / LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  begin_after_previous();
  if (blockIdx.x >= kv_blocks) {
    rotate_queries<D, kQPassesFew>(p, (blockIdx.x - kv_blocks) * 4 + warp);
    return;
  }
  const KvCache& c = p.cache;
  const long long unit = blockIdx.x * 4ll + warp;
  if (unit >= static_cast<long long>(p.batch.N) * c.heads) return;
  const int n = static_cast<int>(unit / c.heads), head = static_cast<int>(unit % c.heads);
  const int b = kv_seq_of_query(p.batch, n);
  const KvSeq s = kv_seq(p.batch, c, b);
  const int pos = s.pos0 + n - s.q0;
  if (n < s.q0 || n >= s.q0 + s.nq) return;
  if (s.pos0 < 0 || pos >= s.len) {
    if (lane == 0) raise_status(p.status, kDevArg);
    return;
  }
  const int r_lo = pos & (c.page - 1);
  if (r_lo != 0 && pos != s.pos0) return;
  const int p0 = pos - r_lo, r_hi = min(s.len - p0, c.page);
  const int page = kv_page(p.batch, c, b, pos);
  if (page < 0 || page >= c.num_pages) {
    if (lane == 0) raise_status(p.status, kDevArg);
    return;
  }
  const size_t block = static_cast<size_t>(page) * c.heads + head;
  float k_held = 0.f, v_held = 0.f;
  if (r_lo > 0) {
    k_held = c.k_scale[block];
    v_held = c.v_scale[block];
  }
  const int j = lane % LPR, sub = lane / LPR, h = p.rot >> 4;
  const uint16_t* k = reinterpret_cast<const uint16_t*>(p.k) + static_cast<size_t>(head) * D;
  const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v) + static_cast<size_t>(head) * D;
  const float limit = 448.f * pow2f(kKvMaxExp);
  Chunk kc, vc;
  bool bad = false;
  auto take = [&](int base) {            // rows base .. base + RPP - 1
    const int r = base + sub;
    const bool live = r < r_hi;
    uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
    Turn t;
    bool on = false, fine = true;
    if (live) {
      const size_t tok = static_cast<size_t>(s.q0 + (p0 + r - s.pos0));
      kr = kv_load(reinterpret_cast<const uint4*>(k + tok * p.k_stride) + j);
      vr = kv_load(reinterpret_cast<const uint4*>(v + tok * p.v_stride) + j);
      if (p.cos != nullptr) {
        fine = p0 + r < p.table_rows;
        if (!fine) raise_status(p.status, kDevArg);
        on = fine && j < 2 * h;
        if (on) load_turn(t, p, p0 + r, j, h);
      }
    }
    kc = unpack(kr, p.bf16);
    vc = unpack(vr, p.bf16);
    if (p.cos != nullptr) rotate<LPR>(kc, t, j, h, p.interleaved, on);
#pragma unroll
    for (int e = 0; e < 8; ++e) fine = fine && fabsf(kc.x[e]) <= limit && fabsf(vc.x[e]) <= limit;
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, fine);
    constexpr uint32_t row_mask = LPR == 32 ? 0xFFFFFFFFu : (1u << LPR) - 1u;
    bad = ((votes >> (sub * LPR)) & row_mask) != row_mask;
  };
  float k_max = 0.f, v_max = 0.f;
  for (int base = r_lo; base < r_hi; base += RPP) {
    take(base);
    if (!bad) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        k_max = fmaxf(k_max, fabsf(kc.x[e]));
        v_max = fmaxf(v_max, fabsf(vc.x[e]));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    k_max = fmaxf(k_max, __shfl_xor_sync(0xFFFFFFFFu, k_max, o));
    v_max = fmaxf(v_max, __shfl_xor_sync(0xFFFFFFFFu, v_max, o));
  }
  int ke = scale_exp(k_max), ve = scale_exp(v_max);
  if (r_lo > 0) {                        // tokens held before: their codes follow a larger scale
    ke = max(ke, exp_above(k_held));
    ve = max(ve, exp_above(v_held));
    const float k_by = k_held * pow2f(-ke), v_by = v_held * pow2f(-ve);
    for (int r = sub; r < r_lo && (k_by != 1.f || v_by != 1.f); r += RPP) {
      const size_t o = (block * c.page + r) * D + j * 8;
      if (k_by != 1.f) {
        uint2* w = reinterpret_cast<uint2*>(c.k_codes + o);
        *w = rescale_codes(*w, k_by);
      }
      if (v_by != 1.f) {
        uint2* w = reinterpret_cast<uint2*>(c.v_codes + o);
        *w = rescale_codes(*w, v_by);
      }
    }
  }
  if (lane == 0) {
    c.k_scale[block] = pow2f(ke);
    c.v_scale[block] = pow2f(ve);
  }
  const float k_inv = pow2f(-ke), v_inv = pow2f(-ve);
  for (int base = r_lo; base < r_hi; base += RPP) {
    if (r_hi - r_lo > RPP) take(base);
    const int r = base + sub;
    if (r >= r_hi) continue;             // no collective operation follows in this pass
    const size_t o = (block * c.page + r) * D + j * 8;
    *reinterpret_cast<uint2*>(c.k_codes + o) = bad ? make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu) : encode(kc, k_inv);
    *reinterpret_cast<uint2*>(c.v_codes + o) = bad ? make_uint2(0u, 0u) : encode(vc, v_inv);
  }
}

// One page and head, 16 rows per warp.  Pages that can be touched are numbered
// without a scan: sequence b's n tokens touch at most (n + 2 page - 2) / page
// pages, so its numbers start at (cu_q[b] + b (2 page - 2)) / page; numbers
// beyond what it touches are empty.
template <int D>
__global__ void __launch_bounds__(256, 3) kv_append_kernel(const AppendParams p, long long kv_blocks) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, PASSES = 16 / RPP;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  begin_after_previous();
  if (blockIdx.x >= kv_blocks) {
    rotate_queries<D, kQPassesMany>(p, (blockIdx.x - kv_blocks) * warps + warp);
    return;
  }
  const KvCache& c = p.cache;
  const int head = blockIdx.x % c.heads;
  const long long slot = blockIdx.x / c.heads;
  const int step = 2 * c.page - 2;
  int lo = 0, hi = p.batch.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((kv_load(p.batch.cu_q + mid) + static_cast<long long>(mid) * step) >> c.page_log2 <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int b = lo;
  const KvSeq s = kv_seq(p.batch, c, b);
  if (s.nq == 0) return;
  const bool past = s.pos0 > s.len - s.nq;                    // its last tokens have no page
  if (s.pos0 < 0 || past) {
    if (threadIdx.x == 0) raise_status(p.status, kDevArg);
    if (!past) return;
  }
  const long long first_page = s.pos0 >> c.page_log2;
  const long long at = first_page + slot - ((kv_load(p.batch.cu_q + b) + static_cast<long long>(b) * step) >> c.page_log2);
  if (at < first_page || at << c.page_log2 >= s.len) return;
  const int page = kv_load(p.batch.page_table + static_cast<size_t>(b) * p.batch.width + at);
  if (page < 0 || page >= c.num_pages) {
    if (threadIdx.x == 0) raise_status(p.status, kDevArg);
    return;
  }
  const int p0 = static_cast<int>(at) << c.page_log2;         // position of the page's row 0
  const int r_lo = max(s.pos0 - p0, 0), r_hi = min(s.len - p0, c.page);
  const size_t block = static_cast<size_t>(page) * c.heads + head;
  float k_held = 0.f, v_held = 0.f;
  if (r_lo > 0) {
    k_held = c.k_scale[block];
    v_held = c.v_scale[block];
  }

  const int j = lane % LPR, sub = lane / LPR;
  const uint16_t* k = reinterpret_cast<const uint16_t*>(p.k) + static_cast<size_t>(head) * D;
  const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v) + static_cast<size_t>(head) * D;
  const int h = p.rot >> 4;
  const float limit = 448.f * pow2f(kKvMaxExp);
  float k_max = 0.f, v_max = 0.f;
  uint32_t bad_rows = 0;
  // Rows are read and rotated twice, for the maximum and for the codes (the second time
  // from L2): kept in registers, 64 of them, they left room for half the warps, and the
  // queries' rotation in the same launch lives on warps (8192 tokens: 53 -> 45 us).
  constexpr int AT_ONCE = 4;             // passes whose loads are in flight together
  auto load = [&](int i, uint4& kr, uint4& vr) {
    const int r = warp * 16 + i * RPP + sub;
    kr = vr = make_uint4(0, 0, 0, 0);
    if (r >= r_lo && r < r_hi) {
      const size_t n = static_cast<size_t>(s.q0 + (p0 + r - s.pos0));
      kr = kv_load(reinterpret_cast<const uint4*>(k + n * p.k_stride) + j);
      vr = kv_load(reinterpret_cast<const uint4*>(v + n * p.v_stride) + j);
    }
  };
  auto keys = [&](int i, const uint4& kr, bool& fine) {
    const int r = warp * 16 + i * RPP + sub;
    const bool live = r >= r_lo && r < r_hi;
    Chunk kc = unpack(kr, p.bf16);
    fine = true;
    if (p.cos != nullptr) {
      fine = !live || p0 + r < p.table_rows;
      const bool on = live && fine && j < 2 * h;
      Turn t;
      if (on) load_turn(t, p, p0 + r, j, h);
      rotate<LPR>(kc, t, j, h, p.interleaved, on);
    }
    return kc;
  };
#pragma unroll 1
  for (int i0 = 0; i0 < PASSES; i0 += AT_ONCE) {
    uint4 kr[AT_ONCE], vr[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) load(i0 + i, kr[i], vr[i]);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      bool fine;
      const Chunk kc = keys(i0 + i, kr[i], fine);
      if (!fine) raise_status(p.status, kDevArg);
      const Chunk vc = unpack(vr[i], p.bf16);
      float ka = 0.f, va = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = fabsf(kc.x[e]), z = fabsf(vc.x[e]);
        fine = fine && a <= limit && z <= limit;
        ka = fmaxf(ka, a);
        va = fmaxf(va, z);
      }
      const uint32_t votes = __ballot_sync(0xFFFFFFFFu, fine);
      constexpr uint32_t row_mask = LPR == 32 ? 0xFFFFFFFFu : (1u << LPR) - 1u;
      if (((votes >> (sub * LPR)) & row_mask) != row_mask) {
        bad_rows |= 1u << (i0 + i);
      } else {
        k_max = fmaxf(k_max, ka);
        v_max = fmaxf(v_max, va);
      }
    }
  }
  __shared__ float red[2][8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    k_max = fmaxf(k_max, __shfl_xor_sync(0xFFFFFFFFu, k_max, o));
    v_max = fmaxf(v_max, __shfl_xor_sync(0xFFFFFFFFu, v_max, o));
  }
  if (lane == 0) {
    red[0][warp] = k_max;
    red[1][warp] = v_max;
  }
  __syncthreads();
  for (int w = 0; w < warps; ++w) {
    k_max = fmaxf(k_max, red[0][w]);
    v_max = fmaxf(v_max, red[1][w]);
  }
  int ke = scale_exp(k_max), ve = scale_exp(v_max);
  float k_by = 1.f, v_by = 1.f;
  if (r_lo > 0) {                                             // tokens held before
    ke = max(ke, exp_above(k_held));
    ve = max(ve, exp_above(v_held));
    k_by = k_held * pow2f(-ke);
    v_by = v_held * pow2f(-ve);
  }
  const float k_inv = pow2f(-ke), v_inv = pow2f(-ve);
  if (threadIdx.x == 0) {
    c.k_scale[block] = pow2f(ke);
    c.v_scale[block] = pow2f(ve);
  }
#pragma unroll 1
  for (int i0 = 0; i0 < PASSES; i0 += AT_ONCE) {
    uint4 kr[AT_ONCE], vr[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) load(i0 + i, kr[i], vr[i]);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int r = warp * 16 + (i0 + i) * RPP + sub;
      const size_t o = (block * c.page + r) * D + j * 8;
      bool fine;
      const Chunk kc = keys(i0 + i, kr[i], fine);
      if (r >= r_lo && r < r_hi) {
        const bool bad = (bad_rows >> (i0 + i)) & 1u;
        const Chunk vc = unpack(vr[i], p.bf16);
        *reinterpret_cast<uint2*>(c.k_codes + o) = bad ? make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu) : encode(kc, k_inv);
        *reinterpret_cast<uint2*>(c.v_codes + o) = bad ? make_uint2(0u, 0u) : encode(vc, v_inv);
      } else if (r < r_lo) {
        if (k_by != 1.f) {
          uint2* w = reinterpret_cast<uint2*>(c.k_codes + o);
          *w = rescale_codes(*w, k_by);
        }
        if (v_by != 1.f) {
          uint2* w = reinterpret_cast<uint2*>(c.v_codes + o);
          *w = rescale_codes(*w, v_by);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const int page = p.cache.page;
  // Up to eight tokens a sequence (on average): a warp for each token and head.  Beyond, a
  // block for each page, whose rows share the loads' latency.  64 sequences (8 KV heads, 32
  // query heads of 128, in us): 1 token each 6.3 by warps and 15.6 by pages, 8 each 10.4 and
  // 16.6, 16 each 16.9 and 17.2, 64 each 40 and 31; 8192 tokens of one sequence 81 and 45.
  const bool few = p.batch.N <= 8ll * p.batch.B;
  const long long slots = (p.batch.N + static_cast<long long>(p.batch.B) * (2 * page - 2)) / page;
  const long long kv_blocks = few ? (static_cast<long long>(p.batch.N) * p.cache.heads + 3) / 4 : slots * p.cache.heads;
  const int warps = few ? 4 : page / 16;
  const int rows = (few ? kQPassesFew : kQPassesMany) * (32 / (p.dim / 8));
  const long long units = p.q != nullptr ? static_cast<long long>(p.batch.N) * ((p.q_heads + rows - 1) / rows) : 0;
  const long long blocks = kv_blocks + (units + warps - 1) / warps;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  if (blocks == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(blocks);
  cudaError_t e;
  if (p.dim == 128) {
    e = few ? launch_overlapped(kv_append_few_kernel<128>, grid, 128, 0, stream, p, kv_blocks)
            : launch_overlapped(kv_append_kernel<128>, grid, warps * 32, 0, stream, p, kv_blocks);
  } else {
    e = few ? launch_overlapped(kv_append_few_kernel<64>, grid, 128, 0, stream, p, kv_blocks)
            : launch_overlapped(kv_append_kernel<64>, grid, warps * 32, 0, stream, p, kv_blocks);
  }
  count_launches(1);
  return e;
}

}  // namespace ltk

// k_kv_tile.cu -- attention over the paged e4m3 cache for many query rows per KV
// head (prefill chunks, one KV head shared by many query heads), on the tensor
// cores: S = Q K^T and O += P V as tcgen05 products with S, P and O in tensor memory.
//
//   t_j = c_row * ks * (q . k_j) + log2(vs),  w_j = 2^(t_j - M)   (exponents in base 2)
//   O = sum_j w_j vcode_j,  l = sum_j w_j / vs,  out = O / l,  lse = (M + log2 l) ln 2
//
// as in the kernel for few rows: the value scale is folded into the weight's
// exponent, weights go to the product as f16 at most 2^15, codes become f16
// exactly, queries after a power-of-two scaling of their row; M, l and O are fp32.
//
// Rows of a KV head are (query, head in group) pairs, 128 to an MMA tile.  A key
// tile is 128 keys.  Two streams (one warpgroup of softmax threads each, one
// thread per row) keep the tensor cores busy while the other stream's weights
// are computed:
//   pair mode:  the streams are two row tiles that share every key tile;
//   solo mode:  one row tile, the streams take alternate key tiles and their
//               results are merged at the end.  With at most 64 rows the tile
//               holds them twice, so the streams' threads sit on different schedulers.
// Roles: warps 0-3 and 4-7 softmax, 8-11 loader (codes from global memory through
// registers, e4m3 to f16, 128-byte-swizzled shared memory; a listed key is as good
// as a paged one), warp 12 issues the MMAs.
#include "kv_internal.cuh"

namespace ltk {
namespace {

constexpr int kTileRows = 128;
constexpr int kKeys = 128;
constexpr int kThreads = 13 * 32;
constexpr float kMinusHuge = -1e30f;
constexpr float kBoost = 8.f;            // as in the kernel for few rows
constexpr float kSlack = 7.f;

struct Unit {                            // one work item, written by the loader
  int n_tiles;                           // key tiles; -1: no more items
  int first;                             // ordinal of the first of them
  int rows;                              // live rows
  int row0;                              // first row: row r is query q0 + r / group, head r % group
  int q0;
  int pos0;                              // position of query q0
  int p_lo, p_hi;                        // smallest and largest position of the rows
  int head;
  int skip, tile0;                       // ordinals below skip are the sinks' tiles, the rest start at tile0
  int item;
};

struct Meta {                            // scales of a key tile's eight 16-key groups
  float ks[8];
  float lv[8];                           // log2(vs) + kBoost
  float iv[8];                           // 1 / vs
  uint32_t valid[4];                     // listed keys: bit per key
};

struct Ctrl {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], ofull[2];
  uint64_t ufull[2], uempty[2], qempty, mfull, mempty, drained;
  uint32_t tmem;
  int abort_flag;
  Unit unit[2];
  Meta meta[4];
  // score factor of each row by unit slot: pair mode [2][256]; solo mode [2][128], then
  // stream 1's (M, l) [128][2]
  float rowf[512];
};

template <int D>
struct TileShape {
  static constexpr int kOperand = kKeys * D * 2;              // one f16 operand tile
  static constexpr int kQ = 2 * kOperand;                     // pair: two row tiles; solo: two buffers
  static constexpr int kStage = 2 * kOperand;                 // K and V
  static constexpr int kMerge = kTileRows * 64 * 4;           // solo mode: 64 columns of stream 1's O
  static constexpr int kBytes = kQ + 2 * kStage + kMerge + static_cast<int>(sizeof(Ctrl));
};
static_assert(TileShape<128>::kBytes <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\tmbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\tselp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t a, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(a));
}
__device__ __forceinline__ void tmem_ld32_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_st32f(uint32_t a, const float (&v)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[16 * h + i]);
    tmem_st16(a + 16 * h, w);
  }
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of the value operand: rows of 128 bytes hold 64 consecutive d of one
// key (N contiguous), 8-row atoms 1024 bytes apart along the keys (stride offset),
// 128-byte-wide halves `lead` bytes apart along d (leading offset).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// f16 operands, fp32 result; the second operand with N contiguous when b_mn.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

struct TileParams {
  AttnParams a;
  int pair;                              // 1: pair mode
  int n_split;                           // pieces of each unit's key tiles
  int row_tiles;                         // listed keys: row tiles of a group
  long long items;
};

__device__ __forceinline__ int unit_rows(const TileParams& p) { return p.pair ? 2 * kTileRows : kTileRows; }

// Dense units are numbered without a scan: sequence b's start at
// cu_q[b] * group / rows + b, which leaves room for every row tile.
__device__ __forceinline__ long long slot_start(const TileParams& p, int b) {
  return static_cast<long long>(__ldg(p.a.batch.cu_q + b)) * p.a.group / unit_rows(p) + b;
}

// Work item to unit; false: nothing there.
template <bool SEL>
__device__ bool decode_item(const TileParams& p, long long item, Unit& u, int& b, int& len) {
  const AttnParams& a = p.a;
  const int s = static_cast<int>(item % p.n_split);
  const long long rest = item / p.n_split;
  u.item = static_cast<int>(min(item, 0x7FFFFFFFll));
  u.head = static_cast<int>(rest % a.cache.heads);
  const long long slot = rest / a.cache.heads;
  int total;
  if constexpr (SEL) {
    const int n = static_cast<int>(slot / p.row_tiles);
    u.row0 = static_cast<int>(slot % p.row_tiles) * kTileRows;
    u.rows = min(a.group - u.row0, kTileRows);
    b = kv_seq_of_query(a.batch, n);
    const KvSeq q = kv_seq(a.batch, a.cache, b);
    u.q0 = n;
    u.pos0 = (n >= q.q0 && n < q.q0 + q.nq) ? q.pos0 + n - q.q0 : -1;
    u.p_lo = u.p_hi = u.pos0;
    u.skip = u.tile0 = 0;
    len = a.k;
    total = (a.k + kKeys - 1) / kKeys;
  } else {
    int lo = 0, hi = a.batch.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (slot_start(p, mid) <= slot) lo = mid; else hi = mid - 1;
    }
    b = lo;
    const KvSeq q = kv_seq(a.batch, a.cache, b);
    const long long row0 = (slot - slot_start(p, b)) * unit_rows(p);
    const long long all = static_cast<long long>(q.nq) * a.group;
    if (row0 < 0 || row0 >= all) return false;
    u.row0 = static_cast<int>(row0);
    u.rows = static_cast<int>(min(all - row0, static_cast<long long>(unit_rows(p))));
    u.q0 = q.q0;
    u.pos0 = q.pos0;
    u.p_lo = q.pos0 + u.row0 / a.group;
    u.p_hi = q.pos0 + (u.row0 + u.rows - 1) / a.group;
    len = q.len;
    u.skip = u.tile0 = 0;
    total = u.p_hi >= 0 ? u.p_hi / kKeys + 1 : 0;
    if (total > 0 && a.window > 0) {
      u.tile0 = max(u.p_lo - a.window + 1, 0) / kKeys;
      u.skip = min((min(a.sinks, u.p_hi + 1) + kKeys - 1) / kKeys, u.tile0);
      total = u.skip + total - u.tile0;
    }
  }
  u.first = static_cast<int>(static_cast<long long>(total) * s / p.n_split);
  u.n_tiles = static_cast<int>(static_cast<long long>(total) * (s + 1) / p.n_split) - u.first;
  return true;
}

// --- loader ---------------------------------------------------------------------------------
// Thread mapping of a 128-key tile: warp w holds rows 32 w .. 32 w + 31 (two whole
// 16-key groups); a lane's NI rows and its 16-byte chunk of codes are chosen so that
// a quarter warp's 16-byte shared stores fall on distinct banks (two rows of
// different parity, four chunks).
template <int D>
struct Map {
  static constexpr int NI = D == 128 ? 8 : 4;
  static __device__ __forceinline__ int row(int lane, int i) {
    return D == 128 ? (lane >> 4) * 2 + ((lane >> 2) & 1) + 4 * i : (lane >> 2) + 8 * i;
  }
  static __device__ __forceinline__ int chunk(int lane) { return D == 128 ? (lane & 3) + 4 * ((lane >> 3) & 1) : lane & 3; }
};

// 16 codes to two swizzled 16-byte chunks of f16 (by != 0: times an f16x2 factor).
template <int D, bool SCALED>
__device__ __forceinline__ void store_codes(uint32_t base, int row, int chunk, const uint4& codes, __half2 by) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = e4m3x2_to_f16x2(w[i] & 0xFFFFu);
    h[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
  }
  if constexpr (SCALED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), by);
      h[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  const uint32_t line = base + (chunk >> 2) * (kKeys * 128) + row * 128;
  const int c0 = (2 * chunk) & 7;
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(line + ((c0 ^ (row & 7)) << 4)), "r"(h[0]), "r"(h[1]), "r"(h[2]),
               "r"(h[3])
               : "memory");
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(line + (((c0 + 1) ^ (row & 7)) << 4)), "r"(h[4]), "r"(h[5]),
               "r"(h[6]), "r"(h[7])
               : "memory");
}

// What a lane holds of one key tile on its way to shared memory.
template <int D>
struct Tile {
  uint4 k[Map<D>::NI], v[Map<D>::NI];
  float ks[Map<D>::NI], vs[Map<D>::NI];  // listed: per row; dense: [0], [1] the warp's two groups
  uint32_t valid;                        // bit i: row i is live
};
template <int D>
struct Ids {
  int key[Map<D>::NI];                   // listed: key position or -1
  int page[Map<D>::NI];                  // listed: per row; dense: [0], [1]
};

template <int D, bool SEL>
__device__ __forceinline__ void fetch_keys(const TileParams& p, const Unit& u, int ord, int w, int lane, Ids<D>& ids) {
  if constexpr (SEL) {
#pragma unroll
    for (int i = 0; i < Map<D>::NI; ++i) {
      const int at = ord * kKeys + 32 * w + Map<D>::row(lane, i);
      ids.key[i] = at < p.a.k ? __ldg(p.a.idx + static_cast<size_t>(u.q0) * p.a.k + at) : -1;
    }
  }
}
__device__ __forceinline__ int tile_of(const Unit& u, int ord) { return ord < u.skip ? ord : ord - u.skip + u.tile0; }

template <int D, bool SEL>
__device__ __forceinline__ void fetch_pages(const TileParams& p, const Unit& u, int b, int len, int ord, int w, Ids<D>& ids) {
  const int* table = p.a.batch.page_table + static_cast<size_t>(b) * p.a.batch.width;
  if constexpr (SEL) {
#pragma unroll
    for (int i = 0; i < Map<D>::NI; ++i) {
      if (ids.key[i] < 0 || ids.key[i] > u.pos0) ids.key[i] = -1;
      ids.page[i] = ids.key[i] >= 0 ? __ldg(table + (ids.key[i] >> p.a.cache.page_log2)) : -1;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = tile_of(u, ord) * kKeys + 32 * w + 16 * h;
      ids.page[h] = key < len ? __ldg(table + (key >> p.a.cache.page_log2)) : -1;
    }
  }
}

// Row i's place in the cache, -1 if it has none.
template <int D, bool SEL>
__device__ __forceinline__ long long row_at(const TileParams& p, const Unit& u, int len, int ord, int w, int lane, int i,
                                            const Ids<D>& ids) {
  const KvCache& c = p.a.cache;
  int page, off;
  if constexpr (SEL) {
    page = ids.page[i];
    off = ids.key[i] & (c.page - 1);
    if (ids.key[i] < 0) return -1;
  } else {
    constexpr int kPerGroup = Map<D>::NI / 2;
    page = ids.page[i / kPerGroup];
    const int key = tile_of(u, ord) * kKeys + 32 * w + Map<D>::row(lane, i);
    if (key >= len) return -1;
    off = key & (c.page - 1);
  }
  if (page < 0 || page >= c.num_pages) return -1;
  return (static_cast<long long>(page) * c.heads + u.head) * c.page + off;
}

template <int D, bool SEL>
__device__ __forceinline__ void load_half(const TileParams& p, const Unit& u, int len, int ord, int w, int lane, const Ids<D>& ids,
                                          bool values, Tile<D>& t) {
  const KvCache& c = p.a.cache;
  const uint8_t* codes = values ? c.v_codes : c.k_codes;
  const float* scale = values ? c.v_scale : c.k_scale;
  uint32_t valid = 0;
#pragma unroll
  for (int i = 0; i < Map<D>::NI; ++i) {
    const long long r = row_at<D, SEL>(p, u, len, ord, w, lane, i, ids);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r >= 0) x = __ldg(reinterpret_cast<const uint4*>(codes + static_cast<size_t>(r) * D) + Map<D>::chunk(lane));
    if (values) t.v[i] = x; else t.k[i] = x;
    if constexpr (SEL) {
      const bool listed = ids.key[i] >= 0;
      float sc = 0.f;
      if (r >= 0) {
        sc = __ldg(scale + static_cast<size_t>(ids.page[i]) * c.heads + u.head);
      } else if (listed && !values) {    // a page outside the pool: the key is NaN
        sc = __int_as_float(0x7FC00000);
        raise_status(p.a.status, kDevArg);
      }
      if (values) t.vs[i] = sc; else t.ks[i] = sc;
      if (listed) valid |= 1u << i;
    }
  }
  if constexpr (!SEL) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = tile_of(u, ord) * kKeys + 32 * w + 16 * h;
      float sc = 1.f;
      if (ids.page[h] >= 0 && ids.page[h] < c.num_pages) {
        sc = __ldg(scale + static_cast<size_t>(ids.page[h]) * c.heads + u.head);
      } else if (key < len && !values) {
        sc = __int_as_float(0x7FC00000);
        raise_status(p.a.status, kDevArg);
      }
      if (values) t.vs[h] = sc; else t.ks[h] = sc;
    }
  }
  if (!values) t.valid = valid;
}

// Listed keys come from blocks of different scales: the codes are multiplied by
// 64 * scale / (largest scale of the 16-key group), exact in f16 for ratios down
// to 2^-21 (an e4m3 code is a multiple of 2^-9, f16's smallest step 2^-24).
template <int D>
__device__ __forceinline__ float group_scale(const float (&s)[Map<D>::NI], int h) {
  constexpr int kPer = Map<D>::NI / 2;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = fmaxf(m, s[h * kPer + i]);
  m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
  m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
  if constexpr (D == 64) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
  return m > 0.f ? m : 1.f;
}

template <int D, bool SEL>
__device__ __forceinline__ void store_half(uint32_t base, int w, int lane, const uint4 (&x)[Map<D>::NI], const float (&s)[Map<D>::NI],
                                           float (&group)[2]) {
  constexpr int kPer = Map<D>::NI / 2;
  if constexpr (SEL) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float top = group_scale<D>(s, h);
      const float inv = 64.f / top;
      group[h] = top * (1.f / 64.f);
#pragma unroll
      for (int i = h * kPer; i < (h + 1) * kPer; ++i)
        store_codes<D, true>(base, 32 * w + Map<D>::row(lane, i), Map<D>::chunk(lane), x[i], __float2half2_rn(s[i] * inv));
    }
  } else {
    group[0] = s[0];
    group[1] = s[1];
#pragma unroll
    for (int i = 0; i < Map<D>::NI; ++i)
      store_codes<D, false>(base, 32 * w + Map<D>::row(lane, i), Map<D>::chunk(lane), x[i], __half2());
  }
}

// Query rows [r0, r0 + 128) of the unit to an operand tile; factor[r] = what turns
// the products into base-2 exponents.  `mask`: rows repeat with this period.
template <int D>
__device__ void load_queries(const TileParams& p, const Unit& u, uint32_t base, float* factor, int r0, int mask, int w, int lane) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, PASSES = 32 / RPP;
  const AttnParams& a = p.a;
  const int j = lane % LPR, sub = lane / LPR;
#pragma unroll 1
  for (int p0 = 0; p0 < PASSES; p0 += 4) {
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int local = 32 * w + (p0 + i) * RPP + sub;
      const int r = r0 + (local & mask);
      raw[i] = make_uint4(0, 0, 0, 0);
      if (r < u.rows) {
        const int row = u.row0 + r;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (static_cast<size_t>(u.q0) + row / a.group) * a.q_stride +
                              static_cast<size_t>(u.head * a.group + row % a.group) * D;
        raw[i] = __ldg(reinterpret_cast<const uint4*>(src) + j);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int local = 32 * w + (p0 + i) * RPP + sub;
      const uint32_t ws[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      float2 f[4];
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = kv_unpack16(ws[e], a.bf16);
        amax = fmaxf(amax, fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
      }
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 8;      // the largest element to [2^8, 2^9)
      e = amax > 0.f && amax < __int_as_float(0x7F800000) ? max(e, -118) : 0;
      const float by = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (j == 0) factor[local] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      uint32_t h[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = kv_pack16(f[q].x * by, f[q].y * by, false);
      const uint32_t line = base + (j >> 3) * (kTileRows * 128) + local * 128;
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(line + (((j & 7) ^ (local & 7)) << 4)), "r"(h[0]), "r"(h[1]),
                   "r"(h[2]), "r"(h[3])
                   : "memory");
    }
  }
}

template <int D, bool SEL>
__global__ void __launch_bounds__(kThreads, 1) kv_tile_kernel(const TileParams p) {
  using S = TileShape<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + S::kQ + 2 * S::kStage + S::kMerge);
  const uint32_t q_sm = smem_u32(smem), stage_sm = q_sm + S::kQ;
  float* merge = reinterpret_cast<float*>(smem + S::kQ + 2 * S::kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttnParams& a = p.a;
  const bool pair = p.pair != 0;
  volatile int* abort_flag = &ctrl->abort_flag;
  int* status = a.status;

  if (warp == 12) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&ctrl->kfull[i]), 128);
        mbar_init(smem_u32(&ctrl->kempty[i]), 1);
        mbar_init(smem_u32(&ctrl->vfull[i]), 128);
        mbar_init(smem_u32(&ctrl->vempty[i]), 1);
        mbar_init(smem_u32(&ctrl->sfull[i]), 2);
        mbar_init(smem_u32(&ctrl->pfull[i]), 128);
        mbar_init(smem_u32(&ctrl->ofull[i]), 1);
        mbar_init(smem_u32(&ctrl->ufull[i]), 128);
        mbar_init(smem_u32(&ctrl->uempty[i]), 256 + 2);
      }
      mbar_init(smem_u32(&ctrl->qempty), 1);
      mbar_init(smem_u32(&ctrl->mfull), 128);
      mbar_init(smem_u32(&ctrl->mempty), 128);
      mbar_init(smem_u32(&ctrl->drained), 1);
      ctrl->abort_flag = 0;
      mbar_fence_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(&ctrl->tmem), 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem;

  if (warp >= 8 && warp < 12) {
    // ================= loader =================
    const int w = warp - 8;
    const int ltid = tid - 256;
    int un = 0;                          // units published
    int cnt[2] = {0, 0};                 // tiles loaded by stream (pair mode: [0] counts all)
    bool ok = true;
    for (long long item = blockIdx.x; ok; item += gridDim.x) {
      Unit u;
      int b = 0, len = 0;
      const bool more = item < p.items;
      if (more && !decode_item<SEL>(p, item, u, b, len)) continue;
      Ids<D> ids;
      Tile<D> t;
      if (more && u.n_tiles > 0) {
        fetch_keys<D, SEL>(p, u, u.first, w, lane, ids);
        fetch_pages<D, SEL>(p, u, b, len, u.first, w, ids);
        load_half<D, SEL>(p, u, len, u.first, w, lane, ids, false, t);
        load_half<D, SEL>(p, u, len, u.first, w, lane, ids, true, t);
        if (u.n_tiles > 1) fetch_keys<D, SEL>(p, u, u.first + 1, w, lane, ids);
      }
      const int us = un & 1;
      if (un >= 2 && !mbar_wait(smem_u32(&ctrl->uempty[us]), ((un >> 1) - 1) & 1, abort_flag, status)) break;
      if (!more) u.n_tiles = -1;
      if (ltid == 0) ctrl->unit[us] = u;
      if (more && u.n_tiles > 0) {
        if (pair) {
          if (un >= 1 && !mbar_wait(smem_u32(&ctrl->qempty), (un - 1) & 1, abort_flag, status)) break;
          load_queries<D>(p, u, q_sm, ctrl->rowf + us * 256, 0, 127, w, lane);
          if (u.rows > kTileRows) load_queries<D>(p, u, q_sm + S::kOperand, ctrl->rowf + us * 256 + 128, kTileRows, 127, w, lane);
        } else {
          load_queries<D>(p, u, q_sm + us * S::kOperand, ctrl->rowf + us * 128, 0, u.rows <= 64 ? 63 : 127, w, lane);
        }
        fence_async_smem();
      }
      mbar_arrive(smem_u32(&ctrl->ufull[us]));
      ++un;
      if (!more) break;
#pragma unroll 1
      for (int i = 0; i < u.n_tiles; ++i) {
        const int ord = u.first + i;
        const bool next = i + 1 < u.n_tiles;
        const int x = pair ? 0 : i & 1;
        const int n = cnt[x];
        const int st = pair ? n & 1 : x, use = pair ? n >> 1 : n;
        const int slot = pair ? n & 3 : x * 2 + (n & 1);
        if (next) fetch_pages<D, SEL>(p, u, b, len, ord + 1, w, ids);
        if (use > 0 && !mbar_wait(smem_u32(&ctrl->kempty[st]), (use - 1) & 1, abort_flag, status)) { ok = false; break; }
        float gk[2], gv[2];
        store_half<D, SEL>(stage_sm + st * S::kStage, w, lane, t.k, t.ks, gk);
        // the tile's scales, before K is announced
        Meta& m = ctrl->meta[slot];
        if constexpr (SEL) {
          gv[0] = group_scale<D>(t.vs, 0) * (1.f / 64.f);
          gv[1] = group_scale<D>(t.vs, 1) * (1.f / 64.f);
          uint32_t bits = 0;
#pragma unroll
          for (int r = 0; r < Map<D>::NI; ++r)
            if ((t.valid >> r) & 1u) bits |= 1u << Map<D>::row(lane, r);
          bits = __reduce_or_sync(0xFFFFFFFFu, bits);
          if (lane == 0) m.valid[w] = bits;
        } else {
          gv[0] = t.vs[0];
          gv[1] = t.vs[1];
        }
        if (lane < 2) {
          m.ks[2 * w + lane] = lane ? gk[1] : gk[0];
          const float g = lane ? gv[1] : gv[0];
          m.lv[2 * w + lane] = __log2f(g) + kBoost;
          m.iv[2 * w + lane] = __frcp_rn(g);
        }
        fence_async_smem();
        mbar_arrive(smem_u32(&ctrl->kfull[st]));
        if (next) load_half<D, SEL>(p, u, len, ord + 1, w, lane, ids, false, t);
        if (use > 0 && !mbar_wait(smem_u32(&ctrl->vempty[st]), (use - 1) & 1, abort_flag, status)) { ok = false; break; }
        store_half<D, SEL>(stage_sm + st * S::kStage + S::kOperand, w, lane, t.v, t.vs, gv);
        fence_async_smem();
        mbar_arrive(smem_u32(&ctrl->vfull[st]));
        if (next) load_half<D, SEL>(p, u, len, ord + 1, w, lane, ids, true, t);
        if (i + 2 < u.n_tiles) fetch_keys<D, SEL>(p, u, ord + 2, w, lane, ids);
        ++cnt[x];
      }
    }
  } else if (warp == 12) {
    // ================= MMA issue =================
    if (lane == 0) {
      constexpr uint32_t id_qk = idesc_f16(kTileRows, kKeys, false), id_pv = idesc_f16(kTileRows, D, true);
      auto qk = [&](int x, uint32_t q_tile, int st) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * (kTileRows * 128) + (k & 3) * 32;
          tc_mma<false>(tmem + x * kKeys, smem_desc_sw128(q_tile + off), smem_desc_sw128(stage_sm + st * S::kStage + off), id_qk,
                        k > 0);
        }
        tc_commit(smem_u32(&ctrl->sfull[x]));
        mbar_arrive(smem_u32(&ctrl->sfull[x]));   // passes on what the loader wrote beside K
      };
      auto pv = [&](int x, int st, bool first) {
        const uint32_t v = stage_sm + st * S::kStage + S::kOperand;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts(tmem + 256 + x * D, tmem + x * kKeys + k * 8, desc_mn(v + k * 2048, kKeys * 128), id_pv, !first || k > 0);
      };
      if (pair) {
        int c = 0, nu = 0;
        int sp[2] = {0, 0};              // weights awaited by stream
        bool ok = true;
        while (ok) {
          const int us = nu & 1;
          if (!mbar_wait(smem_u32(&ctrl->ufull[us]), (nu >> 1) & 1, abort_flag, status)) break;
          const int n = ctrl->unit[us].n_tiles;
          const bool two = ctrl->unit[us].rows > kTileRows;
          if (n < 0) break;
          ++nu;
          if (n > 0) {
            if (!mbar_wait(smem_u32(&ctrl->kfull[c & 1]), (c >> 1) & 1, abort_flag, status)) break;
            tc_fence_after();
            qk(0, q_sm, c & 1);
            if (two) qk(1, q_sm + S::kOperand, c & 1);
            tc_commit(smem_u32(&ctrl->kempty[c & 1]));
            for (int i = 0; i < n && ok; ++i, ++c) {
              const int st = c & 1, ns = (c + 1) & 1;
              const bool next = i + 1 < n;
              if (!mbar_wait(smem_u32(&ctrl->vfull[st]), (c >> 1) & 1, abort_flag, status) ||
                  !mbar_wait(smem_u32(&ctrl->pfull[0]), sp[0] & 1, abort_flag, status)) { ok = false; break; }
              ++sp[0];
              tc_fence_after();
              pv(0, st, i == 0);
              if (!next) tc_commit(smem_u32(&ctrl->ofull[0]));
              if (next) {
                if (!mbar_wait(smem_u32(&ctrl->kfull[ns]), ((c + 1) >> 1) & 1, abort_flag, status)) { ok = false; break; }
                tc_fence_after();
                qk(0, q_sm, ns);
              }
              if (two) {
                if (!mbar_wait(smem_u32(&ctrl->pfull[1]), sp[1] & 1, abort_flag, status)) { ok = false; break; }
                ++sp[1];
                tc_fence_after();
                pv(1, st, i == 0);
              }
              tc_commit(smem_u32(&ctrl->vempty[st]));
              if (two && next) qk(1, q_sm + S::kOperand, ns);
              if (two && !next) tc_commit(smem_u32(&ctrl->ofull[1]));
              if (next) tc_commit(smem_u32(&ctrl->kempty[ns]));
            }
            tc_commit(smem_u32(&ctrl->qempty));
          } else {
            mbar_arrive(smem_u32(&ctrl->qempty));
          }
          mbar_arrive(smem_u32(&ctrl->uempty[us]));
          mbar_arrive(smem_u32(&ctrl->uempty[us]));
        }
      } else {
        // Each stream walks its own key tiles through the units.  Neither may hold up the
        // other (a stream without a tile in some unit runs ahead, and what it waits for can
        // depend on the other's next product), so both are polled.
        int cu[2] = {0, 0}, left[2] = {0, 0}, cnt[2] = {0, 0}, fresh[2] = {1, 1};
        bool pending[2] = {false, false}, done[2] = {false, false};
        uint64_t since = globaltimer_ns();
        while (!(done[0] && done[1])) {
          bool progress = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (done[x]) continue;
            if (pending[x]) {
              if (!mbar_test(smem_u32(&ctrl->pfull[x]), cnt[x] & 1) || !mbar_test(smem_u32(&ctrl->vfull[x]), cnt[x] & 1)) continue;
              tc_fence_after();
              pv(x, x, fresh[x]);
              fresh[x] = 0;
              tc_commit(smem_u32(&ctrl->vempty[x]));
              pending[x] = false;
              progress = true;
              ++cnt[x];
              if (--left[x] == 0) {
                tc_commit(smem_u32(&ctrl->ofull[x]));
                tc_commit(smem_u32(&ctrl->uempty[cu[x] & 1]));
                ++cu[x];
              }
            }
            while (left[x] == 0) {       // the stream's next unit with a tile for it
              const int us = cu[x] & 1;
              if (!mbar_test(smem_u32(&ctrl->ufull[us]), (cu[x] >> 1) & 1)) break;
              const int n = ctrl->unit[us].n_tiles;
              progress = true;
              if (n < 0) {
                done[x] = true;
                break;
              }
              left[x] = x == 0 ? (n + 1) >> 1 : n >> 1;
              fresh[x] = 1;
              if (left[x] == 0) {
                mbar_arrive(smem_u32(&ctrl->uempty[us]));
                ++cu[x];
              }
            }
            if (left[x] == 0 || !mbar_test(smem_u32(&ctrl->kfull[x]), cnt[x] & 1)) continue;
            tc_fence_after();
            qk(x, q_sm + (cu[x] & 1) * S::kOperand, x);
            tc_commit(smem_u32(&ctrl->kempty[x]));
            pending[x] = true;
            progress = true;
          }
          if (progress) {
            since = globaltimer_ns();
          } else {
            if (*abort_flag) break;
            if (globaltimer_ns() - since > kWaitLimitNs) {
              *abort_flag = 1;
              raise_status(status, kDevTimeout);
              break;
            }
          }
        }
      }
      // every MMA issued has finished before the tensor memory is given back
      tc_commit(smem_u32(&ctrl->drained));
      mbar_drain(smem_u32(&ctrl->drained), 0);
    }
    __syncwarp();
  } else {
    // ================= softmax =================
    const int x = warp >> 2;             // stream
    const int r = tid & 127;             // tensor-memory lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + x * kKeys, o_col = tmem + lanes + 256 + x * D;
    const float inf = __int_as_float(0x7F800000);
    int sn = 0, on = 0, mn = 0;          // scores, results and merges seen
    int pc = 0;                          // pair mode: tiles seen by the CTA
    for (int un = 0;; ++un) {
      const int us = un & 1;
      if (!mbar_wait(smem_u32(&ctrl->ufull[us]), (un >> 1) & 1, abort_flag, status)) break;
      const Unit u = ctrl->unit[us];
      if (u.n_tiles < 0) break;
      const bool twice = !pair && u.rows <= 64;
      const int row = pair ? x * kTileRows + r : twice ? r & 63 : r;
      const bool live = row < u.rows && (!twice || (r >> 6) == x);
      const bool warp_live = __any_sync(0xFFFFFFFFu, live);
      const int mine = pair ? (x == 0 || u.rows > kTileRows ? u.n_tiles : 0) : x == 0 ? (u.n_tiles + 1) >> 1 : u.n_tiles >> 1;
      const int qi = (u.row0 + row) / a.group;
      const int pos = live ? (SEL ? u.pos0 : u.pos0 + qi) : -1;
      const float f = mine > 0 ? (pair ? ctrl->rowf[us * 256 + row] : ctrl->rowf[us * 128 + r]) : 0.f;
      float M = kMinusHuge, l = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < mine; ++i) {
        const int ord = u.first + (pair ? i : 2 * i + x);
        const Meta& m = ctrl->meta[pair ? (pc + i) & 3 : x * 2 + (sn & 1)];
        if (!mbar_wait(smem_u32(&ctrl->sfull[x]), sn & 1, abort_flag, status)) { ok = false; break; }
        ++sn;
        tc_fence_after();
        if (warp_live) {
          const int key0 = tile_of(u, ord) * kKeys;
          bool masked;
          uint32_t vw[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
          if constexpr (SEL) {
#pragma unroll
            for (int c = 0; c < 4; ++c) vw[c] = m.valid[c];
            masked = (vw[0] & vw[1] & vw[2] & vw[3]) != 0xFFFFFFFFu;
          } else {
            masked = !(key0 + kKeys - 1 <= u.p_lo &&
                       (a.window <= 0 || key0 > u.p_hi - a.window || key0 + kKeys <= a.sinks));
            if (masked) {
              // this row's visible keys of the tile as bits
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                auto below = [&](int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };   // keys < n
                const int k0 = key0 + 32 * c;
                uint32_t seen = below(pos + 1 - k0);
                if (a.window > 0) seen &= ~below(pos - a.window + 1 - k0) | below(a.sinks - k0);
                vw[c] = seen;
              }
            }
          }
          float mx = -inf;
          float s[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld32(s_col + 32 * c, s);
            tmem_ld32_wait(s);
            if (masked) {
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = (vw[c] >> e) & 1u ? s[e] : -inf;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float g = s[16 * h];
#pragma unroll
              for (int e = 1; e < 16; ++e) g = fmaxf(g, s[16 * h + e]);
              mx = fmaxf(mx, fmaf(g, f * m.ks[2 * c + h], m.lv[2 * c + h]));
            }
          }
          if (__any_sync(0xFFFFFFFFu, mx > M + (kBoost + kSlack))) {
            const float next = fmaxf(M, mx - kBoost);
            const float by = exp2_approx(M - next);
            M = next;
            l *= by;
            if (i > 0) {                 // scores are complete, so the last value product is too
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                tmem_ld32(o_col + 32 * c, s);
                tmem_ld32_wait(s);
#pragma unroll
                for (int e = 0; e < 32; ++e) s[e] *= by;
                tmem_st32f(o_col + 32 * c, s);
              }
              tmem_st_wait();
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld32(s_col + 32 * c, s);
            tmem_ld32_wait(s);
            if (masked) {
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = (vw[c] >> e) & 1u ? s[e] : -inf;
            }
            uint32_t pk[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float fa = f * m.ks[2 * c + h], fb = m.lv[2 * c + h] - M;
              float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float w0 = exp2_approx(fmaf(s[16 * h + e], fa, fb)), w1 = exp2_approx(fmaf(s[16 * h + e + 1], fa, fb));
                sum0 += w0;
                sum1 += w1;
                pk[8 * h + e / 2] = kv_pack16(w0, w1, false);
              }
              l = fmaf(sum0 + sum1, m.iv[2 * c + h], l);
            }
            tmem_st16(s_col + 16 * c, pk);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&ctrl->pfull[x]));
      }
      if (!ok) break;
      pc += u.n_tiles;
      if (mine > 0) {
        if (!mbar_wait(smem_u32(&ctrl->ofull[x]), on & 1, abort_flag, status)) break;
        ++on;
        tc_fence_after();
      }
      // solo mode: stream 1 hands its rows to stream 0
      const bool merged = !pair && u.n_tiles > 1;
      float by0 = 1.f, by1 = 0.f;
      const int partner = twice ? (r & 63) : r;           // row of the hand-over buffer
      const int rounds = twice || D == 64 ? 1 : 2;        // 64-column rounds when 128 rows fill the buffer
      constexpr int kCols = D;
      float* ml = ctrl->rowf + 256;
      if (merged && x == 1) {
        const int cols = kCols / rounds;
        for (int h = 0; h < rounds && ok; ++h) {
          if (mn > 0 && !mbar_wait(smem_u32(&ctrl->mempty), (mn - 1) & 1, abort_flag, status)) { ok = false; break; }
          ++mn;
          if (h == 0 && (!twice || r >= 64)) {
            ml[2 * partner] = M;
            ml[2 * partner + 1] = l;
          }
          if (warp_live) {
            for (int c = 0; c < cols / 32; ++c) {
              float s[32];
              tmem_ld32(o_col + h * cols + 32 * c, s);
              tmem_ld32_wait(s);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<float4*>(merge + partner * cols + (((c * 8 + e) ^ (r & 7)) << 2)) =
                    make_float4(s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]);
            }
          }
          mbar_arrive(smem_u32(&ctrl->mfull));
        }
        if (!ok) break;
      }
      if (!merged || x == 0) {
        if (!(x == 1 && (!pair || u.rows <= kTileRows))) {
          // this thread's row goes out: whole result, or a part when the keys are split
          const bool part = p.n_split > 1;
          float* pd = nullptr;
          size_t at = 0;
          if (live) {
            const int rr = u.row0 + row;
            at = (static_cast<size_t>(u.q0) + rr / a.group) * a.q_heads + u.head * a.group + rr % a.group;
            if (part) pd = a.part + static_cast<size_t>(u.item) * unit_rows(p) * (D + 2);
          }
          for (int h = 0; h < (merged ? rounds : 1) && ok; ++h) {
            const int cols = merged ? kCols / rounds : kCols;
            if (merged) {
              if (!mbar_wait(smem_u32(&ctrl->mfull), mn & 1, abort_flag, status)) { ok = false; break; }
              ++mn;
              if (h == 0) {
                const float M1 = ml[2 * partner], l1 = ml[2 * partner + 1];
                const float next = fmaxf(M, M1);
                by0 = exp2_approx(M - next);
                by1 = exp2_approx(M1 - next);
                M = next;
                l = l * by0 + l1 * by1;
              }
            }
            const float inv = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
            if (warp_live) {
              for (int c = 0; c < cols / 32; ++c) {
                float s[32];
                if (mine > 0) {
                  tmem_ld32(o_col + h * cols + 32 * c, s);
                  tmem_ld32_wait(s);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  float4 o1 = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (merged) o1 = *reinterpret_cast<const float4*>(merge + partner * cols + (((c * 8 + e) ^ (r & 7)) << 2));
                  const float* of = reinterpret_cast<const float*>(&o1);
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const float own = mine > 0 ? s[4 * e + q] * by0 : 0.f;
                    s[4 * e + q] = merged ? fmaf(of[q], by1, own) * inv : own * inv;
                  }
                }
                if (live) {
                  const int col = h * cols + 32 * c;
                  if (part) {
                    float4* dst = reinterpret_cast<float4*>(pd + unit_rows(p) * 2 + static_cast<size_t>(row) * D + col);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[e] = make_float4(s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]);
                  } else {
                    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at * D + col);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      dst[e] = make_uint4(kv_pack16(s[8 * e], s[8 * e + 1], a.bf16), kv_pack16(s[8 * e + 2], s[8 * e + 3], a.bf16),
                                          kv_pack16(s[8 * e + 4], s[8 * e + 5], a.bf16),
                                          kv_pack16(s[8 * e + 6], s[8 * e + 7], a.bf16));
                  }
                }
              }
            }
            if (merged) mbar_arrive(smem_u32(&ctrl->mempty));
          }
          if (!ok) break;
          if (live) {
            if (part) {
              pd[2 * row] = M;
              pd[2 * row + 1] = l;
            } else if (a.lse != nullptr) {
              a.lse[at] = l == 0.f ? -inf : (M - kBoost + log2f(l)) * 0.69314718055994530942f;
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&ctrl->uempty[us]));
    }
    // dense: queries that belong to no sequence have no unit
    if constexpr (!SEL) {
      if (x == 1 && p.n_split == 1) {
        for (long long n = blockIdx.x * 128ll + r; n < a.batch.N; n += gridDim.x * 128ll) {
          const KvSeq q = kv_seq(a.batch, a.cache, kv_seq_of_query(a.batch, static_cast<int>(n)));
          if (n >= q.q0 && n < q.q0 + q.nq) continue;
          uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + n * a.q_heads * D;
          for (int i = 0; i < a.q_heads * D; ++i) o[i] = 0;
          if (a.lse != nullptr)
            for (int i = 0; i < a.q_heads; ++i) a.lse[n * a.q_heads + i] = -inf;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of split units in their order: one CTA per unit.
template <int D, bool SEL>
__global__ void __launch_bounds__(256) kv_join_kernel(const TileParams p) {
  const AttnParams& a = p.a;
  const int rows_max = unit_rows(p);
  Unit u;
  int b, len;
  const long long base = static_cast<long long>(blockIdx.x) * p.n_split;
  const bool there = decode_item<SEL>(p, base, u, b, len);
  if (there) {
    for (int i = threadIdx.x; i < u.rows * (D / 4); i += 256) {
      const int r = i / (D / 4), ch = i % (D / 4);
      float M = kMinusHuge, l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < p.n_split; ++s) {
        const float* src = a.part + static_cast<size_t>(base + s) * rows_max * (D + 2);
        const float2 ml = *reinterpret_cast<const float2*>(src + 2 * r);
        const float4 v = *reinterpret_cast<const float4*>(src + rows_max * 2 + static_cast<size_t>(r) * D + ch * 4);
        const float next = fmaxf(M, ml.x);
        const float x = exp2_approx(M - next), y = exp2_approx(ml.x - next);
        M = next;
        l = l * x + ml.y * y;
        acc = make_float4(acc.x * x + v.x * y, acc.y * x + v.y * y, acc.z * x + v.z * y, acc.w * x + v.w * y);
      }
      const int rr = u.row0 + r;
      const size_t at = (static_cast<size_t>(u.q0) + rr / a.group) * a.q_heads + u.head * a.group + rr % a.group;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at * D)[ch] =
          make_uint2(kv_pack16(acc.x * inv, acc.y * inv, a.bf16), kv_pack16(acc.z * inv, acc.w * inv, a.bf16));
      if (ch == 0 && a.lse != nullptr)
        a.lse[at] = l == 0.f ? -__int_as_float(0x7F800000) : (M - kBoost + log2f(l)) * 0.69314718055994530942f;
    }
  }
  if constexpr (!SEL) {
    for (long long n = blockIdx.x; n < a.batch.N; n += gridDim.x) {
      const KvSeq q = kv_seq(a.batch, a.cache, kv_seq_of_query(a.batch, static_cast<int>(n)));
      if (n >= q.q0 && n < q.q0 + q.nq) continue;
      uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + n * a.q_heads * D;
      for (int i = threadIdx.x; i < a.q_heads * D; i += 256) o[i] = 0;
      if (a.lse != nullptr)
        for (int i = threadIdx.x; i < a.q_heads; i += 256) a.lse[n * a.q_heads + i] = -__int_as_float(0x7F800000);
    }
  }
}

constexpr int kSplitItems = 2;           // split units fill at most this many waves of CTAs

template <int D, bool SEL>
cudaError_t launch_tile(TileParams& p, long long units, int num_sms, cudaStream_t stream) {
  const int grid = static_cast<int>(p.items < num_sms ? p.items : num_sms);
  kv_tile_kernel<D, SEL><<<grid, kThreads, TileShape<D>::kBytes, stream>>>(p);
  count_launches(1);
  if (p.n_split > 1) {
    kv_join_kernel<D, SEL><<<static_cast<unsigned>(units), 256, 0, stream>>>(p);
    count_launches(1);
  }
  return cudaGetLastError();
}

template <int D, bool SEL>
cudaError_t init_tile() {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kv_tile_kernel<D, SEL>), cudaFuncAttributeMaxDynamicSharedMemorySize,
                              TileShape<D>::kBytes);
}

}  // namespace

size_t kv_tile_part_floats(int num_sms) { return static_cast<size_t>(kSplitItems) * num_sms * 2 * kTileRows * (128 + 2); }

cudaError_t kv_tile_init() {
  cudaError_t e = init_tile<128, false>();
  if (e == cudaSuccess) e = init_tile<128, true>();
  if (e == cudaSuccess) e = init_tile<64, false>();
  if (e == cudaSuccess) e = init_tile<64, true>();
  return e;
}

cudaError_t launch_kv_tile(const AttnParams& a, int max_q, int num_sms, cudaStream_t stream) {
  TileParams p{};
  p.a = a;
  const bool sel = a.idx != nullptr;
  long long units, tiles;
  if (sel) {
    p.row_tiles = (a.group + kTileRows - 1) / kTileRows;
    units = static_cast<long long>(a.batch.N) * p.row_tiles * a.cache.heads;
    tiles = (a.k + kKeys - 1) / kKeys;
  } else {
    p.pair = static_cast<long long>(max_q) * a.group > kTileRows;
    const int rows = p.pair ? 2 * kTileRows : kTileRows;
    units = (static_cast<long long>(a.batch.N) * a.group / rows + a.batch.B) * a.cache.heads;
    tiles = (static_cast<long long>(a.batch.width) * a.cache.page + kKeys - 1) / kKeys;
  }
  // Too few units to fill the GPU: cut each one's keys, two key tiles to a piece at least.
  const long long room = static_cast<long long>(kSplitItems) * num_sms / units;
  const long long most = (tiles + 1) / 2;
  const long long split = room < most ? room : most;
  p.n_split = static_cast<int>(split > 1 ? split : 1);
  p.items = units * p.n_split;
  if (a.dim == 128) return sel ? launch_tile<128, true>(p, units, num_sms, stream) : launch_tile<128, false>(p, units, num_sms, stream);
  return sel ? launch_tile<64, true>(p, units, num_sms, stream) : launch_tile<64, false>(p, units, num_sms, stream);
}

}  // namespace ltk

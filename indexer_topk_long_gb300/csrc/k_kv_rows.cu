// k_kv_rows.cu -- attention over the paged e4m3 cache for few query rows per KV
// head (decode): each code is read once and meets at most 16 rows, so the cache
// stream bounds the kernel.
//
//   t_j = c_row * ks_j * (q . k_j) + log2(vs_j)       (exponents in base 2)
//   w_j = 2^(t_j - M),  O = sum_j w_j * vcode_j,  l = sum_j w_j / vs_j
//   out = O / l,  lse = (M + log2 l) ln 2
//
// ks, vs are the blocks' scales.  Folding log2(vs) into the exponent keeps the
// weights that meet the value codes at most 2^(kBoost + kSlack) for any scales,
// so they go to the matrix product as f16: 11 significant bits down to 2^-22 of
// the running maximum's weight.  Sums, M and l are fp32.  K and V codes become f16
// exactly; queries (bf16 or f16) become f16 after a power-of-two scaling of the
// row, exact but for elements below 2^-22 of the row's largest.
//
// Work: the (sequence or query, 16-row group, KV head) units' key tiles of 128
// form one line that is cut into equal pieces, one per CTA, so ragged lengths
// need no plan on the host.  A unit cut by a border is merged by the last of its
// CTAs in a fixed order.  Each of a CTA's 4 warps takes 32 keys of a tile through
// its own ring of asynchronous 16-byte copies (no block barrier in the loop).
//
// Keys are the products' rows (S^T = K Q^T, O^T = V^T P) and the query rows their columns, 8 or
// 16: a small group leaves few columns empty, and a lane's weights are of few keys.  P comes
// from the scores' layout by an 8 x 8 transposition across the warp.
//
// Measured (8 KV heads of 4 query heads, D = 128): one sequence of 262144 tokens 94 us, 537 MB
// at 5.7 TB/s, 84% of the copy rate; 64 sequences of 128 to 32768 tokens 141 us, 795 MB at 5.6
// TB/s, 83% (query rows as the products' rows, 16 with 12 of them empty: 97 and 153 us); 16 x 2
// queries of 1000 listed keys 24 us; 2048 listed keys for 64 heads of one KV head 14 us and 777
// tokens 8 us, which is latency.  The look for blocks of zeros is 0.3% of long streams and up to
// 2% of listed keys.  What is left of long streams: the first data come after 5 us, since all SMs
// ask at once, and of an SM's three CTAs the last gets the least of its issue slots and ends up to
// 10% after the first, alone and too few to fill memory.
#include "kv_internal.cuh"

namespace ltk {
namespace {

constexpr int kWarps = 4;
// 12 warps an SM: with 8, the dependent arithmetic of two warps a scheduler bound the kernel.
constexpr int kCtasPerSm = 3;
constexpr int kThreads = kWarps * 32;
constexpr int kGroups = 2;               // 16-key groups a warp takes from a tile
constexpr int kWarpKeys = 16 * kGroups;
constexpr int kTileKeys = kWarps * kWarpKeys;
constexpr int kStages = 2;               // 8 KB each and warp at D = 128: 64 KB in flight an SM
constexpr float kMinusHuge = -3e38f;     // running maximum of a row that has seen nothing
// A weight at the running maximum is 2^kBoost; the maximum is only moved when a
// score exceeds it by more than kSlack, so weights stay below 2^15 < f16's 65504.
constexpr float kBoost = 8.f;
constexpr float kSlack = 7.f;

template <int D, int RT>
struct RowsSmem {
  static constexpr int kRows = 8 * RT;                        // of a unit
  static constexpr int kStageBytes = kWarpKeys * D * 2;
  static constexpr int kMetaFloats = 3 * kWarpKeys;           // ks, vs, valid of each key
  static constexpr int kWarpBytes = kStages * (kStageBytes + kMetaFloats * 4);
  static constexpr int kBytes = kWarps * kWarpBytes + kWarps * kRows * 2 * 4;   // and each row's (M, l)
  // at a piece's end a warp's results take the place of the stage it has just read
  static_assert(kStageBytes >= kRows * D * 4, "merge buffer");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit elements across the warp (row lane / 4, columns 2 (lane % 4) ..), transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Where 16-byte chunk `chunk` of row r of a warp's results lies in its row of the merge buffer:
// a quarter warp's stores are two chunks of every other row of eight.
template <int D>
__device__ __forceinline__ int merge_place(int r, int chunk) {
  return chunk ^ (D == 128 ? (r >> 1) & 3 : ((r >> 1) & 1) | ((r >> 2) & 1) << 2);
}

// A row's new running maximum, kBoost below its largest score; where fp32 holds scores to 16 and
// rounding put it too far below for f16 weights, the largest score itself.
__device__ __forceinline__ float below_top(float top, float next) { return top - next > kSlack + kBoost ? top : next; }

// Row r of a 16-key group and 16-byte chunk: byte offset in the group's codes.  Lanes
// of one quarter warp read chunks of two neighbouring rows (K) or one or two
// chunks of four rows of equal parity (V); the placement keeps each on distinct
// banks.
template <int D>
__device__ __forceinline__ int place(int r, int chunk) {
  if constexpr (D == 128) {
    return r * 128 + ((chunk ^ (r & 6) ^ ((r & 1) << 2)) << 4);
  } else {
    const int slot = (r & ~1) | ((r ^ (r >> 1)) & 1);
    return slot * 64 + ((chunk ^ (((slot >> 2) & 1) << 1)) << 4);
  }
}

// The place of row i * (rows a warp copies at once) + r, given row r's: `at` = place(r, chunk).
template <int D>
__device__ __forceinline__ uint32_t place_next(uint32_t at, int i) {
  return (D == 128 ? at ^ ((i & 1) << 6) : at) + i * 512;
}

struct Unit {
  int q0;          // first query of the unit's sequence (selected: the query)
  int nq;          // its queries (selected: 1)
  int pos0;        // position of the first
  int len;         // cached tokens (selected: list length)
  int head;        // KV head
  int row0;        // first row of the unit: row r is query r / group, head r % group
  int tile0;       // first tile of the unit's window
  int skip;        // tiles [0, skip) are the sinks'
  int b;
  int page0;       // see KvSeq
};

// Where a cursor stands: unit u of its sequence, key tile t of n_tiles.
struct Cursor {
  int left;              // tiles to go
  int t, n_tiles;
  int u;                 // unit within the sequence (dense) or -1
  long long unit;        // unit number (selected)
  Unit w;
};

template <int RT>
__device__ __forceinline__ int groups_of(int rows) { return (rows + 8 * RT - 1) / (8 * RT); }

// Key tiles of sequence s that some query sees: sinks' tiles, then from the first
// query's window start to the end.
__device__ __forceinline__ int tiles_of(const AttnParams& p, const KvSeq& s, int* skip, int* tile0) {
  if (s.nq == 0 || s.len == 0) return 0;
  const int n = (s.len + kTileKeys - 1) / kTileKeys;
  *skip = 0;
  *tile0 = 0;
  if (p.window <= 0) return n;
  const int lo = min(max(max(s.pos0, 0) - p.window + 1, 0) / kTileKeys, n - 1);   // (queries past the table see none of them)
  const int sk = min((min(p.sinks, s.len) + kTileKeys - 1) / kTileKeys, lo);
  *skip = sk;
  *tile0 = lo;
  return sk + n - lo;
}

template <bool SEL, int RT>
__device__ __forceinline__ void enter_unit(const AttnParams& p, Cursor& c) {
  if constexpr (SEL) {
    const int rg = groups_of<RT>(p.group);
    const int per = rg * p.cache.heads;
    const int n = static_cast<int>(c.unit / per), r = static_cast<int>(c.unit % per);
    const int b = kv_seq_of_query(p.batch, n);
    const KvSeq s = kv_seq(p.batch, p.cache, b);
    c.w.b = b;
    c.w.q0 = n;
    c.w.nq = 1;
    c.w.pos0 = (n >= s.q0 && n < s.q0 + s.nq) ? s.pos0 + n - s.q0 : -1;
    c.w.len = p.k;
    c.w.head = r / rg;
    c.w.row0 = (r % rg) * 8 * RT;
    c.w.skip = c.w.tile0 = 0;
    c.n_tiles = (p.k + kTileKeys - 1) / kTileKeys;
  } else {
    const int rg = groups_of<RT>(c.w.nq * p.group);
    c.w.head = c.u / rg;
    c.w.row0 = (c.u % rg) * 8 * RT;
  }
}

// Dense: stand on unit u of sequence b (whose tile count is known to be > 0).
template <bool STEPS>
__device__ __forceinline__ void enter_seq(const AttnParams& p, Cursor& c, int b) {
  const KvSeq s = kv_seq<STEPS>(p.batch, p.cache, b);
  c.w.b = b;
  c.w.q0 = s.q0;
  c.w.nq = s.nq;
  c.w.pos0 = s.pos0;
  c.w.len = s.len;
  c.w.page0 = s.page0;
  c.n_tiles = tiles_of(p, s, &c.w.skip, &c.w.tile0);
}

// One tile forward.
template <bool SEL, bool STEPS, int RT>
__device__ __forceinline__ void advance(const AttnParams& p, Cursor& c) {
  --c.left;
  if (++c.t < c.n_tiles || c.left <= 0) return;
  c.t = 0;
  if constexpr (SEL) {
    ++c.unit;
    enter_unit<SEL, RT>(p, c);
  } else {
    if (++c.u >= groups_of<RT>(c.w.nq * p.group) * p.cache.heads) {
      c.u = 0;
      int b = c.w.b;
      do {
        enter_seq<STEPS>(p, c, ++b);
      } while (c.n_tiles == 0 && b + 1 < p.batch.B);
    }
    enter_unit<SEL, RT>(p, c);
  }
}

struct Feed {            // what the next tile's copies need, fetched a step ahead
  int key;               // selected: this lane's key position as listed, -1 none
  int page[kGroups];     // dense: the groups' pages, -1 beyond the length
};

template <int D, bool SEL, bool STEPS, int RT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv_rows_kernel(const AttnParams p, const int grid) {
  using S = RowsSmem<D, RT>;
  constexpr int kRows = S::kRows;
  constexpr int KS = D / 16;             // k-steps of the score product
  constexpr int NT = D / 8;              // elements of a row's result that a lane holds
  constexpr int CPR = D / 16;            // 16-byte chunks in a row of codes
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ long long sh_start;
  __shared__ long long sh_warp[kWarps];
  __shared__ int sh_b;
  __shared__ int sh_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, cq = lane & 3;

  begin_after_previous();
  // --- this CTA's piece of the line -------------------------------------------------------
  long long total;
  int n_cta = grid;                      // CTAs with work: every one has a tile at least
  Cursor head{};
  if constexpr (SEL) {
    const int tiles = (p.k + kTileKeys - 1) / kTileKeys;
    total = static_cast<long long>(p.batch.N) * groups_of<RT>(p.group) * p.cache.heads * tiles;
    n_cta = static_cast<int>(min(static_cast<long long>(grid), total));
  } else {
    const int each = (p.batch.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * each, p.batch.B), b1 = min(b0 + each, p.batch.B);
    long long mine = 0;
    int sk, t0;
    for (int b = b0; b < b1; ++b) {
      const KvSeq s = kv_seq<STEPS>(p.batch, p.cache, b);
      mine += static_cast<long long>(tiles_of(p, s, &sk, &t0)) * groups_of<RT>(s.nq * p.group) * p.cache.heads;
    }
    long long incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) sh_warp[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh_warp[w];
      total += sh_warp[w];
    }
    n_cta = static_cast<int>(min(static_cast<long long>(grid), max(total, 1ll)));
    const long long start = blockIdx.x * total / n_cta;
    if (mine > 0 && start >= before && start < before + mine) {
      long long x = before;
      for (int b = b0; b < b1; ++b) {
        const KvSeq s = kv_seq<STEPS>(p.batch, p.cache, b);
        const long long n = static_cast<long long>(tiles_of(p, s, &sk, &t0)) * groups_of<RT>(s.nq * p.group) * p.cache.heads;
        if (start < x + n) {
          sh_b = b;
          sh_start = x;
          break;
        }
        x += n;
      }
    }
    __syncthreads();
  }
  const long long start = blockIdx.x * total / n_cta;
  const long long end = blockIdx.x < n_cta ? (blockIdx.x + 1) * total / n_cta : start;
  if (start < end) {
    head.left = static_cast<int>(end - start);
    if constexpr (SEL) {
      const int tiles = (p.k + kTileKeys - 1) / kTileKeys;
      head.unit = start / tiles;
      head.t = static_cast<int>(start % tiles);
    } else {
      enter_seq<STEPS>(p, head, sh_b);
      const long long in = start - sh_start;
      head.u = static_cast<int>(in / head.n_tiles);
      head.t = static_cast<int>(in % head.n_tiles);
    }
    enter_unit<SEL, RT>(p, head);
  }

  unsigned char* ring = smem + warp * S::kWarpBytes;
  float* meta = reinterpret_cast<float*>(ring + kStages * S::kStageBytes);
  const uint32_t ring_u = smem_u32(ring), meta_u = smem_u32(meta);
  float* merge_ml = reinterpret_cast<float*>(smem + kWarps * S::kWarpBytes);    // [warp][16][2]

  // --- producer: one tile's 32 keys of this warp into a stage -----------------------------
  Cursor pc = head;                      // producer cursor
  Feed feed;
  auto fetch = [&]() {                   // index or pages of the next tile to produce
    feed.key = -1;
#pragma unroll
    for (int h = 0; h < kGroups; ++h) feed.page[h] = -1;
    if (pc.left <= 0) return;
    if constexpr (SEL) {
      const int slot = pc.t * kTileKeys + warp * kWarpKeys + lane;
      if (slot < p.k) feed.key = kv_load(p.idx + static_cast<size_t>(pc.w.q0) * p.k + slot);
    } else {
      const int tile = pc.t < pc.w.skip ? pc.t : pc.t - pc.w.skip + pc.w.tile0;
      const int key0 = tile * kTileKeys + warp * kWarpKeys;
      const int* table = p.batch.page_table + static_cast<size_t>(pc.w.b) * p.batch.width + (STEPS ? pc.w.page0 : 0);
#pragma unroll
      for (int h = 0; h < kGroups; ++h)
        if (key0 + 16 * h < pc.w.len) feed.page[h] = kv_load(table + ((key0 + 16 * h) >> p.cache.page_log2));
    }
  };
  int stage_in = 0;
  auto produce = [&]() {
    if (pc.left > 0) {
      const uint32_t kd = ring_u + stage_in * S::kStageBytes, vd = kd + kWarpKeys * D;
      float* m = meta + stage_in * S::kMetaFloats;
      const uint32_t mu = meta_u + stage_in * S::kMetaFloats * 4;
      constexpr int kPer = CPR / 2;      // copies of a group, lane and operand
      const int cr = lane / CPR, ch = lane % CPR;
      const uint32_t at0 = place<D>(cr, ch);
      if constexpr (SEL) {
        const int key = feed.key <= pc.w.pos0 ? feed.key : -1;
        int page = -1;
        if (key >= 0) {
          page = kv_page(p.batch, p.cache, pc.w.b, key);
          if (page < 0 || page >= p.cache.num_pages) {
            raise_status(p.status, kDevArg);
            page = -2;
          }
        }
        long long row = -1;
        m[2 * kWarpKeys + lane] = key >= 0 ? 1.f : 0.f;
        if (page >= 0) {
          const size_t blk = static_cast<size_t>(page) * p.cache.heads + pc.w.head;
          row = static_cast<long long>(blk) * p.cache.page + (key & (p.cache.page - 1));
          cp_async4(mu + lane * 4, p.cache.k_scale + blk);
          cp_async4(mu + (kWarpKeys + lane) * 4, p.cache.v_scale + blk);
        } else {
          m[lane] = page == -2 ? __int_as_float(0x7FC00000) : 1.f;
          m[kWarpKeys + lane] = 1.f;
        }
#pragma unroll
        for (int h = 0; h < kGroups; ++h)
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int r = i * (32 / CPR) + cr;
            const long long rr = __shfl_sync(0xFFFFFFFFu, row, 16 * h + r);
            const size_t o = rr >= 0 ? static_cast<size_t>(rr) * D + ch * 16 : 0;
            const uint32_t at = 16 * h * D + place_next<D>(at0, i);
            cp_async16(kd + at, p.cache.k_codes + o, rr >= 0);
            cp_async16(vd + at, p.cache.v_codes + o, rr >= 0);
          }
      } else {
        const int tile = pc.t < pc.w.skip ? pc.t : pc.t - pc.w.skip + pc.w.tile0;
        const int key0 = tile * kTileKeys + warp * kWarpKeys;
#pragma unroll
        for (int h = 0; h < kGroups; ++h) {
          const int first = key0 + 16 * h;
          if (first >= pc.w.len) break;
          const bool known = feed.page[h] >= 0 && feed.page[h] < p.cache.num_pages;
          if (!known) raise_status(p.status, kDevArg);
          const size_t blk = known ? static_cast<size_t>(feed.page[h]) * p.cache.heads + pc.w.head : 0;
          if (lane == 0) {
            if (known) {
              cp_async4(mu + 8 * h, p.cache.k_scale + blk);
              cp_async4(mu + 8 * h + 4, p.cache.v_scale + blk);
            } else {
              m[2 * h] = __int_as_float(0x7FC00000);
              m[2 * h + 1] = 1.f;
            }
          }
          const size_t o = (blk * p.cache.page + (first & (p.cache.page - 1))) * D + lane * 16;
          const uint8_t *ks = p.cache.k_codes + o, *vs = p.cache.v_codes + o;
          const int rows = known ? pc.w.len - first : 0;      // of the group's 16
          if (rows >= 16) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const uint32_t at = 16 * h * D + place_next<D>(at0, i);
              cp_async16(kd + at, ks + i * 512);
              cp_async16(vd + at, vs + i * 512);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const bool on = i * (32 / CPR) + cr < rows;
              const uint32_t at = 16 * h * D + place_next<D>(at0, i);
              cp_async16(kd + at, on ? ks + i * 512 : p.cache.k_codes, on);
              cp_async16(vd + at, on ? vs + i * 512 : p.cache.v_codes, on);
            }
          }
        }
      }
      advance<SEL, STEPS, RT>(p, pc);
      fetch();
    }
    cp_commit();
    stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
  };
  fetch();
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) produce();

  // Dense: rows of sequences whose queries see no token have no tile on the line.
  if constexpr (!SEL) {
    for (long long n = blockIdx.x; n < p.batch.N && !(STEPS && p.step == 1); n += grid) {
      const KvSeq s = kv_seq<STEPS>(p.batch, p.cache, kv_seq_of_query(p.batch, static_cast<int>(n)));
      if (s.len > 0 && n >= s.q0 && n < s.q0 + s.nq) continue;
      for (int i = tid; i < p.q_heads * D; i += kThreads) reinterpret_cast<uint16_t*>(p.out)[n * p.q_heads * D + i] = 0;
      if (p.lse != nullptr)
        for (int i = tid; i < p.q_heads; i += kThreads) p.lse[n * p.q_heads + i] = -__int_as_float(0x7F800000);
    }
  }

  // --- consumer ---------------------------------------------------------------------------
  // Rows of tile x: 8 x + 2 cq and the next; results: elements g NT .. of both.
  uint32_t qf[RT][KS][2];
  float o[RT][NT / 2][4];                // [.][i]: elements 2 i of both rows, then 2 i + 1
  float M[RT][2], l[RT][2], crow[RT][2];
  int prow[RT][2];                       // the rows' query positions, -1: no such row
  int stage_out = 0;
  long long at = start;                  // where head stands on the line

#pragma unroll 1
  while (head.left > 0) {
    // a unit's piece: tiles [head.t, t_end)
    const int t_begin = head.t;
    const int t_end = min(head.n_tiles, head.t + head.left);
    const int rows_all = head.w.nq * p.group;
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      // as an operand a lane holds row 8 x + g
      const int r = head.w.row0 + g + 8 * x;
      const bool on = r < rows_all;
      const int qi = r / p.group;
      uint4 raw[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (on) {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + (static_cast<size_t>(head.w.q0) + qi) * p.q_stride +
                              static_cast<size_t>(head.w.head * p.group + r % p.group) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)   // chunk cq of each 64 elements: 16 elements, 32 bytes
          raw[i] = kv_load(reinterpret_cast<const uint4*>(src + (i >> 1) * 64 + cq * 16) + (i & 1));
      }
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t ws[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = kv_unpack16(ws[j], p.bf16);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // the row's largest element goes to [2^8, 2^9)
      int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 8;
      e = amax > 0.f && amax < __int_as_float(0x7F800000) ? max(e, -118) : 0;
      const float by = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      const float scale = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      const int pos = on ? (SEL ? head.w.pos0 : max(head.w.pos0 + (STEPS ? qi * p.batch.advance : qi), -1)) : -1;   // (from -1 any window is within 32 bits)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        crow[x][n] = __shfl_sync(0xFFFFFFFFu, scale, (2 * cq + n) * 4);
        prow[x][n] = __shfl_sync(0xFFFFFFFFu, pos, (2 * cq + n) * 4);
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t ws[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = kv_unpack16(ws[j], p.bf16);
          // words 2 i' and 2 i' + 1 of a chunk are k-step i' (bytes 0-1 and 2-3 of a code word)
          const int word = i * 4 + j;
          qf[x][word >> 1][word & 1] = kv_pack16(f.x * by, f.y * by, false);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < RT; ++x) {
#pragma unroll
      for (int i = 0; i < NT / 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[x][i][j] = 0.f;
      M[x][0] = M[x][1] = kMinusHuge;
      // a query past the page table sees a page that is not there: NaN
#pragma unroll
      for (int n = 0; n < 2; ++n) l[x][n] = !SEL && prow[x][n] >= head.w.len ? __int_as_float(0x7FC00000) : 0.f;
    }
    const int p_lo = SEL ? 0 : head.w.pos0 + head.w.row0 / p.group * (STEPS ? p.batch.advance : 1);
    const int p_hi = SEL ? 0 : head.w.pos0 + min(head.w.row0 + kRows - 1, rows_all - 1) / p.group * (STEPS ? p.batch.advance : 1);
    if (!SEL && p_hi >= head.w.len && tid == 0) raise_status(p.status, kDevArg);

#pragma unroll 1
    for (int t = t_begin; t < t_end; ++t) {
      __syncwarp();                      // the stage that is filled next has been read by every lane
      produce();
      cp_wait<kStages - 1>();
      __syncwarp();
      unsigned char* kp = ring + stage_out * S::kStageBytes;
      unsigned char* vp = kp + kWarpKeys * D;
      float* m = meta + stage_out * S::kMetaFloats;
      stage_out = stage_out + 1 == kStages ? 0 : stage_out + 1;
      const int tile = SEL ? t : (t < head.w.skip ? t : t - head.w.skip + head.w.tile0);
      const int key0 = tile * kTileKeys + warp * kWarpKeys;
      if (!SEL && (key0 >= head.w.len || key0 > p_hi)) continue;
      {
        // a key of a block without a value scale: zeros, see kKvLeastScale
        float* vs = SEL ? m + kWarpKeys + lane : m + 2 * (lane >> 4) + 1;
        const bool zeros = (SEL || key0 + (lane & 16) < head.w.len) && !(*vs > 0.f);
        if (__any_sync(0xFFFFFFFFu, zeros)) {
          if (zeros) {
            *vs = kKvLeastScale;
#pragma unroll 1
            for (int i = 0; i < CPR; ++i)
              *reinterpret_cast<uint4*>(vp + (lane & 16) * D + place<D>(lane & 15, i)) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
      }

      float s[RT][kGroups][4] = {};
#pragma unroll
      for (int half = 0; half < D / 64; ++half)
#pragma unroll
        for (int h = 0; h < kGroups; ++h) {
          const uint4 a = *reinterpret_cast<const uint4*>(kp + 16 * h * D + place<D>(g, half * 4 + cq));
          const uint4 b = *reinterpret_cast<const uint4*>(kp + 16 * h * D + place<D>(g + 8, half * 4 + cq));
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t k[4];
            e4m3x4_to_f16(aw[i], k[0], k[2]);
            e4m3x4_to_f16(bw[i], k[1], k[3]);
#pragma unroll
            for (int x = 0; x < RT; ++x) mma_f16(s[x][h], k, qf[x][half * 4 + i][0], qf[x][half * 4 + i][1]);
          }
        }
      // element e of s[x][h]: key 16 h + g + 8 (e >> 1), row 8 x + 2 cq + (e & 1)
      const bool inside = !SEL && key0 + kWarpKeys - 1 <= p_lo &&
                          (p.window <= 0 || key0 > p_hi - p.window || key0 + kWarpKeys <= p.sinks);
      float iv[kGroups][2];              // 1 / vs of the lane's keys
      float mx[RT][2];
#pragma unroll
      for (int x = 0; x < RT; ++x) mx[x][0] = mx[x][1] = -__int_as_float(0x7F800000);
#pragma unroll
      for (int h = 0; h < kGroups; ++h) {
        float ks[2], lv[2];
        bool valid[2] = {true, true};
        if constexpr (SEL) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int at0 = 16 * h + 8 * n + g;
            const float vs = m[kWarpKeys + at0];
            ks[n] = m[at0];
            lv[n] = __log2f(vs) + kBoost;
            iv[h][n] = __frcp_rn(vs);
            valid[n] = m[2 * kWarpKeys + at0] != 0.f;
          }
        } else {
          // a group beyond the length was not copied: its keys are masked, its values skipped
          const float2 sc = key0 + 16 * h < head.w.len ? *reinterpret_cast<const float2*>(m + 2 * h) : make_float2(1.f, 1.f);
          ks[0] = ks[1] = sc.x;
          lv[0] = lv[1] = __log2f(sc.y) + kBoost;
          iv[h][0] = iv[h][1] = __frcp_rn(sc.y);
        }
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kk = e >> 1, n = e & 1;
            float t = fmaf(s[x][h][e], ks[kk] * crow[x][n], lv[kk]);
            if constexpr (SEL) {
              if (!valid[kk]) t = -__int_as_float(0x7F800000);
            } else if (!inside) {
              const int key = key0 + 16 * h + g + 8 * kk;
              const bool seen = key <= prow[x][n] && (p.window <= 0 || key > prow[x][n] - p.window || key < p.sinks);
              if (!seen) t = -__int_as_float(0x7F800000);
            }
            s[x][h][e] = t;
            mx[x][n] = fmaxf(mx[x][n], t);
          }
      }
      bool outgrown = false;
#pragma unroll
      for (int x = 0; x < RT; ++x)
#pragma unroll
        for (int n = 0; n < 2; ++n) outgrown = outgrown || mx[x][n] - M[x][n] > kSlack + kBoost;
      if (__any_sync(0xFFFFFFFFu, outgrown)) {
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float top = mx[x][n];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            const float next = fmaxf(M[x][n], below_top(top, top - kBoost));
            const float by = exp2_approx(M[x][n] - next);
            M[x][n] = next;
            l[x][n] *= by;
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) {
              o[x][i][n] *= by;
              o[x][i][2 + n] *= by;
            }
          }
      }
#pragma unroll
      for (int h = 0; h < kGroups; ++h) {
        if (!SEL && key0 + 16 * h >= head.w.len) break;       // not copied
        uint32_t pf[RT][2];
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const float w0 = exp2_approx(s[x][h][2 * kk] - M[x][0]), w1 = exp2_approx(s[x][h][2 * kk + 1] - M[x][1]);
            l[x][0] = fmaf(w0, iv[h][kk], l[x][0]);
            l[x][1] = fmaf(w1, iv[h][kk], l[x][1]);
            pf[x][kk] = transposed(kv_pack16(w0, w1, false));
          }
        // values: this lane's keys 2 cq, 2 cq + 1 (and + 8), its g-th D / 8 elements
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * cq + (i & 1) + 8 * (i >> 1);
          const unsigned char* row = vp + 16 * h * D;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + place<D>(r, g));
            vw[i][0] = v.x;
            vw[i][1] = v.y;
            vw[i][2] = v.z;
            vw[i][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(row + place<D>(r, g >> 1) + (g & 1) * 8);
            vw[i][0] = v.x;
            vw[i][1] = v.y;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          // elements 4 w .. 4 w + 3 of the lane's, each of two neighbouring keys
          const uint32_t v[4] = {vw[0][w], vw[1][w], vw[2][w], vw[3][w]};
          const uint32_t a01 = __byte_perm(v[0], v[1], 0x5140), a23 = __byte_perm(v[0], v[1], 0x7362);
          const uint32_t b01 = __byte_perm(v[2], v[3], 0x5140), b23 = __byte_perm(v[2], v[3], 0x7362);
          uint32_t e01[4], e23[4];
          e4m3x4_to_f16(a01, e01[0], e01[1]);
          e4m3x4_to_f16(b01, e01[2], e01[3]);
          e4m3x4_to_f16(a23, e23[0], e23[1]);
          e4m3x4_to_f16(b23, e23[2], e23[3]);
#pragma unroll
          for (int x = 0; x < RT; ++x) {
            mma_f16(o[x][2 * w], e01, pf[x][0], pf[x][1]);
            mma_f16(o[x][2 * w + 1], e23, pf[x][0], pf[x][1]);
          }
        }
      }
    }

    // --- the piece's end: warps of the CTA, then CTAs of the unit -------------------------
    // All warps have read the same number of stages, so the free one is the same for all.
    const int spare = stage_out == 0 ? kStages - 1 : stage_out - 1;
    auto merge_of = [&](int w) { return reinterpret_cast<float*>(smem + w * S::kWarpBytes + spare * S::kStageBytes); };
    __syncwarp();
#pragma unroll
    for (int x = 0; x < RT; ++x)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[x][n] += __shfl_xor_sync(0xFFFFFFFFu, l[x][n], d);
        const int r = 8 * x + 2 * cq + n;
        if (head.w.row0 + r >= rows_all) continue;             // no such row
        if (g == 0) {
          merge_ml[(warp * kRows + r) * 2] = M[x][n];
          merge_ml[(warp * kRows + r) * 2 + 1] = l[x][n];
        }
        float* dst = merge_of(warp) + r * D;
#pragma unroll
        for (int i = 0; i < NT / 2; i += 2)
          *reinterpret_cast<float4*>(dst + merge_place<D>(r, (g * NT + 2 * i) >> 2) * 4) =
              make_float4(o[x][i][n], o[x][i][2 + n], o[x][i + 1][n], o[x][i + 1][2 + n]);
      }
    __syncthreads();
    const int rows = min(rows_all - head.w.row0, kRows);
    const bool whole = t_begin == 0 && t_end == head.n_tiles;
    // Contributors of this unit and its place in the workspace.
    const long long u0 = at - t_begin, u1 = u0 + head.n_tiles;       // the unit on the line
    const int c0 = static_cast<int>(((u0 + 1) * n_cta - 1) / total), c1 = static_cast<int>((u1 * n_cta - 1) / total);
    constexpr int kSlot = kRows * (D + 2);
    float* mine = p.part + static_cast<size_t>(2 * blockIdx.x + (t_begin == 0 ? 1 : 0)) * kSlot;
    // the first step's result for a row's piece ch, asked for before it is needed
    const bool joined = STEPS && p.step == 2 && head.w.page0 > 0;
    struct Before {
      float lse;
      float4 o;
    };
    auto place_of = [&](int r) {
      const int row = head.w.row0 + r;
      return (static_cast<size_t>(head.w.q0) + row / p.group) * p.q_heads + head.w.head * p.group + row % p.group;
    };
    auto before_of = [&](int r, int ch) {
      Before b{};
      if (joined) {
        const size_t at = place_of(r);
        b.lse = kv_load(p.mid_lse + at);
        b.o = kv_load(reinterpret_cast<const float4*>(p.mid + at * D) + ch);
      }
      return b;
    };
    auto write_row = [&](int r, int ch, float4 v, float m2, float sum, const Before& b) {
      const size_t at = place_of(r);
      const RowEnd e = row_end(b.lse, joined, m2 - kBoost, sum);
      v = make_float4(v.x * e.own, v.y * e.own, v.z * e.own, v.w * e.own);
      if (STEPS && p.step == 1) {
        reinterpret_cast<float4*>(p.mid + at * D)[ch] = v;
        if (ch == 0) p.mid_lse[at] = e.lse2;
        return;
      }
      if (joined) {
        const float4 o = b.o;
        v = make_float4(fmaf(o.x, e.mid, v.x), fmaf(o.y, e.mid, v.y), fmaf(o.z, e.mid, v.z), fmaf(o.w, e.mid, v.w));
      }
      uint2 w;
      w.x = kv_pack16(v.x, v.y, p.bf16);
      w.y = kv_pack16(v.z, v.w, p.bf16);
      reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at * D)[ch] = w;
      if (ch == 0 && p.lse != nullptr) p.lse[at] = e.lse2 * 0.69314718055994530942f;
    };
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), ch = i % (D / 4);
      const Before b = before_of(r, ch);
      float mx = kMinusHuge;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, merge_ml[(w * kRows + r) * 2]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float by = exp2_approx(merge_ml[(w * kRows + r) * 2] - mx);
        sum = fmaf(merge_ml[(w * kRows + r) * 2 + 1], by, sum);
        const int at = merge_place<D>(r, ch);
        const float4 v = *reinterpret_cast<const float4*>(merge_of(w) + r * D + at * 4);
        acc.x = fmaf(v.x, by, acc.x);
        acc.y = fmaf(v.y, by, acc.y);
        acc.z = fmaf(v.z, by, acc.z);
        acc.w = fmaf(v.w, by, acc.w);
      }
      if (whole) {
        write_row(r, ch, acc, mx, sum, b);
      } else {
        __stcg(reinterpret_cast<float4*>(mine + kRows * 2 + r * D) + ch, acc);
        if (ch == 0) __stcg(reinterpret_cast<float2*>(mine) + r, make_float2(mx, sum));
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) sh_last = atomicAdd(p.counters + c0, 1) == c1 - c0;
      __syncthreads();
      if (sh_last) {
        __threadfence();
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
          const int r = i / (D / 4), ch = i % (D / 4);
          float mx = kMinusHuge, sum = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int cta = c0; cta <= c1; ++cta) {
            const float* src = p.part + static_cast<size_t>(2 * cta + (cta == c0 ? 1 : 0)) * kSlot;
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(src) + r);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + kRows * 2 + r * D) + ch);
            const float next = fmaxf(mx, ml.x);
            const float a = exp2_approx(mx - next), b = exp2_approx(ml.x - next);
            mx = next;
            sum = sum * a + ml.y * b;
            acc.x = acc.x * a + v.x * b;
            acc.y = acc.y * a + v.y * b;
            acc.z = acc.z * a + v.z * b;
            acc.w = acc.w * a + v.w * b;
          }
          write_row(r, ch, acc, mx, sum, before_of(r, ch));
        }
        if (tid == 0) p.counters[c0] = 0;
      }
    }
    __syncthreads();
    // to the next unit
    const int n = t_end - t_begin;
    at += n;
    head.left -= n - 1;
    head.t = t_end - 1;
    advance<SEL, STEPS, RT>(p, head);
  }
  cp_wait<0>();
}

template <int D, bool SEL, bool STEPS, int RT>
cudaError_t init_rows() {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kv_rows_kernel<D, SEL, STEPS, RT>),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, RowsSmem<D, RT>::kBytes);
}

template <int D, bool SEL, bool STEPS>
cudaError_t launch_rows(const AttnParams& p, bool narrow, int grid, cudaStream_t stream) {
  return narrow ? launch_overlapped(kv_rows_kernel<D, SEL, STEPS, 1>, grid, kThreads, RowsSmem<D, 1>::kBytes, stream, p, grid)
                : launch_overlapped(kv_rows_kernel<D, SEL, STEPS, 2>, grid, kThreads, RowsSmem<D, 2>::kBytes, stream, p, grid);
}
template <int D>
cudaError_t launch_rows(const AttnParams& p, bool narrow, int grid, cudaStream_t stream) {
  if (p.idx != nullptr) return launch_rows<D, true, false>(p, narrow, grid, stream);
  return p.step != 0 ? launch_rows<D, false, true>(p, narrow, grid, stream) : launch_rows<D, false, false>(p, narrow, grid, stream);
}

}  // namespace

size_t kv_rows_part_floats(int num_sms) { return static_cast<size_t>(2) * kCtasPerSm * num_sms * kRowsPerUnit * (128 + 2); }
int kv_rows_counters(int num_sms) { return kCtasPerSm * num_sms; }

cudaError_t kv_rows_init() {
  const cudaError_t e[] = {init_rows<128, false, false, 1>(), init_rows<128, false, false, 2>(), init_rows<128, true, false, 1>(),
                           init_rows<128, true, false, 2>(),  init_rows<128, false, true, 1>(),  init_rows<128, false, true, 2>(),
                           init_rows<64, false, false, 1>(),  init_rows<64, false, false, 2>(),  init_rows<64, true, false, 1>(),
                           init_rows<64, true, false, 2>(),   init_rows<64, false, true, 1>(),   init_rows<64, false, true, 2>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_kv_rows(const AttnParams& p, int max_q, int num_sms, cudaStream_t stream) {
  const bool sel = p.idx != nullptr;
  const int grid = kCtasPerSm * num_sms;
  const bool narrow = static_cast<long long>(p.group) * (sel ? 1 : max_q) <= 8;
  count_launches(1);
  return p.dim == 128 ? launch_rows<128>(p, narrow, grid, stream) : launch_rows<64>(p, narrow, grid, stream);
}

}  // namespace ltk

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
// Roles: warps 0-3 and 4-7 softmax, 8-11 key loader, 12-15 value loader (codes from
// global memory through registers, e4m3 to f16, 128-byte-swizzled shared memory; a
// listed key is as good as a paged one), warp 16 issues the MMAs, warp 17 walks the
// CTA's work, warps 18 and 19 bring the queries.
// Work: all units' key tiles form one line, cut into equal pieces, one per CTA; a
// unit cut by a border is merged by the last of its CTAs in a fixed order.
//
// Bound by the products, and by the softmax that feeds them: a pair's key tile takes four
// 128-cubes, 2050 cycles of the tensor cores at D = 128, and 2 x 128 x 128 exponentials, 1024
// cycles of each scheduler's exp2 unit.  2048 queries at the end of 32768 tokens, 8 KV heads of
// 4: 778 us, 1.37 PFLOP/s, 72% of the matrix rate (some 20 us of it is that a warp's lanes agree on
// whether a wait was given up).  Small work is bound by what a unit costs to
// begin and end (lookups, queries, the first tile's maxima, the joining of pieces: some 20 us):
// 24 ragged chunks of 1362 tokens with a window of 1024, D = 64, 42 us.
#include "kv_tensor.cuh"

namespace ltk {
namespace {

constexpr int kLoaders = 4;              // warps that load a tile of an operand, 32 keys each
// Warps of each role and registers a thread (launched evenly, then moved between the
// warpgroups so that no role spills in its loop).  Narrow form (at most 64 rows): the two
// streams' rows lie in the two halves of one row tile, so one warpgroup serves both, and
// its place goes to a second set of loaders, one set for each stream.
template <int D, bool NARROW>
struct Roles {
  static constexpr int kSoftmaxWarps = NARROW ? 4 : 8, kStreamWarps = kSoftmaxWarps / 2;
  static constexpr int kSets = NARROW ? 2 : 1;                // of key and value loaders
  static constexpr int kLoad = kSoftmaxWarps, kRest = kLoad + kSets * 2 * kLoaders;
  static constexpr int kThreads = (kRest + 4) * 32;
  static constexpr int kLaunchRegs = NARROW ? 80 : 96;
  static constexpr int kSoftmaxRegs = NARROW ? 112 : D == 64 ? 128 : 120, kLoadRegs = 72, kRestRegs = NARROW || D == 64 ? 80 : 96;
  static_assert(kSoftmaxWarps / 4 * kSoftmaxRegs + kSets * 2 * kLoadRegs + kRestRegs <= kThreads / 128 * kLaunchRegs, "register split");
};

struct Unit {                            // a piece of a work unit
  int n_tiles;                           // key tiles; -1: no more pieces
  int first;                             // ordinal of the first of them
  int rows;                              // live rows
  int row0;                              // first row: row r is query q0 + r / group, head r % group
  int q0;
  int pos0;                              // position of query q0
  int p_lo, p_hi;                        // smallest and largest position of the rows
  int head;
  int skip, tile0;                       // ordinals below skip are the sinks' tiles, the rest start at tile0
  int b;                                 // sequence
  int len;                               // cached tokens (listed: list length)
  int part;                              // -1: the whole unit; else its place in the workspace
  int c0, c1;                            // CTAs that hold the unit's pieces
};

struct Meta {                            // scales of a key tile's eight 16-key groups
  float ks[8];
  float lv[8];                           // log2(vs) + kBoost
  float iv[8];                           // 1 / vs
  uint32_t valid[4];                     // listed keys: bit per key
};

struct Ctrl {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], ofull[2];
  uint64_t ufull[2], uempty[2], qfull[2], qempty, qraw, mfull, mempty, drained, wg[2];
  uint32_t tmem;
  int abort_flag;
  int last[2];
  Unit unit[2];
  Meta meta[4];
  // solo mode: score factor of each row by unit slot [2][128], then stream 1's (M, l) [128][2]
  float rowf[512];
  long long at, left;                    // the CTA's piece of the line
  int slot, head, t;                     // where it begins
  Unit first;                            // dense: the row tile there, decoded
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

struct TileParams {
  AttnParams a;
  int pair;                              // 1: pair mode
  int rows;                              // rows of a unit
  uint32_t group_magic;                  // 2^32 / group rounded up (0 for a group of 1)
  int row_tiles;                         // listed keys: row tiles of a group
  int slots;                             // row tiles over all sequences (an upper bound when dense)
};


// Dense row tiles are numbered without a scan: sequence b's start at
// cu_q[b] * group / rows + b, which leaves room for every row tile.
__device__ __forceinline__ long long slot_start(const TileParams& p, int b) {
  return static_cast<long long>(kv_load(p.a.batch.cu_q + b)) * p.a.group / p.rows + b;
}

// Row tile `slot`: its fields, and the number of its key tiles (at least 1 on the
// line, so that rows that see nothing are written too); 0: nothing there.  `b`:
// where to begin looking for the sequence, -1 anywhere.
template <bool SEL>
__device__ int decode_slot(const TileParams& p, int slot, int b, Unit& u, int& tiles) {
  const AttnParams& a = p.a;
  if constexpr (SEL) {
    const int n = slot / p.row_tiles;
    u.row0 = (slot - n * p.row_tiles) * p.rows;
    u.rows = min(a.group - u.row0, p.rows);
    u.b = kv_seq_of_query(a.batch, n);
    const KvSeq q = kv_seq(a.batch, a.cache, u.b);
    u.q0 = n;
    u.pos0 = (n >= q.q0 && n < q.q0 + q.nq) ? q.pos0 + n - q.q0 : -1;
    u.p_lo = u.p_hi = u.pos0;
    u.skip = u.tile0 = 0;
    u.len = a.k;
    tiles = (a.k + kKeys - 1) / kKeys;
    return tiles;
  } else {
    if (b < 0) {
      int lo = 0, hi = a.batch.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (slot_start(p, mid) <= slot) lo = mid; else hi = mid - 1;
      }
      b = lo;
    } else {
      while (b + 1 < a.batch.B && slot_start(p, b + 1) <= slot) ++b;
    }
    u.b = b;
    const KvSeq q = kv_seq(a.batch, a.cache, b);
    const long long row0 = (slot - slot_start(p, b)) * p.rows;
    const long long all = static_cast<long long>(q.nq) * a.group;
    tiles = 0;
    if (row0 < 0 || row0 >= all) return 0;
    u.row0 = static_cast<int>(row0);
    u.rows = static_cast<int>(min(all - row0, static_cast<long long>(p.rows)));
    u.q0 = q.q0;
    u.pos0 = q.pos0;
    u.p_lo = q.pos0 + u.row0 / a.group;
    u.p_hi = q.pos0 + (u.row0 + u.rows - 1) / a.group;
    u.len = q.len;
    u.skip = u.tile0 = 0;
    const int last = min(u.p_hi, u.len - 1);                  // (queries past the table: see kv_seq)
    tiles = last >= 0 ? last / kKeys + 1 : 0;
    if (tiles > 0 && a.window > 0) {
      u.tile0 = min(max(max(u.p_lo, 0) - a.window + 1, 0) / kKeys, tiles);
      u.skip = min((min(a.sinks, last + 1) + kKeys - 1) / kKeys, u.tile0);
      tiles = u.skip + tiles - u.tile0;
    }
    return max(tiles, 1);
  }
}

// --- loader ---------------------------------------------------------------------------------
// Thread mapping of an operand's 128-key tile: warp w holds the keys 32 w .. (two
// 16-key groups); a lane's NI rows and its 16-byte chunk of codes are chosen so that
// a quarter warp's 16-byte shared stores fall on distinct banks (two rows of
// different parity, four chunks).  Row i is row 0 plus kStep * i.
template <int D>
struct Map {
  static constexpr int NI = D == 128 ? 8 : 4;
  static constexpr int kStep = 32 / NI;
  static __device__ __forceinline__ int row0(int lane) { return D == 128 ? (lane >> 4) * 2 + ((lane >> 2) & 1) : lane >> 2; }
  static __device__ __forceinline__ int chunk(int lane) { return D == 128 ? (lane & 3) + 4 * ((lane >> 3) & 1) : lane & 3; }
};

__device__ __forceinline__ int tile_of(const Unit& u, int ord) { return ord < u.skip ? ord : ord - u.skip + u.tile0; }
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

// Listed keys come from blocks of different scales: the codes are multiplied by
// 64 * scale / (largest scale of the 16-key group), exact in f16 for ratios down
// to 2^-21 (an e4m3 code is a multiple of 2^-9, f16's smallest step 2^-24).
// s: this lane's row's scale; returns its group's.
__device__ __forceinline__ float group_scale(float s) {
  float m = fmaxf(s, 0.f);               // a NaN (page outside the pool) counts as 0
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m > 0.f ? m : kKvLeastScale;
}

// Codes pass the little L1 that the operands leave: page tables and indices stay in it.
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// A warp's 32 rows of codes (16 a lane and row) to swizzled f16 rows.  at: the lane's
// place of row 0's first chunk of f16 in the operand; rows kStep apart lie kStep * 128
// bytes apart, and their swizzle differs in one bit where kStep is 4.
template <int D, bool SEL>
__device__ __forceinline__ void store_rows(uint32_t at, int lane, const uint4 (&x)[Map<D>::NI], uint32_t factor) {
#pragma unroll
  for (int i = 0; i < Map<D>::NI; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) e4m3x4_to_f16(w[e], h[2 * e], h[2 * e + 1]);
    if constexpr (SEL) {
      const uint32_t by = __shfl_sync(0xFFFFFFFFu, factor, Map<D>::row0(lane) + Map<D>::kStep * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[e]), *reinterpret_cast<const __half2*>(&by));
        h[e] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    const uint32_t to = (at ^ ((Map<D>::kStep * i & 7) << 4)) + Map<D>::kStep * i * 128;
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to ^ 16u), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]) : "memory");
  }
}

// Queries come in two steps, since a round trip to memory for every few rows would hold
// up the next unit: all rows by asynchronous copies to where their f16 form will stand
// (16-bit elements either way), then converted in place by convert_query.
//
// The copies, by warps w = 0, 1: rows [r0, r0 + 128) of the unit; rows repeat with period mask + 1,
// rows past the unit's are zero.
template <int D>
__device__ __forceinline__ void copy_queries(const TileParams& p, const Unit& u, uint32_t base, int r0, int mask, int w, int lane) {
  constexpr int LPR = D / 8, RPP = 32 / LPR;
  const AttnParams& a = p.a;
  const int j = lane % LPR;
  // row0 + r is head (row0 % group + r) % group of query row0 / group + (row0 % group + r) / group:
  // one division, then products with 2^32 / group rounded up, exact for the at most
  // 256 + group rows meant here while group^2 stays below 2^31
  const int q0 = u.row0 / a.group, g0 = u.row0 - q0 * a.group;
  const uint16_t* head = reinterpret_cast<const uint16_t*>(a.q) + (static_cast<size_t>(u.q0) + q0) * a.q_stride +
                         static_cast<size_t>(u.head) * a.group * D + j * 8;
  const uint32_t column = base + (j >> 3) * (kTileRows * 128);
#pragma unroll 4
  for (int i = 0; i < 64 / RPP; ++i) {
    const int local = 64 * w + lane / LPR + i * RPP;
    const int r = r0 + (local & mask);
    const bool on = r < u.rows;
    const int x = g0 + r;
    const int qi = a.group == 1 ? x : a.group > 32768 ? x / a.group : static_cast<int>(__umulhi(static_cast<uint32_t>(x), p.group_magic));
    const uint16_t* src = on ? head + qi * a.q_stride + (x - qi * a.group) * D : reinterpret_cast<const uint16_t*>(a.q);
    const uint32_t to = column + local * 128 + (((j & 7) ^ (local & 7)) << 4);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(on ? 16 : 0) : "memory");
  }
}
template <int D, bool SEL, bool NARROW>
__global__ void __launch_bounds__(Roles<D, NARROW>::kThreads, 1) kv_tile_kernel(const __grid_constant__ TileParams p) {
  using S = TileShape<D>;
  using R = Roles<D, NARROW>;
  constexpr int kThreads = R::kThreads;
  constexpr int NI = Map<D>::NI;
  extern __shared__ __align__(1024) unsigned char smem[];
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + S::kQ + 2 * S::kStage + S::kMerge);
  const uint32_t q_sm = smem_u32(smem), stage_sm = q_sm + S::kQ;
  float* merge = reinterpret_cast<float*>(smem + S::kQ + 2 * S::kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // uniform
  const AttnParams& a = p.a;
  const bool pair = !NARROW && p.pair != 0;
  volatile int* abort_flag = &ctrl->abort_flag;
  int* status = a.status;

  if (warp == R::kRest) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&ctrl->kfull[i]), kLoaders);
        mbar_init(smem_u32(&ctrl->kempty[i]), 1);
        mbar_init(smem_u32(&ctrl->vfull[i]), kLoaders);
        mbar_init(smem_u32(&ctrl->vempty[i]), 1);
        mbar_init(smem_u32(&ctrl->sfull[i]), 2);
        mbar_init(smem_u32(&ctrl->pfull[i]), R::kStreamWarps);
        mbar_init(smem_u32(&ctrl->ofull[i]), 1);
        mbar_init(smem_u32(&ctrl->ufull[i]), 1);
        mbar_init(smem_u32(&ctrl->uempty[i]), R::kSoftmaxWarps + R::kSets * 2 * kLoaders + 2 + 2);
        mbar_init(smem_u32(&ctrl->qfull[i]), pair ? 8 : 2);
        mbar_init(smem_u32(&ctrl->wg[i]), 32 * R::kStreamWarps);
      }
      mbar_init(smem_u32(&ctrl->qempty), 1);
      mbar_init(smem_u32(&ctrl->qraw), 2);
      mbar_init(smem_u32(&ctrl->mfull), R::kStreamWarps);
      mbar_init(smem_u32(&ctrl->mempty), R::kStreamWarps);
      mbar_init(smem_u32(&ctrl->drained), 1);
      ctrl->abort_flag = 0;
      mbar_fence_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(&ctrl->tmem), 512);
  }

  begin_after_previous();

  // --- this CTA's piece of the line (head, row tile, key tile), every CTA one tile at least ---
  long long total;
  int n_cta = gridDim.x;
  {
    Unit u;
    int tiles;
    if constexpr (SEL) {
      tiles = (a.k + kKeys - 1) / kKeys;
      // Whole units in turn for as many waves as there are (neighbouring queries choose many
      // of the same keys, so they run at the same time and L2 serves them); the line holds the rest.
      const long long units = static_cast<long long>(p.slots) * a.cache.heads;
      const long long whole = units / gridDim.x * gridDim.x;
      total = (units - whole) * tiles;
      n_cta = static_cast<int>(min(static_cast<long long>(n_cta), max(total, 1ll)));
      if (tid == 0) {
        const long long at = blockIdx.x * total / n_cta;
        const long long unit = whole + at / tiles;
        ctrl->at = at;
        ctrl->left = blockIdx.x < n_cta ? (blockIdx.x + 1) * total / n_cta - at : 0;
        ctrl->t = static_cast<int>(at % tiles);
        ctrl->head = static_cast<int>(unit % a.cache.heads);
        ctrl->slot = static_cast<int>(unit / a.cache.heads);
      }
    } else {
      long long* sums = reinterpret_cast<long long*>(smem);   // free until the first queries come
      // Row tiles are numbered by cu_q, so it has to rise within [0, N]; else nothing is done.
      bool rises = true;
      for (int i = tid; i < a.batch.B; i += kThreads) {
        const int at = kv_load(a.batch.cu_q + i), to = kv_load(a.batch.cu_q + i + 1);
        rises = rises && at >= 0 && at <= to && to <= a.batch.N;
      }
      const int each = (p.slots + kThreads - 1) / kThreads;
      const int s0 = min(tid * each, p.slots), s1 = min(s0 + each, p.slots);
      long long mine = 0;
      int b = -1, n = 0;
      for (int s = s0; s < s1; ++s) {
        n = decode_slot<SEL>(p, s, b, u, tiles);
        mine += n;
        b = u.b;
      }
      long long incl = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sums[warp] = incl;
      if (tid == 0) ctrl->left = 0;
      const bool wrong = __syncthreads_or(rises ? 0 : 1) != 0;
      if (wrong && tid == 0) raise_status(status, kDevArg);
      long long before = incl - mine, one = 0;                // one: a head's tiles
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        one += sums[w];
      }
      total = wrong ? 0 : one * a.cache.heads;
      n_cta = static_cast<int>(min(static_cast<long long>(n_cta), max(total, 1ll)));
      if (total > 0 && blockIdx.x < n_cta) {
        const long long at = blockIdx.x * total / n_cta;
        const long long in = at % one;
        if (in >= before && in < before + mine) {
          long long x = before;
          b = -1;
          for (int s = s0; s < s1; ++s) {
            if (each > 1) n = decode_slot<SEL>(p, s, b, u, tiles);   // else still at hand
            b = u.b;
            if (in < x + n) {
              u.n_tiles = n;             // on the line, and to see
              u.first = tiles;
              ctrl->first = u;
              ctrl->at = at;
              ctrl->left = (blockIdx.x + 1) * total / n_cta - at;
              ctrl->t = static_cast<int>(in - x);
              ctrl->slot = s;
              ctrl->head = static_cast<int>(at / one);
              break;
            }
            x += n;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem;

  if (warp >= R::kRest) {
    if constexpr (R::kRestRegs < R::kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kRestRegs));
    if (warp == R::kRest + 1) {
      // ================= the CTA's pieces, one after the other =================
      if (lane == 0) {
        long long at = ctrl->at, left = ctrl->left;
        int slot = ctrl->slot, head = ctrl->head, t = ctrl->t, b = -1;
        const int waves = SEL ? static_cast<int>(static_cast<long long>(p.slots) * a.cache.heads / gridDim.x) : 0;
        for (int un = 0;; ++un) {
          Unit u{};
          int tiles = 0, n = 0;
          if (un < waves) {
            const long long unit = static_cast<long long>(un) * gridDim.x + blockIdx.x;
            const int at_slot = static_cast<int>(unit / a.cache.heads);
            u.n_tiles = decode_slot<SEL>(p, at_slot, -1, u, tiles);
            u.head = static_cast<int>(unit - static_cast<long long>(at_slot) * a.cache.heads);
            u.part = -1;
          } else if (left > 0) {
            if (!SEL && un == 0) {
              u = ctrl->first;
              n = u.n_tiles;
              tiles = u.first;
            } else {
              n = decode_slot<SEL>(p, slot, b, u, tiles);
            }
            b = u.b;
            const int end = static_cast<int>(min(static_cast<long long>(n), t + left));
            const long long u0 = at - t, u1 = u0 + n;
            u.head = head;
            u.first = t;
            u.n_tiles = min(end, tiles) - t;
            u.c0 = static_cast<int>(((u0 + 1) * n_cta - 1) / total);
            u.c1 = static_cast<int>((u1 * n_cta - 1) / total);
            u.part = t == 0 && end == n ? -1 : 2 * static_cast<int>(blockIdx.x) + (t == 0 ? 1 : 0);
            at += end - t;
            left -= end - t;
            t = 0;
            if constexpr (SEL) {
              if (++head == a.cache.heads) {
                head = 0;
                ++slot;
              }
            } else if (++slot == p.slots) {
              slot = 0;
              ++head;
              b = -1;
            }
          } else {
            u.n_tiles = -1;
          }
          const int us = un & 1;
          if (un >= 2 && !lane_wait(smem_u32(&ctrl->uempty[us]), ((un >> 1) - 1) & 1, abort_flag, status)) break;
          if (!SEL && u.n_tiles >= 0 && u.p_hi >= u.len && u.p_hi >= 0) raise_status(status, kDevArg);
          ctrl->unit[us] = u;
          mbar_arrive(smem_u32(&ctrl->ufull[us]));
          if (u.n_tiles < 0) break;
          if (!SEL && left > 0) {
            // on to the next row tile with something in it (there is one: the line goes on)
            Unit v;
            int vt;
            for (int looked = 0; looked <= p.slots && decode_slot<SEL>(p, slot, b, v, vt) == 0; ++looked) {
              b = v.b;
              if (++slot == p.slots) {
                slot = 0;
                ++head;
                b = -1;
              }
            }
          }
        }
      }
    } else if (warp >= R::kRest + 2) {
      // ================= queries =================
      for (int un = 0;; ++un) {
        const int us = un & 1;
        if (!warp_wait(smem_u32(&ctrl->ufull[us]), (un >> 1) & 1, abort_flag, status)) break;
        const Unit& u = ctrl->unit[us];
        if (u.n_tiles < 0) break;
        // Pair mode: one buffer.  Also a unit without tiles waits for the one before it to be done
        // with, or qraw could complete a second phase before a softmax warp has seen the first.
        if (pair && un >= 1 && !warp_wait(smem_u32(&ctrl->qempty), (un - 1) & 1, abort_flag, status)) break;
        if (u.n_tiles > 0) {
          const int w = warp - R::kRest - 2;
          if (pair) {                    // the softmax threads convert their rows
            copy_queries<D>(p, u, q_sm, 0, 127, w, lane);
            if (u.rows > kTileRows) copy_queries<D>(p, u, q_sm + S::kOperand, kTileRows, 127, w, lane);
          } else {                       // two buffers, converted here ahead of their use
            copy_queries<D>(p, u, q_sm + us * S::kOperand, 0, u.rows <= 64 ? 63 : 127, w, lane);
          }
          asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
          __syncwarp();
          if (!pair) {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              const int row = 64 * w + 32 * i + lane;
              ctrl->rowf[us * 128 + row] = convert_query<D, kTileRows>(a, q_sm + us * S::kOperand, row);
            }
            fence_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(pair ? &ctrl->qraw : &ctrl->qfull[us]));
          mbar_arrive(smem_u32(&ctrl->uempty[us]));
        }
      }
    } else if (elect_one()) {
      // ================= MMA issue =================
      auto commit = [&](uint64_t* bar) { tc_commit(smem_u32(bar)); };
      auto arrive = [&](uint64_t* bar) { mbar_arrive(smem_u32(bar)); };
      auto wait = [&](uint64_t* bar, uint32_t parity) { return lane_wait(smem_u32(bar), parity, abort_flag, status); };
      auto test = [&](uint64_t* bar, uint32_t parity) { return mbar_test(smem_u32(bar), parity); };
      constexpr uint32_t id_qk = idesc_f16(kTileRows, kKeys, false), id_pv = idesc_f16(kTileRows, D, true);
      auto qk = [&](int x, uint32_t q_tile, int st) {
        const uint64_t q_d = operand_desc(q_tile, 16), k_d = operand_desc(stage_sm + st * S::kStage, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * (kTileRows * 128) + (k & 3) * 32) >> 4;
          mma_ss(tmem + x * kKeys, q_d + off, k_d + off, id_qk, k > 0);
        }
        commit(&ctrl->sfull[x]);
        arrive(&ctrl->sfull[x]);         // passes on what the loader wrote beside K
      };
      auto pv = [&](int x, int st, bool first) {
        const uint64_t v_d = operand_desc(stage_sm + st * S::kStage + S::kOperand, kKeys * 128);
        const uint32_t d = tmem + 256 + x * D, w = tmem + x * kKeys;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) mma_ts(d, w + k * 8, v_d + k * (2048 >> 4), id_pv, !first || k > 0);
      };
      if (pair) {
        int c = 0, nu = 0;
        int sp[2] = {0, 0};              // weights awaited by stream
        bool ok = true;
        while (ok) {
          const int us = nu & 1;
          if (!wait(&ctrl->ufull[us], (nu >> 1) & 1)) break;
          const int n = ctrl->unit[us].n_tiles;
          const bool two = ctrl->unit[us].rows > kTileRows;
          if (n < 0) break;
          if (!wait(&ctrl->qfull[us], (nu >> 1) & 1)) break;
          ++nu;
          if (n > 0) {
            if (!wait(&ctrl->kfull[c & 1], (c >> 1) & 1)) break;
            tc_fence_after();
            qk(0, q_sm, c & 1);
            if (two) qk(1, q_sm + S::kOperand, c & 1);
            commit(&ctrl->kempty[c & 1]);
            for (int i = 0; i < n && ok; ++i, ++c) {
              const int st = c & 1, ns = (c + 1) & 1;
              const bool next = i + 1 < n;
              if (!wait(&ctrl->vfull[st], (c >> 1) & 1) ||
                  !wait(&ctrl->pfull[0], sp[0] & 1)) { ok = false; break; }
              ++sp[0];
              tc_fence_after();
              pv(0, st, i == 0);
              if (!next) commit(&ctrl->ofull[0]);
              if (next) {
                if (!wait(&ctrl->kfull[ns], ((c + 1) >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                qk(0, q_sm, ns);
              }
              if (two) {
                if (!wait(&ctrl->pfull[1], sp[1] & 1)) { ok = false; break; }
                ++sp[1];
                tc_fence_after();
                pv(1, st, i == 0);
              }
              commit(&ctrl->vempty[st]);
              if (two && next) qk(1, q_sm + S::kOperand, ns);
              if (two && !next) commit(&ctrl->ofull[1]);
              if (next) commit(&ctrl->kempty[ns]);
            }
            commit(&ctrl->qempty);
          } else {
            arrive(&ctrl->qempty);
          }
          arrive(&ctrl->uempty[us]);
          arrive(&ctrl->uempty[us]);
        }
      } else {
        // Each stream walks its own key tiles through the units.  Neither may hold up the
        // other (a stream without a tile in some unit runs ahead, and what it waits for can
        // depend on the other's next product), so both are polled.
        int cu[2] = {0, 0}, left[2] = {0, 0}, cnt[2] = {0, 0}, fresh[2] = {1, 1};
        bool pending[2] = {false, false}, done[2] = {false, false};
        uint64_t since = globaltimer_ns();
        int idle = 0;
        while (!(done[0] && done[1])) {
          bool progress = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (done[x]) continue;
            if (pending[x]) {
              if (!test(&ctrl->pfull[x], cnt[x] & 1) || !test(&ctrl->vfull[x], cnt[x] & 1)) continue;
              tc_fence_after();
              pv(x, x, fresh[x]);
              fresh[x] = 0;
              commit(&ctrl->vempty[x]);
              pending[x] = false;
              progress = true;
              ++cnt[x];
              if (--left[x] == 0) {
                commit(&ctrl->ofull[x]);
                commit(&ctrl->uempty[cu[x] & 1]);
                ++cu[x];
              }
            }
            while (left[x] == 0) {       // the stream's next unit with a tile for it
              const int us = cu[x] & 1;
              if (!test(&ctrl->ufull[us], (cu[x] >> 1) & 1)) break;
              const int n = ctrl->unit[us].n_tiles;
              if (n >= 0 && !test(&ctrl->qfull[us], (cu[x] >> 1) & 1)) break;
              progress = true;
              if (n < 0) {
                done[x] = true;
                break;
              }
              left[x] = x == 0 ? (n + 1) >> 1 : n >> 1;
              fresh[x] = 1;
              if (left[x] == 0) {
                arrive(&ctrl->uempty[us]);
                ++cu[x];
              }
            }
            if (left[x] == 0 || !test(&ctrl->kfull[x], cnt[x] & 1)) continue;
            tc_fence_after();
            qk(x, q_sm + (cu[x] & 1) * S::kOperand, x);
            commit(&ctrl->kempty[x]);
            pending[x] = true;
            progress = true;
          }
          if (progress) {
            idle = 0;
          } else if ((++idle & 255) == 0) {
            if (idle == 256) since = globaltimer_ns();
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
      commit(&ctrl->drained);
      mbar_drain(smem_u32(&ctrl->drained), 0);
    }
    __syncwarp();
  } else if (warp >= R::kLoad) {
    // ================= loaders =================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kLoadRegs));
    const int set = NARROW ? (warp - R::kLoad) / (2 * kLoaders) : 0;   // narrow: the stream it loads for
    const bool values = ((warp - R::kLoad) / kLoaders & 1) != 0;
    const int w = (warp - R::kLoad) & (kLoaders - 1);
    const KvCache& c = a.cache;
    const uint8_t* codes = values ? c.v_codes : c.k_codes;
    uint64_t* full = values ? ctrl->vfull : ctrl->kfull;
    uint64_t* empty = values ? ctrl->vempty : ctrl->kempty;
    const int lrow = Map<D>::row0(lane), lchunk = Map<D>::chunk(lane);
    const uint32_t at0 = stage_sm + (values ? S::kOperand : 0) + (lchunk >> 2) * (kKeys * 128) + (32 * w + lrow) * 128 +
                         ((((2 * lchunk) & 7) ^ (lrow & 7)) << 4);
    int cnt[2] = {0, 0};                 // tiles loaded by stream (pair mode: [0] counts all)
    bool ok = true;
    for (int un = 0; ok; ++un) {
      const int us = un & 1;
      if (!warp_wait(smem_u32(&ctrl->ufull[us]), (un >> 1) & 1, abort_flag, status)) break;
      const Unit& u = ctrl->unit[us];   // stays in shared memory: a spilled copy would be read back from L2
      if (u.n_tiles < 0) break;
      const int* table = a.batch.page_table + static_cast<size_t>(u.b) * a.batch.width;
      const int begin = u.first + set, end = u.first + u.n_tiles;
      constexpr int kStep = R::kSets;    // a set's tiles lie that far apart
      // A tile's lookups run ahead of its data, each a whole tile ahead of its use: its
      // page (listed: first its key) is asked for two tiles before its codes are.
      struct Look {
        int key;                         // listed: lane's row's position
        int page, page2;                 // listed: the row's page; dense: the warp's two groups'
      };
      auto key_of = [&](int ord) {
        const int i = ord * kKeys + 32 * w + lane;
        return ord < end && i < a.k ? kv_load(a.idx + static_cast<size_t>(u.q0) * a.k + i) : -1;
      };
      auto look = [&](int ord, int key) {
        Look k{-1, -1, -1};
        if constexpr (SEL) {
          k.key = key <= u.pos0 ? key : -1;
          if (k.key >= 0) k.page = kv_page(a.batch, c, u.b, k.key);
        } else if (ord < end) {
          const int first = tile_of(u, ord) * kKeys + 32 * w;
          if (first < u.len) k.page = kv_load(table + (first >> c.page_log2));
          if (first + 16 < u.len) k.page2 = kv_load(table + ((first + 16) >> c.page_log2));
        }
        return k;
      };
      // Where a tile's rows are: listed, the lane's row; dense, the groups' first rows and
      // how many of the 32 there are.
      struct Place {
        uint32_t row, row2;
        int rows;
        float ks, vs;                    // listed: the lane's row's; dense: group (lane & 1)'s
        bool listed;
      };
      auto place_tile = [&](int ord, const Look& k) {
        Place t{kNoRow, kNoRow, 0, 0.f, 0.f, false};
        if constexpr (SEL) {
          t.listed = k.key >= 0;
          if (t.listed) {
            if (k.page >= 0 && k.page < c.num_pages) {
              const uint32_t blk = static_cast<uint32_t>(k.page) * c.heads + u.head;
              t.row = blk * c.page + (k.key & (c.page - 1));
              t.ks = kv_load(c.k_scale + blk);
              t.vs = kv_load(c.v_scale + blk);
            } else {
              raise_status(status, kDevArg);
              t.ks = __int_as_float(0x7FC00000);
            }
          }
        } else {
          const int key = tile_of(u, ord) * kKeys + 32 * w;
          t.rows = u.len - key;
          const bool known1 = k.page >= 0 && k.page < c.num_pages, known2 = k.page2 >= 0 && k.page2 < c.num_pages;
          const uint32_t b1 = known1 ? static_cast<uint32_t>(k.page) * c.heads + u.head : 0;
          const uint32_t b2 = known2 ? static_cast<uint32_t>(k.page2) * c.heads + u.head : 0;
          if (known1) t.row = b1 * c.page + (key & (c.page - 1));
          if (known2) t.row2 = b2 * c.page + ((key + 16) & (c.page - 1));
          const int h = lane & 1;
          t.ks = t.vs = 1.f;
          if (h ? known2 : known1) {
            t.ks = kv_load(c.k_scale + (h ? b2 : b1));
            t.vs = kv_load(c.v_scale + (h ? b2 : b1));
          } else if (key + 16 * h < u.len) {
            raise_status(status, kDevArg);
            t.ks = __int_as_float(0x7FC00000);
          }
        }
        return t;
      };
      uint4 x[NI];
      auto load_tile = [&](const Place& t) {
        if constexpr (SEL) {
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const uint32_t r = __shfl_sync(0xFFFFFFFFu, t.row, lrow + Map<D>::kStep * i);
            x[i] = make_uint4(0, 0, 0, 0);
            if (r != kNoRow) x[i] = load_codes(codes + static_cast<size_t>(r) * D + lchunk * 16);
          }
        } else {
          const uint8_t* p1 = codes + (static_cast<size_t>(t.row) + lrow) * D + lchunk * 16;
          const uint8_t* p2 = codes + (static_cast<size_t>(t.row2) + lrow) * D + lchunk * 16;
          const int n1 = t.row != kNoRow ? t.rows - lrow : 0, n2 = t.row2 != kNoRow ? t.rows - lrow : 0;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int r = Map<D>::kStep * i;
            x[i] = make_uint4(0, 0, 0, 0);
            if (r < (i < NI / 2 ? n1 : n2))
              x[i] = load_codes((i < NI / 2 ? p1 : p2) + (i < NI / 2 ? r : r - 16) * D);
          }
        }
      };
      Place cur{};
      Look near{}, far{};                // of the next tile and the one after it
      int far_key = -1;                  // listed: of the tile after those
      if (begin < end) {
        int key = -1, near_key = -1, then_key = -1;
        if constexpr (SEL) {
          key = key_of(begin);
          near_key = key_of(begin + kStep);
          then_key = key_of(begin + 2 * kStep);
          far_key = key_of(begin + 3 * kStep);
        }
        const Look first = look(begin, key);
        near = look(begin + kStep, near_key);
        far = look(begin + 2 * kStep, then_key);
        cur = place_tile(begin, first);
        load_tile(cur);
      }
#pragma unroll 1
      for (int ord = begin; ord < end; ord += kStep) {
        const int sx = NARROW ? set : pair ? 0 : (ord - begin) & 1;
        const int n = cnt[sx];
        const int st = pair ? n & 1 : sx, use = pair ? n >> 1 : n;
        Place next{};
        if (ord + kStep < end) next = place_tile(ord + kStep, near);
        uint32_t factor = 0;
        float kg = cur.ks, vg = cur.vs;
        if constexpr (SEL) {
          const float top = group_scale(values ? cur.vs : cur.ks);
          const __half2 f2 = __float2half2_rn((values ? cur.vs : cur.ks) * (64.f / top));
          factor = *reinterpret_cast<const uint32_t*>(&f2);
          if (!values) {
            kg = top * (1.f / 64.f);
            vg = group_scale(cur.vs) * (1.f / 64.f);
          }
        }
        if constexpr (!SEL) {            // groups whose values are zeros, see kKvLeastScale
          const uint32_t zeros = __ballot_sync(0xFFFFFFFFu, !(vg > 0.f));
          if (zeros != 0) {
            if (!(vg > 0.f)) vg = kKvLeastScale;
#pragma unroll
            for (int i = 0; i < NI; ++i)
              if (values && (zeros >> (i < NI / 2 ? 0 : 1) & 1u) != 0) x[i] = make_uint4(0, 0, 0, 0);
          }
        }
        const float lv = __log2f(vg) + kBoost, iv = __frcp_rn(vg);
        if (use > 0 && !warp_wait(smem_u32(&empty[st]), (use - 1) & 1, abort_flag, status)) { ok = false; break; }
        if (!values) {                   // the tile's scales go with its keys
          Meta& m = ctrl->meta[pair ? n & 3 : sx * 2 + (n & 1)];
          if constexpr (SEL) {
            const uint32_t bits = __ballot_sync(0xFFFFFFFFu, cur.listed);
            if (lane == 0) m.valid[w] = bits;
          }
          const int gi = SEL ? lane >> 4 : lane & 1;
          if (SEL ? (lane & 15) == 0 : lane < 2) {
            m.ks[2 * w + gi] = kg;
            m.lv[2 * w + gi] = lv;
            m.iv[2 * w + gi] = iv;
          }
        }
        store_rows<D, SEL>(at0 + st * S::kStage, lane, x, factor);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&full[st]));
        if (ord + kStep < end) load_tile(next);
        near = far;
        far = look(ord + 3 * kStep, far_key);
        if constexpr (SEL) far_key = key_of(ord + 4 * kStep);
        cur = next;
        ++cnt[sx];
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctrl->uempty[us]));
    }
  } else {
    // ================= softmax =================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftmaxRegs));
    const int x = NARROW ? warp >> 1 : warp >> 2;             // stream
    const int r = tid & 127;             // tensor-memory lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + x * kKeys, o_col = tmem + lanes + 256 + x * D;
    const float inf = __int_as_float(0x7F800000);
    int sn = 0, on = 0, mn = 0, wn = 0;  // scores, results, merges and meetings seen
    int pc = 0;                          // pair mode: tiles seen by the CTA
    for (int un = 0;; ++un) {
      const int us = un & 1;
      if (!warp_wait(smem_u32(&ctrl->ufull[us]), (un >> 1) & 1, abort_flag, status)) break;
      const Unit& u = ctrl->unit[us];   // stays in shared memory: a spilled copy would be read back from L2
      if (u.n_tiles < 0) break;
      const bool twice = NARROW || (!pair && u.rows <= 64);
      const int row = pair ? x * kTileRows + r : twice ? r & 63 : r;
      const bool live = row < u.rows && (!twice || (r >> 6) == x);
      const bool warp_live = __any_sync(0xFFFFFFFFu, live);
      const int mine = pair ? (x == 0 || u.rows > kTileRows ? u.n_tiles : 0) : x == 0 ? (u.n_tiles + 1) >> 1 : u.n_tiles >> 1;
      const int pos = live ? (SEL ? u.pos0 : max(u.pos0 + (u.row0 + row) / a.group, -1)) : -1;
      float f = 0.f;                     // scores to base-2 exponents
      if (pair) {
        if (!warp_wait(smem_u32(&ctrl->qraw), un & 1, abort_flag, status)) break;
        if (mine > 0) {
          f = convert_query<D, kTileRows>(a, q_sm + x * S::kOperand, r);
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->qfull[us]));
      } else {
        if (!warp_wait(smem_u32(&ctrl->qfull[us]), (un >> 1) & 1, abort_flag, status)) break;
        if (mine > 0) f = ctrl->rowf[us * 128 + r];
      }
      if (!live) f = 0.f;
      // a query past the page table sees a page that is not there: NaN
      float M = kMinusHuge, l = !SEL && pos >= u.len ? __int_as_float(0x7FC00000) : 0.f;
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < mine; ++i) {
        const int ord = u.first + (pair ? i : 2 * i + x);
        const Meta& m = ctrl->meta[pair ? (pc + i) & 3 : x * 2 + (sn & 1)];
        if (!warp_wait(smem_u32(&ctrl->sfull[x]), sn & 1, abort_flag, status)) { ok = false; break; }
        ++sn;
        tc_fence_after();
        if (warp_live) {
          const int key0 = tile_of(u, ord) * kKeys;
          bool masked;
          if constexpr (SEL) {
            masked = (m.valid[0] & m.valid[1] & m.valid[2] & m.valid[3]) != 0xFFFFFFFFu;
          } else {
            masked = !(key0 + kKeys - 1 <= u.p_lo && (a.window <= 0 || key0 > u.p_hi - a.window || key0 + kKeys <= a.sinks));
          }
          // 32-column pieces from here on still want their weights: all when the tile is masked
          // or the unit's first, else none, or those from where a weight outgrew the slack.
          int from = masked || i == 0 ? 0 : 4;
          if (from != 0) {
            // One pass with the maximum as it stands, half a tile at a time; a half's weights
            // stay in registers until it is known that none outgrew the slack (a group's sum
            // bounds each of its weights), since they take the place of scores.
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t pk[32];
              float s[2][16];
              float l1 = l, most = 0.f;
              tmem_ld32x16(s_col + 64 * hf, s[0]);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float (&v)[16] = s[c & 1];
                tmem_wait_ld_tied(v);
                if (c < 3) tmem_ld32x16(s_col + 64 * hf + 16 * (c + 1), s[(c + 1) & 1]);
                const float fa = f * m.ks[4 * hf + c], fb = m.lv[4 * hf + c] - M;
                const uint64_t fa2 = pack2(fa, fa), fb2 = pack2(fb, fb);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float2 t0 = unpack2(fma2(pack2(v[e], v[e + 1]), fa2, fb2)), t1 = unpack2(fma2(pack2(v[e + 2], v[e + 3]), fa2, fb2));
                  const float w0 = exp2_approx(t0.x), w1 = exp2_approx(t0.y), w2 = exp2_approx(t1.x), w3 = exp2_approx(t1.y);
                  sum0 = add2(sum0, pack2(w0, w1));
                  sum1 = add2(sum1, pack2(w2, w3));
                  pk[8 * c + e / 2] = pack_f16(w0, w1);
                  pk[8 * c + e / 2 + 1] = pack_f16(w2, w3);
                }
                const float2 sm = unpack2(add2(sum0, sum1));
                most = fmaxf(most, sm.x + sm.y);
                l1 = fmaf(sm.x + sm.y, m.iv[4 * hf + c], l1);
              }
              if (__any_sync(0xFFFFFFFFu, most > 32768.f)) {
                from = 2 * hf;
                break;
              }
              l = l1;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pk[16 * c + e];
                tmem_st16(s_col + 32 * hf + 16 * c, w);
              }
            }
          }
          // The general form: 32 columns at a time with masks, the maximum moving as it must.
#pragma unroll 1
          for (int c = from; c < 4; ++c) {
            float s[32];
            tmem_ld32(s_col + 32 * c, s);
            uint32_t seen = 0xFFFFFFFFu;   // this row's visible keys of the 32
            if (masked) {
              if constexpr (SEL) {
                seen = m.valid[c];
              } else {
                auto below = [&](int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };   // keys < n
                const int k0 = key0 + 32 * c;
                seen = below(pos + 1 - k0);
                if (a.window > 0) seen &= ~below(static_cast<int>(static_cast<uint32_t>(pos) - a.window + 1 - k0)) | below(a.sinks - k0);
              }
            }
            const float fa0 = f * m.ks[2 * c], fa1 = f * m.ks[2 * c + 1], fb0 = m.lv[2 * c], fb1 = m.lv[2 * c + 1];
            tmem_ld32_wait(s);
            float mx[4] = {-inf, -inf, -inf, -inf};
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float t = fmaf(s[e], e < 16 ? fa0 : fa1, e < 16 ? fb0 : fb1);
              s[e] = (seen >> e) & 1u ? t : -inf;   // after the scale, which may be NaN (a page outside the pool)
              mx[e & 3] = fmaxf(mx[e & 3], s[e]);
            }
            const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (__any_sync(0xFFFFFFFFu, most - M > kBoost + kSlack)) {
              // What was summed and stored so far follows the new maximum, by a power of two, so
              // that the tile's stored f16 weights are not rounded again (but for subnormal ones).
              const float top = fmaxf(M, below_top(most, ceilf(most - kBoost)));
              const float by = exp2_approx(M - top);
              M = top;
              l *= by;
              uint32_t w[16];
              float v[16];
              if (i > 0) {               // scores are complete, so the last value product is too
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                  tmem_ld32x16(o_col + 16 * q, v);
                  tmem_wait_ld_tied(v);
#pragma unroll
                  for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[e] * by);
                  tmem_st16(o_col + 16 * q, w);
                }
              }
#pragma unroll 1
              for (int q = 0; q < c; ++q) {        // weights of this tile (f16 would end the factor at 2^-24)
                tmem_st_wait();
                tmem_ld32x16(s_col + 16 * q, v);
                tmem_wait_ld_tied(v);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 y = kv_unpack16(__float_as_uint(v[e]), false);
                  w[e] = pack_f16(y.x * by, y.y * by);
                }
                tmem_st16(s_col + 16 * q, w);
              }
            }
            uint32_t pk[16];
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float w0 = exp2_approx(s[e] - M), w1 = exp2_approx(s[e + 1] - M);
              sum[(e >> 4) * 2] += w0;
              sum[(e >> 4) * 2 + 1] += w1;
              pk[e / 2] = pack_f16(w0, w1);
            }
            l = fmaf(sum[0] + sum[1], m.iv[2 * c], fmaf(sum[2] + sum[3], m.iv[2 * c + 1], l));
            tmem_st16(s_col + 16 * c, pk);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->pfull[x]));
      }
      if (!ok) break;
      pc += u.n_tiles;
      if (mine > 0) {
        if (!warp_wait(smem_u32(&ctrl->ofull[x]), on & 1, abort_flag, status)) break;
        ++on;
        tc_fence_after();
      }
      // solo mode: stream 1 hands its rows to stream 0
      const bool merged = !pair && u.n_tiles > 1;
      float by0 = 1.f, by1 = 0.f;
      const int partner = twice ? (r & 63) : r;           // row of the hand-over buffer
      const int rounds = twice || D == 64 ? 1 : 2;        // 64-column rounds when 128 rows fill the buffer
      float* ml = ctrl->rowf + 256;
      const bool writer = pair ? x == 0 || u.rows > kTileRows : x == 0;
      if (merged && x == 1) {
        const int cols = D / rounds;
        for (int h = 0; h < rounds && ok; ++h) {
          if (mn > 0 && !warp_wait(smem_u32(&ctrl->mempty), (mn - 1) & 1, abort_flag, status)) { ok = false; break; }
          ++mn;
          if (h == 0 && (!twice || r >= 64)) {
            ml[2 * partner] = M;
            ml[2 * partner + 1] = l;
          }
          if (warp_live) {
#pragma unroll 1
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
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctrl->mfull));
        }
        if (!ok) break;
      }
      if (writer) {
        // this thread's row goes out: whole result, or a piece to be joined
        const bool part = u.part >= 0;
        const int rows_max = p.rows;
        constexpr int kRowFloats = D + 2;
        float* pd = a.part + static_cast<size_t>(max(u.part, 0)) * rows_max * kRowFloats;
        size_t at = 0;
        if (live) {
          const int rr = u.row0 + row;
          const int qi = rr / a.group;
          at = (static_cast<size_t>(u.q0) + qi) * a.q_heads + u.head * a.group + (rr - qi * a.group);
        }
        auto write_out = [&](int col, const float (&s)[32], float inv) {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at * D + col);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(kv_pack16(s[8 * e] * inv, s[8 * e + 1] * inv, a.bf16),
                                kv_pack16(s[8 * e + 2] * inv, s[8 * e + 3] * inv, a.bf16),
                                kv_pack16(s[8 * e + 4] * inv, s[8 * e + 5] * inv, a.bf16),
                                kv_pack16(s[8 * e + 6] * inv, s[8 * e + 7] * inv, a.bf16));
        };
        for (int h = 0; h < (merged ? rounds : 1) && ok; ++h) {
          const int cols = merged ? D / rounds : D;
          if (merged) {
            if (!warp_wait(smem_u32(&ctrl->mfull), mn & 1, abort_flag, status)) { ok = false; break; }
            ++mn;
            if (h == 0) {
              const float M1 = ml[2 * partner], l1 = ml[2 * partner + 1];
              const float top = fmaxf(M, M1);
              by0 = exp2_approx(M - top);
              by1 = exp2_approx(M1 - top);
              M = top;
              l = l * by0 + l1 * by1;
            }
          }
          const float inv = l == 0.f ? 0.f : 1.f / l;
          if (warp_live) {
#pragma unroll 1
            for (int c = 0; c < cols / 32; ++c) {
              float s[32];
              if (mine > 0) {
                tmem_ld32(o_col + h * cols + 32 * c, s);
                tmem_ld32_wait(s);
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) s[e] = 0.f;
              }
              if (merged) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 o1 = *reinterpret_cast<const float4*>(merge + partner * cols + (((c * 8 + e) ^ (r & 7)) << 2));
                  s[4 * e] = fmaf(o1.x, by1, s[4 * e] * by0);
                  s[4 * e + 1] = fmaf(o1.y, by1, s[4 * e + 1] * by0);
                  s[4 * e + 2] = fmaf(o1.z, by1, s[4 * e + 2] * by0);
                  s[4 * e + 3] = fmaf(o1.w, by1, s[4 * e + 3] * by0);
                }
              }
              if (live) {
                const int col = h * cols + 32 * c;
                if (part) {
                  // column-major in pieces of four, so that a warp's stores lie side by side
                  float4* dst = reinterpret_cast<float4*>(pd + rows_max * 2) + static_cast<size_t>(col / 4) * rows_max + row;
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    __stcg(dst + static_cast<size_t>(e) * rows_max, make_float4(s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]));
                } else {
                  write_out(col, s, inv);
                }
              }
            }
          }
          __syncwarp();
          if (merged && lane == 0) mbar_arrive(smem_u32(&ctrl->mempty));
        }
        if (!ok) break;
        auto write_lse = [&](float m2, float sum) {
          if (a.lse != nullptr) a.lse[at] = sum == 0.f ? -inf : (m2 - kBoost + log2f(sum)) * 0.69314718055994530942f;
        };
        if (!part) {
          if (live) write_lse(M, l);
        } else {
          if (live) __stcg(reinterpret_cast<float2*>(pd) + row, make_float2(M, l));
          // the last of the unit's CTAs joins the pieces in their order
          __threadfence();
          mbar_arrive(smem_u32(&ctrl->wg[x]));
          if (!warp_wait(smem_u32(&ctrl->wg[x]), wn & 1, abort_flag, status)) break;
          ++wn;
          if (r == 0) {
            int* count = a.counters + 2 * u.c0 + x;
            const bool last = atomicAdd(count, 1) == u.c1 - u.c0;
            if (last) *count = 0;
            ctrl->last[x] = last;
          }
          mbar_arrive(smem_u32(&ctrl->wg[x]));
          if (!warp_wait(smem_u32(&ctrl->wg[x]), wn & 1, abort_flag, status)) break;
          ++wn;
          if (*reinterpret_cast<volatile int*>(&ctrl->last[x]) && live) {
            __threadfence();
            const size_t slot_floats = static_cast<size_t>(rows_max) * kRowFloats;
            float top = kMinusHuge, sum = 0.f;
#pragma unroll 4
            for (int cta = u.c0; cta <= u.c1; ++cta) {
              const float2 v = __ldcg(reinterpret_cast<const float2*>(a.part + (2 * cta + (cta == u.c0 ? 1 : 0)) * slot_floats) + row);
              const float next = fmaxf(top, v.x);
              sum = sum * exp2_approx(top - next) + v.y * exp2_approx(v.x - next);
              top = next;
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float s[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = 0.f;
#pragma unroll 1
              for (int cta = u.c0; cta <= u.c1; ++cta) {
                const float* src = a.part + (2 * cta + (cta == u.c0 ? 1 : 0)) * slot_floats;
                const float by = exp2_approx(__ldcg(src + 2 * row) - top);
                const float4* o4 = reinterpret_cast<const float4*>(src + rows_max * 2) + static_cast<size_t>(8 * c) * rows_max + row;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 v = __ldcg(o4 + static_cast<size_t>(e) * rows_max);
                  s[4 * e] = fmaf(v.x, by, s[4 * e]);
                  s[4 * e + 1] = fmaf(v.y, by, s[4 * e + 1]);
                  s[4 * e + 2] = fmaf(v.z, by, s[4 * e + 2]);
                  s[4 * e + 3] = fmaf(v.w, by, s[4 * e + 3]);
                }
              }
              write_out(32 * c, s, inv);
            }
            write_lse(top, sum);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctrl->uempty[us]));
    }
    // dense: queries that belong to no sequence have no unit
    if constexpr (!SEL) {
      if (x == 1) {
        constexpr int kMine = 32 * R::kStreamWarps;             // this stream's threads
        for (long long n = blockIdx.x * static_cast<long long>(kMine) + (r & (kMine - 1)); n < a.batch.N;
             n += gridDim.x * static_cast<long long>(kMine)) {
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
  if (warp == R::kRest) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool SEL, bool NARROW>
cudaError_t init_tile() {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kv_tile_kernel<D, SEL, NARROW>),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, TileShape<D>::kBytes);
}

template <int D, bool SEL>
cudaError_t launch_tile(const TileParams& p, int num_sms, cudaStream_t stream) {
  count_launches(1);
  if constexpr (!SEL) {
    if (p.rows <= 64)
      return launch_overlapped(kv_tile_kernel<D, SEL, true>, num_sms, Roles<D, true>::kThreads, TileShape<D>::kBytes, stream, p);
  }
  return launch_overlapped(kv_tile_kernel<D, SEL, false>, num_sms, Roles<D, false>::kThreads, TileShape<D>::kBytes, stream, p);
}

}  // namespace

size_t kv_tile_part_floats(int num_sms) { return static_cast<size_t>(2) * num_sms * 2 * kTileRows * (128 + 2); }
int kv_tile_counters(int num_sms) { return 2 * num_sms; }

cudaError_t kv_tile_init() {
  const cudaError_t e[6] = {init_tile<128, false, false>(), init_tile<128, false, true>(), init_tile<128, true, false>(),
                            init_tile<64, false, false>(),  init_tile<64, false, true>(),  init_tile<64, true, false>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

// Pairs where a sequence has more rows than a tile and there is work for all SMs.  A pair takes
// as long for a key tile as a single one, but there are half as many units to spread, their
// queries have one buffer, and so each costs more to begin and end.  Two KV heads of 8 query
// heads, D = 128, in us: 16 x 256 queries of 1100 keys (15 pairs' tiles an SM) 82 in pairs and 104
// in single tiles, 1 x 1024 of 4096 (13.5) 66 and 61, 4 x 256 of 1100 (3.8) 50 and 43, 1 x 64 of
// 16384 (3.4) 111 and 66.
bool kv_tile_pairs(const AttnParams& a, int max_q, int num_sms) {
  double keys = static_cast<double>(a.batch.width) * a.cache.page;
  if (a.window > 0) keys = fmin(keys, static_cast<double>(a.window) + a.sinks + max_q);
  const double pairs = a.cache.heads * (static_cast<double>(a.batch.N) * a.group / (2 * kTileRows) + 0.5 * a.batch.B);
  return static_cast<long long>(a.group) * max_q > kTileRows && pairs * (keys / kKeys) >= 14.0 * num_sms;
}

cudaError_t launch_kv_tile(const AttnParams& a, int max_q, int num_sms, cudaStream_t stream) {
  TileParams p{};
  p.a = a;
  p.group_magic = static_cast<uint32_t>((0x100000000ull + a.group - 1) / a.group);
  const bool sel = a.idx != nullptr;
  // Rows that one KV head's keys meet at a time: a pair of tiles, one tile, or a narrow one
  // (max_q is a hint: more rows make more units).
  const long long most = static_cast<long long>(a.group) * (sel ? 1 : max_q);
  p.pair = !sel && kv_tile_pairs(a, max_q, num_sms);
  p.rows = p.pair ? 2 * kTileRows : most <= 64 && !sel ? 64 : kTileRows;
  if (sel) {
    p.row_tiles = (a.group + p.rows - 1) / p.rows;
    p.slots = a.batch.N * p.row_tiles;
  } else {
    p.slots = static_cast<int>(static_cast<long long>(a.batch.N) * a.group / p.rows) + a.batch.B;
  }
  if (a.dim == 128) return sel ? launch_tile<128, true>(p, num_sms, stream) : launch_tile<128, false>(p, num_sms, stream);
  return sel ? launch_tile<64, true>(p, num_sms, stream) : launch_tile<64, false>(p, num_sms, stream);
}

}  // namespace ltk

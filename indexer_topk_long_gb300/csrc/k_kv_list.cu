// k_kv_list.cu -- attention over listed keys of the paged e4m3 cache for up to 64
// query rows (the query heads of one token that share a KV head), on the tensor cores.
//
//   t_jr = f_r * ks_j * (k_j . q_r) + log2(vs_j),  w_jr = 2^(t_jr - M_r)
//   O_r = sum_j w_jr vcode_j,  l_r = sum_j w_jr / vs_j,  out = O / l,  lse = (M + log2 l) ln 2
//
// as in the other attention kernels: each key's value scale is folded into its weights'
// exponent, weights meet the value codes as f16 of at most 2^15, codes become f16 exactly,
// queries after a power-of-two scaling; M, l and O are fp32.
//
// Every query has keys of its own, so a product's 128 rows cannot be filled with queries;
// they are filled with keys instead, and the (at most 64) query rows are its columns:
//   S^T [keys x rows] = K Q^T,  O^T [d x rows] += V^T P.
// A softmax thread holds one key and half of the rows, so a key's scales, place and mask are
// one thread's scalars, and l is kept by thread until the unit ends.  The row maxima are shared
// by the four warps of a half: each tile they vote whether a weight outgrew its f16 range
// (always at a unit's first tile), and only then find new maxima together.
//
// Way of a tile of 128 keys: one of two warps looks the keys up (list, page table, scales;
// each step a tile ahead of the one that needs it); four warps each for K and V copy the
// code rows of their 32 keys to shared memory asynchronously, several tiles ahead, and turn
// them to f16: K to tensor memory, as the first operand of S^T, V to shared memory; one
// thread issues the products; eight warps do the softmax and store P to shared memory.
// Work: units (query, KV head) in whole waves over the CTAs, so that neighbouring queries,
// which choose many of the same keys, run at the same time; the rest as one line of tiles
// cut into equal pieces, a unit cut by a border being joined by the last of its CTAs.
//
// 8192 queries of 2048 keys each, 64 heads on one KV head, D = 128, in a cache of 1M tokens:
// 1063 us, 0.52 PFLOP/s and 4.3 GB of code rows at 4.0 TB/s out of L2.  Bound by the softmax
// warps: a tile takes them some 1900 cycles (scores from tensor memory, 32 rows' weights, the
// vote, P to shared memory) while the products need 640 and the conversions 1300; then a unit
// costs as much as another two tiles to end and begin.  What was tried: 128 query rows a product,
// half of them empty, with both codes converted through registers 1764 us; rows gathered by TMA,
// four to an instruction, 2960 (an instruction took 60 cycles); 16 softmax warps of 16 rows 1318
// against 1255 for 8 of 32; scores asked for a tile ahead 1193 against 1132; loops unrolled less,
// so that the roles' code stays near the schedulers, 1630 -> 1300; P stored after all weights are
// made, its fence behind the vote, 1107 -> 1075.
#include <cstddef>

#include "kv_tensor.cuh"

namespace ltk {
namespace {

constexpr int kRows = kListRows;         // query rows of a unit, at most
constexpr int kHalf = kRows / 2;         // rows of a softmax thread
constexpr int kWarpK = 8, kWarpV = 12, kWarpMma = 16, kWarpUnits = 17, kWarpLook = 18;   // 0 - 7: softmax
constexpr int kThreads = 640;
constexpr int kRingK = 2, kRingV = 3;       // tiles of codes on their way
constexpr int kMetas = 8;                // tiles that are looked up
// Pieces in hand, and how far they are told ahead of their queries.  Keys are looked up as far
// as kRingV tiles ahead of the conversion, which with units of one tile are as many units:
// pieces told later than that, and the conversion would wait for its own products.
constexpr int kPieces = 8, kAhead = 5;
static_assert(kRingK <= kRingV && kAhead >= kRingV + 2 && kPieces >= kAhead + 3 && kMetas > kRingV + 2, "lookups ahead");
// Registers a thread by role; all start with 96.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 120, kConvertRegs = 72, kRestRegs = 96;
static_assert(2 * kSoftmaxRegs + 2 * kConvertRegs + kRestRegs <= 5 * kLaunchRegs, "register split");
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

struct Piece {                           // a piece of a unit
  int n_tiles;                           // -1: no more pieces
  int first;                             // its first tile
  int q;                                 // query
  int head;
  int pos;                               // the query's position, -1: in no sequence
  int b;
  int part;                              // -1: the whole unit; else its place in the workspace
  int c0, c1;                            // CTAs that hold the unit's pieces
};

struct alignas(16) Meta {                // of a tile's keys; written four at a time
  uint32_t k_row[kKeys];                 // code rows, in the order of row_slot; kNoRow: zeros
  uint32_t v_row[kKeys];
  float ks[kKeys];
  float vs[kKeys];                       // -1: nothing listed there
  int end;                               // no tile: the CTA's work ends here
};

struct Ctrl {
  uint64_t look_full[kMetas], look_empty[kMetas];    // lookups
  uint64_t kfull[2], kempty[2], vfull[2], done[2];   // f16 operands; done: the tile's value product
  uint64_t sfull[2], pfull[2], ufull[kPieces], uempty[kPieces], qfull[2], qempty[2], ofull, drained;
  uint32_t tmem;
  int abort_flag;
  int last[2];
  Piece piece[kPieces];
  Meta meta[kMetas];
  float factor[kPieces];                 // scores to base-2 exponents, for key scales of 1; negative: see row_exp
  alignas(16) float minus_max[kRows];    // by row: minus the running maximum
  float most[4][kRows];                  // by warp: maxima, and at the end sums
  float by[kRows];                       // what rows' sums are multiplied by
  alignas(16) uint8_t row_exp[kPieces][kRows];       // exponents of rows scaled by themselves, see convert_queries
};

static_assert(offsetof(Ctrl, meta) % 16 == 0 && sizeof(Meta) % 16 == 0 && offsetof(Meta, vs) % 16 == 0 &&
              offsetof(Ctrl, most) % 8 == 0 && offsetof(Ctrl, by) % 8 == 0, "vector accesses");

template <int D>
struct Shape {
  static constexpr int kCodes = kKeys * D;                    // codes of a tile of K or V
  static constexpr int kV = kKeys * 256;                      // f16 values; for D = 64 half of it is unused
  static constexpr int kP = kKeys * kRows * 2;
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kAtV = (kRingK + kRingV) * kCodes, kAtP = kAtV + 2 * kV, kAtQ = kAtP + 2 * kP;
  static constexpr int kAtCtrl = kAtQ + 2 * kQ;
  static constexpr int kBytes = kAtCtrl + static_cast<int>(sizeof(Ctrl));
};
static_assert(Shape<128>::kBytes <= 232448, "shared memory of a CTA");

struct ListParams {
  AttnParams a;
  int tiles;                             // of a unit
};

// Meeting of the four softmax warps of half x, telling all whether any lane says so.  Every wait in
// between is bounded and every warp comes to every meeting, so none is left waiting.
__device__ __forceinline__ bool meet_any(int x, bool here) {
  uint32_t any;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(any)
               : "r"(here ? 1 : 0), "r"(1 + x)
               : "memory");
  return any != 0;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Reduces 32 values of every lane over the warp: lane i gets value i's result.
template <class F>
__device__ __forceinline__ float reduce_across(float (&v)[32], int lane, F op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float mine = upper ? v[j + o] : v[j], theirs = upper ? v[j] : v[j + o];
      v[j] = op(mine, __shfl_xor_sync(0xFFFFFFFFu, theirs, o));
    }
  }
  return v[0];
}
// Byte of 16-byte chunk c of a row of D codes, so that eight lanes reading a chunk of eight
// rows, or eight chunks of a row (half a row of each of two), meet distinct banks.
template <int D>
__device__ __forceinline__ int code_at(int row, int c) {
  return row * D + ((c ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4);
}
// Largest of a chunk's eight 16-bit magnitudes, which compare as integers, infinities and NaN from
// `bound` on; those count as 0 when `finite`.
__device__ __forceinline__ uint32_t chunk_most(const uint4& x, bool finite, uint32_t bound) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t m = w[e] & 0x7FFF7FFFu;
    if (finite) m = ((m & 0xFFFFu) < bound ? m & 0xFFFFu : 0u) | ((m >> 16) < bound ? m & 0xFFFF0000u : 0u);
    most = __vmaxu2(most, m);
  }
  return max(most & 0xFFFFu, most >> 16);
}
// Exponent of the power of two that takes a largest element to [2^14, 2^15).
__device__ __forceinline__ int query_exp(uint32_t most, bool bf16) {
  return max(static_cast<int>(__float_as_uint(kv_unpack16(most, bf16).x) >> 23) - 127 - 14, -118);
}
__device__ __forceinline__ void scale_chunk(uint32_t at, const uint4& x, int e, bool bf16) {
  const float by = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = kv_unpack16(w[j], bf16);
    w[j] = kv_pack16(f.x * by, f.y * by, false);
  }
  sts128(at, w[0], w[1], w[2], w[3]);
}
// The unit's queries, copied as they are, to f16 in place, by one warp.  As a rule all times one
// power of two, for the largest (finite) element: elements from 2^-29 of the largest on keep f16's
// 11 bits, smaller ones an error of 2^-40 of the largest, which in a row whose own largest is 2^-16
// of that is 2^-24.  Where eight elements lie below 2^-16 together (and not all are 0) every row gets
// a power of its own, and row_exp what turns its scores into the others', as biased fp32 exponents;
// a head's results do not depend on how large the others' queries are.  Returns what turns the
// products into base-2 exponents, negative in the second case.
template <int D>
__device__ __forceinline__ float convert_queries(const AttnParams& a, uint32_t q_sm, uint8_t* row_exp, int lane) {
  const uint32_t bound = a.bf16 ? 0x7F80u : 0x7C00u;
  constexpr int kChunks = kRows * D / 8;
  uint32_t most = 0, least = ~0u;        // least: less 1, so that zeros are left out
#pragma unroll 4
  for (int i = lane; i < kChunks; i += 32) {
    const uint32_t m = chunk_most(lds128(q_sm + i * 16), false, bound);
    most = max(most, m);
    least = min(least, m - 1);
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (most >= bound) {                   // some are not finite: without them
    most = 0;
#pragma unroll 1
    for (int i = lane; i < kChunks; i += 32) most = max(most, chunk_most(lds128(q_sm + i * 16), true, bound));
    most = __reduce_max_sync(0xFFFFFFFFu, most);
  }
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  const int e = most != 0 ? query_exp(most, a.bf16) : 0;
  const float factor = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  if (least < most && kv_unpack16(least + 1, a.bf16).x < kv_unpack16(most, a.bf16).x * 0x1p-16f) {
    // eight lanes to a row (of 64 elements; D = 128: then the other 64), four rows a step
#pragma unroll 1
    for (int i = lane; i < kRows * 8; i += 32) {
      const uint4 x = lds128(q_sm + i * 16);
      uint4 y = make_uint4(0, 0, 0, 0);
      if constexpr (D == 128) y = lds128(q_sm + kRows * 128 + i * 16);
      uint32_t m = max(chunk_most(x, true, bound), chunk_most(y, true, bound));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const int er = m != 0 ? max(query_exp(m, a.bf16), e - 126) : e;
      scale_chunk(q_sm + i * 16, x, er, a.bf16);
      if constexpr (D == 128) scale_chunk(q_sm + kRows * 128 + i * 16, y, er, a.bf16);
      if ((lane & 7) == 0) row_exp[i >> 3] = static_cast<uint8_t>(127 + er - e);
    }
    return -factor;
  }
#pragma unroll 4
  for (int i = lane; i < kChunks; i += 32) scale_chunk(q_sm + i * 16, lds128(q_sm + i * 16), e, a.bf16);
  return factor;
}
// A copying lane's rows (lanes of a row share them) lie side by side: kStep rows to an
// instruction, key % kStep which of them, key % 32 / kStep which instruction.
template <int D>
__device__ __forceinline__ int row_slot(int key) {
  constexpr int kStep = 32 / (D / 16), kAsks = 32 / kStep;
  return (key & ~31) + (key & (kStep - 1)) * kAsks + (key & 31) / kStep;
}
// S^T = K Q^T with K from tensor memory, and O^T += V^T P with both operands' rows of keys.
constexpr uint32_t kIdescS = (1u << 4) | (static_cast<uint32_t>(kRows >> 3) << 17) | (static_cast<uint32_t>(kKeys >> 4) << 24);
constexpr uint32_t kIdescO = kIdescS | (1u << 15) | (1u << 16);

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_list_kernel(const __grid_constant__ ListParams p) {
  using S = Shape<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + S::kAtCtrl);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // uniform
  const AttnParams& a = p.a;
  const KvCache& c = a.cache;
  volatile int* abort_flag = &ctrl->abort_flag;
  int* status = a.status;
  auto wait = [&](uint64_t* bar, int phase) { return warp_wait(smem_u32(bar), phase & 1, abort_flag, status); };
  auto arrive = [&](uint64_t* bar) { mbar_arrive(smem_u32(bar)); };

  if (warp == kWarpMma) {
    if (lane == 0) {
      for (int i = 0; i < kMetas; ++i) {
        mbar_init(smem_u32(&ctrl->look_full[i]), 1);
        mbar_init(smem_u32(&ctrl->look_empty[i]), 8 + 4);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&ctrl->kfull[i]), 4);
        mbar_init(smem_u32(&ctrl->kempty[i]), 1);
        mbar_init(smem_u32(&ctrl->vfull[i]), 4);
        mbar_init(smem_u32(&ctrl->done[i]), 1);
        mbar_init(smem_u32(&ctrl->sfull[i]), 2);
        mbar_init(smem_u32(&ctrl->qfull[i]), 1);
        mbar_init(smem_u32(&ctrl->qempty[i]), 1);
        mbar_init(smem_u32(&ctrl->pfull[i]), 8);
      }
      for (int i = 0; i < kPieces; ++i) {
        mbar_init(smem_u32(&ctrl->ufull[i]), 1);
        mbar_init(smem_u32(&ctrl->uempty[i]), 8 + 2 + 1);
      }
      mbar_init(smem_u32(&ctrl->ofull), 1);
      mbar_init(smem_u32(&ctrl->drained), 1);
      ctrl->abort_flag = 0;
      mbar_fence_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(&ctrl->tmem), 512);
  }
  begin_after_previous();
  const long long units = static_cast<long long>(a.batch.N) * c.heads;
  const int waves = static_cast<int>(units / gridDim.x);
  const long long whole = static_cast<long long>(waves) * gridDim.x, total = (units - whole) * p.tiles;
  const int n_cta = static_cast<int>(min(static_cast<long long>(gridDim.x), max(total, 1ll)));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem;
  const uint32_t s_col = tmem, o_col = tmem + 2 * kRows, k_col = tmem + 3 * kRows;   // S twice, O, K twice

  if (warp >= kWarpMma) {
    if (warp == kWarpUnits) {
      // ================= the CTA's pieces, one after the other; their queries =================
      long long at = blockIdx.x < n_cta ? blockIdx.x * total / n_cta : 0;
      long long left = blockIdx.x < n_cta ? (blockIdx.x + 1) * total / n_cta - at : 0;
      auto tell = [&](int un) {          // piece un; -1 tiles after the last
        Piece u{};
        u.n_tiles = -1;
        u.part = -1;
        long long unit = -1;
        if (un < waves) {
          unit = static_cast<long long>(un) * gridDim.x + blockIdx.x;
          u.n_tiles = p.tiles;
        } else if (left > 0) {
          const long long in = at / p.tiles, u0 = in * p.tiles;
          unit = whole + in;
          u.first = static_cast<int>(at - u0);
          u.n_tiles = static_cast<int>(min(static_cast<long long>(p.tiles - u.first), left));
          u.c0 = static_cast<int>(((u0 + 1) * n_cta - 1) / total);
          u.c1 = static_cast<int>(((u0 + p.tiles) * n_cta - 1) / total);
          if (u.n_tiles < p.tiles) u.part = 2 * static_cast<int>(blockIdx.x) + (u.first == 0 ? 1 : 0);
          at += u.n_tiles;
          left -= u.n_tiles;
        }
        if (unit >= 0) {
          u.q = static_cast<int>(unit / c.heads);
          u.head = static_cast<int>(unit - static_cast<long long>(u.q) * c.heads);
          u.b = kv_seq_of_query(a.batch, u.q);
          const KvSeq s = kv_seq(a.batch, c, u.b);
          u.pos = u.q >= s.q0 && u.q < s.q0 + s.nq ? s.pos0 + u.q - s.q0 : -1;
        }
        const int us = un % kPieces;
        if (un >= kPieces && !wait(&ctrl->uempty[us], un / kPieces - 1)) return false;
        if (lane == 0) {
          ctrl->piece[us] = u;
          arrive(&ctrl->ufull[us]);
        }
        return true;
      };
      bool ok = true;
#pragma unroll 1
      for (int told = 0, un = 0; ok; ++un) {
        while (ok && told <= un + kAhead) ok = tell(told++);
        __syncwarp();
        const int us = un % kPieces;
        if (!ok || ctrl->piece[us].n_tiles < 0) break;
        if (un >= 2 && !wait(&ctrl->qempty[un & 1], (un >> 1) - 1)) break;
        // rows past the group are zero
        const uint32_t q_sm = base + S::kAtQ + (un & 1) * S::kQ;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + static_cast<size_t>(ctrl->piece[us].q) * a.q_stride +
                              static_cast<size_t>(ctrl->piece[us].head) * a.group * D;
        constexpr int kChunks = D / 8;
#pragma unroll 4
        for (int i = lane; i < kRows * kChunks; i += 32) {
          const int r = i / kChunks, j = i % kChunks;
          const bool on = r < a.group;
          const uint32_t to = q_sm + (j >> 3) * (kRows * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(on ? src + r * D + j * 8 : src), "r"(on ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        const float factor = convert_queries<D>(a, q_sm, ctrl->row_exp[us], lane);
        if (lane == 0) ctrl->factor[us] = factor;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&ctrl->qfull[un & 1]);
      }
    } else if (warp >= kWarpLook) {
      // ================= lookups: each warp every other tile =================
      // This lane's keys: 4 lane .. 4 lane + 3 of the tile.
      const int odd = warp - kWarpLook;
      int n0 = 0;                        // the CTA's tiles before this piece
      bool ok = true;
      auto slot_free = [&](int n) { return n < kMetas || wait(&ctrl->look_empty[n % kMetas], n / kMetas - 1); };
      for (int un = 0; ok; ++un) {
        const int us = un % kPieces;
        if (!wait(&ctrl->ufull[us], un / kPieces)) break;
        const Piece u = ctrl->piece[us];
        if (u.n_tiles < 0) {
          if ((n0 & 1) == odd && slot_free(n0) && lane == 0) {
            ctrl->meta[n0 % kMetas].end = 1;
            arrive(&ctrl->look_full[n0 % kMetas]);
          }
          break;
        }
        const int* list = a.idx + static_cast<size_t>(u.q) * a.k;
        const int end = u.first + u.n_tiles;
        auto keys_of = [&](int ord, int (&key)[4]) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = ord * kKeys + 4 * lane + e;
            key[e] = ord < end && i < a.k ? kv_load(list + i) : -1;
          }
        };
        // a key past its query's position does not count
        auto pages_of = [&](int (&key)[4], int (&page)[4]) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (key[e] > u.pos) key[e] = -1;
            page[e] = key[e] >= 0 ? kv_page(a.batch, c, u.b, key[e]) : -1;
          }
        };
        struct Rows {
          uint32_t row[4];
          float ks[4], vs[4];
        };
        auto rows_of = [&](const int (&key)[4], const int (&page)[4], Rows& r) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            r.row[e] = kNoRow;
            r.ks[e] = 0.f;
            r.vs[e] = -1.f;
            if (key[e] >= 0) {
              if (page[e] >= 0 && page[e] < c.num_pages) {
                const uint32_t blk = static_cast<uint32_t>(page[e]) * c.heads + u.head;
                r.row[e] = blk * c.page + (key[e] & (c.page - 1));
                r.ks[e] = kv_load(c.k_scale + blk);
                r.vs[e] = kv_load(c.v_scale + blk);
              } else {
                raise_status(status, kDevArg);
                r.ks[e] = __int_as_float(0x7FC00000);
                r.vs[e] = 1.f;
              }
            }
          }
        };
        // Each lookup is asked for a tile before the next one needs it.
        const int begin = u.first + ((n0 & 1) ^ odd);
        int key0[4], page0[4], key1[4], page1[4], key2[4];
        Rows now;
        keys_of(begin, key0);
        keys_of(begin + 2, key1);
        keys_of(begin + 4, key2);
        pages_of(key0, page0);
        pages_of(key1, page1);
        rows_of(key0, page0, now);
#pragma unroll 1
        for (int ord = begin; ord < end; ord += 2) {
          const int n = n0 + ord - u.first;
          if (!slot_free(n)) { ok = false; break; }
          Meta& meta = ctrl->meta[n % kMetas];
          uint32_t v_row[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v_row[e] = now.row[e];
            if (now.row[e] != kNoRow && !(now.vs[e] > 0.f)) {   // a block without a scale holds zeros
              v_row[e] = kNoRow;
              now.vs[e] = kKvLeastScale;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            meta.k_row[row_slot<D>(4 * lane + e)] = now.row[e];
            meta.v_row[row_slot<D>(4 * lane + e)] = v_row[e];
          }
          *reinterpret_cast<float4*>(&meta.ks[4 * lane]) = make_float4(now.ks[0], now.ks[1], now.ks[2], now.ks[3]);
          *reinterpret_cast<float4*>(&meta.vs[4 * lane]) = make_float4(now.vs[0], now.vs[1], now.vs[2], now.vs[3]);
          if (lane == 0) meta.end = 0;
          __syncwarp();
          if (lane == 0) arrive(&ctrl->look_full[n % kMetas]);
          rows_of(key1, page1, now);
#pragma unroll
          for (int e = 0; e < 4; ++e) key1[e] = key2[e];
          pages_of(key1, page1);
          keys_of(ord + 6, key2);
        }
        n0 += u.n_tiles;
        __syncwarp();
        if (ok && lane == 0) arrive(&ctrl->uempty[us]);
      }
    } else if (elect_one()) {
      // ================= MMA issue =================
      auto lwait = [&](uint64_t* bar, int phase) { return lane_wait(smem_u32(bar), phase & 1, abort_flag, status); };
      auto commit = [&](uint64_t* bar) { tc_commit(smem_u32(bar)); };
      int un = 0;                        // the next piece whose scores are to be issued
      auto next_piece = [&]() {          // its tiles; -1 at the end
        if (!lwait(&ctrl->ufull[un % kPieces], un / kPieces)) return -1;
        const int tiles = ctrl->piece[un % kPieces].n_tiles;
        mbar_arrive(smem_u32(&ctrl->uempty[un % kPieces]));
        if (tiles < 0 || !lwait(&ctrl->qfull[un & 1], un >> 1)) return -1;
        ++un;
        return tiles;
      };
      auto scores = [&](int t) {         // of the CTA's tile t, in piece un - 1
        const uint64_t q_d = operand_desc(base + S::kAtQ + ((un - 1) & 1) * S::kQ, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * (kRows * 128) + (k & 3) * 32) >> 4;
          mma_ts(s_col + (t & 1) * kRows, k_col + (t & 1) * (D / 2) + k * 8, q_d + off, kIdescS, k > 0);
        }
        commit(&ctrl->sfull[t & 1]);
        mbar_arrive(smem_u32(&ctrl->sfull[t & 1]));   // passes on what was looked up beside the keys
        commit(&ctrl->kempty[t & 1]);
      };
      // Scores run a tile ahead of the value products, but not into the next piece: while its
      // first are made, the softmax warps still bring the last results out.
      int n = next_piece(), ahead = n, i = 0;   // tiles of the piece at hand, its scores to do, its products done
      int t = 0, t_scores = 0;
      bool ok = n > 0;
      while (ok) {
        if (ahead > 0 && t_scores <= t + 1) {
          if (!lwait(&ctrl->kfull[t_scores & 1], t_scores >> 1)) break;
          tc_fence_after();
          scores(t_scores++);
          if (--ahead == 0) commit(&ctrl->qempty[(un - 1) & 1]);
          if (t_scores <= t + 1 && ahead > 0) continue;
        }
        if (!lwait(&ctrl->vfull[t & 1], t >> 1) || !lwait(&ctrl->pfull[t & 1], t >> 1)) break;
        tc_fence_after();
        const uint64_t v_d = operand_desc(base + S::kAtV + (t & 1) * S::kV, kKeys * 128);
        const uint64_t p_d = operand_desc(base + S::kAtP + (t & 1) * S::kP, 16);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ss(o_col, v_d + k * (2048 >> 4), p_d + k * (2048 >> 4), kIdescO, i > 0 || k > 0);
        commit(&ctrl->done[t & 1]);
        ++t;
        if (++i == n) {
          commit(&ctrl->ofull);
          n = ahead = next_piece();
          i = 0;
          ok = n > 0;
        }
      }
      // every MMA issued has finished before the tensor memory is given back
      commit(&ctrl->drained);
      mbar_drain(smem_u32(&ctrl->drained), 0);
    }
    __syncwarp();
  } else if (warp >= kWarpK) {
    // ================= codes to f16 =================
    // Each warp copies the rows of its own 32 keys and converts them, so its copies need no
    // barrier: a tile's slot is asked for again as soon as the warp has read it.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
    const bool values = warp >= kWarpV;
    const int w = warp & 3, ring = values ? kRingV : kRingK;
    const uint32_t codes_sm = base + (values ? kRingK * S::kCodes : 0);
    const uint8_t* codes = values ? c.v_codes : c.k_codes;
    int stop = 0x7FFFFFFF;               // the CTA's tiles, once known
    bool ok = true;
    auto ask = [&](int n) {
      if (n < stop) {
        const Meta& meta = ctrl->meta[n % kMetas];
        if (!wait(&ctrl->look_full[n % kMetas], n / kMetas)) {
          ok = false;
        } else if (meta.end != 0) {
          stop = n;
        } else {
          constexpr int kLanes = D / 16, kStep = 32 / kLanes, kAsks = 32 / kStep;   // lanes of a row, rows and number of asks
          const int chunk = lane % kLanes, first = 32 * w + lane / kLanes;
          const uint32_t* rows = (values ? meta.v_row : meta.k_row) + row_slot<D>(first);
          const uint32_t to = codes_sm + n % ring * S::kCodes;
          const uint32_t to0 = to + code_at<D>(first, chunk), to1 = to + code_at<D>(first + kStep, chunk);
          const uint8_t* src = codes + chunk * 16;
          uint32_t row[kAsks];
#pragma unroll
          for (int e = 0; e < kAsks; e += 4) {
            const uint4 r = *reinterpret_cast<const uint4*>(rows + e);
            row[e] = r.x, row[e + 1] = r.y, row[e + 2] = r.z, row[e + 3] = r.w;
          }
#pragma unroll
          for (int e = 0; e < kAsks; ++e)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((e & 1 ? to1 - kStep * D : to0) + e * kStep * D),
                         "l"(src + (row[e] == kNoRow ? 0 : static_cast<size_t>(row[e]) * D)), "r"(row[e] == kNoRow ? 0 : 16)
                         : "memory");
          if (values) {
            __syncwarp();
            if (lane == 0) arrive(&ctrl->look_empty[n % kMetas]);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int n = 0; n < ring && ok; ++n) ask(n);
#pragma unroll 1
    for (int n = 0; ok && n < stop; ++n) {
      if (!values) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRingK - 1) : "memory");
        __syncwarp();
        if (n >= 2 && !wait(&ctrl->kempty[n & 1], (n >> 1) - 1)) break;
        tc_fence_after();
        const uint32_t from = codes_sm + n % kRingK * S::kCodes;
        const uint32_t to = k_col + (n & 1) * (D / 2) + (static_cast<uint32_t>(w * 32) << 16);
#pragma unroll 2
        for (int j = 0; j < D / 32; ++j) {
          uint32_t h[16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 x = lds128(from + code_at<D>(32 * w + lane, 2 * j + e));
            e4m3x4_to_f16(x.x, h[8 * e], h[8 * e + 1]);
            e4m3x4_to_f16(x.y, h[8 * e + 2], h[8 * e + 3]);
            e4m3x4_to_f16(x.z, h[8 * e + 4], h[8 * e + 5]);
            e4m3x4_to_f16(x.w, h[8 * e + 6], h[8 * e + 7]);
          }
          tmem_st16(to + 16 * j, h);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(&ctrl->kfull[n & 1]);
        ask(n + kRingK);
      } else {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRingV - 1) : "memory");
        __syncwarp();
        const uint32_t from = codes_sm + n % kRingV * S::kCodes;
        // a quarter warp reads and writes 16-byte pieces on distinct banks: two rows of
        // different parity, four chunks of each
        constexpr int kStep = D == 128 ? 4 : 8, NI = 32 / kStep;
        const int row0 = 32 * w + (D == 128 ? (lane >> 4) * 2 + ((lane >> 2) & 1) : lane >> 2);
        const int chunk = D == 128 ? (lane & 3) + 4 * (((lane >> 2) ^ (lane >> 3)) & 1) : lane & 3;
        if (n >= 2 && !wait(&ctrl->done[n & 1], (n >> 1) - 1)) break;
        const uint32_t to = base + S::kAtV + (n & 1) * S::kV + (chunk >> 2) * (kKeys * 128);
#pragma unroll 4
        for (int e = 0; e < NI; ++e) {
          const int r = row0 + kStep * e;
          const uint4 x = lds128(from + code_at<D>(r, chunk));
          uint32_t h[8];
          e4m3x4_to_f16(x.x, h[0], h[1]);
          e4m3x4_to_f16(x.y, h[2], h[3]);
          e4m3x4_to_f16(x.z, h[4], h[5]);
          e4m3x4_to_f16(x.w, h[6], h[7]);
          const uint32_t at = to + r * 128 + ((((2 * chunk) & 7) ^ (r & 7)) << 4);
          sts128(at, h[0], h[1], h[2], h[3]);
          sts128(at ^ 16u, h[4], h[5], h[6], h[7]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&ctrl->vfull[n & 1]);
        ask(n + kRingV);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ================= softmax: thread = key of a tile; at the end thread = d =================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp >> 2, t = tid & 127, w = warp & 3;      // rows 32 x .., the thread's key and d
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    const uint32_t o_at = o_col + lanes + x * kHalf;
    const float inf = __int_as_float(0x7F800000);
    const bool idle = x * kHalf >= a.group;                   // no rows: their columns may hold anything
    float* minus_max = ctrl->minus_max + x * kHalf;
    float (*most)[kRows] = ctrl->most;
    float* by = ctrl->by + x * kHalf;
    int n = 0;
    bool ok = true;
    for (int un = 0;; ++un) {
      const int us = un % kPieces;
      if (meet_any(x, !wait(&ctrl->ufull[us], un / kPieces))) break;
      const Piece& u = ctrl->piece[us];
      if (u.n_tiles < 0) break;
      ok = wait(&ctrl->qfull[un & 1], un >> 1);
      if (t < kHalf) minus_max[t] = -kMinusHuge;
      if (meet_any(x, !ok)) break;
      const float factor = fabsf(ctrl->factor[us]);
      const bool uneven = ctrl->factor[us] < 0.f;
      uint64_t l2[kHalf / 2];            // this thread's keys' share of l
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) l2[i] = 0;
      const int tiles = u.n_tiles;
#pragma unroll 1
      for (int i = 0; i < tiles; ++i, ++n) {
        const Meta& meta = ctrl->meta[n % kMetas];
        // (the products of tile n - 2 were issued before these scores, so P's place is free too)
        ok = wait(&ctrl->sfull[n & 1], n >> 1);
        tc_fence_after();
        if (idle) {
          if (meet_any(x, !ok)) { ok = false; break; }
        } else {
          const uint32_t s_at = s_col + lanes + (n & 1) * kRows + x * kHalf;
          const uint32_t p_at = base + S::kAtP + (n & 1) * S::kP + t * 128;
          const float ks = meta.ks[t] * factor, vs = meta.vs[t];
          const float lv = vs > 0.f ? __log2f(vs) + kBoost : -inf, iv = vs > 0.f ? __frcp_rn(vs) : 0.f;
          const uint64_t ks2 = pack2(ks, ks), lv2 = pack2(lv, lv), iv2 = pack2(iv, iv);
          // the maxima may do (with rows scaled by themselves they are found anew for every tile, so
          // that only that path, and not the usual one, has to bring their scores into line)
          bool fresh = i > 0 && !uneven;
          uint64_t w2[kHalf / 2];
#pragma unroll 1
          while (true) {
            float s[32];
            tmem_ld32(s_at, s);
            tmem_ld32_wait(s);
            if (!fresh) {
              if (uneven) {
#pragma unroll
                for (int g = 0; g < kHalf / 4; ++g) {
                  const uint32_t e4 = reinterpret_cast<const uint32_t*>(ctrl->row_exp[us] + x * kHalf)[g];
#pragma unroll
                  for (int r = 0; r < 4; ++r) s[4 * g + r] *= __uint_as_float((e4 >> (8 * r) & 0xFFu) << 23);
                }
              }
              // new maxima: over the tile's keys by warp, then over the warps
              float v[32];
#pragma unroll
              for (int r = 0; r < kHalf; ++r) v[r] = fmaxf(fmaf(s[r], ks, lv), kMinusHuge);
              most[w][x * kHalf + lane] = reduce_across(v, lane, [](float p, float q) { return fmaxf(p, q); });
              if (meet_any(x, !ok)) { ok = false; break; }
              if (t < kHalf) {
                const int r = x * kHalf + t;
                const float high = fmaxf(fmaxf(most[0][r], most[1][r]), fmaxf(most[2][r], most[3][r]));
                const float old = -minus_max[t], next = fmaxf(old, below_top(high, high - kBoost));
                by[t] = exp2_approx(old - next);
                minus_max[t] = -next;
              }
              // sums so far follow; O after its last product
              if (i > 0) ok = wait(&ctrl->done[(n - 1) & 1], (n - 1) >> 1);
              if (meet_any(x, !ok)) { ok = false; break; }
              if (i > 0) {
                tc_fence_after();
#pragma unroll
                for (int r = 0; r < kHalf / 2; ++r) {
                  const float2 f = *reinterpret_cast<const float2*>(&by[2 * r]);
                  l2[r] = mul2(l2[r], pack2(f.x, f.y));
                }
#pragma unroll 1
                for (int q = 0; q < kHalf / 16; ++q) {
                  float o[16];
                  uint32_t o2[16];
                  tmem_ld32x16(o_at + 16 * q, o);
                  tmem_wait_ld_tied(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o2[e] = __float_as_uint(o[e] * by[16 * q + e]);
                  tmem_st16(o_at + 16 * q, o2);
                }
                tmem_st_wait();
              }
            }
            __half2 top = __float2half2_rn(0.f);
            uint32_t h[kHalf / 2];       // stored at the end: a store would hold back the loads of maxima after it
#pragma unroll
            for (int r = 0; r < kHalf; r += 2) {
              const float4 m = *reinterpret_cast<const float4*>(&minus_max[r & ~3]);
              // (rounded as the maxima are, before they are taken off)
              const float2 z = unpack2(add2(fma2(pack2(s[r], s[r + 1]), ks2, lv2), r & 2 ? pack2(m.z, m.w) : pack2(m.x, m.y)));
              const float w0 = exp2_approx(z.x), w1 = exp2_approx(z.y);
              w2[r >> 1] = pack2(w0, w1);
              h[r >> 1] = pack_f16(w0, w1);
              top = __hmax2(top, *reinterpret_cast<const __half2*>(&h[r >> 1]));
            }
#pragma unroll
            for (int g = 0; g < kHalf / 8; ++g)
              sts128(p_at + (((x * (kHalf / 8) + g) ^ (t & 7)) << 4), h[4 * g], h[4 * g + 1], h[4 * g + 2], h[4 * g + 3]);
            // a weight past its range: once more with new maxima (they hold for this tile)
            if (!fresh) break;
            const bool big = __half2float(__hmax(__low2half(top), __high2half(top))) > 32768.f;
            if (!meet_any(x, big || !ok)) break;
            fresh = false;
          }
          if (!ok) break;
          fence_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive(&ctrl->pfull[n & 1]);
#pragma unroll
          for (int r = 0; r < kHalf / 2; ++r) l2[r] = fma2(w2[r], iv2, l2[r]);
        }
        if (lane == 0) {
          if (idle) arrive(&ctrl->pfull[n & 1]);
          arrive(&ctrl->look_empty[n % kMetas]);
        }
      }
      if (!ok) break;                    // all four warps alike
      float l[kHalf];
#pragma unroll
      for (int r = 0; r < kHalf / 2; ++r) {
        const float2 v = unpack2(l2[r]);
        l[2 * r] = v.x;
        l[2 * r + 1] = v.y;
      }
      most[w][x * kHalf + lane] = reduce_across(l, lane, [](float p, float q) { return p + q; });
      meet_any(x, false);
      const bool part = u.part >= 0;
      constexpr int kPart = kRows * (D + 2);                  // floats of a part: (M, l) by row, then O
      float* pd = a.part + static_cast<size_t>(max(u.part, 0)) * kPart;
      const size_t row_at = static_cast<size_t>(u.q) * a.q_heads + static_cast<size_t>(u.head) * a.group;
      const int row = x * kHalf + t, rows = min(a.group - x * kHalf, kHalf);   // rows of this half
      auto write_lse = [&](float m2, float sum) {
        if (a.lse != nullptr) a.lse[row_at + row] = sum == 0.f ? -inf : (m2 - kBoost + log2f(sum)) * 0.69314718055994530942f;
      };
      if (t < kHalf) {
        const float sum = most[0][row] + most[1][row] + (most[2][row] + most[3][row]);
        by[t] = sum == 0.f ? 0.f : 1.f / sum;
        if (part) __stcg(reinterpret_cast<float2*>(pd) + row, make_float2(-minus_max[t], sum));
        else if (t < rows) write_lse(-minus_max[t], sum);
      }
      ok = wait(&ctrl->ofull, un);
      if (meet_any(x, !ok)) break;
      tc_fence_after();
      uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (row_at + x * kHalf) * D + t;
      float* po = pd + 2 * kRows + x * kHalf * D + t;
#pragma unroll 1
      for (int q = 0; 16 * q < rows; ++q) {
        float v[16];
        tmem_ld32x16(o_at + 16 * q, v);
        tmem_wait_ld_tied(v);
        if (t >= D) {
        } else if (part) {
#pragma unroll
          for (int e = 0; e < 16; ++e) __stcg(po + (16 * q + e) * D, v[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const int r = 16 * q + e;
            const uint32_t two = kv_pack16(v[e] * by[r], v[e + 1] * by[r + 1], a.bf16);
            if (r < rows) out[r * D] = static_cast<uint16_t>(two);
            if (r + 1 < rows) out[(r + 1) * D] = static_cast<uint16_t>(two >> 16);
          }
        }
      }
      if (part) {
        // the last of the unit's CTAs joins the pieces in their order
        __threadfence();
        meet_any(x, false);
        if (t == 0) {
          int* count = a.counters + 2 * u.c0 + x;
          const bool last = atomicAdd(count, 1) == u.c1 - u.c0;
          if (last) *count = 0;
          ctrl->last[x] = last;
        }
        meet_any(x, false);
        if (*reinterpret_cast<volatile int*>(&ctrl->last[x])) {
          __threadfence();
          auto part_of = [&](int cta) { return a.part + static_cast<size_t>(2 * cta + (cta == u.c0 ? 1 : 0)) * kPart; };
          if (t < rows) {
            float top = kMinusHuge, sum = 0.f;
            for (int cta = u.c0; cta <= u.c1; ++cta) {
              const float2 v = __ldcg(reinterpret_cast<const float2*>(part_of(cta)) + row);
              const float next = fmaxf(top, v.x);
              sum = sum * exp2_approx(top - next) + v.y * exp2_approx(v.x - next);
              top = next;
            }
            most[0][row] = top;
            by[t] = sum == 0.f ? 0.f : 1.f / sum;
            write_lse(top, sum);
          }
          meet_any(x, false);
          if (t < D) {
#pragma unroll 1
            for (int q = 0; 16 * q < rows; ++q) {
              float v[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = 0.f;
#pragma unroll 1
              for (int cta = u.c0; cta <= u.c1; ++cta) {
                const float* src = part_of(cta);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const int r = x * kHalf + 16 * q + e;
                  v[e] = fmaf(__ldcg(src + 2 * kRows + r * D + t), exp2_approx(__ldcg(src + 2 * r) - most[0][r]), v[e]);
                }
              }
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (16 * q + e < rows)
                  out[static_cast<size_t>(16 * q + e) * D] = static_cast<uint16_t>(kv_pack16(v[e] * by[16 * q + e], 0.f, a.bf16));
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(&ctrl->uempty[us]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t init_list() {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kv_list_kernel<D>), cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Shape<D>::kBytes);
}

}  // namespace

size_t kv_list_part_floats(int num_sms) { return static_cast<size_t>(2) * num_sms * kRows * (128 + 2); }
int kv_list_counters(int num_sms) { return 2 * num_sms; }

cudaError_t kv_list_init() {
  const cudaError_t e = init_list<128>();
  return e != cudaSuccess ? e : init_list<64>();
}

cudaError_t launch_kv_list(const AttnParams& a, int num_sms, cudaStream_t stream) {
  ListParams p;
  p.a = a;
  p.tiles = (a.k + kKeys - 1) / kKeys;
  count_launches(1);
  return a.dim == 128 ? launch_overlapped(kv_list_kernel<128>, num_sms, kThreads, Shape<128>::kBytes, stream, p)
                      : launch_overlapped(kv_list_kernel<64>, num_sms, kThreads, Shape<64>::kBytes, stream, p);
}

}  // namespace ltk

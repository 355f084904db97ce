// kv_internal.cuh -- paged 8-bit key/value cache: layout, batch description and
// device helpers shared by the append and attention kernels.
//
// Cache of one layer: codes [num_pages, heads, page, dim] (e4m3), one fp32 scale
// for each (page, head); a held value is code * scale.  The pages of sequence b
// are page_table[b, 0..]; its token at position p lies in page
// page_table[b, p / page], row p % page.  Offsets into the cache are 64-bit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ltk_internal.cuh"

namespace ltk {

// Range of a block's scale exponent: scale = 2^e, kKvMinExp <= e <= kKvMaxExp.
// Within it the ratio of two blocks' scales stays far inside fp32 (see the
// attention kernels, which fold log2(v_scale) into the exponent of a weight).
constexpr int kKvMinExp = -40;
constexpr int kKvMaxExp = 40;
// A block whose value scale is 0 holds zeros.  Its keys count like any others: their weights are
// made as if the scale were this one, the smallest that append writes, so that they push no other
// weight out of its range, and meet zeros instead of the block's codes.
constexpr float kKvLeastScale = 0x1p-40f;
// Positions are below this, and no window is larger (it would hide nothing more), so that what is
// made of a row's position, a window and a tile near it stays within 32 bits.
constexpr int kKvMaxPos = 0x7FFFFC00;
constexpr int kDevArg = 1;               // device status: an index outside its table

struct KvCache {
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
  long long num_pages;
  int heads;                             // KV heads
  int page;                              // tokens per page: 16, 32, 64 or 128
  int page_log2;
};

struct KvBatch {
  const int* page_table;                 // [B, width]
  const int* seq_lens;                   // [B] cached tokens, this step's among them
  const int* cu_q;                       // [B + 1] first query (token) of each sequence
  int width;
  int B;
  int N;
  // Attention in two steps (see AttnParams::step): tokens at each sequence's start that are left
  // out, whole pages (null: none), and how far a query's position lies behind the one before: 1, or
  // 0 where every query of a sequence sees all of its keys.
  const int* start;
  int advance;
};

// A load that sees what the kernel before on the stream wrote.  Kernels here start while that one
// still runs (see begin_after_previous), so nothing it writes is read-only for their lifetime, and
// the non-coherent path (ld.global.nc, __ldg) may answer from lines that were read before the wait.
template <class T>
__device__ __forceinline__ T kv_load(const T* p) { return *p; }

// Queries [q0, q0 + nq) of sequence b, the position of its first query, and how many of its
// tokens have a column in the page table.  cu_q is clamped to the batch.  A sequence that is
// longer than its table has queries at positions len and beyond.
// STEPS: one of the two steps of an attention.  With left-out tokens, lengths and positions count from the first one that is not.
struct KvSeq {
  int q0, nq, len, pos0;
  int page0;                             // column of the page table that holds position 0
};
template <bool STEPS = false>
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& bt, const KvCache& c, int b) {
  KvSeq s;
  s.q0 = min(max(kv_load(bt.cu_q + b), 0), bt.N);
  s.nq = min(max(kv_load(bt.cu_q + b + 1), s.q0), bt.N) - s.q0;
  const int start = STEPS && bt.start != nullptr ? kv_load(bt.start + b) : 0;
  const long long room = min(static_cast<long long>(bt.width) << c.page_log2, static_cast<long long>(kKvMaxPos)) - start;
  const int tokens = max(kv_load(bt.seq_lens + b), 0) - start;
  s.len = static_cast<int>(min(static_cast<long long>(tokens), room));
  s.pos0 = tokens - (!STEPS || bt.advance ? s.nq : 1);                  // negative when a sequence is shorter than its queries
  s.page0 = start >> c.page_log2;
  return s;
}

// Sequence of query n: the last b with cu_q[b] <= n.  First looked for where it is
// when every sequence has as many queries (a decode step: one look, no search).
__device__ __forceinline__ int kv_seq_of_query(const KvBatch& bt, int n) {
  const int guess = static_cast<int>(static_cast<long long>(n) * bt.B / bt.N);
  const int at = kv_load(bt.cu_q + guess), next = kv_load(bt.cu_q + guess + 1);
  if (at <= n && n < next) return guess;
  int lo = 0, hi = bt.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (kv_load(bt.cu_q + mid) <= n) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Page of position pos of sequence b; -1, which is no page, past the table.
__device__ __forceinline__ int kv_page(const KvBatch& bt, const KvCache& c, int b, int pos) {
  const int at = pos >> c.page_log2;
  return at < bt.width ? kv_load(bt.page_table + static_cast<size_t>(b) * bt.width + at) : -1;
}

// Four e4m3 codes to four f16 values (exact), in order: lo holds the first two.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// 2^x, one MUFU instruction (2 ulp); 0 for -inf and for results below fp32's normal range.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two packed 16-bit values to fp32.
__device__ __forceinline__ float2 kv_unpack16(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t kv_pack16(float lo, float hi, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A kernel's start overlaps the end of the one before it on the stream: begin_after_previous
// waits until that one is done and its writes can be seen, so a kernel calls it, in every
// thread, before it touches global memory; the next kernel may then start in its turn, as
// soon as every CTA of this one has, and wait at its own.
__device__ __forceinline__ void begin_after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... Params, class... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

struct AppendParams {
  KvCache cache;
  KvBatch batch;
  int dim;
  int bf16;                              // else f16
  const void* k;                         // [N, heads, dim], rows k_stride elements apart
  const void* v;
  long long k_stride, v_stride;
  const float* cos;                      // [table_rows, rot / 2], null: no rotation
  const float* sin;
  int rot;
  int table_rows;
  int interleaved;
  const void* q;                         // [N, q_heads, dim] or null
  long long q_stride;
  int q_heads;
  void* q_out;                           // [N, q_heads, dim] contiguous
  int* status;
};
cudaError_t launch_kv_append(const AppendParams& p, int num_sms, cudaStream_t stream);

struct ReadParams {
  KvCache cache;
  KvBatch batch;                         // cu_q: the rows of each sequence's last tokens
  int dim;
  int bf16;
  const float* cos;                      // [table_rows, rot / 2], null: keys as they are held
  const float* sin;
  int rot;
  int table_rows;
  int interleaved;
  void* k_out;                           // [N, heads, dim] contiguous
  void* v_out;
  int* status;
};
cudaError_t launch_kv_read(const ReadParams& p, int num_sms, cudaStream_t stream);

// What sequences share (k_kv_share.cu): from the page tables to the two batches of an attention in
// two steps.  All arrays are of the workspace.
struct ShareParams {
  KvCache cache;
  KvBatch batch;
  const int* groups;                     // [num_groups + 1] first sequence of each, null: one group of all
  int num_groups;
  int* common;                           // [B] pages in common with the group's first sharing sequence
  int* lead;                             // [num_groups] that sequence
  int* least;                            // [num_groups] pages that all sharing sequences have in common
  int* sharing;                          // [num_groups] how many these are
  int* start;                            // [B] second step: tokens left out
  int* lens;                             // [B] first step: the lead's shared tokens, others 0
  int* cu;                               // [B + 1] first step: all of a group's queries are its lead's
  int* counter;                          // zero between calls
  int* status;
};
cudaError_t launch_kv_share(const ShareParams& p, cudaStream_t stream);
cudaError_t launch_kv_groups(const ShareParams& p, cudaStream_t stream);   // checks the groups only

struct AttnParams {
  KvCache cache;
  KvBatch batch;
  int dim;
  int bf16;
  const void* q;                         // [N, q_heads, dim], rows q_stride elements apart
  long long q_stride;
  int q_heads;
  int group;                             // q_heads / cache.heads
  float scale_log2;                      // softmax scale * log2(e)
  int window;                            // 0: none
  int sinks;
  const int* idx;                        // [N, k] selected positions, or null (dense)
  int k;
  void* out;                             // [N, q_heads, dim]
  float* lse;                            // [N, q_heads] or null
  // Attention in two steps, over keys that sequences share and over each one's own: the first
  // leaves its results here in fp32, the second joins them with its own.
  int step;                              // 0: all at once, 1: the first, 2: the second
  float* mid;                            // [N, q_heads, dim]
  float* mid_lse;                        // [N, q_heads], base 2
  int units;                             // sequences that have queries, for the choice of kernel
  double share;                          // of the tokens that a table has room for: how long sequences are taken to be
  float* part;                           // workspace: partial results
  int* counters;                         // workspace: zero between calls
  int* status;
};

// First step, tensor-core tiles: a unit whose key tiles several CTAs hold is not joined by the last of them, but by a
// kernel of its own, from this, by the first of its CTAs.
struct KvPiece {
  int last;                              // the last of its CTAs; -1: no such unit begins here
  int rows, row0, q0, head;
};

// What turns a row's sum over values into its result: result = own * (weighted sum) + mid * (the
// first step's result).  m2, sum: base-2 maximum and sum of weights; at: the row's place.
struct RowEnd {
  float own, mid;
  float lse2;                            // base-2 logarithm of the sum of exponentials
};
__device__ __forceinline__ RowEnd row_end(float before, bool joined, float m2, float sum);
__device__ __forceinline__ RowEnd row_end(const AttnParams& p, size_t at, bool joined, float m2, float sum) {
  return row_end(joined ? kv_load(p.mid_lse + at) : 0.f, joined, m2, sum);
}
// before: the first step's logarithm
__device__ __forceinline__ RowEnd row_end(float before, bool joined, float m2, float sum) {
  RowEnd e;
  e.own = sum == 0.f ? 0.f : 1.f / sum;
  e.lse2 = sum == 0.f ? -__int_as_float(0x7F800000) : m2 + log2f(sum);
  e.mid = 0.f;
  if (joined) {
    const float top = fmaxf(before, e.lse2);
    if (top > -__int_as_float(0x7F800000)) {
      const float a = exp2_approx(before - top), b = exp2_approx(e.lse2 - top), by = 1.f / (a + b);
      e.mid = a * by;
      e.own *= b * by;
      e.lse2 = top + log2f(a + b);
    }
  }
  return e;
}

// Attention for few rows per KV head (k_kv_rows.cu).
constexpr int kRowsPerUnit = 16;
size_t kv_rows_part_floats(int num_sms);   // workspace floats
int kv_rows_counters(int num_sms);
cudaError_t kv_rows_init();                // kernel attributes on the current device
cudaError_t launch_kv_rows(const AttnParams& p, int max_q, int num_sms, cudaStream_t stream);

// Attention for many rows per KV head, on the tensor cores (k_kv_tile.cu).
size_t kv_tile_part_floats(int num_sms);   // and behind them the pieces
int kv_tile_counters(int num_sms);
cudaError_t kv_tile_init();
bool kv_tile_pairs(const AttnParams& p, int max_q, int num_sms);   // whether its units are pairs of row tiles
cudaError_t launch_kv_tile(const AttnParams& p, int max_q, int num_sms, cudaStream_t stream);

// Attention over listed keys for up to kListRows rows per KV head, on the tensor cores
// (k_kv_list.cu).
constexpr int kListRows = 64;
size_t kv_list_part_floats(int num_sms);
int kv_list_counters(int num_sms);
cudaError_t kv_list_init();
cudaError_t launch_kv_list(const AttnParams& p, int num_sms, cudaStream_t stream);
}  // namespace ltk

struct ltk_kv {
  ltk::KvCache cache;
  int dim = 0;
  int engine = 0;
  int device = 0;
  int num_sms = 0;
  float* part = nullptr;
  int* counters = nullptr;
  int num_counters = 0;
  int* status = nullptr;
};

namespace ltk {

// What the entry points share (kv_api.cu).
ltk_status kv_cuda_fail(cudaError_t e, const char* what);
ltk_status kv_check_batch(const ltk_kv* h, const ltk_kv_batch* b);
// Checks of an attention call and its parameters, all but the results' places; LTK_OK with
// p->batch.N 0: nothing to do.
ltk_status kv_attention_params(const ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* q, long long q_stride,
                               int q_heads, int max_q, float scale, AttnParams* p);
// About how long the chosen kernel takes, in us.
double kv_attention_us(const ltk_kv* h, const AttnParams& p, int max_q);
// Chooses the kernel and starts it.
cudaError_t kv_launch_attention(const ltk_kv* h, const AttnParams& p, int max_q, cudaStream_t stream);
inline bool kv_aligned(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool kv_aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline KvBatch kv_batch_of(const ltk_kv_batch* b) {
  return KvBatch{b->page_table, b->seq_lens, b->cu_q, b->table_width, b->B, b->N, nullptr, 1};
}

}  // namespace ltk

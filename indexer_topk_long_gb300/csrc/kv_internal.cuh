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
};

// A load that sees what the kernel before on the stream wrote.  Kernels here start while that one
// still runs (see begin_after_previous), so nothing it writes is read-only for their lifetime, and
// the non-coherent path (ld.global.nc, __ldg) may answer from lines that were read before the wait.
template <class T>
__device__ __forceinline__ T kv_load(const T* p) { return *p; }

// Queries [q0, q0 + nq) of sequence b, the position of its first query, and how many of its
// tokens have a column in the page table.  cu_q is clamped to the batch.  A sequence that is
// longer than its table has queries at positions len and beyond.
struct KvSeq {
  int q0, nq, len, pos0;
};
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& bt, const KvCache& c, int b) {
  KvSeq s;
  s.q0 = min(max(kv_load(bt.cu_q + b), 0), bt.N);
  s.nq = min(max(kv_load(bt.cu_q + b + 1), s.q0), bt.N) - s.q0;
  const long long room = min(static_cast<long long>(bt.width) << c.page_log2, static_cast<long long>(kKvMaxPos));
  const int tokens = max(kv_load(bt.seq_lens + b), 0);
  s.len = static_cast<int>(min(static_cast<long long>(tokens), room));
  s.pos0 = tokens - s.nq;                // negative when a sequence is shorter than its queries
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
  float* part;                           // workspace: partial results
  int* counters;                         // workspace: zero between calls
  int* status;
};

// Attention for few rows per KV head (k_kv_rows.cu).
constexpr int kRowsPerUnit = 16;
size_t kv_rows_part_floats(int num_sms);   // workspace floats
int kv_rows_counters(int num_sms);
cudaError_t kv_rows_init();                // kernel attributes on the current device
cudaError_t launch_kv_rows(const AttnParams& p, int max_q, int num_sms, cudaStream_t stream);

// Attention for many rows per KV head, on the tensor cores (k_kv_tile.cu).
size_t kv_tile_part_floats(int num_sms);
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

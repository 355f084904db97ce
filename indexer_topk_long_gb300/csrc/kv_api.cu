// kv_api.cu -- C ABI of the paged 8-bit key/value cache: validation on the host,
// the handle with its workspace, and the launches of append and attention.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>

#include "kv_internal.cuh"

using namespace ltk;

namespace ltk {

ltk_status kv_cuda_fail(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return LTK_OK;
  if (std::getenv("LTK_DEBUG")) std::fprintf(stderr, "ltk: %s: %s\n", what, cudaGetErrorString(e));
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? LTK_ERR_NOMEM : LTK_ERR_CUDA;
}

ltk_status kv_check_batch(const ltk_kv* h, const ltk_kv_batch* b) {
  if (h == nullptr || b == nullptr) return LTK_ERR_ARG;
  if (b->B < 0 || b->N < 0 || b->table_width < 0) return LTK_ERR_ARG;
  if (b->N == 0) return LTK_OK;
  if (b->B == 0 || b->table_width == 0) return LTK_ERR_ARG;
  if (static_cast<long long>(b->table_width) * h->cache.page > INT_MAX) return LTK_ERR_ARG;   // positions are int32
  if (!kv_aligned4(b->page_table) || !kv_aligned4(b->seq_lens) || !kv_aligned4(b->cu_q)) return LTK_ERR_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return LTK_ERR_ARG;
  return LTK_OK;
}

}  // namespace ltk

namespace {

// Rows of 16-bit elements, each row a whole number of 16-byte pieces.
bool rows_ok(const void* p, long long stride, int heads, int dim) {
  return kv_aligned(p) && stride >= static_cast<long long>(heads) * dim && stride % 8 == 0;
}

// Which kernel.  The one for few rows goes over a head's keys once for every 16 rows; the tile
// kernels once for 64 (narrow, listed), 128 or 256 (pairs), but each of their units, and the
// kernel as a whole, takes longer to begin and end.  Both are estimated in microseconds of one
// SM, T tiles of 128 keys a unit, and shared out over the SMs:
//   few rows    2.0 + 0.75 T for 16 rows (D = 64: 1.4 + 0.51 T)
//   listed      5.0 + 0.96 T (4.5 + 0.94 T), and 7 for the kernel
//   dense       3.0 + 1.8 T for 64 or 128 rows, 8 + 1.8 T for a pair (D = 64: 1.4 T), and 12
//               for the kernel
// For instance (D = 128), by few rows and by tiles: listed, k = 2048, one KV head of 64 rows, 32
// queries 26 and 27 us, 128 queries 57 and 35, 4096 queries 1398 and 542; of 32 rows, 64 queries
// 26 and 27, 4096 queries 706 and 514; dense, a window of 1024 over 24 ragged chunks (D = 64) 72
// and 41, chunks of 2048 queries ten times as long by few rows.
// How long sequences are is only known on the device: 0.6 of the page table is assumed.  Over
// 130 dense batches (1 to 128 sequences, even and ragged, 98 to 32768 tokens) what this takes
// is 2% more on average than the better of the two.
// The first step of a shared attention has few and long units, whose keys many CTAs read in a row: 64 rows
// take 1.16 T there (D = 64: 0.77 T), 128 rows 1.5 T (1.1 T), and as there is a step after it in any case, all but
// 2 of what it takes to begin and end overlaps.  Both steps, the first by few rows and by tiles (us, 32 heads on 8):
// 32 rows of 32768 tokens 70 and 57, of 131072 139 and 104; 4 groups of 48 rows, 8192 tokens 80 and 58, 131072 730
// and 292 (D = 64: 55 and 45, 418 and 203); of 20 rows, 8192 tokens 57 and 55 (42 and 45).
struct Estimate {
  bool by_rows;
  double us;                             // of the GPU
};
Estimate kv_estimate(const AttnParams& p, int max_q, int num_sms) {
  const double rows = static_cast<double>(p.group) * (p.idx != nullptr ? 1 : max_q);
  double keys = p.k;
  if (p.idx == nullptr) {
    keys = static_cast<double>(p.batch.width) * p.cache.page * p.share;
    if (p.window > 0) keys = std::min(keys, static_cast<double>(p.window) + p.sinks + max_q);
  }
  const double T = std::ceil(keys / 128.0);
  // units of r rows: every query its own (listed), or every sequence's queries, at least one
  auto units = [&](double r) {
    if (p.idx != nullptr) return p.batch.N * std::ceil(p.group / r);
    return std::max<double>(p.units, static_cast<double>(p.batch.N) * p.group / r + 0.5 * p.units);
  };
  const bool wide = p.dim == 128;
  const double by_rows = units(16) * (wide ? 2.0 + 0.75 * T : 1.4 + 0.51 * T);
  if (rows <= kRowsPerUnit) return {true, p.cache.heads * by_rows / num_sms};
  double by_tiles, start;
  if (p.idx != nullptr && p.group <= kListRows) {
    by_tiles = units(64) * (wide ? 5.0 + 0.96 * T : 4.5 + 0.94 * T);
    start = 7.0;
  } else {
    const bool pair = p.idx == nullptr && kv_tile_pairs(p, max_q, num_sms);
    const bool first = p.step == 1 && !pair;
    const double tile = !first ? (wide ? 1.8 : 1.4) : rows <= 64 ? (wide ? 1.16 : 0.77) : (wide ? 1.5 : 1.1);
    by_tiles = units(pair ? 256 : rows <= 64 ? 64 : 128) * ((pair ? 8.0 : 3.0) + tile * T);
    start = p.step == 1 ? 2.0 : 12.0;
  }
  if (p.cache.heads * (by_rows - by_tiles) <= start * num_sms) return {true, p.cache.heads * by_rows / num_sms};
  return {false, p.cache.heads * by_tiles / num_sms + start};
}

}  // namespace

namespace ltk {

ltk_status kv_attention_params(const ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* q, long long q_stride,
                               int q_heads, int max_q, float scale, AttnParams* p) {
  const ltk_status s = kv_check_batch(h, batch);
  if (s != LTK_OK) return s;
  if (dtype != LTK_BF16 && dtype != LTK_F16) return LTK_ERR_ARG;
  if (q_heads < 1 || q_heads % h->cache.heads != 0) return LTK_ERR_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return LTK_ERR_ARG;
  if (max_q < 0) return LTK_ERR_ARG;
  if (q_heads > (1 << 20) || static_cast<long long>(batch->N) * (q_heads / h->cache.heads) > INT_MAX / 2)
    return LTK_ERR_UNSUPPORTED;
  *p = AttnParams{};
  if (batch->N == 0) return LTK_OK;
  if (!rows_ok(q, q_stride, q_heads, h->dim)) return LTK_ERR_ARG;
  p->cache = h->cache;
  p->batch = kv_batch_of(batch);
  p->dim = h->dim;
  p->bf16 = dtype == LTK_BF16;
  p->q = q;
  p->q_stride = q_stride;
  p->q_heads = q_heads;
  p->group = q_heads / h->cache.heads;
  p->scale_log2 = scale * 1.44269504088896340736f;
  p->units = batch->B;
  p->share = 0.6;
  p->part = h->part;
  p->counters = h->counters;
  p->status = h->status;
  return LTK_OK;
}

double kv_attention_us(const ltk_kv* h, const AttnParams& p, int max_q) {
  return kv_estimate(p, max_q > 0 ? max_q : p.batch.N, h->num_sms).us;
}

cudaError_t kv_launch_attention(const ltk_kv* h, const AttnParams& p, int max_q, cudaStream_t stream) {
  const int most_q = max_q > 0 ? max_q : p.batch.N;
  const bool by_rows = h->engine == 0 ? kv_estimate(p, most_q, h->num_sms).by_rows : h->engine == 1;
  if (by_rows) return launch_kv_rows(p, most_q, h->num_sms, stream);
  return p.idx != nullptr && p.group <= kListRows ? launch_kv_list(p, h->num_sms, stream)
                                                  : launch_kv_tile(p, most_q, h->num_sms, stream);
}

}  // namespace ltk

extern "C" {

ltk_status ltk_kv_create(const ltk_kv_config* cfg, ltk_kv** out) {
  if (out == nullptr) return LTK_ERR_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->num_pages < 1 || cfg->heads < 1) return LTK_ERR_ARG;
  if (cfg->num_pages > INT_MAX || cfg->heads > 65535) return LTK_ERR_ARG;
  if (cfg->engine < 0 || cfg->engine > 2) return LTK_ERR_ARG;
  if (cfg->page != 16 && cfg->page != 32 && cfg->page != 64 && cfg->page != 128) return LTK_ERR_UNSUPPORTED;
  // a code row's number is 32 bits in the kernels (more rows than that do not fit the device)
  if (cfg->num_pages * cfg->heads > 0xFFFFFFFEll / cfg->page) return LTK_ERR_UNSUPPORTED;
  if (cfg->dim != 64 && cfg->dim != 128) return LTK_ERR_UNSUPPORTED;
  if (!kv_aligned(cfg->k_codes) || !kv_aligned(cfg->v_codes)) return LTK_ERR_ARG;
  if (!kv_aligned(cfg->k_scale) || !kv_aligned(cfg->v_scale)) return LTK_ERR_ARG;
  ltk_kv* h = new (std::nothrow) ltk_kv();
  if (h == nullptr) return LTK_ERR_NOMEM;
  h->cache.k_codes = static_cast<uint8_t*>(cfg->k_codes);
  h->cache.v_codes = static_cast<uint8_t*>(cfg->v_codes);
  h->cache.k_scale = cfg->k_scale;
  h->cache.v_scale = cfg->v_scale;
  h->cache.num_pages = cfg->num_pages;
  h->cache.heads = cfg->heads;
  h->cache.page = cfg->page;
  h->cache.page_log2 = cfg->page == 16 ? 4 : cfg->page == 32 ? 5 : cfg->page == 64 ? 6 : 7;
  h->dim = cfg->dim;
  h->engine = cfg->engine;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  const size_t part_floats = std::max({kv_rows_part_floats(h->num_sms), kv_tile_part_floats(h->num_sms), kv_list_part_floats(h->num_sms)});
  h->num_counters = std::max({kv_rows_counters(h->num_sms), kv_tile_counters(h->num_sms), kv_list_counters(h->num_sms)});
  const size_t counters = static_cast<size_t>(h->num_counters) * 4;
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->part), part_floats * 4);
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->counters), counters);
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->status), 4);
  if (e == cudaSuccess) e = cudaMemset(h->counters, 0, counters);
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, 4);
  if (e == cudaSuccess) e = kv_rows_init();
  if (e == cudaSuccess) e = kv_tile_init();
  if (e == cudaSuccess) e = kv_list_init();
  if (e == cudaSuccess) e = cudaDeviceSynchronize();   // the workspace is zero for calls on any stream
  if (e != cudaSuccess) {
    const ltk_status s = kv_cuda_fail(e, "ltk_kv_create");
    ltk_kv_destroy(h);
    return s;
  }
  *out = h;
  return LTK_OK;
}

void ltk_kv_destroy(ltk_kv* h) {
  if (h == nullptr) return;
  cudaDeviceSynchronize();
  cudaFree(h->part);
  cudaFree(h->counters);
  cudaFree(h->status);
  delete h;
}

ltk_status ltk_kv_append(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* k, long long k_stride,
                         const void* v, long long v_stride, const float* cos_table, const float* sin_table,
                         int table_rows, int rot, int interleaved, const void* q, long long q_stride, int q_heads,
                         void* q_out, void* stream) {
  const ltk_status s = kv_check_batch(h, batch);
  if (s != LTK_OK) return s;
  if (dtype != LTK_BF16 && dtype != LTK_F16) return LTK_ERR_ARG;
  if ((cos_table == nullptr) != (sin_table == nullptr)) return LTK_ERR_ARG;
  if (interleaved != 0 && interleaved != 1) return LTK_ERR_ARG;
  if (cos_table != nullptr) {
    if (table_rows < 1 || rot < 16 || rot > h->dim) return LTK_ERR_ARG;
    if (rot % 16 != 0) return LTK_ERR_UNSUPPORTED;
    if (!kv_aligned(cos_table) || !kv_aligned(sin_table)) return LTK_ERR_ARG;
  }
  if ((q == nullptr) != (q_out == nullptr)) return LTK_ERR_ARG;
  if (q != nullptr && q_heads < 1) return LTK_ERR_ARG;
  if (batch->N == 0) return LTK_OK;
  if (!rows_ok(k, k_stride, h->cache.heads, h->dim) || !rows_ok(v, v_stride, h->cache.heads, h->dim)) return LTK_ERR_ARG;
  if (q != nullptr && (!rows_ok(q, q_stride, q_heads, h->dim) || !kv_aligned(q_out))) return LTK_ERR_ARG;
  AppendParams p{};
  p.cache = h->cache;
  p.batch = kv_batch_of(batch);
  p.dim = h->dim;
  p.bf16 = dtype == LTK_BF16;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.cos = cos_table;
  p.sin = sin_table;
  p.rot = cos_table != nullptr ? rot : 0;
  p.table_rows = table_rows;
  p.interleaved = interleaved;
  p.q = q;
  p.q_stride = q_stride;
  p.q_heads = q_heads;
  p.q_out = q_out;
  p.status = h->status;
  const cudaError_t e = launch_kv_append(p, h->num_sms, static_cast<cudaStream_t>(stream));
  if (e == cudaErrorInvalidConfiguration) return LTK_ERR_UNSUPPORTED;
  return kv_cuda_fail(e, "ltk_kv_append");
}

static ltk_status kv_attend(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* q, long long q_stride,
                            int q_heads, int max_q, float scale, int window, int sinks, const int* idx, int k,
                            void* out, float* lse, void* stream) {
  AttnParams p;
  const ltk_status s = kv_attention_params(h, batch, dtype, q, q_stride, q_heads, max_q, scale, &p);
  if (s != LTK_OK) return s;
  if (window < 0 || sinks < 0) return LTK_ERR_ARG;
  if (batch->N == 0) return LTK_OK;
  if (!kv_aligned(out)) return LTK_ERR_ARG;
  if (lse != nullptr && !kv_aligned4(lse)) return LTK_ERR_ARG;
  p.window = std::min(window, kKvMaxPos);
  p.sinks = sinks;
  p.idx = idx;
  p.k = k;
  p.out = out;
  p.lse = lse;
  return kv_cuda_fail(kv_launch_attention(h, p, max_q, static_cast<cudaStream_t>(stream)), "kv attention");
}

ltk_status ltk_kv_attention(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* q, long long q_stride,
                            int q_heads, int max_q, float scale, int window, int sinks, void* out, float* lse,
                            void* stream) {
  return kv_attend(h, batch, dtype, q, q_stride, q_heads, max_q, scale, window, sinks, nullptr, 0, out, lse, stream);
}

ltk_status ltk_kv_attention_selected(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* q,
                                     long long q_stride, int q_heads, const int* idx, int k, float scale, void* out,
                                     float* lse, void* stream) {
  if (k < 1 || k > (1 << 24)) return LTK_ERR_ARG;
  if (batch != nullptr && batch->N > 0 && !kv_aligned4(idx)) return LTK_ERR_ARG;
  return kv_attend(h, batch, dtype, q, q_stride, q_heads, 1, scale, 0, 0, idx, k, out, lse, stream);
}

ltk_status ltk_kv_status(ltk_kv* h, int* device_status, void* stream) {
  if (h == nullptr || device_status == nullptr) return LTK_ERR_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int value = 0;
  cudaError_t e = cudaMemcpyAsync(&value, h->status, 4, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->status, 0, 4, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  // A call that gave up half way may have left its counters, and the status holds the first error
  // only, so any error clears them: on the stream, ahead of the calls that come after.
  if (e == cudaSuccess && value != LTK_OK) {
    e = cudaMemsetAsync(h->counters, 0, static_cast<size_t>(h->num_counters) * 4, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (e != cudaSuccess) return kv_cuda_fail(e, "ltk_kv_status");
  *device_status = value;
  return LTK_OK;
}

}  // extern "C"

// kv_share_api.cu -- C ABI of what is shared and read back from the paged cache: attention of groups
// of sequences that begin with the same pages, and tokens back in 16 bits.
#include <algorithm>
#include <climits>

#include "kv_internal.cuh"

using namespace ltk;

namespace {

constexpr unsigned long long kPiece = 256;
unsigned long long rounded(unsigned long long n) { return (n + kPiece - 1) / kPiece * kPiece; }

// The workspace of a call, in order; with base 0 its size.
struct Space {
  float *mid, *mid_lse;
  int *common, *lead, *least, *sharing, *start, *lens, *cu;
  unsigned long long bytes;
};
Space space_of(char* base, unsigned long long B, unsigned long long N, unsigned long long q_heads, unsigned long long dim) {
  Space s{};
  auto take = [&](unsigned long long elements) {
    void* at = base == nullptr ? nullptr : base + s.bytes;
    s.bytes += rounded(4 * elements);
    return at;
  };
  s.mid = static_cast<float*>(take(N * q_heads * dim));
  s.mid_lse = static_cast<float*>(take(N * q_heads));
  s.common = static_cast<int*>(take(B));
  s.lead = static_cast<int*>(take(B));
  s.least = static_cast<int*>(take(B));
  s.sharing = static_cast<int*>(take(B));
  s.start = static_cast<int*>(take(B));
  s.lens = static_cast<int*>(take(B));
  s.cu = static_cast<int*>(take(B + 1));
  return s;
}

}  // namespace

extern "C" {

ltk_status ltk_kv_shared_bytes(const ltk_kv* h, int B, int N, int q_heads, unsigned long long* bytes) {
  if (h == nullptr || bytes == nullptr || B < 0 || N < 0 || q_heads < 1) return LTK_ERR_ARG;
  if (q_heads > (1 << 20)) return LTK_ERR_UNSUPPORTED;
  *bytes = space_of(nullptr, B, N, q_heads, h->dim).bytes;
  return LTK_OK;
}

ltk_status ltk_kv_attention_shared(ltk_kv* h, const ltk_kv_batch* batch, const int* groups, int num_groups, int dtype,
                                   const void* q, long long q_stride, int q_heads, int max_q, float scale, void* out,
                                   float* lse, void* workspace, unsigned long long workspace_bytes, void* stream) {
  AttnParams p;
  ltk_status s = kv_attention_params(h, batch, dtype, q, q_stride, q_heads, max_q, scale, &p);
  if (s != LTK_OK) return s;
  if (batch->N == 0) return LTK_OK;
  if (groups != nullptr && (!kv_aligned4(groups) || num_groups < 1 || num_groups > batch->B)) return LTK_ERR_ARG;
  if (!kv_aligned(out) || (lse != nullptr && !kv_aligned4(lse)) || !kv_aligned(workspace)) return LTK_ERR_ARG;
  const Space w = space_of(static_cast<char*>(workspace), batch->B, batch->N, q_heads, h->dim);
  if (workspace_bytes < w.bytes) return LTK_ERR_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int G = groups != nullptr ? num_groups : 1;
  const int mean_q = static_cast<int>((static_cast<long long>(batch->N) + G - 1) / G);
  const ShareParams share{p.cache, p.batch, groups, G, w.common, w.lead, w.least, w.sharing, w.start, w.lens, w.cu, h->counters, h->status};
  p.out = out;
  p.lse = lse;
  AttnParams first = p;
  first.batch.advance = 0;
  first.units = G;
  first.step = 1;
  first.mid = w.mid;
  first.mid_lse = w.mid_lse;
  AttnParams second = p;
  second.batch.start = w.start;
  second.step = 2;
  second.mid = w.mid;
  second.mid_lse = w.mid_lse;
  // Two steps cost two launches more, the way through memory between them and units that begin and end twice, 20 us in
  // all, which little work does not repay, nor many rows a sequence: its own rows fill the tiles then, and L2 serves what
  // sequences share.  Four fifths of the tokens are taken to be shared.  In one step and in two (us): 4 sequences of 1040
  // tokens, 8 heads of 64, 9 and 17; 47 of up to 16700 in 6 groups, 14 query heads of 64 on 2, 30 and 44; 16 x 226
  // queries behind 8192 tokens, 32 heads of 128 on 8, 443 and 513; 128 sequences of 33000 tokens 1008 and 108.  Over
  // 70 batches (2 to 121 sequences in 1 to 5 groups, prompts of 544 to 241270 tokens) what this and the choice of the first
  // step's kernel take is 1.5% more on average than the best of the three, and more than 10% in three of them.
  first.share = 0.8 * p.share;
  second.share = 0.2 * p.share;
  if (h->engine == 0 && kv_attention_us(h, p, max_q) <= kv_attention_us(h, first, mean_q) + kv_attention_us(h, second, max_q) + 20.0) {
    cudaError_t e = groups != nullptr ? launch_kv_groups(share, st) : cudaSuccess;
    if (e == cudaSuccess) e = kv_launch_attention(h, p, max_q, st);
    return kv_cuda_fail(e, "kv shared attention");
  }
  cudaError_t e = launch_kv_share(share, st);
  if (e != cudaSuccess) return kv_cuda_fail(e, "kv shared attention");
  // all of a group's queries over what it shares, without a mask
  first.batch.seq_lens = w.lens;
  first.batch.cu_q = w.cu;
  e = kv_launch_attention(h, first, mean_q, st);
  if (e != cudaSuccess) return kv_cuda_fail(e, "kv shared attention");
  // each sequence's rest, joined with that
  return kv_cuda_fail(kv_launch_attention(h, second, max_q, st), "kv shared attention");
}

ltk_status ltk_kv_read(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const float* cos_table, const float* sin_table,
                       int table_rows, int rot, int interleaved, void* k_out, void* v_out, void* stream) {
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
  if (batch->N == 0) return LTK_OK;
  if (!kv_aligned(k_out) || !kv_aligned(v_out)) return LTK_ERR_ARG;
  ReadParams p{};
  p.cache = h->cache;
  p.batch = kv_batch_of(batch);
  p.dim = h->dim;
  p.bf16 = dtype == LTK_BF16;
  p.cos = cos_table;
  p.sin = sin_table;
  p.rot = cos_table != nullptr ? rot : 0;
  p.table_rows = table_rows;
  p.interleaved = interleaved;
  p.k_out = k_out;
  p.v_out = v_out;
  p.status = h->status;
  return kv_cuda_fail(launch_kv_read(p, h->num_sms, static_cast<cudaStream_t>(stream)), "ltk_kv_read");
}

}  // extern "C"

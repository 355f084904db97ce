// k_kv_read.cu -- tokens of the paged e4m3 cache back to 16 bits.
//
//   v = code * vs;  k = code * ks, and with a rotation table, for each rotated pair (i, j),
//   k[i] = x[i] cos + x[j] sin,  k[j] = x[j] cos - x[i] sin       (append's turn, taken back)
//
// in fp32, rounded once at the end.  A CTA takes a run of tokens: it first looks up where each of
// them lies, then its threads take 8 elements at a time in the order of the output, which is
// contiguous.
//
// Bound by memory: 3 bytes an element of k and v.  131072 tokens of 8 KV heads of 128: 126 us, 95% of the
// copy rate; 24 ragged runs of 200 to 9000 tokens, 2 heads of 64, turned back: 7 us, of which 3.7 are bytes.
#include "kv_internal.cuh"

namespace ltk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 256;          // of a CTA
constexpr int kUnroll = 4;               // pieces of 8 elements a thread has in flight, of k and v each

struct Place {
  int block;                             // page * heads, -1: no such token, -2: no row of any sequence
  int row;                               // row in the page
  int pos;
};

__device__ __forceinline__ uint2 load8(const uint8_t* p) { return kv_load(reinterpret_cast<const uint2*>(p)); }

// 8 codes to fp32 values; a block whose scale is 0 holds zeros.
__device__ __forceinline__ void values8(const uint2& c, float scale, float (&x)[8]) {
  uint32_t h[4];
  e4m3x4_to_f16(c.x, h[0], h[1]);
  e4m3x4_to_f16(c.y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = kv_unpack16(h[i], false);
    x[2 * i] = scale == 0.f ? 0.f : f.x * scale;
    x[2 * i + 1] = scale == 0.f ? 0.f : f.y * scale;
  }
}
__device__ __forceinline__ uint4 packed8(const float (&x)[8], bool bf16) {
  return make_uint4(kv_pack16(x[0], x[1], bf16), kv_pack16(x[2], x[3], bf16), kv_pack16(x[4], x[5], bf16),
                    kv_pack16(x[6], x[7], bf16));
}

template <int D, bool TURN>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadParams p, const int tokens) {
  constexpr int kPieces = D / 8;         // of a row
  __shared__ Place places[kMaxTokens];
  const int tid = threadIdx.x;
  const int n0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * tokens, static_cast<long long>(p.batch.N)));
  const int count = min(tokens, p.batch.N - n0);
  const KvCache& c = p.cache;
  const float nan = __int_as_float(0x7FC00000);
  begin_after_previous();
  for (int i = tid; i < count; i += kThreads) {
    const int b = kv_seq_of_query(p.batch, n0 + i);
    const KvSeq s = kv_seq(p.batch, c, b);
    Place t{-2, 0, 0};
    if (n0 + i >= s.q0 && n0 + i < s.q0 + s.nq) {
      t.pos = s.pos0 + n0 + i - s.q0;
      const int page = t.pos >= 0 && t.pos < s.len ? kv_page(p.batch, c, b, t.pos) : -1;
      const bool known = page >= 0 && page < c.num_pages && (!TURN || t.pos < p.table_rows);
      t.block = known ? page * c.heads : -1;
      t.row = t.pos & (c.page - 1);
      if (!known) raise_status(p.status, kDevArg);
    }
    places[i] = t;
  }
  __syncthreads();
  const int per_token = c.heads * kPieces, all = count * per_token;
  uint4* k_out = reinterpret_cast<uint4*>(p.k_out) + static_cast<size_t>(n0) * per_token;
  uint4* v_out = reinterpret_cast<uint4*>(p.v_out) + static_cast<size_t>(n0) * per_token;
#pragma unroll 1
  for (int at0 = tid; at0 < all; at0 += kThreads * kUnroll) {
    uint2 kc[kUnroll], vc[kUnroll], other[kUnroll];
    float ks[kUnroll], vs[kUnroll];
    int pos[kUnroll], piece[kUnroll];
    bool on[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = at0 + u * kThreads;
      const int i = at / per_token, rest = at - i * per_token;
      const int head = rest / kPieces;
      piece[u] = rest % kPieces;
      kc[u] = vc[u] = other[u] = make_uint2(0, 0);
      ks[u] = vs[u] = nan;
      pos[u] = -1;
      on[u] = at < all && places[i].block != -2;
      if (on[u] && places[i].block >= 0) {
        const int blk = places[i].block + head;
        const size_t from = (static_cast<size_t>(blk) * c.page + places[i].row) * D + piece[u] * 8;
        kc[u] = load8(c.k_codes + from);
        vc[u] = load8(c.v_codes + from);
        ks[u] = kv_load(c.k_scale + blk);
        vs[u] = kv_load(c.v_scale + blk);
        if (TURN) {
          pos[u] = places[i].pos;
          const int half = p.rot >> 4;   // pieces of a half
          if (!p.interleaved && piece[u] < 2 * half) other[u] = load8(c.k_codes + from + (piece[u] < half ? half : -half) * 8);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!on[u]) continue;
      const int at = at0 + u * kThreads;
      float x[8];
      values8(kc[u], ks[u], x);
      if (TURN && pos[u] >= 0 && piece[u] * 8 < p.rot) {
        const size_t row = static_cast<size_t>(pos[u]) * (p.rot >> 1);
        if (p.interleaved) {
          const float4 cs = kv_load(reinterpret_cast<const float4*>(p.cos + row) + piece[u]);
          const float4 sn = kv_load(reinterpret_cast<const float4*>(p.sin + row) + piece[u]);
          const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * cv[e] + b * sv[e];
            x[2 * e + 1] = b * cv[e] - a * sv[e];
          }
        } else {
          const int half = p.rot >> 4;
          const bool low = piece[u] < half;
          const float4* cp = reinterpret_cast<const float4*>(p.cos + row) + 2 * (low ? piece[u] : piece[u] - half);
          const float4* sp = reinterpret_cast<const float4*>(p.sin + row) + 2 * (low ? piece[u] : piece[u] - half);
          float y[8];
          values8(other[u], ks[u], y);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 cs = kv_load(cp + h), sn = kv_load(sp + h);
            const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * h + e] = x[4 * h + e] * cv[e] + (low ? y[4 * h + e] : -y[4 * h + e]) * sv[e];
          }
        }
      }
      k_out[at] = packed8(x, p.bf16);
      values8(vc[u], vs[u], x);
      v_out[at] = packed8(x, p.bf16);
    }
  }
}

template <int D>
cudaError_t launch_read(const ReadParams& p, int grid, int tokens, cudaStream_t stream) {
  return p.rot > 0 ? launch_overlapped(kv_read_kernel<D, true>, grid, kThreads, 0, stream, p, tokens)
                   : launch_overlapped(kv_read_kernel<D, false>, grid, kThreads, 0, stream, p, tokens);
}

}  // namespace

cudaError_t launch_kv_read(const ReadParams& p, int num_sms, cudaStream_t stream) {
  // A CTA's run of tokens: 16 turns of its threads where there is work for all SMs, fewer where not.
  const long long per_token = static_cast<long long>(p.cache.heads) * (p.dim / 8);
  long long tokens = 16ll * kThreads / per_token;
  tokens = tokens < (p.batch.N + 4 * num_sms - 1) / (4 * num_sms) ? tokens : (p.batch.N + 4 * num_sms - 1) / (4 * num_sms);
  tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
  const int grid = static_cast<int>((p.batch.N + tokens - 1) / tokens);
  count_launches(1);
  return p.dim == 128 ? launch_read<128>(p, grid, static_cast<int>(tokens), stream)
                      : launch_read<64>(p, grid, static_cast<int>(tokens), stream);
}

}  // namespace ltk

// kv_tensor.cuh -- what the attention kernels on the tensor cores share: bounded
// waits, tcgen05 instructions and descriptors, packed fp32 arithmetic, and the
// conversion of query rows to f16.
#pragma once

#include "kv_internal.cuh"

namespace ltk {

constexpr int kTileRows = 128;           // rows of a product
constexpr int kKeys = 128;               // keys of a tile
// Weights are 2^(t - M + kBoost), so that f16 holds those down to 2^-22 of the largest to 11
// bits (2^-21 where M moves by whole powers of two only); M moves once a weight passes 2^kSlack
// times its first place (at most 2^15 in f16).
constexpr float kMinusHuge = -3e38f;     // running maximum of a row that has seen nothing
constexpr float kBoost = 8.f;
constexpr float kSlack = 7.f;

// A row's new running maximum, kBoost below its largest score; where fp32 holds scores to 16 and
// rounding put it too far below for f16 weights, the largest score itself.
__device__ __forceinline__ float below_top(float top, float next) { return top - next > kSlack + kBoost ? top : next; }

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

// Bounded wait of a whole warp, the same answer for all its lanes: false when another role
// gave up or the wait exceeds kWaitLimitNs (then this one gives up: abort flag and status).
// It sleeps from the second look on, since polling takes issue slots from the softmax.
__device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      raise_status(status, kDevTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(0xFFFFFFFFu, lane_wait(bar, parity, abort_flag, status)) != 0;
}

// MMAs are issued by one lane that elect.sync picks.  Behind elect.sync the compiler
// keeps descriptors in uniform registers and an MMA costs four instructions; behind
// `lane == 0` it moved each operand there first, and with busy softmax warps on the
// scheduler a 128-cube took 780 to 2800 cycles to issue instead of 513 to 590.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
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
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of an operand in 128-byte-swizzled rows (8-row atoms 1024 bytes apart).
// Scores' operands have the contraction contiguous (leading offset unused); the value
// operand's rows of 128 bytes hold 64 consecutive d of one key (N contiguous), and its
// 128-byte-wide halves lie `lead` bytes apart along d.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, uint32_t lead) {
  return static_cast<uint64_t>(((saddr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16)) |
         (static_cast<uint64_t>((1024u >> 4) | (1u << 14) | (2u << 29)) << 32);
}
// f16 operands, fp32 result; the second operand with N contiguous when b_mn.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// A row of a ROWS-row operand of queries, by one thread: the row times a power of two that takes its
// largest element to [2^8, 2^9), as f16; returns what turns the products into base-2
// exponents.  The row as it is: where its f16 form goes, copied there before, or at `from` in global memory
// (null: zeros).
template <int D, int ROWS, bool COPIED>
__device__ __forceinline__ float convert_query(const AttnParams& a, uint32_t base, int row, const uint16_t* from) {
  auto at = [&](int c) { return base + (c >> 3) * (ROWS * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4); };
  uint32_t w[D / 8][4];
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    if constexpr (COPIED) {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[c][0]), "=r"(w[c][1]), "=r"(w[c][2]), "=r"(w[c][3]) : "r"(at(c)));
    } else {
      const uint4 v = from != nullptr ? kv_load(reinterpret_cast<const uint4*>(from) + c) : make_uint4(0, 0, 0, 0);
      w[c][0] = v.x;
      w[c][1] = v.y;
      w[c][2] = v.z;
      w[c][3] = v.w;
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < D / 8; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = kv_unpack16(w[c][e], a.bf16);
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
  int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 8;
  e = amax > 0.f && amax < __int_as_float(0x7F800000) ? max(e, -118) : 0;
  const float by = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = kv_unpack16(w[c][i], a.bf16);
      w[c][i] = kv_pack16(f.x * by, f.y * by, false);
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(c)), "r"(w[c][0]), "r"(w[c][1]), "r"(w[c][2]), "r"(w[c][3])
                 : "memory");
  }
  return a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// The same of a row copied there before.
template <int D, int ROWS>
__device__ __forceinline__ float convert_query(const AttnParams& a, uint32_t base, int row) {
  return convert_query<D, ROWS, true>(a, base, row, nullptr);
}

// Two fp32 products and sums at once.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace ltk

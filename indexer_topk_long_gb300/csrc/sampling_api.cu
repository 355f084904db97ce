// sampling_api.cu -- C ABI of the token sampler: validation on the host and the launch.
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "sampling_internal.cuh"

using namespace ltk;

namespace {

bool aligned_to(const void* p, unsigned n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool one_or_each(const void* p) { return p == nullptr || aligned_to(p, 4); }

}  // namespace

extern "C" ltk_status ltk_sample_tokens(const void* logits, int dtype, long long row_stride, int B, int V, const ltk_sampling* s,
                                        const float* u, int* token, float* logp, void* stream) {
  if (dtype != LTK_BF16 && dtype != LTK_F16 && dtype != LTK_F32) return LTK_ERR_ARG;
  if (s == nullptr || B < 0 || V < 1 || row_stride < V) return LTK_ERR_ARG;
  if (!one_or_each(s->temperature) || !one_or_each(s->top_k) || !one_or_each(s->top_p) || !one_or_each(s->min_p)) return LTK_ERR_ARG;
  if (s->temperature == nullptr && !(s->temperature_all >= 0.f && std::isfinite(s->temperature_all))) return LTK_ERR_ARG;
  if (s->top_p == nullptr && !(s->top_p_all >= 0.f)) return LTK_ERR_ARG;
  if (s->min_p == nullptr && !(s->min_p_all >= 0.f && s->min_p_all <= 1.f)) return LTK_ERR_ARG;
  SamplingParams p{};
  p.logits = logits;
  p.stride = row_stride;
  p.dtype = dtype;
  p.B = B;
  p.V = V;
  p.temperature = s->temperature;
  p.top_k = s->top_k;
  p.top_p = s->top_p;
  p.min_p = s->min_p;
  p.temperature_all = s->temperature_all;
  p.top_k_all = s->top_k_all;
  p.top_p_all = s->top_p_all;
  p.min_p_all = s->min_p_all;
  p.u = u;
  p.token = token;
  p.logp = logp;
  // The entry point's own limits.  The kernel takes kMostElements of a row in each of kMaxCtas CTAs, and V weights of 2^44
  // have to stay below 2^64 in all: 2^20 - 1 elements of any type.
  if (V > (dtype == LTK_F32 ? 360000 : 720000)) return LTK_ERR_UNSUPPORTED;
  if (B == 0) return LTK_OK;
  if (!aligned_to(logits, dtype == LTK_F32 ? 4 : 2) || !aligned_to(u, 4) || !aligned_to(token, 4) || !aligned_to(logp, 4)) return LTK_ERR_ARG;
  int device = 0, num_sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess && !sampling_plan(p, num_sms)) return LTK_ERR_UNSUPPORTED;
  if (e == cudaSuccess) e = launch_sampling(p, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) return LTK_OK;
  if (std::getenv("LTK_DEBUG")) std::fprintf(stderr, "ltk: ltk_sample_tokens: %s\n", cudaGetErrorString(e));
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? LTK_ERR_NOMEM : LTK_ERR_CUDA;
}

// sampling_internal.cuh -- parameters of the token sampler.
#pragma once

#include "ltk_internal.cuh"

namespace ltk {

struct SamplingParams {
  const void* logits;                    // [B, V], rows stride elements apart
  long long stride;
  int dtype;
  int B, V;
  // one value for each row, or null: the one for all
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all;
  int top_k_all;
  float top_p_all;
  float min_p_all;
  const float* u;                        // [B]
  int* token;                            // [B]
  float* logp;                           // [B]
  int ctas;                              // of a row
  int per;                               // 16-byte pieces of a CTA's slice
};
// Sets ctas and per; false: too many rows.
bool sampling_plan(SamplingParams& p, int num_sms);
cudaError_t launch_sampling(const SamplingParams& p, cudaStream_t stream);

}  // namespace ltk

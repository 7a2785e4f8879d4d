// Launch interface of the token-by-token delta rule (kda_recurrent.cu).
#pragma once

#include <cuda_runtime.h>

#include "kda_prompt.cuh"

namespace kda {

struct RecurrentParams {
  const uint16_t *q, *k, *v, *g;  // [n_tokens, H, 128]
  const uint16_t *beta;           // [n_tokens, H]
  const float *A_log, *dt_bias;   // [H], [H, 128]
  float lower_bound, q_scale;
  void *state;  // [n_slots, H, 128, 128], FP32 or BF16
  long long slot_stride;
  uint16_t *out;  // [n_tokens, H, 128]
  int H;
  int max_len;  // requests of more tokens are someone else's (inert ones are not)
  bool beside;  // may start beside the kernel before it in the stream
  PromptMaps maps;
};

// Host checks of the rule's own operands (the maps' are check_prompt_maps).
int check_rule(const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v, const kda_bf16 *raw_g,
               const kda_bf16 *raw_beta, const float *A_log, const float *dt_bias,
               float lower_bound, float q_scale, const void *state_pool, int state_dtype,
               int64_t slot_stride, int H, const kda_bf16 *out);

// The decays of a prompt multiply over any number of tokens: they must not
// exceed 1 (false for NaN).  The lower end is the verify kernels' own.
inline bool prompt_gate_ok(float lower_bound) {
  return lower_bound >= -10.0f && lower_bound <= 0.0f;
}

int launch_recurrent(const RecurrentParams &p, bool bf16, cudaStream_t stream);

}  // namespace kda

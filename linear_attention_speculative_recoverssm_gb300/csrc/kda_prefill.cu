// kda_prefill: the gated delta rule over ragged prompts.
#include <cuda_runtime.h>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prompt.cuh"
#include "kda_recurrent.cuh"

extern "C" {

int64_t kda_prefill_workspace_bytes(int n_tokens, int B, int H) {
  if (n_tokens < 0 || B < 0 || H < 1 || H > KDA_PROMPT_MAX_HEADS) return -1;
  return 0;
}

int kda_prefill(const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v, const kda_bf16 *raw_g,
                const kda_bf16 *raw_beta, const float *A_log, const float *dt_bias,
                float lower_bound, float q_scale, void *state_pool, int state_dtype,
                int64_t slot_stride, int n_slots, const int32_t *sources,
                const int32_t *destinations, const int32_t *boundaries,
                const int32_t *boundary_lens, const int32_t *query_start_loc, int n_tokens,
                kda_bf16 *out, void *workspace, int64_t workspace_bytes, int B, int H, int Q,
                int null_slot, int32_t *status, void *stream) {
  const int64_t need = kda_prefill_workspace_bytes(n_tokens, B, H);
  if (need < 0) return KDA_ERR_ARG;
  if (B > 0 && n_tokens > 0 && workspace_bytes < need) return KDA_ERR_ARG;
  return kda_recurrent(q, k, v, raw_g, raw_beta, A_log, dt_bias, lower_bound, q_scale, state_pool,
                       state_dtype, slot_stride, n_slots, sources, destinations, boundaries,
                       boundary_lens, query_start_loc, n_tokens, out, B, H, Q, null_slot, status,
                       stream);
}

}  // extern "C"

// The token-by-token delta rule (kda_recurrent.cu): its launch interface, and a
// token's operands, which the chunked form's chain shares.
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

// -- one token's operands: what every token-by-token form makes of it ---------

__device__ __forceinline__ float4 bf16x4_to_f32(uint32_t lo, uint32_t hi) {
  return make_float4(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u),
                     __uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
}

// One token's operands as loaded, four channels to a lane.
struct RawToken {
  uint2 q, k, g, v;
  uint16_t beta;
};

// Row `row` of the activations.
__device__ __forceinline__ RawToken load_token(const RecurrentParams &p, long long row, int lane) {
  const long long base = row * kDim;
  RawToken t;
  t.q = __ldg(reinterpret_cast<const uint2 *>(p.q + base) + lane);
  t.k = __ldg(reinterpret_cast<const uint2 *>(p.k + base) + lane);
  t.g = __ldg(reinterpret_cast<const uint2 *>(p.g + base) + lane);
  t.v = __ldg(reinterpret_cast<const uint2 *>(p.v + base) + lane);
  t.beta = __ldg(p.beta + row);
  return t;
}

// The same, worked out: the lane's channels of d, kn and qn, and kn . qn (with
// q_scale) and beta.
struct Token {
  float4 d, k, q;
  float kq, beta;
};

// `a` is exp(A_log) of the head, `dt` the lane's channels' bias.
__device__ __forceinline__ Token make_token(const RecurrentParams &p, const RawToken &r, float a,
                                            float4 dt) {
  Token t;
  const float4 q = bf16x4_to_f32(r.q.x, r.q.y), k = bf16x4_to_f32(r.k.x, r.k.y);
  const float4 g = bf16x4_to_f32(r.g.x, r.g.y);
  float qq = q.x * q.x + q.y * q.y + q.z * q.z + q.w * q.w;
  float kk = k.x * k.x + k.y * k.y + k.z * k.z + k.w * k.w;
  float kq = k.x * q.x + k.y * q.y + k.z * q.z + k.w * q.w;
  qq = warp_sum(qq);
  kk = warp_sum(kk);
  kq = warp_sum(kq);
  const float qs = rsqrtf(qq + kNormEps) * p.q_scale, ks = rsqrtf(kk + kNormEps);
  t.d = make_float4(gate_decay(a, g.x, dt.x, p.lower_bound), gate_decay(a, g.y, dt.y, p.lower_bound),
                    gate_decay(a, g.z, dt.z, p.lower_bound),
                    gate_decay(a, g.w, dt.w, p.lower_bound));
  t.k = make_float4(k.x * ks, k.y * ks, k.z * ks, k.w * ks);
  t.q = make_float4(q.x * qs, q.y * qs, q.z * qs, q.w * qs);
  t.kq = kq * qs * ks;
  t.beta = 1.f / (1.f + __expf(-bf16_bits_to_f32(r.beta)));
  return t;
}

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

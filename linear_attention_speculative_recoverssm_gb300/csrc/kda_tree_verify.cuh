// The delta rule over trees: arguments, a request's tree, and the vectors and
// coefficients that a (request, head) needs, made by its CTA's warps.
//
// For node t with path a_0 = t, a_1 = parent, .. up to a root, kn and qn the
// normalised key and query, d the decays:
//   X_k[t] = d_{a_0} d_{a_1} .. kn_t, X_q[t] the same of qn_t (down from the
//   checkpoint);
//   A[t][j] = kn_{a_{j+1}} . (d_{a_0} .. d_{a_j} kn_t), B[t][j] the same of
//   qn_t, and B_self[t] = kn_t . qn_t.
// A warp takes a node and walks up its path, multiplying as it goes: no
// decay is divided by, so that any gate will do, and other branches, whatever
// they hold, are never met.
#pragma once

#include <cuda_runtime.h>

#include "kda_tree.cuh"

namespace kda {

struct TreeVerifyParams {
  TreeMaps maps;
  const uint16_t *q, *k, *v, *g, *beta;
  const float *A_log, *dt_bias;
  float lower_bound, q_scale;
  void *state;
  long long slot_stride;
  const float *corr;
  const uint16_t *kg;
  long long corr_stride, kg_stride;
  float *node_corr;
  uint16_t *out;
  int H;
};

// The variant on the tensor cores (kda_tree_verify_mma.cu).
int launch_tree_mma(const TreeVerifyParams &p, bool bf16, int sms, cudaStream_t stream);

// Coefficients of a node, in shared memory: A[0 .. 6], B[0 .. 6], B_self, beta.
constexpr int kTreeCoefs = 16;
constexpr int kCoefB = kTreeDepth - 1, kCoefSelf = 2 * (kTreeDepth - 1),
              kCoefBeta = kCoefSelf + 1;

__device__ __forceinline__ float4 bf16x4(uint2 x) {
  return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                     __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
}

__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, a.x * b.x)));
}

__device__ __forceinline__ float4 scale4(float4 a, float s) {
  return make_float4(a.x * s, a.y * s, a.z * s, a.w * s);
}

// The decays of a lane's four channels.
__device__ __forceinline__ float4 decay4(float a, float4 g, float4 dt, float lower_bound) {
  return make_float4(gate_decay(a, g.x, dt.x, lower_bound), gate_decay(a, g.y, dt.y, lower_bound),
                     gate_decay(a, g.z, dt.z, lower_bound), gate_decay(a, g.w, dt.w, lower_bound));
}

// A node's operands as a warp asks for them: 4 channels a lane.
struct NodeInputs {
  uint2 q, k, g;
  uint16_t beta;
};

__device__ __forceinline__ NodeInputs node_inputs(const TreeVerifyParams &p, long long row,
                                                  int lane) {
  NodeInputs x;
  x.q = __ldg(reinterpret_cast<const uint2 *>(p.q + row * kDim) + lane);
  x.k = __ldg(reinterpret_cast<const uint2 *>(p.k + row * kDim) + lane);
  x.g = __ldg(reinterpret_cast<const uint2 *>(p.g + row * kDim) + lane);
  x.beta = __ldg(p.beta + row);
  return x;
}

// Norms and decay of a node: kn and d to shared memory for its descendants,
// qn handed back.
__device__ __forceinline__ float4 node_operands(const TreeVerifyParams &p, const NodeInputs &x,
                                                float a, float4 dt, int lane, float *kn, float *d) {
  const float4 k = bf16x4(x.k), q = bf16x4(x.q);
  float kk = dot4(k, k), qq = dot4(q, q);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    kk += __shfl_xor_sync(0xffffffffu, kk, o);
    qq += __shfl_xor_sync(0xffffffffu, qq, o);
  }
  sts4(kn + 4 * lane, scale4(k, rsqrtf(kk + kNormEps)));
  sts4(d + 4 * lane, decay4(a, bf16x4(x.g), dt, p.lower_bound));
  return scale4(q, rsqrtf(qq + kNormEps) * p.q_scale);
}

// Node t's way up: its coefficients (all but beta) into `coef`, and what
// reaches the checkpoint in xk, xq.  kn, d: [nodes][128].
__device__ __forceinline__ void node_walk(const int8_t *parent, int t, float4 qn, const float *kn,
                                          const float *d, int lane, float *coef, float4 &xk,
                                          float4 &xq) {
  xk = lds4(kn + t * kDim + 4 * lane);
  xq = qn;
  float v[kTreeCoefs];
#pragma unroll
  for (int i = 0; i < kTreeCoefs; ++i) v[i] = 0.f;
  v[kCoefSelf] = dot4(xk, xq);
  int s = t;
#pragma unroll
  for (int j = 0; j < kTreeDepth; ++j) {
    const float4 ds = lds4(d + s * kDim + 4 * lane);
    xk = fmul4(xk, ds);
    xq = fmul4(xq, ds);
    s = parent[s];
    if (s < 0) break;  // (the same in every lane)
    if (j < kTreeDepth - 1) {
      const float4 ks = lds4(kn + s * kDim + 4 * lane);
      v[j] = dot4(xk, ks);
      v[kCoefB + j] = dot4(xq, ks);
    }
  }
  // lane l of each half warp ends with value l
  reduce_scatter<kTreeCoefs, 16>(v, lane);
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
  if (lane < kCoefBeta) coef[lane] = v[0];
}

// The replay's operands: kp[t] = kn_t times the decays behind token t, and
// the product of all, Dn, in place of the recorded tokens' keys and decays.
// One thread a channel; kp and dec are [kMaxQ][128].
__device__ __forceinline__ void replay_suffix(float *kp, const float *dec, float *dn, int n, int c) {
  float behind = 1.f;
  for (int t = n - 1; t >= 0; --t) {
    kp[t * kDim + c] *= behind;
    behind *= dec[t * kDim + c];
  }
  dn[c] = behind;
}

}  // namespace kda

// The delta rule over trees of drafted tokens, from the checkpoint, the
// pending replay folded in:
//   S_n = S_0 diag(D_n) + sum_t u_t kp_t^T (written back iff n > 0),
//   w_t = S_n X_k[t], y_t = S_n X_q[t],
//   u_t = beta_t (v_t - w_t - sum_j A[t][j] u_{a_j}),
//   o_t = y_t + sum_j B[t][j] u_{a_j} + B_self[t] u_t
// over the ancestors a_j of t: no node's state is formed, and the page is
// read once and written at most once.
#include <cuda_runtime.h>

#include <cmath>

#include "kda_launch.h"
#include "kda_tree_verify.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------------------
// Windows of a few nodes: a CTA an item, or a slice of its rows, its part of the
// state in registers, products by FMA.  (Larger ones: kda_tree_verify_mma.cu.)
// ---------------------------------------------------------------------------

constexpr int kTrThreads = 256;
constexpr int kTrWarps = kTrThreads / 32;
constexpr int kTrNodes = 8;  // room for windows of up to kTrMaxQ nodes
constexpr int kTrMaxQ = 6;
constexpr int kTrFewNodes = 4;  // windows that go by FMA however many items there are

// Shared memory of a CTA whose windows hold up to `nodes` (a multiple of 4)
// nodes, in floats: X, [2 nodes][128]; kn and d, [nodes][128] each, whose
// place the products w and y take afterwards; u, [nodes][rows]; coefficients;
// the replay's kp, decays and corrections, and D_n.
struct RowsLayout {
  int x, kn, d, wy, u, coef, kp, dec, ru, dn, floats;
};

__host__ __device__ constexpr RowsLayout rows_layout(int nodes, int rows) {
  RowsLayout l{};
  l.x = 0;
  l.kn = l.x + 2 * nodes * kDim;
  l.d = l.kn + nodes * kDim;
  l.wy = l.kn;
  const int wy = 2 * nodes * (rows + 4), knd = 2 * nodes * kDim;
  l.u = l.wy + (wy > knd ? wy : knd);
  l.coef = l.u + nodes * rows;
  l.kp = l.coef + nodes * kTreeCoefs;
  l.dec = l.kp + kMaxQ * kDim;
  l.ru = l.dec + kMaxQ * kDim;
  l.dn = l.ru + kMaxQ * kDim;
  l.floats = l.dn + kDim;
  return l;
}

template <bool BF16>
__device__ __forceinline__ float4 state_load(const void *state, long long at) {
  if constexpr (BF16) {
    return bf16x4(__ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(state) + at)));
  } else {
    return __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(state) + at));
  }
}

// ROWS rows of the page a CTA; 8 lanes a row, ROWS / 32 rows a lane, channels
// 4 (lane + 8 j) + 0 .. 3 of each.
template <int ROWS, bool BF16>
__global__ void __launch_bounds__(kTrThreads) kda_tree_rows_kernel(const TreeVerifyParams p,
                                                                   int nodes) {
  constexpr int RPT = ROWS / (kTrThreads / 8), kSplit = kDim / ROWS, kPitch = ROWS + 4;
  extern __shared__ __align__(16) float mem[];
  __shared__ __align__(16) int8_t parent[kTreeNodes];
  __shared__ int good;
  const TreeMaps &mp = p.maps;
  const RowsLayout l = rows_layout(nodes, ROWS);
  const int item = blockIdx.x / kSplit, slice = blockIdx.x % kSplit;
  const int b = item / p.H, h = item - b * p.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const TreeRequest r = tree_request(mp, b);
  if (r.error == KDA_OK && r.slot < 0) {
    for (int t = tid / (ROWS / 8); t < r.n; t += kTrThreads / (ROWS / 8))
      *reinterpret_cast<uint4 *>(p.out + ((long long)(r.t0 + t) * p.H + h) * kDim + slice * ROWS +
                                 tid % (ROWS / 8) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  if (warp == 0) {
    const bool ok = r.error == KDA_OK && load_tree(mp, r, parent, lane);
    if (lane == 0) {
      good = ok;
      if (!ok && slice == 0) report(mp.status, KDA_ERR_ARG);
    }
  }
  __syncthreads();
  if (!good) return;
  // the rows are asked for first
  const int group = tid >> 3, sub = tid & 7;
  const long long page = r.slot * p.slot_stride + (long long)h * kDim * kDim;
  const long long base = page + (long long)(slice * ROWS + group * RPT) * kDim + 4 * sub;
  float4 s[RPT][4];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = state_load<BF16>(p.state, base + i * kDim + 32 * j);
  float *x = mem + l.x, *kn = mem + l.kn, *d = mem + l.d, *coef = mem + l.coef;
  const float a = expf(p.A_log[h]);
  const float4 dt = __ldg(reinterpret_cast<const float4 *>(p.dt_bias + h * kDim) + lane);
  const int n = r.pending;
  for (int t = warp; t < n; t += kTrWarps) {
    const uint16_t *rec = p.kg + r.row * p.kg_stride + ((long long)h * mp.rq + t) * 2 * kDim;
    const float4 k = bf16x4(__ldg(reinterpret_cast<const uint2 *>(rec) + lane));
    const float4 g = bf16x4(__ldg(reinterpret_cast<const uint2 *>(rec + kDim) + lane));
    const float4 u = __ldg(reinterpret_cast<const float4 *>(p.corr + r.row * p.corr_stride +
                                                            ((long long)h * mp.rq + t) * kDim) +
                           lane);
    sts4(mem + l.kp + t * kDim + 4 * lane, scale4(k, rsqrtf(warp_sum(dot4(k, k)) + kNormEps)));
    sts4(mem + l.dec + t * kDim + 4 * lane, decay4(a, g, dt, p.lower_bound));
    sts4(mem + l.ru + t * kDim + 4 * lane, u);
  }
  for (int t = warp; t < r.n; t += kTrWarps) {
    const NodeInputs in = node_inputs(p, (long long)(r.t0 + t) * p.H + h, lane);
    const float4 qn = node_operands(p, in, a, dt, lane, kn + t * kDim, d + t * kDim);
    sts4(x + (2 * t + 1) * kDim + 4 * lane, qn);  // until the walk
    if (lane == 0) coef[t * kTreeCoefs + kCoefBeta] = sigmoidf_fast(bf16_bits_to_f32(in.beta));
  }
  __syncthreads();
  for (int t = warp; t < r.n; t += kTrWarps) {
    float4 xk, xq;
    node_walk(parent, t, lds4(x + (2 * t + 1) * kDim + 4 * lane), kn, d, lane,
              coef + t * kTreeCoefs, xk, xq);
    sts4(x + 2 * t * kDim + 4 * lane, xk);
    sts4(x + (2 * t + 1) * kDim + 4 * lane, xq);
  }
  if (n > 0 && tid < kDim) replay_suffix(mem + l.kp, mem + l.dec, mem + l.dn, n, tid);
  __syncthreads();
  if (n > 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 dn = lds4(mem + l.dn + 4 * sub + 32 * j);
#pragma unroll
      for (int i = 0; i < RPT; ++i) s[i][j] = fmul4(s[i][j], dn);
    }
    for (int t = 0; t < n; ++t) {
      float u[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) u[i] = mem[l.ru + t * kDim + slice * ROWS + group * RPT + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 k = lds4(mem + l.kp + t * kDim + 4 * sub + 32 * j);
#pragma unroll
        for (int i = 0; i < RPT; ++i) s[i][j] = ffma4s(u[i], k, s[i][j]);
      }
    }
    if constexpr (!BF16) {
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          stg4(static_cast<float *>(p.state) + base + i * kDim + 32 * j, s[i][j]);
    }
  }
  // w and y, four nodes (eight vectors) at a time; lane `sub` of a row's
  // eight ends with vector `sub` of them
  float *wy = mem + l.wy;
  for (int t = 0; t < r.n; t += 4) {
    float v[8 * RPT];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2 acc[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 xv = lds4(x + (2 * t + e) * kDim + 4 * sub + 32 * j);
#pragma unroll
        for (int i = 0; i < RPT; ++i) acc[i] = dot4_acc(s[i][j], xv, acc[i]);
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i) v[e * RPT + i] = acc[i].x + acc[i].y;
    }
    reduce_scatter<8 * RPT, 8>(v, lane);
#pragma unroll
    for (int i = 0; i < RPT; ++i) wy[(2 * t + sub) * kPitch + group * RPT + i] = v[i];
  }
  __syncthreads();
  // a thread a row: down the nodes, each behind its ancestors
  if (tid < ROWS) {
    float *u = mem + l.u;
    const long long first = (long long)r.t0 * p.H + h;
    const int row = slice * ROWS + tid;
    for (int t = 0; t < r.n; ++t) {
      const float *c = coef + t * kTreeCoefs;
      float w = wy[2 * t * kPitch + tid], o = wy[(2 * t + 1) * kPitch + tid];
      const long long at = (first + (long long)t * p.H) * kDim + row;
      const float v = bf16_bits_to_f32(__ldg(p.v + at));
      int j = 0;
      for (int s2 = parent[t]; s2 >= 0; s2 = parent[s2], ++j) {
        const float us = u[s2 * ROWS + tid];
        w = fmaf(c[j], us, w);
        o = fmaf(c[kCoefB + j], us, o);
      }
      const float ut = c[kCoefBeta] * (v - w);
      u[t * ROWS + tid] = ut;
      p.node_corr[at] = ut;
      p.out[at] = f32_to_bf16_bits(fmaf(c[kCoefSelf], ut, o));
    }
  }
}

template <int ROWS, bool BF16>
int launch_rows(const TreeVerifyParams &p, cudaStream_t stream) {
  const int nodes = round_up(p.maps.Q, 4);
  const int bytes = rows_layout(nodes, ROWS).floats * 4;
  const auto kernel = kda_tree_rows_kernel<ROWS, BF16>;
  // (the largest call's, always: another thread's call may come in between)
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           rows_layout(kTrNodes, ROWS).floats * 4) != cudaSuccess)
    return KDA_ERR_CUDA;
  kernel<<<(unsigned)p.maps.B * p.H * (kDim / ROWS), kTrThreads, bytes, stream>>>(p, nodes);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace
}  // namespace kda

extern "C" int kda_tree_verify(
    const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v, const kda_bf16 *raw_g,
    const kda_bf16 *raw_beta, const float *A_log, const float *dt_bias, float lower_bound,
    float q_scale, void *state_pool, int state_dtype, int64_t slot_stride, int n_slots,
    const int32_t *state_slots, const int32_t *parents, const int32_t *query_start_loc,
    int n_tokens, const int32_t *record_rows, const int32_t *pending, const float *corr,
    const kda_bf16 *key_gate, int64_t corr_row_stride, int64_t kg_row_stride, int n_rows, int rq,
    float *node_corr, kda_bf16 *out, int B, int H, int Q, int null_slot, int32_t *status,
    void *stream) {
  kda::TreeVerifyParams p;
  const bool replay = pending != nullptr;
  p.maps = kda::TreeMaps{parents, state_slots, replay ? record_rows : nullptr, pending,
                         query_start_loc, n_tokens, n_slots, replay ? n_rows : B, rq, B, Q,
                         null_slot, status};
  if (const int rc = kda::check_tree_maps(p.maps, H); rc != KDA_OK) return rc;
  if (state_dtype != KDA_STATE_F32 && state_dtype != KDA_STATE_BF16) return KDA_ERR_UNSUPPORTED;
  if (!(lower_bound >= -10.0f && lower_bound <= 10.0f)) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(q_scale)) return KDA_ERR_ARG;
  if (parents == nullptr && Q > KDA_TREE_MAX_DEPTH) return KDA_ERR_ARG;
  if ((corr == nullptr) == replay || (key_gate == nullptr) == replay) return KDA_ERR_ARG;
  const bool bf16 = state_dtype == KDA_STATE_BF16;
  if (replay && bf16) return KDA_ERR_UNSUPPORTED;
  if (replay && (rq < 1 || rq > KDA_MAX_WINDOW)) return KDA_ERR_ARG;
  // One warp of each of the tensor cores' CTAs looks through its requests, 0.6 us
  // for each without nodes (2^24: 70 ms), while the others' waits run towards their
  // limit of 2 s.
  if (Q > kda::kTrFewNodes && B > KDA_PLAN_MAX_REQUESTS) return KDA_ERR_ARG;
  if (B == 0 || (n_tokens == 0 && !replay)) return KDA_OK;
  if (!A_log || !dt_bias || !state_pool || !state_slots || n_slots < 1) return KDA_ERR_ARG;
  if (n_tokens > 0 && (!q || !k || !v || !raw_g || !raw_beta || !node_corr || !out))
    return KDA_ERR_ARG;
  const int64_t D = (int64_t)H * KDA_HEAD_DIM;
  if (slot_stride < D * KDA_HEAD_DIM) return KDA_ERR_ARG;
  if (replay && (n_rows < 1 || (record_rows == nullptr && n_rows < B) ||
                 corr_row_stride < D * rq || kg_row_stride < 2 * D * rq))
    return KDA_ERR_ARG;
  if (!kda::tree_aligned16(q) || !kda::tree_aligned16(k) || !kda::tree_aligned16(v) ||
      !kda::tree_aligned16(raw_g) || !kda::tree_aligned16(dt_bias) ||
      !kda::tree_aligned16(state_pool) || !kda::tree_aligned16(node_corr) ||
      !kda::tree_aligned16(out) || !kda::tree_aligned16(corr) || !kda::tree_aligned16(key_gate) ||
      (slot_stride * (bf16 ? 2 : 4)) % 16 != 0 ||
      (replay && (corr_row_stride % 4 != 0 || kg_row_stride % 8 != 0)))
    return KDA_ERR_ALIGN;
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = raw_g;
  p.beta = raw_beta;
  p.A_log = A_log;
  p.dt_bias = dt_bias;
  p.lower_bound = lower_bound;
  p.q_scale = q_scale;
  p.state = state_pool;
  p.slot_stride = slot_stride;
  p.corr = corr;
  p.kg = key_gate;
  p.corr_stride = corr_row_stride;
  p.kg_stride = kg_row_stride;
  p.node_corr = node_corr;
  p.out = out;
  p.H = H;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  const int sms = kda::device_sm_count(dev);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Windows of a few nodes by FMA, and of few items by a CTA for every 32 rows;
  // all others on the tensor cores.  FP32 pages with a replay, us by FMA (by rows
  // of 32 / by whole pages) and on the tensor cores: 4 nodes, 32 items 13 / 15 and
  // 15, 192 items 25 / 19 and 25, 1536 items 130 / 74 and 74; 6 nodes, 32 items 15
  // and 17, 192 items 21 and 25, 512 items 37 and 37, 1536 items 87 and 74; 8 nodes,
  // 1536 items 95 and 75; 15 nodes, 32 items 23 / 25 and 17.  Pages that are only
  // read, FP32 (and BF16): 6 nodes, 512 items 29 and 27 (27 and 25), 1536 items 64 and
  // 52 (61 and 45), 8192 items 289 and 199 (267 and 173); 4 nodes, 512 items 23 and 27
  // (22 and 23), 1536 items 50 and 52 (47 and 44), 8192 items 212 and 199 (195 and
  // 172; with a replay 328 and 314).
  if (Q > kda::kTrMaxQ || (Q > kda::kTrFewNodes && (long long)B * H > 4LL * sms))
    return kda::launch_tree_mma(p, bf16, sms, st);
  if ((long long)B * H * 4 <= sms)
    return bf16 ? kda::launch_rows<32, true>(p, st) : kda::launch_rows<32, false>(p, st);
  return bf16 ? kda::launch_rows<128, true>(p, st) : kda::launch_rows<128, false>(p, st);
}

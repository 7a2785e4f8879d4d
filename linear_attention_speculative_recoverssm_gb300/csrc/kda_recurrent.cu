// kda_recurrent: the gated delta rule token by token, the state taken from
// and left in slots of the pool.  Per (request, head) item and token
//   S <- S diag(d); u = beta (v - S kn); S <- S + u kn^T; o = S qn,
// d, kn, qn, beta as in the verify kernels.  The rows of S (value channels)
// never meet, so a warp owns 16 rows for the whole window, in registers:
// lane l holds key channels 4 l .. 4 l + 3 of each.  With S_d = S diag(d),
//   w = S_d kn, y = S_d qn, u = beta (v - w), o = y + u (kn . qn),
// so one pass over the rows gives both products, the 32 partial sums of a
// token (w and y of 16 rows) go through one reduce-scatter (31 shuffles)
// that leaves row r's w in lane r and its y in lane 16 + r, and the update
// needs u of each row from its lane (16 shuffles).  State traffic is one
// read and one write of the page whatever the window; at one token that is
// all there is to do, and the kernel streams pages.
#include <cuda_runtime.h>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prompt.cuh"
#include "kda_recurrent.cuh"

namespace kda {
namespace {

constexpr int kRecRows = 16;  // state rows of a warp

__device__ __forceinline__ float4 bf16x4_to_f32(uint2 b) {
  return make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                     __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
}

// The 16 rows of a page from `row0`, to and from registers.
template <bool BF16>
__device__ __forceinline__ void load_rows(const void *page, int row0, int lane,
                                          float4 (&s)[kRecRows]) {
  if constexpr (BF16) {
    const uint2 *g = reinterpret_cast<const uint2 *>(page) + row0 * (kDim / 4) + lane;
    uint2 raw[kRecRows];
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) raw[r] = __ldcs(g + r * (kDim / 4));
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) s[r] = bf16x4_to_f32(raw[r]);
  } else {
    const float4 *g = reinterpret_cast<const float4 *>(page) + row0 * (kDim / 4) + lane;
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) s[r] = __ldcs(g + r * (kDim / 4));
  }
}

template <bool BF16>
__device__ __forceinline__ void store_rows(void *page, int row0, int lane,
                                           const float4 (&s)[kRecRows]) {
  if constexpr (BF16) {
    // the page's own type: rounded once, here
    uint2 *g = reinterpret_cast<uint2 *>(page) + row0 * (kDim / 4) + lane;
#pragma unroll
    for (int r = 0; r < kRecRows; ++r)
      __stcs(g + r * (kDim / 4),
             make_uint2(pack_bf16x2(s[r].x, s[r].y), pack_bf16x2(s[r].z, s[r].w)));
  } else {
    float4 *g = reinterpret_cast<float4 *>(page) + row0 * (kDim / 4) + lane;
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) __stcs(g + r * (kDim / 4), s[r]);
  }
}

// One token's operands of a head as loaded: 4 key channels per lane, and the
// value of row `lane & 15` of the warp.
struct RawToken {
  uint2 q, k, g;
  uint16_t v, beta;
};

__device__ __forceinline__ RawToken load_token(const RecurrentParams &p, long long row, int lane,
                                               int vrow) {
  RawToken t;
  const long long base = row * kDim;
  t.q = __ldg(reinterpret_cast<const uint2 *>(p.q + base) + lane);
  t.k = __ldg(reinterpret_cast<const uint2 *>(p.k + base) + lane);
  t.g = __ldg(reinterpret_cast<const uint2 *>(p.g + base) + lane);
  t.v = __ldg(p.v + base + vrow);
  t.beta = __ldg(p.beta + row);
  return t;
}

template <bool BF16>
__global__ void __launch_bounds__(256, 2) kda_recurrent_kernel(const RecurrentParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H;
  const int row0 = (blockIdx.y * (blockDim.x >> 5) + warp) * kRecRows;
  // launched behind a chain, this grid needs nothing of it but ends after it
  if (p.beside && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) grid_dependency_wait();
  const PromptRequest r = prompt_request(p.maps, b);
  if (r.error != KDA_OK && h == 0 && row0 == 0 && lane == 0) report(p.maps.status, r.error);
  if (r.n == 0) return;
  if (r.n > p.max_len && r.dst >= 0) return;
  if (r.dst < 0) {  // inert: zero outputs
    for (int t = 0; t < r.n; ++t)
      if (lane < kRecRows)
        p.out[((long long)(r.t0 + t) * p.H + h) * kDim + row0 + lane] = 0;
    return;
  }
  const long long head = (long long)h * kDim * kDim * (BF16 ? 2 : 4);
  const long long slot_bytes = p.slot_stride * (BF16 ? 2 : 4);
  char *pool = reinterpret_cast<char *>(p.state) + head;
  float4 s[kRecRows];
  if (r.src >= 0) {
    load_rows<BF16>(pool + r.src * slot_bytes, row0, lane, s);
  } else {
#pragma unroll
    for (int i = 0; i < kRecRows; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float a = expf(p.A_log[h]);
  const float4 dt = *reinterpret_cast<const float4 *>(p.dt_bias + h * kDim + 4 * lane);
  const int vrow = row0 + (lane & (kRecRows - 1));
  RawToken next = load_token(p, (long long)r.t0 * p.H + h, lane, vrow);
  for (int t = 0; t < r.n; ++t) {
    const RawToken cur = next;
    if (t + 1 < r.n) next = load_token(p, (long long)(r.t0 + t + 1) * p.H + h, lane, vrow);
    float4 q = bf16x4_to_f32(cur.q), k = bf16x4_to_f32(cur.k);
    const float4 g = bf16x4_to_f32(cur.g);
    const float4 d = make_float4(gate_decay(a, g.x, dt.x, p.lower_bound),
                                 gate_decay(a, g.y, dt.y, p.lower_bound),
                                 gate_decay(a, g.z, dt.z, p.lower_bound),
                                 gate_decay(a, g.w, dt.w, p.lower_bound));
    float qq = q.x * q.x + q.y * q.y + q.z * q.z + q.w * q.w;
    float kk = k.x * k.x + k.y * k.y + k.z * k.z + k.w * k.w;
    float kq = k.x * q.x + k.y * q.y + k.z * q.z + k.w * q.w;
    qq = warp_sum(qq);
    kk = warp_sum(kk);
    kq = warp_sum(kq);
    const float qs = rsqrtf(qq + kNormEps) * p.q_scale, ks = rsqrtf(kk + kNormEps);
    q = make_float4(q.x * qs, q.y * qs, q.z * qs, q.w * qs);
    k = make_float4(k.x * ks, k.y * ks, k.z * ks, k.w * ks);
    kq *= qs * ks;
    float part[2 * kRecRows];
#pragma unroll
    for (int i = 0; i < kRecRows; ++i) {
      s[i] = fmul4(s[i], d);
      const float2 z = make_float2(0.f, 0.f);
      const float2 w = dot4_acc(s[i], k, z), y = dot4_acc(s[i], q, z);
      part[i] = w.x + w.y;
      part[kRecRows + i] = y.x + y.y;
    }
    reduce_scatter<2 * kRecRows, 32>(part, lane);
    // lane i < 16: w of row i; lane 16 + i: y of row i
    const float beta = 1.f / (1.f + __expf(-bf16_bits_to_f32(cur.beta)));
    const float w = __shfl_sync(0xffffffffu, part[0], lane & (kRecRows - 1));
    const float u = beta * (bf16_bits_to_f32(cur.v) - w);  // of row lane & 15
    if (lane >= kRecRows)
      p.out[((long long)(r.t0 + t) * p.H + h) * kDim + vrow] =
          f32_to_bf16_bits(fmaf(u, kq, part[0]));
#pragma unroll
    for (int i = 0; i < kRecRows; ++i) s[i] = ffma4s(__shfl_sync(0xffffffffu, u, i), k, s[i]);
    if (t + 1 == r.m) store_rows<BF16>(pool + r.bnd * slot_bytes, row0, lane, s);
  }
  store_rows<BF16>(pool + r.dst * slot_bytes, row0, lane, s);
}

}  // namespace

int check_rule(const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v, const kda_bf16 *raw_g,
               const kda_bf16 *raw_beta, const float *A_log, const float *dt_bias,
               float lower_bound, float q_scale, const void *state_pool, int state_dtype,
               int64_t slot_stride, int H, const kda_bf16 *out) {
  if (!q || !k || !v || !raw_g || !raw_beta || !A_log || !dt_bias || !state_pool || !out)
    return KDA_ERR_ARG;
  if (!(q_scale - q_scale == 0.f)) return KDA_ERR_ARG;  // (infinite or NaN)
  if (slot_stride < (int64_t)H * kDim * kDim) return KDA_ERR_ARG;
  const auto aligned = [](const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
  if (!aligned(q) || !aligned(k) || !aligned(v) || !aligned(raw_g) || !aligned(state_pool) ||
      !aligned(out) || !aligned(dt_bias) ||
      ((slot_stride * (state_dtype == KDA_STATE_F32 ? 4 : 2)) & 15) != 0)
    return KDA_ERR_ALIGN;
  return KDA_OK;
}

int launch_recurrent(const RecurrentParams &p, bool bf16, cudaStream_t stream) {
  const int items = p.maps.B * p.H;
  const int warps = 8;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = p.beside ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(items, kDim / kRecRows / warps);
  cfg.blockDim = dim3(32 * warps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = bf16 ? kda_recurrent_kernel<true> : kda_recurrent_kernel<false>;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return KDA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda

extern "C" int kda_recurrent(
    const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v, const kda_bf16 *raw_g,
    const kda_bf16 *raw_beta, const float *A_log, const float *dt_bias, float lower_bound,
    float q_scale, void *state_pool, int state_dtype, int64_t slot_stride, int n_slots,
    const int32_t *sources, const int32_t *destinations, const int32_t *boundaries,
    const int32_t *boundary_lens, const int32_t *query_start_loc, int n_tokens, kda_bf16 *out,
    int B, int H, int Q, int null_slot, int32_t *status, void *stream) {
  if (state_dtype != KDA_STATE_F32 && state_dtype != KDA_STATE_BF16) return KDA_ERR_UNSUPPORTED;
  if (!kda::prompt_gate_ok(lower_bound)) return KDA_ERR_UNSUPPORTED;
  int rc = kda::check_prompt_maps(sources, destinations, boundaries, boundary_lens,
                                  query_start_loc, n_tokens, n_slots, B, H, Q, null_slot);
  if (rc != KDA_OK) return rc;
  if (B == 0 || n_tokens == 0) return KDA_OK;
  rc = kda::check_rule(q, k, v, raw_g, raw_beta, A_log, dt_bias, lower_bound, q_scale, state_pool,
                       state_dtype, slot_stride, H, out);
  if (rc != KDA_OK) return rc;
  const kda::RecurrentParams p{q, k, v, raw_g, raw_beta, A_log, dt_bias, lower_bound, q_scale,
                               state_pool, slot_stride, out, H, 0x7fffffff, false,
                               kda::make_prompt_maps(sources, destinations, boundaries,
                                                     boundary_lens, query_start_loc, n_tokens,
                                                     n_slots, B, Q, null_slot, status)};
  return kda::launch_recurrent(p, state_dtype == KDA_STATE_BF16,
                               static_cast<cudaStream_t>(stream));
}

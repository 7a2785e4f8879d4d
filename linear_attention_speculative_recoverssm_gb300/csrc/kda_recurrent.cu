// kda_recurrent: the gated delta rule token by token, the state taken from
// and left in slots of the pool.  Per (request, head) item and token
//   S <- S diag(d); u = beta (v - S kn); S <- S + u kn^T; o = S qn,
// d, kn, qn, beta as in the verify kernels.  The rows of S (value channels)
// never meet, so a warp owns 16 rows for the whole window, in registers, and
// the page moves once each way whatever the window.  With S_d = S diag(d),
//   w = S_d kn, y = S_d qn, u = beta (v - w), o = y + u (kn . qn):
// one pass over the rows gives both products.
//
// Two kernels, by the window that the caller allows:
//  - one token (kda_recurrent_one): moving the pages is all there is to do.  A
//    warp's load covers a whole FP32 row (512 bytes; lane l holds channels
//    4 l .. 4 l + 3 of each row), every warp makes the token's operands for
//    itself, and none waits for another.  The token is asked for before the
//    page, so that its operands are made while the rows arrive (behind the
//    rows: 654 us).  512 requests of 64 heads, FP32: 616 us, 6.97 TB/s (a
//    copy measures 6.77); the other kernel 662.
//  - more (kda_recurrent_group): lane 8 g + j holds 16 channels of rows g,
//    g + 4, g + 8, g + 12, so that the eight partial sums of a lane go through
//    one reduce-scatter over eight lanes (7 shuffles, where a row to a warp
//    takes 31) and u comes back by 4 instead of 16; a token's operands are
//    made once for the CTA, a token a warp, eight tokens at a time, from rows
//    asked for a step ahead (8 tokens of 32 heads, one request: 6.7 us, asked
//    for when needed 8.5; 100 requests 109 and 114).  100 requests of 32 heads,
//    3 tokens, BF16: 60 us, 3.7 TB/s; the other kernel 82.  What bounds it is
//    its form, a token after the other: each is a chain of sums, shuffles and an
//    update behind the one before, and the 16 warps an SM that the rows'
//    registers leave room for do not cover it.  (The verify kernels take a whole
//    window's products from the state as loaded, and move pages at 80 % of a
//    copy's rate with 8 tokens each.)
#include <cuda_runtime.h>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prompt.cuh"
#include "kda_recurrent.cuh"

namespace kda {
namespace {

constexpr int kRecRows = 16;  // state rows of a warp
constexpr int kGroup = 8;     // tokens whose operands are made at a time,
constexpr int kGroupWarps = 4;  // by so many warps

// What both kernels do first: this item's request, reported if it is wrong,
// its outputs zeroed if it is inert.  False: nothing is left to do.
__device__ __forceinline__ bool begin_item(const RecurrentParams &p, int b, int h, int row0,
                                           int lane, PromptRequest &r) {
  // launched behind a chain, this grid needs nothing of it but ends after it
  if (p.beside && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) grid_dependency_wait();
  r = prompt_request(p.maps, b);
  if (r.error != KDA_OK && h == 0 && row0 == 0 && lane == 0) report(p.maps.status, r.error);
  if (r.n == 0) return false;
  if (r.dst < 0) {
    for (int t = lane >> 4; t < r.n; t += 2)
      p.out[((long long)(r.t0 + t) * p.H + h) * kDim + row0 + (lane & 15)] = 0;
    return false;
  }
  return r.n <= p.max_len;
}

// -- one token ---------------------------------------------------------------

template <bool BF16>
__device__ __forceinline__ void store_whole(void *page, int row0, int lane,
                                            const float4 (&s)[kRecRows]) {
#pragma unroll
  for (int i = 0; i < kRecRows; ++i) {
    if constexpr (BF16)  // the page's own type: rounded once, here
      __stcs(reinterpret_cast<uint2 *>(page) + (row0 + i) * (kDim / 4) + lane,
             make_uint2(pack_bf16x2(s[i].x, s[i].y), pack_bf16x2(s[i].z, s[i].w)));
    else
      __stcs(reinterpret_cast<float4 *>(page) + (row0 + i) * (kDim / 4) + lane, s[i]);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(256, 2) kda_recurrent_one(const RecurrentParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H;
  const int row0 = (blockIdx.y * (blockDim.x >> 5) + warp) * kRecRows;
  PromptRequest r;
  if (!begin_item(p, b, h, row0, lane, r)) return;
  const long long elem = BF16 ? 2 : 4;
  char *pool = reinterpret_cast<char *>(p.state) + (long long)h * kDim * kDim * elem;
  const long long slot_bytes = p.slot_stride * elem;
  const float a = expf(p.A_log[h]);
  const float4 dt = *reinterpret_cast<const float4 *>(p.dt_bias + h * kDim + 4 * lane);
  const long long at = (long long)r.t0 * p.H + h;
  const int row = row0 + (lane & (kRecRows - 1));
  const float v = bf16_bits_to_f32(__ldg(p.v + at * kDim + row));
  const RawToken raw = load_token(p, at, lane);
  float4 s[kRecRows];
  if (r.src < 0) {
#pragma unroll
    for (int i = 0; i < kRecRows; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  } else if constexpr (BF16) {
    const uint2 *g = reinterpret_cast<const uint2 *>(pool + r.src * slot_bytes) +
                     row0 * (kDim / 4) + lane;
    uint2 x[kRecRows];
#pragma unroll
    for (int i = 0; i < kRecRows; ++i) x[i] = __ldcs(g + i * (kDim / 4));
#pragma unroll
    for (int i = 0; i < kRecRows; ++i) s[i] = bf16x4_to_f32(x[i].x, x[i].y);
  } else {
    const float4 *g = reinterpret_cast<const float4 *>(pool + r.src * slot_bytes) +
                      row0 * (kDim / 4) + lane;
#pragma unroll
    for (int i = 0; i < kRecRows; ++i) s[i] = __ldcs(g + i * (kDim / 4));
  }
  const Token t = make_token(p, raw, a, dt);
  float part[2 * kRecRows];
#pragma unroll
  for (int i = 0; i < kRecRows; ++i) {
    s[i] = fmul4(s[i], t.d);
    const float2 z = make_float2(0.f, 0.f);
    const float2 w = dot4_acc(s[i], t.k, z), y = dot4_acc(s[i], t.q, z);
    part[i] = w.x + w.y;
    part[kRecRows + i] = y.x + y.y;
  }
  reduce_scatter<2 * kRecRows, 32>(part, lane);
  // lane i < 16: w of row i; lane 16 + i: y of row i
  const float w = __shfl_sync(0xffffffffu, part[0], lane & (kRecRows - 1));
  const float u = t.beta * (v - w);  // of row lane & 15
  if (lane >= kRecRows) p.out[at * kDim + row] = f32_to_bf16_bits(fmaf(u, t.kq, part[0]));
#pragma unroll
  for (int i = 0; i < kRecRows; ++i) s[i] = ffma4s(__shfl_sync(0xffffffffu, u, i), t.k, s[i]);
  if (r.m > 0) store_whole<BF16>(pool + r.bnd * slot_bytes, row0, lane, s);
  store_whole<BF16>(pool + r.dst * slot_bytes, row0, lane, s);
}

// -- more --------------------------------------------------------------------

// The key channels of lane part j, as the m-th four: 16-byte pieces of a page's
// row, eight lanes side by side (BF16: two fours to a piece).
template <bool BF16>
__device__ __forceinline__ constexpr int key_of(int j, int m) {
  return BF16 ? 64 * (m >> 1) + 8 * j + 4 * (m & 1) : 32 * m + 4 * j;
}

// Rows `row`, row + 4, row + 8 and row + 12, to and from registers.
template <bool BF16>
__device__ __forceinline__ void load_rows(const void *page, int row, int j, float4 (&s)[4][4]) {
  if constexpr (BF16) {
    uint4 raw[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        raw[i][m] = __ldcs(reinterpret_cast<const uint4 *>(page) +
                           (row + 4 * i) * (kDim / 8) + 8 * m + j);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        s[i][2 * m] = bf16x4_to_f32(raw[i][m].x, raw[i][m].y);
        s[i][2 * m + 1] = bf16x4_to_f32(raw[i][m].z, raw[i][m].w);
      }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m)
        s[i][m] = __ldcs(reinterpret_cast<const float4 *>(page) +
                         (row + 4 * i) * (kDim / 4) + 8 * m + j);
  }
}

template <bool BF16>
__device__ __forceinline__ void store_rows(void *page, int row, int j, const float4 (&s)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      // the page's own type: rounded once, here
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float4 a = s[i][2 * m], b = s[i][2 * m + 1];
        __stcs(reinterpret_cast<uint4 *>(page) + (row + 4 * i) * (kDim / 8) + 8 * m + j,
               make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                          pack_bf16x2(b.z, b.w)));
      }
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m)
        __stcs(reinterpret_cast<float4 *>(page) + (row + 4 * i) * (kDim / 4) + 8 * m + j, s[i][m]);
    }
  }
}

// Operands of a group's tokens.
struct __align__(16) GroupOps {
  float d[kGroup][kDim], k[kGroup][kDim], q[kGroup][kDim];
  uint2 v[kGroup][kDim / 4];  // BF16
  float kq[kGroup], beta[kGroup];
};

// One token of a group on a warp's rows; `out` is the head's row of it.
template <bool BF16>
__device__ __forceinline__ void step_rows(const GroupOps &sm, int t, int lane, int row,
                                          float4 (&s)[4][4], uint16_t *out) {
  const int j = lane & 7;
  float part[8];
  float4 k[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int c = key_of<BF16>(j, m);
    const float4 d = lds4(&sm.d[t][c]), q = lds4(&sm.q[t][c]);
    k[m] = lds4(&sm.k[t][c]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i][m] = fmul4(s[i][m], d);
      const float2 z = make_float2(0.f, 0.f);
      const float2 w = dot4_acc(s[i][m], k[m], z), y = dot4_acc(s[i][m], q, z);
      part[i] = m == 0 ? w.x + w.y : part[i] + (w.x + w.y);
      part[4 + i] = m == 0 ? y.x + y.y : part[4 + i] + (y.x + y.y);
    }
  }
  reduce_scatter<8, 8>(part, lane);
  // lane j < 4 of eight: w of its row j; 4 + j: y of row j
  const float w = __shfl_sync(0xffffffffu, part[0], lane & ~4);
  const float v =
      bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(sm.v[t])[row + 4 * (lane & 3)]);
  const float u = sm.beta[t] * (v - w);  // of row lane & 3
  if (j >= 4) out[row + 4 * (j - 4)] = f32_to_bf16_bits(fmaf(u, sm.kq[t], part[0]));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float ui = __shfl_sync(0xffffffffu, u, (lane & ~7) + i);
#pragma unroll
    for (int m = 0; m < 4; ++m) s[i][m] = ffma4s(ui, k[m], s[i][m]);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(32 * kGroupWarps, 4)
    kda_recurrent_group(const RecurrentParams p) {
  __shared__ GroupOps ops[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H;
  const int row0 = (blockIdx.y * kGroupWarps + warp) * kRecRows;
  PromptRequest r;
  if (!begin_item(p, b, h, row0, lane, r)) return;  // (all of the CTA alike)
  const int j = lane & 7, row = row0 + (lane >> 3);
  const long long elem = BF16 ? 2 : 4;
  char *pool = reinterpret_cast<char *>(p.state) + (long long)h * kDim * kDim * elem;
  const long long slot_bytes = p.slot_stride * elem;
  const float a = expf(p.A_log[h]);
  const float4 dt = *reinterpret_cast<const float4 *>(p.dt_bias + h * kDim + 4 * lane);
  const long long t0 = (long long)r.t0 * p.H + h;
  // A warp makes every fourth token's operands, and asks for the one after it
  // first: across groups too, so that it arrives under the steps between.
  const auto ask = [&](int t) {
    return load_token(p, t0 + (long long)(t < r.n ? t : r.n - 1) * p.H, lane);
  };
  RawToken next = ask(warp);
  float4 s[4][4];
  if (r.src >= 0) {
    load_rows<BF16>(pool + r.src * slot_bytes, row, j, s);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) s[i][m] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int g0 = 0; g0 < r.n; g0 += kGroup) {
    GroupOps &sm = ops[(g0 / kGroup) & 1];
    const int n = r.n - g0 < kGroup ? r.n - g0 : kGroup;
    for (int i = warp; i < n; i += kGroupWarps) {
      const RawToken raw = next;
      next = ask(g0 + i + kGroupWarps);
      const Token t = make_token(p, raw, a, dt);
      sm.v[i][lane] = raw.v;
      sts4(&sm.d[i][4 * lane], t.d);
      sts4(&sm.k[i][4 * lane], t.k);
      sts4(&sm.q[i][4 * lane], t.q);
      if (lane == 0) {
        sm.kq[i] = t.kq;
        sm.beta[i] = t.beta;
      }
    }
    // (one barrier a group: the buffer before the last has been read by all
    // that have come here)
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      step_rows<BF16>(sm, t, lane, row, s, p.out + (t0 + (long long)(g0 + t) * p.H) * kDim);
      if (g0 + t + 1 == r.m) store_rows<BF16>(pool + r.bnd * slot_bytes, row, j, s);
    }
  }
  store_rows<BF16>(pool + r.dst * slot_bytes, row, j, s);
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
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  const int sms = device_sm_count(dev);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = p.beside ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // One token, few items: their rows over more CTAs, so that more SMs take part
  // (32 items: 5.2 us by 64-thread CTAs, 5.9 by 256); many: CTAs as large as
  // the SM's registers hold whole (32768 items: 616 us by 256 threads, 637 by
  // 128, 645 by 64).
  const bool one = p.maps.Q == 1;
  const int warps = !one ? kGroupWarps : (items >= sms ? 8 : 2);
  cfg.gridDim = dim3(items, kDim / kRecRows / warps);
  cfg.blockDim = dim3(32 * warps);
  const auto kernel = one ? (bf16 ? kda_recurrent_one<true> : kda_recurrent_one<false>)
                          : (bf16 ? kda_recurrent_group<true> : kda_recurrent_group<false>);
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

// kda_prefill_conv: the layer's short convolution and SiLU over ragged
// prompts (the convolution of kda_layer_prologue for windows of any length):
//   out_t = BF16(silu(bias + sum_{i<4} w_i s_{t+i})),
//   s = [3 window entries (zeros without a source), x_0 .. x_{n-1}],
// and the last three entries of s after n (and after m) tokens become the
// destination's (the boundary's) window.  Nothing but bandwidth: 6 D bytes
// read and 6 D written per token.  A thread takes 8 channels (16-byte
// accesses) and a run of kTokens consecutive tokens, keeping the three
// entries before the current one in registers, so x is read once but for the
// three entries before each run.
#include <cuda_runtime.h>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prompt.cuh"

namespace kda {
namespace {

constexpr int kPcThreads = 128;
constexpr int kPcTokens = 16;  // tokens of a CTA

struct ConvParams {
  const uint16_t *x, *w, *bias;  // [n_tokens, 3 D], [3, 4, D], [3 D] or nullptr
  uint16_t *window;              // [n_slots, 3 D, width]
  long long slot_stride;
  int width, H;
  uint16_t *q, *k, *v;  // [n_tokens, H, 128]
  PromptMaps maps;
};

// The last b with qsl[b] <= t, in [0, B - 1] (0 when there is none): a
// 32-way search by the whole warp.  For offsets that decrease somewhere it
// ends all the same, on a request whose window the caller checks.
__device__ __forceinline__ int find_request(const int32_t *qsl, int B, int t, int lane) {
  int lo = 0, hi = B;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && qsl[at] <= t;
    const uint32_t votes = __ballot_sync(0xffffffffu, below);
    const int last = votes == 0 ? 0 : 31 - __clz(votes);
    const int end = lo + (last + 1) * step;
    lo += last * step;
    hi = end < hi ? end : hi;
  }
  return lo;
}

__device__ __forceinline__ float silu_f32(float z) { return __fdividef(z, 1.f + __expf(-z)); }

struct Eight {
  float f[8];
};

__device__ __forceinline__ Eight unpack8(uint4 b) {
  Eight e;
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e.f[2 * i] = __uint_as_float(w[i] << 16);
    e.f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return e;
}

__device__ __forceinline__ uint4 pack8(const uint16_t (&e)[8]) {
  return make_uint4(e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16),
                    e[4] | ((uint32_t)e[5] << 16), e[6] | ((uint32_t)e[7] << 16));
}

__global__ void __launch_bounds__(kPcThreads) kda_prefill_conv_kernel(const ConvParams p) {
  const PromptMaps &mp = p.maps;
  const int lane = threadIdx.x & 31;
  // every window is looked at once, by the first channel CTAs
  if (blockIdx.y == 0) {
    const long long per = (mp.B + gridDim.x - 1) / gridDim.x;
    for (long long b = blockIdx.x * per + threadIdx.x; b < (blockIdx.x + 1) * per && b < mp.B;
         b += kPcThreads) {
      const PromptRequest r = prompt_request(mp, (int)b);
      if (r.error != KDA_OK) report(mp.status, r.error);
    }
  }
  const int D = p.H * kDim;
  const int group = blockIdx.y * kPcThreads + threadIdx.x;
  const bool active = group < 3 * D / 8;
  const int ch = active ? 8 * group : 0, part = ch / D, hc = ch - part * D;
  const int first = blockIdx.x * kPcTokens;
  const int past = first + kPcTokens < mp.n_tokens ? first + kPcTokens : mp.n_tokens;
  Eight w[4], bias;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = unpack8(__ldg(reinterpret_cast<const uint4 *>(p.w + (long long)(part * 4 + i) * D + hc)));
  bias = p.bias != nullptr ? unpack8(__ldg(reinterpret_cast<const uint4 *>(p.bias + ch)))
                           : unpack8(make_uint4(0, 0, 0, 0));
  uint16_t *out = part == 0 ? p.q : (part == 1 ? p.k : p.v);
  const auto input = [&](int t) {
    return __ldg(reinterpret_cast<const uint4 *>(p.x + (long long)t * (3 * D) + ch));
  };
  int b = mp.qsl != nullptr ? find_request(mp.qsl, mp.B, first, lane) : first / mp.Q;
  for (; b < mp.B; ++b) {  // the requests that reach into this run
    const PromptRequest r = prompt_request(mp, b);
    if (r.n == 0) continue;
    if (r.t0 >= past) break;
    // A request's first three tokens belong to the run of its first: that
    // run alone reads the source's window, so it may then write the
    // destination's and the boundary's, which may be the same slot.
    const bool starts = r.t0 >= first;
    int t = starts ? r.t0 : (first > r.t0 + 3 ? first : r.t0 + 3);
    int end = past;
    if (starts && end < r.t0 + 3) end = r.t0 + 3;
    if (end > r.t0 + r.n) end = r.t0 + r.n;
    // an inert request is skipped: the step over its tokens writes zeros
    if (!active || r.dst < 0 || t >= end) continue;
    uint4 h0, h1, h2;  // the three entries before token t
    if (starts) {
      uint16_t e[3][8];
      const uint16_t *win = p.window + (long long)(r.src < 0 ? 0 : r.src) * p.slot_stride +
                            (long long)ch * p.width;
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int i = 0; i < 3; ++i) e[i][c] = r.src >= 0 ? win[c * p.width + i] : (uint16_t)0;
      h0 = pack8(e[0]);
      h1 = pack8(e[1]);
      h2 = pack8(e[2]);
      // entries n - 3 .. n - 1 are what the request leaves, m - 3 .. m - 1
      // its boundary's
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        const int slot = which == 0 ? r.bnd : r.dst, at = which == 0 ? r.m : r.n;
        if (slot < 0) continue;
        uint16_t *to = p.window + (long long)slot * p.slot_stride + (long long)ch * p.width;
#pragma unroll 1
        for (int i = 0; i < 3; ++i) {
          const int j = at - 3 + i;  // >= -2: at >= 1
          const uint4 v = j >= 0 ? input(r.t0 + j) : (j == -1 ? h2 : h1);
          const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int c = 0; c < 8; ++c) to[c * p.width + i] = (uint16_t)(vw[c / 2] >> (16 * (c & 1)));
        }
      }
    } else {
      h0 = input(t - 3);
      h1 = input(t - 2);
      h2 = input(t - 1);
    }
    Eight s0 = unpack8(h0), s1 = unpack8(h1), s2 = unpack8(h2);
#pragma unroll 4
    for (; t < end; ++t) {
      const Eight x = unpack8(input(t));
      uint32_t res[4];
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        float z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // in tap order, as in kda_layer_prologue
          float acc = fmaf(s0.f[c + e], w[0].f[c + e], bias.f[c + e]);
          acc = fmaf(s1.f[c + e], w[1].f[c + e], acc);
          acc = fmaf(s2.f[c + e], w[2].f[c + e], acc);
          acc = fmaf(x.f[c + e], w[3].f[c + e], acc);
          z[e] = silu_f32(acc);
        }
        res[c / 2] = pack_bf16x2(z[0], z[1]);
      }
      *reinterpret_cast<uint4 *>(out + (long long)t * D + hc) =
          make_uint4(res[0], res[1], res[2], res[3]);
      s0 = s1;
      s1 = s2;
      s2 = x;
    }
  }
}

inline bool aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace
}  // namespace kda

extern "C" int kda_prefill_conv(
    const kda_bf16 *x, const kda_bf16 *conv_weight, const kda_bf16 *conv_bias,
    kda_bf16 *conv_state, int64_t conv_slot_stride, int conv_width, int n_slots,
    const int32_t *sources, const int32_t *destinations, const int32_t *boundaries,
    const int32_t *boundary_lens, const int32_t *query_start_loc, int n_tokens, kda_bf16 *q,
    kda_bf16 *k, kda_bf16 *v, int B, int H, int Q, int null_slot, int32_t *status, void *stream) {
  const int rc = kda::check_prompt_maps(sources, destinations, boundaries, boundary_lens,
                                        query_start_loc, n_tokens, n_slots, B, H, Q, null_slot);
  if (rc != KDA_OK) return rc;
  if (conv_width < 3 || conv_width > KDA_MAX_WINDOW + 2) return KDA_ERR_ARG;
  if (B == 0 || n_tokens == 0) return KDA_OK;
  if (!x || !conv_weight || !conv_state || !q || !k || !v) return KDA_ERR_ARG;
  if (conv_slot_stride < 3LL * H * KDA_HEAD_DIM * conv_width) return KDA_ERR_ARG;
  if (!kda::aligned16(x) || !kda::aligned16(conv_weight) ||
      (conv_bias != nullptr && !kda::aligned16(conv_bias)) || !kda::aligned16(conv_state) ||
      !kda::aligned16(q) || !kda::aligned16(k) || !kda::aligned16(v) || conv_slot_stride % 8 != 0)
    return KDA_ERR_ALIGN;
  kda::ConvParams p;
  p.x = x;
  p.w = conv_weight;
  p.bias = conv_bias;
  p.window = conv_state;
  p.slot_stride = conv_slot_stride;
  p.width = conv_width;
  p.H = H;
  p.q = q;
  p.k = k;
  p.v = v;
  p.maps = kda::make_prompt_maps(sources, destinations, boundaries, boundary_lens,
                                 query_start_loc, n_tokens, n_slots, B, Q, null_slot, status);
  const int groups = 3 * H * KDA_HEAD_DIM / 8;
  const dim3 grid((n_tokens + kda::kPcTokens - 1) / kda::kPcTokens,
                  (groups + kda::kPcThreads - 1) / kda::kPcThreads);
  kda::kda_prefill_conv_kernel<<<grid, kda::kPcThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

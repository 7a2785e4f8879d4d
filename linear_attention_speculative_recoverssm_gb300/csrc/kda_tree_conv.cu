// The layer's short convolution over trees of drafted tokens: per node and
// channel
//   out = BF16(silu(bias + sum_{i<4} w_i s_i)),
// s_3 the node's own input, s_2 .. s_0 those of its three nearest ancestors,
// and of the request's window above a root.
//
// What bounds it: HBM, 4 bytes a node and channel (one input, one output) and
// the windows' sectors once a request.  A CTA takes a request's nodes, or a
// run of them, in 512 channels, four a thread (eight take the registers of
// twice the warps).  Every node asks for its own input and its ancestors'; those
// were asked for just before, and come from the first-level cache.
#include <cuda_runtime.h>

#include "kda_launch.h"
#include "kda_silu.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kTcThreads = 128;

struct TreeConvParams {
  TreeMaps maps;
  const uint16_t *x, *w, *bias, *window;
  long long slot_stride;
  int width, H, run;
  uint16_t *q, *k, *v;
};

struct Four {
  float2 a, b;
};

__device__ __forceinline__ Four unpack4(uint2 x) {
  return Four{make_float2(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u)),
              make_float2(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u))};
}

// Entry `at` of a thread's four channels' windows, `width` entries each.
__device__ __forceinline__ uint2 window_entry(const uint16_t *win, int width, int at) {
  return make_uint2((uint32_t)__ldg(win + at) | (uint32_t)__ldg(win + width + at) << 16,
                    (uint32_t)__ldg(win + 2 * width + at) |
                        (uint32_t)__ldg(win + 3 * width + at) << 16);
}

__global__ void __launch_bounds__(kTcThreads, 8) kda_tree_conv_kernel(const TreeConvParams p) {
  __shared__ int8_t parent[kTreeNodes];
  __shared__ char4 above[kTreeNodes];  // x, y, z: the nearest ancestor first
  __shared__ int good;
  const TreeMaps &mp = p.maps;
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int D = p.H * kDim;
  const int group = blockIdx.y * kTcThreads + threadIdx.x;
  const bool active = group < 3 * D / 4;
  const int ch = active ? 4 * group : 0, part = ch / D, hc = ch - part * D;
  const TreeRequest r = tree_request(mp, b);
  if (r.error == KDA_OK && r.slot < 0) return;
  const int first = blockIdx.z * p.run;
  const int past = r.n - first > p.run ? first + p.run : r.n;
  // the first nodes' inputs, and the entries above a root (the newest first),
  // are asked for before the tree is looked at
  constexpr int kAhead = 4;
  const uint16_t *x = p.x + (long long)r.t0 * (3 * D) + ch;
  uint2 next[kAhead], h1, h2, h3;
  if (r.error == KDA_OK && first < past) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      next[i] = __ldg(reinterpret_cast<const uint2 *>(
          x + (long long)(first + i < past ? first + i : first) * (3 * D)));
    const uint16_t *win = p.window + r.slot * p.slot_stride + (long long)ch * p.width;
    const int off = r.pending > 0 ? r.pending - 1 : 0;
    h1 = window_entry(win, p.width, off + 2);
    h2 = window_entry(win, p.width, off + 1);
    h3 = window_entry(win, p.width, off);
  }
  if (threadIdx.x < 32) {
    const bool ok = r.error == KDA_OK && load_tree(mp, r, parent, lane);
    if (lane == 0) {
      good = ok;
      if (!ok && blockIdx.y == 0 && blockIdx.z == 0) report(mp.status, KDA_ERR_ARG);
    }
    if (ok) {
#pragma unroll
      for (int i = 0; i < kTreeNodes / 32; ++i) {
        const int t = lane + 32 * i;
        const int a = parent[t];
        const int c = a >= 0 ? parent[a] : a - 1;
        const int e = c >= 0 ? parent[c] : c - 1;
        above[t] = make_char4((char)a, (char)c, (char)e, 0);
      }
    }
  }
  Four w[4], bias;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = unpack4(__ldg(reinterpret_cast<const uint2 *>(p.w + (long long)(part * 4 + i) * D + hc)));
  bias = unpack4(p.bias != nullptr ? __ldg(reinterpret_cast<const uint2 *>(p.bias + ch))
                                   : make_uint2(0, 0));
  __syncthreads();
  if (!good || !active || first >= past) return;
  uint16_t *out = (part == 0 ? p.q : (part == 1 ? p.k : p.v)) + (long long)r.t0 * D + hc;
  const auto input = [&](int a) {
    return a >= 0 ? __ldg(reinterpret_cast<const uint2 *>(x + (long long)a * (3 * D)))
                  : (a == -1 ? h1 : (a == -2 ? h2 : h3));
  };
  const auto step = [&](uint2 own, int t) {
    const char4 up = above[t];
    const Four s3 = unpack4(own), s2 = unpack4(input(up.x)), s1 = unpack4(input(up.y)),
               s0 = unpack4(input(up.z));
    // in tap order, as in kda_layer_prologue
    Four z{ffma2(s0.a, w[0].a, bias.a), ffma2(s0.b, w[0].b, bias.b)};
    z = Four{ffma2(s1.a, w[1].a, z.a), ffma2(s1.b, w[1].b, z.b)};
    z = Four{ffma2(s2.a, w[2].a, z.a), ffma2(s2.b, w[2].b, z.b)};
    z = Four{ffma2(s3.a, w[3].a, z.a), ffma2(s3.b, w[3].b, z.b)};
    *reinterpret_cast<uint2 *>(out + (long long)t * D) =
        make_uint2(silu_pair(z.a), silu_pair(z.b));
  };
  // the next four nodes are asked for while four are worked on
#pragma unroll 1
  for (int t = first; t < past; t += kAhead) {
    uint2 own[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) own[i] = next[i];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + kAhead + i < past) next[i] = input(t + kAhead + i);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + i < past) step(own[i], t + i);
  }
}

}  // namespace
}  // namespace kda

extern "C" int kda_tree_conv(const kda_bf16 *x, const kda_bf16 *conv_weight,
                             const kda_bf16 *conv_bias, const kda_bf16 *conv_state,
                             int64_t conv_slot_stride, int conv_width, int n_slots,
                             const int32_t *state_slots, const int32_t *record_rows,
                             const int32_t *pending, int n_rows, const int32_t *parents,
                             const int32_t *query_start_loc, int n_tokens, kda_bf16 *q,
                             kda_bf16 *k, kda_bf16 *v, int B, int H, int Q, int null_slot,
                             int32_t *status, void *stream) {
  kda::TreeConvParams p;
  p.maps = kda::TreeMaps{parents, state_slots, record_rows, pending, query_start_loc,
                         n_tokens, n_slots, n_rows, conv_width - 2, B, Q, null_slot, status};
  if (const int rc = kda::check_tree_maps(p.maps, H); rc != KDA_OK) return rc;
  if (conv_width < 3 || conv_width > KDA_MAX_WINDOW + 2) return KDA_ERR_ARG;
  if (parents == nullptr && Q > KDA_TREE_MAX_DEPTH) return KDA_ERR_ARG;
  if (B == 0 || n_tokens == 0) return KDA_OK;
  if (!x || !conv_weight || !conv_state || !state_slots || !q || !k || !v || n_slots < 1)
    return KDA_ERR_ARG;
  // (the record rows only find the pending counts)
  if (pending == nullptr) {
    p.maps.record_rows = nullptr;
    p.maps.n_rows = B;
  } else if (n_rows < 1 || (record_rows == nullptr && n_rows < B)) {
    return KDA_ERR_ARG;
  }
  if (conv_slot_stride < 3LL * H * KDA_HEAD_DIM * conv_width) return KDA_ERR_ARG;
  if (!kda::tree_aligned16(x) || !kda::tree_aligned16(conv_weight) ||
      (conv_bias != nullptr && !kda::tree_aligned16(conv_bias)) ||
      !kda::tree_aligned16(conv_state) || !kda::tree_aligned16(q) || !kda::tree_aligned16(k) ||
      !kda::tree_aligned16(v) || conv_slot_stride % 8 != 0)
    return KDA_ERR_ALIGN;
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
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  const int sms = kda::device_sm_count(dev);
  const int channels = (3 * H * KDA_HEAD_DIM / 4 + kda::kTcThreads - 1) / kda::kTcThreads;
  // whole requests where they fill the SMs, else runs of their nodes
  int run = Q;
  while (run > 2 && (long long)B * channels * ((Q - 1) / run + 1) < 4LL * sms) run = (run + 1) / 2;
  p.run = run;
  const dim3 grid(B, channels, (Q - 1) / run + 1);
  kda::kda_tree_conv_kernel<<<grid, kda::kTcThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

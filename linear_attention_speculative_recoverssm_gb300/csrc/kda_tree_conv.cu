// The layer's short convolution over trees of drafted tokens: per node and
// channel
//   out = BF16(silu(bias + sum_{i<4} w_i s_i)),
// s_3 the node's own input, s_2 .. s_0 those of its three nearest ancestors,
// and of the request's window above a root.
//
// Its floor is HBM's, 4 bytes a node and channel (one input, one output) and
// the windows' sectors once a request.  A CTA takes a request's nodes, or a
// run of them, in 512 channels, four a thread.  All inputs are copied to shared
// memory at once, asynchronously, and a node's four taps read there: window
// entries and inputs alike, without a branch.
//
// 128 trees of up to 33 nodes, 64 heads (326 MB): 84 us, 3.9 TB/s (a copy: 6.7),
// with 55% of the issue slots and 44% of shared memory's wavefronts: no unit is
// at its end.  Four channels of a node take 87 warp instructions, 32 of them
// addresses and copies, loads and stores of 8 bytes, and the rows leave room for a
// third of an SM's warps to cover their latencies.  By events around the call 89 us; by
// loads four nodes ahead in place of the copies 109, two channels a thread 112;
// loops unrolled further, or the first half of the nodes begun while the rest is
// on its way, gain nothing.
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

// 8-byte asynchronous copy global -> shared.
__device__ __forceinline__ void cp_async8(void *smem_dst, const void *gmem_src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(smem_dst)), "l"(gmem_src)
               : "memory");
}

__global__ void __launch_bounds__(kTcThreads) kda_tree_conv_kernel(const TreeConvParams p) {
  // rows of this CTA's channels: the window's three entries, the oldest first,
  // then the nodes' inputs; a thread reads what it copied itself
  extern __shared__ uint2 rows[];
  __shared__ int8_t parent[kTreeNodes];
  __shared__ uint2 taps[kTreeNodes];  // a node's four rows, the oldest first
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
  // All is asked for before the tree is looked at (ancestors come before their
  // nodes).  A warp's windows, one piece of memory, take the places of its last
  // nodes' inputs until three entries of each channel are picked from them.
  if (r.error == KDA_OK && first < past) {
    const int late = past > p.width ? past - p.width : 0;
    const int warp_ch = 4 * (group - lane), warp_at = threadIdx.x - lane;
    uint2 *const held = rows + (3 + late) * kTcThreads + warp_at;
    const auto held_at = [&](int byte) {  // of the warp's windows
      return reinterpret_cast<char *>(held + (byte >> 8) * kTcThreads) + (byte & 255);
    };
    if (warp_ch < 3 * D) {
      const uint16_t *win = p.window + r.slot * p.slot_stride + (long long)warp_ch * p.width;
      for (int i = lane; i < 16 * p.width; i += 32) cp_async16(held_at(16 * i), win + 8 * i);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const uint16_t *x = p.x + (long long)r.t0 * (3 * D) + ch;
    uint2 *to = rows + 3 * kTcThreads + threadIdx.x;
    int t = 0;
    for (; t < late; ++t, x += 3 * D, to += kTcThreads) cp_async8(to, x);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    const int off = r.pending > 0 ? r.pending - 1 : 0;
    uint2 h[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      uint32_t e[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        e[c] = *reinterpret_cast<const uint16_t *>(held_at(2 * ((4 * lane + c) * p.width + off + i)));
      h[i] = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
    }
    __syncwarp();
    for (; t < past; ++t, x += 3 * D, to += kTcThreads) cp_async8(to, x);
#pragma unroll
    for (int i = 0; i < 3; ++i) rows[i * kTcThreads + threadIdx.x] = h[i];
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
        // (row of node or entry s: s + 3)
        taps[t] = make_uint2((uint32_t)(e + 3) | (uint32_t)(c + 3) << 16,
                             (uint32_t)(a + 3) | (uint32_t)(t + 3) << 16);
      }
    }
  }
  Four w[4], bias;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = unpack4(__ldg(reinterpret_cast<const uint2 *>(p.w + (long long)(part * 4 + i) * D + hc)));
  bias = unpack4(p.bias != nullptr ? __ldg(reinterpret_cast<const uint2 *>(p.bias + ch))
                                   : make_uint2(0, 0));
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (!good || !active || first >= past) return;
  uint16_t *out =
      (part == 0 ? p.q : (part == 1 ? p.k : p.v)) + (long long)(r.t0 + first) * D + hc;
  const uint2 *mine = rows + threadIdx.x;
#pragma unroll 2
  for (int t = first; t < past; ++t, out += D) {
    const uint2 tap = taps[t];
    const Four s0 = unpack4(mine[(tap.x & 0xffffu) * kTcThreads]),
               s1 = unpack4(mine[(tap.x >> 16) * kTcThreads]),
               s2 = unpack4(mine[(tap.y & 0xffffu) * kTcThreads]),
               s3 = unpack4(mine[(tap.y >> 16) * kTcThreads]);
    // in tap order, as in kda_layer_prologue
    Four z{ffma2(s0.a, w[0].a, bias.a), ffma2(s0.b, w[0].b, bias.b)};
    z = Four{ffma2(s1.a, w[1].a, z.a), ffma2(s1.b, w[1].b, z.b)};
    z = Four{ffma2(s2.a, w[2].a, z.a), ffma2(s2.b, w[2].b, z.b)};
    z = Four{ffma2(s3.a, w[3].a, z.a), ffma2(s3.b, w[3].b, z.b)};
    *reinterpret_cast<uint2 *>(out) = make_uint2(silu_pair(z.a), silu_pair(z.b));
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
  constexpr int kRow = kda::kTcThreads * (int)sizeof(uint2);
  // (the largest call's, always: another thread's call may come in between)
  if (cudaFuncSetAttribute(kda::kda_tree_conv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (3 + KDA_TREE_MAX_NODES) * kRow) != cudaSuccess)
    return KDA_ERR_CUDA;
  const int bytes = (3 + (Q > conv_width ? Q : conv_width)) * kRow;
  kda::kda_tree_conv_kernel<<<grid, kda::kTcThreads, bytes, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

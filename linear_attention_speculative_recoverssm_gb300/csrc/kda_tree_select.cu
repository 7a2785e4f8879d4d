// The accepted path of a tree to the front of its request's records and
// convolution window:
//   corr[r, h, i] = node_corr[t_i, h], key_gate[r, h, i] = (k, raw_g)[t_i, h],
//   W <- [W[off + 1], W[off + 2], x[t_0] .. x[t_{m-1}]]
// (an eager request's window: its last three inputs).
//
// Its floor is HBM's, and copies are all there is.  Record CTAs take a
// request's heads, 8 at a time (a warp a head, 16 bytes a lane); window CTAs
// take 1024 channels of a request: their window, one piece of memory, goes
// through shared memory whole, where a thread rewrites the few entries of its
// four channels, and comes back in 16-byte pieces.
//
// 256 requests, 64 heads (285 MB of what has to move, 323 with the entries that
// are kept): 72 us, 4.0 TB/s (a copy: 6.7).  No unit is at its end: HBM is at 57%,
// the shared memory's path, which windows take twice on their way through registers
// and where an entry is 2 bytes, at 62%; a window's CTA reads, rewrites and writes it
// one after the other.  By events around the call 80 us, by one
// channel a thread 95.
#include <cuda_runtime.h>

#include "kda_launch.h"
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kTsThreads = 256;
constexpr int kTsHeads = kTsThreads / 32;
constexpr int kTsChannels = 4 * kTsThreads;
constexpr int kTsMaxWidth = KDA_MAX_WINDOW + 2;

struct TreeSelectParams {
  TreeMaps maps;
  const int32_t *path, *accepted;
  const uint8_t *eager;
  const uint16_t *k, *g, *x;
  const float *node_corr;
  float *corr;
  uint16_t *kg, *window;
  long long corr_stride, kg_stride, slot_stride;
  int width, H, rq;    // (maps.rq is what the pending counts are clamped to)
  int most;            // the longest path that fits
  int record_ctas;     // CTAs of a request that move records
};

__global__ void __launch_bounds__(kTsThreads, 5) kda_tree_select_kernel(const TreeSelectParams p) {
  __shared__ __align__(16) uint16_t rows[kTsChannels * kTsMaxWidth];
  const TreeMaps &mp = p.maps;
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int m = p.accepted[b];
  // (behind nothing accepted the convolution's window moves without any token)
  const TreeRequest r = tree_request(mp, b, m != 0);
  const int32_t *path = p.path + (long long)b * kTreeDepth;
  bool ok = r.error == KDA_OK;
  const bool moves = !ok && m == 0 && r.slot >= 0;
  if (ok && r.slot >= 0 && r.row >= 0) {
    ok = m >= 0 && m <= p.most;
    const int4 lo = reinterpret_cast<const int4 *>(path)[0],
               hi = reinterpret_cast<const int4 *>(path)[1];
    const int nodes[kTreeDepth] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < kTreeDepth; ++i) ok = ok && (i >= m || (nodes[i] >= 0 && nodes[i] < r.n));
  }
  if (!ok && blockIdx.y == 0 && threadIdx.x == 0) report(mp.status, KDA_ERR_ARG);
  if (!(ok || moves) || r.slot < 0 || r.row < 0) return;
  if ((int)blockIdx.y < p.record_ctas) {
    const int h = blockIdx.y * kTsHeads + (threadIdx.x >> 5);
    if (h >= p.H) return;
    const long long at = (long long)r.t0 * p.H + h;
    float *corr = p.corr + r.row * p.corr_stride + (long long)h * p.rq * kDim;
    uint16_t *kg = p.kg + r.row * p.kg_stride + (long long)h * p.rq * 2 * kDim;
    const uint16_t *half = lane < 16 ? p.k : p.g;
    // (three at a time: more registers leave fewer CTAs on an SM)
#pragma unroll 1
    for (int i0 = 0; i0 < m; i0 += 3) {
      float4 u[3];
      uint4 e[3];
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i0 + i < m) {
          const long long row = at + (long long)__ldg(path + i0 + i) * p.H;
          u[i] = __ldcs(reinterpret_cast<const float4 *>(p.node_corr + row * kDim) + lane);
          e[i] = __ldcs(reinterpret_cast<const uint4 *>(half + row * kDim) + (lane & 15));
        }
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i0 + i < m) {
          reinterpret_cast<float4 *>(corr + (i0 + i) * kDim)[lane] = u[i];
          reinterpret_cast<uint4 *>(kg + (i0 + i) * 2 * kDim)[lane] = e[i];
        }
    }
    return;
  }
  const int D3 = 3 * p.H * kDim;
  const int ch0 = ((int)blockIdx.y - p.record_ctas) * kTsChannels;
  const int count = D3 - ch0 < kTsChannels ? D3 - ch0 : kTsChannels;
  uint4 *memory = reinterpret_cast<uint4 *>(p.window + r.slot * p.slot_stride + (long long)ch0 * p.width);
  uint4 *staged = reinterpret_cast<uint4 *>(rows);
  const int pieces = count * p.width / 8;  // (count is a multiple of 128)
  for (int i = threadIdx.x; i < pieces; i += kTsThreads) staged[i] = memory[i];
  const int c = 4 * threadIdx.x;
  uint2 in[kTreeDepth];
  if (c < count) {
#pragma unroll
    for (int i = 0; i < kTreeDepth; ++i)
      if (i < m)
        in[i] = __ldg(reinterpret_cast<const uint2 *>(
            p.x + ((long long)r.t0 + __ldg(path + i)) * D3 + ch0 + c));
  }
  __syncthreads();
  if (c < count) {
    uint16_t *const w = rows + c * p.width;
    const auto get = [&](int i) {
      return make_uint2(w[i] | (uint32_t)w[p.width + i] << 16,
                        w[2 * p.width + i] | (uint32_t)w[3 * p.width + i] << 16);
    };
    const auto set = [&](int i, uint2 v) {
      w[i] = (uint16_t)v.x, w[p.width + i] = (uint16_t)(v.x >> 16);
      w[2 * p.width + i] = (uint16_t)v.y, w[3 * p.width + i] = (uint16_t)(v.y >> 16);
    };
    const int off = r.pending > 0 ? r.pending - 1 : 0;
    if (m == 0 || (p.eager != nullptr && p.eager[b] != 0)) {
      // the last three of the window's and the path's (in order: what an
      // entry takes lies at its place or behind)
      for (int i = 0; i < 3; ++i) {
        const int j = m + i;
        uint2 v = make_uint2(0, 0);
        if (j < 3) v = get(off + j);
#pragma unroll
        for (int e = 0; e < kTreeDepth; ++e)
          if (j - 3 == e) v = in[e];
        set(i, v);
      }
    } else {
      for (int i = 0; i < 2; ++i) set(i, get(off + 1 + i));
#pragma unroll
      for (int i = 0; i < kTreeDepth; ++i)
        if (i < m) set(2 + i, in[i]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pieces; i += kTsThreads) memory[i] = staged[i];
}

}  // namespace
}  // namespace kda

extern "C" int kda_tree_select(const int32_t *path, const int32_t *accepted,
                               const uint8_t *eager, const kda_bf16 *k, const kda_bf16 *raw_g,
                               const float *node_corr,
                               const int32_t *state_slots, const int32_t *record_rows,
                               const int32_t *pending, float *corr, kda_bf16 *key_gate,
                               int64_t corr_row_stride, int64_t kg_row_stride, int n_rows, int rq,
                               const kda_bf16 *x, kda_bf16 *conv_state, int64_t conv_slot_stride,
                               int conv_width, int n_slots, const int32_t *query_start_loc,
                               int n_tokens, int B, int H, int Q, int null_slot, int32_t *status,
                               void *stream) {
  kda::TreeSelectParams p;
  const bool windows = conv_state != nullptr;
  p.maps = kda::TreeMaps{nullptr, state_slots, record_rows, windows ? pending : nullptr,
                         query_start_loc, n_tokens, n_slots, n_rows, rq, B, Q, null_slot, status};
  if (const int rc = kda::check_tree_maps(p.maps, H); rc != KDA_OK) return rc;
  if (rq < 1 || rq > KDA_MAX_WINDOW) return KDA_ERR_ARG;
  if (windows && (conv_width < 3 || conv_width > KDA_MAX_WINDOW + 2)) return KDA_ERR_ARG;
  if (B == 0) return KDA_OK;
  if (!path || !accepted || !state_slots || !corr || !key_gate || n_slots < 1 || n_rows < 1 ||
      (record_rows == nullptr && n_rows < B))
    return KDA_ERR_ARG;
  if (n_tokens > 0 && (!k || !raw_g || !node_corr || (windows && !x))) return KDA_ERR_ARG;
  if (!windows && x != nullptr) return KDA_ERR_ARG;
  const int64_t D = (int64_t)H * KDA_HEAD_DIM;
  if (corr_row_stride < D * rq || kg_row_stride < 2 * D * rq ||
      (windows && conv_slot_stride < 3 * D * conv_width))
    return KDA_ERR_ARG;
  if (!kda::tree_aligned16(path) || !kda::tree_aligned16(k) || !kda::tree_aligned16(raw_g) ||
      !kda::tree_aligned16(node_corr) || !kda::tree_aligned16(corr) ||
      !kda::tree_aligned16(key_gate) || !kda::tree_aligned16(x) ||
      !kda::tree_aligned16(conv_state) || corr_row_stride % 4 != 0 || kg_row_stride % 8 != 0 ||
      (windows && conv_slot_stride % 8 != 0))
    return KDA_ERR_ALIGN;
  p.path = path;
  p.accepted = accepted;
  p.eager = eager;
  p.k = k;
  p.g = raw_g;
  p.x = x;
  p.node_corr = node_corr;
  p.corr = corr;
  p.kg = key_gate;
  p.window = conv_state;
  p.corr_stride = corr_row_stride;
  p.kg_stride = kg_row_stride;
  p.slot_stride = conv_slot_stride;
  p.width = conv_width;
  p.H = H;
  p.rq = rq;
  p.most = windows && conv_width - 2 < rq ? conv_width - 2 : rq;
  if (windows) p.maps.rq = conv_width - 2;  // what kda_tree_conv clamps the pending counts to
  p.record_ctas = (H + kda::kTsHeads - 1) / kda::kTsHeads;
  const int window_ctas =
      windows ? (3 * H * KDA_HEAD_DIM + kda::kTsChannels - 1) / kda::kTsChannels : 0;
  const dim3 grid(B, p.record_ctas + window_ctas);
  kda::kda_tree_select_kernel<<<grid, kda::kTsThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

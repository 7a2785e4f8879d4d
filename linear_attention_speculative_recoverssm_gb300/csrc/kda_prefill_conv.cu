// kda_prefill_conv: the layer's short convolution and SiLU over ragged
// prompts (the convolution of kda_layer_prologue for windows of any length):
//   out_t = BF16(silu(bias + sum_{i<4} w_i s_{t+i})),
//   s = [3 window entries (zeros without a source), x_0 .. x_{n-1}],
// and the last three entries of s after n (and after m) tokens become the
// destination's (the boundary's) window.  6 D bytes read and 6 D written per
// token and nothing used twice: bandwidth, if enough is in flight and the
// arithmetic (4 FMA, 2 functions of the special unit per element) stays under
// it.  A thread takes 4 channels and a run of consecutive tokens, keeping the
// three entries before the current one in registers, so x is read once but for
// the three entries before each run; 8 tokens are asked for at a time.  4
// channels a thread and not 8: 80 registers, 24 warps an SM (8 channels: 127,
// 16 warps).  16384 tokens, 32 heads: 138 us, 5.8 TB/s (of 6.77 measured for a
// copy); 8 channels and runs of 16 tokens: 215.  Short prompts are windows above
// all: a thread's four are neighbours, and move whole (entry by entry, 4096
// requests of one token took 809 us in place of 281).
#include <cuda_runtime.h>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prompt.cuh"
#include "kda_silu.cuh"

namespace kda {
namespace {

constexpr int kPcThreads = 128;
constexpr int kAhead = 8;      // tokens whose loads are in flight at a time

struct ConvParams {
  const uint16_t *x, *w, *bias;  // [n_tokens, 3 D], [3, 4, D], [3 D] or nullptr
  uint16_t *window;              // [n_slots, 3 D, width]
  long long slot_stride;
  int H;
  int run;  // tokens of a CTA
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

struct Four {
  float2 a, b;
};

__device__ __forceinline__ Four unpack4(uint2 x) {
  return Four{make_float2(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u)),
              make_float2(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u))};
}

// The windows of a thread's four channels, W entries each, one after the other:
// halfword c W + i.
template <int W>
struct Windows {
  static constexpr int kWords = 2 * W;
  uint32_t w[kWords];
  // (16-byte pieces where W is even, else 8-byte ones)
  __device__ __forceinline__ void load(const uint16_t *at) {
    if constexpr (W % 2 == 0) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const uint4 x = reinterpret_cast<const uint4 *>(at)[i];
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint2 x = reinterpret_cast<const uint2 *>(at)[i];
        w[2 * i] = x.x, w[2 * i + 1] = x.y;
      }
    }
  }
  __device__ __forceinline__ void store(uint16_t *at) const {
    if constexpr (W % 2 == 0) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i)
        reinterpret_cast<uint4 *>(at)[i] =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        reinterpret_cast<uint2 *>(at)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
    }
  }
  __device__ __forceinline__ uint32_t get(int h) const {
    return h & 1 ? w[h / 2] >> 16 : w[h / 2] & 0xffffu;
  }
  __device__ __forceinline__ void set(int h, uint32_t x) {  // x's low half
    w[h / 2] = __byte_perm(w[h / 2], x, h & 1 ? 0x5410 : 0x3254);
  }
  __device__ __forceinline__ uint2 entry(int i) const {  // of the four channels
    return make_uint2(get(i) | get(W + i) << 16, get(2 * W + i) | get(3 * W + i) << 16);
  }
  __device__ __forceinline__ void set_entry(int i, uint2 x) {
    set(i, x.x);
    set(W + i, x.x >> 16);
    set(2 * W + i, x.y);
    set(3 * W + i, x.y >> 16);
  }
};

template <int W>
__global__ void __launch_bounds__(kPcThreads, 6) kda_prefill_conv_kernel(const ConvParams p) {
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
  const bool active = group < 3 * D / 4;
  const int ch = active ? 4 * group : 0, part = ch / D, hc = ch - part * D;
  const int first = blockIdx.x * p.run;
  const int past = mp.n_tokens - first > p.run ? first + p.run : mp.n_tokens;
  Four w[4], bias;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = unpack4(__ldg(reinterpret_cast<const uint2 *>(p.w + (long long)(part * 4 + i) * D + hc)));
  bias = unpack4(p.bias != nullptr ? __ldg(reinterpret_cast<const uint2 *>(p.bias + ch))
                                   : make_uint2(0, 0));
  uint16_t *out = (part == 0 ? p.q : (part == 1 ? p.k : p.v)) + hc;
  const uint16_t *x = p.x + ch;
  const auto input = [&](int t) {
    return __ldg(reinterpret_cast<const uint2 *>(x + (long long)t * (3 * D)));
  };
  int b = mp.qsl != nullptr ? find_request(mp.qsl, mp.B, first, lane) : first / mp.Q;
  for (; b < mp.B; ++b) {  // the requests that reach into this run
    const PromptRequest r = prompt_request(mp, b);
    if (r.t0 >= past) break;  // (a window without tokens lies somewhere too)
    if (r.n == 0) continue;
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
    uint2 h0, h1, h2;  // the three entries before token t
    if (starts) {
      h0 = h1 = h2 = make_uint2(0, 0);
      if (r.src >= 0) {
        Windows<W> win;
        win.load(p.window + r.src * p.slot_stride + (long long)ch * W);
        h0 = win.entry(0);
        h1 = win.entry(1);
        h2 = win.entry(2);
      }
      // entries n - 3 .. n - 1 are what the request leaves, m - 3 .. m - 1
      // its boundary's
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        const int slot = which == 0 ? r.bnd : r.dst, at = which == 0 ? r.m : r.n;
        if (slot < 0) continue;
        uint16_t *to = p.window + slot * p.slot_stride + (long long)ch * W;
        Windows<W> win;
        if (W > 3) win.load(to);  // (what the other entries hold stays)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const int j = at - 3 + i;  // >= -2: at >= 1
          win.set_entry(i, j >= 0 ? input(r.t0 + j) : (j == -1 ? h2 : h1));
        }
        win.store(to);
      }
    } else {
      h0 = input(t - 3);
      h1 = input(t - 2);
      h2 = input(t - 1);
    }
    Four s0 = unpack4(h0), s1 = unpack4(h1), s2 = unpack4(h2);
    const auto step = [&](uint2 raw, int at) {
      const Four in = unpack4(raw);
      // in tap order, as in kda_layer_prologue
      Four z{ffma2(s0.a, w[0].a, bias.a), ffma2(s0.b, w[0].b, bias.b)};
      z = Four{ffma2(s1.a, w[1].a, z.a), ffma2(s1.b, w[1].b, z.b)};
      z = Four{ffma2(s2.a, w[2].a, z.a), ffma2(s2.b, w[2].b, z.b)};
      z = Four{ffma2(in.a, w[3].a, z.a), ffma2(in.b, w[3].b, z.b)};
      *reinterpret_cast<uint2 *>(out + (long long)at * D) =
          make_uint2(silu_pair(z.a), silu_pair(z.b));
      s0 = s1;
      s1 = s2;
      s2 = in;
    };
    // kAhead tokens are asked for at a time
    for (; end - t >= kAhead; t += kAhead) {
      uint2 raw[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) raw[i] = input(t + i);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) step(raw[i], t + i);
    }
    for (; t < end; ++t) step(input(t), t);
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
  p.H = H;
  p.q = q;
  p.k = k;
  p.v = v;
  p.maps = kda::make_prompt_maps(sources, destinations, boundaries, boundary_lens,
                                 query_start_loc, n_tokens, n_slots, B, Q, null_slot, status);
  const int channels = (3 * H * KDA_HEAD_DIM / 4 + kda::kPcThreads - 1) / kda::kPcThreads;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  const int sms = kda::device_sm_count(dev);
  if (sms < 1) return KDA_ERR_CUDA;
  // Long runs where they leave every SM its fill (16384 tokens, 32 heads: 171
  // us by runs of 16 tokens, 153 by 32, 147 by 64); a few tokens are a chain of
  // loads, and run side by side (37 tokens: 7 us by 4, 13 by 16); and so do short
  // windows (4096 of one token: 281 us by runs of 8, 294 by 64; 512 of three: 53
  // by 16, 60 by 64).
  int run = 64;
  while (run > 4 && ((long long)((n_tokens - 1) / run + 1) * channels < 4 * sms ||
                     run > 8LL * n_tokens / B))
    run /= 2;
  p.run = run;
  const dim3 grid((n_tokens - 1) / run + 1, channels);
  const auto kernel = [&] {
    switch (conv_width) {
      case 3: return kda::kda_prefill_conv_kernel<3>;
      case 4: return kda::kda_prefill_conv_kernel<4>;
      case 5: return kda::kda_prefill_conv_kernel<5>;
      case 6: return kda::kda_prefill_conv_kernel<6>;
      case 7: return kda::kda_prefill_conv_kernel<7>;
      case 8: return kda::kda_prefill_conv_kernel<8>;
      case 9: return kda::kda_prefill_conv_kernel<9>;
      default: return kda::kda_prefill_conv_kernel<10>;
    }
  }();
  static_assert(KDA_MAX_WINDOW + 2 == 10, "an instance for every width");
  kernel<<<grid, kda::kPcThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// kda_prefill: the gated delta rule over ragged prompts, in chunks of 64
// tokens (kda_prefill.cuh).  Five kernels: the list of chunks, what each
// needs of itself (the preparation, all chunks at once), the chain of each
// (request, head) through its chunks, token by token what is too short for a
// chunk, or inert, and once more what the chain's parts did not hold.
#include <cuda_runtime.h>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prefill.cuh"

namespace kda {
namespace {

// Windows of at most so many tokens go through the token-by-token kernel, where
// a call has none longer: 40 tokens of 1 / 4 / 32 requests of 32 heads take 30 /
// 36 / 159 us there and 38 / 40 / 161 as a chunk each, 48 tokens 34 / 41 / 189
// and 36 / 40 / 161.  Beside longer ones fewer, since that kernel finds room
// only as the chain ends: prompts of 63 x 24 and 2000 tokens take 292 us with
// 24 and 337 with 16 in its place, 37 and 5 x 1600 tokens 368 with 24 and 385
// with 40.
constexpr int kShortLen = 40, kMixedLen = 24;
constexpr int kListThreads = 1024;

// Segments: where a call has far fewer (request, head) items than there are
// SMs, the chain of a long prompt leaves the others idle, and the preparation
// of the next segment runs there meanwhile.  A chunk takes an SM of the chain
// some 3 us, and one of the preparation 6: up to a quarter of the SMs' items,
// the rest of the SMs prepare two chunks of each while the chain goes through
// one, and a segment can be twice the one before it.  Then the chain starts
// after a short first one, and there are few.  With more items the chain fills
// the GPU by itself, and a segment only costs its launches and the state's way
// through memory.  One prompt of 16384 tokens, us in one segment / in eight of
// 32 chunks / in four from 18 chunks on: 8 heads 757 / 818 / 751, 32 heads 1022 /
// 932 / 845, 48 heads 1197 / 1046 / 1171, 64 heads 1384 / 1455 / 1613.  (The
// workspace's size depends on it, so it goes by the SMs of a GB300, not of the
// device at hand.)
constexpr int kSms = 152;
constexpr int kSegItems = 3 * kSms / 8, kSegChunks = 32, kMaxSegments = 16;
constexpr int kSegDoubleItems = kSms / 4, kSegFirst = 16;

struct Workspace {
  int64_t chunks, bases, order, lost, redo, carry, images, bytes;  // offsets
  int64_t max_chunks;
};

// Of windows of up to Q tokens.  Chunks end at a request's boundary (if there
// are any) and at its end, so a request of n tokens has at most n / 64 + 2 (+ 1),
// and one with any has more than kMixedLen.  A call without windows longer than
// kShortLen has none.
Workspace workspace_layout(int64_t n_tokens, int64_t B, int64_t H, int64_t Q, bool boundaries) {
  const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  const int64_t longest = Q < n_tokens ? Q : n_tokens, cuts = boundaries ? 2 : 1;
  Workspace w = {};
  if (longest <= kShortLen || B < 1) return w;
  const int64_t most = n_tokens / (kMixedLen + 1), with = B == 1 || B < most ? B : most;
  const int64_t by_tokens = n_tokens / kChunk + cuts * with;
  const int64_t by_windows = with * ((longest - 1) / kChunk + cuts);
  w.max_chunks = by_windows < by_tokens ? by_windows : by_tokens;
  w.chunks = 256;
  const bool segments = B * H <= kSegItems;
  w.bases = up(w.chunks + w.max_chunks * (int64_t)sizeof(PrefillChunk));
  w.order = up(w.bases + B * 4 * (segments ? kMaxSegments : 1));
  w.lost = up(w.order + B * (int64_t)sizeof(PrefillRequest));
  w.redo = up(w.lost + (segments ? B * H * 4 : 0));
  w.carry = up(w.redo + B * H * (int64_t)sizeof(PrefillRedo));
  w.images = up(w.carry + (segments ? B * H * kDim * kDim * 4 : 0));
  w.bytes = w.images + w.max_chunks * H * (int64_t)kImgBytes;
  return w;
}

__device__ __forceinline__ int chunks_of(int n) { return (n + kChunk - 1) / kChunk; }

// `mine` chunks of every lane's request, from its chunk `done` on, to the list
// at `at`: a warp writes those of its 32 requests one after the other.
__device__ __forceinline__ void write_chunks(const PrefillParams &p, int at, int mine, int done,
                                             int t0, int first, int m, int n) {
  const int lane = threadIdx.x & 31;
  uint32_t some = __ballot_sync(0xffffffffu, mine > 0);
  while (some != 0) {
    const int l = __ffs(some) - 1;
    some &= some - 1;
    const int f = __shfl_sync(0xffffffffu, first, l), c = __shfl_sync(0xffffffffu, mine, l);
    const int w = __shfl_sync(0xffffffffu, at, l), t = __shfl_sync(0xffffffffu, t0, l);
    const int mm = __shfl_sync(0xffffffffu, m, l), nn = __shfl_sync(0xffffffffu, n, l);
    for (int j = lane; j < c; j += 32) {
      const int k = done + j;  // the request's chunk
      const int from = k < f ? k * kChunk : mm + (k - f) * kChunk;
      const int end = k < f ? mm : nn;
      p.chunks[w + j] = PrefillChunk{t + from, min(kChunk, end - from)};
    }
  }
}

// The same as below for up to 32 requests, a lane each: no barriers, and no
// second look at the requests (4 prompts: 3.7 us against 6.7).
__global__ void __launch_bounds__(32) kda_prefill_list_warp_kernel(const PrefillParams p) {
  const int b = threadIdx.x, B = p.r.maps.B;
  grid_launch_dependents();
  int first = 0, rest = 0, t0 = 0, m = 0, n = 0;
  if (b < B) {
    const PromptRequest r = prompt_request(p.r.maps, b);
    if (r.error != KDA_OK) report(p.r.maps.status, r.error);
    if (r.n > p.short_len && r.dst >= 0) {
      t0 = r.t0;
      n = r.n;
      m = r.m;
      first = chunks_of(m);
      rest = chunks_of(n - m);
    }
  }
  const int all = first + rest;
  int kept = all, place = 0;  // longest first
  for (int l = 0; l < B; ++l) {
    const int other = __shfl_sync(0xffffffffu, all, l);
    place += other > all || (other == all && l < b);
  }
  long long base = 0, start = 0;
  int room = p.max_chunks;  // the list ends where the first request was cut off
  for (int seg = 0; seg < p.segments; ++seg) {
    const int done = seg_from(p, seg);
    int mine = min(max(all - done, 0), seg_from(p, seg + 1) - done);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (b >= o) inc += y;
    }
    if (b == 0) p.seg_first[seg] = (int)min(base, (long long)room);
    const long long at = base + inc - mine;
    base += __shfl_sync(0xffffffffu, inc, 31);
    // (cut off where windows that overlap ask for more than there is room for)
    const bool fits = at + mine <= room;
    if (!fits) {
      report(p.r.maps.status, KDA_ERR_ARG);
      mine = 0;
      kept = min(kept, done);
    }
    const uint32_t cut = __ballot_sync(0xffffffffu, !fits);
    if (cut != 0)
      room = (int)min((long long)room, __shfl_sync(0xffffffffu, at, __ffs(cut) - 1));
    if (seg == 0) start = fits ? at : -1;
    if (b < B) p.bases[seg * B + b] = fits ? (int)at : -1;
    write_chunks(p, (int)at, mine, done, t0, first, m, n);
  }
  if (b == 0) p.seg_first[p.segments] = (int)min(base, (long long)room);
  if (b == 0) *p.n_redo = 0;
  if (b < B) p.order[place] = PrefillRequest{b, kept, first, (int)start};
}

// One CTA: the chunks of every request, by segment and then in order of the
// requests, and the requests by falling number of chunks (a counting sort: the
// chain's longest items start first).
__global__ void __launch_bounds__(kListThreads) kda_prefill_list_kernel(const PrefillParams p) {
  __shared__ long long warp_sums[kListThreads / 32];  // (windows may overlap: no bound on a sum)
  __shared__ int bins[kListThreads];
  __shared__ int room;  // the list ends where the first request was cut off
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.r.maps.B;
  grid_launch_dependents();
  bins[tid] = 0;
  if (tid == 0) room = p.max_chunks;
  __syncthreads();
  long long base = 0;
  for (int seg = 0; seg < p.segments; ++seg) {
    if (tid == 0) p.seg_first[seg] = (int)min(base, (long long)room);
    for (int b0 = 0; b0 < B; b0 += kListThreads) {
      const int b = b0 + tid;
      int first = 0, rest = 0, t0 = 0, m = 0, n = 0;
      if (b < B) {
        const PromptRequest r = prompt_request(p.r.maps, b);
        if (seg == 0 && r.error != KDA_OK) report(p.r.maps.status, r.error);
        if (r.n > p.short_len && r.dst >= 0) {
          t0 = r.t0;
          n = r.n;
          m = r.m;
          first = chunks_of(m);
          rest = chunks_of(n - m);
        }
      }
      // (the last segment takes what is left: there is nothing where Q is kept)
      const int done = seg_from(p, seg), all = first + rest;
      int mine = min(max(all - done, 0), seg_from(p, seg + 1) - done);
      long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) warp_sums[warp] = inc;
      __syncthreads();
      long long s = warp_sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      const long long total = __shfl_sync(0xffffffffu, s, 31);
      const long long before = warp > 0 ? __shfl_sync(0xffffffffu, s, warp - 1) : 0;
      const long long at = base + before + inc - mine;
      base += total;
      // (windows that overlap can ask for more chunks than there is room for:
      // such a request is cut off, and reported)
      const bool fits = at + mine <= p.max_chunks;
      if (!fits) {
        report(p.r.maps.status, KDA_ERR_ARG);
        mine = 0;
        if (at < p.max_chunks) atomicMin(&room, (int)at);
      }
      if (b < B) {
        p.bases[seg * B + b] = fits ? (int)at : -1;
        if (seg == 0) atomicAdd(&bins[min(all, kListThreads - 1)], 1);
      }
      write_chunks(p, (int)at, mine, done, t0, first, m, n);
      __syncthreads();
    }
  }
  if (tid == 0) p.seg_first[p.segments] = (int)min(base, (long long)room);
  if (tid == 0) *p.n_redo = 0;
  // bins, longest first -> where each begins
  const int bin = kListThreads - 1 - tid;
  const int mine = bins[bin];
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int s = (int)warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  bins[bin] = inc - mine + (warp > 0 ? __shfl_sync(0xffffffffu, s, warp - 1) : 0);
  __syncthreads();
  for (int b = tid; b < B; b += kListThreads) {
    const PromptRequest r = prompt_request(p.r.maps, b);
    PrefillRequest q{b, 0, 0, p.bases[b]};
    if (r.n > p.short_len && r.dst >= 0) {
      q.bnd_chunks = chunks_of(r.m);
      q.chunks = q.bnd_chunks + chunks_of(r.n - r.m);
    }
    const int at = atomicAdd(&bins[min(q.chunks, kListThreads - 1)], 1);
    // (cut off where there was no room)
    for (int seg = 0; seg < p.segments; ++seg)
      if (p.bases[seg * B + b] < 0) q.chunks = min(q.chunks, seg_from(p, seg));
    p.order[at] = q;
  }
}

}  // namespace
}  // namespace kda

extern "C" {

int64_t kda_prefill_workspace_bytes(int n_tokens, int B, int H) {
  return kda_prefill_workspace_bytes_for(n_tokens, B, H, n_tokens > 1 ? n_tokens : 1, 1);
}

int64_t kda_prefill_workspace_bytes_for(int n_tokens, int B, int H, int Q, int has_boundaries) {
  if (n_tokens < 0 || B < 0 || H < 1 || H > KDA_PROMPT_MAX_HEADS || Q < 1) return -1;
  return kda::workspace_layout(n_tokens, B, H, Q, has_boundaries != 0).bytes;
}

int kda_prefill(const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v, const kda_bf16 *raw_g,
                const kda_bf16 *raw_beta, const float *A_log, const float *dt_bias,
                float lower_bound, float q_scale, void *state_pool, int state_dtype,
                int64_t slot_stride, int n_slots, const int32_t *sources,
                const int32_t *destinations, const int32_t *boundaries,
                const int32_t *boundary_lens, const int32_t *query_start_loc, int n_tokens,
                kda_bf16 *out, void *workspace, int64_t workspace_bytes, int B, int H, int Q,
                int null_slot, int32_t *status, void *stream) {
  if (state_dtype != KDA_STATE_F32 && state_dtype != KDA_STATE_BF16) return KDA_ERR_UNSUPPORTED;
  if (!kda::prompt_gate_ok(lower_bound)) return KDA_ERR_UNSUPPORTED;
  int rc = kda::check_prompt_maps(sources, destinations, boundaries, boundary_lens,
                                  query_start_loc, n_tokens, n_slots, B, H, Q, null_slot);
  if (rc != KDA_OK) return rc;
  if (B == 0 || n_tokens == 0) return KDA_OK;
  rc = kda::check_rule(q, k, v, raw_g, raw_beta, A_log, dt_bias, lower_bound, q_scale, state_pool,
                       state_dtype, slot_stride, H, out);
  if (rc != KDA_OK) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = state_dtype == KDA_STATE_BF16;
  const int longest = Q < n_tokens ? Q : n_tokens;
  kda::PrefillParams p;
  p.r = kda::RecurrentParams{q, k, v, raw_g, raw_beta, A_log, dt_bias, lower_bound, q_scale,
                             state_pool, slot_stride, out, H, kda::kShortLen, false,
                             kda::make_prompt_maps(sources, destinations, boundaries,
                                                   boundary_lens, query_start_loc, n_tokens,
                                                   n_slots, B, Q, null_slot, status)};
  if (longest <= kda::kShortLen) return kda::launch_recurrent(p.r, bf16, st);
  const kda::Workspace w = kda::workspace_layout(n_tokens, B, H, Q, boundaries != nullptr);
  if (!workspace || workspace_bytes < w.bytes) return KDA_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return KDA_ERR_ALIGN;
  if (w.max_chunks * H > 0x7fffffffLL) return KDA_ERR_ARG;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  // a single request of any length is one launch less by chunks alone
  p.short_len = B == 1 ? 0 : kda::kMixedLen;
  p.max_chunks = (int)w.max_chunks;
  // the longest request's chunks: its own and one more where its boundary
  // cuts one in two
  const int most = (longest - 1) / kda::kChunk + 1 + (boundaries != nullptr ? 1 : 0);
  p.segments = 1;
  p.seg_doubles = false;
  const long long heads = (long long)B * H;
  if (heads <= kda::kSegDoubleItems && most >= 2 * kda::kSegFirst) {
    p.seg_doubles = true;
    while (p.segments < kda::kMaxSegments && kda::kSegFirst * ((2LL << p.segments) - 1) <= most)
      ++p.segments;
  } else if (heads <= kda::kSegItems && most >= 2 * kda::kSegChunks) {
    p.segments = (most + kda::kSegChunks / 2) / kda::kSegChunks;
    if (p.segments > kda::kMaxSegments) p.segments = kda::kMaxSegments;
  }
  const int parts = p.seg_doubles ? (1 << p.segments) - 1 : p.segments;
  p.seg_chunks = (most + parts - 1) / parts;
  p.seg_first = reinterpret_cast<int *>(ws);
  static_assert(4 * (kda::kMaxSegments + 1) <= 128, "n_redo behind them");
  p.n_redo = reinterpret_cast<int *>(ws + 128);
  p.lost = reinterpret_cast<int *>(ws + w.lost);
  p.redo = reinterpret_cast<kda::PrefillRedo *>(ws + w.redo);
  p.bases = reinterpret_cast<int *>(ws + w.bases);
  p.carry = reinterpret_cast<float *>(ws + w.carry);
  p.chunks = reinterpret_cast<kda::PrefillChunk *>(ws + w.chunks);
  p.order = reinterpret_cast<kda::PrefillRequest *>(ws + w.order);
  p.images = ws + w.images;
  if (B <= 32)
    kda::kda_prefill_list_warp_kernel<<<1, 32, 0, st>>>(p);
  else
    kda::kda_prefill_list_kernel<<<1, kda::kListThreads, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  // From here on each kernel is launched as the one before it starts, and
  // waits, where it needs to, for that one to end.
  for (int seg = 0; seg < p.segments; ++seg) {
    rc = kda::launch_prefill_prep(p, seg, st);
    if (rc != KDA_OK) return rc;
    rc = kda::launch_prefill_chain(p, seg, bf16, st);
    if (rc != KDA_OK) return rc;
  }
  if (p.short_len != 0) {
    p.r.beside = true;
    p.r.max_len = p.short_len;
    rc = kda::launch_recurrent(p.r, bf16, st);
    if (rc != KDA_OK) return rc;
  }
  return kda::launch_prefill_redo(p, bf16, st);
}

}  // extern "C"

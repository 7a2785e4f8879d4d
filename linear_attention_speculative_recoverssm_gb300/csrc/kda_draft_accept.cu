// Drafted tokens against the target's probabilities, and the token behind
// the accepted path.
//
// The path needs a few weights only: u_a q(x) < p(x) down a chain, running
// sums over siblings in a tree; every CTA of a request works it out for
// itself, a lane a node.  The token behind it is drawn by inverse CDF from
// one row of the target's weights (less the refused draft's row): the first i
// whose running sum exceeds s Z.  A cluster of up to 8 CTAs takes a request, each
// its share of the row; a warp adds up 512 weights at a time; the sums of
// those tiles are scanned, the CTAs' totals go round through distributed
// shared memory, and the tile with the crossing is read again.
//
// What bounds it: HBM, for the rows (each read once, but for one tile); a
// single request's half a dozen loads that depend on one another.  256 chains
// with drafts, 131072 FP32 weights (268 MB): 58 us, 4.6 TB/s (a copy: 6.7), 44%
// of the issue slots.  By events around the call 70 us behind a cache full of
// written lines, which go back to memory meanwhile, 60 behind one of read lines, 59
// a pass of eight; one request 17.  64 trees of up to 24 nodes, 100003 BF16 weights:
// 25 us for 13 MB, which no unit's rate explains: seven rounds of tiles a CTA, each
// with one tile (32 bytes a lane) on its way.
//
// Precision.  The answer is an index, which must not depend on the order of
// the sums: a row's running sums lie 1e-5 apart and less, where FP32 sums
// would be off by 1e-7.  So p - q is taken exactly (its rounding error is
// itself a float), and sums are pairs of floats (48 bits) in the tiles,
// doubles behind them: FP64 for each weight would cost more than reading it.
#include <cuda_runtime.h>

#include <type_traits>

#include "kda_launch.h"
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kDaMaxCtas = 8;  // of a request
constexpr int kDaThreads = 256;
constexpr int kDaWarps = kDaThreads / 32;
constexpr int kDaTile = 512;
constexpr int kDaPer = kDaTile / 32;  // weights a lane
constexpr int kDaOccupancy = 2;       // CTAs an SM
constexpr int kDaTiles = KDA_MAX_VOCAB / kDaTile;  // of a CTA, at most

struct AcceptParams {
  TreeMaps maps;
  const void *target, *draft;
  long long target_stride, draft_stride;
  int vocab;
  const int32_t *tokens;
  const float *u, *u_next;
  int32_t *accepted, *path, *next;
};

// A sum of floats as hi + lo, |lo| within half a unit of hi's last place or
// so (Knuth's two-sum).
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x, float err) {
    const float t = hi + x;
    const float z = t - hi;
    lo += ((hi - (t - z)) + (x - z)) + err;
    hi = t;
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

__device__ __forceinline__ float weight_at(const float *row, int i) { return __ldg(row + i); }
__device__ __forceinline__ float weight_at(const uint16_t *row, int i) {
  return bf16_bits_to_f32(__ldg(row + i));
}

// kDaPer weights of a tile: 16-byte pieces where the rows allow it, else one
// by one, lane by lane; index(j) is where a lane's j-th lies in the tile.
template <typename T, bool VEC>
struct TileAccess {
  static constexpr int kPiece = VEC ? 16 / (int)sizeof(T) : 1;
  static __device__ __forceinline__ int index(int j, int lane) {
    return (j / kPiece) * (32 * kPiece) + lane * kPiece + j % kPiece;
  }
  // as they are in memory: pieces, or a weight each
  static constexpr int kRaw = VEC ? kDaPer / kPiece : kDaPer;
  using Raw = typename std::conditional<VEC, uint4, T>::type;
  static __device__ __forceinline__ void load(const T *row, int first, int vocab, int lane,
                                              Raw (&raw)[kRaw]) {
#pragma unroll
    for (int c = 0; c < kRaw; ++c) {
      const int i = first + index(c * kPiece, lane);
      raw[c] = Raw{};
      if constexpr (VEC) {
        if (i + kPiece <= vocab) {
          raw[c] = __ldg(reinterpret_cast<const uint4 *>(row + i));
        } else if (i < vocab) {  // the row's last piece, in part
          T last[kPiece];
#pragma unroll
          for (int e = 0; e < kPiece; ++e) last[e] = i + e < vocab ? row[i + e] : T(0);
          memcpy(&raw[c], last, 16);
        }
      } else {
        if (i < vocab) raw[c] = __ldg(row + i);
      }
    }
  }
  static __device__ __forceinline__ void values(const Raw (&raw)[kRaw], float (&w)[kDaPer]) {
#pragma unroll
    for (int c = 0; c < kRaw; ++c) {
      if constexpr (VEC) {
        const uint32_t x[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int e = 0; e < kPiece; ++e)
          w[c * kPiece + e] =
              sizeof(T) == 4 ? __uint_as_float(x[e % 4])
                             : __uint_as_float(e & 1 ? x[e / 2 % 4] & 0xffff0000u
                                                     : x[e / 2 % 4] << 16);
      } else if constexpr (sizeof(T) == 4) {
        w[c] = raw[c];
      } else {
        w[c] = bf16_bits_to_f32(raw[c]);
      }
    }
  }
};

// What the CTA's warps need of the walk, and the scan's numbers.
struct AcceptSmem {
  alignas(16) int8_t parent[kTreeNodes];
  int token[kTreeNodes];
  float p[kTreeNodes];
  int last, refused;           // the path's last node; the refused child of a chain or -1
  int n_removed;
  int removed[kTreeNodes];  // tokens of the refused children of a tree
  bool ok;
  Sum2 tile[kDaTiles];
  double warp_sum[kDaWarps];
  double total[2][kDaMaxCtas];  // written by every CTA of the cluster
  int best, any;
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void store_to_rank(double *mine, int rank, double x) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(there)
               : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(there), "d"(x) : "memory");
}

// Nodes of the tree whose parent is `a`, as two words of bits.
__device__ __forceinline__ void children_of(const int8_t *parent, int a, uint32_t (&bits)[2]) {
  const uint32_t all = (uint32_t)(uint8_t)a * 0x01010101u;
  bits[0] = bits[1] = 0;
#pragma unroll
  for (int w = 0; w < kTreeNodes / 4; ++w) {
    const uint32_t eq = __vcmpeq4(reinterpret_cast<const uint32_t *>(parent)[w], all);
    bits[w / 8] |= (((eq & 0x08040201u) * 0x01010101u) >> 24) << (4 * (w % 8));
  }
}

// Warp 0: the accepted path, from the root.  False: the request's tree or
// tokens are bad.
template <typename T>
__device__ bool walk(const AcceptParams &p, const TreeRequest &r, int b, int lane, bool writes,
                     AcceptSmem &sm) {
  bool good = load_tree(p.maps, r, sm.parent, lane);
  const T *target = static_cast<const T *>(p.target), *draft = static_cast<const T *>(p.draft);
  float u[2], qx[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    u[i] = qx[i] = 0.f;
    sm.token[t] = -1;
    sm.p[t] = 0.f;
    const int a = sm.parent[t];
    if (!good || t >= r.n) continue;
    if (t == 0) {
      good = a < 0;
      continue;
    }
    const int x = p.tokens[r.t0 + t];
    if (a < 0 || x < 0 || x >= p.vocab) {
      good = false;
      continue;
    }
    sm.token[t] = x;
    u[i] = p.u[r.t0 + a];
    const float w = weight_at(target + (long long)(r.t0 + a) * p.target_stride, x);
    sm.p[t] = w > 0.f ? w : 0.f;
    if (draft != nullptr) qx[i] = weight_at(draft + (long long)(r.t0 + t) * p.draft_stride, x);
  }
  // (tokens and weights are there for the other lanes: a vote orders no memory)
  __syncwarp();
  if (!__all_sync(0xffffffffu, good)) return false;
  // (nodes past the window are nobody's children)
  const uint32_t live[2] = {r.n >= 32 ? 0xffffffffu : (1u << r.n) - 1u,
                            r.n >= 64 ? 0xffffffffu : (r.n <= 32 ? 0u : (1u << (r.n - 32)) - 1u)};
  uint32_t sib[2][2];
  bool fresh[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    children_of(sm.parent, sm.parent[t], sib[i]);
    // those before t
    sib[i][0] &= live[0] & (t >= 32 ? 0xffffffffu : (1u << t) - 1u);
    sib[i][1] &= live[1] & (t < 32 ? 0u : (1u << (t - 32)) - 1u);
    fresh[i] = t > 0 && t < r.n;
    if (fresh[i])
#pragma unroll
      for (int w = 0; w < 2; ++w)
        for (uint32_t m = sib[i][w]; m != 0; m &= m - 1)
          if (sm.token[32 * w + __ffs(m) - 1] == sm.token[t]) fresh[i] = false;
  }
  const uint32_t firsts[2] = {__ballot_sync(0xffffffffu, fresh[0]),
                              __ballot_sync(0xffffffffu, fresh[1])};
  uint32_t taken[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    bool take = false;
    if (fresh[i] && draft != nullptr) {
      // (products of floats are exact in doubles)
      take = (double)u[i] * (double)qx[i] < (double)sm.p[t];
    } else if (fresh[i]) {
      double before = 0.0;
#pragma unroll
      for (int w = 0; w < 2; ++w)
        for (uint32_t m = sib[i][w] & firsts[w]; m != 0; m &= m - 1)
          before += (double)sm.p[32 * w + __ffs(m) - 1];
      take = !((double)u[i] < before) && (double)u[i] < before + (double)sm.p[t];
    }
    taken[i] = __ballot_sync(0xffffffffu, take);
  }
  int cur = 0, n = 1, node = lane == 0 ? 0 : -1;  // lane i < 8: the path's i-th node
  uint32_t kids[2];
  const int up0 = sm.parent[lane], up1 = sm.parent[lane + 32];
  while (true) {
    kids[0] = __ballot_sync(0xffffffffu, up0 == cur) & live[0];
    kids[1] = __ballot_sync(0xffffffffu, up1 == cur) & live[1];
    const uint32_t m0 = kids[0] & taken[0], m1 = kids[1] & taken[1];
    if ((m0 | m1) == 0 || n == kTreeDepth) break;  // (no path is longer)
    cur = m0 != 0 ? __ffs(m0) - 1 : 31 + __ffs(m1);
    if (lane == n) node = cur;
    ++n;
  }
  const int n0 = __popc(kids[0]);
  int refused = -1, n_removed = 0;
  if (draft != nullptr) {
    refused = kids[0] != 0 ? __ffs(kids[0]) - 1 : -1;
  } else {
    n_removed = n0 + __popc(kids[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (kids[i] >> lane & 1u)
        sm.removed[(i ? n0 : 0) + __popc(kids[i] & ((1u << lane) - 1u))] = sm.token[lane + 32 * i];
  }
  if (lane == 0) {
    sm.last = cur;
    sm.refused = refused;
    sm.n_removed = n_removed;
  }
  if (writes) {
    if (lane == 0) p.accepted[b] = n;
    if (lane < kTreeDepth) p.path[(long long)b * kTreeDepth + lane] = node;
  }
  return true;
}

// The sums of a CTA's tiles of weights max(p - q, 0), p without the removed
// tokens, or p, a warp a tile; the next tile is on its way meanwhile.
template <typename T, bool VEC, bool DIFF>
__device__ __forceinline__ void tile_sums(const T *prow, const T *qrow, int n_removed, int vocab,
                                          int first, int tiles, AcceptSmem &sm) {
  using A = TileAccess<T, VEC>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  typename A::Raw p_raw[A::kRaw], q_raw[A::kRaw];
  const auto ask = [&](int i) {
    A::load(prow, (first + i) * kDaTile, vocab, lane, p_raw);
    if (DIFF) A::load(qrow, (first + i) * kDaTile, vocab, lane, q_raw);
  };
  if (warp < tiles) ask(warp);
  for (int i = warp; i < tiles; i += kDaWarps) {
    float w[kDaPer], q[kDaPer];
    A::values(p_raw, w);
    if (DIFF) A::values(q_raw, q);
    if (i + kDaWarps < tiles) ask(i + kDaWarps);
    if (!DIFF) {
#pragma unroll
      for (int j = 0; j < kDaPer; ++j) w[j] = w[j] > 0.f ? w[j] : 0.f;
      for (int k = 0; k < n_removed; k += 32) {
        const int x = k + lane < n_removed ? sm.removed[k + lane] : -1;
        for (uint32_t m = __ballot_sync(0xffffffffu, x >= 0 && x / kDaTile == first + i); m != 0;
             m &= m - 1) {
          const int at = __shfl_sync(0xffffffffu, x, __ffs(m) - 1) % kDaTile;
#pragma unroll
          for (int j = 0; j < kDaPer; ++j)
            if (A::index(j, lane) == at) w[j] = 0.f;
        }
      }
    }
    Sum2 s{0.f, 0.f}, s2{0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kDaPer; ++j) {
      float x = w[j], err = 0.f;
      if (DIFF) {
        // (what the difference's rounding leaves out is itself a float)
        const float d = w[j] - q[j];
        const bool more = w[j] > q[j];
        err = more ? (w[j] - d) - q[j] : 0.f;
        x = more ? d : 0.f;
      }
      if (j % 2) {
        s2.add(x, err);
      } else {
        s.add(x, err);
      }
    }
    s.add(s2.hi, s2.lo);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const float hi = __shfl_xor_sync(0xffffffffu, s.hi, o);
      const float lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
      s.add(hi, lo);
    }
    if (lane == 0) sm.tile[i] = s;
  }
}

// Sums of the doubles of threads 0 .. t, for every thread t of the CTA.
__device__ __forceinline__ double block_scan(double x, AcceptSmem &sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm.warp_sum[warp] = x;
  __syncthreads();
  double before = 0.0;
  for (int i = 0; i < warp; ++i) before += sm.warp_sum[i];
  __syncthreads();
  return before + x;
}

template <typename T>
__global__ void __launch_bounds__(kDaThreads, kDaOccupancy)
    kda_draft_accept_kernel(const AcceptParams p, int ctas) {
  __shared__ AcceptSmem sm;
  const TreeMaps &mp = p.maps;
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int tid = threadIdx.x, lane = tid & 31;
  cluster_arrive();  // waited for before the first store to another CTA
  const TreeRequest r = tree_request(mp, b);
  const bool live = r.error == KDA_OK && r.slot >= 0 && r.n > 0;
  if (tid < 32) {
    const bool ok = live && walk<T>(p, r, b, lane, rank == 0, sm);
    if (lane == 0) {
      sm.ok = ok;
      sm.best = 0x7fffffff;
      sm.any = -1;
    }
    if (!ok && rank == 0) {
      if (lane == 0) {
        if (live || r.error != KDA_OK) report(mp.status, KDA_ERR_ARG);
        p.accepted[b] = 0;
        p.next[b] = -1;
      }
      if (lane < kTreeDepth) p.path[(long long)b * kTreeDepth + lane] = -1;
    }
  }
  __syncthreads();
  if (!sm.ok) {  // (every CTA of the request alike)
    cluster_wait();
    return;
  }
  const T *prow = static_cast<const T *>(p.target) + (long long)(r.t0 + sm.last) * p.target_stride;
  const T *qrow = sm.refused < 0 ? nullptr
                                 : static_cast<const T *>(p.draft) +
                                       (long long)(r.t0 + sm.refused) * p.draft_stride;
  int n_removed = sm.n_removed;
  const bool vec = ((reinterpret_cast<uintptr_t>(prow) | reinterpret_cast<uintptr_t>(qrow)) & 15) == 0;
  const int all = (p.vocab + kDaTile - 1) / kDaTile, per = (all + ctas - 1) / ctas;
  const int first = rank * per;
  const int tiles = first >= all ? 0 : (all - first < per ? all - first : per);
  const int each = (tiles + kDaThreads - 1) / kDaThreads;
  double mine, upto, before, whole, goal;
  int owner, pass = 0;
  for (;; ++pass) {
    if (qrow != nullptr) {
      if (vec) {
        tile_sums<T, true, true>(prow, qrow, 0, p.vocab, first, tiles, sm);
      } else {
        tile_sums<T, false, true>(prow, qrow, 0, p.vocab, first, tiles, sm);
      }
    } else if (vec) {
      tile_sums<T, true, false>(prow, qrow, n_removed, p.vocab, first, tiles, sm);
    } else {
      tile_sums<T, false, false>(prow, qrow, n_removed, p.vocab, first, tiles, sm);
    }
    __syncthreads();
    // a thread takes `each` tiles, one after the other
    mine = 0.0;
    for (int i = tid * each; i < (tid + 1) * each && i < tiles; ++i) mine += sm.tile[i].value();
    upto = block_scan(mine, sm);
    if (pass == 0) cluster_wait();
    if (tid == kDaThreads - 1)
#pragma unroll 1
      for (int i = 0; i < ctas; ++i) store_to_rank(&sm.total[pass][rank], i, upto);
    cluster_arrive();
    cluster_wait();
    // the same in every CTA: the total, and whose share holds the crossing
    whole = 0.0;
    for (int i = 0; i < ctas; ++i) whole += sm.total[pass][i];
    if (whole > 0.0 || pass == 1 || (qrow == nullptr && n_removed == 0)) break;
    qrow = nullptr;  // nothing is left without them: p itself
    n_removed = 0;
  }
  if (!(whole > 0.0 && whole <= 1.7976931348623157e308)) {
    if (rank == 0 && tid == 0) {
      report(mp.status, KDA_ERR_ARG);
      p.next[b] = -1;
    }
    return;
  }
  float s = p.u_next[b];
  s = s > 0.f ? s : 0.f;
  goal = (double)s * whole;
  // (a running sum that rounding leaves below: the last weight above zero)
  owner = -1;
  double sum = 0.0;
  before = 0.0;
#pragma unroll 1
  for (int i = 0; i < ctas; ++i) {
    const double t = sm.total[pass][i];
    if (t > 0.0) {
      owner = i;
      before = sum;
    }
    sum += t;
    if (t > 0.0 && sum > goal) break;
  }
  if (owner != rank) return;
  // the tile of the crossing, among the thread's
  double from = before + (upto - mine);
  for (int i = tid * each; i < (tid + 1) * each && i < tiles; ++i) {
    const bool some = sm.tile[i].hi > 0.f;
    from += sm.tile[i].value();
    if (some && from > goal) {
      atomicMin(&sm.best, i);
      break;
    }
    if (some) atomicMax(&sm.any, i);
  }
  __syncthreads();
  const int tile = sm.best != 0x7fffffff ? sm.best : sm.any;
  // (what lies before it, from the thread that has the sum)
  if (tid == tile / each) {
    from = before + (upto - mine);
    for (int i = tid * each; i < tile; ++i) from += sm.tile[i].value();
    sm.warp_sum[0] = from;
  }
  __syncthreads();
  const double start = sm.warp_sum[0];
  if (tid == 0) {
    sm.best = 0x7fffffff;
    sm.any = -1;
  }
  __syncthreads();
  // its weights again, two a thread, in their order
  double w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = (first + tile) * kDaTile + 2 * tid + j;
    w[j] = 0.0;
    if (i < p.vocab) {
      const float x = weight_at(prow, i), y = qrow != nullptr ? weight_at(qrow, i) : 0.f;
      bool out = !(x > y);
      for (int k = 0; k < n_removed; ++k) out = out || sm.removed[k] == i;
      if (!out) w[j] = (double)x - (double)y;
    }
  }
  const double end = block_scan(w[0] + w[1], sm);
  const double at[2] = {start + (end - w[1]), start + end};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = (first + tile) * kDaTile + 2 * tid + j;
    if (w[j] > 0.0 && at[j] > goal) atomicMin(&sm.best, i);
    if (w[j] > 0.0) atomicMax(&sm.any, i);
  }
  __syncthreads();
  if (tid == 0) p.next[b] = sm.best != 0x7fffffff ? sm.best : sm.any;
}

}  // namespace
}  // namespace kda

extern "C" int kda_draft_accept(const void *target, const void *draft, int probs_dtype,
                                int64_t target_row_stride, int64_t draft_row_stride, int vocab,
                                const int32_t *tokens, const int32_t *parents,
                                const float *accept_uniforms, const float *sample_uniforms,
                                const int32_t *state_slots, const int32_t *query_start_loc,
                                int n_tokens, int32_t *accepted, int32_t *path,
                                int32_t *next_tokens, int B, int Q, int null_slot,
                                int32_t *status, void *stream) {
  kda::AcceptParams p;
  p.maps = kda::TreeMaps{parents, state_slots, nullptr, nullptr, query_start_loc, n_tokens,
                         0x7fffffff, 0x7fffffff, 1, B, Q, null_slot, status};
  if (const int rc = kda::check_tree_maps(p.maps, 1); rc != KDA_OK) return rc;
  if (probs_dtype != KDA_PROBS_F32 && probs_dtype != KDA_PROBS_BF16) return KDA_ERR_UNSUPPORTED;
  if (parents == nullptr ? Q > KDA_TREE_MAX_DEPTH : draft != nullptr) return KDA_ERR_ARG;
  if (vocab < 1 || vocab > KDA_MAX_VOCAB) return KDA_ERR_ARG;
  if (B == 0) return KDA_OK;
  if (B > 0x7fffffff / kda::kDaMaxCtas) return KDA_ERR_ARG;
  if (!sample_uniforms || !accepted || !path || !next_tokens) return KDA_ERR_ARG;
  if (n_tokens > 0 && (!target || !tokens || !accept_uniforms)) return KDA_ERR_ARG;
  if (target_row_stride < vocab || (draft != nullptr && draft_row_stride < vocab))
    return KDA_ERR_ARG;
  const uintptr_t mask = probs_dtype == KDA_PROBS_F32 ? 3 : 1;
  if (((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft)) & mask) != 0)
    return KDA_ERR_ALIGN;
  p.target = target;
  p.draft = draft;
  p.target_stride = target_row_stride;
  p.draft_stride = draft_row_stride;
  p.vocab = vocab;
  p.tokens = tokens;
  p.u = accept_uniforms;
  p.u_next = sample_uniforms;
  p.accepted = accepted;
  p.path = path;
  p.next = next_tokens;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  const int sms = kda::device_sm_count(dev);
  // As many CTAs a request as run all at once, two to an SM.  131072 FP32 weights
  // and drafts, us by 1 / 2 / 4 / 8 CTAs a request: 64 requests 54 / 38 / 33 / 40,
  // 128 requests 58 / 48 / 48 / 62, 256 requests 72 / 72 / 81 / 97.
  int ctas = kda::kDaMaxCtas;
  while (ctas > 1 && (long long)B * ctas > (long long)kda::kDaOccupancy * sms) ctas /= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * ctas));
  cfg.blockDim = dim3(kda::kDaThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      probs_dtype == KDA_PROBS_F32
          ? cudaLaunchKernelEx(&cfg, kda::kda_draft_accept_kernel<float>, p, ctas)
          : cudaLaunchKernelEx(&cfg, kda::kda_draft_accept_kernel<uint16_t>, p, ctas);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

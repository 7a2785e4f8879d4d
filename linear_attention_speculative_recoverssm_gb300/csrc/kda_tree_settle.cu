// Which requests of a step of trees go on to kda_tree_select and
// kda_defer_commit, and which are left as they were before the step.
//
// kda_tree_verify leaves a request that it reports alone: its replay is still
// pending.  A pending count of zero behind such a step would lose the tokens
// accepted before it, so those requests get no record row here, and what
// follows passes them by.  Where the replays were folded in otherwise (a flush),
// such a request keeps its row, and nothing of the step is accepted.  Nor is
// anything of a path that records or windows cannot hold: its count as the
// pending one would replay what an earlier step left in the records.
//
// A warp a request, integer work only.  What bounds it is latency: two or three
// loads that depend on one another, and walks up the tree in shared memory.  One
// request to 256 of 64 nodes take 6 us by events around the call, trees and paths
// at once, or 4096 requests, 8; the launch and the events are some 5 of them.
#include <cuda_runtime.h>

#include "kda_launch.h"
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kTlWarps = 8;

struct TreeSettleParams {
  TreeMaps maps;
  const int32_t *served, *path;
  int32_t *accepted, *rows;
  int most;  // the longest path that fits
  bool folded;
};

__global__ void __launch_bounds__(32 * kTlWarps) kda_tree_settle_kernel(const TreeSettleParams p) {
  __shared__ int8_t parents[kTlWarps][kTreeNodes];
  const TreeMaps &mp = p.maps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x * kTlWarps + warp;
  if (b >= mp.B) return;
  const int slot = mp.state_slots[b];
  const int row = mp.record_rows != nullptr ? mp.record_rows[b] : b;
  int to = row, count = p.accepted != nullptr ? p.accepted[b] : 0;
  bool ok = true;
  if (slot > mp.null_slot && row >= 0) {
    const TreeRequest r = tree_request(mp, b);
    const bool left = p.served != nullptr && p.served[b] < 0;
    ok = !left && r.error == KDA_OK &&
         (mp.parents == nullptr || load_tree(mp, r, parents[warp], lane));
    if (!ok) {
      if (left || !p.folded || slot >= mp.n_slots || row >= mp.n_rows) to = -1;
    } else if (p.path != nullptr) {
      bool fits = count >= 0 && count <= p.most;
      if (fits && lane < count) {
        const int t = p.path[(long long)b * kTreeDepth + lane];
        fits = t >= 0 && t < r.n;
      }
      ok = __all_sync(0xffffffffu, fits);
    }
    if (!ok) count = 0;
  }
  __syncwarp();  // (`rows` may be `served` or record_rows: all lanes have read)
  if (lane != 0) return;
  if (!ok) report(mp.status, KDA_ERR_ARG);
  p.rows[b] = to;
  if (p.accepted != nullptr) p.accepted[b] = count;
}

}  // namespace
}  // namespace kda

extern "C" int kda_tree_settle(const int32_t *path, int32_t *accepted, int most,
                               const int32_t *state_slots, int n_slots,
                               const int32_t *record_rows, const int32_t *served, int n_rows,
                               const int32_t *parents, const int32_t *query_start_loc,
                               int n_tokens, int folded, int32_t *rows, int B, int Q,
                               int null_slot, int32_t *status, void *stream) {
  kda::TreeSettleParams p;
  p.maps = kda::TreeMaps{parents, state_slots, record_rows, nullptr, query_start_loc,
                         n_tokens, n_slots, n_rows, 1, B, Q, null_slot, status};
  if (const int rc = kda::check_tree_maps(p.maps, 1); rc != KDA_OK) return rc;
  if (B == 0) return KDA_OK;
  if (!state_slots || !rows || n_slots < 1 || n_rows < 1 || (record_rows == nullptr && n_rows < B))
    return KDA_ERR_ARG;
  if (path != nullptr && (accepted == nullptr || most < 0 || most > KDA_TREE_MAX_DEPTH))
    return KDA_ERR_ARG;
  p.path = path;
  p.most = most;
  p.served = served;
  p.accepted = accepted;
  p.rows = rows;
  p.folded = folded != 0;
  const unsigned ctas = ((unsigned)B + kda::kTlWarps - 1) / kda::kTlWarps;
  kda::kda_tree_settle_kernel<<<ctas, 32 * kda::kTlWarps, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

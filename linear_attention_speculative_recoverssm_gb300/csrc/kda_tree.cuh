// What the tree operators share (kda_tree_conv, kda_tree_verify,
// kda_draft_accept, kda_tree_select): a request's window, its tree and its
// slots, and their checks.
#pragma once

#include "kda_device.cuh"

namespace kda {

constexpr int kTreeNodes = KDA_TREE_MAX_NODES;
constexpr int kTreeDepth = KDA_TREE_MAX_DEPTH;
static_assert(kTreeNodes == 64, "a warp's lanes take two nodes each");

// Windows and slots of every request of a call.
struct TreeMaps {
  const int32_t *parents;      // [n_tokens], within the request; nullptr: a chain
  const int32_t *state_slots;  // [B] or nullptr (every request is live)
  const int32_t *record_rows;  // [B] or nullptr (row b)
  const int32_t *pending;      // [n_rows] or nullptr (no replay pending)
  const int32_t *qsl;          // [B + 1] or nullptr (windows of Q tokens)
  int n_tokens, n_slots, n_rows, rq, B, Q, null_slot;
  int32_t *status;
};

// One request: its window t0 .. t0 + n - 1, its slot (-1: inert), its record
// row (-1: none) and its pending count (0 .. rq).
struct TreeRequest {
  int t0, n, slot, row, pending;
  int error;  // KDA_OK or what to report
};

// A bad window ends it, or where none is needed is an empty one, error set.
__device__ __forceinline__ TreeRequest tree_request(const TreeMaps &p, int b,
                                                    bool needs_window = true) {
  TreeRequest r;
  r.error = KDA_OK;
  r.slot = r.row = -1;
  r.pending = 0;
  if (p.qsl != nullptr) {
    r.t0 = p.qsl[b];
    const long long end = p.qsl[b + 1];
    const long long n = end - r.t0;
    if (r.t0 < 0 || n < 0 || n > p.Q || end > p.n_tokens) {
      r.error = KDA_ERR_ARG;
      r.t0 = r.n = 0;
      if (needs_window) return r;
    } else {
      r.n = (int)n;
    }
  } else {
    r.t0 = b * p.Q;
    r.n = p.Q;
  }
  const int slot = p.state_slots != nullptr ? p.state_slots[b] : p.null_slot + 1;
  if (slot <= p.null_slot) return r;
  const int row = p.record_rows != nullptr ? p.record_rows[b] : b;
  if (slot >= p.n_slots || row >= p.n_rows) {
    r.error = KDA_ERR_ARG;
    r.n = 0;
    return r;
  }
  r.slot = slot;
  r.row = row < 0 ? -1 : row;
  if (p.pending != nullptr && r.row >= 0) {
    const int n = p.pending[r.row];
    r.pending = n < 0 ? 0 : (n > p.rq ? p.rq : n);
  }
  return r;
}

// Depth of node t (1: hangs on the checkpoint) in a tree whose parents (all
// below their children, -1 or more) are in shared memory; kTreeDepth + 1 for
// anything deeper.
__device__ __forceinline__ int tree_depth(const int8_t *parent, int t) {
  int d = 0;
  for (int a = t; a >= 0 && d <= kTreeDepth; a = parent[a]) ++d;
  return d;
}

// The request's parents into shared memory (entries n .. kTreeNodes - 1: -1),
// by one warp; true where they are a tree: parent[t] in -1 .. t - 1 and no
// path of more than kTreeDepth tokens.
__device__ __forceinline__ bool load_tree(const TreeMaps &p, const TreeRequest &r,
                                          int8_t *parent, int lane) {
  bool good = true;
  __syncwarp();  // (the tree that was there before is read)
#pragma unroll
  for (int i = 0; i < kTreeNodes / 32; ++i) {
    const int t = lane + 32 * i;
    int a = -1;
    if (t < r.n) {
      a = p.parents != nullptr ? p.parents[r.t0 + t] : t - 1;
      if (a < -1 || a >= t) {
        good = false;
        a = -1;
      }
    }
    parent[t] = (int8_t)a;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kTreeNodes / 32; ++i) {
    const int t = lane + 32 * i;
    if (t < r.n) good = good && tree_depth(parent, t) <= kTreeDepth;
  }
  return __all_sync(0xffffffffu, good);
}

// Host-side checks of the maps (before the operator's own).  A (token, head)
// row number fits 31 bits; byte and element offsets are 64-bit.
inline int check_tree_maps(const TreeMaps &m, int H) {
  if (m.B < 0 || H < 1 || H > KDA_PROMPT_MAX_HEADS || m.Q < 1 || m.Q > kTreeNodes ||
      m.n_tokens < 0 || m.null_slot < -1)
    return KDA_ERR_ARG;
  if (m.B == 0) return KDA_OK;
  if ((long long)m.B * H > 0x7fffffffLL || (long long)m.n_tokens * H > 0x7fffffffLL)
    return KDA_ERR_ARG;
  if (m.qsl == nullptr && (long long)m.n_tokens != (long long)m.B * m.Q) return KDA_ERR_ARG;
  return KDA_OK;
}

inline bool tree_aligned16(const void *ptr) {
  return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0;
}

}  // namespace kda

// What the prompt operators share (kda_prefill_conv, kda_prefill,
// kda_recurrent): a request's window, the slots its state is read from and
// written to, and their checks.
#pragma once

#include "kda_device.cuh"

namespace kda {

// Slots of every request of a call, and the packed windows' bounds.
struct PromptMaps {
  const int32_t *sources, *destinations;  // [B]
  const int32_t *bnd_slots, *bnd_lens;    // [B] or nullptr
  const int32_t *qsl;                     // [B + 1] or nullptr (windows of Q tokens)
  int n_tokens, n_slots, B, Q, null_slot;
  int32_t *status;
};

// One request: its window t0 .. t0 + n - 1 and its slots.  `n` is 0 for a
// request of which nothing is read or written (an empty window, or one that
// was reported).  src < 0: it starts from the zero state.  dst < 0: inert,
// only its outputs are written (zeros).  bnd < 0: no boundary state; else
// the state after `m` <= n tokens goes to slot bnd.
struct PromptRequest {
  int t0, n, src, dst, bnd, m;
  int error;  // KDA_OK or what to report
};

__device__ __forceinline__ PromptRequest prompt_request(const PromptMaps &p, int b) {
  PromptRequest r;
  r.error = KDA_OK;
  r.src = r.dst = r.bnd = -1;
  r.m = 0;
  if (p.qsl != nullptr) {
    r.t0 = p.qsl[b];
    const long long end = p.qsl[b + 1];
    const long long n = end - r.t0;
    if (r.t0 < 0 || n < 0 || n > p.Q || end > p.n_tokens) {
      r.error = KDA_ERR_ARG;
      r.t0 = r.n = 0;
      return r;
    }
    r.n = (int)n;
  } else {
    r.t0 = b * p.Q;
    r.n = p.Q;
  }
  if (r.n == 0) return r;
  const int src = p.sources[b], dst = p.destinations[b];
  int bnd = p.null_slot, m = 0;
  if (p.bnd_slots != nullptr) {
    bnd = p.bnd_slots[b];
    m = p.bnd_lens[b];
  }
  if (dst <= p.null_slot) return r;  // inert whatever its other slots hold
  const bool crosses = m > 0 && bnd > p.null_slot;
  if (src >= p.n_slots || dst >= p.n_slots || (crosses && bnd >= p.n_slots)) {
    r.error = KDA_ERR_ARG;
    r.n = 0;
    return r;
  }
  // slots are >= 0 from here on whatever null_slot is
  r.dst = dst;
  if (src > p.null_slot) r.src = src;
  if (crosses) {
    r.bnd = bnd;
    r.m = m < r.n ? m : r.n;
  }
  return r;
}

// Host-side checks of the maps (before the operator's own).  Every index
// the kernels make from 32-bit sizes stays inside the types they use: a
// (token, head) row number fits 31 bits, byte and element offsets are 64-bit.
inline int check_prompt_maps(const int32_t *sources, const int32_t *destinations,
                             const int32_t *boundaries, const int32_t *boundary_lens,
                             const int32_t *qsl, int n_tokens, int n_slots, int B, int H, int Q,
                             int null_slot) {
  if (B < 0 || H < 1 || H > KDA_PROMPT_MAX_HEADS || Q < 1 || n_tokens < 0 || null_slot < -1)
    return KDA_ERR_ARG;
  if (B == 0) return KDA_OK;
  if ((long long)B * H > 0x7fffffffLL || (long long)n_tokens * H > 0x7fffffffLL)
    return KDA_ERR_ARG;
  if (qsl == nullptr && (long long)n_tokens != (long long)B * Q) return KDA_ERR_ARG;
  if (n_tokens == 0) return KDA_OK;
  if (!sources || !destinations || n_slots < 1) return KDA_ERR_ARG;
  if ((boundaries == nullptr) != (boundary_lens == nullptr)) return KDA_ERR_ARG;
  return KDA_OK;
}

inline PromptMaps make_prompt_maps(const int32_t *sources, const int32_t *destinations,
                                   const int32_t *boundaries, const int32_t *boundary_lens,
                                   const int32_t *qsl, int n_tokens, int n_slots, int B, int Q,
                                   int null_slot, int32_t *status) {
  PromptMaps m;
  m.sources = sources;
  m.destinations = destinations;
  m.bnd_slots = boundaries;
  m.bnd_lens = boundary_lens;
  m.qsl = qsl;
  m.n_tokens = n_tokens;
  m.n_slots = n_slots;
  m.B = B;
  m.Q = Q;
  m.null_slot = null_slot;
  m.status = status;
  return m;
}

}  // namespace kda

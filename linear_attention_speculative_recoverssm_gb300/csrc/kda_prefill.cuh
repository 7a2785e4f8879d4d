// The chunked gated delta rule: what its three kernels share.
//
// A chunk is 64 consecutive tokens of a request (fewer at its end and at its
// boundary).  With G_t the sum of the log decays from the chunk's first
// token to t (per key channel), the tokens of a chunk and the state S before
// it give
//   L_ts = beta_t sum_c kn_tc kn_sc e^{G_tc - G_sc}  (s < t),
//   T = (I + L)^-1 diag(beta),
//   A_ts = sum_c qn_tc kn_sc e^{G_tc - G_sc}         (s <= t),
//   R = V - Kd S^T, Kd_t = kn_t e^{G_t};  U = T R;
//   O = Qd S^T + A U, Qd_t = qn_t e^{G_t};
//   S <- S diag(e^{G_end}) + U^T Ke, Ke_t = kn_t e^{G_end - G_t}.
// The preparation kernel (kda_prefill_prep.cu) makes T, A, Kd, Qd, Ke of
// every (chunk, head) at once, as shared-memory images in the layouts that
// the matrix instructions read; the chain kernel (kda_prefill_chain.cu) takes
// each (request, head) through its chunks.
//
// Every entry of the images is at most 1 in size (unit keys and queries,
// decays <= 1, and T_ts is minus beta_t k_t applied to what is left of a
// state beta_s k_s after contractions: at most beta_s).  They are held as FP16
// times powers of two, Kd and A 2^10, Qd 2^4, Ke 2^6 (kda_prefill_chain.cu says
// why), and T 2^14 over p, the power of two above the chunk's largest beta: what
// a nearly closed write gate leaves is as small as the gate.  "hi" and "lo" are
// x rounded to FP16 and the rest rounded again, 22 bits together where neither
// is subnormal (x above 2^-24 for Kd, 2^-20 for Ke, 2^-28 p for T) and 2^-25 of
// the held value below.  hi.hi + hi.lo + lo.hi leaves 2^-22 of a product.
#pragma once

#include <cuda_fp16.h>

#include "kda_recurrent.cuh"

namespace kda {

constexpr int kChunk = 64;
constexpr float kImgScale = 1024.f;           // Kd, A
constexpr float kImgQdScale = 16.f, kImgKeScale = 64.f;
constexpr float kImgTScale = 16384.f;         // over the chunk's p

// Image of one (chunk, head): byte offsets of its parts.  Rows of 128 bytes
// (64 FP16), the 16-byte pieces of row r at position piece ^ (r & 7); K = 128
// operands are two such blocks of 64 rows, channels 0 .. 63 and 64 .. 127.
constexpr uint32_t kImgBlock = kChunk * 128;             // 8 KB
constexpr uint32_t kImgKdHi = 0;                         // [t][channel]
constexpr uint32_t kImgKdLo = kImgKdHi + 2 * kImgBlock;
constexpr uint32_t kImgQdHi = kImgKdLo + 2 * kImgBlock;  // [t][channel]
constexpr uint32_t kImgQdLo = kImgQdHi + 2 * kImgBlock;
constexpr uint32_t kImgTHi = kImgQdLo + 2 * kImgBlock;   // [t][s]
constexpr uint32_t kImgTLo = kImgTHi + kImgBlock;
constexpr uint32_t kImgKeHi = kImgTLo + kImgBlock;       // [s][channel]
constexpr uint32_t kImgKeLo = kImgKeHi + 2 * kImgBlock;
constexpr uint32_t kImgAHi = kImgKeLo + 2 * kImgBlock;   // [t][s]
constexpr uint32_t kImgALo = kImgAHi + kImgBlock;
constexpr uint32_t kImgDecay = kImgALo + kImgBlock;      // e^{G_end}, 128 FP32
// Behind the decays, FP32, what bounds the states to come (kScal..)
constexpr uint32_t kImgTail = (128 + 32) * 4;            // decays and scalars
constexpr uint32_t kImgBytes = kImgDecay + kImgTail;
// Scalars, by their place behind the decays: kEndFactor (the largest e^{G_end})^2
// (four values, whose maximum it is); kLeftFactor (the largest decay from the
// end of block 0 .. 2, of 16 tokens, to the chunk's)^2 (four values each); p; and
// p + 64 p^2.
constexpr int kScalEnd = 128, kScalLeft = 132, kScalBeta = 144, kScalValue = 145;
constexpr float kEndFactor = 2.03f / 4096.f, kLeftFactor = 130.f;

// x - h, by a multiply-add of FP16 factors to an FP32 sum: exact for h = x
// rounded to FP16, and no conversion of h, which shares its unit with the
// roundings (two conversions and a packed multiply-add: 3.1 us a chunk and not
// 2.8).
__device__ __forceinline__ float2 less_half(float2 x, __half2 h) {
  const uint16_t minus_one = 0xBC00;
  float2 d;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;"
      : "=f"(d.x)
      : "h"(__half_as_ushort(__low2half(h))), "h"(minus_one), "f"(x.x));
  asm("fma.rn.f32.f16 %0, %1, %2, %3;"
      : "=f"(d.y)
      : "h"(__half_as_ushort(__high2half(h))), "h"(minus_one), "f"(x.y));
  return d;
}

struct PrefillChunk {
  int t0, count;  // tokens t0 .. t0 + count - 1 of the packed activations
};

struct __align__(16) PrefillRequest {
  int b;
  int chunks;      // all of its chunks
  int bnd_chunks;  // chunks up to its boundary; 0: none
  int base;        // its first chunk of segment 0
};

// A (request, head) of which a chain's parts lost something (LostRows): by its
// place in the chain's grid, and which of its four groups of 32 rows.
struct PrefillRedo {
  int item, groups;
};

// The chunks go by segments of every request, seg_from(s) .. seg_from(s + 1) - 1
// of each at a time: the preparation of one and then its chain, whose CTAs leave the state to the
// next segment's in FP32.  The next preparation runs beside the chain.
struct PrefillParams {
  RecurrentParams r;
  int short_len;  // requests of at most so many tokens go token by token
  int max_chunks;
  int segments, seg_chunks;
  bool seg_doubles;  // each segment twice the one before, the first seg_chunks
  int *seg_first;           // [segments + 1], the segments' first chunks
  PrefillChunk *chunks;     // [max_chunks], by segment, then request
  int *bases;               // [segments, B], a request's first chunk of each
  PrefillRequest *order;    // [B], by falling number of chunks
  float *carry;             // [B, H, 128, 128] (segments > 1)
  int *lost;                // [B, H], the groups lost so far (segments > 1)
  int *n_redo;
  PrefillRedo *redo;        // [B * H], the first n_redo
  uint8_t *images;          // [max_chunks, H, kImgBytes]
};

__host__ __device__ __forceinline__ int seg_from(const PrefillParams &p, int s) {
  return p.seg_chunks * (p.seg_doubles ? (1 << s) - 1 : s);
}

// One segment.  A preparation that is not the first may start as soon as the
// chain before it has, and ends after it.
int launch_prefill_prep(const PrefillParams &p, int segment, cudaStream_t stream);
int launch_prefill_chain(const PrefillParams &p, int segment, bool bf16, cudaStream_t stream);
// After the last segment's chain: what `redo` lists once more, from its source.
int launch_prefill_redo(const PrefillParams &p, bool bf16, cudaStream_t stream);

}  // namespace kda

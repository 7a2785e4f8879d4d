// The chain of the chunked delta rule: one CTA takes a (request, head)
// through its chunks, its state on the chip throughout.  Everything is
// transposed so that a value channel v is a row: S^T [v][key channel],
// W = (S Kd^T), U, O [v][token].  Rows never meet, a thread owns a quarter of one,
// and per chunk (kda_prefill.cuh for the operands)
//   E0  S <- S e^{G_end} + dS of the chunk before; S as FP16 parts to TMEM
//   M1  W = S Kd^T, O = S Qd^T
//   E1  R = V - W as FP16 parts to TMEM
//   M2  U = R T^T
//   E2  U as FP16 parts to TMEM (over R)
//   M3  dS = U Ke;  M4  O += U A^T
// with M on the tensor cores (M = 128 rows, the first operand in TMEM, the
// second the image in shared memory) and E on warps 0-15: warp w holds lanes
// (rows) 32 (w & 3) .. and quarter w >> 2 of the columns.  O leaves while the
// next chunk's M1 runs.  Warp 16 issues the MMAs, warp 17 the copies.  All
// products take hi.hi + hi.lo + lo.hi.  (With the high parts alone for O, 16
// prompts took 578 us in place of 639 and one of 16384 tokens 832 in place of
// 890, and 15 % of the outputs rounded to another BF16 value than the exact
// ones; now fewer than 0.5 % do.)
//
// FP16 parts of a row are taken times powers of two: S times 2^6 f, U times f,
// R times a factor fr of its own, so that with the images' scales dS comes out
// in the state's units and both terms of O alike.  A part ends at 2^-24, so
// each factor is as large as what it holds allows, and follows what S, U and R
// themselves can be: of the state a chunk began with only what its decays leave
// counts, values behind a nearly closed write gate count for R and not for U.
// With B a bound of |S| over the row, V the largest |v| of the chunk and p at
// least its largest beta,
//   |R| <= V + sqrt(128) B,  |U| <= (p + 64 p^2) V + sqrt(128) p B
// (unit keys; a row's norm grows by at most beta |v| a token), and B itself is
//   max |S before| max e^{G_end} + 8 |U'|_2,
// U' being U times the largest decay from the end of its block of 16 tokens to
// the chunk's (the sum of 64 of them is at most 8 times their norm); (x + y)^2
// <= 2 x^2 + 2 y^2 makes Z = (f B)^2 of their squares.  f is kept while
// Z < 2^18 and f (p + 64 p^2) V < 2^14, which hold S and U below 2^15, and one
// of them is not 2^10 or 2^5 below that.  All of it is known before dS is, from
// a chunk's image and U: the rows' quarters exchange squares while M3 runs, and
// nothing waits between dS and S but the arithmetic; M3 and M1 go by halves of
// the key channels, E0 of the one under the other's MMAs.  For states that last
// B is some 2^5 above |S|: U's parts keep 2^-29 of U's size, and more where
// much is forgotten, so that a chunk may leave some 2^-14 of the sizes in it.
// Where a chunk leaves less in all rows of a group of 32 (those of one warp), or
// has tokens whose sizes are as far below the largest, or something in it is not
// finite, the parts cannot hold it.
// The chain finds that when it has the next state's sizes; the group's rows then
// go through the chunks once more, from the source, in a second kernel behind
// it, which looks before it goes on and does such a chunk token by token
// (CAREFUL): 150 us for such a chunk, 5 for the others.  (Both in one kernel left
// every chunk's path too few registers: 16384 tokens took 895 us in place of 843.)
// The state itself stays in FP32, in registers: an accumulator that is added
// to over and over loses up to a unit of its last place each time, so dS is
// summed apart, smallest parts first.
//
// What bounds it: a chunk's products and passes depend on one another, some 6.2 K
// cycles (3.2 us) of which the tensor cores run 2.8 K, with 8 CTAs on the GPU (751
// us for 256 chunks) nearly as with 32; 265 chunks of 32 heads in 16 prompts take
// 245 us, most of them the longest prompt's 78 chunks.  TMEM and shared memory
// hold one item an SM.  (One factor for R, S and U, from bounds that know no
// decay, was 0.2 us a chunk less, and lost what the above keeps.)  Eight row
// warps in place of 16 took longer, and so did the outputs' stores between R and
// U (2 to 6 %): what the other warps split then waits.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prefill.cuh"
#include "kda_tcgen05.cuh"
#include "kda_tensor_map.h"

namespace kda {
namespace {

constexpr int kRowWarps = 16;
constexpr int kChainThreads = 32 * (kRowWarps + 2);  // and the MMA and copy warps
constexpr int kParts = kRowWarps / 4;  // threads of a row
constexpr int kKeys = kDim / kParts, kToks = kChunk / kParts;  // their columns
constexpr uint32_t kPartA = kImgQdHi;                 // Kd: 32 KB
constexpr uint32_t kPartQ = kImgTHi - kImgQdHi;       // Qd: 32 KB
constexpr uint32_t kPartB = kImgKeHi - kImgTHi;       // T: 16 KB
constexpr uint32_t kPartC = kImgDecay - kImgKeHi;     // Ke, A: 48 KB
// Buffers of each.  C is released last, a chunk's end, and needed soonest: a
// second one takes 2 to 3 % off the chain (of the others or of v: nothing).
constexpr int kBufA = 1, kBufQ = 1, kBufB = 1, kBufC = 2;
constexpr uint32_t kVBytes = kChunk * kDim * 2;       // 16 KB

// TMEM columns
constexpr uint32_t kColDs = 0;      // dS, 128
constexpr uint32_t kColSHi = 128;   // 64: 128 FP16 per row
constexpr uint32_t kColSLo = 192;
constexpr uint32_t kColW = 256;     // W, then U: 64
constexpr uint32_t kColO = 320;     // two buffers of 64
constexpr uint32_t kColRHi = 448;   // R, then U: 32
constexpr uint32_t kColRLo = 480;
constexpr uint32_t kTmemCols = 512;

// kind::f16, FP32 accumulator, A and B FP16, M = 128; `mn`: B is MN-major
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t n, bool mn) {
  return (1u << 4) | ((mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

struct ChainSmem {
  // (multiples of 1024 bytes)
  uint8_t a[kBufA][kPartA], q[kBufQ][kPartQ], b[kBufB][kPartB], c[kBufC][kPartC];
  uint8_t v[kVBytes];
  float decay[4][kImgTail / 4];  // decays and scalars of chunk i at i & 3
  PrefillChunk chunk[4];  // chunk i at i & 3, there when its v is
  // [chunk parity][part][row]: the largest |S|, squares of U', in parts' units; the
  // next |v|; squares of U over the part's block of tokens
  float4 peak[2][kParts][128];
  uint32_t kept[4][kParts];  // by row warps w & 3 and part: what a chunk left (CAREFUL)
  float2 next[128];          // by row: f of the next chunk and most_r's bits
  float least[128];          // by row: see is_lost
  int lost;                  // the groups of rows that parts lost something of, a bit each
  // The item: its request, head, chunks and boundary as the row warps need them
  // (what they keep in registers costs them others in every chunk).
  struct {
    int b, h, n, bnd_at, ends;
  } item;
  uint64_t a_full[kBufA], a_free[kBufA], q_full[kBufQ], q_free[kBufQ];
  uint64_t b_full[kBufB], b_free[kBufB], c_full[kBufC], c_free[kBufC];
  uint64_t v_full, v_free, d_full[4];
  uint64_t s_ready[2], r_ready, u_ready, w_full, u_full, ds_full[2], o_full, drained;
  uint64_t factors[4], advanced[4], token[4];  // of the four warps of the same rows
  uint32_t tmem;
};
static_assert(kPartA % 1024 == 0 && kPartB % 1024 == 0 && kPartC % 1024 == 0, "swizzle atoms");

// A 128-byte swizzled MN-major operand: LBO between blocks of 64 N elements,
// SBO between groups of 8 K rows.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kImgBlock >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p;
}

// D[tmem] (+)= A[tmem, 128 x 16] . B[N x 16]^T, issued by the lane with
// `lead` while the whole warp runs along: what is the same in every lane then
// lives in uniform registers, which the instruction takes its operands from.
// (In a branch of one lane each operand is moved there first, some 50 cycles
// an issue against the 32 that N = 64 takes to execute.)
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                        bool accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
      : "memory");
}

// 16 FP32 columns of this warp's lanes; waits for the load.
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ void tmem_store_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// floor(log2 |x|) (128 for infinities and NaN, -127 for zero).
__device__ __forceinline__ int exponent(float x) {
  return (int)((__float_as_uint(x) >> 23) & 255u) - 127;
}

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// f for a row of zeros, and for the bounds B and V' = (p + 64 p^2) V.
constexpr int kMostExp = 90;
__device__ __forceinline__ float row_factor(float b, float v) {
  return pow2(min(max(min(8 - exponent(b), 13 - exponent(v)) - 2, -109), kMostExp));
}

// The larger; NaN where one is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

__device__ __forceinline__ float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float pow2_inverse(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// Two values as FP16 and what that leaves; `most` the largest |hi| so far.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo, __half2 &most) {
  const __half2 h = __float22half2_rn(x);
  most = __hmax2_nan(most, __habs2(h));
  const __half2 l = __float22half2_rn(less_half(x, h));
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}

// A part of a state page's row (kKeys key channels).
template <bool BF16>
__device__ __forceinline__ void load_state(const void *page, int row, int part,
                                           float2 (&s)[kKeys / 2]) {
  if constexpr (BF16) {
    const uint4 *g = reinterpret_cast<const uint4 *>(page) + row * (kDim / 8) + part * (kKeys / 8);
#pragma unroll
    for (int i = 0; i < kKeys / 8; ++i) {
      const uint4 x = __ldcs(g + i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[4 * i + j] = make_float2(__uint_as_float(w[j] << 16),
                                   __uint_as_float(w[j] & 0xffff0000u));
    }
  } else {
    const float4 *g =
        reinterpret_cast<const float4 *>(page) + row * (kDim / 4) + part * (kKeys / 4);
#pragma unroll
    for (int i = 0; i < kKeys / 4; ++i) {
      const float4 x = __ldcs(g + i);
      s[2 * i] = make_float2(x.x, x.y);
      s[2 * i + 1] = make_float2(x.z, x.w);
    }
  }
}

// The same to memory, times `f`.
template <bool BF16>
__device__ __forceinline__ void store_state(void *page, int row, int part,
                                            const float2 (&s)[kKeys / 2], float f) {
  const float2 ff = make_float2(f, f);
  if constexpr (BF16) {
    uint4 *g = reinterpret_cast<uint4 *>(page) + row * (kDim / 8) + part * (kKeys / 8);
#pragma unroll
    for (int i = 0; i < kKeys / 8; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = fmul2(s[4 * i + j], ff);
        w[j] = pack_bf16x2(x.x, x.y);
      }
      g[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    float4 *g = reinterpret_cast<float4 *>(page) + row * (kDim / 4) + part * (kKeys / 4);
#pragma unroll
    for (int i = 0; i < kKeys / 4; ++i) {
      const float2 x = fmul2(s[2 * i], ff), y = fmul2(s[2 * i + 1], ff);
      g[i] = make_float4(x.x, x.y, y.x, y.y);
    }
  }
}

// The MMAs of one product: hi and lo parts, STEPS K = 16 steps each, smallest
// first.
template <int STEPS, typename BDesc>
__device__ __forceinline__ void mma_part(uint32_t d, uint32_t a, BDesc b, uint32_t idesc,
                                         bool accumulate, uint32_t lead) {
#pragma unroll
  for (int ks = 0; ks < STEPS; ++ks)
    umma_ts(d, a + 8 * ks, b(ks), idesc, accumulate || ks > 0, lead);
}
template <int STEPS, typename BDesc>
__device__ __forceinline__ void mma_split(uint32_t d, uint32_t a_hi, uint32_t a_lo, BDesc hi,
                                          BDesc lo, uint32_t idesc, bool accumulate,
                                          uint32_t lead) {
  mma_part<STEPS>(d, a_lo, hi, idesc, accumulate, lead);
  mma_part<STEPS>(d, a_hi, lo, idesc, true, lead);
  mma_part<STEPS>(d, a_hi, hi, idesc, true, lead);
}

// K-major parts: a K step is 32 bytes of a 128-byte row, 4 to a block.
struct KMajor {
  uint64_t desc;
  __device__ __forceinline__ explicit KMajor(uint32_t at) : desc(umma_desc_sw128(at)) {}
  __device__ __forceinline__ uint64_t operator()(int ks) const {
    return desc + (uint64_t)(((uint32_t)(ks >> 2) * kImgBlock + (uint32_t)(ks & 3) * 32u) >> 4);
  }
  __device__ __forceinline__ KMajor block(int i) const {  // K steps from 4 i on
    KMajor b = *this;
    b.desc += (uint64_t)((uint32_t)i * kImgBlock >> 4);
    return b;
  }
};
// The MMAs of a product with T or A, which have nothing above their diagonals:
// K step ks (columns 16 ks .. 16 ks + 15) only from row 16 ks on, N = 64 - 16 ks
// (all of N: 1.5 % longer, 16384 tokens).
__device__ __forceinline__ void mma_lower(uint32_t d, uint32_t a_hi, uint32_t a_lo, KMajor hi,
                                          KMajor lo, bool accumulate, uint32_t lead) {
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const KMajor &b = j == 1 ? lo : hi;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      umma_ts(d + 16 * ks, (j == 0 ? a_lo : a_hi) + 8 * ks,
              b(ks) + (uint64_t)((uint32_t)ks * 2048u >> 4), idesc_f16(64 - 16 * ks, false),
              accumulate || j > 0 || ks > 0, lead);
  }
}
// MN-major parts: a K step is 16 rows of 128 bytes.
struct MnMajor {
  uint64_t desc;
  __device__ __forceinline__ explicit MnMajor(uint32_t at) : desc(umma_desc_mn_sw128(at)) {}
  __device__ __forceinline__ uint64_t operator()(int ks) const {
    return desc + (uint64_t)((uint32_t)ks * 2048u >> 4);
  }
  __device__ __forceinline__ MnMajor block(int i) const {  // N from 64 i on
    MnMajor b = *this;
    b.desc += (uint64_t)((uint32_t)i * kImgBlock >> 4);
    return b;
  }
};

// A chunk's tokens one after the other in FP32, its outputs stored and the
// state `s` (as it is, not scaled) advanced: by the four warps of the same
// rows, for a chunk that the parts cannot hold.  2.4 us a token (its operands by
// 128 shuffles a warp), 150 a chunk, with 16 warps at it.  What a row's parts
// add up goes through their places in sm.peak of the chunk before,
// which have been read (each token's by turns in two of the four floats).
// False: a wait ran out.
__device__ __noinline__ bool rows_by_token(const RecurrentParams &r, ChainSmem &sm, int chunk,
                                           int h, int row, int part, volatile float *state) {
  float2 s[kKeys / 2];
#pragma unroll
  for (int e = 0; e < kKeys / 2; ++e) s[e] = make_float2(state[2 * e], state[2 * e + 1]);
  const int lane = row & 31;
  const PrefillChunk ck = sm.chunk[chunk & 3];
  const float a = expf(r.A_log[h]);
  const float4 dt = *reinterpret_cast<const float4 *>(r.dt_bias + h * kDim + 4 * lane);
  uint64_t *const bar = &sm.token[row >> 5];
  bool ok = true;
  static_assert(kChunk % 2 == 0, "the barrier ends on the parity that it began with");
#pragma unroll 1
  for (int t = 0; t < kChunk && ok; ++t) {
    Token tk;
    float v = 0.f;
    const long long at = (long long)(ck.t0 + min(t, ck.count - 1)) * r.H + h;
    if (t < ck.count) {
      tk = make_token(r, load_token(r, at, lane), a, dt);
      v = bf16_bits_to_f32(r.v[at * kDim + row]);
      // (channel c of a token is held by lane c / 4)
      const auto of = [&](const float4 &x, int e) {
        const int from = (kKeys / 4) * part + (e >> 1);
        return (e & 1) ? make_float2(__shfl_sync(0xffffffffu, x.z, from),
                                     __shfl_sync(0xffffffffu, x.w, from))
                       : make_float2(__shfl_sync(0xffffffffu, x.x, from),
                                     __shfl_sync(0xffffffffu, x.y, from));
      };
      float2 w = make_float2(0.f, 0.f), y = w;
#pragma unroll
      for (int e = 0; e < kKeys / 2; ++e) {
        s[e] = fmul2(s[e], of(tk.d, e));
        w = ffma2(s[e], of(tk.k, e), w);
        y = ffma2(s[e], of(tk.q, e), y);
      }
      reinterpret_cast<float2 *>(&sm.peak[(chunk + 1) & 1][part][row])[t & 1] =
          make_float2(w.x + w.y, y.x + y.y);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, (uint32_t)t & 1u));
    if (t >= ck.count || !ok) continue;
    float w = 0.f, y = 0.f;
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
      const float2 x = reinterpret_cast<const float2 *>(&sm.peak[(chunk + 1) & 1][j][row])[t & 1];
      w += x.x;
      y += x.y;
    }
    const float u = tk.beta * (v - w);
    if (part == 0) r.out[at * kDim + row] = f32_to_bf16_bits(fmaf(u, tk.kq, y));
#pragma unroll
    for (int e = 0; e < kKeys / 2; ++e) {
      const int from = (kKeys / 4) * part + (e >> 1);
      const float k0 = __shfl_sync(0xffffffffu, (e & 1) ? tk.k.z : tk.k.x, from);
      const float k1 = __shfl_sync(0xffffffffu, (e & 1) ? tk.k.w : tk.k.y, from);
      s[e] = ffma2(make_float2(u, u), make_float2(k0, k1), s[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < kKeys / 2; ++e) {
    state[2 * e] = s[e].x;
    state[2 * e + 1] = s[e].y;
  }
  return ok;
}

// Zeros to the outputs of an inert request's head.
__device__ __forceinline__ void zero_inert(const PrefillParams &p, int b, int h) {
  const PromptRequest rq = prompt_request(p.r.maps, b);
  if (rq.dst >= 0) return;
  for (int i = threadIdx.x; i < rq.n * (kDim / 8); i += kChainThreads)
    *reinterpret_cast<uint4 *>(p.r.out +
                               ((long long)(rq.t0 + i / (kDim / 8)) * p.r.H + h) * kDim +
                               i % (kDim / 8) * 8) = make_uint4(0, 0, 0, 0);
}

// CAREFUL: the redo list's items, all of their chunks, every segment's.
template <bool BF16, bool CAREFUL>
__global__ void __launch_bounds__(kChainThreads, 1)
    kda_prefill_chain_kernel(const __grid_constant__ PrefillParams p,
                             const __grid_constant__ CUtensorMap v_map, int segment) {
  // (the swizzle atoms want 1024 bytes; there is no other shared memory)
  extern __shared__ __align__(1024) uint8_t chain_raw[];
  const int H = p.r.H;
  ChainSmem &sm = *reinterpret_cast<ChainSmem *>(chain_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto give_up = [&] {
    report(p.r.maps.status, KDA_ERR_TIMEOUT);
    if constexpr (CAREFUL) atomicOr(&sm.lost, 1);  // (goes to no other item)
  };
  // what does not need the preparation, while its last CTAs may still run
  const auto init_barriers = [&] {
    const auto init = [](uint64_t *full, uint64_t *free, int n) {
      for (int i = 0; i < n; ++i) {
        mbar_init(full + i, 1);
        mbar_init(free + i, 1);
      }
    };
    init(sm.a_full, sm.a_free, kBufA);
    init(sm.q_full, sm.q_free, kBufQ);
    init(sm.b_full, sm.b_free, kBufB);
    init(sm.c_full, sm.c_free, kBufC);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.d_full[i], 1);
      mbar_init(&sm.d_full[i + 2], 1);
      mbar_init(&sm.s_ready[i], kRowWarps / 2);
      mbar_init(&sm.ds_full[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.factors[i], 1);
      mbar_init(&sm.advanced[i], kParts);
      mbar_init(&sm.token[i], kParts);
    }
    mbar_init(&sm.v_full, 1);
    mbar_init(&sm.v_free, kRowWarps);
    mbar_init(&sm.r_ready, kRowWarps);
    mbar_init(&sm.u_ready, kRowWarps);
    mbar_init(&sm.w_full, 1);
    mbar_init(&sm.u_full, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.drained, 1);
    mbar_init_fence();
    sm.lost = 0;
  };
  if (!CAREFUL && threadIdx.x == 0) init_barriers();
  if (!CAREFUL && warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
  grid_dependency_wait();
  // (only now: the next kernel may count on what this one has waited for)
  grid_launch_dependents();
  int listed = blockIdx.x;
  const int n_listed = CAREFUL ? __ldcg(p.n_redo) : 0;
  if constexpr (CAREFUL) {
    if (listed >= n_listed) return;
    if (threadIdx.x == 0) init_barriers();
    if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
  }
  while (!CAREFUL || listed < n_listed) {
  PrefillRedo redo{(int)blockIdx.x, 15};
  if constexpr (CAREFUL)
    redo = PrefillRedo{__ldcg(&p.redo[listed].item), __ldcg(&p.redo[listed].groups)};
  const PrefillRequest req = p.order[redo.item / H];
  const int b = req.b, h = redo.item % H;
  // this segment's chunks: done, done + 1 .. done + n - 1 of the request's
  const int done = CAREFUL ? 0 : seg_from(p, segment);
  const int n = CAREFUL ? req.chunks : max(min(req.chunks, seg_from(p, segment + 1)) - done, 0);
  const bool starts = CAREFUL || segment == 0;
  const bool ends = done + n == req.chunks;
  const int bnd_at = req.bnd_chunks > 0 ? req.bnd_chunks - done : -1;  // in its chunks
  const int base = starts ? req.base : p.bases[segment * p.r.maps.B + b];
  const int src = prompt_request(p.r.maps, b).src;  // (of segment 0)
  if (threadIdx.x == 0) {
    if (!starts) sm.lost = p.lost[b * H + h];
    sm.item.b = b, sm.item.h = h, sm.item.n = n, sm.item.bnd_at = bnd_at, sm.item.ends = ends;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  // the list's place of chunk i, and its image
  const auto place = [&](int i) {
    if constexpr (!CAREFUL) return base + i;
    int s = 0;
    while (s + 1 < p.segments && seg_from(p, s + 1) <= i) ++s;
    return p.bases[s * p.r.maps.B + b] + i - seg_from(p, s);
  };
  const auto image = [&](int i) {
    return p.images + ((long long)place(i) * H + h) * kImgBytes;
  };

  if (n == 0) {
    if (segment == 0 && p.short_len == 0) zero_inert(p, b, h);
  } else if (warp == kRowWarps + 1) {
    // -- copies ---------------------------------------------------------------
    bool ok = true;
    int n_v = 0, n_a = 0, n_q = 0, n_b = 0, n_c = 0;  // copies issued of each kind
    PrefillChunk coming = p.chunks[place(0)];  // the next chunk whose v is copied
    const auto load_v = [&](int i) {
      uint64_t *bar = &sm.v_full;
      if (i >= 1) ok = ok && mbar_wait_bounded(&sm.v_free, (uint32_t)(i - 1) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      n_v = i + 1;
      if (lane != 0) return;
      // 64 rows whatever the count: one copy (a copy a row took the warp some
      // 75 cycles each); what is past it, rows of others or the zeros past the
      // activations, is not used
      const PrefillChunk ck = coming;
      coming = p.chunks[place(min(i + 1, n - 1))];
      // (the places of chunk i - 4: its outputs and state were done before any
      // row warp released v of chunk i - 1)
      sm.chunk[i & 3] = ck;
      mbar_arrive_expect_tx(&sm.d_full[i & 3], kImgTail);
      bulk_g2s(sm.decay[i & 3], image(i) + kImgDecay, kImgTail, &sm.d_full[i & 3]);
      mbar_arrive_expect_tx(bar, kVBytes);
      tma_load_3d(sm.v, &v_map, 0, h, ck.t0, bar);
    };
    const auto load_part = [&](int i, int buffers, uint64_t *full, uint64_t *free, uint8_t *dst,
                               uint32_t at, uint32_t bytes, int &issued) {
      const int use = i / buffers, which = i - use * buffers;
      if (use >= 1) ok = ok && mbar_wait_bounded(free + which, (uint32_t)(use - 1) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      issued = i + 1;
      if (lane != 0) return;
      mbar_arrive_expect_tx(full + which, bytes);
      bulk_g2s(dst + which * bytes, image(i) + at, bytes, full + which);
    };
    load_v(0);
    for (int i = 0; i < n && ok; ++i) {
      load_part(i, kBufA, sm.a_full, sm.a_free, sm.a[0], 0, kPartA, n_a);
      if (ok && i + 1 < n) load_v(i + 1);
      if (ok) load_part(i, kBufB, sm.b_full, sm.b_free, sm.b[0], kImgTHi, kPartB, n_b);
      if (ok) load_part(i, kBufQ, sm.q_full, sm.q_free, sm.q[0], kImgQdHi, kPartQ, n_q);
      if (ok) load_part(i, kBufC, sm.c_full, sm.c_free, sm.c[0], kImgKeHi, kPartC, n_c);
    }
    if (!ok) {
      // every copy issued lands before the CTA can exit: the last phase in
      // use of each barrier
      if (lane == 0) give_up();
      const auto settle = [&](uint64_t *bar, int uses) {
        if (uses > 0) mbar_wait_bounded(bar, (uint32_t)(uses - 1) & 1u);
      };
      const auto settle_all = [&](uint64_t *bar, int buffers, int uses) {
        for (int j = 0; j < buffers; ++j) settle(bar + j, (uses - j + buffers - 1) / buffers);
      };
      settle_all(sm.a_full, kBufA, n_a);
      settle_all(sm.q_full, kBufQ, n_q);
      settle_all(sm.b_full, kBufB, n_b);
      settle_all(sm.c_full, kBufC, n_c);
      settle_all(sm.d_full, 4, n_v);
      settle(&sm.v_full, n_v);
    }
  } else if (warp == kRowWarps) {
    // -- tensor cores: the whole warp, converged ------------------------------
    const uint32_t lead = elect_one();
    const auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = uniform(tmem);
    const uint32_t base_a = uniform(smem_u32(sm.a)), base_q = uniform(smem_u32(sm.q));
    const uint32_t base_b = uniform(smem_u32(sm.b)), base_c = uniform(smem_u32(sm.c));
    constexpr uint32_t k64 = idesc_f16(64, false), k64mn = idesc_f16(64, true);
    const uint32_t w = tm + kColW, s_hi = tm + kColSHi, s_lo = tm + kColSLo;
    const uint32_t r_hi = tm + kColRHi, r_lo = tm + kColRLo;
    const auto commit = [&](uint64_t *bar) {
      if (lead) umma_commit(bar);
      __syncwarp();
    };
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const uint32_t ph = (uint32_t)i & 1u;
      const uint32_t o = tm + kColO + 64u * ph;
      const uint32_t ia = (uint32_t)i % kBufA, iq = (uint32_t)i % kBufQ;
      const uint32_t ib = (uint32_t)i % kBufB, ic = (uint32_t)i % kBufC;
      const uint32_t sa = base_a + ia * kPartA, sq = base_q + iq * kPartQ;
      const uint32_t sb = base_b + ib * kPartB, sc = base_c + ic * kPartC;
      const KMajor kd_hi(sa + kImgKdHi), kd_lo(sa + kImgKdLo);
      const KMajor qd_hi(sq), qd_lo(sq + kImgQdLo - kImgQdHi), t_hi(sb), t_lo(sb + kImgBlock);
      const KMajor a_hi(sc + 4 * kImgBlock), a_lo(sc + 5 * kImgBlock);
      const MnMajor ke_hi(sc), ke_lo(sc + 2 * kImgBlock);
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm.a_full[ia], (uint32_t)(i / kBufA) & 1u));
      for (int half = 0; half < 2 && ok; ++half) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm.s_ready[half], ph));
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = 32u * half;  // four K steps of TMEM columns
        mma_split<4>(w, s_hi + at, s_lo + at, kd_hi.block(half), kd_lo.block(half), k64, half > 0,
                     lead);
      }
      if (!ok) break;
      commit(&sm.w_full);
      commit(&sm.a_free[ia]);
      // (of O a third under the rows' way from W to R, the rest under theirs from
      // U to its parts)
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm.q_full[iq], (uint32_t)(i / kBufQ) & 1u));
      if (!ok) break;
      mma_part<8>(o, s_hi, qd_hi, k64, false, lead);
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm.b_full[ib], (uint32_t)(i / kBufB) & 1u) &&
                                       mbar_wait_bounded(&sm.r_ready, ph));
      if (!ok) break;
      tc_fence_after();
      mma_lower(w, r_hi, r_lo, t_hi, t_lo, false, lead);
      commit(&sm.u_full);
      commit(&sm.b_free[ib]);
      mma_part<8>(o, s_lo, qd_hi, k64, true, lead);
      mma_part<8>(o, s_hi, qd_lo, k64, true, lead);
      commit(&sm.q_free[iq]);
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm.c_full[ic], (uint32_t)(i / kBufC) & 1u) &&
                                       mbar_wait_bounded(&sm.u_ready, ph));
      if (!ok) break;
      tc_fence_after();
      for (int half = 0; half < 2; ++half) {
        mma_split<4>(tm + kColDs + 64u * half, r_hi, r_lo, ke_hi.block(half), ke_lo.block(half),
                     k64mn, false, lead);
        commit(&sm.ds_full[half]);
      }
      mma_lower(o, r_hi, r_lo, a_hi, a_lo, true, lead);
      commit(&sm.o_full);
      commit(&sm.c_free[ic]);
    }
    if (!ok && lead) give_up();
    // nothing of this CTA's is in flight when its columns are released
    commit(&sm.drained);
    mbar_wait_bounded(&sm.drained, 0u);
  } else {
    // -- rows -------------------------------------------------------------------
    const int row = 32 * (warp & 3) + lane, qt = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    // The pages' addresses are made where they are used, from values that are
    // read anew each time: kept through the loop they would take registers that
    // it has not got.
    const auto now = [](const int &x) { return *const_cast<const volatile int *>(&x); };
    const auto page = [&](int slot) {
      return reinterpret_cast<char *>(p.r.state) +
             ((long long)slot * p.r.slot_stride + (long long)now(sm.item.h) * kDim * kDim) *
                 (BF16 ? 2 : 4);
    };
    const auto carry = [&] {
      return p.carry + ((long long)now(sm.item.b) * H + now(sm.item.h)) * kDim * kDim;
    };
    const auto request = [&] { return prompt_request(p.r.maps, now(sm.item.b)); };
    float2 s[kKeys / 2];  // this row's key channels from kKeys qt on
    const int group = warp & 3;
    // (rows that are not to be done again run along, from zeros)
    const bool live = !CAREFUL || ((redo.groups >> group) & 1);
    if (!starts) {
      load_state<false>(carry(), row, qt, s);
    } else {
      if (src >= 0 && live) {
        load_state<BF16>(page(src), row, qt, s);
      } else {
#pragma unroll
        for (int i = 0; i < kKeys / 2; ++i) s[i] = make_float2(0.f, 0.f);
      }
    }
    constexpr float kDown = 1.f / kImgScale;
    constexpr float kUnit = kImgKeScale, kPerUnit = 1.f / kImgKeScale;  // S's factor over f
    static_assert(kImgKeScale * kImgQdScale == kImgScale, "both terms of O alike");
    const auto f2 = [](uint32_t x, uint32_t y) {
      return make_float2(__uint_as_float(x), __uint_as_float(y));
    };
    const auto both = [](float x) { return make_float2(x, x); };
    const int half = 2 * qt / kParts;  // of the key channels
    bool bad = false;
    const auto wait = [&](uint64_t *bar, uint32_t parity) {
      bad = __any_sync(0xffffffffu, bad || !mbar_wait_bounded(bar, parity));
      return !bad;
    };
    // v of chunk i: this row's tokens from kToks qt on, and their peak
    uint32_t v2[kToks / 2];
    const auto load_v = [&](int i) {
      if (!wait(&sm.v_full, (uint32_t)i & 1u)) return 0.f;
      const int count = sm.chunk[i & 3].count;
      const uint16_t *v = reinterpret_cast<const uint16_t *>(sm.v) + kToks * qt * kDim + row;
      const int left = count - kToks * qt;
      if (left >= kToks) {
#pragma unroll
        for (int j = 0; j < kToks / 2; ++j)
          v2[j] = (uint32_t)v[2 * j * kDim] | ((uint32_t)v[(2 * j + 1) * kDim] << 16);
      } else {
#pragma unroll
        for (int j = 0; j < kToks / 2; ++j) {
          const uint32_t x = 2 * j < left ? v[2 * j * kDim] : 0u;
          v2[j] = x | (2 * j + 1 < left ? (uint32_t)v[(2 * j + 1) * kDim] << 16 : 0u);
        }
      }
      __nv_bfloat162 peak = __float2bfloat162_rn(0.f);
#pragma unroll
      for (int j = 0; j < kToks / 2; ++j)
        peak = __hmax2(peak, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&v2[j])));
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_free);
      return fmaxf(__low2float(peak), __high2float(peak));
    };
    // the sum of what this row's parts left at [i & 1], of |S| and |v| the largest,
    // of the blocks' U the smallest
    const auto joined = [&](int i) {
      float4 m = sm.peak[i & 1][0][row];
#pragma unroll
      for (int j = 1; j < kParts; ++j) {
        const float4 x = sm.peak[i & 1][j][row];
        m = make_float4(max_nan(m.x, x.x), m.y + x.y, fmaxf(m.z, x.z), fminf(m.w, x.w));
      }
      return m;
    };
    const auto max4 = [](const float *x) {
      const float4 v = lds4(x);
      return fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
    };
    const auto largest = [&] {  // of this part's s
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < kKeys / 2; ++e) m = max_nan(m, max_nan(fabsf(s[e].x), fabsf(s[e].y)));
      return m;
    };
    sm.peak[1][qt][row] = make_float4(largest(), 0.f, load_v(0), 0.f);
    wait(&sm.d_full[0], 0u);
    bad = named_bar_or(1, 32 * kRowWarps, bad);
    // s holds the state times 2^6 f from here on; inv = 1 / f
    float f, inv;
    int most_r;  // no |R| of the chunk reaches 2^most_r
    {
      const float4 m = joined(1);
      const float v = m.z * sm.decay[0][kScalValue];
      f = row_factor(m.x, is_finite(v) ? v : 0.f);
      inv = pow2_inverse(f);
      most_r = max(exponent(m.x) + 4, exponent(m.z)) + 2;
    }
#pragma unroll
    for (int e = 0; e < kKeys / 2; ++e) s[e] = fmul2(s[e], both(f * kUnit));
    const auto is_marked = [&] { return ((now(sm.lost) >> group) & 1) != 0; };
    // The parts end a fixed way below what they could hold, 2^-24 / f, and what
    // of that reaches the state measures some 2^-27 / f.  A chunk is lost for a
    // group of rows that is left with nothing above 2^-12 / f: 2^-15 of its largest
    // entry.  So it is where a block of 16 tokens has no U above that,
    // nor had the state before the chunk: of its outputs not enough would be left
    // (values before an outlying one).
    constexpr float kLeast = 0x1p-12f;
    // (CAREFUL) Before the next chunk: where that is so for the largest of the
    // four parts' entries, the chunk is done again token by token, from the state
    // before it.  Its parts are still in TMEM, and hold it to 2^-19 of its rows;
    // where they would not, `by_token` was set before dS was there.  All four
    // warps come to that together: one whose rows all keep more says so, and
    // only one that cannot waits for what the others say.
    bool by_token = false;
    const auto check = [&](int i) {
      uint32_t mine = 0xffffffffu;  // (every row keeps enough)
      bool finite = true;
      const float top = largest();
      const bool doubt = !by_token && live &&
                         !__all_sync(0xffffffffu, top >= kLeast * kUnit || f == pow2(kMostExp));
      if (doubt) {
        // (a row that is not finite asks for nothing)
        const float n = top * (inv * kPerUnit);
        finite = is_finite(n);
        mine = __reduce_max_sync(0xffffffffu, finite ? __float_as_uint(n) : 0u);
      }
      if (lane == 0) {
        sm.kept[group][qt] = mine;
        mbar_arrive(&sm.advanced[group]);
      }
      if (!doubt || !wait(&sm.advanced[group], (uint32_t)i & 1u)) return;
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < kParts; ++j) most = max(most, sm.kept[group][j]);
      const float floor = kLeast * __uint_as_float(__reduce_max_sync(
                                       0xffffffffu, finite ? __float_as_uint(inv) : 0u));
      by_token = most != 0xffffffffu && __uint_as_float(most) < floor && floor > 0x1p-100f;
      if (by_token) {
        uint32_t d[16];
        tmem_load16(lanes + kColSHi + (uint32_t)(kKeys / 2 * qt), d);
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e)
          s[e] = __half22float2(*reinterpret_cast<const __half2 *>(&d[e]));
        tmem_load16(lanes + kColSLo + (uint32_t)(kKeys / 2 * qt), d);
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e)
          s[e] = ffma2(both(1.f), s[e], __half22float2(*reinterpret_cast<const __half2 *>(&d[e])));
      }
    };
    // The same of rows whose largest are brought together, times f; `least` is
    // kLeast times the present f over the chunk's.
    const auto is_lost = [&](float top, float least) {
      const float n = top * inv, floor = least * inv;
      const bool finite = is_finite(n);
      const uint32_t most = __reduce_max_sync(0xffffffffu, finite ? __float_as_uint(n) : 0u);
      const uint32_t worst = __reduce_max_sync(0xffffffffu, finite ? __float_as_uint(floor) : 0u);
      return most < worst && __uint_as_float(worst) > 0x1p-100f;
    };
    float f_next = f;
    bool changes = false;   // for any row of the warp
    // (else) What the rows' warps go by after chunk i.
    const auto take = [&](int i) {
      if (!wait(&sm.factors[group], (uint32_t)i & 1u)) return false;
      const float2 x = sm.next[row];
      f_next = x.x;
      most_r = __float_as_int(x.y);
      changes = __any_sync(0xffffffffu, f_next != f);
      return true;
    };
    // S <- S e^{G_end} + dS of chunk i
    const auto advance = [&](int i) {
      if constexpr (!CAREFUL) {  // (while dS is on its way: after it, 2 % longer)
        if (!take(i)) return;
      }
      if (!wait(&sm.ds_full[half], (uint32_t)i & 1u)) return;
      tc_fence_after();
      if (CAREFUL && by_token) return check(i);
      const float *dec = sm.decay[i & 3] + kKeys * qt;
#pragma unroll
      for (int j = 0; j < kKeys / 16; ++j) {
        uint32_t d[16];
        tmem_load16(lanes + kColDs + (uint32_t)(kKeys * qt + 16 * j), d);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 g = lds4(dec + 16 * j + 2 * e);
          float2 &x = s[8 * j + e], &y = s[8 * j + e + 1];
          x = ffma2(x, make_float2(g.x, g.y), f2(d[2 * e], d[2 * e + 1]));
          y = ffma2(y, make_float2(g.z, g.w), f2(d[2 * e + 2], d[2 * e + 3]));
        }
      }
      if constexpr (CAREFUL) check(i);
    };
    // the outputs of chunk i
    const auto emit = [&](int i, float inv) {
      if (!wait(&sm.o_full, (uint32_t)i & 1u)) return;
      if (CAREFUL && (by_token || !live)) {
        by_token = false;  // (they are there)
        return;
      }
      tc_fence_after();
      const float f = p.r.q_scale * kDown * inv;
      const uint32_t step = (uint32_t)H * kDim;
      const PrefillChunk ck = sm.chunk[i & 3];
#pragma unroll
      for (int k = 0; k < kToks / 16; ++k) {
        const int t = kToks * qt + 16 * k;
        uint32_t d[16];
        tmem_load16(lanes + kColO + 64u * (i & 1) + (uint32_t)t, d);
        uint16_t *o = p.r.out + (long long)(ck.t0 + t) * step + now(sm.item.h) * kDim + row;
        const int left = ck.count - t;
        if (left >= 16) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[j * step] = f32_to_bf16_bits(__uint_as_float(d[j]) * f);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < left) o[j * step] = f32_to_bf16_bits(__uint_as_float(d[j]) * f);
        }
      }
    };
    // the state to a page; to the next segment (slot < 0)
    const auto store = [&](int slot) {
      if (slot < 0) store_state<false>(carry(), row, qt, s, inv * kPerUnit);
      else store_state<BF16>(page(slot), row, qt, s, inv * kPerUnit);
    };
    // The state after the boundary.  The chain keeps the source as it is while
    // it may have to go again: where the boundary's slot is the source, the
    // destination's holds it until the end.
    const auto store_boundary = [&] {
      const PromptRequest r = request();
      if (CAREFUL ? live : !is_marked()) store(!CAREFUL && r.bnd == r.src ? r.dst : r.bnd);
    };
    const auto settle_boundary = [&] {
      const PromptRequest r = request();
      if (r.bnd < 0 || r.bnd != r.src || now(sm.item.bnd_at) > now(sm.item.n)) return;  // (cut off)
      constexpr int kPieces = kKeys * (BF16 ? 2 : 4) / 16;
      const long long at = ((long long)row * kParts + qt) * kPieces;
      const uint4 *const from = reinterpret_cast<const uint4 *>(page(r.dst)) + at;
      uint4 *const to = reinterpret_cast<uint4 *>(page(r.bnd)) + at;
#pragma unroll 1
      for (int e = 0; e < kPieces; ++e) to[e] = from[e];
    };
    // What a state that is ready goes through.
    const auto rescale = [&] {
      if (changes) {
        if (!CAREFUL && qt == kParts - 1) sm.least[row] *= f_next * inv;
        // (one after the other: the factors' quotient may be out of range)
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e) s[e] = fmul2(fmul2(s[e], both(f_next)), both(inv));
        f = f_next;
        inv = pow2_inverse(f);
        changes = false;
      }
    };
    const auto pass = [&](int i, float inv_before) {
      // (what the factors are made of goes to memory at once: the registers are
      // wanted)
      float *const peak = reinterpret_cast<float *>(&sm.peak[i & 1][qt][row]);
      // S as parts
      {
        __half2 most = __float2half2_rn(0.f);
#pragma unroll
        for (int j = 0; j < kKeys / 16; ++j) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split2(s[8 * j + e], hi[e], lo[e], most);
          tmem_store8(lanes + kColSHi + (uint32_t)(kKeys / 2 * qt + 8 * j), hi);
          tmem_store8(lanes + kColSLo + (uint32_t)(kKeys / 2 * qt + 8 * j), lo);
        }
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_ready[half]);
        const float2 x = __half22float2(most);
        peak[0] = max_nan(x.x, x.y);
      }
      if (i > 0) emit(i - 1, inv_before);
      // R = V - W
      const float fr = pow2(min(max(15 - most_r, -113), 100));
      const float w = -kDown * kPerUnit * fr * inv;
      if (!wait(&sm.w_full, (uint32_t)i & 1u)) return false;
      tc_fence_after();
      __half2 unused = __float2half2_rn(0.f);
      {
#pragma unroll
        for (int k = 0; k < kToks / 16; ++k) {
          uint32_t d[16], hi[8], lo[8];
          tmem_load16(lanes + kColW + (uint32_t)(kToks * qt + 16 * k), d);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t vv = v2[8 * k + j];
            const float2 v = make_float2(__uint_as_float(vv << 16),
                                         __uint_as_float(vv & 0xffff0000u));
            split2(ffma2(f2(d[2 * j], d[2 * j + 1]), both(w), fmul2(v, both(fr))), hi[j],
                   lo[j], unused);
          }
          tmem_store8(lanes + kColRHi + (uint32_t)(kToks / 2 * qt + 8 * k), hi);
          tmem_store8(lanes + kColRLo + (uint32_t)(kToks / 2 * qt + 8 * k), lo);
        }
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.r_ready);
      }
      peak[2] = 0.f;
      if (i + 1 < now(sm.item.n)) {
        peak[2] = load_v(i + 1);
        if (!wait(&sm.d_full[(i + 1) & 3], (uint32_t)((i + 1) >> 2) & 1u)) return false;
      }
      // U: T's scale and R's off, its own on (f p / fr is at most 4)
      const float *const tail = sm.decay[i & 3];
      const float by = f * tail[kScalBeta] * (pow2_inverse(fr) * (1.f / kImgTScale));
      static_assert(kToks == 16, "a part's tokens are a block of the scalars'");
      const float left = qt < kParts - 1 ? max4(tail + kScalLeft + 4 * qt) : kLeftFactor;
      // (a block past the chunk's tokens has no U; one of zeros, as of padding, to a
      // state of zeros has lost none: [i + 1] still holds its largest |v|)
      const bool past = kToks * qt >= sm.chunk[i & 3].count;
      const bool blank = sm.peak[(i + 1) & 1][qt][row].z == 0.f && peak[0] == 0.f;
      float2 uu[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      if (!wait(&sm.u_full, (uint32_t)i & 1u)) return false;
      tc_fence_after();
      {
#pragma unroll
        for (int k = 0; k < kToks / 16; ++k) {
          uint32_t d[16], hi[8], lo[8];
          tmem_load16(lanes + kColW + (uint32_t)(kToks * qt + 16 * k), d);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 u = fmul2(f2(d[2 * j], d[2 * j + 1]), both(by));
            uu[j & 1] = ffma2(u, u, uu[j & 1]);
            split2(u, hi[j], lo[j], unused);
          }
          tmem_store8(lanes + kColRHi + (uint32_t)(kToks / 2 * qt + 8 * k), hi);
          tmem_store8(lanes + kColRLo + (uint32_t)(kToks / 2 * qt + 8 * k), lo);
        }
        const float u2 = (uu[0].x + uu[0].y) + (uu[1].x + uu[1].y);
        peak[1] = left * u2;
        peak[3] = past || (blank && u2 == 0.f) ? __int_as_float(0x7f800000) : u2;
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.u_ready);
      }
      // under M3: every row's sums are there once all warps have arrived.  One
      // of a row's four warps, of those whose half of dS comes last, works out
      // what all of them go by (an E's four warps share a scheduler: all four
      // would take it 350 issue slots a chunk)
      if (CAREFUL || qt == kParts - 1) {  // (of the last chunk: what was lost before it)
        if (!wait(&sm.u_ready, (uint32_t)i & 1u)) return false;
        const float4 m = joined(i);
        const float z = fmaf(m.x * m.x, max4(tail + kScalEnd), m.y);
        // (a chunk whose V is infinite goes token by token, from this state)
        const float v0 = m.z * sm.decay[(i + 1) & 3][kScalValue];
        const float v = is_finite(v0) ? v0 : 0.f, fv = f * v;
        const bool keep = z < 0x1p18f && fv < 0x1p14f &&
                          (z >= 0x1p8f || fv >= 0x1p9f || f == pow2(kMostExp));
        // (CAREFUL: a state that its parts would not give back; a fresh one is
        // zeros)
        const float least = CAREFUL || i == 0 ? 0.f : sm.least[row];
        const float top = kPerUnit * m.x;  // of f |S|
        const bool low = CAREFUL ? top < 0x1p-12f && f != pow2(kMostExp) && (i > 0 || src >= 0)
                                 : top < least;
        const bool little = top < kLeast && m.w < kLeast * kLeast;
        if (__any_sync(0xffffffffu, !keep || low || little)) {
          // An infinity or a NaN of one token is in the U of all of its chunk's
          // (zeros of T times it), and not of those before it by the rule.  (A
          // state that is not finite spoils all that follows by either.)
          const bool wild = __any_sync(0xffffffffu, !is_finite(m.y) && is_finite(m.x));
          const bool thin = wild || is_lost(fmaxf(top, sqrt_fast(m.w)), kLeast);
          if constexpr (CAREFUL) by_token = live && (__any_sync(0xffffffffu, low) || thin);
          else if ((thin || is_lost(top, least)) && lane == 0) atomicOr(&sm.lost, 1 << group);
          f_next = keep ? f : row_factor(sqrt_fast(z) * inv, v);
          if constexpr (CAREFUL) changes = __any_sync(0xffffffffu, f_next != f);
        }
        // (sqrt(128) B is below 2^4 B, and of the sum each at most half)
        most_r = max(((exponent(z) + 1) >> 1) - exponent(f) + 4, exponent(m.z)) + 2;
        if constexpr (!CAREFUL) {
          sm.next[row] = make_float2(f_next, __int_as_float(most_r));
          sm.least[row] = kLeast;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.factors[group]);
        }
      }
      return true;
    };
    if constexpr (!CAREFUL) {
      for (int i = 0; i < now(sm.item.n); ++i) {
        const float inv_before = inv;
        if (i > 0) {
          advance(i - 1);
          if (bad) break;
          if (i == now(sm.item.bnd_at)) store_boundary();
          rescale();
        }
        if (!pass(i, inv_before)) break;
      }
      if (!bad) advance(now(sm.item.n) - 1);
      if (!bad && now(sm.item.n) == now(sm.item.bnd_at)) store_boundary();
    } else {
      // (by token: through memory, so that what the chunks need in registers is
      // not kept in them meanwhile)
      volatile float held[kKeys + kToks / 2 + 3];
      for (int i = 0;;) {
        const float inv_before = inv;
        if (i > 0) rescale();
        if (!pass(i, inv_before)) break;
        advance(i);
        if (bad) break;
        if (by_token) {
#pragma unroll
          for (int e = 0; e < kKeys / 2; ++e) {
            held[2 * e] = s[e].x * (inv * kPerUnit);
            held[2 * e + 1] = s[e].y * (inv * kPerUnit);
          }
#pragma unroll
          for (int e = 0; e < kToks / 2; ++e) held[kKeys + e] = __uint_as_float(v2[e]);
          held[kKeys + kToks / 2] = f;
          held[kKeys + kToks / 2 + 1] = f_next;
          held[kKeys + kToks / 2 + 2] = __int_as_float(most_r);
          if (!rows_by_token(p.r, sm, i, now(sm.item.h), row, qt, held)) {
            bad = true;
            break;
          }
          f = held[kKeys + kToks / 2];
          f_next = held[kKeys + kToks / 2 + 1];
          most_r = __float_as_int(held[kKeys + kToks / 2 + 2]);
          inv = pow2_inverse(f);
          changes = __any_sync(0xffffffffu, f_next != f);
#pragma unroll
          for (int e = 0; e < kKeys / 2; ++e)
            s[e] = fmul2(make_float2(held[2 * e], held[2 * e + 1]), both(f * kUnit));
#pragma unroll
          for (int e = 0; e < kToks / 2; ++e) v2[e] = __float_as_uint(held[kKeys + e]);
        }
        ++i;
        if (i == now(sm.item.bnd_at)) store_boundary();
        if (i == now(sm.item.n)) break;
      }
    }
    if constexpr (!CAREFUL) {
      // the last chunk's, whose state nothing else brings together
      const int n = now(sm.item.n);
      sm.peak[n & 1][qt][row].x = kPerUnit * largest();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.advanced[group]);
      if (!bad && wait(&sm.advanced[group], 0u) && is_lost(joined(n).x, kLeast) && lane == 0)
        atomicOr(&sm.lost, 1 << group);
      __syncwarp();
    }
    if (!bad) {
      const bool marked = !CAREFUL && is_marked();
      const bool ends = now(sm.item.ends) != 0;
      if (ends && !CAREFUL && !marked) settle_boundary();
      if (live && !(ends && marked)) store(ends ? request().dst : -1);
      emit(now(sm.item.n) - 1, inv);
    }
    if (bad && lane == 0) give_up();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (!CAREFUL) {
    if (n > 0 && threadIdx.x == 0) {
      if (p.segments > 1) p.lost[b * H + h] = sm.lost;
      if (ends && sm.lost != 0) p.redo[atomicAdd(p.n_redo, 1)] = PrefillRedo{redo.item, sm.lost};
    }
    break;
  }
  if (sm.lost != 0) break;
  listed += gridDim.x;
  if (listed < n_listed) {
    // (no wait or arrival is left of the item before)
    if (threadIdx.x == 0) {
      constexpr int kBars = (offsetof(ChainSmem, tmem) - offsetof(ChainSmem, a_full)) / 8;
      for (int j = 0; j < kBars; ++j) mbar_inval(sm.a_full + j);
      init_barriers();
    }
    __syncthreads();
  }
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(sm.tmem, kTmemCols);
  }
}

}  // namespace

// The chain of a segment; of what the redo list holds (segment < 0).
static int launch_chain(const PrefillParams &p, int segment, bool bf16, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  constexpr uint32_t kSmem = sizeof(ChainSmem);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(2 * kSmem > 228 * 1024, "one CTA per SM: its TMEM allocation never waits");
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    for (const auto kernel : {kda_prefill_chain_kernel<false, false>,
                              kda_prefill_chain_kernel<true, false>,
                              kda_prefill_chain_kernel<false, true>,
                              kda_prefill_chain_kernel<true, true>})
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)kSmem) != cudaSuccess)
        return KDA_ERR_CUDA;
    configured.fetch_or(bit);
  }
  // v [n_tokens, H, 128] as a 3-D tensor, a chunk's rows of one head a copy
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return KDA_ERR_CUDA;
  const cuuint64_t dims[3] = {(cuuint64_t)kDim, (cuuint64_t)p.r.H,
                              (cuuint64_t)p.r.maps.n_tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)kDim * 2, (cuuint64_t)p.r.H * kDim * 2};
  const cuuint32_t box[3] = {(cuuint32_t)kDim, 1, (cuuint32_t)kChunk};
  const cuuint32_t estride[3] = {1, 1, 1};
  CUtensorMap v_map;
  if (encode(&v_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(p.r.v), dims,
             strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
      CUDA_SUCCESS)
    return KDA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int items = p.r.maps.B * p.r.H, sms = device_sm_count(dev);
  cfg.gridDim = dim3((unsigned)(segment < 0 && sms > 0 && sms < items ? sms : items));
  cfg.blockDim = dim3(kChainThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel =
      segment < 0 ? (bf16 ? kda_prefill_chain_kernel<true, true> : kda_prefill_chain_kernel<false, true>)
                  : (bf16 ? kda_prefill_chain_kernel<true, false> : kda_prefill_chain_kernel<false, false>);
  if (cudaLaunchKernelEx(&cfg, kernel, p, v_map, segment) != cudaSuccess) return KDA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int launch_prefill_chain(const PrefillParams &p, int segment, bool bf16, cudaStream_t stream) {
  return launch_chain(p, segment, bf16, stream);
}

int launch_prefill_redo(const PrefillParams &p, bool bf16, cudaStream_t stream) {
  return launch_chain(p, -1, bf16, stream);
}

}  // namespace kda

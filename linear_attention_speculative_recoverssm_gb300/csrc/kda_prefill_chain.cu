// The chain of the chunked delta rule: one CTA takes a (request, head)
// through its chunks, its state on the chip throughout.  Everything is
// transposed so that a value channel v is a row: S^T [v][key channel],
// W = (S Kd^T), U, O [v][token].  Rows never meet, a thread owns half of one,
// and per chunk (kda_prefill.cuh for the operands)
//   E0  S <- S e^{G_end} + dS of the chunk before; S as FP16 parts to TMEM
//   M1  W = S Kd^T, O = S Qd^T
//   E1  R = V - W as FP16 parts to TMEM
//   M2  U = R T^T
//   E2  U as FP16 parts to TMEM (over R)
//   M3  dS = U Ke;  M4  O += U A^T
// with M on the tensor cores (M = 128 rows, the first operand in TMEM, the
// second the image in shared memory) and E on warps 0-7: warp w holds lanes
// (rows) 32 (w & 3) .. and half w >> 2 of the columns.  O leaves while the
// next chunk's M1 runs.  Warp 8 issues the MMAs, warp 9 the copies.
//
// FP16 parts of a row are taken times a power of two that brings the largest
// of |S| and |v| over the row to 2^8 .. 2^9.  R is then below 12.4 2^9, and
// U below 76 2^9 < 65504 (a row of the state grows by at most beta |v| a
// token), so one factor a chunk serves S, R, U and O, and their accumulators
// share it.  The state itself stays in FP32, in registers: an accumulator
// that is added to over and over loses up to a unit of its last place each
// time, so dS is summed apart, smallest parts first.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prefill.cuh"
#include "kda_tcgen05.cuh"

namespace kda {
namespace {

constexpr int kChainThreads = 320;  // E warps 0-7, MMA warp 8, copy warp 9
constexpr uint32_t kPartA = kImgTHi;                  // Kd, Qd: 48 KB
constexpr uint32_t kPartB = kImgKeHi - kImgTHi;       // T: 16 KB
constexpr uint32_t kPartC = kImgDecay - kImgKeHi;     // Ke, A: 40 KB
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
  uint8_t a[kPartA], b[kPartB], c[kPartC];  // each a multiple of 1024 bytes
  uint8_t v[2][kVBytes];
  float decay[2][kDim];
  float peak[2][2][128];  // [chunk parity][column half][row]
  uint64_t a_full, a_free, b_full, b_free, c_full, c_free, v_full[2], v_free[2], d_full[2];
  uint64_t s_ready, r_ready, u_ready, w_full, u_full, ds_full, o_full, drained;
  uint32_t tmem;
};
static_assert(kPartA % 1024 == 0 && kPartB % 1024 == 0 && kPartC % 1024 == 0, "swizzle atoms");

// A 128-byte swizzled MN-major operand: LBO between blocks of 64 N elements,
// SBO between groups of 8 K rows.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kImgBlock >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// D[tmem] (+)= A[tmem, 128 x 16] . B[N x 16]^T
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_store_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 2^(8 - e) for m in [2^e, 2^(e+1)), at most 2^100 (zero rows)
__device__ __forceinline__ float row_scale(float m) {
  const int e = (int)((__float_as_uint(m) >> 23) & 255u);
  const int s = 127 + 8 + 127 - e;
  return __uint_as_float((uint32_t)(s > 227 ? 227 : s) << 23);
}

__device__ __forceinline__ float pow2_inverse(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// Two values as FP16 and what that leaves.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __float22half2_rn(x);
  const float2 f = __half22float2(h);
  const __half2 l = __float22half2_rn(ffma2(f, make_float2(-1.f, -1.f), x));
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}

template <bool BF16>
__device__ __forceinline__ void load_state(const void *page, int row, int half, float2 (&s)[32]) {
  if constexpr (BF16) {
    const uint4 *g = reinterpret_cast<const uint4 *>(page) + row * (kDim / 8) + half * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 x = __ldcs(g + i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[4 * i + j] = make_float2(__uint_as_float(w[j] << 16),
                                   __uint_as_float(w[j] & 0xffff0000u));
    }
  } else {
    const float4 *g = reinterpret_cast<const float4 *>(page) + row * (kDim / 4) + half * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float4 x = __ldcs(g + i);
      s[2 * i] = make_float2(x.x, x.y);
      s[2 * i + 1] = make_float2(x.z, x.w);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store_state(void *page, int row, int half,
                                            const float2 (&s)[32]) {
  if constexpr (BF16) {
    uint4 *g = reinterpret_cast<uint4 *>(page) + row * (kDim / 8) + half * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      g[i] = make_uint4(pack_bf16x2(s[4 * i].x, s[4 * i].y),
                        pack_bf16x2(s[4 * i + 1].x, s[4 * i + 1].y),
                        pack_bf16x2(s[4 * i + 2].x, s[4 * i + 2].y),
                        pack_bf16x2(s[4 * i + 3].x, s[4 * i + 3].y));
  } else {
    float4 *g = reinterpret_cast<float4 *>(page) + row * (kDim / 4) + half * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      g[i] = make_float4(s[2 * i].x, s[2 * i].y, s[2 * i + 1].x, s[2 * i + 1].y);
  }
}

// The MMAs of one product: hi and lo parts, `steps` K = 16 steps each,
// smallest first.  `bstep(ks)`: byte offset of step ks in an operand part.
template <typename BDesc>
__device__ __forceinline__ void mma_split(uint32_t d, uint32_t a_hi, uint32_t a_lo, int steps,
                                          uint32_t idesc, BDesc hi, BDesc lo) {
  for (int ks = 0; ks < steps; ++ks) umma_ts(d, a_lo + 8 * ks, hi(ks), idesc, ks > 0);
  for (int ks = 0; ks < steps; ++ks) umma_ts(d, a_hi + 8 * ks, lo(ks), idesc, true);
  for (int ks = 0; ks < steps; ++ks) umma_ts(d, a_hi + 8 * ks, hi(ks), idesc, true);
}

// K-major parts: a K step is 32 bytes of a 128-byte row, 4 to a block.
struct KMajor {
  uint32_t base;
  __device__ __forceinline__ uint64_t operator()(int ks) const {
    return umma_desc_sw128(base + (uint32_t)(ks >> 2) * kImgBlock + (uint32_t)(ks & 3) * 32u);
  }
};
// MN-major parts: a K step is 16 rows of 128 bytes.
struct MnMajor {
  uint32_t base;
  __device__ __forceinline__ uint64_t operator()(int ks) const {
    return umma_desc_mn_sw128(base + (uint32_t)ks * 2048u);
  }
};

template <bool BF16>
__global__ void __launch_bounds__(kChainThreads, 1) kda_prefill_chain_kernel(const PrefillParams p) {
  extern __shared__ uint8_t chain_raw[];
  const int H = p.r.H;
  const int b = p.order[blockIdx.x / H], h = blockIdx.x % H;
  const PrefillRequest req = p.requests[b];
  const int n = req.chunks;
  if (n == 0) return;
  ChainSmem &sm = *reinterpret_cast<ChainSmem *>(
      chain_raw + ((1024u - (smem_u32(chain_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t *status = p.r.maps.status;
  if (threadIdx.x == 0) {
    mbar_init(&sm.a_full, 1);
    mbar_init(&sm.a_free, 1);
    mbar_init(&sm.b_full, 1);
    mbar_init(&sm.b_free, 1);
    mbar_init(&sm.c_full, 1);
    mbar_init(&sm.c_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_free[i], 8);
      mbar_init(&sm.d_full[i], 1);
    }
    mbar_init(&sm.s_ready, 8);
    mbar_init(&sm.r_ready, 8);
    mbar_init(&sm.u_ready, 8);
    mbar_init(&sm.w_full, 1);
    mbar_init(&sm.u_full, 1);
    mbar_init(&sm.ds_full, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.drained, 1);
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const uint8_t *images = p.images + ((long long)req.base * H + h) * kImgBytes;
  const long long img_step = (long long)H * kImgBytes;

  if (warp == 9) {
    // -- copies ---------------------------------------------------------------
    bool ok = true;
    const auto load_v = [&](int i) {
      const PrefillChunk ck = p.chunks[req.base + i];
      uint64_t *bar = &sm.v_full[i & 1];
      if (i >= 2) ok = ok && mbar_wait_bounded(&sm.v_free[i & 1], (uint32_t)((i >> 1) - 1) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)ck.count * kDim * 2);
      __syncwarp();
      for (int t = lane; t < ck.count; t += 32)
        bulk_g2s(sm.v[i & 1] + t * kDim * 2,
                 p.r.v + ((long long)(ck.t0 + t) * H + h) * kDim, kDim * 2, bar);
    };
    const auto load_part = [&](int i, uint64_t *full, uint64_t *free, uint8_t *dst, uint32_t at,
                               uint32_t bytes) {
      if (i >= 1) ok = ok && mbar_wait_bounded(free, (uint32_t)(i - 1) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || lane != 0) return;
      mbar_arrive_expect_tx(full, bytes);
      bulk_g2s(dst, images + i * img_step + at, bytes, full);
    };
    load_v(0);
    int issued = 0;  // parts A, B, C and the decays of chunks 0 .. issued - 1
    int part = 0;    // and so many parts of the next one
    for (int i = 0; i < n && ok; ++i) {
      part = 0;
      load_part(i, &sm.a_full, &sm.a_free, sm.a, 0, kPartA);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.d_full[i & 1], kDim * 4);
        bulk_g2s(sm.decay[i & 1], images + i * img_step + kImgDecay, kDim * 4, &sm.d_full[i & 1]);
      }
      part = 1;
      load_part(i, &sm.b_full, &sm.b_free, sm.b, kPartA, kPartB);
      if (!ok) break;
      part = 2;
      load_part(i, &sm.c_full, &sm.c_free, sm.c, kPartA + kPartB, kPartC);
      if (!ok) break;
      issued = i + 1;
      part = 0;
      if (i + 1 < n) load_v(i + 1);
    }
    if (!ok) {
      // every copy issued lands before the CTA can exit: each barrier's last
      // phase in use
      if (lane == 0) report(status, KDA_ERR_TIMEOUT);
      const auto settle = [&](uint64_t *bar, int uses) {
        if (uses > 0) mbar_wait_bounded(bar, (uint32_t)(uses - 1) & 1u);
      };
      const int a = issued + (part >= 1), bb = issued + (part >= 2);
      settle(&sm.a_full, a);
      settle(&sm.b_full, bb);
      settle(&sm.c_full, issued);
      settle(&sm.d_full[0], (a + 1) / 2);
      settle(&sm.d_full[1], a / 2);
      const int v = issued + 1 < n ? issued + 1 : n;  // (at most so many: a wait may run out)
      settle(&sm.v_full[0], (v + 1) / 2);
      settle(&sm.v_full[1], v / 2);
    }
  } else if (warp == 8) {
    // -- tensor cores ---------------------------------------------------------
    if (lane == 0) {
      bool ok = true;
      const uint32_t a = smem_u32(sm.a), bt = smem_u32(sm.b), c = smem_u32(sm.c);
      for (int i = 0; i < n; ++i) {
        const uint32_t ph = (uint32_t)i & 1u;
        const uint32_t o = tmem + kColO + 64u * ph;
        ok = mbar_wait_bounded(&sm.a_full, ph) && mbar_wait_bounded(&sm.s_ready, ph);
        if (!ok) break;
        tc_fence_after();
        mma_split(tmem + kColW, tmem + kColSHi, tmem + kColSLo, 8, idesc_f16(64, false),
                  KMajor{a + kImgKdHi}, KMajor{a + kImgKdLo});
        umma_commit(&sm.w_full);
        for (int ks = 0; ks < 8; ++ks)
          umma_ts(o, tmem + kColSHi + 8 * ks, KMajor{a + kImgQd}(ks), idesc_f16(64, false),
                  ks > 0);
        umma_commit(&sm.a_free);
        ok = mbar_wait_bounded(&sm.b_full, ph) && mbar_wait_bounded(&sm.r_ready, ph);
        if (!ok) break;
        tc_fence_after();
        mma_split(tmem + kColW, tmem + kColRHi, tmem + kColRLo, 4, idesc_f16(64, false),
                  KMajor{bt}, KMajor{bt + kImgBlock});
        umma_commit(&sm.u_full);
        umma_commit(&sm.b_free);
        ok = mbar_wait_bounded(&sm.c_full, ph) && mbar_wait_bounded(&sm.u_ready, ph);
        if (!ok) break;
        tc_fence_after();
        mma_split(tmem + kColDs, tmem + kColRHi, tmem + kColRLo, 4, idesc_f16(128, true),
                  MnMajor{c}, MnMajor{c + 2 * kImgBlock});
        umma_commit(&sm.ds_full);
        for (int ks = 0; ks < 4; ++ks)
          umma_ts(o, tmem + kColRHi + 8 * ks, KMajor{c + 4 * kImgBlock}(ks),
                  idesc_f16(64, false), true);
        umma_commit(&sm.o_full);
        umma_commit(&sm.c_free);
      }
      if (!ok) report(status, KDA_ERR_TIMEOUT);
      // nothing of this CTA's is in flight when its columns are released
      umma_commit(&sm.drained);
      mbar_wait_bounded(&sm.drained, 0u);
    }
  } else {
    // -- rows -------------------------------------------------------------------
    const int row = 32 * (warp & 3) + lane, hf = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const long long elem = BF16 ? 2 : 4;
    char *pool = reinterpret_cast<char *>(p.r.state) + (long long)h * kDim * kDim * elem;
    const long long slot_bytes = p.r.slot_stride * elem;
    const PromptRequest rq = prompt_request(p.r.maps, b);
    float2 s[32];  // this row's key channels 64 hf .. 64 hf + 63
    if (rq.src >= 0) {
      load_state<BF16>(pool + rq.src * slot_bytes, row, hf, s);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = make_float2(0.f, 0.f);
    }
    constexpr float kDown = 1.f / kImgScale;
    float inv = 0.f;  // 1 / the chunk before's row scale
    int t0 = 0, count = 0;
    bool bad = false;
    // S <- S e^{G_end} + dS of chunk i
    const auto advance = [&](int i) {
      bad = bad || !mbar_wait_bounded(&sm.d_full[i & 1], (uint32_t)(i >> 1) & 1u) ||
            !mbar_wait_bounded(&sm.ds_full, (uint32_t)i & 1u);
      bad = __any_sync(0xffffffffu, bad);
      if (bad) return;
      tc_fence_after();
      const float2 f = make_float2(inv * kDown, inv * kDown);
      const float *dec = sm.decay[i & 1] + 64 * hf;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t d[32];
        tmem_load32(lanes + kColDs + 64u * hf + 32u * j, d);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float4 g = lds4(dec + 32 * j + 2 * e);
          float2 &x = s[16 * j + e], &y = s[16 * j + e + 1];
          x = ffma2(x, make_float2(g.x, g.y),
                    fmul2(f, make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1]))));
          y = ffma2(y, make_float2(g.z, g.w),
                    fmul2(f, make_float2(__uint_as_float(d[2 * e + 2]),
                                         __uint_as_float(d[2 * e + 3]))));
        }
      }
    };
    // the outputs of chunk i (at t0, count: still that chunk's)
    const auto emit = [&](int i, int t0, int count) {
      bad = bad || !mbar_wait_bounded(&sm.o_full, (uint32_t)i & 1u);
      bad = __any_sync(0xffffffffu, bad);
      if (bad) return;
      tc_fence_after();
      uint32_t d[32];
      tmem_load32(lanes + kColO + 64u * (i & 1) + 32u * hf, d);
      const float f = p.r.q_scale * kDown * inv;
      uint16_t *o = p.r.out + ((long long)(t0 + 32 * hf) * H + h) * kDim + row;
      const int left = count - 32 * hf;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < left) o[(long long)j * H * kDim] = f32_to_bf16_bits(__uint_as_float(d[j]) * f);
    };
    for (int i = 0; i < n; ++i) {
      const PrefillChunk ck = p.chunks[req.base + i];
      // v of the chunk: this row's tokens 32 hf .. 32 hf + 31
      uint32_t v2[16];
      float peak = 0.f;
      bad = bad || !mbar_wait_bounded(&sm.v_full[i & 1], (uint32_t)(i >> 1) & 1u);
      {
        const uint16_t *v = reinterpret_cast<const uint16_t *>(sm.v[i & 1]) + 32 * hf * kDim + row;
        const int left = ck.count - 32 * hf;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t x = 2 * j < left ? v[2 * j * kDim] : 0u;
          const uint32_t y = 2 * j + 1 < left ? v[(2 * j + 1) * kDim] : 0u;
          v2[j] = x | (y << 16);
          peak = fmaxf(peak, fmaxf(fabsf(__uint_as_float(x << 16)),
                                   fabsf(__uint_as_float(y << 16))));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_free[i & 1]);
      }
      if (i > 0) {
        advance(i - 1);
        if (i == req.bnd_chunks && !bad)
          store_state<BF16>(pool + rq.bnd * slot_bytes, row, hf, s);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) peak = fmaxf(peak, fmaxf(fabsf(s[e].x), fabsf(s[e].y)));
      sm.peak[i & 1][hf][row] = peak;
      bad = named_bar_or(1, 256, bad);
      if (bad) break;
      const float scale = row_scale(fmaxf(peak, sm.peak[i & 1][hf ^ 1][row]));
      {
        const float2 f = make_float2(scale, scale);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) split2(fmul2(s[16 * j + e], f), hi[e], lo[e]);
          tmem_store16(lanes + kColSHi + 32u * hf + 16u * j, hi);
          tmem_store16(lanes + kColSLo + 32u * hf + 16u * j, lo);
        }
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_ready);
      }
      if (i > 0) emit(i - 1, t0, count);
      inv = pow2_inverse(scale);
      t0 = ck.t0;
      count = ck.count;
      // R = V - W
      bad = bad || !mbar_wait_bounded(&sm.w_full, (uint32_t)i & 1u);
      bad = __any_sync(0xffffffffu, bad);
      if (!bad) {
        tc_fence_after();
        uint32_t d[32], hi[16], lo[16];
        tmem_load32(lanes + kColW + 32u * hf, d);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 w = make_float2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]));
          const float2 v = make_float2(__uint_as_float(v2[j] << 16),
                                       __uint_as_float(v2[j] & 0xffff0000u));
          split2(ffma2(w, make_float2(-kDown, -kDown), fmul2(v, make_float2(scale, scale))),
                 hi[j], lo[j]);
        }
        tmem_store16(lanes + kColRHi + 16u * hf, hi);
        tmem_store16(lanes + kColRLo + 16u * hf, lo);
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.r_ready);
        bad = !mbar_wait_bounded(&sm.u_full, (uint32_t)i & 1u);
      }
      // U
      bad = __any_sync(0xffffffffu, bad);
      if (!bad) {
        tc_fence_after();
        uint32_t d[32], hi[16], lo[16];
        tmem_load32(lanes + kColW + 32u * hf, d);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          split2(fmul2(make_float2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1])),
                       make_float2(kDown, kDown)),
                 hi[j], lo[j]);
        tmem_store16(lanes + kColRHi + 16u * hf, hi);
        tmem_store16(lanes + kColRLo + 16u * hf, lo);
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.u_ready);
      }
    }
    if (!bad) advance(n - 1);
    if (!bad) {
      if (n == req.bnd_chunks) store_state<BF16>(pool + rq.bnd * slot_bytes, row, hf, s);
      store_state<BF16>(pool + rq.dst * slot_bytes, row, hf, s);
      emit(n - 1, t0, count);
    }
    if (bad && lane == 0) report(status, KDA_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

int launch_prefill_chain(const PrefillParams &p, bool bf16, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  constexpr uint32_t kSmem = sizeof(ChainSmem) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(2 * kSmem > 228 * 1024, "one CTA per SM: its TMEM allocation never waits");
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute(kda_prefill_chain_kernel<false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(kda_prefill_chain_kernel<true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSmem) != cudaSuccess)
      return KDA_ERR_CUDA;
    configured.fetch_or(bit);
  }
  const unsigned grid = (unsigned)(p.r.maps.B * p.r.H);
  if (bf16) kda_prefill_chain_kernel<true><<<grid, kChainThreads, kSmem, stream>>>(p);
  else kda_prefill_chain_kernel<false><<<grid, kChainThreads, kSmem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda

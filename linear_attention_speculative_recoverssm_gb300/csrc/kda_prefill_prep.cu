// The preparation of the chunked delta rule: the images of every (chunk,
// head) (kda_prefill.cuh).  One CTA of 8 warps each; warps 2 i and 2 i + 1
// own the 16 tokens of block i, half the channels each, in the layout of an
// m16n8k8 operand: lane 4 g + j holds tokens g and g + 8 and eight
// consecutive channels of every 32.
//
// The products need e^{G_t - G_s} per channel, whose two factors must stay
// representable.  Within a block of 16 they are taken from its middle,
// 2^(G_t - mid) and 2^(mid - G_s), at most 2^116 with the steepest gate, and
// the 16 x 16 products run in TF32 (8 exponent bits) straight from the
// registers that hold the factors.  Between blocks a border lies between s
// and t, and both factors, from t back to it and from it back to s, are at
// most 1: blocks 0-1 | 2-3 with the border at token 32, blocks 0 | 1 and
// 2 | 3 with theirs at 16 and 48, in FP16 parts through shared memory.  The
// key products take hi.hi + hi.lo + lo.hi (their errors reach the state);
// the query products hi alone, 2^-12 of values whose result rounds to BF16.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prefill.cuh"

namespace kda {
namespace {

constexpr int kPrepThreads = 256;
constexpr uint32_t kXPitch = 272;  // bytes of a 128-channel FP16 row, padded
constexpr uint32_t kXBytes = kChunk * kXPitch;
constexpr uint32_t kYBytes = 32 * kXPitch;
constexpr int kLPitch = 68;  // floats
constexpr int kDPitch = 17;

// Shared memory, by phases: the FP16 operands of the products between
// blocks, then (in their place) L, its inverse and a scratch matrix.
struct PrepSmem {
  union {
    struct {
      uint8_t x16_hi[kXBytes], x16_lo[kXBytes], x32_hi[kXBytes], x32_lo[kXBytes];
      uint8_t y16[kYBytes], y32[kYBytes];
    } x;
    struct {
      float L[kChunk * kLPitch], X[kChunk * kLPitch], Y[32 * kLPitch];
    } s;
  } u;
  float fac[4][4][128];        // [kind][block][channel], times 1024
  float tot[2][4][128];        // log2 decays of a block's two halves
  float part[4][2][16 * kDPitch];  // a block's products over channels 64 .. 127
  float norm[2][kChunk][2];    // sums of squares per channel half
  float beta[kChunk];
};

__device__ __forceinline__ float tf32_hi(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return __uint_as_float(r);
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], const float (&a)[4], float b0, float b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
        "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Eight values as FP16 (hi), and what that leaves (lo).
__device__ __forceinline__ uint4 half8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void split8(const float (&x)[8], uint4 &hi, uint4 &lo) {
  uint32_t w[4], v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x[2 * i] - f.x, x[2 * i + 1] - f.y);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
    v[i] = *reinterpret_cast<const uint32_t *>(&l);
  }
  hi = make_uint4(w[0], w[1], w[2], w[3]);
  lo = make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void unpack8f(uint4 b, float (&f)[8]) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void scaled8(const float (&x)[8], const float *fac, float (&out)[8]) {
  const float4 a = lds4(fac), b = lds4(fac + 4);
  const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = x[i] * f[i];
}

// Where the 16-byte piece of channels c .. c + 7 (or columns) of row t lies.
__device__ __forceinline__ uint32_t img_at(int t, int c) {
  return (uint32_t)(c >> 6) * kImgBlock + (uint32_t)t * 128u +
         (uint32_t)((((c & 63) >> 3) ^ (t & 7)) << 4);
}

__global__ void __launch_bounds__(kPrepThreads, 2) kda_prefill_prep_kernel(const PrefillParams p) {
  extern __shared__ __align__(16) uint8_t prep_raw[];
  PrepSmem &sm = *reinterpret_cast<PrepSmem *>(prep_raw);
  const int chunk = blockIdx.x / p.r.H, h = blockIdx.x - chunk * p.r.H;
  if (chunk >= *p.n_chunks) return;
  const PrefillChunk ck = p.chunks[chunk];
  uint8_t *img = p.images + ((long long)chunk * p.r.H + h) * kImgBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = warp >> 1, hf = warp & 1, g = lane >> 2, tig = lane & 3;
  const int row[2] = {16 * blk + g, 16 * blk + g + 8};
  const int ch0 = hf * 64 + tig * 8;  // slices add 0 and 32

  // -- loads; log2 decays and their sums over the block's tokens ------------
  uint4 kraw[2][2], qraw[2][2];  // [slice][token]
  float d[2][2][8];              // log2 decay sums around the block's middle
  {
    uint4 graw[2][2];
#pragma unroll
    for (int sl = 0; sl < 2; ++sl)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        kraw[sl][r] = qraw[sl][r] = graw[sl][r] = make_uint4(0, 0, 0, 0);
        if (row[r] < ck.count) {
          const long long at =
              ((long long)(ck.t0 + row[r]) * p.r.H + h) * kDim + ch0 + 32 * sl;
          kraw[sl][r] = __ldg(reinterpret_cast<const uint4 *>(p.r.k + at));
          graw[sl][r] = __ldg(reinterpret_cast<const uint4 *>(p.r.g + at));
          qraw[sl][r] = __ldg(reinterpret_cast<const uint4 *>(p.r.q + at));
        }
      }
    if (threadIdx.x < kChunk) {
      float b = 0.f;
      if ((int)threadIdx.x < ck.count)
        b = 1.f / (1.f + __expf(-bf16_bits_to_f32(
                             p.r.beta[(long long)(ck.t0 + threadIdx.x) * p.r.H + h])));
      sm.beta[threadIdx.x] = b;
    }
    const float al = expf(p.r.A_log[h]) * kLog2e, lb2 = p.r.lower_bound * kLog2e;
#pragma unroll
    for (int sl = 0; sl < 2; ++sl) {
      const float4 da = *reinterpret_cast<const float4 *>(p.r.dt_bias + h * kDim + ch0 + 32 * sl);
      const float4 db =
          *reinterpret_cast<const float4 *>(p.r.dt_bias + h * kDim + ch0 + 32 * sl + 4);
      const float dt[8] = {da.x, da.y, da.z, da.w, db.x, db.y, db.z, db.w};
      float ta[8], tb[8];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float raw[8];
        unpack8f(graw[sl][r], raw);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x = lb2 * __fdividef(1.f, 1.f + exp2f_fast(fmaf(-al, raw[e], -al * dt[e])));
          if (row[r] >= ck.count) x = 0.f;
          // inclusive sum over the 8 tokens of this half
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, x, 4 * o);
            if (g >= o) x += y;
          }
          const float t = __shfl_sync(0xffffffffu, x, 28 + tig);
          d[sl][r][e] = r == 0 ? x - t : x;
          if (r == 0) ta[e] = t;
          else tb[e] = t;
        }
      }
      if (g == 0) {
        float *pa = &sm.tot[0][blk][ch0 + 32 * sl], *pb = &sm.tot[1][blk][ch0 + 32 * sl];
        sts4(pa, make_float4(ta[0], ta[1], ta[2], ta[3]));
        sts4(pa + 4, make_float4(ta[4], ta[5], ta[6], ta[7]));
        sts4(pb, make_float4(tb[0], tb[1], tb[2], tb[3]));
        sts4(pb + 4, make_float4(tb[4], tb[5], tb[6], tb[7]));
      }
    }
  }
  // -- norms: sums of squares over this warp's channels ----------------------
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float ks = 0.f, qs = 0.f;
#pragma unroll
    for (int sl = 0; sl < 2; ++sl) {
      float f[8];
      unpack8f(kraw[sl][r], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ks = fmaf(f[e], f[e], ks);
      unpack8f(qraw[sl][r], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) qs = fmaf(f[e], f[e], qs);
    }
    ks += __shfl_xor_sync(0xffffffffu, ks, 1);
    qs += __shfl_xor_sync(0xffffffffu, qs, 1);
    ks += __shfl_xor_sync(0xffffffffu, ks, 2);
    qs += __shfl_xor_sync(0xffffffffu, qs, 2);
    if (tig == 0) {
      sm.norm[hf][row[r]][0] = ks;
      sm.norm[hf][row[r]][1] = qs;
    }
  }
  __syncthreads();

  // -- per (block, channel) factors, times the images' scale -----------------
  // kind 0: from a token to the chunk's start (on 2^(G_t - mid))
  //      1: from the chunk's end back to a token (on 2^(mid - G_s))
  //      2, 3: to the border at 16 / 48, and at 32 (even and first blocks
  //            hold the columns s, odd and last ones the rows t)
  {
    const int c = threadIdx.x & 127;
    float ta[4], tb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ta[j] = sm.tot[0][j][c];
      tb[j] = sm.tot[1][j][c];
    }
    const float t0 = ta[0] + tb[0], t1 = ta[1] + tb[1], t2 = ta[2] + tb[2], t3 = ta[3] + tb[3];
    const auto put = [&](int kind, int j, float x) {
      sm.fac[kind][j][c] = kImgScale * exp2f_fast(x);
    };
    if (threadIdx.x < 128) {
      put(0, 0, ta[0]);
      put(0, 1, t0 + ta[1]);
      put(1, 0, tb[0] + t1 + t2 + t3);
      put(1, 1, tb[1] + t2 + t3);
      put(2, 0, tb[0]);
      put(2, 1, ta[1]);
      put(3, 0, tb[0] + t1);
      put(3, 1, tb[1]);
      reinterpret_cast<float *>(img + kImgDecay)[c] = exp2f_fast(t0 + t1 + t2 + t3);
    } else {
      put(0, 2, t0 + t1 + ta[2]);
      put(0, 3, t0 + t1 + t2 + ta[3]);
      put(1, 2, tb[2] + t3);
      put(1, 3, tb[3]);
      put(2, 2, tb[2]);
      put(2, 3, ta[3]);
      put(3, 2, ta[2]);
      put(3, 3, t2 + ta[3]);
    }
  }
  float rk[2], rq[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    rk[r] = rsqrtf(sm.norm[0][row[r]][0] + sm.norm[1][row[r]][0] + kNormEps);
    rq[r] = rsqrtf(sm.norm[0][row[r]][1] + sm.norm[1][row[r]][1] + kNormEps);
  }
  __syncthreads();

  // -- the block's own products, and the operands of everything else ---------
  float dk[2][4], dq[2][4];  // [n-tile] 16 x 8 of kn kn^T and qn kn^T
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) dk[n][i] = dq[n][i] = 0.f;
#pragma unroll
  for (int sl = 0; sl < 2; ++sl) {
    const int c = ch0 + 32 * sl;
    float kf[2][8], kg[2][8], qf[2][8];  // kn 2^(G - mid), kn 2^(mid - G), qn 2^(G - mid)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float k[8], q[8];
      unpack8f(kraw[sl][r], k);
      unpack8f(qraw[sl][r], q);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = exp2f_fast(d[sl][r][e]), b = exp2f_fast(-d[sl][r][e]);
        const float kn = k[e] * rk[r];
        kf[r][e] = kn * f;
        kg[r][e] = kn * b;
        qf[r][e] = q[e] * rq[r] * f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      // columns tig and tig + 4 of the operand are channels e and e + 1
      float a[4] = {kf[0][e], kf[1][e], kf[0][e + 1], kf[1][e + 1]};
      float ah[4], alo[4], aq[4] = {qf[0][e], qf[1][e], qf[0][e + 1], qf[1][e + 1]};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ah[i] = tf32_hi(a[i]);
        alo[i] = a[i] - ah[i];
        aq[i] = tf32_hi(aq[i]);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float b0 = tf32_hi(kg[n][e]), b1 = tf32_hi(kg[n][e + 1]);
        mma_tf32(dk[n], alo, b0, b1);
        mma_tf32(dk[n], ah, kg[n][e] - b0, kg[n][e + 1] - b1);
        mma_tf32(dk[n], ah, b0, b1);
        mma_tf32(dq[n], aq, b0, b1);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float x[8];
      uint4 hi, lo;
      const uint32_t at = img_at(row[r], c);
      scaled8(kf[r], &sm.fac[0][blk][c], x);
      split8(x, hi, lo);
      *reinterpret_cast<uint4 *>(img + kImgKdHi + at) = hi;
      *reinterpret_cast<uint4 *>(img + kImgKdLo + at) = lo;
      scaled8(qf[r], &sm.fac[0][blk][c], x);
      *reinterpret_cast<uint4 *>(img + kImgQd + at) = half8(x);
      scaled8(kg[r], &sm.fac[1][blk][c], x);
      split8(x, hi, lo);
      *reinterpret_cast<uint4 *>(img + kImgKeHi + at) = hi;
      *reinterpret_cast<uint4 *>(img + kImgKeLo + at) = lo;
      const uint32_t xat = (uint32_t)row[r] * kXPitch + (uint32_t)c * 2;
      scaled8((blk & 1) ? kf[r] : kg[r], &sm.fac[2][blk][c], x);
      split8(x, hi, lo);
      *reinterpret_cast<uint4 *>(sm.u.x.x16_hi + xat) = hi;
      *reinterpret_cast<uint4 *>(sm.u.x.x16_lo + xat) = lo;
      scaled8(blk >= 2 ? kf[r] : kg[r], &sm.fac[3][blk][c], x);
      split8(x, hi, lo);
      *reinterpret_cast<uint4 *>(sm.u.x.x32_hi + xat) = hi;
      *reinterpret_cast<uint4 *>(sm.u.x.x32_lo + xat) = lo;
      if (blk & 1) {
        scaled8(qf[r], &sm.fac[2][blk][c], x);
        *reinterpret_cast<uint4 *>(sm.u.x.y16 +
                                   (uint32_t)((blk >> 1) * 16 + g + 8 * r) * kXPitch + c * 2) =
            half8(x);
      }
      if (blk >= 2) {
        scaled8(qf[r], &sm.fac[3][blk][c], x);
        *reinterpret_cast<uint4 *>(sm.u.x.y32 +
                                   (uint32_t)((blk - 2) * 16 + g + 8 * r) * kXPitch + c * 2) =
            half8(x);
      }
    }
  }
  if (hf == 1) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = (g + 8 * (i >> 1)) * kDPitch + 8 * n + 2 * tig + (i & 1);
        sm.part[blk][0][at] = dk[n][i];
        sm.part[blk][1][at] = dq[n][i];
      }
  }
  __syncthreads();

  // -- products between blocks: warps 0-3 the quarters of rows 32 .. 63 by
  //    columns 0 .. 31, warps 4 and 5 blocks 1 by 0 and 3 by 2 ---------------
  float ok[2][4], oq[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) ok[n][i] = oq[n][i] = 0.f;
  int r0 = 0, c0 = 0;
  if (warp < 6) {
    const uint8_t *xh = sm.u.x.x32_hi, *xl = sm.u.x.x32_lo, *y = sm.u.x.y32;
    int y0;
    if (warp < 4) {
      r0 = 32 + 16 * (warp >> 1);
      c0 = 16 * (warp & 1);
      y0 = r0 - 32;
    } else {
      r0 = 32 * (warp - 4) + 16;
      c0 = r0 - 16;
      y0 = 16 * (warp - 4);
      xh = sm.u.x.x16_hi;
      xl = sm.u.x.x16_lo;
      y = sm.u.x.y16;
    }
    const uint32_t arow = (uint32_t)(lane & 15) * kXPitch + (uint32_t)(lane >> 4) * 16;
    const uint32_t brow = (uint32_t)((lane & 7) + ((lane >> 4) << 3)) * kXPitch +
                          (uint32_t)((lane >> 3) & 1) * 16;
    const uint32_t ah0 = smem_u32(xh) + r0 * kXPitch + arow;
    const uint32_t al0 = smem_u32(xl) + r0 * kXPitch + arow;
    const uint32_t aq0 = smem_u32(y) + y0 * kXPitch + arow;
    const uint32_t bh0 = smem_u32(xh) + c0 * kXPitch + brow;
    const uint32_t bl0 = smem_u32(xl) + c0 * kXPitch + brow;
#pragma unroll 2
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t ah[4], al[4], aq[4], bh[4], bl[4];
      ldmatrix4(ah, ah0 + ks * 32);
      ldmatrix4(al, al0 + ks * 32);
      ldmatrix4(aq, aq0 + ks * 32);
      ldmatrix4(bh, bh0 + ks * 32);
      ldmatrix4(bl, bl0 + ks * 32);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        mma_f16(ok[n], al, bh[2 * n], bh[2 * n + 1]);
        mma_f16(ok[n], ah, bl[2 * n], bl[2 * n + 1]);
        mma_f16(ok[n], ah, bh[2 * n], bh[2 * n + 1]);
        mma_f16(oq[n], aq, bh[2 * n], bh[2 * n + 1]);
      }
    }
  }
  __syncthreads();  // the operands have been read: L and X take their place

  float *L = sm.u.s.L, *X = sm.u.s.X, *Y = sm.u.s.Y;
  const auto put_a = [&](int t, int s, float x0, float x1) {  // s even
    const __half2 a = __floats2half2_rn(x0, x1);
    *reinterpret_cast<__half2 *>(img + kImgA + img_at(t, s & ~7) + (s & 7) * 2) = a;
  };
  if (warp < 6) {
    constexpr float kUnit = 1.f / (kImgScale * kImgScale);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const int t = r0 + g + 4 * i, s = c0 + 8 * n + 2 * tig;
        const float b = sm.beta[t] * kUnit;
        L[t * kLPitch + s] = b * ok[n][i];
        L[t * kLPitch + s + 1] = b * ok[n][i + 1];
        put_a(t, s, oq[n][i] * (kImgScale * kUnit), oq[n][i + 1] * (kImgScale * kUnit));
      }
  }
  if (hf == 0) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const int tl = g + 4 * i, s0 = 8 * n + 2 * tig, t = 16 * blk + tl;
        const float *pk = &sm.part[blk][0][tl * kDPitch + s0];
        const float *pq = &sm.part[blk][1][tl * kDPitch + s0];
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // (above the diagonal the factors may have overflowed: dropped, not
          // multiplied by zero)
          L[t * kLPitch + 16 * blk + s0 + e] =
              s0 + e < tl ? sm.beta[t] * (dk[n][i + e] + pk[e]) : 0.f;
          a[e] = s0 + e <= tl ? (dq[n][i + e] + pq[e]) * kImgScale : 0.f;
        }
        put_a(t, 16 * blk + s0, a[0], a[1]);
      }
  } else {
    // A above its diagonal blocks: zeros
    for (int i = lane; i < 16 * (6 - 2 * blk); i += 32) {
      const int t = 16 * blk + (i & 15), piece = 2 * (blk + 1) + (i >> 4);
      *reinterpret_cast<uint4 *>(img + kImgA + img_at(t, 8 * piece)) = make_uint4(0, 0, 0, 0);
    }
  }
  __syncthreads();

  // -- X = (I + L)^-1: its diagonal blocks by columns, then the rest ---------
  if (warp < 4) {
    const int j = lane & 15;
    float x[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) x[t] = t == j ? 1.f : 0.f;
    const float *Lb = L + (16 * warp) * kLPitch + 16 * warp;
#pragma unroll
    for (int t = 0; t < 15; ++t)
#pragma unroll
      for (int u = t + 1; u < 16; ++u) x[u] = fmaf(-Lb[u * kLPitch + t], x[t], x[u]);
    if (lane < 16) {
#pragma unroll
      for (int t = 0; t < 16; ++t) X[(16 * warp + t) * kLPitch + 16 * warp + j] = x[t];
    }
  }
  __syncthreads();
  {
    // X10 = -X11 (L10 X00) and X32 = -X33 (L32 X22), 16 x 16 each
    const int pr = threadIdx.x >> 7, r = (threadIdx.x & 127) >> 3, c = (threadIdx.x & 7) * 2;
    const int lo = 32 * pr, hi = lo + 16;
    float y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float l = L[(hi + r) * kLPitch + lo + k];
      const float2 x = *reinterpret_cast<const float2 *>(&X[(lo + k) * kLPitch + lo + c]);
      y0 = fmaf(l, x.x, y0);
      y1 = fmaf(l, x.y, y1);
    }
    *reinterpret_cast<float2 *>(&Y[r * kLPitch + 32 * pr + c]) = make_float2(y0, y1);
    __syncthreads();
    float z0 = 0.f, z1 = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float l = X[(hi + r) * kLPitch + hi + k];
      const float2 x = *reinterpret_cast<const float2 *>(&Y[k * kLPitch + 32 * pr + c]);
      z0 = fmaf(l, x.x, z0);
      z1 = fmaf(l, x.y, z1);
    }
    *reinterpret_cast<float2 *>(&X[(hi + r) * kLPitch + lo + c]) = make_float2(-z0, -z1);
    // above the diagonal of the two halves
    *reinterpret_cast<float2 *>(&X[(lo + r) * kLPitch + hi + c]) = make_float2(0.f, 0.f);
    __syncthreads();
  }
  {
    // the lower left 32 x 32: -X[32.., 32..] (L[32.., ..32] X[..32, ..32])
    const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < 32; ++k) y = ffma4s(L[(32 + r) * kLPitch + k], lds4(&X[k * kLPitch + c]), y);
    sts4(&Y[r * kLPitch + c], y);
    __syncthreads();
    float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < 32; ++k)
      z = ffma4s(-X[(32 + r) * kLPitch + 32 + k], lds4(&Y[k * kLPitch + c]), z);
    sts4(&X[(32 + r) * kLPitch + c], z);
    __syncthreads();
  }
  // -- T = X diag(beta) ------------------------------------------------------
  {
    const int t = threadIdx.x >> 2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int s0 = (threadIdx.x & 3) * 16 + 8 * e;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = s0 + i <= t ? X[t * kLPitch + s0 + i] * (sm.beta[s0 + i] * kImgScale) : 0.f;
      uint4 hi, lo;
      split8(x, hi, lo);
      const uint32_t at = img_at(t, s0);
      *reinterpret_cast<uint4 *>(img + kImgTHi + at) = hi;
      *reinterpret_cast<uint4 *>(img + kImgTLo + at) = lo;
    }
  }
}

}  // namespace

int launch_prefill_prep(const PrefillParams &p, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute(kda_prefill_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(PrepSmem)) != cudaSuccess)
      return KDA_ERR_CUDA;
    configured.fetch_or(bit);
  }
  static_assert(2 * (sizeof(PrepSmem) + 1024) <= 228 * 1024, "two CTAs per SM");
  kda_prefill_prep_kernel<<<(unsigned)(p.max_chunks * p.r.H), kPrepThreads, sizeof(PrepSmem),
                            stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda

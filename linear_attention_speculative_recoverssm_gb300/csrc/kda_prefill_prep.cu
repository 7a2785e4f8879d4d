// The preparation of the chunked delta rule: the images of every (chunk,
// head) (kda_prefill.cuh).  One CTA of 8 warps each; warps 2 i and 2 i + 1
// own the 16 tokens of block i.
//
// The products need e^{G_t - G_s} per channel, whose two factors must stay
// representable.  Within a block of 16 they are taken from its middle,
// 2^(G_t - mid) and 2^(mid - G_s), at most 2^116 with the steepest gate, and
// the 16 x 16 products run in TF32 (8 exponent bits) straight from the
// registers that hold the factors: lane 4 g + j of a warp holds tokens g and
// g + 8 and eight consecutive channels of every 32, half of the channels in
// each of the two warps.  Between blocks a border lies between s and t, and
// both factors, from t back to it and from it back to s, are at most 1:
// blocks 0-1 | 2-3 with the border at token 32, blocks 0 | 1 and 2 | 3 with
// theirs at 16 and 48, in FP16 parts through shared memory.  The key products
// and the query products take hi.hi + hi.lo + lo.hi.
//
// The references are powers of two: with B_i the sum of the log2 decays
// before block i rounded to an integer, a row operand is R_t = kn_t
// 2^(G_t - B_i) and a column operand C_s = kn_s 2^(B_{i+1} - G_s), split into
// FP16 parts once; from another block's border, or the chunk's start, they
// are the same parts times an exact 2^n.
//
// What bounds it: 265 chunks of 32 heads read 0.42 GB and write 1.1 GB, 225 us at
// a copy's rate, and take 373.  16 warps an SM is what registers (128, with 20
// bytes spilled) and shared memory leave room for; they issue every other cycle,
// the operands' pass on exponents, FP16 splits and their stores.  (Splits by a
// conversion of the high part in place of a multiply-add of FP16 to FP32: 382.)
// With the high parts of the query operands alone it took 327; then, laid out
// without care for banks, and with A and T stored from registers, 342, and with
// an item to a CTA, without the next one's inputs on their way, 415.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/kda_recoverssm.h"
#include "kda_launch.h"
#include "kda_prefill.cuh"
#include "kda_tensor_map.h"

namespace kda {
namespace {

constexpr int kPrepThreads = 256;
constexpr uint32_t kXPitch = 256;  // bytes of a 128-channel FP16 row
constexpr uint32_t kXBytes = kChunk * kXPitch;
constexpr uint32_t kX3Bytes = 48 * kXPitch;  // three blocks' rows
// Pitches (floats): rows four or eight banks apart, as their readers want.
constexpr int kLPitch = 36, kL16Pitch = 20, kXPitchF = 68, kYPitch = 40, kLtPitch = 20;
constexpr int kLtSize = 16 * kLtPitch + 16;  // (two blocks apart by half the banks)
constexpr uint32_t kRowsBytes = kChunk * kDim * 2;  // a chunk's rows of an input

// Where columns c .. c + 3 of row r of a 16 x 16 block lie: pieces of 16 bytes,
// of eight rows one each meet every bank.
__device__ __forceinline__ int part_at(int r, int c) {
  return 16 * r + (((c >> 2) ^ ((r >> 1) & 3)) << 2);
}

// Shared memory, by phases: the FP16 operands of the products between blocks;
// then, in their place, L between blocks, X = (I + L)^-1 and a scratch matrix,
// and behind those the next item's q, k and raw_g as they arrive.
struct PrepSmem {
  union {
    struct {
      // (before they hold operands, x16_hi and x16_lo hold the log2 decay
      // sums of each half block: of a 16-byte piece's eight channels the first
      // and last four)
      uint8_t x16_hi[kXBytes], x16_lo[kXBytes];
      // of 32, blocks 0 .. 2 (block 3's are its rows of 48 times powers of two)
      uint8_t x32_hi[kX3Bytes], x32_lo[kX3Bytes];
      uint8_t y_hi[kX3Bytes], y_lo[kX3Bytes];  // query rows of blocks 1 .. 3
    } x;
    struct {
      float L[32 * kLPitch];          // rows 32 .. 63 by columns 0 .. 31
      float L16[2][16 * kL16Pitch];   // blocks 1 by 0, 3 by 2
      float X[kChunk * kXPitchF], Y[32 * kYPitch];
    } s;
    struct {
      uint8_t before[2 * kXBytes];    // (the decay sums are made from g)
      uint8_t g[kRowsBytes], q[kRowsBytes], k[kRowsBytes];
    } in;
  } u;
  union {
    struct {
      union {
        float fac[3][4][128];        // [R, C, Ke][block][channel], times their scales
        float Lt[4][kLtSize];        // then the diagonal blocks of L, transposed
      };
      uint16_t pow[4][128];    // FP16 2^n: of Kd and Qd
      uint16_t pow32[2][128];  // of the operands at 32, blocks 0 and 3
      float tot[2][4][128];    // log2 decays of a block's two halves
      float norm[2][kChunk][2];  // sums of squares per channel half
    };
    __align__(16) uint8_t a[2 * kImgBlock];  // then the image's A
  };
  union {
    // a block's products kn kn^T and qn kn^T, over either half of the channels
    __align__(16) float part[4][2][2][16 * 16];
    uint8_t t[2 * kImgBlock];  // then the image's T
  };
  float beta[kChunk];
  uint64_t landed;  // the item's q, k and raw_g are there
};
static_assert(sizeof(PrepSmem::u.s) <= sizeof(PrepSmem::u.in.before), "inputs behind X");

// q, k and raw_g [n_tokens, H, 128] as 3-D tensors, a chunk's rows of one head
// a copy.
struct PrepMaps {
  CUtensorMap g, q, k;
};

// Rows r of 256 bytes: 16-byte pieces, each 128-byte half permuted so that
// one piece of eight consecutive rows, and four pieces of two, meet every
// bank once.
__device__ __forceinline__ uint32_t x_at(int r, int piece) {
  const int f = ((r & 1) << 2) | ((r >> 1) & 3);
  return (uint32_t)r * kXPitch + (uint32_t)(piece >> 3) * 128u +
         (uint32_t)(((piece & 7) ^ f) << 4);
}

// 2^x, as exp2f_fast but for results below 2^-126, which are not flushed.
__device__ __forceinline__ float exp2f_subnormal(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest of a warp's non-negative values.
__device__ __forceinline__ float warp_max(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// The power of two above the chunk's largest beta, 2^-100 at least: every warp
// for itself.
__device__ __forceinline__ float beta_power(const float *beta, int lane) {
  const float m = warp_max(fmaxf(beta[lane], beta[lane + 32]));
  const int e = (int)(__float_as_uint(m) >> 23) + 1;
  return __uint_as_float((uint32_t)min(max(e, 27), 128) << 23);
}

// The leading 11 bits of x (truncated).
__device__ __forceinline__ float tf32_hi(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffffe000u);
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

__device__ __forceinline__ uint32_t h2_bits(__half2 h) {
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight values (four pairs) as FP16, and what that leaves.
__device__ __forceinline__ void split8(const float2 (&x)[4], uint4 &hi, uint4 &lo) {
  uint32_t w[4], v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __float22half2_rn(x[i]);
    w[i] = h2_bits(h);
    v[i] = h2_bits(__float22half2_rn(less_half(x[i], h)));
  }
  hi = make_uint4(w[0], w[1], w[2], w[3]);
  lo = make_uint4(v[0], v[1], v[2], v[3]);
}

// Eight FP16 values times powers of two.
__device__ __forceinline__ uint4 scale8(uint4 x, uint4 f) {
  uint4 r;
  const auto mul = [](uint32_t a, uint32_t b) {
    return h2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&a),
                           *reinterpret_cast<const __half2 *>(&b)));
  };
  r.x = mul(x.x, f.x);
  r.y = mul(x.y, f.y);
  r.z = mul(x.z, f.z);
  r.w = mul(x.w, f.w);
  return r;
}

// An operand's 16 x 16 tile times powers of two by channel: the first and the
// last eight channels' at this lane's place.
__device__ __forceinline__ void scale_rows(uint32_t (&x)[4], uint32_t p0, uint32_t p1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = i < 2 ? p0 : p1;
    x[i] = h2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&x[i]),
                           *reinterpret_cast<const __half2 *>(&p)));
  }
}

__device__ __forceinline__ float2 bf16x2_f32(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ void unpack4x2(uint4 b, float2 (&f)[4]) {
  f[0] = bf16x2_f32(b.x);
  f[1] = bf16x2_f32(b.y);
  f[2] = bf16x2_f32(b.z);
  f[3] = bf16x2_f32(b.w);
}

__device__ __forceinline__ void load4x2(const float *p, float2 (&f)[4]) {
  const float4 a = lds4(p), b = lds4(p + 4);
  f[0] = make_float2(a.x, a.y);
  f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y);
  f[3] = make_float2(b.z, b.w);
}

// C[16 x 8] = A[16 x 8 steps] B[8 steps x 8], FP32 operands in shared memory
// as TF32 parts, from step `first` on.
__device__ __forceinline__ void tile_mm(float (&c)[4], const float *A, int lda, const float *B,
                                        int ldb, int first, int steps, int lane) {
  const int g = lane >> 2, t = lane & 3;
  float c1[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = 0.f;
  for (int ks = first; ks < steps; ++ks) {
    const float a[4] = {A[g * lda + 8 * ks + t], A[(g + 8) * lda + 8 * ks + t],
                        A[g * lda + 8 * ks + t + 4], A[(g + 8) * lda + 8 * ks + t + 4]};
    const float b0 = B[(8 * ks + t) * ldb + g], b1 = B[(8 * ks + t + 4) * ldb + g];
    float h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = tf32_hi(a[i]);
      l[i] = a[i] - h[i];
    }
    const float h0 = tf32_hi(b0), h1 = tf32_hi(b1);
    mma_tf32(c1, l, h0, h1);
    mma_tf32(c2, h, b0 - h0, b1 - h1);
    mma_tf32(c, h, h0, h1);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] += c1[i] + c2[i];
}

// Shared memory to global memory, asynchronously (the writes were fenced and
// waited for); both 16-byte aligned.
__device__ __forceinline__ void bulk_store(uint8_t *to, const uint8_t *from, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to),
               "r"(smem_u32(from)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// This thread's stores but the N last have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void bulk_stores_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Where the 16-byte piece of channels c .. c + 7 (or columns) of row t lies.
__device__ __forceinline__ uint32_t img_at(int t, int c) {
  return (uint32_t)(c >> 6) * kImgBlock + (uint32_t)t * 128u +
         (uint32_t)((((c & 63) >> 3) ^ (t & 7)) << 4);
}

__device__ __forceinline__ int pair_of(int tid) {
  return (tid & 32) | ((tid & 14) << 1) | ((tid & 16) >> 3) | (tid & 1);
}

__global__ void __launch_bounds__(kPrepThreads, 2)
    kda_prefill_prep_kernel(const PrefillParams p, const __grid_constant__ PrepMaps maps,
                            int segment) {
  extern __shared__ __align__(1024) uint8_t prep_raw[];
  PrepSmem &sm = *reinterpret_cast<PrepSmem *>(prep_raw);
  const int H = p.r.H;
  // The first segment waits for the list; the others start once the chain
  // before them has seen the preparation before it, and so the list, complete.
  if (segment == 0) grid_dependency_wait();
  grid_launch_dependents();
  const int first = p.seg_first[segment];
  const int n_items = (p.seg_first[segment + 1] - first) * H;
  if ((int)blockIdx.x >= n_items) {
    if (blockIdx.x == 0 && threadIdx.x == 0) grid_dependency_wait();
    return;
  }
  // CTAs stay, two to an SM.  An item's rows arrive (one copy each) while the
  // one before it takes its last steps, which need little of the shared memory.
  const auto fetch = [&](const PrefillChunk &ck, int h) {
    mbar_arrive_expect_tx(&sm.landed, 3 * kRowsBytes);
    tma_load_3d(sm.u.in.g, &maps.g, 0, h, ck.t0, &sm.landed);
    tma_load_3d(sm.u.in.q, &maps.q, 0, h, ck.t0, &sm.landed);
    tma_load_3d(sm.u.in.k, &maps.k, 0, h, ck.t0, &sm.landed);
  };
  uint16_t braw = 0;
  float a_log = 0.f;
  float2 dt = make_float2(0.f, 0.f);
  const auto load_head = [&](int tid, const PrefillChunk &ck, int h) {
    braw = __ldg(p.r.beta + (long long)(ck.t0 + min(tid & 63, ck.count - 1)) * H + h);
    a_log = __ldg(p.r.A_log + h);
    dt = __ldg(reinterpret_cast<const float2 *>(p.r.dt_bias + h * kDim) + pair_of(tid));
  };
  int chunk = blockIdx.x / H, h = blockIdx.x - chunk * H;
  const int chunk_step = gridDim.x / H, h_step = gridDim.x - chunk_step * H;
  const PrefillChunk *const chunks = p.chunks + first;
  uint8_t *const images = p.images + (long long)first * H * kImgBytes;
  PrefillChunk ck = chunks[chunk];
  if (threadIdx.x == 0) {
    mbar_init(&sm.landed, 1);
    mbar_init_fence();
    fetch(ck, h);
  }
  load_head(threadIdx.x, ck, h);
  __syncthreads();
  uint32_t phase = 0;
  for (int item = blockIdx.x; item < n_items; item += gridDim.x, phase ^= 1u) {
  // (a value that the compiler takes for new each time: the many addresses
  // that follow from it are then made again, not kept through the loop in
  // registers that the steps need)
  int tid = threadIdx.x;
  asm volatile("" : "+r"(tid));
  const int warp = tid >> 5, lane = tid & 31;
  const int blk = warp >> 1, hf = warp & 1, g = lane >> 2, tig = lane & 3;
  const int row[2] = {16 * blk + g, 16 * blk + g + 8};
  const int ch0 = hf * 64 + tig * 8;  // slices add 0 and 32
  // A pair of channels, for the decays: half a warp takes the first four
  // channels of eight pieces, the other half the last four.
  const int pr = pair_of(tid);
  const int last = ck.count - 1;
  uint8_t *img = images + (long long)item * kImgBytes;
  // the next item
  chunk += chunk_step;
  h += h_step;
  if (h >= H) {
    h -= H;
    ++chunk;
  }
  const bool more = item + (int)gridDim.x < n_items;
  const PrefillChunk next = chunks[more ? chunk : 0];

  const bool here = mbar_wait_bounded(&sm.landed, phase);
  if (tid == 0) bulk_stores_read<1>();  // A's place is free (T, asked for last, may not be)
  if (__syncthreads_or(!here)) {  // (nothing else can run out in this kernel)
    if (tid == 0) {
      report(p.r.maps.status, KDA_ERR_TIMEOUT);
      mbar_wait_bounded(&sm.landed, phase);  // (once more for the copies in flight)
    }
    break;
  }
  // Rows past the chunk's tokens take its last token's inputs (their own may
  // be another request's) and get no weight: decay 1, kn = qn = 0, beta = 0.
  // (rows g and g + 1 lie in the same banks: odd rows take their slices the
  // other way round)
  uint4 kraw[2][2], qraw[2][2];  // [slice][token]
  const bool odd = g & 1;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t at = (uint32_t)min(row[r], last) * (kDim * 2) + (uint32_t)ch0 * 2;
    const uint32_t at0 = at + (odd ? 64u : 0u), at1 = at + (odd ? 0u : 64u);
    const auto swap = [&](uint4 &x, uint4 &y) {
      const uint4 u = odd ? y : x;
      y = odd ? x : y;
      x = u;
    };
    kraw[0][r] = *reinterpret_cast<const uint4 *>(sm.u.in.k + at0);
    kraw[1][r] = *reinterpret_cast<const uint4 *>(sm.u.in.k + at1);
    swap(kraw[0][r], kraw[1][r]);
    qraw[0][r] = *reinterpret_cast<const uint4 *>(sm.u.in.q + at0);
    qraw[1][r] = *reinterpret_cast<const uint4 *>(sm.u.in.q + at1);
    swap(qraw[0][r], qraw[1][r]);
  }
  // -- log2 decays and their sums over each half of the block: a thread takes
  //    two channels and the block's 16 tokens in turn -------------------------
  {
    const int c = 2 * pr;
    if (tid < kChunk)
      sm.beta[tid] = tid <= last ? 1.f / (1.f + __expf(-bf16_bits_to_f32(braw))) : 0.f;
    const float al = expf(a_log) * kLog2e, lb2 = p.r.lower_bound * kLog2e;
    const float2 off = make_float2(-al * dt.x, -al * dt.y), nal = make_float2(-al, -al);
    uint8_t *to = ((pr & 2) ? sm.u.x.x16_lo : sm.u.x.x16_hi) + (pr & 1) * 8 + 16 * blk * kXPitch;
    const uint32_t at = x_at(0, pr >> 2);
    const uint8_t *from = sm.u.in.g + 4 * pr;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = 8 * r + i;
        const uint32_t raw = *reinterpret_cast<const uint32_t *>(
            from + (uint32_t)min(16 * blk + t, last) * (kDim * 2));
        const float2 z = ffma2(nal, bf16x2_f32(raw), off);
        const float w = 16 * blk + t <= last ? lb2 : 0.f;
        sum.x += __fdividef(w, 1.f + exp2f_fast(z.x));
        sum.y += __fdividef(w, 1.f + exp2f_fast(z.y));
        *reinterpret_cast<float2 *>(to + (at ^ x_at(i, 0) ^ (i * kXPitch)) + t * kXPitch) = sum;
      }
      *reinterpret_cast<float2 *>(&sm.tot[r][blk][c]) = sum;
    }
  }
  // -- norms: sums of squares over this warp's channels ----------------------
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float2 ks = make_float2(0.f, 0.f), qs = ks;
#pragma unroll
    for (int sl = 0; sl < 2; ++sl) {
      float2 f[4];
      unpack4x2(kraw[sl][r], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) ks = ffma2(f[e], f[e], ks);
      unpack4x2(qraw[sl][r], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) qs = ffma2(f[e], f[e], qs);
    }
    float kk = ks.x + ks.y, qq = qs.x + qs.y;
    kk += __shfl_xor_sync(0xffffffffu, kk, 1);
    qq += __shfl_xor_sync(0xffffffffu, qq, 1);
    kk += __shfl_xor_sync(0xffffffffu, kk, 2);
    qq += __shfl_xor_sync(0xffffffffu, qq, 2);
    if (tig == 0) {
      sm.norm[hf][row[r]][0] = kk;
      sm.norm[hf][row[r]][1] = qq;
    }
  }
  __syncthreads();

  // -- per (block, channel) factors -------------------------------------------
  // With ph_i what the rounding of B_i leaves, summed block by block so that a
  // block's own size, not the sum's, sets the error:
  //   R = kn 2^(G - mid) fac[0], fac[0] = 2^(mid - before + ph_i)
  //   C = kn 2^(mid - G) fac[1], fac[1] = 2^(after - mid - ph_{i+1})
  //   Ke = kn 2^(mid - G) fac[2], from the chunk's end
  {
    const int c = tid & 127;
    float ta[4], tb[4], ph[5], B[5];
    ph[0] = B[0] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ta[j] = sm.tot[0][j][c];
      tb[j] = sm.tot[1][j][c];
      const float x = ph[j] + (ta[j] + tb[j]), n = rintf(x);
      ph[j + 1] = x - n;
      B[j + 1] = B[j] + n;
    }
    // 2^n, n <= 0 an integer (FP16 has it down to 2^-24)
    const auto power = [](float n) {
      return __half_as_ushort(__float2half_rn(exp2f_fast(fmaxf(n, -60.f))));
    };
    if (tid < 128) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sm.fac[0][j][c] = kImgScale * exp2f_fast(ta[j] + ph[j]);
        sm.pow[j][c] = power(B[j]);
      }
      float *const tail = reinterpret_cast<float *>(img + kImgDecay);
      const float end =
          exp2f_fast((ta[0] + tb[0]) + (ta[1] + tb[1]) + (ta[2] + tb[2]) + (ta[3] + tb[3]));
      tail[c] = end;
      const float most = warp_max(end);
      if (lane == 0) tail[kScalEnd + warp] = kEndFactor * (most * most);
    } else {
      float *const tail = reinterpret_cast<float *>(img + kImgDecay);
      float rest = 0.f;
#pragma unroll
      for (int j = 3; j >= 0; --j) {
        sm.fac[1][j][c] = kImgScale * exp2f_fast(tb[j] - ph[j + 1]);
        // (2^-115 and less where a half block forgets that much, times 2^115: not
        // flushed where it is subnormal, which leaves Ke to 2^-34; 6: its scale)
        sm.fac[2][j][c] = exp2f_subnormal(tb[j] + rest + 6.f);
        static_assert(kImgKeScale == 64.f, "2^6");
        if (j < 3) {
          const float most = warp_max(exp2f_fast(rest));
          if (lane == 0) tail[kScalLeft + 4 * j + warp - 4] = kLeftFactor * (most * most);
        }
        rest += ta[j] + tb[j];
      }
      sm.pow32[0][c] = power(B[2] - B[1]);
      sm.pow32[1][c] = power(B[3] - B[2]);
      const float p2 = beta_power(sm.beta, lane);
      if (tid == 128) {
        tail[kScalBeta] = p2;
        tail[kScalValue] = p2 + 64.f * p2 * p2;
      }
    }
  }
  // (queries at Qd's scale throughout)
  constexpr float kQDown = kImgQdScale / kImgScale;
  float rk[2], rq[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    rk[r] = rsqrtf(sm.norm[0][row[r]][0] + sm.norm[1][row[r]][0] + kNormEps);
    rq[r] = rsqrtf(sm.norm[0][row[r]][1] + sm.norm[1][row[r]][1] + kNormEps) * kQDown;
    if (row[r] > last) rk[r] = rq[r] = 0.f;
  }
  if (tid == 0) bulk_stores_read<0>();  // and T's
  __syncthreads();

  // -- the block's own products, and the operands of everything else ---------
  float dk[2][4], dq[2][4];  // [n-tile] 16 x 8 of kn kn^T and qn kn^T
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) dk[n][i] = dq[n][i] = 0.f;
  // Token g's places; token g + 8 lies 8 rows further, and slice 1 four pieces
  // on, which flips bit 6 of the permuted place.
  const uint32_t img0 = img_at(row[0], ch0), x0 = x_at(row[0], ch0 >> 3);
  const uint32_t y0 = x_at((max(blk, 1) - 1) * 16 + g, ch0 >> 3);
#pragma unroll
  for (int sl = 0; sl < 2; ++sl) {
    const int c = ch0 + 32 * sl;
    uint8_t *const im = img + (img0 ^ (64u * sl));
    const uint32_t xs = x0 ^ (64u * sl);
    float2 kf[2][4], kg[2][4], qf[2][4];  // kn 2^(G - mid), kn 2^(mid - G), qn 2^(G - mid)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float2 k[4], q[4];
      unpack4x2(kraw[sl][r], k);
      unpack4x2(qraw[sl][r], q);
      const float4 d0 = *reinterpret_cast<const float4 *>(sm.u.x.x16_hi + xs + 8 * r * kXPitch);
      const float4 d1 = *reinterpret_cast<const float4 *>(sm.u.x.x16_lo + xs + 8 * r * kXPitch);
      float2 d[4] = {make_float2(d0.x, d0.y), make_float2(d0.z, d0.w), make_float2(d1.x, d1.y),
                     make_float2(d1.z, d1.w)};
      if (r == 0) {
        float2 mid[4];
        load4x2(&sm.tot[0][blk][c], mid);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = make_float2(d[e].x - mid[e].x, d[e].y - mid[e].y);
      }
      const float2 rk2 = make_float2(rk[r], rk[r]), rq2 = make_float2(rq[r], rq[r]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = make_float2(exp2f_fast(d[e].x), exp2f_fast(d[e].y));
        const float2 b = make_float2(exp2f_fast(-d[e].x), exp2f_fast(-d[e].y));
        const float2 kn = fmul2(k[e], rk2);
        kf[r][e] = fmul2(kn, f);
        kg[r][e] = fmul2(kn, b);
        qf[r][e] = fmul2(fmul2(q[e], rq2), f);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // columns tig and tig + 4 of the operand are channels 2 e and 2 e + 1
      const float a[4] = {kf[0][e].x, kf[1][e].x, kf[0][e].y, kf[1][e].y};
      const float aq[4] = {qf[0][e].x, qf[1][e].x, qf[0][e].y, qf[1][e].y};
      float ah[4], al[4], qh[4], ql[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ah[i] = tf32_hi(a[i]);
        al[i] = a[i] - ah[i];
        qh[i] = tf32_hi(aq[i]);
        ql[i] = aq[i] - qh[i];
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float h0 = tf32_hi(kg[n][e].x), h1 = tf32_hi(kg[n][e].y);
        const float l0 = kg[n][e].x - h0, l1 = kg[n][e].y - h1;
        mma_tf32(dk[n], al, h0, h1);
        mma_tf32(dk[n], ah, l0, l1);
        mma_tf32(dk[n], ah, h0, h1);
        mma_tf32(dq[n], ql, h0, h1);
        mma_tf32(dq[n], qh, l0, l1);
        mma_tf32(dq[n], qh, h0, h1);
      }
    }
    const uint4 pow32 = *reinterpret_cast<const uint4 *>(&sm.pow32[blk >> 1][c]);
    const auto times = [](const float2 (&x)[4], const float2 (&f)[4], float2 (&y)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmul2(x[e], f[e]);
    };
    const auto put = [](uint8_t *at, uint4 x) { *reinterpret_cast<uint4 *>(at) = x; };
    {
      float2 fac[4], x[4];
      uint4 hi, lo;
      load4x2(&sm.fac[2][blk][c], fac);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        times(kg[r], fac, x);
        split8(x, hi, lo);
        put(im + 1024 * r + kImgKeHi, hi);
        put(im + 1024 * r + kImgKeLo, lo);
      }
    }
    if (blk < 3) {  // columns: of the border at 16 / 48 (even blocks), at 32 (0 and 1)
      float2 fac[4], x[4];
      uint4 hi, lo;
      load4x2(&sm.fac[1][blk][c], fac);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t xat = xs + 8 * r * kXPitch;
        times(kg[r], fac, x);
        split8(x, hi, lo);
        if (!(blk & 1)) {
          put(sm.u.x.x16_hi + xat, hi);
          put(sm.u.x.x16_lo + xat, lo);
        }
        if (blk < 2) {
          put(sm.u.x.x32_hi + xat, blk == 0 ? scale8(hi, pow32) : hi);
          put(sm.u.x.x32_lo + xat, blk == 0 ? scale8(lo, pow32) : lo);
        }
      }
    }
    {  // rows: of the chunk's start, of 16 / 48 (odd blocks), of 32 (2 and 3)
      float2 fac[4], x[4];
      uint4 hi, lo;
      load4x2(&sm.fac[0][blk][c], fac);
      const uint4 pow0 = *reinterpret_cast<const uint4 *>(&sm.pow[blk][c]);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t xat = xs + 8 * r * kXPitch;
        times(kf[r], fac, x);
        split8(x, hi, lo);
        put(im + 1024 * r + kImgKdHi, blk == 0 ? hi : scale8(hi, pow0));
        put(im + 1024 * r + kImgKdLo, blk == 0 ? lo : scale8(lo, pow0));
        if (blk & 1) {
          put(sm.u.x.x16_hi + xat, hi);
          put(sm.u.x.x16_lo + xat, lo);
        }
        if (blk == 2) {
          put(sm.u.x.x32_hi + xat, hi);
          put(sm.u.x.x32_lo + xat, lo);
        }
        times(qf[r], fac, x);
        split8(x, hi, lo);
        if (blk > 0) {
          put(sm.u.x.y_hi + (y0 ^ (64u * sl)) + 8 * r * kXPitch, hi);
          put(sm.u.x.y_lo + (y0 ^ (64u * sl)) + 8 * r * kXPitch, lo);
        }
        put(im + 1024 * r + kImgQdHi, blk == 0 ? hi : scale8(hi, pow0));
        put(im + 1024 * r + kImgQdLo, blk == 0 ? lo : scale8(lo, pow0));
      }
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const int at = part_at(g + 4 * i, 8 * n + 2 * tig) + 2 * (tig & 1);
      *reinterpret_cast<float2 *>(&sm.part[blk][0][hf][at]) = make_float2(dk[n][i], dk[n][i + 1]);
      *reinterpret_cast<float2 *>(&sm.part[blk][1][hf][at]) = make_float2(dq[n][i], dq[n][i + 1]);
    }
  __syncthreads();

  // -- products between blocks: warps 0-3 the quarters of rows 32 .. 63 by
  //    columns 0 .. 31, warps 4 and 5 blocks 1 by 0 and 3 by 2.  Warps 6 and 7
  //    meanwhile invert the diagonal blocks of I + L, two each, a lane a
  //    column -----------------------------------------------------------------
  // (all start from zero in every warp: what one branch leaves unset would
  // hold its registers around the loop)
  float ok[2][4], oq[2][4], x[16];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) ok[n][i] = oq[n][i] = 0.f;
#pragma unroll
  for (int t = 0; t < 16; ++t) x[t] = 0.f;
  int r0 = 0, c0 = 0;
  if (warp < 6) {
    // rows of block 2 by 32's columns, all others by what is kept of 16 and 48
    // (block 3's by 32's columns times 2^n); columns of 32 by 32's
    if (warp < 4) {
      r0 = 32 + 16 * (warp >> 1);
      c0 = 16 * (warp & 1);
    } else {
      r0 = 32 * (warp - 4) + 16;
      c0 = r0 - 16;
    }
    const bool rows32 = warp < 2, cols32 = warp < 4, scaled = warp == 2 || warp == 3;
    const int ar = lane & 15, br = (lane & 7) + ((lane >> 4) << 3);
    const uint32_t ah0 = smem_u32(rows32 ? sm.u.x.x32_hi : sm.u.x.x16_hi);
    const uint32_t al0 = smem_u32(rows32 ? sm.u.x.x32_lo : sm.u.x.x16_lo);
    const uint32_t bh0 = smem_u32(cols32 ? sm.u.x.x32_hi : sm.u.x.x16_hi);
    const uint32_t bl0 = smem_u32(cols32 ? sm.u.x.x32_lo : sm.u.x.x16_lo);
    const uint32_t qh0 = smem_u32(sm.u.x.y_hi), ql0 = smem_u32(sm.u.x.y_lo);
    // (K step ks: pieces 2 ks and 2 ks + 1 of the rows, bits 5 and 6 of the
    // permuted place within a half)
    const uint32_t a0 = x_at(r0 + ar, lane >> 4), b0 = x_at(c0 + br, (lane >> 3) & 1);
    const uint32_t q0 = x_at(r0 - 16 + ar, lane >> 4);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t ah[4], al[4], qh[4], ql[4], bh[4], bl[4];
      const uint32_t flip = 32u * (ks & 3), half = 128u * (ks >> 2);
      ldmatrix4(ah, ah0 + (a0 ^ flip) + half);
      ldmatrix4(al, al0 + (a0 ^ flip) + half);
      ldmatrix4(qh, qh0 + (q0 ^ flip) + half);
      ldmatrix4(ql, ql0 + (q0 ^ flip) + half);
      ldmatrix4(bh, bh0 + (b0 ^ flip) + half);
      ldmatrix4(bl, bl0 + (b0 ^ flip) + half);
      if (scaled) {
        const uint16_t *const at = &sm.pow32[1][16 * ks + 2 * tig];
        const uint32_t p0 = *reinterpret_cast<const uint32_t *>(at);
        const uint32_t p1 = *reinterpret_cast<const uint32_t *>(at + 8);
        scale_rows(ah, p0, p1);
        scale_rows(al, p0, p1);
        scale_rows(qh, p0, p1);
        scale_rows(ql, p0, p1);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        mma_f16(ok[n], al, bh[2 * n], bh[2 * n + 1]);
        mma_f16(ok[n], ah, bl[2 * n], bl[2 * n + 1]);
        mma_f16(ok[n], ah, bh[2 * n], bh[2 * n + 1]);
        mma_f16(oq[n], ql, bh[2 * n], bh[2 * n + 1]);
        mma_f16(oq[n], qh, bl[2 * n], bl[2 * n + 1]);
        mma_f16(oq[n], qh, bh[2 * n], bh[2 * n + 1]);
      }
    }
  } else {
    r0 = 16 * (2 * (warp - 6) + (lane >> 4));  // the block's first token
    const int bi = r0 >> 4, j = lane & 15;
    float *Lb = sm.Lt[bi];
    const float b = sm.beta[r0 + j];
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
      const float4 p0 = lds4(&sm.part[bi][0][0][part_at(j, c)]);
      const float4 p1 = lds4(&sm.part[bi][0][1][part_at(j, c)]);
      const float v[4] = {p0.x + p1.x, p0.y + p1.y, p0.z + p1.z, p0.w + p1.w};
      // (above the diagonal the factors may have overflowed: dropped, not
      // multiplied by zero)
#pragma unroll
      for (int e = 0; e < 4; ++e) Lb[(c + e) * kLtPitch + j] = c + e < j ? b * v[e] : 0.f;
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < 16; ++t) x[t] = t == j ? 1.f : 0.f;
#pragma unroll
    for (int t = 0; t < 15; ++t) {
#pragma unroll
      for (int u = (t + 1) & ~3; u < 16; u += 4) {
        const float4 l = lds4(Lb + t * kLtPitch + u);
        if (u + 0 > t) x[u] = fmaf(-l.x, x[t], x[u]);
        if (u + 1 > t) x[u + 1] = fmaf(-l.y, x[t], x[u + 1]);
        if (u + 2 > t) x[u + 2] = fmaf(-l.z, x[t], x[u + 2]);
        if (u + 3 > t) x[u + 3] = fmaf(-l.w, x[t], x[u + 3]);
      }
    }
  }
  __syncthreads();  // the operands have been read: L and X take their place

  if (more && tid == 0) {
    fence_proxy_async_smem();
    fetch(next, h);
  }
  float *L = sm.u.s.L, *X = sm.u.s.X, *Y = sm.u.s.Y;
  constexpr float kUnit = 1.f / (kImgScale * kImgScale);
  if (warp < 6) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const int t = g + 4 * i, s = 8 * n + 2 * tig;
        const float b = sm.beta[r0 + t] * kUnit;
        float *to = warp < 4 ? &L[(r0 - 32 + t) * kLPitch + c0 + s]
                             : &sm.u.s.L16[warp - 4][t * kL16Pitch + s];
        *reinterpret_cast<float2 *>(to) = make_float2(b * ok[n][i], b * ok[n][i + 1]);
      }
  } else {
#pragma unroll
    for (int t = 0; t < 16; ++t) X[(r0 + t) * kXPitchF + r0 + (lane & 15)] = x[t];
  }
  __syncthreads();

  // -- the rest of X = (I + L)^-1, block by block; what each step leaves ready
  //    for the images is written under the next ------------------------------
  const auto put_f = [&](float *to, int ld, const float (&c)[4], float sign) {
    *reinterpret_cast<float2 *>(to + g * ld + 2 * tig) = make_float2(sign * c[0], sign * c[1]);
    *reinterpret_cast<float2 *>(to + (g + 8) * ld + 2 * tig) =
        make_float2(sign * c[2], sign * c[3]);
  };
  const auto put_a = [&](int t, int s, float x0, float x1) {  // s even
    const uint32_t at = img_at(t, s & ~7) + (s & 7) * 2;
    const float2 x = make_float2(x0, x1);
    const __half2 hi = __float22half2_rn(x);
    *reinterpret_cast<uint32_t *>(sm.a + at) = h2_bits(hi);
    *reinterpret_cast<uint32_t *>(sm.a + kImgBlock + at) =
        h2_bits(__float22half2_rn(ffma2(__half22float2(hi), make_float2(-1.f, -1.f), x)));
  };
  // X10 = -X11 (L10 X00) and X32 = -X33 (L32 X22), 16 x 8 a warp
  const int lo = 32 * ((warp >> 1) & 1), hi = lo + 16, n16 = 8 * (warp & 1);
  float c[4] = {0.f, 0.f, 0.f, 0.f};
  if (warp < 4) {
    tile_mm(c, sm.u.s.L16[lo / 32], kL16Pitch, &X[lo * kXPitchF + lo + n16], kXPitchF, n16 / 8, 2,
            lane);
    put_f(&Y[lo / 2 * kYPitch + n16], kYPitch, c, 1.f);
  }
  __syncthreads();
  if (warp < 4) {
    tile_mm(c, &X[hi * kXPitchF + hi], kXPitchF, &Y[lo / 2 * kYPitch + n16], kYPitch, 0, 2, lane);
    put_f(&X[hi * kXPitchF + lo + n16], kXPitchF, c, -1.f);
  }
  if (warp < 6) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; i += 2)
        put_a(r0 + g + 4 * i, c0 + 8 * n + 2 * tig, oq[n][i] * (1.f / kImgQdScale),
              oq[n][i + 1] * (1.f / kImgQdScale));
  }
  __syncthreads();
  load_head(tid, next, more ? h : 0);
  // the lower left 32 x 32: -X[32.., 32..] (L[32.., ..32] X[..32, ..32])
  const int m32 = 16 * (warp >> 2), n32 = 8 * (warp & 3);
  tile_mm(c, &L[m32 * kLPitch], kLPitch, &X[n32], kXPitchF, n32 / 8, 4, lane);
  put_f(&Y[m32 * kYPitch + n32], kYPitch, c, 1.f);
  {
    // A: its diagonal blocks, and above them zeros
    const int t = tid & 63, tl = t & 15, bt = t >> 4;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int piece = 2 * (tid >> 6) + e, s0 = 8 * (piece & 1);
      if ((piece >> 1) < bt) continue;  // (below: by the products' own warps)
      float2 v[4];
      constexpr float kAUp = kImgScale / kQDown;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 p0 = lds4(&sm.part[bt][1][0][part_at(tl, s0 + 4 * i)]);
        const float4 p1 = lds4(&sm.part[bt][1][1][part_at(tl, s0 + 4 * i)]);
        const int s = 8 * piece + 4 * i;
        v[2 * i] = make_float2(s <= t ? (p0.x + p1.x) * kAUp : 0.f,
                               s + 1 <= t ? (p0.y + p1.y) * kAUp : 0.f);
        v[2 * i + 1] = make_float2(s + 2 <= t ? (p0.z + p1.z) * kAUp : 0.f,
                                   s + 3 <= t ? (p0.w + p1.w) * kAUp : 0.f);
      }
      uint4 hi, lo;
      split8(v, hi, lo);
      *reinterpret_cast<uint4 *>(sm.a + img_at(t, 8 * piece)) = hi;
      *reinterpret_cast<uint4 *>(sm.a + kImgBlock + img_at(t, 8 * piece)) = lo;
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) bulk_store(img + kImgAHi, sm.a, 2 * kImgBlock);
  tile_mm(c, &X[(32 + m32) * kXPitchF + 32], kXPitchF, &Y[n32], kYPitch, 0, m32 / 8 + 2, lane);
  // -- T = X diag(beta): the lower left quarter from registers, the two on the
  //    diagonal from X, zeros above ------------------------------------------
  static_assert(kImgTScale == 16384.f, "2^14");
  const float t_scale =
      __uint_as_float((268u << 23) - __float_as_uint(beta_power(sm.beta, lane)));  // 2^14 / p
  {
    const float b0 = -sm.beta[n32 + 2 * tig] * t_scale;
    const float b1 = -sm.beta[n32 + 2 * tig + 1] * t_scale;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 v = make_float2(c[i] * b0, c[i + 1] * b1);
      const __half2 h = __float22half2_rn(v);
      const uint32_t at = img_at(32 + m32 + g + 4 * i, n32) + 4u * tig;
      *reinterpret_cast<uint32_t *>(sm.t + at) = h2_bits(h);
      *reinterpret_cast<uint32_t *>(sm.t + kImgBlock + at) =
          h2_bits(__float22half2_rn(ffma2(__half22float2(h), make_float2(-1.f, -1.f), v)));
    }
  }
  {
    const int t = tid & 63, s0 = (t & 32) + 8 * (tid >> 6);
    float2 v[4], b[4];
    load4x2(&X[t * kXPitchF + s0], v);
    load4x2(&sm.beta[s0], b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = fmul2(v[i], fmul2(b[i], make_float2(t_scale, t_scale)));
      // (what lies above the diagonal was not all written)
      v[i] = make_float2(s0 + 2 * i <= t ? y.x : 0.f, s0 + 2 * i + 1 <= t ? y.y : 0.f);
    }
    uint4 th, tl;
    split8(v, th, tl);
    const uint32_t at = img_at(t, s0);
    *reinterpret_cast<uint4 *>(sm.t + at) = th;
    *reinterpret_cast<uint4 *>(sm.t + kImgBlock + at) = tl;
    const uint32_t above = img_at(tid & 31, 32 + 8 * ((tid >> 5) & 3));
    *reinterpret_cast<uint4 *>(sm.t + (tid < 128 ? 0 : kImgBlock) + above) =
        make_uint4(0, 0, 0, 0);
  }
  ck = next;
  fence_proxy_async_smem();
  __syncthreads();  // the next item's decay sums take the place of X
  if (tid == 0) bulk_store(img + kImgTHi, sm.t, 2 * kImgBlock);
  }
  if (threadIdx.x == 0) bulk_stores_done();
  // beside a chain, this grid completes after it
  if (blockIdx.x == 0 && threadIdx.x == 0) grid_dependency_wait();
}

}  // namespace

int launch_prefill_prep(const PrefillParams &p, int segment, cudaStream_t stream) {
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
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return KDA_ERR_CUDA;
  const cuuint64_t dims[3] = {(cuuint64_t)kDim, (cuuint64_t)p.r.H,
                              (cuuint64_t)p.r.maps.n_tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)kDim * 2, (cuuint64_t)p.r.H * kDim * 2};
  const cuuint32_t box[3] = {(cuuint32_t)kDim, 1, (cuuint32_t)kChunk};
  const cuuint32_t estride[3] = {1, 1, 1};
  PrepMaps maps;
  CUtensorMap *const map[3] = {&maps.g, &maps.q, &maps.k};
  const uint16_t *const src[3] = {p.r.g, p.r.q, p.r.k};
  for (int i = 0; i < 3; ++i)
    if (encode(map[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(src[i]), dims,
               strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
      return KDA_ERR_CUDA;
  long long items = (long long)p.max_chunks * p.r.H;
  const long long most = (long long)p.r.maps.B * p.r.H *
                         (seg_from(p, segment + 1) - seg_from(p, segment));
  if (p.segments > 1 && most < items) items = most;
  // (beside a chain: what its CTAs, one to an SM, leave)
  const int sms = device_sm_count(dev), chain = p.r.maps.B * p.r.H;
  const long long room = 2LL * (segment > 0 && chain < sms ? sms - chain : sms);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < room ? items : room));
  cfg.blockDim = dim3(kPrepThreads);
  cfg.dynamicSmemBytes = sizeof(PrepSmem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kda_prefill_prep_kernel, p, maps, segment) != cudaSuccess)
    return KDA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda

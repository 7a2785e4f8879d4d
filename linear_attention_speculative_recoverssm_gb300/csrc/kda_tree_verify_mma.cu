// The delta rule over trees on the tensor cores: two CTAs an SM, each taking
// (request, head) items one after the other.
//
// Per item, S the state page after its replay and X_k, X_q the nodes' vectors:
//   [w; y] = S [X_k; X_q]^T             (tcgen05: M = 128 rows of the page,
//                                        N = two columns a node, K = 128)
//   R_s = v_s - w_s
//   u_t = sum_s T[t][s] R_s, o_t = y_t + sum_s C[t][s] R_s
// s over t and its ancestors, where T inverts u_t = beta_t (R_t - sum A u) and
// C is B T: at most eight terms a node, none of which waits for another.
//
// Operands are BF16 in three parts (24 bits): x = hi + mid + lo, six products
// of parts whose sizes are above 2^-24 of the first's (a BF16 page is its own
// only part: three products).  FP32's exponents, so that no scale is needed.
// TF32 in two parts costs the same tensor time for 22 bits, and twice the
// columns of tensor memory.
//
// The page goes from HBM to registers in the layout of tcgen05.st's 16x256b
// (16 bytes a lane, four lanes to 64 bytes of a row), is replayed there,
// written back from there, split there, and stored to tensor memory as the
// A operand: it never passes through shared memory, which holds the nodes.
// While an item is worked on, the next one's page and operands are fetched to
// L2; the two CTAs of an SM cover each other's waits.
//
// Per group of up to G nodes the warps (1) walk up the nodes' paths, writing
// X in parts and the coefficients A, B; (2) one thread issues the products,
// and meanwhile warp 0 makes T and C; (3) R and y go from tensor memory to
// shared memory, a thread a row; (4) u and o, a warp a node.  A node's
// ancestors are in its group or in an earlier one.
#include <cuda_runtime.h>

#include "kda_launch.h"
#include "kda_tcgen05.cuh"
#include "kda_tree_verify.cuh"

namespace kda {
namespace {

constexpr int kTmThreads = 256;
constexpr int kTmWarps = kTmThreads / 32;
constexpr uint32_t kTmCols = 256;     // of tensor memory, a CTA
constexpr uint32_t kTmPartCols = kDim / 2;  // of one part of the page: two keys a column
constexpr uint32_t kTmD = 3 * kTmPartCols;  // the products
constexpr int kPath = kTreeDepth;           // T and C: t itself and its ancestors

// Instruction descriptor of kind::f16: FP32 accumulator, A and B BF16, both
// K-major, N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__device__ __forceinline__ uint32_t tm_idesc(uint32_t n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((uint32_t)(kDim >> 4) << 24);
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t tm_elect() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p;
}

// D[tmem] (+)= A[tmem, 128 x 16] . B[N x 16]^T, issued by the lane with
// `lead` while its warp runs along (the operands then live in uniform
// registers).
__device__ __forceinline__ void tm_mma(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                       bool accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
      : "memory");
}

// 16 lanes (from taddr's), 32 columns: a thread's registers 4 j .. 4 j + 3 are
// columns 8 j + 2 (lane % 4) + 0, 1 of row lane / 4, then of row lane / 4 + 8.
__device__ __forceinline__ void tm_store_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// 4 columns of this warp's 32 lanes, a lane a thread (no wait).
__device__ __forceinline__ void tm_load4(uint32_t taddr, float (&r)[4]) {
  uint32_t x[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __uint_as_float(x[i]);
}

__device__ __forceinline__ void prefetch_l2(const void *at) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

// A pair's next part: BF16 of both (returned packed), the rest left in them.
__device__ __forceinline__ uint32_t take_part(float2 &x) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(x.y), "f"(x.x));
  x.x -= __uint_as_float(w << 16);
  x.y -= __uint_as_float(w & 0xffff0000u);
  return w;
}

// NC: nodes of the largest window; G: nodes of a group.
template <int NC, int G>
struct TreeMma {
  static constexpr uint32_t kBlock = 2 * G * 128;  // 64 keys of a part of X: rows of 128 bytes
  static constexpr uint32_t kPart = 2 * kBlock;
  // byte offsets of dynamic shared memory, from a 1024-byte boundary
  static constexpr uint32_t kX = 0;
  static constexpr uint32_t kD = kX + 3 * kPart;         // decays [NC][128] FP32
  static constexpr uint32_t kK = kD + NC * kDim * 4;     // keys [NC][128] BF16
  static constexpr uint32_t kR = kK + NC * kDim * 2;     // R of all groups but the last
  static constexpr uint32_t kCoef = kR + (NC - G) * kDim * 4;
  static constexpr uint32_t kTC = kCoef + NC * kTreeCoefs * 4;  // T[8], C[8] of a node
  static constexpr uint32_t kNorm = kTC + NC * 2 * kPath * 4;
  static constexpr uint32_t kAnc = kNorm + NC * 4;  // depth, then the ancestors, a byte each
  static constexpr uint32_t kParent = kAnc + kTreeNodes * 8;
  static constexpr uint32_t kBar = kParent + kTreeNodes;
  static constexpr uint32_t kEnd = kBar + 32;
  // (two CTAs an SM, and no third, whose tensor memory would not be there)
  static constexpr uint32_t kBytes = kEnd + 1024 > 78 * 1024 ? kEnd + 1024 : 78 * 1024;
  static_assert(kBytes <= 113 * 1024, "two CTAs an SM");
  // the replay's operands stand where X comes later; y and the last group's R
  // where X was
  static constexpr uint32_t kReplayK = kX, kReplayD = kReplayK + kMaxQ * kDim * 4,
                            kReplayU = kReplayD + kMaxQ * kDim * 4,
                            kReplayDn = kReplayU + kMaxQ * kDim * 4;
  static_assert(kReplayDn + kDim * 4 <= kD, "the replay's operands in X");
  static_assert(2 * G * kDim * 4 <= 3 * kPart, "y and R in X");
};

// A page's part of a thread: rows 16 rh + lane / 4 + 8 i of the warp's 32,
// keys 16 j + 4 (lane % 4) + 0 .. 3 of the warp's 64.
struct PageRegs {
  float4 s[2][4][2];  // [rh][j][i]
};

template <int NC, int G, bool BF16>
__global__ void __launch_bounds__(kTmThreads, 2) kda_tree_mma_kernel(const TreeVerifyParams p,
                                                                    int n_items) {
  using L = TreeMma<NC, G>;
  extern __shared__ uint8_t raw[];
  uint8_t *mem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  float *decay = reinterpret_cast<float *>(mem + L::kD);
  uint16_t *keys = reinterpret_cast<uint16_t *>(mem + L::kK);
  float *coefs = reinterpret_cast<float *>(mem + L::kCoef);
  float *tc = reinterpret_cast<float *>(mem + L::kTC);
  float *norms = reinterpret_cast<float *>(mem + L::kNorm);
  uint8_t *anc = mem + L::kAnc;
  int8_t *parent = reinterpret_cast<int8_t *>(mem + L::kParent);
  uint64_t *bar = reinterpret_cast<uint64_t *>(mem + L::kBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mem + L::kBar + 8);
  int *good = reinterpret_cast<int *>(mem + L::kBar + 16);
  const TreeMaps &mp = p.maps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quarter = warp & 3, half = warp >> 2;
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(tmem_slot, kTmCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t my_lanes = tmem + ((uint32_t)(32 * quarter) << 16);
  const int begin = (int)((long long)n_items * blockIdx.x / gridDim.x);
  const int end = (int)((long long)n_items * (blockIdx.x + 1) / gridDim.x);
  uint32_t rounds = 0;  // of products, for the barrier's parity
  bool failed = false;
  int request = -1;
  TreeRequest r;
  r.error = KDA_ERR_ARG;
  r.t0 = r.n = r.pending = 0;
  r.slot = r.row = -1;
  bool tree_ok = false;
  for (int item = begin; item < end && !failed; ++item) {
    const int b = item / p.H, h = item - b * p.H;
    if (b != request) {
      request = b;
      r = tree_request(mp, b);
      if (warp == 0) {
        const bool ok = r.error == KDA_OK && (r.slot < 0 || load_tree(mp, r, parent, lane));
        if (lane == 0) {
          *good = ok;
          if (!ok) report(mp.status, KDA_ERR_ARG);
        }
        if (ok && r.slot >= 0) {
#pragma unroll
          for (int i = 0; i < NC / 32 + (NC < 32); ++i) {
            const int t = lane + 32 * i;
            if (t >= NC) break;
            uint8_t path[8];
            int m = 0, a = parent[t];
#pragma unroll
            for (int j = 1; j < 8; ++j) {
              path[j] = (uint8_t)a;
              m += a >= 0;
              a = a >= 0 ? parent[a] : -1;
            }
            path[0] = (uint8_t)m;
            uint2 w;
            w.x = path[0] | path[1] << 8 | path[2] << 16 | (uint32_t)path[3] << 24;
            w.y = path[4] | path[5] << 8 | path[6] << 16 | (uint32_t)path[7] << 24;
            *reinterpret_cast<uint2 *>(anc + 8 * t) = w;
          }
        }
      }
      __syncthreads();
      tree_ok = *good != 0;
      __syncthreads();  // (read before the next request's)
    }
    if (!tree_ok) continue;
    const long long first = (long long)r.t0 * p.H + h;  // the (token, head) row of node 0
    if (r.slot < 0) {
      for (int i = tid; i < r.n * (kDim / 8); i += kTmThreads)
        *reinterpret_cast<uint4 *>(p.out + (first + (long long)(i / (kDim / 8)) * p.H) * kDim +
                                   i % (kDim / 8) * 8) = make_uint4(0, 0, 0, 0);
      continue;
    }
    const int n = r.n, replay = r.pending;
    if (n == 0 && replay == 0) continue;
    const long long page = r.slot * p.slot_stride + (long long)h * kDim * kDim;
    const float a = expf(p.A_log[h]);
    const float4 dt = __ldg(reinterpret_cast<const float4 *>(p.dt_bias + h * kDim) + lane);
    float *const rk = reinterpret_cast<float *>(mem + L::kReplayK);
    float *const rd = reinterpret_cast<float *>(mem + L::kReplayD);
    float *const ru = reinterpret_cast<float *>(mem + L::kReplayU);
    float *const rdn = reinterpret_cast<float *>(mem + L::kReplayDn);
    // ---- the page is asked for
    PageRegs pg;
    uint2 pgb[BF16 ? 16 : 1];
    const long long at = page + (long long)(32 * quarter + lane / 4) * kDim + 64 * half +
                         4 * (lane & 3);
    if constexpr (BF16) {
#pragma unroll
      for (int rh = 0; rh < 2; ++rh)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            pgb[(rh * 4 + j) * 2 + i] = __ldcs(reinterpret_cast<const uint2 *>(
                static_cast<const uint16_t *>(p.state) + at + (16 * rh + 8 * i) * kDim + 16 * j));
    } else {
#pragma unroll
      for (int rh = 0; rh < 2; ++rh)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            pg.s[rh][j][i] = __ldcs(reinterpret_cast<const float4 *>(
                static_cast<const float *>(p.state) + at + (16 * rh + 8 * i) * kDim + 16 * j));
    }
    // ---- the recorded tokens and the nodes: norms and decays
    for (int t = warp; t < replay; t += kTmWarps) {
      const uint16_t *rec = p.kg + r.row * p.kg_stride + ((long long)h * mp.rq + t) * 2 * kDim;
      const float4 k = bf16x4(__ldg(reinterpret_cast<const uint2 *>(rec) + lane));
      const float4 g = bf16x4(__ldg(reinterpret_cast<const uint2 *>(rec + kDim) + lane));
      const float4 u = __ldg(reinterpret_cast<const float4 *>(
                                 p.corr + r.row * p.corr_stride + ((long long)h * mp.rq + t) * kDim) +
                             lane);
      sts4(rk + t * kDim + 4 * lane, scale4(k, rsqrtf(warp_sum(dot4(k, k)) + kNormEps)));
      sts4(rd + t * kDim + 4 * lane, decay4(a, g, dt, p.lower_bound));
      sts4(ru + t * kDim + 4 * lane, u);
    }
#pragma unroll 2
    for (int t = warp; t < n; t += kTmWarps) {
      const long long row = first + (long long)t * p.H;
      const uint2 kb = __ldg(reinterpret_cast<const uint2 *>(p.k + row * kDim) + lane);
      const uint2 gb = __ldg(reinterpret_cast<const uint2 *>(p.g + row * kDim) + lane);
      const uint16_t beta = __ldg(p.beta + row);
      const float4 k = bf16x4(kb);
      const float norm = rsqrtf(warp_sum(dot4(k, k)) + kNormEps);
      *reinterpret_cast<uint2 *>(keys + t * kDim + 4 * lane) = kb;
      sts4(decay + t * kDim + 4 * lane, decay4(a, bf16x4(gb), dt, p.lower_bound));
      if (lane == 0) {
        norms[t] = norm;
        coefs[t * kTreeCoefs + kCoefBeta] = sigmoidf_fast(bf16_bits_to_f32(beta));
      }
    }
    // ---- the next head's page and operands on their way to L2
    if (item + 1 < end && h + 1 < p.H) {
      const char *next = static_cast<const char *>(p.state) + (page + kDim * kDim) * (BF16 ? 2 : 4);
#pragma unroll
      for (int i = 0; i < (BF16 ? 1 : 2); ++i) prefetch_l2(next + (i * kTmThreads + tid) * 128);
      for (int i = tid; i < 8 * n; i += kTmThreads) {
        const long long byte = ((first + 1 + (long long)(i >> 3) * p.H) * kDim) * 2 + (i & 1) * 128;
        const uint16_t *from = (i & 7) < 4 ? ((i & 7) < 2 ? p.k : p.g) : ((i & 7) < 6 ? p.q : p.v);
        prefetch_l2(reinterpret_cast<const char *>(from) + byte);
      }
    }
    if (replay > 0) {
      __syncthreads();
      if (tid < kDim) replay_suffix(rk, rd, rdn, replay, tid);
      __syncthreads();
    }
    // ---- S_n, and its parts to tensor memory
    if constexpr (BF16) {
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            w[4 * j + 2 * i] = pgb[(rh * 4 + j) * 2 + i].x;
            w[4 * j + 2 * i + 1] = pgb[(rh * 4 + j) * 2 + i].y;
          }
        tm_store_16x32(my_lanes + ((uint32_t)(16 * rh) << 16) + 32 * half, w);
      }
    } else {
      if (replay > 0) {
        const float *dn = rdn + 64 * half + 4 * (lane & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 x = lds4(dn + 16 * j);
#pragma unroll
          for (int rh = 0; rh < 2; ++rh)
#pragma unroll
            for (int i = 0; i < 2; ++i) pg.s[rh][j][i] = fmul4(pg.s[rh][j][i], x);
        }
#pragma unroll 1
        for (int t = 0; t < replay; ++t) {
          const float *kp = rk + t * kDim + 64 * half + 4 * (lane & 3);
          const float *up = ru + t * kDim + 32 * quarter + lane / 4;
          float u[2][2];
#pragma unroll
          for (int rh = 0; rh < 2; ++rh)
#pragma unroll
            for (int i = 0; i < 2; ++i) u[rh][i] = up[16 * rh + 8 * i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 x = lds4(kp + 16 * j);
#pragma unroll
            for (int rh = 0; rh < 2; ++rh)
#pragma unroll
              for (int i = 0; i < 2; ++i) pg.s[rh][j][i] = ffma4s(u[rh][i], x, pg.s[rh][j][i]);
          }
        }
        float *to = static_cast<float *>(p.state) + at;
#pragma unroll
        for (int rh = 0; rh < 2; ++rh)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              stg4(to + (16 * rh + 8 * i) * kDim + 16 * j, pg.s[rh][j][i]);
      }
      if (n > 0) {
#pragma unroll
        for (int rh = 0; rh < 2; ++rh)
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float4 &s = pg.s[rh][j][i];
                float2 lo = make_float2(s.x, s.y), hi = make_float2(s.z, s.w);
                w[4 * j + 2 * i] = take_part(lo);
                w[4 * j + 2 * i + 1] = take_part(hi);
                s = make_float4(lo.x, lo.y, hi.x, hi.y);
              }
            tm_store_16x32(my_lanes + ((uint32_t)(16 * rh) << 16) + kTmPartCols * part + 32 * half, w);
          }
      }
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    tc_fence_before();
    __syncthreads();  // the nodes' operands are there, and the replay's are read
    const int groups = (n + G - 1) / G;
    for (int g = 0; g < groups; ++g) {
      const int n0 = g * G, ng = n - n0 < G ? n - n0 : G;
      const int cols = (ng + 7) & ~7;  // of w, and of y behind them
      // ---- (1) paths
#pragma unroll 1
      for (int i = warp; i < ng; i += kTmWarps) {
        const int t = n0 + i;
        const uint2 qb = __ldg(reinterpret_cast<const uint2 *>(p.q + (first + (long long)t * p.H) * kDim) + lane);
        const float4 q = bf16x4(qb);
        float4 xk = scale4(bf16x4(*reinterpret_cast<const uint2 *>(keys + t * kDim + 4 * lane)), norms[t]);
        float4 xq = scale4(q, rsqrtf(warp_sum(dot4(q, q)) + kNormEps) * p.q_scale);
        float v[kTreeCoefs];
#pragma unroll
        for (int c = 0; c < kTreeCoefs; ++c) v[c] = 0.f;
        v[kCoefSelf] = dot4(xk, xq);
        int s = t;
#pragma unroll
        for (int j = 0; j < kTreeDepth; ++j) {
          const float4 ds = lds4(decay + s * kDim + 4 * lane);
          xk = fmul4(xk, ds);
          xq = fmul4(xq, ds);
          s = parent[s];
          if (s < 0) break;  // (the same in every lane)
          if (j < kTreeDepth - 1) {
            const float4 ks = scale4(bf16x4(*reinterpret_cast<const uint2 *>(keys + s * kDim + 4 * lane)), norms[s]);
            v[j] = dot4(xk, ks);
            v[kCoefB + j] = dot4(xq, ks);
          }
        }
        // lane l of each half warp ends with value l
        reduce_scatter<kTreeCoefs, 16>(v, lane);
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
        if (lane < kCoefBeta) coefs[t * kTreeCoefs + lane] = v[0];
        // X's rows i and cols + i: keys 4 lane .. + 3 of 64-key block lane / 16
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int row = w * cols + i;
          uint8_t *to = mem + L::kX + (lane >> 4) * L::kBlock + row * 128 +
                        ((((lane & 15) >> 1) ^ (row & 7)) << 4) + (lane & 1) * 8;
          const float4 x = w ? xq : xk;
          float2 lo = make_float2(x.x, x.y), hi = make_float2(x.z, x.w);
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint32_t c = take_part(lo);
            *reinterpret_cast<uint2 *>(to + part * L::kPart) = make_uint2(c, take_part(hi));
          }
        }
      }
      fence_proxy_async_smem();
      __syncthreads();
      // ---- (2) products; T and C
      if (warp == kTmWarps - 1) {
        tc_fence_after();
        const uint32_t lead = tm_elect();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t idesc = __shfl_sync(0xffffffffu, tm_idesc(2 * cols), 0);
        const uint32_t x0 = __shfl_sync(0xffffffffu, smem_u32(mem + L::kX), 0);
        {
          // the smallest products first
          constexpr int kTerms = BF16 ? 3 : 6;
          constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
          constexpr int kB1[3] = {2, 1, 0};
#pragma unroll
          for (int e = 0; e < kTerms; ++e) {
            const uint32_t pa = BF16 ? 0 : kA[e], pb = BF16 ? kB1[e % 3] : kB[e];
#pragma unroll
            for (int ks = 0; ks < kDim / 16; ++ks)
              tm_mma(tm + kTmD, tm + pa * kTmPartCols + 8 * ks,
                     umma_desc_sw128(x0 + pb * L::kPart + (ks >> 2) * L::kBlock + (ks & 3) * 32),
                     idesc, e > 0 || ks > 0, lead);
          }
          if (lead) umma_commit(bar);
        }
        __syncwarp();
      } else if (warp == 0) {
        // a lane a node, level by level
        for (int level = 0; level < kTreeDepth; ++level) {
          const int t = n0 + lane;
          const bool mine = lane < ng && anc[8 * t] == level;
          if (mine) {
            const float *c = coefs + t * kTreeCoefs;
            const float beta = c[kCoefBeta], self = c[kCoefSelf];
            float ta[kPath], ca[kPath];
#pragma unroll
            for (int j = 0; j < kPath; ++j) ta[j] = ca[j] = 0.f;
#pragma unroll
            for (int i = 1; i < kPath; ++i) {
              if (i > level) break;
              const float *up = tc + anc[8 * t + i] * 2 * kPath;
              const float A = c[i - 1], B = c[kCoefB + i - 1];
              const float4 x = lds4(up), y = lds4(up + 4);
              const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k + i < kPath; ++k) {
                ta[i + k] = fmaf(A, f[k], ta[i + k]);
                ca[i + k] = fmaf(B, f[k], ca[i + k]);
              }
            }
            float *to = tc + t * 2 * kPath;
            ta[0] = -1.f;
#pragma unroll
            for (int j = 0; j < kPath; ++j) {
              ta[j] *= -beta;
              ca[j] = fmaf(self, ta[j], ca[j]);
            }
            sts4(to, make_float4(ta[0], ta[1], ta[2], ta[3]));
            sts4(to + 4, make_float4(ta[4], ta[5], ta[6], ta[7]));
            sts4(to + 8, make_float4(ca[0], ca[1], ca[2], ca[3]));
            sts4(to + 12, make_float4(ca[4], ca[5], ca[6], ca[7]));
          }
          __syncwarp();
        }
      }
      // ---- (3) R and y: four nodes at a time, the halves in turn
      const uint16_t *vp = p.v + (first + (long long)n0 * p.H) * kDim + 32 * quarter + lane;
      constexpr int kChunks = G / 8;  // of a half, at most
      uint16_t vb[kChunks][4];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 8 * c + 4 * half + e;
          vb[c][e] = i < ng ? __ldg(vp + (long long)i * p.H * kDim) : 0;
        }
      const bool ok = mbar_wait_bounded(bar, rounds & 1u);
      ++rounds;
      if (__syncthreads_or(!ok)) {
        if (tid == 0) report(mp.status, KDA_ERR_TIMEOUT);
        failed = true;
        break;
      }
      tc_fence_after();
      const bool last = g + 1 == groups;
      float *const ys = reinterpret_cast<float *>(mem + L::kX);
      float *const rs = reinterpret_cast<float *>(mem + L::kR);
      // R of node t: rs + t * kDim, or in X for the last group's
      float *const rx = ys + (G - n0) * kDim;
      float *const to = (last ? rx : rs) + n0 * kDim + 32 * quarter + lane;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int i0 = 8 * c + 4 * half;
        if (i0 < cols) {
          float w[4], y[4];
          tm_load4(my_lanes + kTmD + i0, w);
          tm_load4(my_lanes + kTmD + cols + i0, y);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            to[(i0 + e) * kDim] = bf16_bits_to_f32(vb[c][e]) - w[e];
            ys[(i0 + e) * kDim + 32 * quarter + lane] = y[e];
          }
        }
      }
      tc_fence_before();
      __syncthreads();
      // ---- (4) u and o
#pragma unroll 1
      for (int i = warp; i < ng; i += kTmWarps) {
        const int t = n0 + i;
        const uint2 path = *reinterpret_cast<const uint2 *>(anc + 8 * t);
        const float *c = tc + t * 2 * kPath;
        const int m = path.x & 0xff;
        float4 x = lds4((last ? rx : rs) + t * kDim + 4 * lane);
        float4 u = scale4(x, c[0]);
        float4 o = ffma4s(c[kPath], x, lds4(ys + i * kDim + 4 * lane));
#pragma unroll
        for (int j = 1; j < kPath; ++j) {
          if (j > m) break;
          const int s = ((j < 4 ? path.x : path.y) >> (8 * (j & 3))) & 0xff;
          x = lds4((s >= n0 && last ? rx : rs) + s * kDim + 4 * lane);
          u = ffma4s(c[j], x, u);
          o = ffma4s(c[kPath + j], x, o);
        }
        const long long row = (first + (long long)t * p.H) * kDim + 4 * lane;
        stg4(p.node_corr + row, u);
        *reinterpret_cast<uint2 *>(p.out + row) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
      }
      __syncthreads();  // X, R and the coefficients may be written again
      tc_fence_after();
    }
  }
  if (failed && warp == kTmWarps - 1) mbar_wait_bounded(bar, (rounds - 1) & 1u);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

template <int NC, int G, bool BF16>
int launch(const TreeVerifyParams &p, int sms, cudaStream_t stream) {
  const auto kernel = kda_tree_mma_kernel<NC, G, BF16>;
  constexpr int bytes = (int)TreeMma<NC, G>::kBytes;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return KDA_ERR_CUDA;
  const int items = p.maps.B * p.H;
  kernel<<<items < 2 * sms ? items : 2 * sms, kTmThreads, bytes, stream>>>(p, items);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

int launch_tree_mma(const TreeVerifyParams &p, bool bf16, int sms, cudaStream_t stream) {
  if (p.maps.Q <= 32)
    return bf16 ? launch<32, 32, true>(p, sms, stream) : launch<32, 32, false>(p, sms, stream);
  return bf16 ? launch<64, 16, true>(p, sms, stream) : launch<64, 16, false>(p, sms, stream);
}

}  // namespace kda

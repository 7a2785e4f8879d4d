// The delta rule over trees on the tensor cores: persistent CTAs, each taking
// (request, head) items one after the other.
//
// Per item, S the state page after its replay, G_t the product of the decays
// down the path to node t:
//   X = [G_t kn_t; G_t qn_t], Y = [kn_s / G_s]    (two rows a node, and one)
//   P = X Y^T                  the products of t's key and query with its
//                              ancestors' keys, decayed from one to the other
//   [w y] = S X^T              (M = 128 rows of the page)
//   R_s = v_s - w_s
//   [u o] = R [T; C]^T + [0 y]
// where T inverts u_t = beta_t (R_t - sum_s P_ts u_s) and C = P_q T: at most
// eight entries a row, at the node and its ancestors.  A path holds at most
// eight decays, each within e^-10 .. e^10, so that 1 / G stays inside FP32.
// Of P only the entries of ancestors are looked at.
//
// Operands are BF16 in three parts (24 bits): x = hi + mid + lo, six products
// of parts whose sizes are above 2^-24 of the first's (a BF16 page is its own
// only part: three products).  FP32's exponents, so that no scale is needed.
// TF32 in two parts costs the same tensor time for 22 bits, and more of tensor
// memory.  (Where a channel's G is within 2^16 of FP32's ends, its last part
// underflows: 16 bits of it are left.)
//
// The page goes from HBM to registers in the layout of tcgen05.st's 16x256b
// (16 bytes a lane, four lanes to 64 bytes of a row), is replayed there,
// written back from there, split there, and stored to tensor memory as the
// A operand.  R goes the same way.  Where shared memory has room beside the
// nodes, a page waits there first (kStaged).
//
// R and [T; C] are multiplied whole, and zero times NaN is NaN: an R that is
// not finite is left out as zero, and the outputs of its node and of those
// below it are made NaN at the end (nothing is looked at where all are finite).
//
// One CTA an SM, whose warps divide the work by its kind and run one behind
// the other, some items apart, as barriers in shared memory let them: the
// requests (validated, their paths listed, copies of their nodes sent for) a
// warp; nodes to X and Y; pages; T and C; R and the outputs; and two warps that
// issue the products, of X and of R.  Each kind is a chain of latencies (shared
// memory, the shuffles of a norm, a product's hand-off); one phase after the
// other by all warps, two CTAs an SM, was slower when it was tried: 804 against
// 646 us (128 windows of 64 nodes and 64 heads), 111 against 97 (48 of up to 32
// nodes, 32 heads), 115 against 113 (100 of 24, BF16 pages).  Later steps took the
// three to 605, 87 and 101.
//
// Those three move 2053, 274 and 243 MB at 3.4, 3.2 and 2.4 TB/s (a copy's rate:
// 6.7).  What bounds them is not HBM but instructions, their fetch, and the
// chains' latencies: 46 thousand warp instructions an item of 64 nodes, 18 of
// 24, half of the issue slots, half of the shared memory's wavefronts, a quarter
// of the tensor pipe's cycles.  The roles' code, all of it in use at once, is
// more than an SM's instruction cache holds: loops are rolled up wherever their
// state allows it (BF16 pages, 24 nodes: the cache's hits from 64 to 84% of the
// requests; with the nodes' tensor copies and R ahead of the outputs 113 -> 101 us).
// At 64 registers a thread 8 to 40 bytes of it are kept in local memory.
//
// Small trees cost what their pages do: 1536 items with a replay take 73 to 76 us
// for 4, 5, 6 and 7 nodes alike (floor 33).  A page has one place in shared memory
// and one in tensor memory, and the next one waits for both.
#include <cuda_runtime.h>

#include <type_traits>

#include "kda_launch.h"
#include "kda_tcgen05.cuh"
#include "kda_tensor_map.h"
#include "kda_tree_verify.cuh"

namespace kda {
namespace {

constexpr uint32_t kTmPartCols = kDim / 2;  // of one part of the page: two keys a column
constexpr uint32_t kTmD = 3 * kTmPartCols;  // w, then u; y, then o
constexpr int kPath = kTreeDepth;           // a node and its ancestors

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

// D[tmem] (+)= A[128 x 16] . B[N x 16]^T, A in tensor memory or in shared
// memory, issued by the lane with `lead` while its warp runs along (the
// operands then live in uniform registers).
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
__device__ __forceinline__ void tm_mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, bool accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
      : "memory");
}

// 16 lanes (from taddr's), 16 columns: a thread's registers 4 j .. 4 j + 3 are
// columns 8 j + 2 (lane % 4) + 0, 1 of row lane / 4, then of row lane / 4 + 8.
__device__ __forceinline__ void tm_store_16x16(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// 4 columns of this warp's 32 lanes, a lane a thread.
__device__ __forceinline__ void tm_store_32x4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c,
                                              uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ void tm_store_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 16 or 8 columns of this warp's 32 lanes, a lane a thread (no wait).
__device__ __forceinline__ void tm_load(uint32_t taddr, float (&r)[16]) {
  uint32_t x[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
        "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]),
        "=r"(x[14]), "=r"(x[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(x[i]);
}
__device__ __forceinline__ void tm_load(uint32_t taddr, float (&r)[8]) {
  uint32_t x[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
        "=r"(x[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(x[i]);
}
__device__ __forceinline__ void tm_load_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *at) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

// A box of a tensor on its way to L2 (coordinates as in tma_load_3d).
__device__ __forceinline__ void prefetch_box(const void *tmap, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// A pair's next part: BF16 of both (returned packed), the rest left in them.
__device__ __forceinline__ uint32_t take_part(float2 &x) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(x.y), "f"(x.x));
  x = __fadd2_rn(x, make_float2(-__uint_as_float(w << 16), -__uint_as_float(w & 0xffff0000u)));
  return w;
}

// mbar_wait_bounded in few instructions: the roles' code, all of it in use at
// once, is more than an SM's instruction cache holds.
__device__ __forceinline__ bool tm_wait(uint64_t *bar, uint32_t parity) {
  static_assert(kWaitLimitNs < 0x7fffffff, "32 bits of the timer");
  uint32_t start = 0, now;
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, 1000000u))) return true;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
    if (start == 0) start = now | 1u;  // (odd: it may lie a nanosecond ahead)
    if ((int)(now - start) > (int)kWaitLimitNs) return false;
  }
}

// A request as its warp hands it to the others: heads h0 .. h1 - 1 of it are this
// CTA's.  n < 0: there is none any more.
struct TreeTask {
  int t0, n, slot, row, pending, h0, h1;
  // per node the number of its ancestors, then they, the nearest first, a byte
  // each; the node itself where there are no more
  uint2 path[kTreeNodes];
};

// Between the groups of warps: `full` when what it names is there, `free` when
// its place may be written again.
struct TreeBars {
  uint64_t task_full[4], task_free[4];
  uint64_t raw_full[2], raw_free[2];  // keys, queries and gates as they are
  uint64_t x_full, x_free, y_free;  // X and Y
  uint64_t n_full;                  // norms and decays, where T's warps take nodes too
  uint64_t p_full, p_free;          // P in tensor memory
  uint64_t a_full, a_free;          // the page's parts
  uint64_t d_full[2], d_free[2];    // w and y, until o is out
  uint64_t t_full, t_free;          // [T; C]
  uint64_t r_full[2], o_full[2];    // R's parts; u and o
  uint64_t done[2];                 // every product that a warp issued
};

// NC: nodes of the largest window.
template <int NC, bool BF16>
struct TreeMma {
  // warps: pages (two to a quarter of the rows; BF16 pages, which are only read,
  // one), R (two), T and C (a lane a row of P), the two that issue, the one with
  // the requests, nodes
  static constexpr int kWarps = 32, kPageWarps = BF16 ? 4 : 8, kRWarps = 8, kTWarps = 2 * NC / 32;
  static constexpr int kR0 = kPageWarps, kT0 = kR0 + kRWarps, kIssue0 = kT0 + kTWarps,
                       kTask0 = kIssue0 + 2, kNode0 = kTask0 + 1, kNodeWarps = kWarps - kNode0;
  // warps that make X and Y: of large trees T's and C's too, which wait meanwhile
  // (64 nodes: 648 -> 605 us)
  static constexpr bool kTHelps = NC > 32;
  static constexpr int kXWarps = kNodeWarps + (kTHelps ? kTWarps : 0);
  // registers a thread: at launch, of pages (whole warpgroups), of the others
  static constexpr int kPageRegs = kPageWarps == 4 ? 120 : 88, kOtherRegs = 56;
  static_assert(kPageWarps * kPageRegs + (kWarps - kPageWarps) * kOtherRegs <= kWarps * 64,
                "what the warps of pages take, the others have given");
  static_assert(kR0 % 4 == 0 && kT0 % 4 == 0, "a warp reaches the tensor memory lanes of its number");
  static constexpr int kThreads = 32 * kWarps;
  // tensor memory: the page, w and y (twice where there is room), P, R (as often)
  static constexpr int kDBufs = NC <= 32 ? 2 : 1;
  // P: by the size of the parts' products, where there is room
  static constexpr int kPParts = NC <= 32 ? 3 : 1;
  static constexpr uint32_t kTmP = kTmD + kDBufs * 2 * NC, kTmR = kTmP + kPParts * NC;
  static_assert(kTmR + kDBufs * 3 * NC / 2 <= 512, "tensor memory");
  // tiles of 128-byte rows (64 keys of a part), 128-byte swizzled
  static constexpr uint32_t kXBlock = 2 * NC * 128, kXPart = 2 * kXBlock;
  // (of Y a block is of all three parts, where one product takes them together)
  static constexpr uint32_t kYBlock = kPParts * NC * 128, kYPart = kPParts == 1 ? 2 * kYBlock : NC * 128;
  static constexpr uint32_t kYBytes = 3 * 2 * NC * 128;
  static constexpr uint32_t kTCPart = 2 * NC * 128;  // [T; C], NC columns of a row used
  // Byte offsets of dynamic shared memory, 1024-byte aligned.  Of trees of more
  // than 32 nodes P and then [T; C] stand where Y was, which is free again when
  // u and o are there; of smaller ones they have places of their own.
  static constexpr bool kOverY = NC > 32;
  static constexpr uint32_t kX = 0;
  static constexpr uint32_t kY = kX + 3 * kXPart;
  static constexpr uint32_t kTC = kOverY ? kY : kY + kYBytes;
  // P, [2 NC][NC] FP32, column c of row r at c ^ (r & 31)
  static constexpr uint32_t kP = kOverY ? kY : kTC + 3 * kTCPart;
  static_assert(!kOverY || (3 * kTCPart <= kYBytes && 2 * NC * NC * 4 <= kYBytes), "over Y");
  // decays [NC][128] FP32; where gates have no place of their own a row's arrive
  // in its first half
  static constexpr uint32_t kD = kOverY ? kY + kYBytes : kP + 2 * NC * NC * 4;
  // Keys and queries [NC][128] BF16.  Where there is room gates stand behind them,
  // and the three come by tensor copies of eight nodes, which the warp with the
  // requests sends for ahead of their turn; else by the nodes' warps' own copies.
  static constexpr int kRawBufs = NC > 32 ? 0 : (BF16 ? 2 : 1), kCopies = kRawBufs > 0 ? kRawBufs : 1;
  static constexpr uint32_t kRows = NC * kDim * 2;
  static constexpr uint32_t kRaw = (kRawBufs > 0 ? 3 : 2) * kRows;
  static constexpr uint32_t kK = kD + NC * kDim * 4;
  static constexpr uint32_t kReplayK = kK + kCopies * kRaw;  // the replay's operands
  static constexpr uint32_t kReplayD = kReplayK + kMaxQ * kDim * 4;
  static constexpr uint32_t kReplayU = kReplayD + kMaxQ * kDim * 4;
  static constexpr uint32_t kReplayDn = kReplayU + kMaxQ * kDim * 4;
  static constexpr uint32_t kDt = kReplayDn + kDim * 4;  // dt_bias of the head
  // per node: P with its ancestors' keys, the nearest's first, and beta
  static constexpr uint32_t kA = kDt + kCopies * kDim * 4;
  static constexpr uint32_t kNorms = kA + NC * kPath * 4;  // of keys, then of queries
  static constexpr uint32_t kBad = kNorms + 2 * NC * 4;    // [NC / 8][128] nodes, a byte's bits
  static constexpr uint32_t kTasks = kBad + kDBufs * NC / 8 * kDim;
  static constexpr uint32_t kParent = kTasks + 4 * sizeof(TreeTask);
  // A page comes here by asynchronous copies, a whole item ahead, 8 KB a warp, where
  // there is room (48 requests of up to 32 nodes: 97 -> 91 us); else to registers, a
  // unit ahead, of BF16 pages four.  A warp's rows of an FP32 page are one piece of
  // memory and one copy, as they are (83 -> 82 us of the kernel alone); those of a BF16 page, whose rows would meet in
  // the banks four times over, go by 16 bytes each to a place of their own.
  static constexpr bool kStaged = NC <= 32;
  static constexpr uint32_t kPage = kStaged ? round_up(kParent + kTreeNodes, 128) : kParent + kTreeNodes;
  static constexpr uint32_t kPageBars = kPage + (kStaged ? kPageWarps * 8192 : 0);  // its parts are there
  static constexpr uint32_t kBars = kPageBars + (kStaged ? kPageWarps * 8 : 0);
  static constexpr uint32_t kSlot = kBars + sizeof(TreeBars);
  static constexpr uint32_t kBytes = kSlot + 8;
  static_assert(kTasks % 8 == 0 && kBars % 8 == 0 && sizeof(TreeTask) % 8 == 0, "alignment");
  static_assert(kBytes <= 227 * 1024 && 2 * kBytes > 228 * 1024, "one CTA an SM");
};

// A thread's part of 16 rows and 32 keys of the page: rows lane / 4 + 8 i, keys 16
// j + 4 (lane % 4) + 0 .. 3.
template <bool BF16>
struct PageUnit {
  using Four = typename std::conditional<BF16, uint2, float4>::type;
  Four s[2][2];  // [j][i]
  __device__ __forceinline__ void load(const void *pool, long long at) {
    const auto *from = reinterpret_cast<const Four *>(static_cast<const char *>(pool) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) s[j][i] = __ldcs(from + (8 * i * kDim + 16 * j) / 4);
  }
  // From a warp's staged rows.  Of BF16, 256 bytes a row, 16-byte piece c of row r
  // stands at place(r, c), where no two of 16 lanes meet in a bank; of FP32 the rows
  // stand as in memory, and pairs of lanes meet.
  static __device__ __forceinline__ int place(int r, int c) {
    return r * 256 + ((c >> 1 ^ (r & 3)) << 5) + (c & 1) * 16;
  }
  __device__ __forceinline__ void load_staged(const uint8_t *rows, int row, int key, int lane) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row + lane / 4 + 8 * i, byte = (key + 16 * j + 4 * (lane & 3)) * (BF16 ? 2 : 4);
        const int at = BF16 ? place(r, byte >> 4) + (byte & 15) : r * (kDim * 4) + byte;
        s[j][i] = *reinterpret_cast<const Four *>(rows + at);
      }
  }
};

// Swizzled place of channels 4 lane .. 4 lane + 3 of a tile's row.
__device__ __forceinline__ uint32_t tile_place(int row, int lane, uint32_t block) {
  return (uint32_t)(lane >> 4) * block + row * 128 + ((((lane & 15) >> 1) ^ (row & 7)) << 4) +
         (lane & 1) * 8;
}

__device__ __forceinline__ void store_parts(uint8_t *to, uint32_t part, float4 x) {
  float2 lo = make_float2(x.x, x.y), hi = make_float2(x.z, x.w);
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    const uint32_t c = take_part(lo);
    *reinterpret_cast<uint2 *>(to + e * part) = make_uint2(c, take_part(hi));
  }
}

// 1 / x, within a unit of the last place (x is far from FP32's ends).
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// j-th byte of a node's path.
__device__ __forceinline__ int path_byte(uint2 path, int j) {
  return ((j < 4 ? path.x : path.y) >> (8 * (j & 3))) & 0xff;
}

// A warp's way through the CTA's items.  A group of warps that has a barrier of
// its own agrees there, item by item, that no wait of any has run out.
struct TreeItems {
  const TreeTask *tasks;
  TreeBars *bars;
  int seq, t0, n, slot, row, pending, h, h1;
  bool ok;  // no wait has run out

  __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) {
    ok = tm_wait(bar, parity) && ok;
    return ok;
  }
  // The next task; false where there is none.
  __device__ __forceinline__ bool load() {
    if (!wait(&bars->task_full[seq & 3], (uint32_t)(seq >> 2) & 1u)) return false;
    const TreeTask &t = tasks[seq & 3];
    t0 = t.t0, n = t.n, slot = t.slot, row = t.row, pending = t.pending, h = t.h0, h1 = t.h1;
    return n >= 0;
  }
  __device__ __forceinline__ bool start(const TreeTask *ts, TreeBars *bs) {
    tasks = ts, bars = bs, seq = 0, ok = true;
    return load();
  }
  // The next item; hands a task's place back behind its last one.
  __device__ __forceinline__ bool next(int lane) {
    if (++h < h1) return true;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->task_free[seq & 3]);
    ++seq;
    return load();
  }
  __device__ __forceinline__ const uint2 *paths() const { return tasks[seq & 3].path; }
};

// k, q, raw_g and v [n_tokens, H, 128] in boxes of eight tokens of a head.
constexpr int kBoxTokens = 8;
struct TreeTokenMaps {
  CUtensorMap of[4];
};

template <int NC, bool BF16>
__global__ void __launch_bounds__(TreeMma<NC, BF16>::kThreads, 1)
    kda_tree_mma_kernel(const TreeVerifyParams p, const __grid_constant__ TreeTokenMaps maps,
                        int n_items) {
  using L = TreeMma<NC, BF16>;
  // (its alignment known, the addresses below are constants, which take no
  // registers)
  extern __shared__ __align__(1024) uint8_t mem[];
  float *const decay = reinterpret_cast<float *>(mem + L::kD);
  float *const coefs = reinterpret_cast<float *>(mem + L::kA);
  TreeTask *const tasks = reinterpret_cast<TreeTask *>(mem + L::kTasks);
  TreeBars *const bars = reinterpret_cast<TreeBars *>(mem + L::kBars);
  uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(mem + L::kSlot);
  const TreeMaps &mp = p.maps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int begin = (int)((long long)n_items * blockIdx.x / gridDim.x);
  const int end = (int)((long long)n_items * (blockIdx.x + 1) / gridDim.x);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->task_full[i], 1);
      // (the warps of R may go through the tasks twice)
      mbar_init(&bars->task_free[i], L::kWarps - 1 + (L::kDBufs > 1 ? L::kRWarps : 0));
    }
    mbar_init(&bars->x_full, L::kXWarps);
    mbar_init(&bars->n_full, L::kNodeWarps);
    mbar_init(&bars->x_free, 1);
    mbar_init(&bars->y_free, 1);
    mbar_init(&bars->p_full, 1);
    mbar_init(&bars->p_free, L::kTWarps);
    mbar_init(&bars->a_full, L::kPageWarps);
    mbar_init(&bars->a_free, 1);
    if (L::kStaged)
      for (int i = 0; i < L::kPageWarps; ++i) mbar_init(reinterpret_cast<uint64_t *>(mem + L::kPageBars) + i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->d_full[i], 1);
      mbar_init(&bars->d_free[i], L::kRWarps);
      mbar_init(&bars->r_full[i], L::kRWarps);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->done[i], 1);
      mbar_init(&bars->raw_full[i], 1);
      mbar_init(&bars->raw_free[i], L::kNodeWarps);
    }
    mbar_init(&bars->t_full, L::kTWarps);
    mbar_init(&bars->t_free, 1);
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const auto page_of = [&](int slot, int h) { return slot * p.slot_stride + (long long)h * kDim * kDim; };
  // a warp's part of what is handed over is done
  const auto arrive = [&](uint64_t *bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // X and Y of `it`, the done-th item with nodes: nodes from the first-th on, a node
  // a warp, four channels a lane
  const auto make_xy = [&](TreeItems &it, const uint16_t *keys, const uint16_t *queries, int first,
                           int done) {
    const float *const norms = reinterpret_cast<const float *>(mem + L::kNorms);
    const int n = it.n, cols = (n + 15) & ~15;
    if (done > 0) {
      it.wait(&bars->x_free, (uint32_t)(done - 1) & 1u);
      it.wait(&bars->y_free, (uint32_t)(done - 1) & 1u);
    }
#pragma unroll 1
    for (int t = first; t < n; t += L::kXWarps) {
      const uint2 path = it.paths()[t];
      const int m = path.x & 0xff;
      float4 g = lds4(decay + t * kDim + 4 * lane);
      const float4 k = scale4(bf16x4(*reinterpret_cast<const uint2 *>(keys + t * kDim + 4 * lane)), norms[t]);
      const float4 q = scale4(bf16x4(*reinterpret_cast<const uint2 *>(queries + t * kDim + 4 * lane)), norms[NC + t]);
      uint2 way = path;
#pragma unroll 1
      for (int j = 0; j < m; ++j) {  // (the same in every lane)
        way = make_uint2(__funnelshift_r(way.x, way.y, 8), way.y >> 8);
        g = fmul4(g, lds4(decay + (way.x & 0xff) * kDim + 4 * lane));
      }
      // (queries stand a multiple of 16 rows behind the keys: the same swizzle)
      uint8_t *const x = mem + L::kX + tile_place(t, lane, L::kXBlock);
      store_parts(x, L::kXPart, fmul4(k, g));
      store_parts(x + cols * 128, L::kXPart, fmul4(q, g));
      store_parts(mem + L::kY + tile_place(t, lane, L::kYBlock), L::kYPart,
                  make_float4(k.x * rcp_fast(g.x), k.y * rcp_fast(g.y), k.z * rcp_fast(g.z),
                              k.w * rcp_fast(g.w)));
    }
    fence_proxy_async_smem();
    arrive(&bars->x_full);
  };
  bool ok = true;
  if (warp < L::kR0) {
    warpgroup_reg_alloc<L::kPageRegs>();
  } else {
    warpgroup_reg_dealloc<L::kOtherRegs>();
  }

  if (warp < L::kR0) {
    // ======== pages: of a quarter's rows half of the keys a warp, of FP32 staged ones
    // half of the rows (and BF16 pages have one warp a quarter)
    // units of 16 rows and 32 keys, those of the same rows first
    constexpr bool kBulk = L::kStaged && !BF16;
    constexpr int kUnits = 32 / L::kPageWarps, kKeys = kBulk ? kDim : 16 * kUnits, kThreads = 32 * L::kPageWarps;
    constexpr int kAhead = L::kStaged ? 0 : BF16 ? 4 : 1, kRecs = kMaxQ / L::kPageWarps;
    uint8_t *const staged = mem + L::kPage + warp * 8192;
    uint64_t *const page_full = reinterpret_cast<uint64_t *>(mem + L::kPageBars) + warp;
    constexpr int kInRow = kKeys / 32;  // units of the same rows
    const auto unit_at = [](int e) { return 16 * (e / kInRow) * kDim + 32 * (e % kInRow); };
    const int quarter = warp & 3, which = warp >> 2;
    const int row0 = 32 * quarter + (kBulk ? 16 * which : 0), key0 = kBulk ? 0 : kKeys * which;
    const uint32_t lanes = tmem + ((uint32_t)row0 << 16);
    float *const rk = reinterpret_cast<float *>(mem + L::kReplayK);
    float *const rd = reinterpret_cast<float *>(mem + L::kReplayD);
    float *const ru = reinterpret_cast<float *>(mem + L::kReplayU);
    float *const rdn = reinterpret_cast<float *>(mem + L::kReplayDn);
    const int k0 = key0 + 4 * (lane & 3);
    TreeItems it;
    int done = 0;  // items with nodes
    uint32_t asked = 0, had = 0;  // pages
    float4 rec_dt;
    float rec_a;
    PageUnit<BF16> pg[L::kStaged ? 1 : kUnits];
    uint2 rec_k[kRecs], rec_g[kRecs];
    float4 rec_u[kRecs];
    // an item's records (a warp one; gates' constants where registers are left for
    // them) and first units, ahead of its turn; and the next head's page on its way
    // to L2
    const auto page_part = [&] {
      return page_of(it.slot, it.h) + (long long)(row0 + lane / 4) * kDim + k0;
    };
    const auto ask = [&] {
      if (kBulk && it.pending > 0) {
        rec_dt = __ldg(reinterpret_cast<const float4 *>(p.dt_bias + it.h * kDim) + lane);
        rec_a = __ldg(p.A_log + it.h);
      }
#pragma unroll
      for (int i = 0; i < kRecs; ++i)
        if (warp + i * L::kPageWarps < it.pending) {
          const long long row = (long long)it.h * mp.rq + warp + i * L::kPageWarps;
          const uint2 *rec = reinterpret_cast<const uint2 *>(p.kg + it.row * p.kg_stride + row * 2 * kDim) + lane;
          rec_k[i] = __ldg(rec);
          rec_g[i] = __ldg(rec + 32);
          rec_u[i] = __ldg(reinterpret_cast<const float4 *>(p.corr + it.row * p.corr_stride + row * kDim) + lane);
        }
      if constexpr (kBulk) {
        if (lane == 0) {
          mbar_arrive_expect_tx(page_full, 8192);
          bulk_g2s(staged, static_cast<const float *>(p.state) + page_of(it.slot, it.h) + row0 * kDim, 8192,
                   page_full);
        }
        ++asked;
      } else if constexpr (L::kStaged) {
        const char *from = static_cast<const char *>(p.state) +
                           (page_of(it.slot, it.h) + row0 * kDim) * 2;
#pragma unroll 2
        for (int i = lane; i < 512; i += 32)
          cp_async16(staged + PageUnit<true>::place(i >> 4, i & 15),
                     from + (i >> 4) * (kDim * 2) + 16 * (i & 15));
      } else {
#pragma unroll
        for (int e = 0; e < kAhead; ++e) pg[e].load(p.state, page_part() + unit_at(e));
      }
      if (it.h + 1 < it.h1)
#pragma unroll
        for (int i = 0; i < (BF16 ? 256 : 512) / kThreads; ++i)
          prefetch_l2(static_cast<const char *>(p.state) + page_of(it.slot, it.h + 1) * (BF16 ? 2 : 4) +
                      (i * kThreads + tid) * 128);
    };
    bool more = it.start(tasks, bars);
    if (more) ask();
    if (named_bar_or(3, kThreads, !it.ok)) more = it.ok = false;
    while (more) {
      const int replay = it.pending;
      const long long page = page_part();
      if (!BF16 && replay > 0) {
#pragma unroll
        for (int i = 0; i < kRecs; ++i)
          if (const int t = warp + i * L::kPageWarps; t < replay) {
            const float4 k = bf16x4(rec_k[i]);
            if (!kBulk) {
              rec_dt = __ldg(reinterpret_cast<const float4 *>(p.dt_bias + it.h * kDim) + lane);
              rec_a = __ldg(p.A_log + it.h);
            }
            sts4(rk + t * kDim + 4 * lane, scale4(k, rsqrtf(warp_sum(dot4(k, k)) + kNormEps)));
            sts4(rd + t * kDim + 4 * lane, decay4(expf(rec_a), bf16x4(rec_g[i]), rec_dt, p.lower_bound));
            sts4(ru + t * kDim + 4 * lane, rec_u[i]);
          }
        named_bar(3, kThreads);
        if (tid < kDim) replay_suffix(rk, rd, rdn, replay, tid);
        named_bar(3, kThreads);
      }
      // S_n, and its parts to tensor memory
      if (it.n > 0 && done > 0) {
        it.wait(&bars->a_free, (uint32_t)(done - 1) & 1u);
        tc_fence_after();
      }
      if (kBulk) {
        it.wait(page_full, had++ & 1u);
      } else if (L::kStaged) {
        cp_async_wait_all();
        __syncwarp();
      }
#pragma unroll(L::kStaged ? 1 : kUnits)
      for (int e = 0; e < kUnits; ++e) {
        PageUnit<BF16> &unit = pg[L::kStaged ? 0 : e];
        const int rh = e / kInRow, k32 = 32 * (e % kInRow);
        if constexpr (L::kStaged) unit.load_staged(staged, 16 * rh, k32, lane);
        if constexpr (!BF16) {
          if (replay > 0) {
            const float *up = ru + row0 + 16 * rh + lane / 4;
            const float *kp = rk + k0 + k32, *dp = rdn + k0 + k32;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 x = lds4(dp + 16 * j);
              unit.s[j][0] = fmul4(unit.s[j][0], x);
              unit.s[j][1] = fmul4(unit.s[j][1], x);
            }
#pragma unroll 1
            for (int t = 0; t < replay; ++t, kp += kDim, up += kDim) {
              const float u0 = up[0], u1 = up[8];
              const float4 x0 = lds4(kp), x1 = lds4(kp + 16);
              unit.s[0][0] = ffma4s(u0, x0, unit.s[0][0]);
              unit.s[0][1] = ffma4s(u1, x0, unit.s[0][1]);
              unit.s[1][0] = ffma4s(u0, x1, unit.s[1][0]);
              unit.s[1][1] = ffma4s(u1, x1, unit.s[1][1]);
            }
            float *to = static_cast<float *>(p.state) + page + unit_at(e);
#pragma unroll
            for (int c = 0; c < 4; ++c) stg4(to + 8 * (c % 2) * kDim + 16 * (c / 2), unit.s[c / 2][c % 2]);
          }
        }
        if (it.n > 0)
#pragma unroll
          for (int part = 0; part < (BF16 ? 1 : 3); ++part) {
            uint32_t w[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              auto &s = unit.s[c / 2][c % 2];
              if constexpr (BF16) {
                w[2 * c] = s.x;
                w[2 * c + 1] = s.y;
              } else {
                float2 lo = make_float2(s.x, s.y), hi = make_float2(s.z, s.w);
                w[2 * c] = take_part(lo);
                w[2 * c + 1] = take_part(hi);
                s = make_float4(lo.x, lo.y, hi.x, hi.y);
              }
            }
            tm_store_16x16(lanes + ((uint32_t)(16 * rh) << 16) + kTmPartCols * part + (key0 + k32) / 2, w);
          }
        if constexpr (!L::kStaged)
          if (e + kAhead < kUnits) pg[e + kAhead].load(p.state, page + unit_at(e + kAhead));
      }
      if (it.n > 0) {
        tm_store_wait();
        tc_fence_before();
        arrive(&bars->a_full);
        ++done;
      }
      more = it.next(lane);
      __syncwarp();  // (the staged rows are read)
      if (more) ask();
      // (the replay's operands are read)
      if (named_bar_or(3, kThreads, !it.ok)) more = it.ok = false;
    }
    if (had < asked) it.wait(page_full, had & 1u);
    if (L::kStaged && !kBulk) cp_async_wait_all();
    ok = it.ok;
  } else if (warp < L::kT0) {
    // ======== R and the outputs: a row a lane, eight nodes at a time
    // Where w and y have two places an item's R comes before the outputs of the
    // one ahead of it, whose product is meanwhile formed.
    const int quarter = warp & 3, which = (warp - L::kR0) >> 2, at = 32 * quarter + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    const long long step = (long long)p.H * kDim;
    const auto agree = [&](bool x) { return named_bar_or(4, 32 * L::kRWarps, x); };
    // R of `it`, its parts to tensor memory; true where an entry is not finite
    const auto front = [&](TreeItems &it, int done) {
      const int n = it.n, cols = (n + 15) & ~15, buf = done % L::kDBufs;
      const uint32_t d = kTmD + buf * 2 * NC, to_r = L::kTmR + buf * (3 * NC / 2);
      uint8_t *const marks = mem + L::kBad + buf * (NC / 8 * kDim) + at;
      const uint16_t *from = p.v + ((long long)it.t0 * p.H + it.h) * kDim + at;
      uint32_t v[8];
      const auto ask = [&](int i0) {
        const uint16_t *x = from + i0 * step;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = __ldg(x);
          if (i0 + i + 1 < n) x += step;  // (behind the last: again the last)
        }
      };
      if (8 * which < n) ask(8 * which);
      it.wait(&bars->d_full[buf], (uint32_t)(done / L::kDBufs) & 1u);
      tc_fence_after();
      bool bad = false;
#pragma unroll 1
      for (int i0 = 8 * which; i0 < cols; i0 += 16) {
        float x[8];
        tm_load(lanes + d + i0, x);
        tm_load_wait();
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = i0 + i < n ? __uint_as_float(v[i] << 16) - x[i] : 0.f;
          all += fabsf(x[i]);
        }
        if (i0 + 16 < n) ask(i0 + 16);
        uint32_t bits = 0;
        if (!(all < __int_as_float(0x7f800000))) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(fabsf(x[i]) < __int_as_float(0x7f800000))) {
              bits |= 1u << i;
              x[i] = 0.f;
            }
          bad = bad || bits != 0;
        }
        marks[i0 / 8 * kDim] = (uint8_t)bits;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 pair = make_float2(x[2 * i], x[2 * i + 1]);
            w[i] = take_part(pair);
            x[2 * i] = pair.x, x[2 * i + 1] = pair.y;
          }
          tm_store_32x4(lanes + to_r + (NC / 2) * part + i0 / 2, w[0], w[1], w[2], w[3]);
        }
        // (u is added up on zeros, o on y)
        tm_store_32x4(lanes + d + i0, 0, 0, 0, 0);
        tm_store_32x4(lanes + d + i0 + 4, 0, 0, 0, 0);
      }
      tm_store_wait();
      tc_fence_before();
      arrive(&bars->r_full[buf]);
      return bad;
    };
    // the outputs of `it`
    const auto back = [&](TreeItems &it, int done, bool any_bad) {
      const int n = it.n, cols = (n + 15) & ~15, buf = done % L::kDBufs;
      const uint32_t d = kTmD + buf * 2 * NC;
      const uint8_t *const marks = mem + L::kBad + buf * (NC / 8 * kDim) + at;
      const long long first = ((long long)it.t0 * p.H + it.h) * kDim + at;
      it.wait(&bars->o_full[buf], (uint32_t)(done / L::kDBufs) & 1u);
      tc_fence_after();
#pragma unroll 1
      for (int i0 = 8 * which; i0 < n; i0 += 16) {
        float u[8], o[8];
        tm_load(lanes + d + i0, u);
        tm_load(lanes + d + cols + i0, o);
        tm_load_wait();
        if (any_bad) {
#pragma unroll 1
          for (int i = 0; i < 8 && i0 + i < n; ++i) {
            const uint2 way = it.paths()[i0 + i];
            bool hit = false;
            for (int j = 0; j <= (int)(way.x & 0xff); ++j) {
              const int s = j == 0 ? i0 + i : path_byte(way, j);
              hit = hit || (marks[(s >> 3) * kDim] >> (s & 7) & 1u);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (hit && e == i) u[e] = o[e] = __int_as_float(0x7fffffff);
          }
        }
        float *to_u = p.node_corr + first + i0 * step;
        uint16_t *to_o = p.out + first + i0 * step;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i0 + i < n) {
            *to_u = u[i];
            *to_o = f32_to_bf16_bits(o[i]);
          }
          to_u += step, to_o += step;
        }
      }
      tc_fence_before();
      arrive(&bars->d_free[buf]);
    };
    // `out` is the item behind `it` (every one in its turn: the tasks of those
    // without nodes are handed back too)
    TreeItems it, out;
    int done = 0;  // items whose R is formed
    bool more = it.start(tasks, bars), first = true, owed = false, was_bad = false;
    out.ok = true;
    if (L::kDBufs > 1) out.start(tasks, bars);
    while (true) {
      const bool live = more && it.n > 0;
      bool bad = false;
      if (live) bad = front(it, done++);
      // (whatever a warp has found, it comes here, where all go on or none)
      if (agree(bad || !it.ok || !out.ok)) {
        bad = agree(bad);
        if (agree(!it.ok || !out.ok)) break;
      }
      if (L::kDBufs == 1) {
        if (live) back(it, done - 1, bad);
        if (bad) agree(false);  // (the marks are read)
      } else {
        if (owed) back(out, live ? done - 2 : done - 1, was_bad);
        if (was_bad) agree(false);
        if (!first && more) out.next(lane);
        first = false, owed = live, was_bad = bad;
      }
      if (!more) break;
      more = it.next(lane);
    }
    ok = it.ok && out.ok;
  } else if (warp < L::kIssue0) {
    // ======== T and C: a lane a row of P, nodes' keys, then their queries
    const int tw = warp - L::kT0, row = 32 * tw + lane;
    float *const mine = reinterpret_cast<float *>(mem + L::kP) + row * NC;
    TreeItems it;
    int done = 0;
    bool more = it.start(tasks, bars);
    if (named_bar_or(2, 32 * L::kTWarps, !it.ok)) more = it.ok = false;
    while (more) {
      const int n = it.n, cols = (n + 15) & ~15;
      if (n == 0) {
        more = it.next(lane);
        if (named_bar_or(2, 32 * L::kTWarps, !it.ok)) more = it.ok = false;
        continue;
      }
      const bool key = row < cols;
      const int t = key ? row : row - cols;
      const bool live = row < 2 * cols && t < n;
      const uint2 path = live ? it.paths()[t] : make_uint2(0, 0);
      const int m = live ? (int)(path.x & 0xff) : -1;
      uint16_t beta = 0;
      if constexpr (L::kTHelps) {
        it.wait(&bars->n_full, (uint32_t)done & 1u);
        const uint16_t *const raw = reinterpret_cast<const uint16_t *>(mem + L::kK);
        make_xy(it, raw, raw + NC * kDim, L::kNodeWarps + tw, done);
      }
      if (live) beta = __ldg(p.beta + (long long)(it.t0 + t) * p.H + it.h);
      // this item's values on their way to L2, and the next head's nodes (elsewhere
      // the warp with the requests sends for them)
      if constexpr (L::kRawBufs == 0)
        for (int i = row; i < n * 8; i += 32 * L::kTWarps) {
          const int what = i >> 1 & 3;
          const long long at = ((long long)(it.t0 + (i >> 3)) * p.H + it.h) * kDim + (i & 1) * (kDim / 2);
          if (what == 0) {
            prefetch_l2(p.v + at);
          } else if (it.h + 1 < it.h1) {
            prefetch_l2((what == 1 ? p.k : (what == 2 ? p.q : p.g)) + at + kDim);
          }
        }
      it.wait(&bars->p_full, (uint32_t)done & 1u);
      tc_fence_after();
      for (int c = 0; c < cols; c += 16) {
        float x[16];
        tm_load(tmem + ((uint32_t)(32 * tw) << 16) + L::kTmP + c, x);
        tm_load_wait();
#pragma unroll
        for (int part = 1; part < L::kPParts; ++part) {
          float y[16];
          tm_load(tmem + ((uint32_t)(32 * tw) << 16) + L::kTmP + part * NC + c, y);
          tm_load_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] += y[i];
        }
        if (row < 2 * cols)
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[(c + i) ^ lane] = x[i];
      }
      tc_fence_before();
      arrive(&bars->p_free);
      // A row's weights: of u_s in u_t (in o_t) over all ways down the path from
      // s, W_s = -sum W_r beta_r A[r][s] over the r between (and P's entry); then
      // R_s enters with W_s beta_s.
      float wt[kPath];
      wt[0] = m < 0 || key ? 1.f : mine[t ^ lane];
#pragma unroll
      for (int j = 1; j < kPath; ++j) wt[j] = j <= m ? mine[path_byte(path, j) ^ lane] : 0.f;
      if (key && live) {
        sts4(coefs + t * kPath, make_float4(wt[1], wt[2], wt[3], wt[4]));
        sts4(coefs + t * kPath + 4, make_float4(wt[5], wt[6], wt[7], sigmoidf_fast(bf16_bits_to_f32(beta))));
#pragma unroll
        for (int j = 1; j < kPath; ++j) wt[j] = 0.f;
      }
      named_bar(2, 32 * L::kTWarps);
      // [T; C] in parts: zeros, and a row's entries
      if (done > 0) it.wait(&bars->t_free, (uint32_t)(done - 1) & 1u);
      uint8_t *const to = mem + L::kTC + row * 128;
      if (row < 2 * cols)
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll 1
          for (int c = 0; c < cols / 8; ++c)
            *reinterpret_cast<uint4 *>(to + e * L::kTCPart + ((c ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
      // step i: wt[k] is the weight of the path's node i + k
      uint2 way = path;
      int s = t;
      float4 x = lds4(coefs + (m < 0 ? 0 : t) * kPath), y = lds4(coefs + (m < 0 ? 0 : t) * kPath + 4);
#pragma unroll 1
      for (int i = 0; i <= m; ++i) {
        float2 w = make_float2(wt[0] * y.w, 0.f);
        const float f[kPath - 1] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z};
#pragma unroll
        for (int k = 1; k < kPath; ++k) wt[k - 1] = fmaf(-w.x, f[k - 1], wt[k]);
        uint8_t *const place = to + (((s >> 3) ^ (row & 7)) << 4) + (s & 7) * 2;
        way = make_uint2(__funnelshift_r(way.x, way.y, 8), way.y >> 8);
        s = way.x & 0xff;  // (behind the last: some node of the path, or 0)
        x = lds4(coefs + s * kPath), y = lds4(coefs + s * kPath + 4);
#pragma unroll
        for (int e = 0; e < 3; ++e)
          *reinterpret_cast<uint16_t *>(place + e * L::kTCPart) = (uint16_t)take_part(w);
      }
      fence_proxy_async_smem();
      arrive(&bars->t_full);
      ++done;
      more = it.next(lane);
      if (named_bar_or(2, 32 * L::kTWarps, !it.ok)) more = it.ok = false;
    }
    ok = it.ok;
  } else if (warp < L::kTask0) {
    // ======== products
    const uint32_t lead = tm_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t x0 = __shfl_sync(0xffffffffu, smem_u32(mem + L::kX), 0);
    const uint32_t y0 = __shfl_sync(0xffffffffu, smem_u32(mem + L::kY), 0);
    const uint32_t c0 = __shfl_sync(0xffffffffu, smem_u32(mem + L::kTC), 0);
    const auto commit = [&](uint64_t *bar) {
      if (lead) umma_commit(bar);
      __syncwarp();
    };
    // parts of A and of B of the six products, the smallest first, two bits each
    constexpr uint32_t kA6 = 2 | 0 << 2 | 1 << 4 | 1 << 6 | 0 << 8 | 0 << 10,
                       kB6 = 0 | 2 << 2 | 1 << 4 | 0 << 6 | 1 << 8 | 0 << 10;
    TreeItems it;
    uint32_t done = 0;
    if (warp == L::kIssue0) {
      for (bool more = it.start(tasks, bars); more; more = it.next(lane)) {
        if (it.n == 0) continue;
        const uint32_t cols = __shfl_sync(0xffffffffu, (uint32_t)(it.n + 15) & ~15u, 0);
        const uint32_t buf = done % L::kDBufs, d = tm + kTmD + buf * 2 * NC;
        it.wait(&bars->x_full, done & 1u);
        if (done > 0) it.wait(&bars->p_free, (done - 1) & 1u);
        if (!it.ok) break;
        tc_fence_after();
        // (M = 128 rows: those behind X's are other operands', and P's rows of them
        // nobody reads.)  A product reads its 128 rows of X from shared memory
        // whatever its N: where tensor memory has room, one takes all parts of Y that
        // go with part e of X, those with part j to P's (e + j)-th.  Products of one
        // size are summed there, so that the small ones' sums are not rounded as the
        // large one's is (all on one, pairs of nodes were off by 51 2^-24).
#pragma unroll 1
        for (uint32_t e = 0; e < (L::kPParts == 1 ? 6 : 3); ++e) {
          const uint32_t x = x0 + (L::kPParts == 1 ? (kA6 >> 2 * e & 3) : e) * L::kXPart;
          const uint32_t y = y0 + (L::kPParts == 1 ? (kB6 >> 2 * e & 3) * L::kYPart : 0);
          const uint32_t columns = L::kPParts == 1 ? cols : (2 - e) * NC + cols;
          const uint32_t p_at = tm + L::kTmP + (L::kPParts == 1 ? 0 : e * NC);
#pragma unroll
          for (int ks = 0; ks < kDim / 16; ++ks)
            tm_mma_ss(p_at, umma_desc_sw128(x + (ks >> 2) * L::kXBlock + (ks & 3) * 32),
                      umma_desc_sw128(y + (ks >> 2) * L::kYBlock + (ks & 3) * 32), tm_idesc(columns),
                      e > 0 || ks > 0, lead);
        }
        commit(&bars->p_full);
        if (!L::kOverY) commit(&bars->y_free);
        it.wait(&bars->a_full, done & 1u);
        if (done >= (uint32_t)L::kDBufs) it.wait(&bars->d_free[buf], (done / L::kDBufs - 1) & 1u);
        if (!it.ok) break;
        tc_fence_after();
#pragma unroll 1
        for (uint32_t e = 0; e < (BF16 ? 3 : 6); ++e) {
          const uint32_t s = tm + (BF16 ? 0 : (kA6 >> 2 * e & 3)) * kTmPartCols;
          const uint32_t x = x0 + (BF16 ? 2 - e : (kB6 >> 2 * e & 3)) * L::kXPart;
#pragma unroll 4
          for (int ks = 0; ks < kDim / 16; ++ks)
            tm_mma(d, s + 8 * ks, umma_desc_sw128(x + (ks >> 2) * L::kXBlock + (ks & 3) * 32),
                   tm_idesc(2 * cols), e > 0 || ks > 0, lead);
        }
        commit(&bars->d_full[buf]);
        commit(&bars->a_free);
        commit(&bars->x_free);
        ++done;
      }
    } else {
      for (bool more = it.start(tasks, bars); more; more = it.next(lane)) {
        if (it.n == 0) continue;
        const uint32_t cols = __shfl_sync(0xffffffffu, (uint32_t)(it.n + 15) & ~15u, 0);
        const uint32_t buf = done % L::kDBufs, d = tm + kTmD + buf * 2 * NC;
        it.wait(&bars->t_full, done & 1u);
        it.wait(&bars->r_full[buf], (done / L::kDBufs) & 1u);
        if (!it.ok) break;
        tc_fence_after();
#pragma unroll 1
        for (uint32_t e = 0; e < 6; ++e)
#pragma unroll 1
          for (uint32_t ks = 0; ks < cols / 16; ++ks)
            tm_mma(d, tm + L::kTmR + buf * (3 * NC / 2) + (kA6 >> 2 * e & 3) * (NC / 2) + 8 * ks,
                   umma_desc_sw128(c0 + (kB6 >> 2 * e & 3) * L::kTCPart + ks * 32),
                   tm_idesc(2 * cols), true, lead);
        commit(&bars->o_full[buf]);
        commit(&bars->t_free);
        if (L::kOverY) commit(&bars->y_free);
        ++done;
      }
    }
    ok = it.ok;
    // every product issued has completed before the columns are released
    commit(&bars->done[warp - L::kIssue0]);
    ok = tm_wait(&bars->done[warp - L::kIssue0], 0u) && ok;
  } else if (warp < L::kNode0) {
    // ======== requests: checked, their paths listed; the inert ones' zeros
    int8_t *const parent = reinterpret_cast<int8_t *>(mem + L::kParent);
    int seq = 0;
    uint32_t sent = 0;  // items whose nodes' rows were sent for
    const auto place = [&] {
      if (seq >= 4)
        ok = tm_wait(&bars->task_free[seq & 3], (uint32_t)((seq >> 2) - 1) & 1u);
      return ok;
    };
    for (int item = begin; item < end && ok;) {
      const int b = item / p.H, h0 = item - b * p.H;
      const int h1 = p.H - h0 < end - item ? p.H : h0 + (end - item);
      item += h1 - h0;
      const TreeRequest r = tree_request(mp, b);
      if (r.error == KDA_OK && r.slot < 0) {
        for (long long i = lane; i < (long long)r.n * (h1 - h0) * (kDim / 8); i += 32) {
          const int c = (int)(i % (kDim / 8)), h = h0 + (int)(i / (kDim / 8) % (h1 - h0));
          const long long t = r.t0 + i / (kDim / 8) / (h1 - h0);
          *reinterpret_cast<uint4 *>(p.out + (t * p.H + h) * kDim + 8 * c) = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      if (r.error != KDA_OK || !load_tree(mp, r, parent, lane)) {
        if (lane == 0) report(mp.status, KDA_ERR_ARG);
        continue;
      }
      if (r.n == 0 && r.pending == 0) continue;
      if (!place()) break;
      TreeTask &task = tasks[seq & 3];
#pragma unroll
      for (int i = 0; i < NC / 32; ++i) {
        const int t = lane + 32 * i;
        uint32_t path[8];
        int a = parent[t];
        path[0] = 0;
#pragma unroll
        for (int j = 1; j < 8; ++j) {
          path[j] = a >= 0 ? a : t;
          path[0] += a >= 0;
          a = a >= 0 ? parent[a] : -1;
        }
        task.path[t] = make_uint2(path[0] | path[1] << 8 | path[2] << 16 | path[3] << 24,
                                  path[4] | path[5] << 8 | path[6] << 16 | path[7] << 24);
      }
      if (lane == 0) {
        task.t0 = r.t0, task.n = r.n, task.slot = r.slot, task.row = r.row;
        task.pending = r.pending, task.h0 = h0, task.h1 = h1;
      }
      arrive(&bars->task_full[seq & 3]);
      ++seq;
      if constexpr (L::kRawBufs > 0) {
        const int boxes = (r.n + kBoxTokens - 1) / kBoxTokens;
        for (int h = h0; h < h1 && boxes > 0; ++h, ++sent) {
          const uint32_t buf = sent % L::kRawBufs;
          if (sent >= (uint32_t)L::kRawBufs)
            ok = tm_wait(&bars->raw_free[buf], (sent / L::kRawBufs - 1) & 1u);
          if (!ok) break;
          if (lane == 0)
            mbar_arrive_expect_tx(&bars->raw_full[buf], 3 * boxes * kBoxTokens * kDim * 2 + kDim * 4);
          __syncwarp();
          const int which = lane >> 3, box = lane & 7;
          if (which < 3 && box < boxes)
            tma_load_3d(mem + L::kK + buf * L::kRaw + which * L::kRows + box * (kBoxTokens * kDim * 2),
                        &maps.of[which], 0, h, r.t0 + kBoxTokens * box, &bars->raw_full[buf]);
          // and to L2 this item's values, and the next one's nodes where they have to
          // wait for their place
          if (which == 3 && box < boxes) prefetch_box(&maps.of[3], 0, h, r.t0 + kBoxTokens * box);
          if (L::kRawBufs == 1 && which < 3 && box < boxes && h + 1 < h1)
            prefetch_box(&maps.of[which], 0, h + 1, r.t0 + kBoxTokens * box);
          if (lane == 31) bulk_g2s(mem + L::kDt + buf * kDim * 4, p.dt_bias + h * kDim, kDim * 4, &bars->raw_full[buf]);
        }
      }
    }
    // (no copy is on its way when the CTA ends)
    for (uint32_t i = sent > (uint32_t)L::kRawBufs ? sent - L::kRawBufs : 0; i < sent; ++i)
      ok = tm_wait(&bars->raw_full[i % L::kCopies], (i / L::kCopies) & 1u) && ok;
    if (ok && place()) {
      if (lane == 0) tasks[seq & 3].n = -1;
      arrive(&bars->task_full[seq & 3]);
    }
  } else {
    // ======== nodes
    constexpr int kThreads = 32 * L::kNodeWarps;
    const int nw = warp - L::kNode0, ntid = tid - 32 * L::kNode0;
    float *const norms = reinterpret_cast<float *>(mem + L::kNorms);
    TreeItems it;
    // where `done`'s operands are, and where a node's gates
    int done = 0;
    const auto raw = [&](int which) {
      return reinterpret_cast<uint16_t *>(mem + L::kK + done % L::kCopies * L::kRaw + which * L::kRows);
    };
    const auto dts = [&] { return reinterpret_cast<float *>(mem + L::kDt + done % L::kCopies * kDim * 4); };
    const auto gates = [&](int t) {
      return L::kRawBufs > 0 ? raw(2) + t * kDim : reinterpret_cast<uint16_t *>(decay + t * kDim);
    };
    // the next item with nodes, whose operands are then on their way
    const auto settle = [&](bool more) {
      while (more && it.n == 0) more = it.next(lane);
      if (named_bar_or(1, kThreads, !it.ok)) return it.ok = false;
      // (T's warps have read the nodes as well)
      if (L::kTHelps && done > 0) it.wait(&bars->x_full, (uint32_t)(done - 1) & 1u);
      if (L::kRawBufs == 0 && more) {
        const int c8 = 8 * (lane & 15);
#pragma unroll 1
        for (int t = nw; t < it.n; t += L::kNodeWarps) {
          const long long at = ((long long)(it.t0 + t) * p.H + it.h) * kDim + c8;
          cp_async16(raw(lane >> 4) + t * kDim + c8, (lane < 16 ? p.k : p.q) + at);
          if (lane < 16) cp_async16(gates(t) + c8, p.g + at);
        }
        if (ntid < kDim / 4) cp_async16(dts() + 4 * ntid, p.dt_bias + it.h * kDim + 4 * ntid);
      }
      return more;
    };
    bool more = settle(it.start(tasks, bars));
    while (more) {
      const int n = it.n;
      const float a = expf(__ldg(p.A_log + it.h));
      const uint16_t *const keys = raw(0), *const queries = raw(1);
      if constexpr (L::kRawBufs > 0) {
        it.wait(&bars->raw_full[done % L::kCopies], (uint32_t)(done / L::kCopies) & 1u);
      } else {
        cp_async_wait_all();
        named_bar(1, kThreads);
      }
      // norms and decays: two nodes a warp, eight channels a lane
      {
        const int hw = lane >> 4, c8 = 8 * (lane & 15);
#pragma unroll 1
        for (int t0 = 2 * nw; t0 < n; t0 += 2 * L::kNodeWarps) {
          const int t = t0 + hw < n ? t0 + hw : t0;
          const uint4 kb = *reinterpret_cast<const uint4 *>(keys + t * kDim + c8);
          const uint4 qb = *reinterpret_cast<const uint4 *>(queries + t * kDim + c8);
          const uint4 gb = *reinterpret_cast<const uint4 *>(gates(t) + c8);
          const float4 ka = bf16x4(make_uint2(kb.x, kb.y)), kc = bf16x4(make_uint2(kb.z, kb.w));
          const float4 qa = bf16x4(make_uint2(qb.x, qb.y)), qc = bf16x4(make_uint2(qb.z, qb.w));
          float kk = dot4(ka, ka) + dot4(kc, kc), qq = dot4(qa, qa) + dot4(qc, qc);
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) {
            kk += __shfl_xor_sync(0xffffffffu, kk, o);
            qq += __shfl_xor_sync(0xffffffffu, qq, o);
          }
          __syncwarp();  // the row's gates are read
          if (t0 + hw < n) {
            uint2 g4 = make_uint2(gb.x, gb.y);
#pragma unroll 1
            for (int e = 0; e < 8; e += 4) {
              sts4(decay + t * kDim + c8 + e, decay4(a, bf16x4(g4), lds4(dts() + c8 + e), p.lower_bound));
              g4 = make_uint2(gb.z, gb.w);
            }
            if ((lane & 15) == 0) {
              norms[t] = rsqrtf(kk + kNormEps);
              norms[NC + t] = rsqrtf(qq + kNormEps) * p.q_scale;
            }
          }
        }
      }
      named_bar(1, kThreads);
      if (L::kTHelps) arrive(&bars->n_full);
      make_xy(it, keys, queries, nw, done);
      if (L::kRawBufs > 0 && lane == 0) mbar_arrive(&bars->raw_free[done % L::kCopies]);
      ++done;
      more = settle(it.next(lane));  // (its barrier: the nodes are read)
    }
    if (L::kRawBufs == 0) cp_async_wait_all();
    ok = it.ok;
  }
  if (!ok && lane == 0) report(mp.status, KDA_ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int NC, bool BF16>
int launch(const TreeVerifyParams &p, int sms, cudaStream_t stream) {
  using L = TreeMma<NC, BF16>;
  const auto kernel = kda_tree_mma_kernel<NC, BF16>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kBytes) !=
      cudaSuccess)
    return KDA_ERR_CUDA;
  TreeTokenMaps maps{};
  if (L::kRawBufs > 0 && p.maps.n_tokens > 0) {
    const auto encode = tensor_map_encoder();
    if (encode == nullptr) return KDA_ERR_CUDA;
    const cuuint64_t dims[3] = {(cuuint64_t)kDim, (cuuint64_t)p.H, (cuuint64_t)p.maps.n_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)kDim * 2, (cuuint64_t)p.H * kDim * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kDim, 1, (cuuint32_t)kBoxTokens};
    const cuuint32_t estride[3] = {1, 1, 1};
    const uint16_t *const src[4] = {p.k, p.q, p.g, p.v};
    for (int i = 0; i < 4; ++i)
      if (encode(&maps.of[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(src[i]),
                 dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return KDA_ERR_CUDA;
  }
  const int items = p.maps.B * p.H;
  kernel<<<items < sms ? items : sms, L::kThreads, L::kBytes, stream>>>(p, maps, items);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

int launch_tree_mma(const TreeVerifyParams &p, bool bf16, int sms, cudaStream_t stream) {
  if (p.maps.Q <= 32) return bf16 ? launch<32, true>(p, sms, stream) : launch<32, false>(p, sms, stream);
  return bf16 ? launch<64, true>(p, sms, stream) : launch<64, false>(p, sms, stream);
}

}  // namespace kda

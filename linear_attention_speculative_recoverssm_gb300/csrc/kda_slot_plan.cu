// kda_slot_plan: packed offsets, block table entries and slot maps from the
// requests' lengths (the align mode's bookkeeping).  Integer work: per
// request a few divisions, and two prefix sums over the requests (tokens,
// and free slots taken).  One cluster of up to 16 CTAs: CTA c owns a
// contiguous part of the requests and sums it; the CTAs exchange their sums
// through distributed shared memory; then each places its requests behind
// what comes before them.  Latency is all there is: three loads that depend
// on one another, two barriers, the scans by shuffles.  48 requests 7 us;
// 8192 requests 14.4 us, most of it the 4 MB of table entries that the prompts
// pass over.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "../../include/kda_recoverssm.h"
#include "kda_device.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

// A thread a request, and many CTAs before large ones, as every SM of the
// cluster stores for itself: 8192 requests take 14.4 us by 16 CTAs of 512,
// 16.7 by 8 of 1024, 23 by 16 of 256 (two requests a thread, worked out twice).
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxCtas = 16;   // the largest cluster
constexpr int kPlanPortable = 8;   // the largest that needs no permission

struct PlanParams {
  const int32_t *computed, *fresh;  // [B]
  int32_t *table;                   // [B, max_blocks]
  long long row_stride;
  int max_blocks;
  const int32_t *free_slots;  // [n_free]
  int n_free;
  const int32_t *free_head;
  int32_t *free_next;
  int32_t *qsl, *sources, *destinations, *bnd_slots, *bnd_lens;
  int B, block_size, null_slot;
  int32_t *status;
};

// What one request needs.  The state after p > 0 tokens is held by block
// (p - 1) / block_size of its row.
struct PlanRequest {
  int tokens;        // of the packed activations, also where nothing else is
  bool live;         // it has tokens and valid lengths
  bool crosses;      // a block ends strictly inside its new tokens' range
  bool new_last, new_bnd;  // a free slot for the last block / the one before
  int cur, last;     // blocks of the state it goes on from (-1: none) and ends in
  int bnd_len;
  int src;           // slot it goes on from, or null
};

__device__ __forceinline__ PlanRequest no_request() {
  PlanRequest r;
  r.tokens = r.bnd_len = r.src = 0;
  r.live = r.crosses = r.new_last = r.new_bnd = false;
  r.cur = r.last = -1;
  return r;
}

__device__ __forceinline__ PlanRequest plan_request(const PlanParams &p, int b, bool say) {
  PlanRequest r = no_request();
  const int c = p.computed[b], n = p.fresh[b];
  r.tokens = n > 0 ? n : 0;
  r.src = p.null_slot;
  const long long end = (long long)c + n;
  if (c < 0 || n < 0 || end > (long long)p.max_blocks * p.block_size || end > 0x7fffffffLL) {
    if (say) report(p.status, KDA_ERR_ARG);
    return r;
  }
  if (n == 0) return r;
  r.cur = c > 0 ? (c - 1) / p.block_size : -1;
  r.last = (int)((end - 1) / p.block_size);
  if (c > 0) {
    r.src = p.table[b * p.row_stride + r.cur];
    if (r.src <= p.null_slot) {  // the state it should go on from is not held
      if (say) report(p.status, KDA_ERR_ARG);
      r.src = p.null_slot;
      return r;
    }
  }
  r.live = true;
  const long long edge = (long long)r.last * p.block_size;
  r.crosses = edge > c;
  r.bnd_len = r.crosses ? (int)(edge - c) : 0;
  r.new_last = r.last != r.cur;
  r.new_bnd = r.crosses && r.last - 1 != r.cur;
  return r;
}

// The two halves of a cluster's barrier (every thread of every CTA does both).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Tokens and free slots, counted.
struct Pair {
  long long tokens;
  int slots;
};

// The sums over the lanes up to and with this one.
__device__ __forceinline__ Pair warp_scan(Pair x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, x.tokens, o);
    const int s = __shfl_up_sync(0xffffffffu, x.slots, o);
    if (lane >= o) {
      x.tokens += t;
      x.slots += s;
    }
  }
  return x;
}

// Sum over the CTA's threads, and over the threads before this one.
__device__ __forceinline__ Pair block_scan(Pair mine, Pair *warp_sums, Pair &total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Pair inc = warp_scan(mine);
  __syncthreads();  // the sums of an earlier scan have been read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  // each warp scans the warps' sums for itself (there are at most 32)
  const Pair sums = warp_scan(lane < (blockDim.x >> 5) ? warp_sums[lane] : Pair{0, 0});
  total.tokens = __shfl_sync(0xffffffffu, sums.tokens, 31);
  total.slots = __shfl_sync(0xffffffffu, sums.slots, 31);
  const long long t = __shfl_sync(0xffffffffu, sums.tokens, (warp + 31) & 31);
  const int s = __shfl_sync(0xffffffffu, sums.slots, (warp + 31) & 31);
  return Pair{(warp ? t : 0) + inc.tokens - mine.tokens, (warp ? s : 0) + inc.slots - mine.slots};
}

__global__ void __launch_bounds__(kPlanThreads) kda_slot_plan_kernel(const PlanParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ Pair warp_sums[32];
  __shared__ Pair cta_sum;
  const int ctas = gridDim.x, rank = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int b_begin = (int)((long long)p.B * rank / ctas);
  const int b_end = (int)((long long)p.B * (rank + 1) / ctas);
  const int head = *p.free_head;
  // this CTA's requests, summed; where each thread has one at most, it is
  // worked out here and kept
  const bool once = b_end - b_begin <= (int)blockDim.x;
  PlanRequest r = no_request();
  Pair sum{0, 0}, total;
  for (int b = b_begin + threadIdx.x; b < b_end; b += blockDim.x) {
    r = plan_request(p, b, once);
    sum.tokens += r.tokens;
    sum.slots += r.new_last + r.new_bnd;
  }
  const Pair before = block_scan(sum, warp_sums, total);
  Pair base{0, 0}, all{0, 0};
  if (ctas == 1) {
    all = total;
    __syncthreads();  // free_head has been read: free_next may be its place
  } else {
    if (threadIdx.x == 0) cta_sum = total;
    cluster.sync();  // every CTA's sum is there, and every CTA has read free_head
    const Pair sums =
        warp_scan(lane < ctas ? *cluster.map_shared_rank(&cta_sum, lane) : Pair{0, 0});
    all.tokens = __shfl_sync(0xffffffffu, sums.tokens, 31);
    all.slots = __shfl_sync(0xffffffffu, sums.slots, 31);
    const long long t = __shfl_sync(0xffffffffu, sums.tokens, (rank + 31) & 31);
    const int s = __shfl_sync(0xffffffffu, sums.slots, (rank + 31) & 31);
    if (rank > 0) base = Pair{t, s};
    cluster_arrive();  // waited for at the end: no CTA leaves while its sum is read
  }
  const bool head_ok = head >= 0 && head <= p.n_free;
  const int avail = head_ok ? p.n_free - head : 0;
  if (rank == ctas - 1 && threadIdx.x == 0) {
    if (!head_ok || all.tokens > 0x7fffffffLL) report(p.status, KDA_ERR_ARG);
    p.qsl[p.B] = all.tokens > 0x7fffffffLL ? 0x7fffffff : (int)all.tokens;
    if (all.slots <= avail) *p.free_next = head + all.slots;
  }
  for (int b0 = b_begin; b0 < b_end; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    Pair at = before;
    if (!once) {
      r = b < b_end ? plan_request(p, b, true) : no_request();
      Pair tile;
      at = block_scan(Pair{r.tokens, r.new_last + r.new_bnd}, warp_sums, tile);
      at.tokens += base.tokens;
      at.slots += base.slots;
      base.tokens += tile.tokens;
      base.slots += tile.slots;
    } else {
      at.tokens += base.tokens;
      at.slots += base.slots;
    }
    const int need = r.new_last + r.new_bnd;
    // A request that the free list has no slots for is not served, and so
    // neither is any behind it that needs one (their places in the list lie
    // further on): the first one's place is how far the list was used.
    const bool served = r.live && (need == 0 || at.slots + need <= avail);
    if (r.live && !served) {
      report(p.status, KDA_ERR_SLOTS);
      if (at.slots <= avail) *p.free_next = head + at.slots;
    }
    if (b < b_end) {
      int dst = p.null_slot, bnd = p.null_slot, len = 0;
      if (served) {
        int32_t *row = p.table + b * p.row_stride;
        int take = head + at.slots;
        if (r.crosses) {
          bnd = r.new_bnd ? p.free_slots[take++] : r.src;
          if (r.new_bnd) row[r.last - 1] = bnd;
          len = r.bnd_len;
        }
        dst = r.new_last ? p.free_slots[take] : r.src;
        if (r.new_last) row[r.last] = dst;
      }
      p.sources[b] = served ? r.src : p.null_slot;
      p.destinations[b] = dst;
      p.bnd_slots[b] = bnd;
      p.bnd_lens[b] = len;
      p.qsl[b] = at.tokens > 0x7fffffffLL ? 0x7fffffff : (int)at.tokens;
    }
    // the blocks that a prompt passes over hold no state: a warp marks the
    // rows of its 32 requests one after the other
    const int skip_from = served ? r.cur + 1 : 0, skip_to = served ? r.last - 1 : 0;
    uint32_t rows = __ballot_sync(0xffffffffu, skip_from < skip_to);
    while (rows != 0) {
      const int l = __ffs(rows) - 1;
      rows &= rows - 1;
      const int from = __shfl_sync(0xffffffffu, skip_from, l);
      const int to = __shfl_sync(0xffffffffu, skip_to, l);
      int32_t *row = p.table + (long long)(b - lane + l) * p.row_stride;
      for (int j = from + lane; j < to; j += 32) row[j] = p.null_slot;
    }
  }
  if (ctas > 1) cluster_wait();
}

}  // namespace
}  // namespace kda

extern "C" int kda_slot_plan(const int32_t *computed_lens, const int32_t *new_lens,
                             int32_t *block_table, int64_t table_row_stride, int max_blocks,
                             const int32_t *free_slots, int n_free, const int32_t *free_head,
                             int32_t *free_next, int32_t *query_start_loc, int32_t *sources,
                             int32_t *destinations, int32_t *boundaries, int32_t *boundary_lens,
                             int B, int block_size, int null_slot, int32_t *status,
                             void *stream) {
  if (B < 0 || B > KDA_PLAN_MAX_REQUESTS || max_blocks < 1 || table_row_stride < max_blocks ||
      n_free < 0 || block_size < 1 || null_slot < -1)
    return KDA_ERR_ARG;
  if (!free_head || !free_next || !query_start_loc) return KDA_ERR_ARG;
  if (B > 0 && (!computed_lens || !new_lens || !block_table || !sources || !destinations ||
                !boundaries || !boundary_lens || (n_free > 0 && !free_slots)))
    return KDA_ERR_ARG;
  kda::PlanParams p;
  p.computed = computed_lens;
  p.fresh = new_lens;
  p.table = block_table;
  p.row_stride = table_row_stride;
  p.max_blocks = max_blocks;
  p.free_slots = free_slots;
  p.n_free = n_free;
  p.free_head = free_head;
  p.free_next = free_next;
  p.qsl = query_start_loc;
  p.sources = sources;
  p.destinations = destinations;
  p.bnd_slots = boundaries;
  p.bnd_lens = boundary_lens;
  p.B = B;
  p.block_size = block_size;
  p.null_slot = null_slot;
  p.status = status;
  int ctas = B < 1 ? 1 : (B - 1) / kda::kPlanThreads + 1;
  if (ctas > kda::kPlanMaxCtas) ctas = kda::kPlanMaxCtas;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(B >= kda::kPlanThreads ? kda::kPlanThreads
                                             : (B < 1 ? 32 : (B + 31) / 32 * 32));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (ctas > kda::kPlanPortable &&
      cudaFuncSetAttribute(kda::kda_slot_plan_kernel,
                           cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return KDA_ERR_CUDA;
  if (cudaLaunchKernelEx(&cfg, kda::kda_slot_plan_kernel, p) != cudaSuccess) return KDA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

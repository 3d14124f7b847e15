// adapter_plan.cu -- groups a step's tokens by adapter.
//
// Sequences are ranked by (adapter, index): rank = number of sequences that come before, counted directly (at most 1024 of them).
// Sums over the ranked sequences then give each its place in the order, and each group of equal adapters its tiles; the tokens'
// places and the tiles are found by binary search.  Every block counts for itself and writes its share of the tokens and tiles.
// Bound: latency of a few dependent rounds; once a step.  1 token 4.4 us, 64 sequences 5.8, 9 of 4493 tokens 7.3, 1024 sequences 35 (each
// thread's count of the 1024, and the scans); with one adapter_add behind it 9.5, 32, 92.
#include "adapter_plan.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"

namespace trellis {
namespace {

constexpr int kThreads = 1024;
constexpr int kPerBlock = 4096;  // tokens of a block
static_assert(kAdapterMaxBatch <= kThreads, "a thread per sequence");

// Sum (or maximum) over the threads up to this one.
template <bool Max>
__device__ __forceinline__ int scan(int v, int* warps) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v = Max ? max(v, u) : v + u;
  }
  __syncthreads();
  if (lane == 31) warps[w] = v;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < w; ++i) before = Max ? max(before, warps[i]) : before + warps[i];
  return Max ? max(v, before) : v + before;
}

__device__ __forceinline__ int total(int v, int* warps) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xFFFFFFFFu, warps[threadIdx.x & 31]);
}

// The last of at[0 .. n) (ascending, at[0] = 0) that is at most x.
__device__ __forceinline__ int last_upto(const int* at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const int32_t* __restrict__ adapter, const int32_t* __restrict__ q_start,
                                                        int batch, int n, int clusters, void* plan) {
  pdl_enter();
  __shared__ int warps[kThreads / 32];
  __shared__ int ids[kThreads];                      // by sequence
  __shared__ int place[kThreads + 1], start[kThreads];  // by rank: first place in the order, first token
  __shared__ int group_first[kThreads + 1], group_tiles[kThreads + 1], group_id[kThreads];
  __shared__ int groups_of_all;
  const int t = threadIdx.x;
  // starts, clamped and ascending
  int from = 0, count = 0;
  {
    int a = t < batch ? __ldcg(q_start + t) : 0;
    a = scan<true>(min(max(a, 0), n), warps);
    place[t] = a;
    __syncthreads();
    if (t < batch) {
      int z = t + 1 < batch ? place[t + 1] : max(min(__ldcg(q_start + batch), n), a);
      from = a;
      count = z - a;
    }
  }
  const int id = t < batch ? __ldcg(adapter + t) : 0;
  ids[t] = id < 0 ? INT32_MAX : id;
  __syncthreads();
  int rank = 0;
  if (t < batch)
    for (int b = 0; b < batch; ++b) rank += ids[b] < ids[t] || (ids[b] == ids[t] && b < t);
  __syncthreads();
  if (t < batch) {
    start[rank] = from;
    group_id[rank] = ids[t];
    group_tiles[rank] = count;
  }
  __syncthreads();
  // from here on a thread is a rank
  const int mine = t < batch ? group_tiles[t] : 0, my_id = t < batch ? group_id[t] : 0;
  const bool head = t < batch && (t == 0 || group_id[t - 1] != my_id);
  const int upto = scan<false>(mine, warps);
  const int group = scan<false>(head ? 1 : 0, warps) - 1;
  if (t < batch) place[t] = upto - mine;
  if (t == batch - 1) place[batch] = upto;
  __syncthreads();
  if (head) {
    group_first[group] = place[t];
    group_id[group] = my_id;  // group <= t, and every thread has read its own
  }
  if (t == batch - 1) {
    groups_of_all = group + 1;
    group_first[group + 1] = place[batch];
  }
  __syncthreads();
  const int groups = groups_of_all, tokens = place[batch];
  const int size = t < groups ? group_first[t + 1] - group_first[t] : 0;
  // The longest tile that needs no more rounds than tiles of 64 do: they are taken by `clusters` at a time, and a last round of few
  // tiles would take as long as a full one.
  int tile = kAdapterTile;
  {
    const auto count_of = [&](int most) { return total((size + most - 1) / most, warps); };
    const int full = count_of(kAdapterTile), rounds = (full + clusters - 1) / clusters;
    if (full >= clusters) {
      int lo = kAdapterLeast, hi = kAdapterTile;  // hi fits
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (count_of(mid) <= rounds * clusters) hi = mid;
        else lo = mid + 1;
      }
      tile = hi;
    }
  }
  const int tiles = (size + tile - 1) / tile;
  const int tiles_upto = scan<false>(tiles, warps);
  if (t < groups) group_tiles[t] = tiles_upto - tiles;
  if (t == groups - 1) group_tiles[groups] = tiles_upto;
  __syncthreads();
  const int all = group_tiles[groups];
  const bool some_without = group_id[groups - 1] == INT32_MAX;
  if (blockIdx.x == 0 && t == 0) {
    AdapterPlanHeader* h = static_cast<AdapterPlanHeader*>(plan);
    h->tiles = all;
    h->with_adapter = some_without ? group_tiles[groups - 1] : all;
    h->reserved[0] = h->reserved[1] = 0;
  }
  int4* out_tiles = const_cast<int4*>(adapter_tiles(plan));
  for (int i = blockIdx.x * kThreads + t; i < all; i += gridDim.x * kThreads) {
    // the tile's group: groups may be empty, so the last that begins at or before i and has tiles
    const int g = last_upto(group_tiles, groups, i);
    const int gsize = group_first[g + 1] - group_first[g], gtiles = group_tiles[g + 1] - group_tiles[g], j = i - group_tiles[g];
    // tiles of a group are as long as one another, to within a token
    const int lo = (int)((int64_t)j * gsize / gtiles), hi = (int)((int64_t)(j + 1) * gsize / gtiles);
    out_tiles[i] = make_int4(group_id[g] == INT32_MAX ? -1 : group_id[g], group_first[g] + lo, hi - lo, 0);
  }
  int32_t* order = const_cast<int32_t*>(adapter_order(plan, batch, n));
  for (int i = blockIdx.x * kThreads + t; i < tokens; i += gridDim.x * kThreads) {
    const int r = last_upto(place, batch, i);
    order[i] = start[r] + i - place[r];
  }
}

}  // namespace

size_t adapter_plan_bytes(int batch, int n) {
  const size_t b = sizeof(AdapterPlanHeader) + (size_t)adapter_max_tiles(batch, n) * sizeof(int4) + (size_t)n * 4;
  return (b + 15) & ~(size_t)15;
}

cudaError_t launch_adapter_plan(const int32_t* adapter, const int32_t* q_start, int batch, int n, void* plan, cudaStream_t st) {
  const int blocks = (n + kPerBlock - 1) / kPerBlock;
  const int most = device_sm_count(), fit = adapter_clusters(), clusters = fit < 1 ? 1 : fit < kAdapterMaxClusters ? fit : kAdapterMaxClusters;
  return launch_pdl(plan_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, st, adapter, q_start, batch, n,
                    clusters, plan);
}

}  // namespace trellis

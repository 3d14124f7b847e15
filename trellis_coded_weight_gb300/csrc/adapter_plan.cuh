// adapter_plan.cuh -- a step's tokens by adapter, as adapter_plan.cu leaves them and adapters.cu reads them.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace trellis {

constexpr int kAdapterTile = 64;  // most tokens of a tile

// A plan: the header, the tiles, the tokens by adapter.
//   tile (adapter, first, tokens, 0): `tokens` tokens of one adapter, from place `first` of the order on.  Tiles come by ascending
//   adapter, those of tokens without one (adapter -1) last.
struct AdapterPlanHeader {
  int tiles, with_adapter;  // tiles in all, and of tokens that have an adapter
  int reserved[2];
};
constexpr int kAdapterLeast = kAdapterTile / 2;  // tiles are not cut shorter than this to fill a round
constexpr int kAdapterMaxClusters = 256;
__host__ __device__ constexpr int64_t adapter_max_tiles(int batch, int n) {
  // every group of tokens has at most one tile that is not full, a group needs a sequence and a token, and a round that is
  // filled up has no more tiles than clusters
  return n / kAdapterTile + (batch < n ? batch : n) + (n >= kAdapterLeast ? kAdapterMaxClusters : 0);
}
int adapter_clusters();  // that add to a projection's output at once on the current device (adapters.cu); 0: none
__host__ __device__ __forceinline__ const int4* adapter_tiles(const void* plan) {
  return reinterpret_cast<const int4*>(static_cast<const char*>(plan) + sizeof(AdapterPlanHeader));
}
__host__ __device__ __forceinline__ const int32_t* adapter_order(const void* plan, int batch, int n) {
  return reinterpret_cast<const int32_t*>(adapter_tiles(plan) + adapter_max_tiles(batch, n));
}

}  // namespace trellis

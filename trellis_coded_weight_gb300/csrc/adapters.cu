// adapters.cu -- adds low-rank adapters to a projection's output (plan: adapter_plan.cuh).
//
//   h = A x  (fp32),  out = bf16(y + scale B h)
// A warp per row of A, then a thread per output.
#include "adapter_plan.cuh"
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"

namespace trellis {
namespace {

constexpr int kThreads = 256;

struct AddParams {
  const uint16_t *x, *y;
  uint16_t* out;
  int64_t x_stride, y_stride, out_stride;
  trellis_adapters_t ad;
  const void* plan;
  int batch, n;
};

__global__ void __launch_bounds__(kThreads) add_kernel(const AddParams p) {
  pdl_enter();
  __shared__ float h[kAdapterMaxRank];
  const AdapterPlanHeader* head = static_cast<const AdapterPlanHeader*>(p.plan);
  const int32_t* order = adapter_order(p.plan, p.batch, p.n);
  const int tiles = head->tiles, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int4 tile = adapter_tiles(p.plan)[t];
    const bool has = tile.x >= 0 && tile.x < p.ad.count;
    int rank = has ? p.ad.ranks ? p.ad.ranks[tile.x] : p.ad.max_rank : 0;
    rank = rank < 0 ? 0 : rank > p.ad.max_rank ? p.ad.max_rank : rank;
    const float scale = has && p.ad.scales ? p.ad.scales[tile.x] : 1.f;
    for (int i = blockIdx.y; i < tile.z; i += gridDim.y) {
      const int64_t token = order[tile.y + i];
      const uint16_t *x = p.x + token * p.x_stride, *y = p.y + token * p.y_stride;
      uint16_t* out = p.out + token * p.out_stride;
      for (int r = warp; r < rank; r += kThreads / 32) {
        const uint16_t* a = p.ad.a + ((int64_t)tile.x * p.ad.max_rank + r) * p.ad.in;
        float s = 0.f;
        for (int k = lane; k < p.ad.in; k += 32) s = fmaf(bf16_to_f32(a[k]), bf16_to_f32(x[k]), s);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) h[r] = s;
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.ad.out; c += kThreads) {
        if (rank == 0) {
          out[c] = y[c];
          continue;
        }
        const uint16_t* b = p.ad.b + ((int64_t)tile.x * p.ad.out + c) * p.ad.max_rank;
        float s = 0.f;
        for (int r = 0; r < rank; ++r) s = fmaf(bf16_to_f32(b[r]), h[r], s);
        out[c] = f32_to_bf16_rn(fmaf(scale, s, bf16_to_f32(y[c])));
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_adapter_add(const uint16_t* x, int64_t x_stride, const uint16_t* y, int64_t y_stride, uint16_t* out,
                               int64_t out_stride, const trellis_adapters_t& ad, const void* plan, int batch, int n,
                               cudaStream_t st) {
  const AddParams p{x, y, out, x_stride, y_stride, out_stride, ad, plan, batch, n};
  const int64_t tiles = adapter_max_tiles(batch, n);
  return launch_pdl(add_kernel, dim3((unsigned)(tiles < 1024 ? tiles : 1024), kAdapterTile), dim3(kThreads), 0, st, p);
}

}  // namespace trellis

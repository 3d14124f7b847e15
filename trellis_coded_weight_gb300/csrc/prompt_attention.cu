// prompt_attention.cu -- causal attention of whole prompts over the paged cache.
//
// A warp per query row goes over the keys that its token sees once, with a running maximum and sum:
//   m' = max(m, s),  l' = l 2^(m - m') + 2^(s - m'),  o' = o 2^(m - m') + 2^(s - m') v
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"
#include "tree_sched.cuh"

namespace trellis {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float e4m3_to_f32(uint8_t v) {
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"((uint32_t)v));
  return f16_to_f32((uint16_t)h);
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) prompt_kernel(const TreeParams p) {
  pdl_enter();
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float kLn2 = 0.693147180559945309f;
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const TreeSeq s = tree_seq(p, b);
    const int64_t rows = (int64_t)s.count * p.hq;
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + warp; r < rows; r += (int64_t)gridDim.x * (kThreads / 32)) {
      const int tok = (int)(r / p.hq), h = (int)(r % p.hq), kvh = h / p.group;
      const uint16_t* q = p.q + (int64_t)(s.start + tok) * p.q_stride + (int64_t)h * D;
      const float ks = p.scales ? p.scales[kvh] : 1.f, vs = p.scales ? p.scales[p.hkv + kvh] : 1.f;
      float x[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = bf16_to_f32(q[lane + 32 * e]);
      for (int pos = 0; pos <= s.prefix + tok; ++pos) {
        int page = p.table[(int64_t)b * p.width + (pos >> p.page_shift)];
        page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
        const int64_t krow = (((int64_t)(page * 2) * p.hkv + kvh) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        const int64_t vrow = krow + ((int64_t)p.hkv << p.page_shift);
        const auto at = [&](int64_t row, int e) {
          const int64_t i = row * D + lane + 32 * e;
          return F8 ? e4m3_to_f32(static_cast<const uint8_t*>(p.pool)[i]) : bf16_to_f32(static_cast<const uint16_t*>(p.pool)[i]);
        };
        float sc = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) sc = fmaf(x[e], at(krow, e), sc);
#pragma unroll
        for (int w = 16; w; w >>= 1) sc += __shfl_xor_sync(0xFFFFFFFFu, sc, w);
        sc *= p.scale_log2 * ks;
        if (sc == -INFINITY) continue;
        const float to = fmaxf(m, sc), a = m == -INFINITY ? 0.f : exp2f(m - to), w = exp2f(sc - to);
        l = l * a + w;
        m = to;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, at(vrow, e), o[e] * a);
      }
      const float f = l == 0.f ? 0.f : vs / l;
      uint16_t* out = p.out + (int64_t)(s.start + tok) * p.out_stride + (int64_t)h * D;
#pragma unroll
      for (int e = 0; e < E; ++e) out[lane + 32 * e] = f32_to_bf16_rn(o[e] * f);
      if (p.lse && lane == 0) p.lse[(int64_t)(s.start + tok) * p.hq + h] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
    }
  }
}

template <int D>
cudaError_t launch_d(const TreeParams& p, bool f8, cudaStream_t st) {
  const dim3 grid(152 * 4, p.batch < 64 ? p.batch : 64);
  return f8 ? launch_pdl(prompt_kernel<D, true>, grid, dim3(kThreads), 0, st, p)
            : launch_pdl(prompt_kernel<D, false>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace

size_t prompt_workspace_bytes(const trellis_cache_t& c, int q_heads) {
  (void)c; (void)q_heads;
  return 1024;
}

cudaError_t launch_prompt_attention(const uint16_t* q, int64_t q_stride, const trellis_cache_t& c, int layer,
                                    const trellis_drafts_t& d, int q_heads, float scale, uint16_t* out,
                                    int64_t out_stride, float* lse, void* workspace, cudaStream_t st) {
  (void)workspace;
  TreeParams p{};
  p.q = q; p.out = out; p.lse = lse;
  p.table = d.table; p.prefix = d.prefix; p.q_start = d.q_start;
  p.scales = c.scales ? c.scales + (int64_t)layer * 2 * c.heads : nullptr;
  p.q_stride = q_stride; p.out_stride = out_stride;
  p.pages = c.pages;
  p.batch = d.batch; p.width = d.width; p.n = d.n; p.max_tokens = d.max_tokens;
  p.hq = q_heads; p.hkv = c.heads; p.group = q_heads / c.heads;
  p.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  p.scale_log2 = scale * kLog2e;
  p.pool = static_cast<uint8_t*>(c.pool) + (int64_t)layer * c.pages * cache_page_bytes(c);
  const bool f8 = c.dtype == TRELLIS_E4M3;
  return c.head_dim == 64 ? launch_d<64>(p, f8, st) : c.head_dim == 128 ? launch_d<128>(p, f8, st) : launch_d<256>(p, f8, st);
}

}  // namespace trellis

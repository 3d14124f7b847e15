// tree_join.cu -- joins the parts of tree attention items that several blocks have shared (tree_sched.cuh).
//
// With m_j, l_j, o_j of the parts:  m = max m_j,  l = sum 2^(m_j - m) l_j,  o = sum 2^(m_j - m) o_j;
// out = o / l,  lse = ln2 (m + log2 l).
// A thread has four columns of a row and goes through the parts in their order, eight at a time, with its own running
// maximum; where an item has many parts four threads share them and join at the end.  The blocks of a shared item (one
// per first block of an item and share of its rows) spread over the GPU.  Bound: latency of the launch and of one or
// two rounds of loads; the parts are still in L2.
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "tree_sched.cuh"

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;       // parts whose loads are in flight
constexpr int kManyParts = 16;  // from here on four threads share them
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct State {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void scale_to(State& s, float m) {
  const float a = s.m == -INFINITY ? 0.f : ex2(s.m - m);
  s.l *= a;
  s.o = make_float4(s.o.x * a, s.o.y * a, s.o.z * a, s.o.w * a);
  s.m = m;
}

template <int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const TreeParams p, int prows, float lift) {
  pdl_enter();
  __shared__ State sh[kThreads];
  const int4 item = __ldcg(p.items + blockIdx.x);
  if (item.x < 0) return;
  const TreeSeq seq = tree_seq(p, item.x);
  const int head = item.y, row0 = item.z * prows, first = blockIdx.x, parts = item.w - first + 1;
  const int rows = min(prows, seq.count * p.group - row0);
  const int64_t part_floats = tree_part_floats(prows, D);
  constexpr int LPR = D / 4;  // threads of a row
  const int sharers = parts >= kManyParts ? 4 : 1;
  const int elems = kThreads / sharers, step = elems / LPR;  // rows at a time
  const int mine = threadIdx.x / elems, e = threadIdx.x % elems, row_in = e % step, col = e / step * 4;
  const float vs = p.scales ? __ldg(p.scales + p.hkv + head) : 1.f;
  for (int r0 = blockIdx.y * step; r0 < rows; r0 += gridDim.y * step) {
    const int r = r0 + row_in;
    State s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (r < rows)
      for (int j0 = mine; j0 < parts; j0 += sharers * kBatch) {
        float m[kBatch], l[kBatch];
        float4 o[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int j = j0 + b * sharers;
          m[b] = -INFINITY;
          l[b] = 0.f;
          o[b] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (j < parts) {
            const float* part = p.part + (int64_t)tree_slot(first + j, j == 0) * part_floats;
            m[b] = __ldcg(part + (int64_t)prows * D + r);
            l[b] = __ldcg(part + (int64_t)prows * D + prows + r);
            o[b] = __ldcg(reinterpret_cast<const float4*>(part + ((int64_t)(col / 4) * prows + r) * 4));
          }
        }
        float mx = s.m;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) mx = fmaxf(mx, m[b]);
        if (mx > s.m) scale_to(s, mx);
        const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const float w = ex2(m[b] - base);
          s.l += w * l[b];
          s.o.x += w * o[b].x;
          s.o.y += w * o[b].y;
          s.o.z += w * o[b].z;
          s.o.w += w * o[b].w;
        }
      }
    if (sharers > 1) {
      __syncthreads();
      sh[threadIdx.x] = s;
      __syncthreads();
      if (mine == 0)
        for (int k = 1; k < 4; ++k) {
          State t = sh[threadIdx.x + k * elems];
          const float mx = fmaxf(s.m, t.m);
          if (mx > -INFINITY) {
            scale_to(s, mx);
            scale_to(t, mx);
          }
          s.l += t.l;
          s.o = make_float4(s.o.x + t.o.x, s.o.y + t.o.y, s.o.z + t.o.z, s.o.w + t.o.w);
        }
    }
    if (r < rows && mine == 0) {
      const float f = s.l == 0.f ? 0.f : vs / s.l;
      const int d = tree_draft(p, row0 + r), hh = row0 + r - d * p.group;
      *reinterpret_cast<uint2*>(p.out + (seq.start + d) * p.out_stride + (int64_t)(head * p.group + hh) * D + col) =
          make_uint2(pack_bf16x2(s.o.x * f, s.o.y * f), pack_bf16x2(s.o.z * f, s.o.w * f));
      if (p.lse && col == 0)
        p.lse[(int64_t)(seq.start + d) * p.hq + head * p.group + hh] = s.l == 0.f ? -INFINITY : kLn2 * (s.m + (log2f(s.l) - lift));
    }
  }
}

}  // namespace

cudaError_t launch_tree_join(const TreeParams& p, int dim, int rows, float lift, int ctas, cudaStream_t st) {
  const int most = p.max_tokens * p.group < rows ? p.max_tokens * p.group : rows;
  // shares of an item's rows: as small as a block's rows with many parts, at most 32
  const int least = kThreads / 4 / (dim / 4) < 1 ? 1 : kThreads / 4 / (dim / 4);
  int y = (most + least - 1) / least;
  if (y > 32) y = 32;
  const dim3 grid((unsigned)ctas, (unsigned)y), block(kThreads);
  if (dim == 64) return launch_pdl(join_kernel<64>, grid, block, 0, st, p, rows, lift);
  if (dim == 128) return launch_pdl(join_kernel<128>, grid, block, 0, st, p, rows, lift);
  return launch_pdl(join_kernel<256>, grid, block, 0, st, p, rows, lift);
}

}  // namespace trellis

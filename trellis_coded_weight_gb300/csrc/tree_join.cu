// tree_join.cu -- joins the parts of tree attention items that several blocks have shared (tree_sched.cuh).
//
// With m_j, l_j, o_j of the parts:  m = max m_j,  l = sum 2^(m_j - m) l_j,  o = sum 2^(m_j - m) o_j;
// out = o / l,  lse = ln2 (m + log2 l).
// A thread has four columns of a row and loads eight parts at a time; where an item has more, up to eight threads share them
// and join at the end.  Eight rows go side by side (128 contiguous bytes of a part).  Where items have
// many rows every block counts the units of work for itself, from the table that the attention kernel has left, and takes its share.  19 parts of 256 rows by 8 heads of 128:
// 6.5 us; a grid of a block per possible item and rows, most of which had none, took 11, and warps that each went through the
// table by themselves 9.  Bound: latency of the launch and of two or three rounds of loads; the parts are still in L2.
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "tree_sched.cuh"

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int kPerSM = 3;
constexpr int kBatch = 8;   // parts whose loads are in flight
constexpr int kRows = 8;    // rows of a unit
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

// direct: block (x, y) takes the item that attention block x was the first to share, and of its units y, y + gridDim.y, ..
template <int D, bool Direct>
__global__ void __launch_bounds__(kThreads, kPerSM) join_kernel(const TreeParams p, int prows, int ctas, float lift) {
  pdl_enter();
  __shared__ State sh[kThreads];
  __shared__ int sums[kThreads / 32];
  __shared__ int4 s_item;
  __shared__ int2 s_at;
  constexpr int LPR = D / 4;  // fours of columns of a row
  const int64_t part_floats = tree_part_floats(prows, D);
  const int tid = threadIdx.x, lane = tid & 31;
  // of a unit's threads as many share a column's parts as the item says, and two at least where a row has fewer columns than
  // there would be threads
  const auto sharers_of = [](int w) { return D == 64 && tree_item_shared(w) == 0 ? 2 : 1 << tree_item_shared(w); };
  const auto units_of = [&](int w) { return (tree_item_rows(w) + kRows - 1) / kRows * (LPR * kRows * sharers_of(w) / kThreads); };
  const auto join = [&](const int4 item, int first, int at) {  // unit `at` of an item whose first part is block `first`'s
    const int head = item.y, row0 = item.z, rows = tree_item_rows(item.w), parts = tree_item_last(item.w) - first + 1;
    const int sharers = sharers_of(item.w), elems = kThreads / sharers, groups = LPR * kRows / elems;  // of columns
    const int mine = tid / elems, e = tid % elems, r = at / groups * kRows + e % kRows;
    const int col = (at % groups * (elems / kRows) + e / kRows) * 4;
    const float vs = p.scales ? __ldg(p.scales + p.hkv + head) : 1.f;
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
        const float base_m = mx == -INFINITY ? 0.f : mx;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const float a = ex2(m[b] - base_m);
          s.l += a * l[b];
          s.o.x += a * o[b].x;
          s.o.y += a * o[b].y;
          s.o.z += a * o[b].z;
          s.o.w += a * o[b].w;
        }
      }
    if (sharers > 1) {
      sh[tid] = s;
      __syncthreads();
      if (mine == 0)
        for (int k = 1; k < sharers; ++k) {
          State t = sh[tid + k * elems];
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
      if (s.l == 0.f) s.o = make_float4(0.f, 0.f, 0.f, 0.f);  // also over values that are not finite
      const int d = tree_draft(p, row0 + r), hh = row0 + r - d * p.group;
      *reinterpret_cast<uint2*>(p.out + (item.x + d) * p.out_stride + (int64_t)(head * p.group + hh) * D + col) =
          make_uint2(pack_bf16x2(s.o.x * f, s.o.y * f), pack_bf16x2(s.o.z * f, s.o.w * f));
      if (p.lse && col == 0)
        p.lse[(int64_t)(item.x + d) * p.hq + head * p.group + hh] = s.l == 0.f ? -INFINITY : kLn2 * (s.m + (log2f(s.l) - lift));
    }
  };
  if constexpr (Direct) {
    const int4 item = __ldcg(p.items + blockIdx.x);
    const int units = units_of(item.w);
    for (int at = blockIdx.y; at < units; at += gridDim.y) {
      join(item, blockIdx.x, at);
      __syncthreads();
    }
    return;
  }
  // units: 8 rows of an item and as many columns as fit; block b has units b, b + gridDim.x, ..
  int unit = blockIdx.x, done = 0;
  for (int base = 0; base < ctas; base += kThreads) {
    const int4 mine_item = base + tid < ctas ? __ldcg(p.items + base + tid) : make_int4(0, 0, 0, 0);
    const int units = units_of(mine_item.w);
    int upto = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    __syncthreads();
    if (lane == 31) sums[tid >> 5] = upto;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < tid >> 5) upto += sums[w];
      sum += sums[w];
    }
    upto += done;
    done += sum;
    for (; unit < done; unit += gridDim.x) {
      __syncthreads();
      if (unit < upto && unit >= upto - units) {
        s_item = mine_item;
        s_at = make_int2(base + tid, unit - (upto - units));
      }
      __syncthreads();
      join(s_item, s_at.x, s_at.y);
    }
  }
}

}  // namespace

template <int D>
static cudaError_t launch_one(const TreeParams& p, int rows, float lift, int ctas, cudaStream_t st) {
  // Few rows of items with a few parts each (as many as if all items were as long) are a few units per item, found without
  // counting: 4 x 1 tokens, 1000 keys, 32/8 heads of 128: 12.2 us for the whole call, 13.5 with the count.  Rows or parts that make
  // more units than four want blocks of their own: 64 drafts, 131072 keys: 119 and 112; 1 x 4096 keys, 16/2 heads of 256: 18.5, 13.7.
  const int most = p.max_tokens * p.group, row_units = (most + kRows - 1) / kRows;
  const int col_units = D / 4 * kRows * (1 << tree_parts_shared(ctas / (p.hkv * p.batch) + 1)) / kThreads;
  if (most <= 16 && col_units <= 4)
    return launch_pdl(join_kernel<D, true>, dim3((unsigned)ctas, row_units * 4u), dim3(kThreads), 0, st, p, rows, ctas, lift);
  // no more blocks than there can be units: of a head's rows an eighth and one per sequence, times shares of the columns
  const int64_t units = (int64_t)p.hkv * (p.n * p.group / kRows + p.n) * (D / 16), fit = (int64_t)kPerSM * device_sm_count();
  return launch_pdl(join_kernel<D, false>, dim3((unsigned)(units < fit ? units : fit)), dim3(kThreads), 0, st, p, rows, ctas, lift);
}

cudaError_t launch_tree_join(const TreeParams& p, int dim, int rows, float lift, int ctas, cudaStream_t st) {
  return dim == 64 ? launch_one<64>(p, rows, lift, ctas, st) : dim == 128 ? launch_one<128>(p, rows, lift, ctas, st)
                                                                        : launch_one<256>(p, rows, lift, ctas, st);
}

}  // namespace trellis

// tree_attention.cu -- attention of drafted tokens over a paged cache (trellis_tree_attention).
//
// For a query row with scores x_p = scale * q.k_p * log2(e) over the positions it sees:
//   m = max x_p,  l = sum 2^(x_p - m),  o = sum 2^(x_p - m) v_p;   out = o / l,  lse = ln2 (m + log2 l)
// computed in one pass over the keys with m, l and o carried along (o and l are scaled by 2^(m_old - m_new) when the
// maximum moves), and joined over disjoint sets of keys by the same rule.
//
// Three kernels do so; all divide the work as tree_sched.cuh says and leave parts of shared items to tree_join.cu:
//   this one                 heads of 64 and 128, up to 16 rows of a key/value head (its group of query heads times the drafts)
//   tree_attention_tc.cu     bf16 heads of 64 and 128, more rows:   tcgen05, 256 rows a block
//   tree_attention_tc1.cu    e4m3 of those, and heads of 256:      tcgen05, 128 rows a block
// Measured on both sides (us, this one / the other; 32/8 heads of 128 unless said otherwise):
//   16 rows: 300 keys 8.2 / 9.5, 4096 keys 11.2 / 12.3, ragged batch of 32 to 2000 37 / 35, 60000 keys 46 / 45;
//            heads of 64, 300 keys 6.9 / 8.7, 60000 keys 29 / 31
//   32 rows: 4096 keys 13.0 / 12.8, ragged batch of 32 to 2048 46 / 35 (e4m3 45 / 37), 131072 keys 126 / 86
// Heads of 256 (e4m3, 16/2 heads): 8 rows, 4096 keys 18.1 / 13.7, 60000 keys 33.5 / 26.4, 300 keys 9.8 / 10.8.
//
// Here a block takes all rows, padded to 16, and its four warps split the keys of a tile between them: scores and outputs
// are warp-level matrix products (m16n8k16) whose accumulators, maxima and sums stay in the registers of one warp
// until the segment ends.  Keys and values arrive as 64-key tiles by tensor copies (TMA, 128-byte swizzle, one box
// per page) issued by a warp of its own, up to eight tiles ahead.  An e4m3 cache stays 8 bits in shared memory and becomes fp16 in
// registers; its queries are fp16 too, each row scaled by a power of two.
//
// Bound: HBM (1 x 131072 keys, 32/8 heads of 128, one token: 86 us, 6.2 TB/s), with e4m3 the latency of the conversions in four
// warps (72 us, 3.7 TB/s; a second group of four warps that takes every other tile: 62, but 61 us for 55 on a ragged batch of
// 64), and for short contexts that of two launches and a segment's start and end (1 x 4096 keys, 40/8 heads: 10.6 us).
#include <cstring>
#include <cuda.h>

#include "common.cuh"
#include "devcache.h"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"
#include "tc_ptx.cuh"
#include "tree_sched.cuh"

namespace trellis {
namespace {

__device__ int g_tree_error = 0;  // set when a bounded wait gives up (trellis_device_error)

constexpr uint64_t kDrainNs = 2000000000ull;  // for copies in flight when a block leaves
constexpr int kRows = 16;  // rows of a block
constexpr int kTile = 64;  // keys per step
// an item's start and end, in steps (64 x 1 token, ragged to 2048 keys, 32/8 heads of 128: 97 us without, 56, 57 with 12)
constexpr int kExtra = 6;
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// c += a (16 x 16) * b (16 x 8), 16-bit operands (bf16, or fp16), fp32 sums.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Two e4m3 (low 16 bits) to two fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ void named_sync(int id, int count) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory"); }

template <int D, bool F8>
struct Cfg {
  static constexpr int WK = 4;                      // warps, along the keys of a tile
  static constexpr int KW = kTile / WK;             // keys of a warp per tile
  static constexpr int Consumers = WK;
  static constexpr int Threads = (Consumers + 1) * 32;
  static constexpr int RowBytes = D * (F8 ? 1 : 2);  // a key or value
  static constexpr int BoxBytes = RowBytes < 128 ? RowBytes : 128;  // of it in one copy: a swizzled row
  static constexpr int Blocks = RowBytes / BoxBytes;
  static constexpr int HalfStage = kTile * RowBytes;  // the keys, or the values, of a tile
  static constexpr int Stage = 2 * HalfStage;
  static constexpr int QBytes = kRows * D * 2;
  static constexpr int Regs = D / 2;                 // output numbers of a lane
  // fp16 weights are lifted to 2^15 at most, so that small ones do not vanish below its smallest numbers
  static constexpr float Lift = F8 ? 15.f : 0.f;
  static constexpr int JoinSlot = (Regs + 4) * 32;   // a warp's outputs, maxima and sums
  static constexpr int Join = WK / 2 * JoinSlot * 4;
  static constexpr int Fixed = QBytes + Join + kRows * 8 + kRows * 4 + (int)sizeof(TreeMap) + 256;
  static constexpr int Fit = (227 * 1024 - 1024 - Fixed) / Stage;
  static constexpr int Stages = Fit > 8 ? 8 : Fit;
  static_assert(D <= 128, "heads of 256 are those of tree_attention_tc1.cu");
  static_assert(Stages >= 2, "two tiles in flight at least");
  static constexpr int Smem = 1024 + Stages * Stage + Fixed;
};

// Offset of 16-byte chunk `chunk` of row `row` in a swizzled tile of kTile rows (copied as Blocks boxes side by side).
template <typename C>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  if constexpr (C::BoxBytes == 128)
    return (uint32_t)((chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
  else  // 64-byte rows, 64-byte swizzle
    return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::Threads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TreeParams p) {
  using C = Cfg<D, F8>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* stages = base;
  uint8_t* sq = stages + C::Stages * C::Stage;
  float* join = reinterpret_cast<float*>(sq + C::QBytes);
  uint64_t* row_mask = reinterpret_cast<uint64_t*>(join + C::Join / 4);
  float* row_fac = reinterpret_cast<float*>(row_mask + kRows);
  TreeMap& seqs = *reinterpret_cast<TreeMap*>(row_fac + kRows);
  uint64_t* full = reinterpret_cast<uint64_t*>(&seqs + 1);
  uint64_t* empty = full + C::Stages;
  volatile int* flags = reinterpret_cast<volatile int*>(empty + C::Stages);  // [0] a wait gave up

  constexpr float kLift = C::Lift;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&map);
    for (int i = 0; i < C::Stages; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, C::Consumers);
    }
    flags[0] = 0;
    tc::fence_mbar_init();
  }
  pdl_enter();
  if (warp == 0) tree_cumulate<kRows, kTile, false, kExtra>(p, seqs);
  __syncthreads();
  const int total = seqs.cum[p.batch];
  const int ctas = tree_ctas_used<kRows, false>(p, total, (int)gridDim.x);
  const int cta = blockIdx.x;
  if (cta >= ctas) {  // fewer steps than blocks
    if (threadIdx.x == 0) p.items[cta] = make_int4(0, 0, 0, 0);
    return;
  }

  TreeWalk<kRows, kTile, false> walk(total, ctas, cta);
  TreeSegment g;
  if (warp == C::Consumers) {
    // ---- the copying warp: every tile of the range, as many ahead as there are stages
    int it = 0, issued = 0;
    bool dead = false;
    while (walk.next(p, seqs, g)) {
      TreePages<kTile> pages(p, g, lane);
      const int len = g.seq.prefix + g.seq.count;
      const int box = p.page_shift < 6 ? 1 << p.page_shift : kTile;  // rows of one copy
      for (int t = 0; t < g.tiles; ++t, ++it) {
        const int s = it % C::Stages;
        const int pos0 = (g.tile0 + t) * kTile;
        // lane i fetches box i of the tile; boxes past the sequence's end are not copied
        const int pos = pos0 + lane * box;
        const bool mine = lane * box < kTile && pos < len;
        int y = 0, page = pages.at(t);
        if (mine) {
          page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
          y = (((page * 2) * p.hkv + g.head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        }
        const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, mine));
        if (it >= C::Stages && !dead) {
          const bool ok = tc::mbar_wait_short(empty + s, (uint32_t)((it / C::Stages) & 1) ^ 1u, p.wait_ns);
          // A consumer that gave up releases tiles it never saw, perhaps before they landed: its flag, set before its
          // arrival, ends the copying too, since a barrier must not be armed again while its copies are in flight.
          if (__any_sync(0xFFFFFFFFu, !ok || flags[0] != 0)) {
            dead = true;
            if (lane == 0) flags[0] = 1;
          }
        }
        if (dead) continue;  // the consumers' waits run out too; what is in flight lands below
        issued = it + 1;
        uint8_t* st = stages + s * C::Stage;
        if (lane == 0) tc::mbar_arrive_expect_tx(full + s, (uint32_t)(2 * boxes * box * C::RowBytes));
        __syncwarp();
        if (mine) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int blk = 0; blk < C::Blocks; ++blk)
              tc::tma_load_2d(st + kv * C::HalfStage + blk * (kTile * C::BoxBytes) + lane * box * C::BoxBytes, &map, full + s,
                              blk * (F8 ? C::BoxBytes : C::BoxBytes / 2), y + kv * (p.hkv << p.page_shift));
        }
      }
    }
    // no copy may land in a block that has left, also where a consumer's wait gave up: see the last ones through
    for (int i = issued > C::Stages ? issued - C::Stages : 0; i < issued; ++i)
      tc::mbar_wait(full + i % C::Stages, (uint32_t)((i / C::Stages) & 1), kDrainNs);
  } else {
    const int wk = warp;
    const int gq = lane >> 2, c4 = lane & 3;  // fragment row and column pair
    const int nthr = C::Consumers * 32;
    int4 shared_item = make_int4(0, 0, 0, 0);  // the item that starts here and ends in a later block
    int it = 0;
    bool dead = false;
    while (walk.next(p, seqs, g)) {
      const int rows = min(kRows, g.seq.count * p.group - g.row_block * kRows);  // rows of this block that exist
      const int row0 = g.row_block * kRows;
      named_sync(1, nthr);  // the previous segment's queries are no longer read
      // ---- queries: row r is draft (row0 + r) / group, head (row0 + r) % group of the key/value head's group
      {
        constexpr int LPR = D / 8;  // lanes of a row
        for (int r = threadIdx.x / LPR; r < kRows; r += nthr / LPR) {
          const int l = threadIdx.x % LPR;
          const int d = tree_draft(p, row0 + r), hh = row0 + r - d * p.group;
          uint4 u = make_uint4(0, 0, 0, 0);
          if (r < rows)
            u = *reinterpret_cast<const uint4*>(p.q + (g.seq.start + d) * p.q_stride +
                                                (int64_t)(g.head * p.group + hh) * D + 8 * l);
          float fac = 1.f;
          if constexpr (F8) {
            float x[8] = {bf16lo_to_f32(u.x), bf16hi_to_f32(u.x), bf16lo_to_f32(u.y), bf16hi_to_f32(u.y),
                          bf16lo_to_f32(u.z), bf16hi_to_f32(u.z), bf16lo_to_f32(u.w), bf16hi_to_f32(u.w)};
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
            constexpr unsigned kLanes = (1u << LPR) - 1;
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kLanes << (lane / LPR * LPR), m, o));
            // the row's largest exponent to 0: fp16 then keeps every bf16 number within 2^-14 of the largest exactly.  At the
            // ends (zero and subnormal rows; the largest exponent) as near as the factor and its reciprocal stay normal numbers.
            uint32_t e = __float_as_uint(m) >> 23;
            e = e == 255 ? 127u : min(max(e, 1u), 253u);  // infinite or NaN rows as they are
            fac = __uint_as_float(e << 23);
            const float inv = __uint_as_float((254u - e) << 23);
            u = make_uint4(pack_f16x2(x[0] * inv, x[1] * inv), pack_f16x2(x[2] * inv, x[3] * inv),
                           pack_f16x2(x[4] * inv, x[5] * inv), pack_f16x2(x[6] * inv, x[7] * inv));
          }
          *reinterpret_cast<uint4*>(sq + r * (D * 2) + ((l ^ (r & 7)) << 4)) = u;
          if (l == 0) {
            row_fac[r] = fac;
            row_mask[r] = r >= rows ? 0ull : p.mask ? p.mask[g.seq.start + d] : d >= 63 ? ~0ull : (2ull << d) - 1;
          }
        }
      }
      named_sync(1, nthr);
      float rc[2];
      uint64_t seen[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = gq + 8 * i;
        rc[i] = p.scale_log2 * row_fac[r] * (F8 && p.scales ? __ldg(p.scales + g.head) : 1.f);
        seen[i] = row_mask[r];
      }
      const uint32_t sq32 = tc::smem_u32(sq);
      constexpr int KS = D / 16;
      uint32_t qa[KS][4];  // query fragments stay in registers
      const auto load_q = [&](uint32_t (&a)[4], int ks) {
        if constexpr (F8) {
          // the order of the 16 numbers of a step is the one the 8-bit keys have in registers: lane column c4 has 4 c4 .. 4 c4 + 3
          const int chunk = 2 * ks + (c4 >> 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = gq + 8 * i;
            const uint2 v = *reinterpret_cast<const uint2*>(sq + r * (D * 2) + ((chunk ^ (r & 7)) << 4) + (c4 & 1) * 8);
            a[i] = v.x;
            a[2 + i] = v.y;
          }
        } else {
          const int r = (lane & 15), chunk = 2 * ks + (lane >> 4);
          ldsm4(a, sq32 + r * (D * 2) + ((chunk ^ (r & 7)) << 4));
        }
      };
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) load_q(qa[ks], ks);

      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      const int len = g.seq.prefix + g.seq.count;

      const int clear = g.seq.prefix / kTile - g.tile0;  // tiles from here on have drafts, or rows past the end, among their keys
      for (int t = 0; t < g.tiles; ++t, ++it) {
        const bool tail = t >= clear;
        const int s = it % C::Stages;
        const bool ok = dead || tc::mbar_wait_short(full + s, (uint32_t)((it / C::Stages) & 1), p.wait_ns);
        if (!__all_sync(0xFFFFFFFFu, ok) && !dead) {
          dead = true;
          if (lane == 0) flags[0] = 1;
        }
        const uint32_t sk = tc::smem_u32(stages + s * C::Stage), sv = sk + C::HalfStage;
        const int key0 = wk * C::KW;                       // this warp's keys of the tile
        const int pos0 = (g.tile0 + t) * kTile + key0;      // their positions

        // ---- scores
        float x[C::KW / 8][4];
#pragma unroll
        for (int i = 0; i < C::KW / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
        if constexpr (F8) {
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
#pragma unroll
            for (int kb = 0; kb < C::KW / 16; ++kb) {
              uint32_t r[4];
              const int row = key0 + kb * 16 + (lane & 15);
              ldsm4(r, sk + tile_at<C>(row, ks + (lane >> 4)));
#pragma unroll
              for (int j = 0; j < 4; ++j) {  // r[0], r[1]: keys 0..7, 8..15 of step ks;  r[2], r[3]: of step ks + 1
                const uint32_t b0 = e4m3x2_to_f16x2(r[j]), b1 = e4m3x2_to_f16x2(r[j] >> 16);
                mma16816<true>(x[kb * 2 + (j & 1)], qa[ks + (j >> 1)], b0, b1);
              }
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int kb = 0; kb < C::KW / 16; ++kb) {
              uint32_t r[4];
              const int row = key0 + kb * 16 + (lane & 7) + ((lane >> 4) << 3);
              ldsm4(r, sk + tile_at<C>(row, 2 * ks + ((lane >> 3) & 1)));
              mma16816<false>(x[kb * 2], qa[ks], r[0], r[1]);
              mma16816<false>(x[kb * 2 + 1], qa[ks], r[2], r[3]);
            }
          }
        }

        // ---- softmax over this warp's keys
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int i = 0; i < C::KW / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i][j] *= rc[j >> 1];
        if (tail)
#pragma unroll
          for (int i = 0; i < C::KW / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int jd = pos0 + i * 8 + c4 * 2 + (j & 1) - g.seq.prefix;
              const bool vis = jd < 0 || (jd < g.seq.count && ((seen[j >> 1] >> jd) & 1ull));
              x[i][j] = vis ? x[i][j] : -INFINITY;
            }
#pragma unroll
        for (int i = 0; i < C::KW / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j >> 1] = fmaxf(mx[j >> 1], x[i][j]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 2));
        }
        if (__any_sync(0xFFFFFFFFu, mx[0] != m[0] || mx[1] != m[1])) {
          float a[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[i] = m[i] == mx[i] ? 1.f : ex2(m[i] - mx[i]);
            l[i] *= a[i];
            m[i] = mx[i];
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] *= a[j >> 1];
        }
        const float ms[2] = {(m[0] == -INFINITY ? 0.f : m[0]) - kLift, (m[1] == -INFINITY ? 0.f : m[1]) - kLift};
        // Weights become 16 bits for the product with the values, which has no wider form at this rate: half a unit of each, 2^-9
        // in bf16 and 2^-12 in fp16 (their sum is that of the unrounded ones).  Off the 64-bit result, relative: 4095 bf16 keys
        // 0.0018, 131072 (tree_attention_tc.cu) 0.0023, of which 0.0017 are the rounding of outputs to bf16.
        uint32_t pa[C::KW / 16][4];
#pragma unroll
        for (int i = 0; i < C::KW / 8; ++i) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e[j] = ex2(x[i][j] - ms[j >> 1]);
            l[j >> 1] += e[j];
          }
          pa[i >> 1][(i & 1) * 2] = F8 ? pack_f16x2(e[0], e[1]) : pack_bf16x2(e[0], e[1]);
          pa[i >> 1][(i & 1) * 2 + 1] = F8 ? pack_f16x2(e[2], e[3]) : pack_bf16x2(e[2], e[3]);
        }

        if (tail) {
          // Values that must not reach a product: rows past the end, whatever their bits, become zeros; drafts with
          // numbers that are not finite (rare) are added to the rows that see them, and become zeros there too.
          uint8_t* tile = stages + s * C::Stage + C::HalfStage;
          const int base_pos = (g.tile0 + t) * kTile, from = max(g.seq.prefix - base_pos, 0);
          constexpr uint32_t kExp = F8 ? 0x7Fu : 0x7F80u;  // bits that are all ones in what is not finite
          constexpr int Chunks = C::RowBytes / 16;
          const auto not_finite = [&](uint32_t w) {
            if constexpr (F8) return (w & 0x7Fu) == 0x7Fu || (w >> 8 & 0x7Fu) == 0x7Fu || (w >> 16 & 0x7Fu) == 0x7Fu || (w >> 24 & 0x7Fu) == 0x7Fu;
            else return (w & kExp) == kExp || (w >> 16 & kExp) == kExp;
          };
          bool odd = false;
          for (int e = from * Chunks + threadIdx.x; e < kTile * Chunks; e += nthr) {
            const int row = e / Chunks;
            uint4* at = reinterpret_cast<uint4*>(tile + tile_at<C>(row, e - row * Chunks));
            if (base_pos + row >= len) *at = make_uint4(0, 0, 0, 0);
            else odd |= not_finite(at->x) || not_finite(at->y) || not_finite(at->z) || not_finite(at->w);
          }
          if (tc::bar_or(odd, 1, nthr)) {
            for (int kk = 0; kk < C::KW; ++kk) {
              const int jd = pos0 + kk - g.seq.prefix;
              if (jd < 0 || jd >= g.seq.count) continue;
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int d = F8 ? (i >> 1) * 16 + c4 * 4 + (j & 1) * 2 + (i & 1) : i * 8 + c4 * 2 + (j & 1);
                  const int byte = F8 ? d : 2 * d;
                  const uint8_t* at = tile + tile_at<C>(key0 + kk, byte >> 4) + (byte & 15);
                  const uint32_t v = F8 ? *at : *reinterpret_cast<const uint16_t*>(at);
                  if ((v & kExp) == kExp && ((seen[j >> 1] >> jd) & 1ull))
                    o[i][j] += F8 ? __int_as_float(0x7FC00000) : bf16_to_f32((uint16_t)v);
                }
            }
            named_sync(1, nthr);
            for (int e = from * Chunks * 16 + threadIdx.x * 2; e < kTile * Chunks * 16; e += nthr * 2) {
              const int row = e / (Chunks * 16), byte = e - row * (Chunks * 16);
              uint16_t* at = reinterpret_cast<uint16_t*>(tile + tile_at<C>(row, byte >> 4) + (byte & 15));
              const uint32_t v = *at;
              if constexpr (F8) *at = (uint16_t)(((v & 0x7Fu) == 0x7Fu ? 0 : v & 0xFFu) | ((v >> 8 & 0x7Fu) == 0x7Fu ? 0 : v & 0xFF00u));
              else if ((v & kExp) == kExp) *at = 0;
            }
            named_sync(1, nthr);
          }
          tc::fence_proxy_async_smem();  // before the next copy into this tile
        }

        // ---- outputs
#pragma unroll
        for (int kb = 0; kb < C::KW / 16; ++kb) {
          const int row = key0 + kb * 16 + (lane & 15);
#pragma unroll
          for (int dc = 0; dc < C::RowBytes / 16; dc += 2) {
            uint32_t r[4];
            ldsm4t(r, sv + tile_at<C>(row, dc + (lane >> 4)));
            if constexpr (F8) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {  // chunk dc + j: its even columns, then its odd ones
                mma16816<true>(o[2 * (dc + j)], pa[kb], e4m3x2_to_f16x2(__byte_perm(r[2 * j], 0, 0x4420)),
                               e4m3x2_to_f16x2(__byte_perm(r[2 * j + 1], 0, 0x4420)));
                mma16816<true>(o[2 * (dc + j) + 1], pa[kb], e4m3x2_to_f16x2(__byte_perm(r[2 * j], 0, 0x4431)),
                               e4m3x2_to_f16x2(__byte_perm(r[2 * j + 1], 0, 0x4431)));
              }
            } else {
              mma16816<false>(o[dc], pa[kb], r[0], r[1]);
              mma16816<false>(o[dc + 1], pa[kb], r[2], r[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(empty + s);
      }

      // ---- the segment's end: sums over the lanes of a row, then over the warps that share rows
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
      }
#pragma unroll
      for (int step = C::WK / 2; step; step >>= 1) {
        float* mine = join + (wk & (step - 1)) * C::JoinSlot + lane;
        if (wk >= step && wk < 2 * step) {
#pragma unroll
          for (int i = 0; i < C::Regs; ++i) mine[i * 32] = o[i >> 2][i & 3];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mine[(C::Regs + i) * 32] = m[i];
            mine[(C::Regs + 2 + i) * 32] = l[i];
          }
        }
        named_sync(1, nthr);
        if (wk < step) {
          float a[2], b[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float om = mine[(C::Regs + i) * 32], nm = fmaxf(m[i], om), base_m = nm == -INFINITY ? 0.f : nm;
            a[i] = ex2(m[i] - base_m);
            b[i] = ex2(om - base_m);
            l[i] = l[i] * a[i] + mine[(C::Regs + 2 + i) * 32] * b[i];
            m[i] = nm;
          }
#pragma unroll
          for (int i = 0; i < C::Regs; ++i) {
            float& v = o[i >> 2][i & 3];
            v = v * a[(i >> 1) & 1] + mine[i * 32] * b[(i >> 1) & 1];
          }
        }
        named_sync(1, nthr);
      }

      if (g.whole) {
        if (wk == 0) {
          const float vs = F8 && p.scales ? __ldg(p.scales + p.hkv + g.head) : 1.f;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = gq + 8 * half;
            if (r >= rows) continue;
            const float f = l[half] == 0.f ? 0.f : vs / l[half];
            const int d = tree_draft(p, row0 + r), hh = row0 + r - d * p.group;
            uint16_t* to = p.out + (g.seq.start + d) * p.out_stride + (int64_t)(g.head * p.group + hh) * D;
            if constexpr (F8) {
#pragma unroll
              for (int i = 0; i < D / 8; i += 2)
                *reinterpret_cast<uint2*>(to + (i >> 1) * 16 + c4 * 4) =
                    make_uint2(pack_bf16x2(o[i][2 * half] * f, o[i + 1][2 * half] * f), pack_bf16x2(o[i][2 * half + 1] * f, o[i + 1][2 * half + 1] * f));
            } else {
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<uint32_t*>(to + i * 8 + c4 * 2) = pack_bf16x2(o[i][2 * half] * f, o[i][2 * half + 1] * f);
            }
            if (p.lse && c4 == 0)
              p.lse[(int64_t)(g.seq.start + d) * p.hq + g.head * p.group + hh] =
                  l[half] == 0.f ? -INFINITY : kLn2 * (m[half] + (log2f(l[half]) - kLift));
          }
        }
        continue;
      }
      // a part, for the joining kernel
      if (wk == 0) {
        float* part = p.part + (int64_t)tree_slot(cta, g.tile0 == 0) * tree_part_floats(kRows, D);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = gq + 8 * half;
          if (r >= rows) continue;
          if constexpr (F8) {
#pragma unroll
            for (int i = 0; i < D / 8; i += 2)
              *reinterpret_cast<float4*>(part + (((i >> 1) * 4 + c4) * kRows + r) * 4) =
                  make_float4(o[i][2 * half], o[i + 1][2 * half], o[i][2 * half + 1], o[i + 1][2 * half + 1]);
          } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<float2*>(part + ((i * 2 + (c4 >> 1)) * kRows + r) * 4 + (c4 & 1) * 2) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
          }
          if (c4 == 0) {
            part[kRows * D + r] = m[half];
            part[kRows * D + kRows + r] = l[half];
          }
        }
      }
      if (threadIdx.x == 0 && g.starts) shared_item = tree_item(g, row0, rows, cta, tree_cta_of(g.last_at, total, ctas));
    }
    if (threadIdx.x == 0) p.items[cta] = shared_item;
  }
  __syncthreads();
  if (threadIdx.x == 0 && flags[0]) atomicCAS(&g_tree_error, 0, 1);
}

// ---------------------------------------------------------------- host

int tree_ctas() { return device_sm_count() < kTreeMaxCtas ? device_sm_count() : kTreeMaxCtas; }

template <int D, bool F8>
cudaError_t launch_d(const CUtensorMap& map, const TreeParams& p, cudaStream_t st) {
  using C = Cfg<D, F8>;
  auto kern = tree_kernel<D, F8>;
  static PerDevice<cudaError_t> attr_of;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const cudaError_t e = attr_of.get(dev, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem);
  }, cudaErrorInvalidDevice);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = launch_pdl(kern, dim3((unsigned)tree_ctas()), dim3(C::Threads), C::Smem, st, map, p);
  return e2 != cudaSuccess ? e2 : launch_tree_join(p, D, kRows, C::Lift, tree_ctas(), st);
}

}  // namespace

size_t tree_workspace_bytes(const trellis_cache_t& c, int batch, int max_tokens, int q_heads) {
  (void)batch;  // parts belong to thread blocks, whatever the batch
  const int group = q_heads / c.heads;
  const int most = max_tokens * group;
  const int rows = tree_tc_fits(c, most) ? tree_tc_rows() : tree_tc1_fits(c, most) ? tree_tc1_rows() : kRows;
  return kTreeMaxCtas * sizeof(int4) + (size_t)tree_part_floats(rows, c.head_dim) * 4 * 2 * tree_ctas();
}

int read_tree_error(int reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_tree_error, sizeof(int)) != cudaSuccess) return -1;
  if (reset && v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  const int w = read_tree_tc_error(reset), x = read_tree_tc1_error(reset);
  return v ? v : w ? w : x;
}

cudaError_t launch_tree_attention(const uint16_t* q, int64_t q_stride, const trellis_cache_t& c, int layer,
                                  const trellis_drafts_t& d, int q_heads, float scale, uint16_t* out,
                                  int64_t out_stride, float* lse, void* workspace, cudaStream_t st) {
  TreeParams p{};
  p.q = q; p.out = out; p.lse = lse;
  p.table = d.table; p.prefix = d.prefix; p.q_start = d.q_start; p.mask = d.mask;
  p.scales = c.scales ? c.scales + (int64_t)layer * 2 * c.heads : nullptr;
  p.q_stride = q_stride; p.out_stride = out_stride;
  p.pages = c.pages;
  p.wait_ns = wait_limit_ns();
  p.batch = d.batch; p.width = d.width; p.n = d.n; p.max_tokens = d.max_tokens;
  p.hq = q_heads; p.hkv = c.heads; p.group = q_heads / c.heads;
  p.group_inv = (((uint64_t)1 << 32) + p.group - 1) / p.group;
  p.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  p.scale_log2 = scale * kLog2e;
  p.items = static_cast<int4*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kTreeMaxCtas * sizeof(int4));

  const auto fn = tensor_map_encoder();
  if (!fn) return cudaErrorNotSupported;
  const int most = d.max_tokens * p.group, elem = (int)cache_elem_bytes(c), row_bytes = c.head_dim * elem;
  const bool f8 = c.dtype == TRELLIS_E4M3, tc = tree_tc_fits(c, most), tc1 = tree_tc1_fits(c, most);
  TreeBox copy{c.page_size < kTile ? c.page_size : kTile, row_bytes < 128 ? row_bytes : 128};
  if (tc) tree_tc_box(c, &copy);
  if (tc1) tree_tc1_box(c, &copy);
  uint8_t* pool = static_cast<uint8_t*>(c.pool) + (int64_t)layer * c.pages * cache_page_bytes(c);
  CUtensorMap map;
  const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)(c.pages * 2 * c.heads * c.page_size)};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)(copy.bytes / elem), (cuuint32_t)copy.rows};
  const cuuint32_t estr[2] = {1, 1};
  if (fn(&map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE,
         copy.bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  p.pool = pool;
  if (tc) return launch_tree_tc(map, p, c, tree_ctas(), st);
  if (tc1) return launch_tree_tc1(map, p, c, tree_ctas(), st);
  if (f8) return c.head_dim == 64 ? launch_d<64, true>(map, p, st) : launch_d<128, true>(map, p, st);
  return c.head_dim == 64 ? launch_d<64, false>(map, p, st) : launch_d<128, false>(map, p, st);
}

}  // namespace trellis

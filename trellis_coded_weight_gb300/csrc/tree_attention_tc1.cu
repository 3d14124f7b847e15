// tree_attention_tc1.cu -- tree attention with the 5th-generation tensor cores for e4m3 caches (any head dim) and heads of
// 256, where tree_attention_tc.cu's two accumulators do not fit.
//
// As there, S = Q K^T and O += P V are tcgen05 MMAs of one issuing thread, P lies in tensor memory over its scores, and two
// softmax warpgroups alternate between the tiles, a thread per row.  Here a block has 128 rows and one accumulator O, so the
// maximum in use is one per row: the warp that has tile i hands its rows' maxima to the warp that has tile i + 1 (an mbarrier
// per warp), before it makes its weights; the groups' sums of weights stay apart until the end.
//
// An e4m3 cache is copied as it is, and a warpgroup of its own turns each tile into fp16 in the layout that the MMAs read
// (exact: 2 bytes of shared memory per number instead of 1, but the products see 16-bit operands and Q keeps its 8
// significant bits).  Q is fp16 then, each row scaled by a power of two, and P fp16 too.  That group also clears what
// must not reach a product.
// Bound: HBM for a cache of 16-bit numbers; the products and the conversion come near it with e4m3.
#include <cstring>
#include <cuda.h>

#include "common.cuh"
#include "devcache.h"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"
#include "tc_ptx.cuh"
#include "tree_sched.cuh"
#include "tree_tc.cuh"

namespace trellis {
namespace {

using namespace tree;

__device__ int g_tree_tc1_error = 0;  // set when a bounded wait gives up (trellis_device_error)

constexpr int kRows = 128;  // rows of a block
constexpr int kSoftmaxWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kConvertWarp = 12;
constexpr int kConvertThreads = 128;

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(r) : "r"(v));
  return r;
}

template <int D, bool F8>
struct Cfg {
  static constexpr int Tile = D == 256 ? 64 : 128;          // keys per step
  static constexpr int Blocks = D / 64;                     // 128-byte blocks of a row of 16-bit numbers
  static constexpr int Slot = Tile * D * 2;                 // the keys, or the values, of a tile
  static constexpr int QTile = kRows * D * 2;
  static constexpr int RawSlot = Tile * D;
  static constexpr int Threads = F8 ? 512 : 384;
  static constexpr int Fixed = QTile + kRows * 8 + kRows * 4 * 4 + (kTreeMaxBatch + 4) * 4 + 1024;
  static constexpr int Room = 227 * 1024 - 1024 - Fixed;
  static constexpr int Slots = D == 256 && F8 ? 3 : D == 64 ? 6 : 4;
  static constexpr int RawFit = (Room - Slots * Slot) / RawSlot;
  static constexpr int RawSlots = F8 ? (RawFit > 8 ? 8 : RawFit) : 0;
  static_assert(Slots * Slot <= Room && (!F8 || RawSlots >= 3), "fits");
  static constexpr int Smem = 1024 + Slots * Slot + RawSlots * RawSlot + Fixed;
  static constexpr int S(int s) { return s * 128; }         // tensor memory columns
  static constexpr int O = 256;
  static constexpr float Lift = F8 ? 7.f : 0.f;             // fp16 weights reach 2^15: 2^kMove times this
};

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::Threads, 1)
    tree_tc1_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TreeParams p) {
  using C = Cfg<D, F8>;
  constexpr int kTile = C::Tile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = base;
  uint8_t* sq = ring + C::Slots * C::Slot;
  uint8_t* raws = sq + C::QTile;
  uint64_t* row_mask = reinterpret_cast<uint64_t*>(raws + C::RawSlots * C::RawSlot);
  float* row_fac = reinterpret_cast<float*>(row_mask + kRows);
  float* row_max = row_fac + kRows;       // in use
  float* row_sum = row_max + kRows;       // [2][rows]
  int* cum = reinterpret_cast<int*>(row_sum + 2 * kRows);
  uint64_t* full = reinterpret_cast<uint64_t*>(cum + kTreeMaxBatch + 4);
  uint64_t* empty = full + C::Slots;
  uint64_t* raw_full = empty + C::Slots;
  uint64_t* raw_empty = raw_full + 8;
  uint64_t* q_ready = raw_empty + 8;
  uint64_t* s_full = q_ready + 1;   // [2] a tile's scores; also: the products of the tile two before it are complete
  uint64_t* p_ready = s_full + 2;   // [2] weights written
  uint64_t* o_done = p_ready + 2;   // each tile's product with the values
  uint64_t* o_full = o_done + 1;    // the segment's last one
  uint64_t* drained = o_full + 1;
  uint64_t* turn = drained + 1;     // [2][4] a warp's row maxima of its tile
  volatile int* flags = reinterpret_cast<volatile int*>(turn + 8);  // [0] a wait gave up, [2] segment with odd values
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(flags) + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&map);
    for (int i = 0; i < C::Slots; ++i) {
      tc::mbar_init(full + i, F8 ? kConvertThreads / 32 : 1);
      tc::mbar_init(empty + i, 1);
    }
    for (int i = 0; i < C::RawSlots; ++i) {
      tc::mbar_init(raw_full + i, 1);
      tc::mbar_init(raw_empty + i, kConvertThreads / 32);
    }
    tc::mbar_init(q_ready, kSoftmaxWarps);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(s_full + s, 1);
      tc::mbar_init(p_ready + s, kSoftmaxWarps / 2);
    }
    tc::mbar_init(o_done, 1);
    tc::mbar_init(o_full, 1);
    tc::mbar_init(drained, 1);
    for (int i = 0; i < 8; ++i) tc::mbar_init(turn + i, 1);
    flags[0] = 0;
    flags[2] = -1;
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  pdl_enter();
  if (warp == 0) tree_cumulate<kRows, kTile, false>(p, cum);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int total = cum[p.batch];
  const int cta = blockIdx.x;
  TreeWalk<kRows, kTile, false> walk(total, tree_ctas_used<false>(total, (int)gridDim.x), cta);
  TreeSegment g;

  if (warp >= kSoftmaxWarps) {
    // F8: 512 threads x 128 registers at launch = 256 x 184 + 256 x 72; else 384 x 168 = 256 x 200 + 128 x 104
    if constexpr (F8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kCopyWarp) {
      // ---- the copying warp: tiles as the cache has them, into the ring or (e4m3) into the raw ring
      constexpr int kSlots = F8 ? C::RawSlots : C::Slots;
      uint64_t* const bar_full = F8 ? raw_full : full;
      uint64_t* const bar_empty = F8 ? raw_empty : empty;
      int it = 0;
      bool dead = false;
      const int box = min(1 << p.page_shift, kTile);  // rows of one copy
      while (!dead && walk.next(p, cum, g)) {
        const int32_t* row = p.table + (int64_t)g.b * p.width;
        const int len = g.seq.prefix + g.seq.count;
        const Order order{g.tiles, true};
        for (int e = 0; e < 2 * g.tiles; ++e, ++it) {
          bool value;
          const int t = order.at(e, &value), s = it % kSlots;
          const int pos = (g.tile0 + t) * kTile + lane * box;  // lane i copies box i of the tile, none past the end
          const bool mine = lane * box < kTile && pos < len;
          int y = 0;
          if (mine) {
            int page = __ldg(row + (pos >> p.page_shift));
            page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
            y = (((page * 2 + (value ? 1 : 0)) * p.hkv + g.head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
          }
          const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, mine));
          if (it >= kSlots) {
            const bool ok = tc::mbar_wait_short(bar_empty + s, (uint32_t)(it / kSlots & 1) ^ 1u, p.wait_ns);
            if (__any_sync(0xFFFFFFFFu, !ok)) {
              dead = true;
              if (lane == 0) flags[0] = 1;
              break;
            }
          }
          if (lane == 0) tc::mbar_arrive_expect_tx(bar_full + s, (uint32_t)(boxes * box * D * (F8 ? 1 : 2)));
          __syncwarp();
          if (mine) {
            if constexpr (F8) {
              tc::tma_load_2d(raws + s * C::RawSlot + lane * box * D, &map, bar_full + s, 0, y);
            } else {
#pragma unroll
              for (int blk = 0; blk < C::Blocks; ++blk)
                tc::tma_load_2d(ring + s * C::Slot + blk * (kTile * 128) + lane * box * 128, &map, bar_full + s, blk * 64, y);
            }
          }
        }
      }
      // no copy may land in a block that has left
      for (int i = it > kSlots ? it - kSlots : 0; i < it; ++i) tc::mbar_wait(bar_full + i % kSlots, (uint32_t)(i / kSlots & 1), kDrainNs);
    } else if (warp == kMmaWarp) {
      // ---- the thread that issues the products, taking the ring's entries in order
      if (lane == 0) {
        bool dead = false, issued = false;
        int seg = 0;
        uint32_t slot = 0, use = 0, ns[2] = {0, 0};
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (!dead && !tc::mbar_wait_short(bar, parity, p.wait_ns)) {
            dead = true;
            flags[0] = 1;
          }
          return !dead;
        };
        constexpr uint32_t kType = F8 ? ~((1u << 7) | (1u << 10)) : ~0u;  // fp16 operands: type fields 0
        const uint32_t id_s = tc::idesc_bf16_f32(128, kTile) & kType, id_o = (tc::idesc_bf16_f32(128, D) & kType) | kBMnMajor;
        const uint64_t q_desc = tc::desc_kmajor(tc::smem_u32(sq), 1024, 2), k_desc = tc::desc_kmajor(tc::smem_u32(ring), 1024, 2),
                       v_desc = desc_mnmajor(tc::smem_u32(ring), kTile * 128);
        const auto take = [&] { return wait(full + slot, use & 1u); };
        const auto release = [&] {
          tc::mma_commit(empty + slot);
          if (++slot == C::Slots) {
            slot = 0;
            ++use;
          }
        };
        const auto scores = [&](int s) {
          const uint64_t b = k_desc + slot * (C::Slot >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_bf16(tmem + C::S(s), q_desc + (uint32_t)(((k >> 2) * (kRows * 128) + (k & 3) * 32) >> 4),
                         b + (uint32_t)(((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4), id_s, k > 0);
          tc::mma_commit(s_full + s);
          issued = true;
          release();
        };
        while (!dead && walk.next(p, cum, g)) {
          const int n = g.tiles;
          if (!wait(q_ready, (uint32_t)(seg & 1))) break;
          tc::fence_after_sync();
          for (int i = 0; i < 2 && i < n; ++i)
            if (take()) scores(i);
          for (int i = 0; i < n; ++i) {
            const int s = i & 1;
            if (!take() || !wait(p_ready + s, ns[s] & 1u)) break;
            ++ns[s];
            tc::fence_after_sync();
            const uint64_t b = v_desc + slot * (C::Slot >> 4);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              mma_ts(tmem + C::O, tmem + C::S(s) + 8 * k, b + (uint32_t)((k * 16 * 128) >> 4), id_o, i > 0 || k > 0);
            tc::mma_commit(o_done);
            release();
            if (i + 1 == n) tc::mma_commit(o_full);
            if (i + 2 < n) {
              if (!take()) break;
              scores(s);
            }
          }
          ++seg;
        }
        // tensor memory is given back once every product issued has completed, also where a wait gave up
        if (issued) {
          tc::mma_commit(drained);
          tc::mbar_wait(drained, 0, kDrainNs);
        }
      }
      __syncwarp();
    } else if (F8 && warp >= kConvertWarp) {
      // ---- e4m3 to fp16, tile by tile in the order of the copies
      const int tid = threadIdx.x - kConvertWarp * 32;
      int it = 0, seg = 0;
      bool dead = false;
      const auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = dead || tc::mbar_wait_short(bar, parity, p.wait_ns);
        if (__any_sync(0xFFFFFFFFu, !ok)) {
          dead = true;
          if (lane == 0) flags[0] = 1;
        }
        return !dead;
      };
      while (!dead && walk.next(p, cum, g)) {
        const Order order{g.tiles, true};
        const int len = g.seq.prefix + g.seq.count;
        for (int e = 0; e < 2 * g.tiles; ++e, ++it) {
          bool value;
          const int t = order.at(e, &value);
          const int rs = F8 ? it % (F8 ? C::RawSlots : 1) : 0, s = it % C::Slots;
          if (!wait(raw_full + rs, (uint32_t)(it / (F8 ? C::RawSlots : 1) & 1))) break;
          if (it >= C::Slots && !wait(empty + s, (uint32_t)(it / C::Slots & 1) ^ 1u)) break;
          const uint8_t* from = raws + rs * C::RawSlot;
          uint8_t* to = ring + s * C::Slot;
          const int pos0 = (g.tile0 + t) * kTile;
          const bool tail = value && pos0 + kTile > g.seq.prefix;
          constexpr int CPR = D / 16, kPer = kTile * CPR / kConvertThreads;  // 16-byte chunks of a row, of a thread
          uint4 u[kPer];
#pragma unroll
          for (int k = 0; k < kPer; ++k) u[k] = *reinterpret_cast<const uint4*>(from + (tid + k * kConvertThreads) * 16);
          if (tail) {
            // values of rows past the end, and those of drafts that are not numbers (the only ones e4m3 has), become zeros
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              const int row = (tid + k * kConvertThreads) / CPR;
              if (pos0 + row >= len) u[k] = make_uint4(0, 0, 0, 0);
              else if (pos0 + row >= g.seq.prefix) {
                bool odd = false;
                const auto clean = [&](uint32_t& w) {
#pragma unroll
                  for (int b = 0; b < 32; b += 8)
                    if ((w >> b & 0x7Fu) == 0x7Fu) { w &= ~(0xFFu << b); odd = true; }
                };
                clean(u[k].x); clean(u[k].y); clean(u[k].z); clean(u[k].w);
                if (odd) flags[2] = seg;
              }
            }
          }
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int idx = tid + k * kConvertThreads, row = idx / CPR, c = idx % CPR;
            uint4 h[2];
            h[0] = make_uint4(e4m3x2_to_f16x2(u[k].x), e4m3x2_to_f16x2(u[k].x >> 16), e4m3x2_to_f16x2(u[k].y), e4m3x2_to_f16x2(u[k].y >> 16));
            h[1] = make_uint4(e4m3x2_to_f16x2(u[k].z), e4m3x2_to_f16x2(u[k].z >> 16), e4m3x2_to_f16x2(u[k].w), e4m3x2_to_f16x2(u[k].w >> 16));
            // eight lanes write eight different places of the banks: half of them their second chunk first
            const int flip = c >> 2 & 1;
            uint8_t* at = to + (c >> 2) * (kTile * 128) + row * 128;
            *reinterpret_cast<uint4*>(at + (((2 * c + flip) & 7) ^ (row & 7)) * 16) = flip ? h[1] : h[0];
            *reinterpret_cast<uint4*>(at + (((2 * c + (flip ^ 1)) & 7) ^ (row & 7)) * 16) = flip ? h[0] : h[1];
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(raw_empty + rs);
            tc::mbar_arrive(full + s);
          }
        }
        ++seg;
      }
    }
  } else {
    if constexpr (F8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax: group s, one thread per row; warp w of a group reaches tensor memory lanes 32 w ..
    const int s = warp >> 2, w4 = warp & 3, r = w4 * 32 + lane;
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const uint32_t t_s = tmem + C::S(s) + lanes, t_o = tmem + C::O + lanes;
    int it0 = 0, done0 = 0, seg = 0, ns = 0, turns = 0;  // turns: the other group's hand-overs of this warp's rows so far
    int4 shared_item = make_int4(-1, 0, 0, 0);
    bool dead = false;
    const auto wait = [&](uint64_t* bar, int count) {
      const bool ok = dead || tc::mbar_wait_short(bar, (uint32_t)(count & 1), p.wait_ns);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        dead = true;
        if (lane == 0) flags[0] = 1;
      }
    };
    while (walk.next(p, cum, g)) {
      const int row0 = g.row_block * kRows, rows = min(kRows, g.seq.count * p.group - row0), n = g.tiles;
      const int len = g.seq.prefix + g.seq.count;
      const float k_scale = F8 && p.scales ? __ldg(p.scales + g.head) : 1.f;
      const uint32_t flip = p.scale_log2 * k_scale < 0.f ? 0x80008000u : 0u;  // a negative scale goes into the queries' signs
      named_sync(1, 256);  // the segment before is finished: its queries, statistics and outputs are no longer read
      // ---- queries
      {
        constexpr int LPR = D / 8, kStep = 256 / LPR, kMost = kRows / kStep < 8 ? kRows / kStep : 8;  // lanes of a row, rows at a time, loads in flight
        const int l = threadIdx.x % LPR;
        for (int r0 = threadIdx.x / LPR; r0 < kRows; r0 += kStep * kMost) {
          uint4 u[kMost];
#pragma unroll
          for (int k = 0; k < kMost; ++k) {
            const int q = r0 + k * kStep, d = (row0 + q) / p.group, hh = (row0 + q) - d * p.group;
            u[k] = make_uint4(0, 0, 0, 0);
            if (q < rows) u[k] = __ldg(reinterpret_cast<const uint4*>(p.q + (g.seq.start + d) * p.q_stride + (int64_t)(g.head * p.group + hh) * D + 8 * l));
          }
#pragma unroll
          for (int k = 0; k < kMost; ++k) {
            const int q = r0 + k * kStep;
            uint4 v = make_uint4(u[k].x ^ flip, u[k].y ^ flip, u[k].z ^ flip, u[k].w ^ flip);
            if constexpr (F8) {
              const float x[8] = {bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y),
                                  bf16lo_to_f32(v.z), bf16hi_to_f32(v.z), bf16lo_to_f32(v.w), bf16hi_to_f32(v.w)};
              float m = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
              for (int o = LPR / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
              // the row's largest exponent to 0: fp16 then keeps every bf16 number within 2^-14 of the largest exactly
              uint32_t e = __float_as_uint(m) >> 23;
              if (e < 2 || e > 252) e = 127;  // zero, subnormal, infinite or NaN rows as they are
              const float inv = __uint_as_float((254u - e) << 23);
              v = make_uint4(pack_f16x2(x[0] * inv, x[1] * inv), pack_f16x2(x[2] * inv, x[3] * inv),
                             pack_f16x2(x[4] * inv, x[5] * inv), pack_f16x2(x[6] * inv, x[7] * inv));
              if (l == 0) row_fac[q] = __uint_as_float(e << 23);
            }
            *reinterpret_cast<uint4*>(sq + (l >> 3) * (kRows * 128) + q * 128 + (((l & 7) ^ (q & 7)) << 4)) = v;
          }
        }
        if (threadIdx.x < kRows) {
          const int d = (row0 + threadIdx.x) / p.group;
          row_mask[threadIdx.x] = threadIdx.x >= rows ? 0ull : p.mask ? __ldg(p.mask + g.seq.start + d) : d >= 63 ? ~0ull : (2ull << d) - 1;
        }
        tc::fence_proxy_async_smem();
        named_sync(1, 256);  // masks and factors
        if (lane == 0) tc::mbar_arrive(q_ready);
      }
      const uint64_t seen = row_mask[r];
      // a scale of 0 too leaves minus infinity where it is
      const float c = fmaxf(fabsf(p.scale_log2 * k_scale) * (F8 ? row_fac[r] : 1.f), 1e-37f);
      const bool active = w4 * 32 < rows;     // warps without a row only keep the count
      float used = -INFINITY, l = 0.f;        // the maximum that l is relative to
      for (int i = s; i < n; i += 2) {
        wait(s_full + s, ns++);
        tc::fence_after_sync();
        if (active) {
          const int pos0 = (g.tile0 + i) * kTile;
          const bool tail = pos0 + kTile > g.seq.prefix;
          constexpr int W = kTile / 32;
          if (tail) {
            // scores that the row does not see become minus infinity, in place: columns before `from` are prefix, drafts
            // come after, then nothing
            const int from = g.seq.prefix - pos0;
            const uint64_t drafts = g.seq.count >= 64 ? seen : seen & ((1ull << g.seq.count) - 1);
#pragma unroll 1
            for (int w = 0; w < W; ++w) {
              const int at = from - 32 * w;  // the first draft's place relative to this word of 32 columns
              uint32_t bits = at >= 32 ? 0xFFFFFFFFu : at > 0 ? (1u << at) - 1 : 0u;
              if (at >= 0 && at < 32) bits |= (uint32_t)(drafts << at);
              else if (at < 0 && at > -64) bits |= (uint32_t)(drafts >> -at);
              uint32_t y[32];
              tc::tmem_ld_32x32b_x32(t_s + 32 * w, y);
              tc::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = bits >> j & 1 ? y[j] : 0xFF800000u;
              tmem_st_x32(t_s + 32 * w, y);
            }
            tmem_st_wait();
          }
          // ---- the row's maximum; the scores stay in registers
          uint32_t x[W][32];
#pragma unroll
          for (int w = 0; w < W; ++w) tc::tmem_ld_32x32b_x32(t_s + 32 * w, x[w]);
          tc::tmem_ld_wait();
          float mx = -INFINITY;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            float a = __uint_as_float(x[w][0]);
#pragma unroll
            for (int j = 1; j < 31; j += 2) a = fmaxf(fmaxf(a, __uint_as_float(x[w][j])), __uint_as_float(x[w][j + 1]));
            mx = fmaxf(mx, fmaxf(a, __uint_as_float(x[w][31])));
          }
          mx *= c;
          // ---- the maximum in use, from the warp that has the tile before; moved, and handed on
          if (i > 0) wait(turn + (1 - s) * 4 + w4, turns + ((i - 1) >> 1));
          const float old = i > 0 ? row_max[r] : -INFINITY;
          const bool move = mx > old + kMove || (old == -INFINITY && mx > -INFINITY);
          const float m = move ? mx : old;
          row_max[r] = m;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(turn + s * 4 + w4);
          if (i > 0 && __any_sync(0xFFFFFFFFu, move)) {
            const float a = move ? ex2(old - m) : 1.f;
            wait(o_done, done0 + i - 1);  // (the product before that is known to be complete)
            tc::fence_after_sync();
#pragma unroll 1
            for (int col = 0; col < D; col += 32) {
              uint32_t y[32];
              tc::tmem_ld_32x32b_x32(t_o + col, y);
              tc::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * a);
              tmem_st_x32(t_o + col, y);
            }
          }
          if (used != m) {
            l *= ex2(used - m);
            used = m;
          }
          // ---- weights, over the scores
          const float ms = m == -INFINITY ? C::Lift : C::Lift - m;
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t e[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float2 y = __ffma2_rn(make_float2(__uint_as_float(x[w][j]), __uint_as_float(x[w][j + 1])), make_float2(c, c), make_float2(ms, ms));
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              sum = __fadd2_rn(sum, y);
              e[j >> 1] = F8 ? pack_f16x2(y.x, y.y) : pack_bf16x2(y.x, y.y);
            }
            tmem_st_x16(t_s + 16 * w, e);
          }
          l += sum.x + sum.y;
          tmem_st_wait();
        }
        if constexpr (!F8) {
          const int pos0 = (g.tile0 + i) * kTile;
          if (pos0 + kTile > g.seq.prefix) {
            // Values that must not reach a product: rows past the end become zeros, whatever their bits; so do numbers of
            // drafts that are not finite (rare), which are added at the end to the rows that see them.
            const int e0 = it0 + (i < n - 1 ? 2 * i + 2 : 2 * n - 1);  // their place in the ring
            wait(full + e0 % C::Slots, e0 / C::Slots);
            uint8_t* tile = ring + e0 % C::Slots * C::Slot;
            const int from = max(g.seq.prefix - pos0, 0);
            constexpr int Chunks = D / 8;
            for (int e = from * Chunks + (threadIdx.x & 127); e < kTile * Chunks; e += 128) {
              const int row = e / Chunks, ch = e - row * Chunks;
              uint4* at = reinterpret_cast<uint4*>(tile + (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
              if (pos0 + row >= len) {
                *at = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint4 v = *at;
              bool odd = false;
              const auto clean = [&](uint32_t& w) {
                if ((w & 0x7F80u) == 0x7F80u) { w &= 0xFFFF0000u; odd = true; }
                if ((w >> 16 & 0x7F80u) == 0x7F80u) { w &= 0xFFFFu; odd = true; }
              };
              clean(v.x); clean(v.y); clean(v.z); clean(v.w);
              if (odd) {
                flags[2] = seg;
                *at = v;
              }
            }
            tc::fence_proxy_async_smem();
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_ready + s);
      }
      // ---- the segment's end
      wait(o_full, seg);
      tc::fence_after_sync();
      it0 += 2 * n;
      done0 += n;
      if (active) turns += (n + s) >> 1;  // tiles of the other group: of group 0 (n + 1) / 2, of group 1 n / 2
      named_sync(1, 256);
      // the last tile's warp has left the final maxima: both groups bring their sums to them
      const float m = active ? row_max[r] : -INFINITY;
      const float mine = used == -INFINITY ? 0.f : l * ex2(used - m);
      row_sum[s * kRows + r] = mine;
      named_sync(1, 256);
      l = mine + row_sum[(1 - s) * kRows + r];
      const bool odd = flags[2] == seg, valid = r < rows;
      const int col0 = s * (D / 2), cols = D / 2;  // each group finishes half of the columns
      const auto fetch = [&](int col, float (&v)[32]) {
        uint32_t x[32];
        tc::tmem_ld_32x32b_x32(t_o + col, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(x[j]);
        if (odd && valid)
          for (int j = 0; j < g.seq.count; ++j) {
            const int pos = g.seq.prefix + j, at = pos - g.tile0 * kTile;
            if (!(seen >> j & 1) || at < 0 || at >= n * kTile) continue;
            int page = __ldg(p.table + (int64_t)g.b * p.width + (pos >> p.page_shift));
            page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
            const int64_t first = (((int64_t)((page * 2 + 1) * p.hkv + g.head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1))) * D + col;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if constexpr (F8) {
                if ((reinterpret_cast<const uint8_t*>(p.pool)[first + k] & 0x7Fu) == 0x7Fu) v[k] = __int_as_float(0x7FC00000);
              } else {
                const uint16_t b = p.pool[first + k];
                if ((b & 0x7F80u) == 0x7F80u) v[k] += bf16_to_f32(b);
              }
            }
          }
      };
      if (g.first == g.last) {
        // finished here: rows go through the queries' place (no longer read) so that a row's numbers are stored together
        const float f = l == 0.f ? 0.f : (F8 && p.scales ? __ldg(p.scales + p.hkv + g.head) : 1.f) / l;
        if (active) {
          uint8_t* stage = sq + r * (D * 2);
#pragma unroll 1
          for (int col = col0; col < col0 + cols; col += 32) {
            float v[32];
            fetch(col, v);
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              *reinterpret_cast<uint4*>(stage + ((((col + j) / 8) ^ (r & 7)) << 4)) =
                  make_uint4(pack_bf16x2(v[j] * f, v[j + 1] * f), pack_bf16x2(v[j + 2] * f, v[j + 3] * f),
                             pack_bf16x2(v[j + 4] * f, v[j + 5] * f), pack_bf16x2(v[j + 6] * f, v[j + 7] * f));
          }
        }
        if (valid && s == 0 && p.lse) {
          const int d = (row0 + r) / p.group, hh = (row0 + r) - d * p.group;
          p.lse[(int64_t)(g.seq.start + d) * p.hq + g.head * p.group + hh] = l == 0.f ? -INFINITY : kLn2 * (m + (log2f(l) - C::Lift));
        }
        tc::fence_before_sync();
        named_sync(1, 256);
        constexpr int LPR = D / 8;
        const int ch = threadIdx.x % LPR;
#pragma unroll 1
        for (int q = threadIdx.x / LPR; q < rows; q += 256 / LPR) {
          const int d = (row0 + q) / p.group, hh = (row0 + q) - d * p.group;
          *reinterpret_cast<uint4*>(p.out + (g.seq.start + d) * p.out_stride + (int64_t)(g.head * p.group + hh) * D + 8 * ch) =
              *reinterpret_cast<const uint4*>(sq + q * (D * 2) + ((ch ^ (q & 7)) << 4));
        }
        ++seg;
        continue;
      }
      // a part, for the joining kernel
      float* part = p.part + (int64_t)tree_slot(cta, g.tile0 == 0) * tree_part_floats(kRows, D);
      if (active)
#pragma unroll 1
        for (int col = col0; col < col0 + cols; col += 32) {
          float v[32];
          fetch(col, v);
          if (valid)
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(part + ((int64_t)(col + j) / 4 * kRows + r) * 4) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      if (valid && s == 0) {
        part[(int64_t)kRows * D + r] = m;
        part[(int64_t)kRows * D + kRows + r] = l;
      }
      tc::fence_before_sync();
      if (threadIdx.x == 0 && g.first == cta) shared_item = make_int4(g.b, g.head, g.row_block, g.last);
      ++seg;
    }
    if (threadIdx.x == 0) p.items[cta] = shared_item;
  }
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && flags[0]) atomicCAS(&g_tree_tc1_error, 0, 3);
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int D, bool F8>
cudaError_t launch_one(const CUtensorMap& map, const TreeParams& p, int ctas, cudaStream_t st) {
  using C = Cfg<D, F8>;
  auto kern = tree_tc1_kernel<D, F8>;
  static PerDevice<cudaError_t> attr_of;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const cudaError_t e = attr_of.get(dev, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem);
  }, cudaErrorInvalidDevice);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = launch_pdl(kern, dim3((unsigned)ctas), dim3(C::Threads), C::Smem, st, map, p);
  return e2 != cudaSuccess ? e2 : launch_tree_join(p, D, kRows, C::Lift, ctas, st);
}

}  // namespace

bool tree_tc1_fits(const trellis_cache_t& c, int rows) { return rows > 16 && (c.dtype == TRELLIS_E4M3 || c.head_dim == 256); }

int tree_tc1_rows() { return kRows; }

void tree_tc1_box(const trellis_cache_t& c, TreeBox* b) {
  const int tile = c.head_dim == 256 ? 64 : 128;
  b->rows = c.page_size < tile ? c.page_size : tile;
  b->bytes = c.dtype == TRELLIS_E4M3 ? c.head_dim : 128;
  b->swizzled = c.dtype != TRELLIS_E4M3;
}

cudaError_t launch_tree_tc1(const CUtensorMap& map, const TreeParams& p, const trellis_cache_t& c, int ctas, cudaStream_t st) {
  if (c.dtype != TRELLIS_E4M3) return launch_one<256, false>(map, p, ctas, st);
  if (c.head_dim == 64) return launch_one<64, true>(map, p, ctas, st);
  if (c.head_dim == 128) return launch_one<128, true>(map, p, ctas, st);
  return launch_one<256, true>(map, p, ctas, st);
}

int read_tree_tc1_error(int reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_tree_tc1_error, sizeof(int)) != cudaSuccess) return -1;
  if (reset && v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_tree_tc1_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

}  // namespace trellis

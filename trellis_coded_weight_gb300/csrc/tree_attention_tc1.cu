// tree_attention_tc1.cu -- tree attention with the 5th-generation tensor cores for e4m3 caches (any head dim) and heads of
// 256, where tree_attention_tc.cu's two accumulators do not fit.
//
// As there, S = Q K^T and O += P V are tcgen05 MMAs of one issuing warp, P lies in tensor memory over its scores (and Q lies
// there too: that leaves shared memory to the rings of tiles), and two softmax warpgroups alternate between the tiles, a
// thread per row.  Here a block has 128 rows and one accumulator O, so the
// maximum in use is one per row: the warp that has tile i hands its rows' maxima to the warp that has tile i + 1 (an mbarrier
// per warp), before it makes its weights; the groups' sums of weights stay apart until the end.
//
// An e4m3 cache is copied as it is.  The scores' MMAs read its keys as they are: Q is split into two 8-bit numbers (each row
// scaled by a power of two first), S = Qhi K^T + Qlo K^T at twice the 16-bit rate.  Qhi is e4m3, with 4 of Q's 8 significant
// bits; what it leaves is a whole number of at most 8 in Q's last place, which e5m2's 3 significant bits hold exactly, and e5m2
// reaches 2^7 further down.  The split is exact down to 2^-13 of the row's largest number, and within 2^-21 of it below, where
// Qhi has fewer bits.  (With e4m3 for Qlo too, 2^-9 and 2^-17: the lse of a row of 256 with one number 2^14 times the others
// was off by 0.13.)  The values become fp16 in shared memory, by a warpgroup of its own (exact), since weights of 4 bits would not do; P is fp16
// then.  That group also clears what must not reach a product.
// Bound: the chain of a tile's scores, weights, conversion and products, 2000 cycles per tile of 64 keys where HBM would take
// 1400: 32 x 4 drafts, ragged to 8200 e4m3 keys, 16/2 heads of 256: 40 us (3.0 TB/s); 1 x 4 drafts, 131072 keys 40 us, bf16 52
// (5.2 TB/s).  Repeating few rows in the lanes that idle, each copy with its part of a tile's keys, made the weights of a tile
// four times as fast and the whole no faster (43 and 49 us): the join of the copies costs more than the chain gains.
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
constexpr int kSoftmaxWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kConvertWarp = 10;
constexpr int kConvertThreads = 128;  // rows of a tile are 8, 16 or 32 apart in a thread's chunks: what it swizzles by stays the same
// an item's start and end, in steps (32 x 4 drafts, ragged to 8200 e4m3 keys, 16/2 heads of 256: 54 us without, 42)
constexpr int kExtra = 7;
constexpr int kOdd = 8;     // segments whose odd values are known at a time

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
  static constexpr int KBytes = D * (F8 ? 1 : 2);           // a key
  static constexpr int KBlock = KBytes < 128 ? KBytes : 128;  // of it in one swizzled row
  static constexpr int KSlot = Tile * KBytes;
  static constexpr int VSlot = Tile * D * 2;                // a tile's values, 16 bits
  static constexpr int RSlot = F8 ? Tile * D : 0;           // as the cache has them
  static constexpr int Threads = F8 ? 448 : 384;
  static constexpr int KSlots = 3, VSlots = 3, RSlots = F8 ? 3 : 0;
  static constexpr int Stage = 32 * D * 2;                  // 32 rows of queries: bf16, or two 8-bit numbers
  static_assert(VSlots + 1 < kOdd, "the converting warps are at most the values' slots and a tile ahead");
  static constexpr int Fixed = Stage + 32 * 4 + kRows * 4 * 3 + (int)sizeof(TreeMap) + 1024;
  static constexpr int Smem = 1024 + KSlots * KSlot + VSlots * VSlot + RSlots * RSlot + Fixed;
  static_assert(Smem <= 227 * 1024, "fits");
  // tensor memory columns: scores, outputs, queries
  static constexpr int S(int s) { return s * Tile; }
  static constexpr int O = 256;
  static constexpr int Q = D == 256 ? 128 : 384;
  static constexpr float Lift = F8 ? 7.f : 0.f;             // fp16 weights reach 2^15: 2^kMove times this
  static constexpr uint32_t KSwizzle = KBlock == 128 ? 2 : 4;  // descriptor: 128-byte or 64-byte
};

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::Threads, 1)
    tree_tc1_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TreeParams p) {
  using C = Cfg<D, F8>;
  constexpr int kTile = C::Tile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* keys = base;
  uint8_t* values = keys + C::KSlots * C::KSlot;
  uint8_t* raws = values + C::VSlots * C::VSlot;
  uint8_t* stage = raws + C::RSlots * C::RSlot;
  float* row_fac = reinterpret_cast<float*>(stage + C::Stage);
  float* row_max = row_fac + 32;          // in use
  float* row_sum = row_max + kRows;       // [2][rows]
  TreeMap& seqs = *reinterpret_cast<TreeMap*>(row_sum + 2 * kRows);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(&seqs + 1);
  uint64_t* k_empty = k_full + 4;
  uint64_t* v_full = k_empty + 4;
  uint64_t* v_empty = v_full + 4;
  uint64_t* r_full = v_empty + 4;   // e4m3: the values as copied
  uint64_t* r_empty = r_full + 4;
  uint64_t* q_ready = r_empty + 4;
  uint64_t* s_full = q_ready + 1;   // [2] a tile's scores; also: the products of the tile two before it are complete
  uint64_t* p_ready = s_full + 2;   // [2] weights written
  uint64_t* o_done = p_ready + 2;   // each tile's product with the values
  uint64_t* o_full = o_done + 1;    // the segment's last one
  uint64_t* drained = o_full + 1;
  uint64_t* turn = drained + 1;     // [2][4] a warp's row maxima of its tile
  volatile int* flags = reinterpret_cast<volatile int*>(turn + 8);  // [0] a wait gave up
  volatile int* odd_of = flags + 4;  // [segment % kOdd] the segment, if it has odd values
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(flags) + 4 + kOdd);

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&map);
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(k_full + i, 1);
      tc::mbar_init(k_empty + i, 1);
      tc::mbar_init(v_full + i, F8 ? kConvertThreads / 32 : 1);
      tc::mbar_init(v_empty + i, 1);
      tc::mbar_init(r_full + i, 1);
      tc::mbar_init(r_empty + i, kConvertThreads / 32);
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
    for (int i = 0; i < kOdd; ++i) odd_of[i] = -1;
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  pdl_enter();
  if (warp == 0) tree_cumulate<kRows, kTile, false, kExtra>(p, seqs);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(*tmem_slot);
  const int total = seqs.cum[p.batch];
  const int cta = blockIdx.x;
  const int ctas = tree_ctas_used<kRows, false>(p, total, (int)gridDim.x);
  TreeWalk<kRows, kTile, false> walk(total, ctas, cta);
  TreeSegment g;

  if (warp >= kSoftmaxWarps) {
    if (warp == kCopyWarp) {
      // ---- the copying warp: keys, and values (e4m3: to be converted), tiles in the order of their use
      int t0 = 0, copied[2] = {0, 0};
      bool dead = false;
      const int box = min(1 << p.page_shift, kTile);  // rows of one copy
      while (!dead && walk.next(p, seqs, g)) {
        TreePages<kTile> pages(p, g, lane);
        const int len = g.seq.prefix + g.seq.count;
        const Order order{g.tiles, true};
        for (int e = 0; e < 2 * g.tiles; ++e) {
          bool value;
          const int t = order.at(e, &value), tile = t0 + t;
          const int slots = !value ? C::KSlots : F8 ? C::RSlots : C::VSlots, s = tile % slots, use = tile / slots;
          uint64_t* const bar = (!value ? k_full : F8 ? r_full : v_full) + s;
          const int pos = (g.tile0 + t) * kTile + lane * box;  // lane i copies box i of the tile, none past the end
          const bool mine = lane * box < kTile && pos < len;
          int y = 0, page = pages.at(t);
          if (mine) {
            page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
            y = (((page * 2 + (value ? 1 : 0)) * p.hkv + g.head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
          }
          const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, mine));
          if (use > 0) {
            const bool ok = tc::mbar_wait_short((!value ? k_empty : F8 ? r_empty : v_empty) + s, (uint32_t)(use & 1) ^ 1u, p.wait_ns);
            if (__any_sync(0xFFFFFFFFu, !ok)) {
              dead = true;
              if (lane == 0) flags[0] = 1;
              break;
            }
          }
          if (lane == 0) tc::mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * C::KBytes));
          __syncwarp();
          copied[value ? 1 : 0] = tile + 1;
          if (mine) {
            uint8_t* const to = !value ? keys + s * C::KSlot : F8 ? raws + s * C::RSlot : values + s * C::VSlot;
#pragma unroll
            for (int blk = 0; blk < C::KBytes / C::KBlock; ++blk)
              tc::tma_load_2d(to + blk * (kTile * C::KBlock) + lane * box * C::KBlock, &map, bar, blk * (F8 ? C::KBlock : C::KBlock / 2), y);
          }
        }
        t0 += g.tiles;
      }
      // no copy may land in a block that has left
      for (int kv = 0; kv < 2; ++kv) {
        const int slots = kv == 0 ? C::KSlots : F8 ? C::RSlots : C::VSlots;
        for (int t = max(0, copied[kv] - slots); t < copied[kv]; ++t)
          tc::mbar_wait((kv == 0 ? k_full : F8 ? r_full : v_full) + t % slots, (uint32_t)(t / slots & 1), kDrainNs);
      }
    } else if (warp == kMmaWarp) {
      // ---- the warp that issues the products
      bool dead = false, issued = false;
      int seg = 0;
      uint32_t ks = 0, kuse = 0, vs = 0, vuse = 0, ns[2] = {0, 0};  // next slots
      const auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = dead || tc::mbar_wait_short(bar, parity, p.wait_ns);
        if (__any_sync(0xFFFFFFFFu, !ok)) {
          dead = true;
          flags[0] = 1;
        }
        return !dead;
      };
      // type fields: bf16 1, fp16 0 of kind::f16; e4m3 0, e5m2 1 of kind::f8f6f4 (of A from bit 7, of B from bit 10)
      constexpr uint32_t kType = F8 ? ~((1u << 7) | (1u << 10)) : ~0u;
      const uint32_t id_s = tc::idesc_bf16_f32(128, kTile) & kType, id_o = (tc::idesc_bf16_f32(128, D) & kType) | kBMnMajor;
      const uint64_t k_desc = tc::desc_kmajor(tc::smem_u32(keys), 8 * C::KBlock, C::KSwizzle),
                     v_desc = desc_mnmajor(tc::smem_u32(values), kTile * 128);
      const auto scores = [&](int s) {
        if (!wait(k_full + ks, kuse & 1u)) return;
        const uint64_t b = k_desc + ks * (C::KSlot >> 4);
#pragma unroll
        for (int h = 0; h < (F8 ? 2 : 1); ++h)
#pragma unroll
          for (int k = 0; k < C::KBytes / 32; ++k) {
            constexpr int kPer = C::KBlock / 32;
            const uint32_t qa = tmem + C::Q + h * (D / 4) + 8 * k;
            const uint64_t ka = b + (uint32_t)((k / kPer * (kTile * C::KBlock) + k % kPer * 32) >> 4);
            if constexpr (F8) mma_ts_f8(tmem + C::S(s), qa, ka, h == 0 ? id_s : id_s | 1u << 7, h > 0 || k > 0);
            else mma_ts(tmem + C::S(s), qa, ka, id_s, k > 0);
          }
        mma_done(s_full + s);
        mma_done(k_empty + ks);
        issued = true;
        if (++ks == C::KSlots) {
          ks = 0;
          ++kuse;
        }
      };
      while (!dead && __any_sync(0xFFFFFFFFu, walk.next(p, seqs, g))) {
        const int n = uniform(g.tiles);
        if (!wait(q_ready, (uint32_t)(seg & 1))) break;
        tc::fence_after_sync();
        for (int i = 0; i < 2 && i < n; ++i) scores(i);
        for (int i = 0; i < n; ++i) {
          const int s = i & 1;
          if (!wait(v_full + vs, vuse & 1u) || !wait(p_ready + s, ns[s] & 1u)) break;
          ++ns[s];
          tc::fence_after_sync();
          const uint64_t b = v_desc + vs * (C::VSlot >> 4);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ts(tmem + C::O, tmem + C::S(s) + 8 * k, b + (uint32_t)((k * 16 * 128) >> 4), id_o, i > 0 || k > 0);
          mma_done(o_done);
          mma_done(v_empty + vs);
          if (++vs == C::VSlots) {
            vs = 0;
            ++vuse;
          }
          if (i + 1 == n) mma_done(o_full);
          if (i + 2 < n) scores(s);
        }
        ++seg;
      }
      // tensor memory is given back once every product issued has completed, also where a wait gave up
      if (issued) {
        mma_done(drained);
        tc::mbar_wait(drained, 0, kDrainNs);
      }
    } else if (F8 && warp >= kConvertWarp) {
      // ---- values, e4m3 to fp16, tile by tile
      const int tid = threadIdx.x - kConvertWarp * 32, row0 = tid / (D / 16), ch = tid % (D / 16);
      constexpr int kBlockChunks = C::KBlock / 16;  // of a swizzled row
      const int from_at = ch / kBlockChunks * (kTile * C::KBlock) + row0 * C::KBlock +
                          ((ch % kBlockChunks) ^ (C::KBlock == 128 ? row0 & 7 : row0 >> 1 & 3)) * 16;
      // a chunk becomes two; eight lanes write eight different places of the banks: half of them their second one first
      const int flip = ch >> 2 & 1, to_at = (ch >> 2) * (kTile * 128) + row0 * 128;
      const int to_first = to_at + (((2 * ch + flip) & 7) ^ (row0 & 7)) * 16, to_second = to_at + (((2 * ch + (flip ^ 1)) & 7) ^ (row0 & 7)) * 16;
      int tile = 0, seg = 0;
      bool dead = false;
      const auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = dead || tc::mbar_wait_short(bar, parity, p.wait_ns);
        if (__any_sync(0xFFFFFFFFu, !ok)) {
          dead = true;
          if (lane == 0) flags[0] = 1;
        }
        return !dead;
      };
      while (!dead && walk.next(p, seqs, g)) {
        const int len = g.seq.prefix + g.seq.count;
        for (int t = 0; t < g.tiles; ++t, ++tile) {
          constexpr int kR = F8 ? C::RSlots : 1;
          const int rs = tile % kR, vs = tile % C::VSlots;
          if (!wait(r_full + rs, (uint32_t)(tile / kR & 1))) break;
          const uint8_t* from = raws + rs * C::RSlot + from_at;
          uint8_t* to = values + vs * C::VSlot;
          const int pos0 = (g.tile0 + t) * kTile;
          const bool tail = pos0 + kTile > g.seq.prefix;
          constexpr int CPR = D / 16, kMine = kTile * CPR / kConvertThreads;  // 16-byte chunks of a row, of this thread
          constexpr int kRowsApart = kConvertThreads / CPR;
          static_assert(kRowsApart % 8 == 0 && kTile % kRowsApart == 0, "a thread's chunks");
          uint4 u[kMine];
#pragma unroll
          for (int k = 0; k < kMine; ++k) u[k] = *reinterpret_cast<const uint4*>(from + k * (kRowsApart * C::KBlock));
          if (tail) {
            // rows past the end, and numbers of drafts that are none (the only ones e4m3 has), become zeros
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
              const int row = row0 + k * kRowsApart;
              if (pos0 + row >= len) u[k] = make_uint4(0, 0, 0, 0);
              else if (pos0 + row >= g.seq.prefix) {
                uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w}, odd = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const uint32_t nan = ((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // the top bit of such bytes
                  odd |= nan;
                  w[j] &= ~((nan >> 7) * 0xFFu);
                }
                u[k] = make_uint4(w[0], w[1], w[2], w[3]);
                if (odd) odd_of[seg % kOdd] = seg;
              }
            }
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(r_empty + rs);
          if (tile >= C::VSlots && !wait(v_empty + vs, (uint32_t)(tile / C::VSlots & 1) ^ 1u)) break;
#pragma unroll
          for (int k = 0; k < kMine; ++k) {
            const uint32_t w[4] = {flip ? u[k].z : u[k].x, flip ? u[k].w : u[k].y, flip ? u[k].x : u[k].z, flip ? u[k].y : u[k].w};
            *reinterpret_cast<uint4*>(to + to_first + k * (kRowsApart * 128)) =
                make_uint4(e4m3x2_to_f16x2(w[0]), e4m3x2_to_f16x2(w[0] >> 16), e4m3x2_to_f16x2(w[1]), e4m3x2_to_f16x2(w[1] >> 16));
            *reinterpret_cast<uint4*>(to + to_second + k * (kRowsApart * 128)) =
                make_uint4(e4m3x2_to_f16x2(w[2]), e4m3x2_to_f16x2(w[2] >> 16), e4m3x2_to_f16x2(w[3]), e4m3x2_to_f16x2(w[3] >> 16));
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(v_full + vs);
        }
        ++seg;
      }
    }
  } else {
    // ---- softmax: group s, one thread per row; warp w of a group reaches tensor memory lanes 32 w ..
    const int s = warp >> 2, w4 = warp & 3, r = w4 * 32 + lane;
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const uint32_t t_s = tmem + C::S(s) + lanes, t_o = tmem + C::O + lanes;
    int t0 = 0, seg = 0, ns = 0, turns = 0;  // turns: the other group's hand-overs of this warp's rows so far
    int4 shared_item = make_int4(0, 0, 0, 0);
    bool dead = false;
    const auto wait = [&](uint64_t* bar, int count) {
      const bool ok = dead || tc::mbar_wait_short(bar, (uint32_t)(count & 1), p.wait_ns);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        dead = true;
        if (lane == 0) flags[0] = 1;
      }
    };
    while (walk.next(p, seqs, g)) {
      const int row0 = g.row_block * kRows, rows = min(kRows, g.seq.count * p.group - row0), n = g.tiles;
      const int len = g.seq.prefix + g.seq.count;
      const float k_scale = F8 && p.scales ? __ldg(p.scales + g.head) : 1.f;
      const uint32_t flip = (p.scale_log2 < 0.f) != (k_scale < 0.f) ? 0x80008000u : 0u;  // a negative scale goes into the queries' signs
      const bool valid = r < rows, active = w4 * 32 < rows;  // warps without a row only keep the count
      const int draft = tree_draft(p, row0 + r), qhead = g.head * p.group + row0 + r - draft * p.group;
      // ---- queries, 32 rows at a time: loaded along the rows, staged, and put into tensor memory by the warps that own the rows,
      // each of the two with half of what is there (bf16: half of the row; e4m3: Qhi, Qlo)
      float fac = 1.f;
      {
        constexpr int LPR = D / 8, kStep = 256 / LPR, kMost = 32 / kStep;  // lanes of a row, rows at a time, loads of a thread
        const int l = threadIdx.x % LPR;
#pragma unroll 1
        for (int rb = 0; rb < rows; rb += 32) {
          uint4 u[kMost];
#pragma unroll
          for (int k = 0; k < kMost; ++k) {
            const int q = rb + k * kStep + threadIdx.x / LPR, d = tree_draft(p, row0 + q), hh = row0 + q - d * p.group;
            u[k] = make_uint4(0, 0, 0, 0);
            if (q < rows) u[k] = *reinterpret_cast<const uint4*>(p.q + (g.seq.start + d) * p.q_stride + (int64_t)(g.head * p.group + hh) * D + 8 * l);
          }
          if (rb > 0) named_sync(1, 256);  // the rows before have been taken
#pragma unroll
          for (int k = 0; k < kMost; ++k) {
            const int q = k * kStep + threadIdx.x / LPR;
            const uint4 v = make_uint4(u[k].x ^ flip, u[k].y ^ flip, u[k].z ^ flip, u[k].w ^ flip);
            uint8_t* const to = stage + q * (D * 2);
            if constexpr (F8) {
              uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
#pragma unroll
              for (int o = LPR / 2; o; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, o));
              // the row's largest number to [2^7, 2^8)
              uint32_t e = max(m2 & 0xFFFFu, m2 >> 16) >> 7;
              const bool none = e == 255;     // infinite or NaN: so are the row's results
              e = none ? 134u : max(e, 8u);   // below 2^-119 the factor is its smallest, 2^-126
              const float inv = __uint_as_float((261u - e) << 23);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float a = bf16lo_to_f32(w[i]) * inv, b = bf16hi_to_f32(w[i]) * inv;
                hi[i] = none ? 0x7F7Fu : e4m3x2(a, b);
                const uint32_t back = e4m3x2_to_f16x2(hi[i]);
                lo[i] = e5m2x2(a - f16_to_f32((uint16_t)back), b - f16_to_f32((uint16_t)(back >> 16)));
              }
              if (l == 0) row_fac[q] = __uint_as_float((e - 7u) << 23);
              const int ch = l >> 1, at = (l & 1) * 8;
              *reinterpret_cast<uint2*>(to + ((ch ^ (q & 3)) << 4) + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
              *reinterpret_cast<uint2*>(to + D + ((ch ^ (q & 3)) << 4) + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            } else {
              *reinterpret_cast<uint4*>(to + ((l ^ (q & 7)) << 4)) = v;
            }
          }
          named_sync(1, 256);
          if (w4 == rb >> 5) {
            constexpr int kChunks = D / 16 < 8 ? D / 16 : 8;  // of 16 bytes, at a time
            const int sw = F8 ? lane & 3 : lane & 7;
            if constexpr (F8) fac = row_fac[lane];
#pragma unroll 1
            for (int c0 = 0; c0 < D / 16; c0 += kChunks) {
              uint32_t y[4 * kChunks];
#pragma unroll
              for (int k = 0; k < kChunks; ++k) {
                const int ch = s * (D / 16) + ((c0 + k) ^ sw);
                const uint4 v = *reinterpret_cast<const uint4*>(stage + lane * (D * 2) + (ch << 4));
                y[4 * k] = v.x;
                y[4 * k + 1] = v.y;
                y[4 * k + 2] = v.z;
                y[4 * k + 3] = v.w;
              }
              const uint32_t to = tmem + C::Q + lanes + s * (D / 4) + 4 * c0;
              if constexpr (kChunks == 8) tmem_st_x32(to, y);
              else tmem_st_x16(to, y);
            }
            tmem_st_wait();
          }
        }
      }
      const uint64_t seen = !valid ? 0ull : p.mask ? p.mask[g.seq.start + draft] : draft >= 63 ? ~0ull : (2ull << draft) - 1;
      // this thread is past the segment before, and so is all that it read of it
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(q_ready);
      // the row's factor first: a small scale is that of large queries
      const float c = score_factor(fabsf(p.scale_log2) * fac * fabsf(k_scale));
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
          // ---- the row's maximum.  Both passes over the scores are loops over 64 columns: reading tensor memory twice costs less
          // than the registers and the code of a step held whole, and a loop over 32 waits twice as often.
          uint32_t x[2][32];
          float mx = -INFINITY;
          const auto largest = [&](const uint32_t (&v)[32]) {
            float a = __uint_as_float(v[0]), b = __uint_as_float(v[1]);
#pragma unroll
            for (int j = 2; j < 30; j += 4) {
              a = fmaxf(fmaxf(a, __uint_as_float(v[j])), __uint_as_float(v[j + 1]));
              b = fmaxf(fmaxf(b, __uint_as_float(v[j + 2])), __uint_as_float(v[j + 3]));
            }
            mx = fmaxf(mx, fmaxf(fmaxf(a, b), fmaxf(__uint_as_float(v[30]), __uint_as_float(v[31]))));
          };
#pragma unroll 1
          for (int w = 0; w < W; w += 2) {
            tc::tmem_ld_32x32b_x32(t_s + 32 * w, x[0]);
            tc::tmem_ld_32x32b_x32(t_s + 32 * w + 32, x[1]);
            tc::tmem_ld_wait();
            largest(x[0]);
            largest(x[1]);
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
            wait(o_done, t0 + i - 1);  // (the product before that is known to be complete)
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
          // ---- weights, over the scores; 16 bits as in tree_attention.cu, of the type that the values have here
          const float ms = m == -INFINITY ? C::Lift : C::Lift - m;
          float2 sum = make_float2(0.f, 0.f);
          const auto weigh = [&](const uint32_t (&v)[32], int w) {
            uint32_t e[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float2 y = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), make_float2(c, c), make_float2(ms, ms));
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              sum = __fadd2_rn(sum, y);
              e[j >> 1] = F8 ? pack_f16x2(y.x, y.y) : pack_bf16x2(y.x, y.y);
            }
            tmem_st_x16(t_s + 16 * w, e);
          };
#pragma unroll 1
          for (int w = 0; w < W; w += 2) {
            tc::tmem_ld_32x32b_x32(t_s + 32 * w, x[0]);
            tc::tmem_ld_32x32b_x32(t_s + 32 * w + 32, x[1]);
            tc::tmem_ld_wait();
            weigh(x[0], w);
            weigh(x[1], w + 1);
          }
          l += sum.x + sum.y;
          tmem_st_wait();
        }
        if constexpr (!F8) {
          const int pos0 = (g.tile0 + i) * kTile;
          if (pos0 + kTile > g.seq.prefix) {
            // Values that must not reach a product: rows past the end become zeros, whatever their bits; so do numbers of
            // drafts that are not finite (rare), which are added at the end to the rows that see them.
            const int vs = (t0 + i) % C::VSlots;
            wait(v_full + vs, (t0 + i) / C::VSlots);
            uint8_t* tile = values + vs * C::VSlot;
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
                odd_of[seg % kOdd] = seg;
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
      t0 += n;
      if (active) turns += (n + s) >> 1;  // tiles of the other group: of group 0 (n + 1) / 2, of group 1 n / 2
      named_sync(1, 256);
      // the last tile's warp has left the final maxima: both groups bring their sums to them
      const float m = active ? row_max[r] : -INFINITY;
      // (l is 0 without a maximum, or NaN where all of the row's scores were: it stays)
      const float mine = used == -INFINITY ? l : l * ex2(used - m);
      row_sum[s * kRows + r] = mine;
      named_sync(1, 256);
      l = mine + row_sum[(1 - s) * kRows + r];
      const bool odd = odd_of[seg % kOdd] == seg;
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
            int page = p.table[(int64_t)g.b * p.width + (pos >> p.page_shift)];
            page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
            const int64_t first = (((int64_t)((page * 2 + 1) * p.hkv + g.head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1))) * D + col;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if constexpr (F8) {
                if ((static_cast<const uint8_t*>(p.pool)[first + k] & 0x7Fu) == 0x7Fu) v[k] = __int_as_float(0x7FC00000);
              } else {
                const uint16_t b = static_cast<const uint16_t*>(p.pool)[first + k];
                if ((b & 0x7F80u) == 0x7F80u) v[k] += bf16_to_f32(b);
              }
            }
          }
      };
      if (g.whole) {
        // finished here
        const float f = l == 0.f ? 0.f : (F8 && p.scales ? __ldg(p.scales + p.hkv + g.head) : 1.f) / l;
        uint16_t* const to = p.out + (int64_t)(g.seq.start + draft) * p.out_stride + (int64_t)qhead * D;
        if (active) {
#pragma unroll 1
          for (int col = col0; col < col0 + cols; col += 32) {
            float v[32];
            fetch(col, v);
            if (valid)
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                *reinterpret_cast<uint4*>(to + col + j) =
                    make_uint4(pack_bf16x2(v[j] * f, v[j + 1] * f), pack_bf16x2(v[j + 2] * f, v[j + 3] * f),
                               pack_bf16x2(v[j + 4] * f, v[j + 5] * f), pack_bf16x2(v[j + 6] * f, v[j + 7] * f));
          }
        }
        if (valid && s == 0 && p.lse)
          p.lse[(int64_t)(g.seq.start + draft) * p.hq + qhead] = l == 0.f ? -INFINITY : kLn2 * (m + (log2f(l) - C::Lift));
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
      if (threadIdx.x == 0 && g.starts) shared_item = tree_item(g, row0, rows, cta, tree_cta_of(g.last_at, total, ctas));
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

// heads of 256, which no other kernel takes, and an e4m3 cache from 17 rows on (measured at tree_attention.cu)
bool tree_tc1_fits(const trellis_cache_t& c, int rows) { return c.head_dim == 256 || (c.dtype == TRELLIS_E4M3 && rows > 16); }

int tree_tc1_rows() { return kRows; }

void tree_tc1_box(const trellis_cache_t& c, TreeBox* b) {
  const int tile = c.head_dim == 256 ? 64 : 128, bytes = (int)(c.head_dim * cache_elem_bytes(c));
  b->rows = c.page_size < tile ? c.page_size : tile;
  b->bytes = bytes < 128 ? bytes : 128;
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

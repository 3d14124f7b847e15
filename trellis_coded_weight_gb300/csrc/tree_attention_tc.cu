// tree_attention_tc.cu -- tree attention with the 5th-generation tensor cores, for more rows per key/value head than
// tree_attention.cu handles at the rate of HBM.
//
// The mathematics is that of tree_attention.cu.  A block takes up to 256 rows of one key/value head and 128 keys per
// step; both products are 128 x N tcgen05 MMAs of one issuing warp with accumulators in tensor memory:
//   S = Q K^T    Q and K in shared memory (128-byte swizzle, along the head dim)
//   O += P V     P in tensor memory over the scores it was made of, V in shared memory (swizzled, along the head dim too)
// Two softmax warpgroups, one thread per row, each own a stream of steps with its own S, O, maximum and sum:
//   up to 128 rows     both streams have the same rows and alternate between the tiles of keys, and are joined at the end
//   up to 256 rows     each has 128 of the rows, and both take every tile
// so that one stream's products run while the other's softmax does.  A stream's maximum is only moved when it has grown by
// more than 2^8: the weights then stay below 2^8, well inside bf16 and fp32, and O is rarely rescaled.
// Keys and values arrive by TMA in a ring of tiles in the order of their use.
// Bound: HBM up to 64 or so rows (16 drafts, 131072 keys, 32/8 heads of 128: 87 us, 6.2 TB/s).  With 256 rows the chain of
// scores, weights and products (a step of both streams 3200 cycles, of which its MMAs take 2150): 64 drafts, 131072 keys 112 us
// (1.2 PFLOP/s); 4 x 64 drafts, 16384 keys, 40/8 heads, where 64 of 320 rows read the cache once more: 115 us (0.75 PFLOP/s).
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

__device__ int g_tree_tc_error = 0;  // set when a bounded wait gives up (trellis_device_error)

constexpr int kTile = 128;                    // keys per step
constexpr int kRows = 256;                    // rows of a block
constexpr int kSoftmaxWarps = 8, kCopyWarp = 8, kMmaWarp = 9;
// an item's start and end, in steps (32 x 8 drafts, ragged to 2048 keys, 32/8 heads of 128: 74 us without, 35, 38 with 12)
constexpr int kExtra = 6;
constexpr int kThreads = 384;  // two softmax warpgroups; one for the copying and the issuing warp, and two that idle

template <int D>
struct Cfg {
  static constexpr int Blocks = D / 64;                     // 128-byte blocks of a row
  static constexpr int Slot = kTile * D * 2;                // the keys, or the values, of a tile
  static constexpr int QTile = 128 * D * 2;
  static constexpr int Fixed = 2 * QTile + kRows * 8 + 4 * 128 * 4 + (int)sizeof(TreeMap) + 512;
  static constexpr int Fit = (227 * 1024 - 1024 - Fixed) / Slot;
  static constexpr int Pairs = Fit >= 8 ? 4 : 2;            // tiles in flight, each in a slot for its keys and one for its values
  static constexpr int Slots = 2 * Pairs;
  static_assert(Fit >= Slots, "keys and values of two tiles");
  static constexpr int Smem = 1024 + Slots * Slot + Fixed;
  // tensor memory columns
  static constexpr int S(int s) { return s * 128; }
  static constexpr int O(int s) { return 256 + s * 128; }
};

// Tile i of a segment that begins at the block's tile t0 is in pair (t0 + i) % Pairs, as that pair's use (t0 + i) / Pairs.
// The number of pairs is even, so the use of a slot before a stream's tile is the same stream's, or of a finished segment:
// a thread that waits for a phase has seen the one before complete, as waits by parity need.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TreeParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = base;
  uint8_t* sq = ring + C::Slots * C::Slot;
  uint64_t* row_mask = reinterpret_cast<uint64_t*>(sq + 2 * C::QTile);
  float* row_stat = reinterpret_cast<float*>(row_mask + kRows);  // [stream][maximum, sum][128]
  TreeMap& seqs = *reinterpret_cast<TreeMap*>(row_stat + 4 * 128);
  uint64_t* full = reinterpret_cast<uint64_t*>(&seqs + 1);
  uint64_t* empty = full + C::Slots;
  uint64_t* q_ready = empty + C::Slots;
  uint64_t* s_full = q_ready + 1;  // [2] scores there; also: the stream's products before them are complete
  uint64_t* p_ready = s_full + 2;  // [2] weights written, values clean
  uint64_t* o_full = p_ready + 2;  // [2] the segment's last product complete
  uint64_t* drained = o_full + 2;
  volatile int* flags = reinterpret_cast<volatile int*>(drained + 1);  // [0] a wait gave up, [2] segment with odd values
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(flags) + 4);

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&map);
    for (int i = 0; i < C::Slots; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, 2);  // both streams, or one twice
    }
    tc::mbar_init(q_ready, kSoftmaxWarps);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(s_full + s, 1);
      tc::mbar_init(p_ready + s, kSoftmaxWarps / 2);
      tc::mbar_init(o_full + s, 1);
    }
    tc::mbar_init(drained, 1);
    flags[0] = 0;
    flags[2] = -1;
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  pdl_enter();
  if (warp == 0) tree_cumulate<kRows, kTile, true, kExtra>(p, seqs);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(*tmem_slot);
  const int total = seqs.cum[p.batch];
  const int cta = blockIdx.x;
  const int ctas = tree_ctas_used<kRows, true>(p, total, (int)gridDim.x);
  TreeWalk<kRows, kTile, true> walk(total, ctas, cta);
  TreeSegment g;
  const auto rows_of = [&](const TreeSegment& x) { return min(kRows, x.seq.count * p.group - x.row_block * kRows); };

  if (warp >= kSoftmaxWarps) {
  if (warp == kCopyWarp) {
    // ---- the copying warp
    int t0 = 0, copied[2] = {0, 0};  // keys, values
    bool dead = false;
    const int box = min(1 << p.page_shift, kTile);  // rows of one copy
    while (!dead && walk.next(p, seqs, g)) {
      TreePages<kTile> pages(p, g, lane);
      const int len = g.seq.prefix + g.seq.count;
      const Order order{g.tiles, rows_of(g) <= 128};
      for (int e = 0; e < 2 * g.tiles; ++e) {
        bool value;
        const int t = order.at(e, &value);
        const int s = (t0 + t) % C::Pairs * 2 + (value ? 1 : 0), use = (t0 + t) / C::Pairs;
        const int pos = (g.tile0 + t) * kTile + lane * box;  // lane i copies box i of the tile, none past the end
        const bool mine = lane * box < kTile && pos < len;
        int y = 0, page = pages.at(t);
        if (mine) {
          page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
          y = (((page * 2 + (value ? 1 : 0)) * p.hkv + g.head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        }
        const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, mine));
        if (use > 0) {
          const bool ok = tc::mbar_wait_short(empty + s, (uint32_t)(use & 1) ^ 1u, p.wait_ns);
          if (__any_sync(0xFFFFFFFFu, !ok)) {
            dead = true;
            if (lane == 0) flags[0] = 1;
            break;
          }
        }
        if (lane == 0) tc::mbar_arrive_expect_tx(full + s, (uint32_t)(boxes * box * D * 2));
        __syncwarp();
        copied[value ? 1 : 0] = t0 + t + 1;
        if (mine)
#pragma unroll
          for (int blk = 0; blk < C::Blocks; ++blk)
            tc::tma_load_2d(ring + s * C::Slot + blk * (kTile * 128) + lane * box * 128, &map, full + s, blk * 64, y);
      }
      t0 += g.tiles;
    }
    // no copy may land in a block that has left
    for (int kv = 0; kv < 2; ++kv)
      for (int t = max(0, copied[kv] - C::Pairs); t < copied[kv]; ++t)
        tc::mbar_wait(full + t % C::Pairs * 2 + kv, (uint32_t)(t / C::Pairs & 1), kDrainNs);
  } else if (warp == kMmaWarp) {
    // ---- the warp that issues the products.  One for both streams: with one each, products of 256 rows measured
    // 153 us against 135 (1 x 64 drafts, 131072 keys).  The tensor cores queue only a few products ahead, so waits sit behind
    // products that are still queued where they can.
    bool dead = false, issued = false;
    int t0 = 0, seg = 0;
    uint32_t ns[2] = {0, 0};
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool ok = dead || tc::mbar_wait_short(bar, parity, p.wait_ns);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        dead = true;
        flags[0] = 1;
      }
      return !dead;
    };
    const uint32_t id_s = tc::idesc_bf16_f32(128, kTile), id_o = tc::idesc_bf16_f32(128, D) | kBMnMajor;
    const uint64_t q_desc = tc::desc_kmajor(tc::smem_u32(sq), 1024, 2), k_desc = tc::desc_kmajor(tc::smem_u32(ring), 1024, 2),
                   v_desc = desc_mnmajor(tc::smem_u32(ring), kTile * 128);
    // tile i's slot for keys (0) or values (1), and the wait for it
    const auto slot_of = [&](int i, uint32_t kv) { return (uint32_t)(t0 + i) % C::Pairs * 2 + kv; };
    const auto take = [&](int i, uint32_t kv) { return wait(full + slot_of(i, kv), (uint32_t)(t0 + i) / C::Pairs & 1u); };
    const auto scores = [&](int s, int qtile, int i) {
      const uint64_t a = q_desc + (uint32_t)(qtile * (C::QTile >> 4)), b = k_desc + slot_of(i, 0) * (C::Slot >> 4);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t step = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
        mma_ss(tmem + C::S(s), a + step, b + step, id_s, k > 0);
      }
      mma_done(s_full + s);
      issued = true;
    };
    const auto outputs = [&](int s, int i, bool fresh) {
      const uint64_t b = v_desc + slot_of(i, 1) * (C::Slot >> 4);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts(tmem + C::O(s), tmem + C::S(s) + 8 * k, b + (uint32_t)((k * 16 * 128) >> 4), id_o, !(fresh && k == 0));
    };
    const auto weights = [&](int s) {  // waits for the stream's
      if (!wait(p_ready + s, ns[s] & 1u)) return false;
      ++ns[s];
      tc::fence_after_sync();
      return true;
    };
    while (!dead && __any_sync(0xFFFFFFFFu, walk.next(p, seqs, g))) {
      const int n = uniform(g.tiles);
      if (!wait(q_ready, (uint32_t)(seg & 1))) break;
      tc::fence_after_sync();
      if (uniform(rows_of(g)) <= 128) {
        for (int i = 0; i < 2 && i < n; ++i)
          if (take(i, 0)) scores(i, 0, i);
        for (int i = 0; i < n; ++i) {
          const int s = i & 1;
          if (!take(i, 1) || !weights(s)) break;
          outputs(s, i, i < 2);
          mma_done(empty + slot_of(i, 1));  // its tile alone: free at once, for both counts
          mma_done(empty + slot_of(i, 1));
          if (i + 2 >= n) mma_done(o_full + s);
          else if (take(i + 2, 0)) scores(s, 0, i + 2);
        }
      } else {
        if (!take(0, 0)) break;
        scores(0, 0, 0);
        scores(1, 1, 0);
        if (!take(0, 1)) break;
        for (int i = 0; i < n; ++i) {
          const bool more = i + 1 < n;
          if (!weights(0)) break;
          outputs(0, i, i == 0);
          if (more) {
            if (!take(i + 1, 0)) break;
            scores(0, 0, i + 1);
          } else {
            mma_done(o_full);
          }
          if (!weights(1)) break;
          outputs(1, i, i == 0);
          if (more) {
            scores(1, 1, i + 1);
            if (!take(i + 1, 1)) break;
          } else {
            mma_done(o_full + 1);
          }
        }
      }
      t0 += n;
      ++seg;
    }
    // tensor memory is given back once every product issued has completed, also where a wait gave up
    if (issued) {
      mma_done(drained);
      tc::mbar_wait(drained, 0, kDrainNs);
    }
  }
  } else {
    // ---- softmax: stream s, one thread per row; warp w of a group reaches tensor memory lanes 32 w ..
    const int s = warp >> 2, lrow = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + C::S(s) + lanes, t_o = tmem + C::O(s) + lanes;
    const float c = score_factor(fabsf(p.scale_log2));
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale goes into the queries' signs
    int t0 = 0, seg = 0, ns = 0, no = 0;
    int4 shared_item = make_int4(0, 0, 0, 0);  // the item that starts here and ends in a later block
    bool dead = false;
    const auto wait = [&](uint64_t* bar, int count) {
      const bool ok = dead || tc::mbar_wait_short(bar, (uint32_t)(count & 1), p.wait_ns);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        dead = true;
        if (lane == 0) flags[0] = 1;
      }
    };
    while (walk.next(p, seqs, g)) {
      const int rows = rows_of(g), row0 = g.row_block * kRows, n = g.tiles;
      const Order order{n, rows <= 128};
      const int len = g.seq.prefix + g.seq.count;
      named_sync(1, 256);  // the segment before is finished: its queries, statistics and outputs are no longer read
      // ---- queries
      {
        constexpr int LPR = D / 8, kStep = 256 / LPR, kMost = D == 128 ? 8 : 4;  // lanes of a row, rows at a time, loads in flight
        const int qrows = (rows + 31) & ~31, l = threadIdx.x % LPR;  // whole warps' rows; what others hold does not matter
        for (int r0 = threadIdx.x / LPR; r0 < qrows; r0 += kStep * kMost) {
          uint4 u[kMost];
#pragma unroll
          for (int k = 0; k < kMost; ++k) {
            const int r = r0 + k * kStep, d = tree_draft(p, row0 + r), hh = row0 + r - d * p.group;
            u[k] = make_uint4(0, 0, 0, 0);
            if (r < rows) u[k] = *reinterpret_cast<const uint4*>(p.q + (g.seq.start + d) * p.q_stride + (int64_t)(g.head * p.group + hh) * D + 8 * l);
          }
#pragma unroll
          for (int k = 0; k < kMost; ++k) {
            const int r = r0 + k * kStep;
            if (r < qrows)
              *reinterpret_cast<uint4*>(sq + (r >> 7) * C::QTile + (l >> 3) * (128 * 128) + (r & 127) * 128 + (((l & 7) ^ (r & 7)) << 4)) =
                make_uint4(u[k].x ^ flip, u[k].y ^ flip, u[k].z ^ flip, u[k].w ^ flip);
          }
        }
        if (threadIdx.x < qrows) {
          const int r = threadIdx.x, d = tree_draft(p, row0 + r);
          row_mask[r] = r >= rows ? 0ull : p.mask ? p.mask[g.seq.start + d] : d >= 63 ? ~0ull : (2ull << d) - 1;
        }
        tc::fence_proxy_async_smem();
        named_sync(1, 256);  // masks
        if (lane == 0) tc::mbar_arrive(q_ready);
      }
      const int r = order.split_keys ? lrow : s * 128 + lrow;  // this thread's row of the block
      const uint64_t seen = row_mask[r];
      float m = -INFINITY, l = 0.f;  // the maximum in use, the sum
      const int first_tile = order.split_keys ? s : 0, tile_step = order.split_keys ? 2 : 1;
      const auto release = [&](int i, int kv) { tc::mbar_arrive(empty + (t0 + i) % C::Pairs * 2 + kv); };
      bool any = false;
      for (int i = first_tile; i < n; i += tile_step) {
        wait(s_full + s, ns++);
        tc::fence_after_sync();
        // Scores that are complete free their keys, and, as a stream's products complete in order, the values of its step before.
        if (threadIdx.x % 128 == 0 && !dead) {
          release(i, 0);
          if (order.split_keys) release(i, 0);
          else if (i > 0) release(i - 1, 1);
        }
        const int pos0 = (g.tile0 + i) * kTile;
        const bool tail = pos0 + kTile > g.seq.prefix;
        if (tail) {
          // scores that the row does not see become minus infinity, in place: columns before `from` are prefix, drafts
          // come after, then nothing
          const int from = g.seq.prefix - pos0;
          const uint64_t drafts = g.seq.count >= 64 ? seen : seen & ((1ull << g.seq.count) - 1);
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
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
        for (int w = 0; w < kTile / 32; w += 2) {
          tc::tmem_ld_32x32b_x32(t_s + 32 * w, x[0]);
          tc::tmem_ld_32x32b_x32(t_s + 32 * w + 32, x[1]);
          tc::tmem_ld_wait();
          largest(x[0]);
          largest(x[1]);
        }
        mx *= c;
        const bool move = mx > m + kMove || (m == -INFINITY && mx > -INFINITY);
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float to = move ? mx : m, a = m == to ? 1.f : ex2(m - to);
          l *= a;
          m = to;
          if (any) {
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
        }
        any = true;
        // ---- weights, over the scores; 16 bits as in tree_attention.cu: bf16, the type of the values they are multiplied with
        const float ms = m == -INFINITY ? 0.f : -m;
        float2 sum = make_float2(0.f, 0.f);
        const auto weigh = [&](const uint32_t (&v)[32], int w) {
          uint32_t e[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float2 y = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), make_float2(c, c), make_float2(ms, ms));
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            sum = __fadd2_rn(sum, y);
            e[j >> 1] = pack_bf16x2(y.x, y.y);
          }
          tmem_st_x16(t_s + 16 * w, e);
        };
#pragma unroll 1
        for (int w = 0; w < kTile / 32; w += 2) {
          tc::tmem_ld_32x32b_x32(t_s + 32 * w, x[0]);
          tc::tmem_ld_32x32b_x32(t_s + 32 * w + 32, x[1]);
          tc::tmem_ld_wait();
          weigh(x[0], w);
          weigh(x[1], w + 1);
        }
        l += sum.x + sum.y;
        tmem_st_wait();
        if (tail) {
          // Values that must not reach a product: rows past the end become zeros, whatever their bits; so do numbers of
          // drafts that are not finite (rare), which are added at the end to the rows that see them.
          const int slot = (t0 + i) % C::Pairs * 2 + 1;
          wait(full + slot, (t0 + i) / C::Pairs);
          uint8_t* tile = ring + slot * C::Slot;
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
              __threadfence_block();
              *at = v;
            }
          }
          tc::fence_proxy_async_smem();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_ready + s);
      }
      // ---- the segment's end
      if (any) {
        wait(o_full + s, no++);
        if (threadIdx.x % 128 == 0 && !dead && !order.split_keys) release(n - 1, 1);
      }
      tc::fence_after_sync();
      t0 += n;
      const bool valid = r < rows;
      float wa = 1.f, wb = 0.f;  // weights of the own stream's and the other's outputs
      bool other = false;
      int col0 = 0, cols = D;
      if (order.split_keys) {
        // both streams have the same rows: each finishes half of the columns
        row_stat[(s * 2) * 128 + lrow] = m;
        row_stat[(s * 2 + 1) * 128 + lrow] = l;
        tc::fence_before_sync();
        named_sync(1, 256);
        tc::fence_after_sync();
        const float om = row_stat[((1 - s) * 2) * 128 + lrow], ol = row_stat[((1 - s) * 2 + 1) * 128 + lrow];
        const float nm = fmaxf(m, om), bm = nm == -INFINITY ? 0.f : nm;
        wa = ex2(m - bm);
        wb = ex2(om - bm);
        l = l * wa + ol * wb;
        m = nm;
        other = s == 0 ? n > 1 : true;  // a single tile is stream 0's
        col0 = s * (D / 2);
        cols = D / 2;
      } else {
        named_sync(1, 256);
      }
      const bool own = any;
      const bool odd = flags[2] == seg;
      const uint32_t t_other = tmem + C::O(1 - s) + lanes;
      const auto fetch = [&](int col, float (&v)[32]) {  // 32 columns of the row, joined
        uint32_t x[32];
        if (own) {
          tc::tmem_ld_32x32b_x32(t_o + col, x);
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(x[j]) * wa;
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
        if (other) {
          tc::tmem_ld_32x32b_x32(t_other + col, x);
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(x[j]) * wb;
        }
        if (odd && valid)
          for (int j = 0; j < g.seq.count; ++j) {
            const int pos = g.seq.prefix + j, at = pos - g.tile0 * kTile;
            if (!(seen >> j & 1) || at < 0 || at >= n * kTile) continue;
            int page = p.table[(int64_t)g.b * p.width + (pos >> p.page_shift)];
            page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
            const uint16_t* vr = static_cast<const uint16_t*>(p.pool) + (((int64_t)((page * 2 + 1) * p.hkv + g.head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1))) * D + col;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint16_t b = vr[k];
              if ((b & 0x7F80u) == 0x7F80u) v[k] += bf16_to_f32(b);
            }
          }
      };
      if (g.whole) {
        // finished here: rows go through the queries' place (no longer read) so that a row's numbers are stored together
        const float f = l == 0.f ? 0.f : 1.f / l;
        uint8_t* stage = sq + (order.split_keys ? 0 : s * C::QTile) + lrow * (D * 2);
#pragma unroll 1
        for (int col = col0; col < col0 + cols; col += 32) {
          float v[32];
          fetch(col, v);
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            *reinterpret_cast<uint4*>(stage + ((((col + j) / 8) ^ (lrow & 7)) << 4)) =
                make_uint4(pack_bf16x2(v[j] * f, v[j + 1] * f), pack_bf16x2(v[j + 2] * f, v[j + 3] * f),
                           pack_bf16x2(v[j + 4] * f, v[j + 5] * f), pack_bf16x2(v[j + 6] * f, v[j + 7] * f));
        }
        if (valid && col0 == 0 && p.lse) {
          const int d = tree_draft(p, row0 + r), hh = row0 + r - d * p.group;
          p.lse[(int64_t)(g.seq.start + d) * p.hq + g.head * p.group + hh] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
        }
        tc::fence_before_sync();
        named_sync(1, 256);
        constexpr int LPR = D / 8;
        const int ch = threadIdx.x % LPR;
#pragma unroll 1
        for (int q = threadIdx.x / LPR; q < rows; q += 256 / LPR) {
          const int d = tree_draft(p, row0 + q), hh = row0 + q - d * p.group;
          *reinterpret_cast<uint4*>(p.out + (g.seq.start + d) * p.out_stride + (int64_t)(g.head * p.group + hh) * D + 8 * ch) =
              *reinterpret_cast<const uint4*>(sq + (q >> 7) * C::QTile + (q & 127) * (D * 2) + ((ch ^ (q & 7)) << 4));
        }
        ++seg;
        continue;
      }
      // a part, for the joining kernel
      float* part = p.part + (int64_t)tree_slot(cta, g.tile0 == 0) * tree_part_floats(kRows, D);
#pragma unroll 1
      for (int col = col0; col < col0 + cols; col += 32) {
        float v[32];
        fetch(col, v);
        if (valid)
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(part + ((int64_t)(col + j) / 4 * kRows + r) * 4) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      }
      if (valid && col0 == 0) {
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
  if (threadIdx.x == 0 && flags[0]) atomicCAS(&g_tree_tc_error, 0, 2);
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_d(const CUtensorMap& map, const TreeParams& p, int ctas, cudaStream_t st) {
  auto kern = tree_tc_kernel<D>;
  static PerDevice<cudaError_t> attr_of;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const cudaError_t e = attr_of.get(dev, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::Smem);
  }, cudaErrorInvalidDevice);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), Cfg<D>::Smem, st, map, p);
  return e2 != cudaSuccess ? e2 : launch_tree_join(p, D, kRows, 0.f, ctas, st);
}

}  // namespace

bool tree_tc_fits(const trellis_cache_t& c, int rows) { return c.dtype == TRELLIS_BF16 && c.head_dim <= 128 && rows > 16; }

int tree_tc_rows() { return kRows; }

void tree_tc_box(const trellis_cache_t& c, TreeBox* b) {
  b->rows = c.page_size < kTile ? c.page_size : kTile;
  b->bytes = 128;
}

cudaError_t launch_tree_tc(const CUtensorMap& map, const TreeParams& p, const trellis_cache_t& c, int ctas, cudaStream_t st) {
  return c.head_dim == 64 ? launch_d<64>(map, p, ctas, st) : launch_d<128>(map, p, ctas, st);
}

int read_tree_tc_error(int reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_tree_tc_error, sizeof(int)) != cudaSuccess) return -1;
  if (reset && v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_tree_tc_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

}  // namespace trellis

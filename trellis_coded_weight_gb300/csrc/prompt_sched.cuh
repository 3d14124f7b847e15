// prompt_sched.cuh -- how the work of a prompt attention call is divided over the GPU.
//
// An item is one key/value head of one sequence and one block of query rows (row r of a sequence and head: token r / group, query
// head r % group of the head's group); it takes one step per 128 keys up to the last one that its last row sees.  Lengths are
// device data, so every thread block plans for itself, in one of two ways:
//   whole  items by falling length, as good as sorted (sequences by falling length, each from its last block to its first); a
//          block takes the next one when it is about to be free (a counter).  What is finished late is then short.
//   split  where items are few or one of them would be longer than a block's share: the steps of all items end to end, cut into
//          equal contiguous ranges, as tree_sched.cuh does, with the parts of an item joined by the same second launch.
// Results do not depend on who computes an item; where one is cut is given by the lengths.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "tree_sched.cuh"

namespace trellis {
namespace prompt {

constexpr int kTile = 128;     // keys of a step
constexpr int kExtra = 2;      // an item's start and end, in steps
constexpr int kJoin = 12;      // what parts and their joining cost, in steps
constexpr int kLeast = 4;      // steps of a range at the least
constexpr int kEntries = 512;  // blocks of rows (of all sequences) that can be split
constexpr int kMaxSeqs = kTreeMaxBatch;

struct Map {
  static constexpr int kCached = 256;
  int4 seq[kCached];            // the first sequences: start, count, prefix
  int cum[kMaxSeqs + 1];        // blocks of rows before the i-th sequence of the order
  uint16_t order[kMaxSeqs];     // sequences by falling length
  int cost[kEntries + 1];       // split: steps before entry e (of all heads)
  int entries, items, total, ctas;
  bool split;
};

__device__ __forceinline__ TreeSeq seq_of(const TreeParams& p, const Map& m, int b) {
  if (b >= Map::kCached) return tree_seq(p, b);
  const int4 v = m.seq[b];
  return TreeSeq{v.x, v.y, v.z};
}

// What a thread block does next: a stretch of one item's steps.
struct Work {
  int b, head;
  int start, first, g0;  // the sequence's first token; the block's first row: its token (of the sequence) and head of the group
  int rows;
  int prefix, len;       // the sequence's
  int tile0, tiles, last;  // of the item's tiles 0 .. last these
  int until;             // the item's last thread block, where it is split
  int n0, n1;            // tiles that rows 0 .. 127, and 128 .. 255, take part in
  int shared0, shared1;  // keys that all of these rows see
  int more;              // 0: nothing is left
};

// Rows 0 .. r of a block: the last one's token, and the keys that it sees.
__device__ __forceinline__ int draft(const TreeParams& p, int x) { return p.group == 1 ? x : (int)__umulhi((uint32_t)x, (uint32_t)p.group_inv); }  // x / group
__device__ __forceinline__ int token_of(const TreeParams& p, const Work& w, int r) { return w.first + draft(p, w.g0 + r); }
__device__ __forceinline__ int seen_by(const TreeParams& p, const Work& w, int r) { return w.prefix + token_of(p, w, r) + 1; }
// Tiles of the stretch that rows r0 .. r1 - 1 (of a stream) take part in.
__device__ __forceinline__ int tiles_of(const TreeParams& p, const Work& w, int r0, int r1) {
  const int z = w.rows < r1 ? w.rows : r1;
  if (z <= r0) return 0;
  const int n = (seen_by(p, w, z - 1) + kTile - 1) / kTile - w.tile0;
  return n < 0 ? 0 : n < w.tiles ? n : w.tiles;
}

template <int ROWS>
__device__ __forceinline__ int blocks_of(const TreeParams& p, const TreeSeq& s) { return (s.count * p.group + ROWS - 1) / ROWS; }  // at most 2^30 rows
// Tiles of block rb of a sequence.
template <int ROWS>
__device__ __forceinline__ int item_tiles(const TreeParams& p, const TreeSeq& s, int rb) {
  const uint32_t z = (uint32_t)(rb + 1) * ROWS, all = (uint32_t)(s.count * p.group);
  return (s.prefix + (int)(((z < all ? z : all) - 1) / (uint32_t)p.group)) / kTile + 1;
}

// Fills the map; by all threads of the block.
template <int ROWS>
__device__ void plan(const TreeParams& p, Map& m, int grid, int* keys) {
  const int n = p.batch, tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  // sequences by falling length: the rank of each is the number of those that come before it
  for (int b = tid; b < kMaxSeqs; b += threads) {
    const TreeSeq s = b < n ? tree_seq(p, b) : TreeSeq{0, 0, 0};
    keys[b] = s.count ? s.prefix + s.count : 0;
    if (b < Map::kCached) m.seq[b] = make_int4(s.start, s.count, s.prefix, 0);
  }
  __syncthreads();
  for (int b = tid; b < n; b += threads) {
    const int mine = keys[b];
    int rank = 0;
    for (int i = 0; i < n; i += 4) {
      const int4 k = *reinterpret_cast<const int4*>(keys + i);
      rank += (k.x > mine || (k.x == mine && i < b)) + (i + 1 < n && (k.y > mine || (k.y == mine && i + 1 < b))) +
              (i + 2 < n && (k.z > mine || (k.z == mine && i + 2 < b))) + (i + 3 < n && (k.w > mine || (k.w == mine && i + 3 < b)));
    }
    m.order[rank] = (uint16_t)b;
  }
  __syncthreads();
  if (tid < 32) {
    int before = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      int v = 0;
      if (i0 + lane < n) v = blocks_of<ROWS>(p, seq_of(p, m, m.order[i0 + lane]));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
      }
      if (i0 + lane < n) m.cum[i0 + lane + 1] = before + v;
      before += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (lane == 0) {
      m.cum[0] = 0;
      m.entries = before;
      m.items = before * p.hkv;
      m.split = false;
      m.total = 0;
      m.ctas = grid;
    }
    __syncwarp();
    if (before > 0 && before <= kEntries && (int64_t)before * p.hkv < 3 * grid) {
      int sum = 0, most = 0;
      bool far = false;  // more steps than 32 bits hold: such items stay whole
      for (int e0 = 0; e0 < before; e0 += 32) {
        int v = 0;
        if (e0 + lane < before) {
          int lo = 0, hi = n;
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (m.cum[mid] <= e0 + lane) lo = mid;
            else hi = mid;
          }
          v = item_tiles<ROWS>(p, seq_of(p, m, m.order[lo]), e0 + lane - m.cum[lo]) + kExtra;
        }
        most = max(most, __reduce_max_sync(0xFFFFFFFFu, v));
        far = far || (int64_t)sum + (int64_t)most * 32 * p.hkv > (1 << 30);
        v *= p.hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
          if (lane >= o) v += u;
        }
        if (e0 + lane < before) m.cost[e0 + lane + 1] = sum + v;
        sum += __shfl_sync(0xFFFFFFFFu, v, 31);
      }
      if (lane == 0) {
        m.cost[0] = 0;
        m.total = sum;
        const int share = sum / grid, whole = before * p.hkv > grid ? max(most, share + most / 2) : most;
        m.split = !far && whole > share + kJoin;
        m.ctas = min(grid, max(1, sum / kLeast));
      }
    }
  }
  __syncthreads();
}

// Fills in what follows from the stretch.
template <int ROWS>
__device__ __forceinline__ void finish(const TreeParams& p, Work& w) {
  w.n0 = tiles_of(p, w, 0, 128);
  w.n1 = ROWS > 128 ? tiles_of(p, w, 128, 256) : 0;
  w.shared0 = seen_by(p, w, 0);
  w.shared1 = w.rows > 128 ? seen_by(p, w, 128) : 0;
}

// Fills the rest of a work from its sequence and block of rows.
template <int ROWS>
__device__ __forceinline__ void describe(const TreeParams& p, Work& w, const TreeSeq& s, int rb) {
  const int row0 = rb * ROWS, rows = s.count * p.group - row0;
  w.start = s.start;
  w.first = (int)((uint32_t)row0 / (uint32_t)p.group);
  w.g0 = row0 - w.first * p.group;
  w.rows = rows < ROWS ? rows : ROWS;
  w.prefix = s.prefix;
  w.len = s.prefix + s.count;
  w.last = item_tiles<ROWS>(p, s, rb) - 1;
  w.more = 1;
}

// Item `i` of the whole ones.
template <int ROWS>
__device__ __forceinline__ Work whole_item(const TreeParams& p, const Map& m, int i) {
  Work w{};
  if ((uint32_t)i >= (uint32_t)m.items) return w;
  const int block = i / p.hkv;
  w.head = i - block * p.hkv;
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (m.cum[mid] <= block) lo = mid;
    else hi = mid;
  }
  w.b = m.order[lo];
  describe<ROWS>(p, w, seq_of(p, m, w.b), m.cum[lo + 1] - 1 - block);  // from the last block to the first
  w.tile0 = 0;
  w.tiles = w.last + 1;
  finish<ROWS>(p, w);
  return w;
}

// The next stretch from `at` on of the range that ends at `end`; moves `at`.
template <int ROWS>
__device__ __forceinline__ Work next_stretch(const TreeParams& p, const Map& m, int& at, int end) {
  while (at < end) {
    Work w{};
    int lo = 0, hi = m.entries;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (m.cost[mid] <= at) lo = mid;
      else hi = mid;
    }
    const int length = (m.cost[lo + 1] - m.cost[lo]) / p.hkv, r = at - m.cost[lo];
    w.head = r / length;
    const int off = r - w.head * length, stop = min(length, off + end - at);
    int s = 0, z = p.batch;
    while (z - s > 1) {
      const int mid = (s + z) >> 1;
      if (m.cum[mid] <= lo) s = mid;
      else z = mid;
    }
    w.b = m.order[s];
    describe<ROWS>(p, w, seq_of(p, m, w.b), lo - m.cum[s]);
    w.tile0 = max(off - kExtra, 0);
    w.tiles = max(stop - kExtra, 0) - w.tile0;
    w.until = tree_cta_of(at - off + length - 1, m.total, m.ctas);
    at += stop - off;
    if (w.tiles > 0) {
      finish<ROWS>(p, w);
      return w;
    }
  }
  return Work{};
}

}  // namespace prompt
}  // namespace trellis

// tree_sched.cuh -- how the work of a tree attention call is divided over the GPU, shared by its kernels.
//
// An item is one key/value head of one sequence and one block of ROWS query rows (row r of a sequence and head:
// draft r / group, query head r % group of the head's group); it takes one step per TILE keys.  Lengths are device
// data, so the division is made on the device: the steps of all items, in the order of (sequence, row block, head,
// tile), are laid end to end and cut into equal contiguous ranges, one per thread block; a step belongs to the range that
// holds its beginning.  A step has length 1, or (HALVES) 2 where its rows fill more than half a block, since it then
// takes that kernel twice as long; an item has some length besides, for what it costs to start and finish it.  An item that falls into one range is finished there.  Otherwise each block
// writes its part (maximum, sum and unnormalised output of its keys, fp32) to the workspace, and a second launch
// (tree_join.cu) joins the parts in their order over the whole GPU: results do not depend on timing, and no block has the
// joining of a long item to itself.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "serving.h"

namespace trellis {

constexpr int kTreeMaxCtas = 1024;   // bound on the grid (sizes the table of shared items)

struct TreeParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t *table, *prefix, *q_start;
  const uint64_t* mask;
  const float* scales;  // [2][hkv] of the layer, or null
  const void* pool;     // the layer's pages, bf16 or e4m3
  int4* items;          // [kTreeMaxCtas]: the item that block c is the first to share (tree_item), or none
  float* part;          // two slots per thread block
  int64_t q_stride, out_stride;
  int64_t pages;
  uint64_t wait_ns;
  uint64_t group_inv;   // ceil(2^32 / group)
  int batch, width, n, max_tokens, hq, hkv, group, page_shift;
  float scale_log2;     // scale * log2(e)
};

// One sequence's lengths, clamped to what the arrays hold.
struct TreeSeq {
  int start, count, prefix;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  int a = __ldcg(p.q_start + b), z = __ldcg(p.q_start + b + 1);
  a = a < 0 ? 0 : a > p.n ? p.n : a;
  z = z < a ? a : z > p.n ? p.n : z;
  const int room = p.width << p.page_shift;
  int c = z - a;
  c = c > p.max_tokens ? p.max_tokens : c;
  c = c > room ? room : c;
  int pre = __ldcg(p.prefix + b);
  pre = pre < 0 ? 0 : pre > room - c ? room - c : pre;
  s.start = a;
  s.count = c;
  s.prefix = pre;
  return s;
}
template <int TILE>
__device__ __forceinline__ int tree_tiles(const TreeSeq& s) { return s.count ? (s.prefix + s.count + TILE - 1) / TILE : 0; }

// Row r of a sequence and head: its draft, without a division (exact: r < 2^16, group <= 2^10).
__device__ __forceinline__ int tree_draft(const TreeParams& p, int r) { return (int)((uint64_t)(uint32_t)r * p.group_inv >> 32); }

// What every thread of a block knows of the sequences, in shared memory: cum[b], the length of the sequences before b, and
// the first kCached sequences themselves.
struct TreeMap {
  static constexpr int kCached = 256;
  int cum[kTreeMaxBatch + 4], items[kTreeMaxBatch + 4];  // items: their number
  int extra;  // length of an item besides its steps
  int4 seq[kCached];  // start, count, prefix
};
__device__ __forceinline__ TreeSeq tree_seq_of(const TreeParams& p, const TreeMap& map, int b) {
  if (b >= TreeMap::kCached) return tree_seq(p, b);
  const int4 v = map.seq[b];
  return TreeSeq{v.x, v.y, v.z};
}

// Fills the map, by one warp.  An item has EXTRA steps before its own (no more than a block's share of the steps): what it costs
// to start and finish one is then counted, and a block with many short items has fewer steps.
template <int ROWS, int TILE, bool HALVES, int EXTRA>
__device__ __forceinline__ void tree_cumulate(const TreeParams& p, TreeMap& map) {
  const int lane = threadIdx.x & 31;
  int before = 0, items = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    int v = 0, n = 0;
    if (b < p.batch) {
      const TreeSeq s = tree_seq(p, b);
      if (b < TreeMap::kCached) map.seq[b] = make_int4(s.start, s.count, s.prefix, 0);
      constexpr int kUnit = HALVES ? ROWS / 2 : ROWS;
      v = tree_tiles<TILE>(s) * ((s.count * p.group + kUnit - 1) / kUnit) * p.hkv;
      n = (s.count * p.group + ROWS - 1) / ROWS * p.hkv;
    }
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, v, o), k = __shfl_up_sync(0xFFFFFFFFu, n, o);
      if (lane >= o) {
        v += u;
        n += k;
      }
    }
    if (b < p.batch) {
      map.cum[b + 1] = before + v;
      map.items[b + 1] = items + n;
    }
    before += __shfl_sync(0xFFFFFFFFu, v, 31);
    items += __shfl_sync(0xFFFFFFFFu, n, 31);
  }
  const int extra = min(EXTRA, before / (int)gridDim.x);
  __syncwarp();
  for (int b = lane; b < p.batch; b += 32) map.cum[b + 1] += extra * map.items[b + 1];
  if (lane == 0) {
    map.cum[0] = 0;
    map.extra = extra;
  }
}

// The blocks' ranges: block c of `ctas` takes [c * total / ctas, (c + 1) * total / ctas); the block that holds `at`:
__device__ __forceinline__ int tree_cta_of(int64_t at, int64_t total, int ctas) { return (int)(((at + 1) * ctas - 1) / total); }
// Blocks in use: no part of an item is left without a step, so ranges are as long as the longest step.
template <int ROWS, bool HALVES>
__device__ __forceinline__ int tree_ctas_used(const TreeParams& p, int total, int grid) {
  const int most = HALVES && p.max_tokens * p.group > ROWS / 2 ? (total + 1) / 2 : total;
  return most < grid ? most : grid;
}

// A stretch of one item's steps inside a block's range.
struct TreeSegment {
  TreeSeq seq;
  int b, head, row_block;
  int tile0, tiles;   // first tile, number of tiles
  bool starts, whole; // the item's first tile is in this range; all of them are
  int last_at;        // where its last step begins
};

// Walks a block's range segment by segment.
template <int ROWS, int TILE, bool HALVES>
struct TreeWalk {
  int at, begin, end, b;
  __device__ __forceinline__ TreeWalk(int total, int ctas, int cta) : at(0), begin(0), end(0), b(-1) {
    if (cta < ctas) {
      begin = at = (int)((int64_t)cta * total / ctas);
      end = (int)((int64_t)(cta + 1) * total / ctas);
    }
  }
  __device__ __forceinline__ bool next(const TreeParams& p, const TreeMap& map, TreeSegment& g) {
    while (at < end) {
      if (b < 0) {  // the last sequence that starts at or before `at`; empty ones are passed over
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (map.cum[mid] <= at) lo = mid;
          else hi = mid;
        }
        b = lo;
      } else {
        while (map.cum[b + 1] <= at) ++b;
      }
      g.b = b;
      g.seq = tree_seq_of(p, map, b);
      const int nt = tree_tiles<TILE>(g.seq), extra = map.extra, r = at - map.cum[b];
      const int block = ((HALVES ? 2 : 1) * nt + extra) * p.hkv;
      g.row_block = r / block;
      const int w = HALVES && g.seq.count * p.group - g.row_block * ROWS > ROWS / 2 ? 2 : 1;
      const int q = r - g.row_block * block;
      const int length = extra + nt * w;
      g.head = q / length;
      const int off = q - g.head * length;             // into the item
      const int stop = off + (end - at) < length ? off + (end - at) : length;
      g.tile0 = (max(off - extra, 0) + w - 1) / w;
      g.tiles = (max(stop - extra, 0) + w - 1) / w - g.tile0;
      g.last_at = at - off + extra + (nt - 1) * w;
      g.starts = g.tile0 == 0;
      g.whole = g.starts && g.last_at < end;
      at += stop - off;
      if (g.tiles > 0) return true;
    }
    return false;
  }
};

// The pages of a segment's tiles, for the warp that copies them: table entries are read 32 boxes (copies of up to a page) at a
// time and a window ahead, since a copy that waits for its own entry costs the warp a trip to memory each time (4 sequences of
// 64 drafts and 16384 keys, 40/8 heads of 128: 132 us so, 122 with the window).
template <int TILE>
struct TreePages {
  const int32_t* row;
  int first, len, shift, box, per, lane, window, prev, now, next;  // per: boxes of a tile
  __device__ __forceinline__ TreePages(const TreeParams& p, const TreeSegment& g, int lane_)
      : row(p.table + (int64_t)g.b * p.width), first(g.tile0 * TILE), len(g.seq.prefix + g.seq.count), shift(p.page_shift),
        box(min(1 << p.page_shift, TILE)), per(TILE / box), lane(lane_), window(0) {
    prev = now = load(0);
    next = load(1);
  }
  __device__ __forceinline__ int load(int w) const {
    const int pos = first + (32 * w + lane) * box;
    return pos < len ? row[pos >> shift] : 0;
  }
  // Page of this lane's box of tile t (lanes below `per`).  Tiles come in order, or up to two behind the last one.
  __device__ __forceinline__ int at(int t) {
    const int i = t * per, w = i >> 5;
    if (w > window) {
      prev = now;
      now = next;
      next = load(w + 1);
      window = w;
    }
    return __shfl_sync(0xFFFFFFFFu, w == window ? now : prev, (i + lane) & 31);
  }
};

__host__ __device__ __forceinline__ int tree_parts_shared(int parts) { return parts <= 8 ? 0 : parts <= 16 ? 1 : parts <= 32 ? 2 : 3; }
// An item for the joining kernel, of parts from block `first` to `last`: its sequence's first draft, head, first row; packed,
// the last block, rows, and (log2) how many share its parts.  Packed 0: no item.
__device__ __forceinline__ int4 tree_item(const TreeSegment& g, int row0, int rows, int first, int last) {
  return make_int4(g.seq.start, g.head, row0, tree_parts_shared(last - first + 1) << 24 | rows << 12 | last);
}
__device__ __forceinline__ int tree_item_last(int w) { return w & 0xFFF; }
__device__ __forceinline__ int tree_item_rows(int w) { return w >> 12 & 0xFFF; }
__device__ __forceinline__ int tree_item_shared(int w) { return w >> 24; }
// The workspace slot of a block's part: a block has at most one part that starts its item and one that does not.
__device__ __forceinline__ int tree_slot(int cta, bool starts_item) { return 2 * cta + (starts_item ? 1 : 0); }
// A part: unnormalised outputs [dim / 4][rows][4], maxima [rows] (log2), sums of weights [rows].
__host__ __device__ constexpr int64_t tree_part_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }

// Joins the parts of shared items, after a kernel over `ctas` blocks of `rows` rows on the stream (tree_join.cu).  lift: log2 of a
// factor that the weights carry.
cudaError_t launch_tree_join(const TreeParams& p, int dim, int rows, float lift, int ctas, cudaStream_t st);

// One copy of a cache's tensor map: rows of head_dim numbers, and bytes of each (128, or 64; also the
// swizzle).
struct TreeBox {
  int rows, bytes;
};

// The tensor-core kernels: where they take a call, the rows of their blocks, and what they need copied.
bool tree_tc_fits(const trellis_cache_t& c, int rows);  // tree_attention_tc.cu
int tree_tc_rows();
void tree_tc_box(const trellis_cache_t& c, TreeBox* b);
cudaError_t launch_tree_tc(const CUtensorMap& map, const TreeParams& p, const trellis_cache_t& c, int ctas, cudaStream_t st);
int read_tree_tc_error(int reset);
bool tree_tc1_fits(const trellis_cache_t& c, int rows);  // tree_attention_tc1.cu
int tree_tc1_rows();
void tree_tc1_box(const trellis_cache_t& c, TreeBox* b);
cudaError_t launch_tree_tc1(const CUtensorMap& map, const TreeParams& p, const trellis_cache_t& c, int ctas, cudaStream_t st);
int read_tree_tc1_error(int reset);

}  // namespace trellis

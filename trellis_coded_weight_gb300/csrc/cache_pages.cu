// cache_pages.cu -- pages of a key/value cache: copied, forked, compacted, and accepted drafts moved
// (trellis_cache_copy, _fork, _compact, _commit).
//
// Fork and compact are two launches each.  A planning kernel of one thread block works on the integers (page table,
// reference counts): a running count over the pages gives the k-th lowest free page, so the result does not depend
// on any order of execution.  It leaves a list of page copies in the workspace.  The copying kernel then moves them in all layers, in
// units of 16 KB spread evenly over the GPU.  The copies are bound by HBM: a compaction that moves 133 MB copies for 40 us, 6.7 TB/s
// read and written; a fork of 159 MB from few sources writes for 50 us, 3.2 TB/s, where a fill of such a size reaches 3.7.  (One load
// of a place for all of its copies changed nothing, and cost small forks 2 us.)  The planning is bound by latency: 6 us for a
// compaction, 10 for a fork, a handful of dependent trips to memory.  Commit is one launch of 12 us for 25 MB: it has to know where a row goes before it can move it.
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"

namespace trellis {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyBlocks = 4;  // of an SM
constexpr int kUnit = 16384;  // bytes of a copying step: four 16-byte loads of each thread in flight

__device__ __forceinline__ uint4 ld_stream(const uint4* p) { return __ldcs(p); }

// ---------------------------------------------------------------- copies of whole pages

struct CopyParams {
  uint8_t* pool;
  const int32_t *src, *dst;
  const int32_t* count;  // device count of the list, or null: `most`
  int64_t page_bytes, layer_bytes, pages;
  int most, layers;
  // compact: entries of the table are renamed on the way
  const int32_t* remap;
  const int32_t* table;
  int32_t* out_table;
  int64_t entries;
};

// A block takes a contiguous range of the units (pair major, then layer, then place in the page), stepping through them
// without divisions; a unit's loads go out before the stores of the one before it.
__global__ void __launch_bounds__(kCopyThreads, kCopyBlocks) copy_pages_kernel(const CopyParams p) {
  pdl_enter();
  const int n = p.count ? __ldcg(p.count) : p.most;
  const int per_page = (int)((p.page_bytes + kUnit - 1) / kUnit);
  const int64_t units = (int64_t)n * p.layers * per_page;
  const int64_t lo = units * blockIdx.x / gridDim.x;
  int left = (int)(units * (blockIdx.x + 1) / gridDim.x - lo);
  int chunk = (int)(lo % per_page), layer = (int)(lo / per_page % p.layers), i = (int)(lo / per_page / p.layers);
  constexpr int kVecs = kUnit / 16 / kCopyThreads;
  struct Unit {
    uint4 v[kVecs];
    uint4* to;
    int vecs;  // of the unit; 0: nothing to move
  };
  const auto fetch = [&](Unit& u) {
    const int64_t src = __ldcg(p.src + i), dst = __ldcg(p.dst + i), at = (int64_t)chunk * kUnit;
    u.vecs = 0;
    if (src >= 0 && src < p.pages && dst >= 0 && dst < p.pages) {
      const int64_t rest = p.page_bytes - at;
      u.vecs = (int)((rest < kUnit ? rest : kUnit) / 16);
      const uint4* from = reinterpret_cast<const uint4*>(p.pool + layer * p.layer_bytes + src * p.page_bytes + at);
      u.to = reinterpret_cast<uint4*>(p.pool + layer * p.layer_bytes + dst * p.page_bytes + at);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const int e = threadIdx.x + j * kCopyThreads;
        if (e < u.vecs) u.v[j] = ld_stream(from + e);
      }
    }
    if (++chunk == per_page) {
      chunk = 0;
      if (++layer == p.layers) {
        layer = 0;
        ++i;
      }
    }
  };
  const auto store = [&](const Unit& u) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int e = threadIdx.x + j * kCopyThreads;
      if (e < u.vecs) u.to[e] = u.v[j];
    }
  };
  Unit a, b;
  if (left > 0) fetch(a);
  for (; left > 0; left -= 2) {
    if (left > 1) fetch(b);
    store(a);
    if (left > 2) fetch(a);
    if (left > 1) store(b);
  }
  for (int64_t e = blockIdx.x * (int64_t)kCopyThreads + threadIdx.x; e < p.entries; e += (int64_t)gridDim.x * kCopyThreads) {
    const int32_t page = p.table[e];
    p.out_table[e] = page >= 0 && page < p.pages ? __ldcg(p.remap + page) : page;
  }
}

cudaError_t launch_copy(CopyParams p, cudaStream_t st) {
  const int64_t units = (int64_t)p.most * p.layers * ((p.page_bytes + kUnit - 1) / kUnit);
  const int64_t full = kCopyBlocks * (int64_t)device_sm_count();
  int64_t grid = units < full ? units : full;
  const int64_t table = (p.entries + kCopyThreads - 1) / kCopyThreads;
  if (grid < table) grid = table < full ? table : full;
  return launch_pdl(copy_pages_kernel, dim3((unsigned)grid), dim3(kCopyThreads), 0, st, p);
}

CopyParams copy_params(const trellis_cache_t& c) {
  CopyParams p{};
  p.pool = static_cast<uint8_t*>(c.pool);
  p.page_bytes = cache_page_bytes(c);
  p.layer_bytes = c.pages * p.page_bytes;
  p.pages = c.pages;
  p.layers = c.layers;
  return p;
}

// ---------------------------------------------------------------- scans of one block

// Inclusive sum of v over the block's threads; the block's total in *total.  Ends with the scratch free again.
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += u;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  if (warp) v += scratch[warp - 1];
  *total = scratch[31];
  __syncthreads();
  return v;
}

// ---------------------------------------------------------------- fork

struct ForkParams {
  int32_t *table, *lens, *refs;
  const int32_t *parent, *child;
  int32_t* status;
  int32_t *count, *src, *dst;  // the list of copies: pairs entries
  int32_t* fresh;              // pages handed out, in order: pairs * width entries
  int32_t* rows_new;           // [pairs][width]
  int64_t pages;
  int pairs, rows, width, room, page_shift;
};

enum : int { kFork = 0, kGrow = 1, kFree = 2, kBad = 3 };

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkParams p) {
  pdl_enter();
  __shared__ int scratch[32];
  __shared__ int s_par[kForkMaxPairs], s_child[kForkMaxPairs], s_len[kForkMaxPairs], s_full[kForkMaxPairs],
      s_need[kForkMaxPairs], s_held[kForkMaxPairs], s_upto[kForkMaxPairs];
  __shared__ uint8_t s_kind[kForkMaxPairs], s_ok[kForkMaxPairs];
  __shared__ int s_copies;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_copies = 0;
  // loads that depend on nothing come first: the planning is a chain of trips to memory
  int32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = tid * 4 + j < p.pages ? p.refs[tid * 4 + j] : 1;

  // 1. what each pair asks for: one warp per pair
  for (int i = warp; i < p.pairs; i += kPlanThreads / 32) {
    const int par = p.parent[i], ch = p.child[i];
    int kind = par == -1 ? kFree : par == ch ? kGrow : kFork;
    if (ch < 0 || ch >= p.rows || par < -1 || par >= p.rows) kind = kBad;
    int held = 0, len = 0, full = 0, need = 0;
    if (kind != kBad) {
      const int32_t first_len = kind != kFree ? p.lens[par] : 0;
      const int32_t first_child = lane < p.width ? p.table[(int64_t)ch * p.width + lane] : -1;
      const int32_t first_parent = kind == kFork && lane < p.width ? p.table[(int64_t)par * p.width + lane] : 0;
      bool more = true;
      for (int e = 0; more && e < p.width; e += 32) {  // leading entries >= 0
        const bool has = e + lane < p.width && (e ? p.table[(int64_t)ch * p.width + e + lane] : first_child) >= 0;
        const unsigned b = __ballot_sync(0xFFFFFFFFu, has);
        const int lead = b == 0xFFFFFFFFu ? 32 : __ffs(~b) - 1;
        held += lead;
        more = lead == 32;
      }
      if (kind != kFree) {
        len = first_len;
        const int64_t most = (int64_t)p.width << p.page_shift;
        if (len < 0 || len > most) kind = kBad;
        else {
          const int64_t want = ((int64_t)len + p.room + (1 << p.page_shift) - 1) >> p.page_shift;
          full = kind == kGrow ? held : len >> p.page_shift;
          const int64_t n = want > full ? want : full;
          need = n > p.width ? p.width + 1 : (int)n;
        }
      }
      // every page that is shared, copied or given up has to be one of the pool
      bool bad = false;
      for (int e = lane; e < held; e += 32) bad |= (e < 32 ? first_child : p.table[(int64_t)ch * p.width + e]) >= p.pages;
      if (kind == kFork) {
        const int used = (len + (1 << p.page_shift) - 1) >> p.page_shift;
        for (int e = lane; e < used; e += 32) {
          const int32_t page = e < 32 ? first_parent : p.table[(int64_t)par * p.width + e];
          bad |= page < 0 || page >= p.pages;
        }
      }
      if (__any_sync(0xFFFFFFFFu, bad)) kind = kBad;
    }
    if (lane == 0) {
      s_par[i] = par; s_child[i] = ch; s_len[i] = len; s_full[i] = full; s_need[i] = need; s_held[i] = held;
      s_kind[i] = (uint8_t)kind;
    }
  }
  __syncthreads();
  int asked;
  {
    int fresh = 0;
    if (tid < p.pairs && (s_kind[tid] == kFork || s_kind[tid] == kGrow) && s_need[tid] <= p.width)
      fresh = s_need[tid] - s_full[tid];
    const int upto = block_scan(fresh, scratch, &asked);
    if (tid < p.pairs) s_upto[tid] = upto;
  }

  // 2. the lowest free pages, as many as are asked for
  int found = 0;
  for (int64_t base = 0; base < p.pages && found < asked; base += kPlanThreads * 4) {
    const int64_t e = base + tid * 4;
    if (base > 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = e + j < p.pages ? p.refs[e + j] : 1;
    const int mine = (r[0] == 0) + (r[1] == 0) + (r[2] == 0) + (r[3] == 0);
    int total;
    int at = found + block_scan(mine, scratch, &total) - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r[j] == 0) {
        if (at < asked) p.fresh[at] = (int32_t)(e + j);
        ++at;
      }
    found += total;
  }
  __syncthreads();
  if (tid < p.pairs) {
    const int fresh = s_need[tid] <= p.width ? s_need[tid] - s_full[tid] : 0;
    s_ok[tid] = s_kind[tid] == kFree ||
                (s_kind[tid] != kBad && s_need[tid] <= p.width && (fresh == 0 || s_upto[tid] <= found));
  }
  __syncthreads();

  // 3. the children's new rows, from the parents as they were; reference counts by commuting additions
  const int64_t cells = (int64_t)p.pairs * p.width;
  for (int64_t x = tid; x < cells; x += kPlanThreads) {
    const int i = (int)(x / p.width), e = (int)(x - (int64_t)i * p.width), kind = s_kind[i];
    if (kind == kBad) continue;
    const int32_t old = p.table[(int64_t)s_child[i] * p.width + e];
    int32_t now = -1;
    if (!s_ok[i]) {
      now = kind == kGrow ? old : -1;
    } else if (kind != kFree) {
      if (e < s_full[i]) {
        now = p.table[(int64_t)s_par[i] * p.width + e];
        if (kind == kFork) atomicAdd(p.refs + now, 1);
      } else if (e < s_need[i]) {
        now = p.fresh[s_upto[i] - (s_need[i] - s_full[i]) + e - s_full[i]];
        atomicAdd(p.refs + now, 1);
      }
    }
    if (kind != kGrow && e < s_held[i]) atomicAdd(p.refs + old, -1);
    p.rows_new[x] = now;
  }
  if (tid < p.pairs && s_kind[tid] == kFork && s_ok[tid] && (s_len[tid] & ((1 << p.page_shift) - 1))) {
    const int at = atomicAdd(&s_copies, 1);  // the order of the list does not matter
    p.src[at] = p.table[(int64_t)s_par[tid] * p.width + s_full[tid]];
    p.dst[at] = p.fresh[s_upto[tid] - (s_need[tid] - s_full[tid])];
  }
  __syncthreads();

  // 4. written back once everything has been read
  for (int64_t x = tid; x < cells; x += kPlanThreads) {
    const int i = (int)(x / p.width), e = (int)(x - (int64_t)i * p.width);
    if (s_kind[i] != kBad) p.table[(int64_t)s_child[i] * p.width + e] = p.rows_new[x];
  }
  if (tid < p.pairs) {
    if (s_kind[tid] == kFork || s_kind[tid] == kFree) p.lens[s_child[tid]] = s_ok[tid] ? s_len[tid] : 0;
    p.status[tid] = s_kind[tid] == kBad ? 2 : s_ok[tid] ? 0 : 1;
  }
  if (tid == 0) *p.count = s_copies;
}

// ---------------------------------------------------------------- compact

struct CompactParams {
  const int32_t* refs;
  int32_t* out_refs;
  int32_t *count, *src, *dst;  // pages / 2 + 1 entries each
  int32_t* remap;              // [pages]
  int64_t pages;
};

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactParams p) {
  pdl_enter();
  __shared__ int scratch[32];
  const int tid = threadIdx.x;
  int mine = 0, live;
  for (int64_t e = tid; e < p.pages; e += kPlanThreads) mine += p.refs[e] > 0;
  block_scan(mine, scratch, &live);
  // the k-th live page at or past `live` goes to the k-th free page before it: as many of the one as of the other
  int holes = 0, high = 0;
  for (int64_t base = 0; base < p.pages; base += kPlanThreads) {
    const int64_t e = base + tid;
    const bool in = e < p.pages, is_live = in && p.refs[e] > 0;
    const bool hole = in && !is_live && e < live, moves = is_live && e >= live;
    int total;  // both counts in one scan: a step adds at most 1024 to either
    const int both = block_scan((hole ? 1 : 0) + (moves ? 1 << 16 : 0), scratch, &total);
    if (hole) p.dst[holes + (both & 0xFFFF) - 1] = (int32_t)e;
    if (moves) p.src[high + (both >> 16) - 1] = (int32_t)e;
    holes += total & 0xFFFF;
    high += total >> 16;
    if (in) {
      p.remap[e] = (int32_t)e;
      p.out_refs[e] = is_live ? p.refs[e] : 0;
    }
  }
  __syncthreads();
  for (int i = tid; i < high; i += kPlanThreads) {
    const int32_t from = p.src[i], to = p.dst[i];
    p.remap[from] = to;
    p.out_refs[to] = p.out_refs[from];
    p.out_refs[from] = 0;
  }
  if (tid == 0) *p.count = high;
}

// ---------------------------------------------------------------- commit

struct CommitParams {
  uint8_t* pool;
  const int32_t *table, *prefix, *path, *accepted;
  int32_t* lens;
  int64_t pages, layer_bytes;
  int width, max_tokens, page_shift, heads, row_vecs;  // row_vecs: 16-byte vectors of one head's row
};

// One block per sequence, layer and share of the 2 * heads rows of a position; a thread owns one 16-byte column of
// such a row and moves it for every accepted draft.  Sources ascend and are never before their destinations, so a
// batch may be loaded whole before it is stored.
__global__ void __launch_bounds__(kCopyThreads) commit_kernel(const CommitParams p) {
  pdl_enter();
  __shared__ int64_t s_src[kTreeMaxTokens], s_dst[kTreeMaxTokens];  // row index within (page, kv, head): page row base
  __shared__ int s_n;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int prefix = p.prefix[b];
  int acc = p.accepted[b];
  acc = acc < 0 ? 0 : acc > p.max_tokens ? p.max_tokens : acc;
  if (tid < 32) {  // the moves, in ascending order
    int n = 0;
    for (int base = 0; base < acc; base += 32) {
      const int i = base + tid;
      bool move = i < acc;
      int64_t from = 0, to = 0;
      if (move) {
        const int j = p.path[(int64_t)b * p.max_tokens + i];
        move = j > i && j < kTreeMaxTokens && prefix >= 0 && (i == 0 || j > p.path[(int64_t)b * p.max_tokens + i - 1]);
        const int64_t a = (int64_t)prefix + j, z = (int64_t)prefix + i, end = (int64_t)p.width << p.page_shift;
        move = move && a < end;
        if (move) {
          const int32_t pa = p.table[(int64_t)b * p.width + (a >> p.page_shift)];
          const int32_t pz = p.table[(int64_t)b * p.width + (z >> p.page_shift)];
          move = pa >= 0 && pa < p.pages && pz >= 0 && pz < p.pages;
          from = ((int64_t)pa * 2 * p.heads << p.page_shift) + (a & ((1 << p.page_shift) - 1));
          to = ((int64_t)pz * 2 * p.heads << p.page_shift) + (z & ((1 << p.page_shift) - 1));
        }
      }
      const unsigned any = __ballot_sync(0xFFFFFFFFu, move);
      if (move) {
        const int at = n + __popc(any & ((1u << tid) - 1));
        s_src[at] = from;
        s_dst[at] = to;
      }
      n += __popc(any);
    }
    if (tid == 0) s_n = n;
  }
  if (blockIdx.y == 0 && blockIdx.z == 0 && tid == 0 && p.lens) p.lens[b] = prefix + acc;
  __syncthreads();
  const int n = s_n;
  const int col = blockIdx.z * kCopyThreads + tid;
  if (col >= 2 * p.heads * p.row_vecs) return;
  const int row = col / p.row_vecs, vec = col - row * p.row_vecs;  // row: kv * heads + head
  uint4* base = reinterpret_cast<uint4*>(p.pool + blockIdx.y * p.layer_bytes) + ((int64_t)row << p.page_shift) * p.row_vecs + vec;
  for (int i0 = 0; i0 < n; i0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i < n) v[i] = base[s_src[i0 + i] * p.row_vecs];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i < n) base[s_dst[i0 + i] * p.row_vecs] = v[i];
  }
}

__global__ void __launch_bounds__(kCopyThreads) commit_lens_kernel(const int32_t* accepted, int32_t* lens, int batch, int max_tokens) {
  pdl_enter();
  const int b = blockIdx.x * kCopyThreads + threadIdx.x;
  if (b >= batch) return;
  const int acc = accepted[b];
  lens[b] += acc < 0 ? 0 : acc > max_tokens ? max_tokens : acc;
}

int page_shift_of(const trellis_cache_t& c) { return c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7; }
int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

}  // namespace

cudaError_t launch_cache_copy(const trellis_cache_t& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t st) {
  CopyParams p = copy_params(c);
  p.src = src; p.dst = dst; p.most = n;
  return launch_copy(p, st);
}

// int32 words: [4] count, then for fork src[pairs], dst[pairs], fresh and rows_new [pairs][width], for compact
// src, dst [pages / 2 + 1] and remap [pages].
size_t cache_workspace_bytes(const trellis_cache_t& c, int pairs, int width) {
  const int64_t fork = 4 + 2 * up4(pairs) + 2 * up4((int64_t)pairs * width);
  const int64_t compact = 4 + 2 * up4(c.pages / 2 + 1) + up4(c.pages);
  return (size_t)(fork > compact ? fork : compact) * 4;
}

cudaError_t launch_cache_fork(const trellis_cache_t& c, int32_t* table, int32_t* lens, int32_t* refs,
                              const int32_t* parent, const int32_t* child, int32_t* status, int pairs, int rows,
                              int width, int room, void* workspace, cudaStream_t st) {
  int32_t* w = static_cast<int32_t*>(workspace);
  ForkParams p{table, lens, refs, parent, child, status};
  p.count = w;
  p.src = w + 4;
  p.dst = p.src + up4(pairs);
  p.fresh = p.dst + up4(pairs);
  p.rows_new = p.fresh + up4((int64_t)pairs * width);
  p.pages = c.pages;
  p.pairs = pairs; p.rows = rows; p.width = width; p.room = room; p.page_shift = page_shift_of(c);
  const cudaError_t e = launch_pdl(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  CopyParams q = copy_params(c);
  q.src = p.src; q.dst = p.dst; q.count = p.count; q.most = pairs;
  return launch_copy(q, st);
}

cudaError_t launch_cache_compact(const trellis_cache_t& c, const int32_t* table, const int32_t* refs,
                                 int32_t* out_table, int32_t* out_refs, int rows, int width, void* workspace,
                                 cudaStream_t st) {
  int32_t* w = static_cast<int32_t*>(workspace);
  const int64_t half = up4(c.pages / 2 + 1);
  CompactParams p{refs, out_refs};
  p.count = w;
  p.src = w + 4;
  p.dst = p.src + half;
  p.remap = p.dst + half;
  p.pages = c.pages;
  const cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  CopyParams q = copy_params(c);
  q.src = p.src; q.dst = p.dst; q.count = p.count; q.most = (int)(c.pages / 2);
  q.remap = p.remap; q.table = table; q.out_table = out_table; q.entries = (int64_t)rows * width;
  return launch_copy(q, st);
}

cudaError_t launch_cache_commit(const trellis_cache_t& c, const int32_t* table, const int32_t* prefix,
                                const int32_t* path, const int32_t* accepted, int32_t* lens, int batch, int width,
                                int max_tokens, cudaStream_t st) {
  CommitParams p{};
  p.pool = static_cast<uint8_t*>(c.pool);
  p.table = table; p.prefix = prefix; p.path = path; p.accepted = accepted;
  // lens in place of prefix is written by a launch of its own: other blocks still read it here
  p.lens = lens == prefix ? nullptr : lens;
  p.pages = c.pages;
  p.layer_bytes = c.pages * cache_page_bytes(c);
  p.width = width; p.max_tokens = max_tokens; p.page_shift = page_shift_of(c); p.heads = c.heads;
  p.row_vecs = (int)(c.head_dim * cache_elem_bytes(c) / 16);
  const unsigned z = (unsigned)((2 * c.heads * p.row_vecs + kCopyThreads - 1) / kCopyThreads);
  cudaError_t e = launch_pdl(commit_kernel, dim3((unsigned)batch, (unsigned)c.layers, z), dim3(kCopyThreads), 0, st, p);
  if (e != cudaSuccess || p.lens) return e;
  return launch_pdl(commit_lens_kernel, dim3((unsigned)((batch + kCopyThreads - 1) / kCopyThreads)), dim3(kCopyThreads), 0, st, accepted,
                    lens, batch, max_tokens);
}

}  // namespace trellis

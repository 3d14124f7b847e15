// token_logprobs.cu -- log probabilities of given tokens with the entropy and the most likely alternatives of each
// row, in one pass over the logits (trellis_token_logprobs).
//
// With c = log2(e) / temperature, R the running maximum of x and y = c (x - R), a row needs
//   s = sum 2^y,   t = sum 2^y y
// and then  lse = R / temperature + ln s,  entropy = ln2 (log2 s - t / s),  log p(x) = (x - R) / temperature - ln s.
// The difference is taken first: it is exact near the maximum, and rows of the type's lowest numbers do not overflow.
// Sums of different references are joined by 2^(c (R - R')), t by t + s c (R - R').
//
// Alternatives: a number's key is its bits made to order like its value, above the complement of its column, so that keys are
// distinct and the larger key is the earlier alternative.  A block keeps the best top_k so far and their last value as
// a threshold; what passes it is appended to a list in shared memory, which is cut back to top_k by counting, for
// each key, the larger ones.  The first chunk's threshold is the top_k-th largest of 64 maxima over 64th parts of the chunk
// (at least top_k numbers reach it), so few numbers pass.  If more pass than the list holds (rows of equal numbers,
// rising rows) the chunk is taken again with such a threshold of its own, and if that fails (many equal numbers), by
// top_k searches for the next key.
//
// A row is split over blocks where there are few rows; the last block to arrive joins the parts in their order, so
// results do not depend on timing.  Bound: HBM for many rows (one read of the logits), latency for one.
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 1024;       // candidates held before they are cut back
constexpr int kCutAt = 192;       // a list longer than this is cut back after its chunk
constexpr int kVecs = 4;          // 16-byte vectors of a thread per chunk
constexpr int kCounters = 4096;   // rows that may be split
constexpr int kGroupThreads = 4;  // threads of one of the 64 parts of a chunk
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kFar = -16384.f;  // 2^kFar is 0: stands in for minus infinity where it would be multiplied

struct Params {
  const void* logits;
  const int32_t* tokens;
  float *logprobs, *lse, *entropy, *top_logprobs;
  int32_t* top_ids;
  uint32_t* counter;            // [n]
  float* sums;                  // [n][splits][4]
  unsigned long long* keys;     // [n][splits][top_k]
  int64_t row_stride;
  int n, vocab, cands, top_k, splits, chunks;
  float c, inv_t;               // log2(e) / temperature, 1 / temperature
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Orders like the value: NaN above all, -0 as +0.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order_bits(uint32_t o) {
  if (o == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ unsigned long long key_of(float x, int col) {
  return (unsigned long long)order_bits(x) << 32 | (uint32_t)~col;
}

struct Sums {
  float r, s, t;  // reference, and the two sums relative to it; s = 0 where nothing counts
};
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float c) {
  // references of sides that hold nothing are minus infinity; NaN stays
  const float r = max_nan(a.r, b.r);
  if (r == -INFINITY) return Sums{r, 0.f, 0.f};
  const float da = max_nan((a.r - r) * c, kFar), db = max_nan((b.r - r) * c, kFar);
  const float ea = ex2(da), eb = ex2(db);
  return Sums{r, a.s * ea + b.s * eb, (a.t + a.s * da) * ea + (b.t + b.s * db) * eb};
}

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& u, float (&x)[8]) {
    x[0] = bf16lo_to_f32(u.x); x[1] = bf16hi_to_f32(u.x);
    x[2] = bf16lo_to_f32(u.y); x[3] = bf16hi_to_f32(u.y);
    x[4] = bf16lo_to_f32(u.z); x[5] = bf16hi_to_f32(u.z);
    x[6] = bf16lo_to_f32(u.w); x[7] = bf16hi_to_f32(u.w);
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f32(*p); }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};

struct Shared {
  unsigned long long list[kList];
  unsigned long long best[kMaxTop];  // cut back: descending
  unsigned long long red[kWarps];
  Sums part[kWarps];
  float group_max[64];
  float threshold;
  int count;
  uint32_t last;
};

// The list's `count` keys cut back to the top_k largest, in descending order; the threshold is the last one's value.
__device__ __forceinline__ void cut_back(Shared& sh, int top_k) {
  const int count = sh.count;  // the caller's barrier precedes this
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const unsigned long long mine = sh.list[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += sh.list[j] > mine;
    if (rank < top_k) sh.best[rank] = mine;
  }
  __syncthreads();
  const int kept = count < top_k ? count : top_k;
  if (threadIdx.x < kept) sh.list[threadIdx.x] = sh.best[threadIdx.x];
  if (threadIdx.x == 0) {
    sh.count = kept;
    sh.threshold = kept == top_k ? from_order_bits((uint32_t)(sh.best[top_k - 1] >> 32)) : -INFINITY;
  }
  __syncthreads();
}

// A value that at least top_k of the chunk's numbers reach (minus infinity if that needs more than 64 parts):
// the top_k-th largest of the 64 parts' maxima.  Ends with a barrier.
__device__ __forceinline__ float chunk_threshold(Shared& sh, float thread_max, int top_k) {
  float g = thread_max;
#pragma unroll
  for (int o = 1; o < kGroupThreads; o <<= 1) g = max_nan(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
  if (threadIdx.x % kGroupThreads == 0) sh.group_max[threadIdx.x / kGroupThreads] = g;
  __syncthreads();
  if (threadIdx.x < 64) {
    const uint32_t mine = order_bits(sh.group_max[threadIdx.x]);
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < 64; ++j) {
      const uint32_t o = order_bits(sh.group_max[j]);
      rank += o > mine || (o == mine && j < (int)threadIdx.x);
    }
    if (rank == top_k - 1) sh.threshold = from_order_bits(mine);
  }
  __syncthreads();
  const float th = sh.threshold;
  __syncthreads();
  return th;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const Params p) {
  pdl_enter();
  constexpr int N = Vec<T>::N, PER = kVecs * N, CHUNK = kThreads * PER;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = blockIdx.x;
  const int64_t row = blockIdx.y;
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  // chunks start on 16-byte boundaries: a row that does not starts `skew` numbers into its first chunk
  const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int first = (int)((int64_t)split * p.chunks / p.splits), last = (int)((int64_t)(split + 1) * p.chunks / p.splits);
  if (tid == 0) {
    sh.count = 0;
    sh.threshold = -INFINITY;
  }
  __syncthreads();

  Sums acc{-INFINITY, 0.f, 0.f};
  bool cut = false;  // the list has been cut back to top_k: its threshold holds for later columns
  for (int ch = first; ch < last; ++ch) {
    // vector v of the thread: columns col0 + v * kThreads * N ..
    const int col0 = ch * CHUNK - skew + tid * N;
    float xs[PER];
    float vmax[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int c0 = col0 + v * kThreads * N;
      float(&e)[N] = *reinterpret_cast<float(*)[N]>(xs + v * N);
      if (c0 >= 0 && c0 + N <= p.vocab) {
        Vec<T>::get(__ldcs(reinterpret_cast<const uint4*>(x + c0)), e);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = c0 + i >= 0 && c0 + i < p.vocab ? Vec<T>::one(x + c0 + i) : -INFINITY;
      }
    }
    float tmax = -INFINITY;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float m = xs[v * N];
#pragma unroll
      for (int i = 1; i < N; ++i) m = max_nan(m, xs[v * N + i]);
      vmax[v] = m;
      tmax = max_nan(tmax, m);
    }
    const float r = max_nan(acc.r, tmax);
    if (r != acc.r && acc.r != -INFINITY) {
      const float d = max_nan((acc.r - r) * p.c, kFar), e = ex2(d);
      acc.t = (acc.t + acc.s * d) * e;
      acc.s *= e;
    }
    acc.r = r;
    if (r != -INFINITY) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float y = max_nan((xs[i] - r) * p.c, kFar);
        const float e = ex2(y);
        acc.s += e;
        acc.t = __fmaf_rn(e, y, acc.t);
      }
    }

    if (p.top_k == 0) continue;
    const float old_th = cut ? sh.threshold : -INFINITY;
    float th = old_th;
    bool strict = cut;  // later columns lose to equal earlier ones once top_k are held
    if (!cut) {
      th = chunk_threshold(sh, tmax, p.top_k);
      strict = false;
    }
    const int held = sh.count;
    __syncthreads();
    for (int attempt = 0;; ++attempt) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (strict ? vmax[v] <= th : vmax[v] < th) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float e = xs[v * N + i];
          const int col = col0 + v * kThreads * N + i;
          if ((strict ? !(e <= th) : !(e < th)) && col >= 0 && col < p.vocab) {
            const int at = atomicAdd(&sh.count, 1);
            if (at < kList) sh.list[at] = key_of(e, col);
          }
        }
      }
      __syncthreads();
      if (sh.count <= kList) break;
      __syncthreads();
      if (tid == 0) sh.count = held;
      if (attempt == 0) {
        // again, with this chunk's own threshold where it is the higher one
        const float own_th = chunk_threshold(sh, tmax, p.top_k);
        if (!(own_th < th) || !cut) {
          if (!(strict && own_th == th)) strict = false;
          th = own_th;
        }
        if (cut && tid == 0) sh.threshold = old_th;
        __syncthreads();
        continue;
      }
      // top_k searches for the largest key below the last one found, among the list and the chunk
      unsigned long long below = ~0ull;
      __syncthreads();
      for (int k = 0; k < p.top_k; ++k) {
        unsigned long long mine = 0;
        for (int i = tid; i < held; i += kThreads)
          if (sh.list[i] < below && sh.list[i] > mine) mine = sh.list[i];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int col = col0 + (i / N) * kThreads * N + i % N;
          if (col >= 0 && col < p.vocab) {
            const unsigned long long key = key_of(xs[i], col);
            if (key < below && key > mine) mine = key;
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const unsigned long long u = __shfl_xor_sync(0xFFFFFFFFu, mine, o);
          mine = u > mine ? u : mine;
        }
        if (lane == 0) sh.red[warp] = mine;
        __syncthreads();
        below = sh.red[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) below = sh.red[w] > below ? sh.red[w] : below;
        if (tid == 0) sh.best[k] = below;
        __syncthreads();
      }
      if (tid < p.top_k) sh.list[tid] = sh.best[tid];
      if (tid == 0) sh.count = p.top_k;  // more than kList numbers passed, so there are top_k
      __syncthreads();
      break;
    }
    if (!cut || sh.count > kCutAt) {
      __syncthreads();
      cut_back(sh, p.top_k);
      cut = sh.count == p.top_k;
    }
  }
  if (p.top_k) {
    __syncthreads();
    cut_back(sh, p.top_k);
  }

  // the block's sums
#pragma unroll
  for (int o = 16; o; o >>= 1)
    acc = join(acc, Sums{__shfl_xor_sync(0xFFFFFFFFu, acc.r, o), __shfl_xor_sync(0xFFFFFFFFu, acc.s, o),
                         __shfl_xor_sync(0xFFFFFFFFu, acc.t, o)}, p.c);
  if (lane == 0) sh.part[warp] = acc;
  __syncthreads();
  acc = sh.part[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) acc = join(acc, sh.part[w], p.c);

  if (p.splits > 1) {
    const int64_t at = row * p.splits + split;
    if (tid < p.top_k) p.keys[at * p.top_k + tid] = tid < sh.count ? sh.list[tid] : 0ull;
    if (tid == 0) *reinterpret_cast<float4*>(p.sums + at * 4) = make_float4(acc.r, acc.s, acc.t, 0.f);
    __syncthreads();
    if (tid == 0) {
      uint32_t old;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p.counter + row) : "memory");
      sh.last = old == (uint32_t)(p.splits - 1);
      if (sh.last) p.counter[row] = 0u;
      sh.count = 0;
    }
    __syncthreads();
    if (!sh.last) return;
    acc = Sums{-INFINITY, 0.f, 0.f};
    for (int i = 0; i < p.splits; ++i) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.sums + (row * p.splits + i) * 4));
      acc = join(acc, Sums{v.x, v.y, v.z}, p.c);
    }
    if (p.top_k) {
      const int total = p.splits * p.top_k;
      for (int base = 0; base < total; base += kList - kMaxTop) {  // as many as fit at a time
        const int n = total - base < kList - kMaxTop ? total - base : kList - kMaxTop;
        for (int i = tid; i < n; i += kThreads) {
          const unsigned long long key = __ldcg(p.keys + row * total + base + i);
          if (key) sh.list[atomicAdd(&sh.count, 1)] = key;
        }
        __syncthreads();
        cut_back(sh, p.top_k);
      }
    }
  }

  const float lns = logf(acc.s);
  const bool none = acc.r == -INFINITY;  // no number above minus infinity in the row
  if (tid == 0) {
    p.lse[row] = none ? -INFINITY : acc.r * p.inv_t + lns;
    p.entropy[row] = none ? 0.f : lns - kLn2 * (acc.t / acc.s);
  }
  const auto logprob = [&](float v) { return none ? -INFINITY : __fmaf_rn(v - acc.r, p.inv_t, -lns); };
  if (tid < p.top_k) {
    const unsigned long long key = sh.list[tid];
    p.top_ids[row * p.top_k + tid] = (int32_t)~(uint32_t)key;
    p.top_logprobs[row * p.top_k + tid] = logprob(from_order_bits((uint32_t)(key >> 32)));
  }
  for (int i = tid; i < p.cands; i += kThreads) {
    const int32_t tok = p.tokens[row * p.cands + i];
    p.logprobs[row * p.cands + i] = tok >= 0 && tok < p.vocab ? logprob(Vec<T>::one(x + tok)) : -INFINITY;
  }
}

// Blocks of a row: as many as make six blocks per SM over all rows, at most one per chunk.
int splits_of(int n, int chunks) {
  const int64_t want = 6 * (int64_t)device_sm_count();
  int64_t s = (want + n - 1) / n;
  if (s > chunks) s = chunks;
  if (s > 64) s = 64;
  if (n > kCounters) s = 1;
  return s < 1 ? 1 : (int)s;
}
// A row may start up to 15 bytes into its first vector: seven bf16 columns more.
int chunks_of(int vocab, int per_chunk) { return (vocab + 7 + per_chunk - 1) / per_chunk; }

}  // namespace

// Counters (always as many, so that a workspace serves calls of any sizes), sums [n][splits][4], keys [n][splits][top_k], for the larger split count of the two types.
size_t logprobs_workspace_bytes(int n, int vocab, int top_k) {
  const int64_t most = chunks_of(vocab, kThreads * kVecs * 4), splits = most < 64 ? most : 64;
  const int64_t rows = n < kCounters ? n : kCounters;  // only split rows use it
  return (size_t)(kCounters * 4 + rows * splits * 16 + (rows * splits * top_k * 8 + 15) / 16 * 16);
}

cudaError_t launch_token_logprobs(const void* logits, int dtype, int64_t row_stride, const int32_t* tokens, int n,
                                  int vocab, int cands, int top_k, float temperature, float* logprobs, float* lse,
                                  float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                                  cudaStream_t st) {
  Params p{};
  p.logits = logits; p.tokens = tokens;
  p.logprobs = logprobs; p.lse = lse; p.entropy = entropy; p.top_logprobs = top_logprobs; p.top_ids = top_ids;
  p.row_stride = row_stride;
  p.n = n; p.vocab = vocab; p.cands = cands; p.top_k = top_k;
  p.c = kLog2e / temperature;
  p.inv_t = 1.f / temperature;
  p.chunks = chunks_of(vocab, kThreads * kVecs * (dtype == TRELLIS_BF16 ? 8 : 4));
  p.splits = splits_of(n, p.chunks);
  char* w = static_cast<char*>(workspace);
  p.counter = reinterpret_cast<uint32_t*>(w);
  w += kCounters * 4;
  p.sums = reinterpret_cast<float*>(w);
  w += (int64_t)(n < kCounters ? n : kCounters) * p.splits * 16;
  p.keys = reinterpret_cast<unsigned long long*>(w);
  const int64_t kMaxRows = 65535;  // rows of one launch (a grid's y)
  for (int64_t r0 = 0; r0 < n; r0 += kMaxRows) {
    Params q = p;
    q.n = (int)(n - r0 < kMaxRows ? n - r0 : kMaxRows);
    const int64_t skip = r0 * row_stride * (dtype == TRELLIS_BF16 ? 2 : 4);
    q.logits = static_cast<const char*>(logits) + skip;
    q.tokens = tokens ? tokens + r0 * cands : nullptr;
    q.logprobs = logprobs ? logprobs + r0 * cands : nullptr;
    q.lse = lse + r0; q.entropy = entropy + r0;
    q.top_ids = top_ids ? top_ids + r0 * top_k : nullptr;
    q.top_logprobs = top_logprobs ? top_logprobs + r0 * top_k : nullptr;
    q.counter = p.counter + (p.splits > 1 ? r0 : 0);
    q.sums = p.sums + r0 * p.splits * 4;
    q.keys = p.keys + r0 * p.splits * top_k;
    const dim3 grid((unsigned)p.splits, (unsigned)q.n);
    const cudaError_t e = dtype == TRELLIS_BF16 ? launch_pdl(logprobs_kernel<uint16_t>, grid, dim3(kThreads), 0, st, q)
                                                : launch_pdl(logprobs_kernel<float>, grid, dim3(kThreads), 0, st, q);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace trellis

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
// distinct and the larger key is the earlier alternative.  While the sums run, each thread only keeps the largest
// number it has met.  The top_k-th largest of 64 maxima (of four threads each) is a threshold that at least top_k
// numbers reach, so only threads whose own maximum reaches it -- about top_k of 256 -- can hold an alternative:
// their numbers are read once more (from L2), what reaches the threshold is listed, and the list is put in order by counting
// larger keys.  Where more numbers reach it than the list holds, many are equal to it: those above it are listed, and
// the first equal ones from the block's first column on; if those above are too many as well, top_k rounds of a tournament
// between the threads take the next key each.
//
// A row is split over blocks where there are few rows; the last block to arrive joins the parts in their order, so
// results do not depend on timing.  Bound: latency for a row (1 x 50257 bf16, 5 alternatives: 7.7 us); for many rows the issue of the
// exponentials and sums, and the tail of alternatives that every block has: 61 x 128256 fp32 12.9 us (2.4 TB/s),
// 256 x 151936 bf16 with 20 alternatives 28 us (2.8 TB/s).
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerSM = 4;          // blocks of an SM at a time
constexpr int kList = 1024;        // numbers that may reach a threshold; kMaxTop * kMaxTop at least (see the join)
constexpr int kBatch = 4;          // 16-byte loads of a thread in flight
constexpr int kMaxSplits = 64;
constexpr int kCounters = 4096;    // rows that may be split
constexpr int kGroupThreads = 4;   // threads of one of the 64 maxima
constexpr float kLn2 = 0.693147180559945309f;
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
  int n, vocab, cands, top_k, splits;
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

// 16 bytes of logits: their numbers, their maximum (NaN if there is one).
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float2 pair(const uint4& u, int i) {
    const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
    return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
    return max_nan(bf16lo_to_f32(m), bf16hi_to_f32(m));
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ uint4 edge(const uint16_t* x, int col, int vocab) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = col + i >= 0 && col + i < vocab ? x[col + i] : 0xFF80u;
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float2 pair(const uint4& u, int i) {
    return i == 0 ? make_float2(__uint_as_float(u.x), __uint_as_float(u.y)) : make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)), max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ uint4 edge(const float* x, int col, int vocab) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = col + i >= 0 && col + i < vocab ? __float_as_uint(x[col + i]) : 0xFF800000u;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Vectors of a row begin on 16-byte boundaries: vector v holds columns v * N - skew .., those outside the row read as
// minus infinity.
template <typename T>
struct Row {
  const T* x;
  int skew, vocab;
  __device__ __forceinline__ int col(int v) const { return v * Vec<T>::N - skew; }
  __device__ __forceinline__ uint4 load(int v) const {
    const int c = col(v);
    if (c >= 0 && c + Vec<T>::N <= vocab) return *reinterpret_cast<const uint4*>(x + c);
    return Vec<T>::edge(x, c, vocab);
  }
};

struct Shared {
  alignas(16) unsigned long long list[kList];
  alignas(16) uint32_t group[64];
  unsigned long long best[kMaxTop];  // descending
  unsigned long long red[kWarps];
  Sums part[kWarps];
  int holders[kThreads];
  float threshold;
  int count, n_holders;
  uint32_t last;
};

// The list's sh.count keys cut back to the top_k largest, in descending order, in sh.best; sh.count follows.  The
// caller's barrier precedes it; ends with a barrier.
__device__ __forceinline__ void cut_back(Shared& sh, int top_k) {
  const int count = sh.count;
  // several threads count for one key where there are few
  const int per = count <= 32 ? 8 : count <= 64 ? 4 : count <= 128 ? 2 : 1;
  for (int i0 = 0; i0 < count; i0 += kThreads / per) {
    const int i = i0 + threadIdx.x / per;
    const unsigned long long mine = i < count ? sh.list[i] : 0ull;
    int rank = 0;
#pragma unroll 4
    for (int j = threadIdx.x % per; j < count; j += per) rank += sh.list[j] > mine;
    for (int o = 1; o < per; o <<= 1) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, o);
    if (i < count && rank < top_k && threadIdx.x % per == 0) sh.best[rank] = mine;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = count < top_k ? count : top_k;
  __syncthreads();
}

// A value that at least top_k of the block's numbers reach: the top_k-th largest of the 64 maxima.  Ends with a
// barrier.
__device__ __forceinline__ float find_threshold(Shared& sh, float thread_max, int top_k) {
  float g = thread_max;
#pragma unroll
  for (int o = 1; o < kGroupThreads; o <<= 1) g = max_nan(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
  if (threadIdx.x % kGroupThreads == 0) sh.group[threadIdx.x / kGroupThreads] = order_bits(g);
  __syncthreads();
  if (threadIdx.x < 64) {
    const uint32_t mine = sh.group[threadIdx.x];
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(sh.group + j);
      rank += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
      rank += (o.x == mine && j < (int)threadIdx.x) + (o.y == mine && j + 1 < (int)threadIdx.x) +
              (o.z == mine && j + 2 < (int)threadIdx.x) + (o.w == mine && j + 3 < (int)threadIdx.x);
    }
    if (rank == top_k - 1) sh.threshold = from_order_bits(mine);
  }
  __syncthreads();
  return sh.threshold;
}

// The largest key up to `most` among the vectors first + of, first + of + kThreads, .. of thread `of`, by a warp.  (A NaN in
// column 0 has the largest key there is.)
template <typename T>
__device__ __forceinline__ unsigned long long next_key(const Row<T>& row, int of, int first, int last, unsigned long long most) {
  constexpr int N = Vec<T>::N;
  unsigned long long best = 0;
  for (int v = first + of + (threadIdx.x & 31) * kThreads; v < last; v += 32 * kThreads) {
    const int c = row.col(v);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i >= 0 && c + i < row.vocab) {
        const unsigned long long key = key_of(Vec<T>::one(row.x + c + i), c + i);
        if (key <= most && key > best) best = key;
      }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long u = __shfl_xor_sync(0xFFFFFFFFu, best, o);
    best = u > best ? u : best;
  }
  return best;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSM) logprobs_kernel(const Params p) {
  pdl_enter();
  constexpr int N = Vec<T>::N;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = blockIdx.x;
  const int64_t row = blockIdx.y;
  Row<T> x;
  x.x = static_cast<const T*>(p.logits) + row * p.row_stride;
  x.skew = (int)((reinterpret_cast<uintptr_t>(x.x) & 15) / sizeof(T));
  x.vocab = p.vocab;
  const int vecs = (p.vocab + x.skew + N - 1) / N;
  const int first = (int)((int64_t)split * vecs / p.splits), last = (int)((int64_t)(split + 1) * vecs / p.splits);
  if (tid == 0) {
    sh.count = 0;
    sh.n_holders = 0;
  }

  // the given tokens' logits are fetched early, by every block of the row: the last one has them when it needs them
  float cand = 0.f;
  bool cand_ok = false;
  if (tid < p.cands) {
    const int32_t tok = p.tokens[row * p.cands + tid];
    cand_ok = tok >= 0 && tok < p.vocab;
    if (cand_ok) cand = Vec<T>::one(x.x + tok);
  }

  // ---- the sums, and each thread's largest number
  Sums acc{-INFINITY, 0.f, 0.f};
  const auto add = [&](const uint4 (&u)[kBatch], int n) {
    float m = acc.r;
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (b < n) m = max_nan(m, Vec<T>::max(u[b]));
    if (m != acc.r && acc.r != -INFINITY) {  // also where m is NaN
      const float d = max_nan((acc.r - m) * p.c, kFar), e = ex2(d);
      acc.t = (acc.t + acc.s * d) * e;
      acc.s *= e;
    }
    acc.r = m;
    if (m == -INFINITY) return;
    const float2 neg = make_float2(-m, -m), cc = make_float2(p.c, p.c);
    float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (b >= n) break;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        float2 y = __fmul2_rn(__fadd2_rn(Vec<T>::pair(u[b], i), neg), cc);
        y.x = max_nan(y.x, kFar);
        y.y = max_nan(y.y, kFar);
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        s = __fadd2_rn(s, e);
        t = __ffma2_rn(e, y, t);
      }
    }
    acc.s += s.x + s.y;
    acc.t += t.x + t.y;
  };
  {
    // the next batch's loads are in flight while one is worked on
    uint4 u[kBatch], next[kBatch];
    int v = first + tid, n = 0, more = 0;
    const auto fetch = [&](uint4 (&to)[kBatch], int at) {
      int k = 0;
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (at + b * kThreads < last) {
          to[b] = x.load(at + b * kThreads);
          k = b + 1;
        }
      return k;
    };
    n = fetch(u, v);
    while (n) {
      v += kBatch * kThreads;
      more = fetch(next, v);
      if (n == kBatch) add(u, kBatch);
      else add(u, n);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) u[b] = next[b];
      n = more;
    }
  }

  // ---- the alternatives
  if (p.top_k) {
    const float th = find_threshold(sh, acc.r, p.top_k);
    if (!(acc.r < th) && first + tid < last) sh.holders[atomicAdd(&sh.n_holders, 1)] = tid;
    __syncthreads();
    const int holders = sh.n_holders;
    // Lists what passes: numbers from the threshold up, or (strict) above it.  The holders' vectors are shared out over all threads
    // (a warp per holder, most of whose lanes have none where parts are short: 174 x 34577, 25 alternatives 14.1 us, 12.3 so).
    const int per = (last - first + kThreads - 1) / kThreads, again = holders * per;  // vectors of a holder, of all
    const auto collect = [&](bool strict) {
      for (int k = tid; k < again; k += kThreads) {
        const int h = k / per, v = first + sh.holders[h] + (k - h * per) * kThreads;
        if (v >= last) continue;
        const uint4 u = x.load(v);
        const float m = Vec<T>::max(u);
        if (strict ? m <= th : m < th) continue;
        const int c = x.col(v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 q = Vec<T>::pair(u, i >> 1);
          const float e = i & 1 ? q.y : q.x;
          if (!(strict ? e <= th : e < th) && c + i >= 0 && c + i < p.vocab) {
            const int at = atomicAdd(&sh.count, 1);
            if (at < kList) sh.list[at] = key_of(e, c + i);
          }
        }
      }
      __syncthreads();
    };
    collect(false);
    bool listed = sh.count <= kList;
    if (!listed) {
      // many numbers equal to the threshold (banned tokens, flat rows): those above it, and the first ones equal to it
      __syncthreads();
      if (tid == 0) sh.count = 0;
      __syncthreads();
      collect(true);
      const int above = sh.count;
      __syncthreads();  // read by all before anyone adds to it: the branch and the loop's end have to be the block's
      listed = above <= kList - 2 * kThreads;
      if (listed) {
        const int end = min(x.col(last), p.vocab);
        for (int c0 = max(x.col(first), 0); c0 < end; c0 += kThreads) {
          const int c = c0 + tid;
          if (c < end && Vec<T>::one(x.x + c) == th) {
            const int at = atomicAdd(&sh.count, 1);
            sh.list[at] = key_of(th, c);
          }
          __syncthreads();
          const bool enough = sh.count - above >= p.top_k;
          __syncthreads();
          if (enough) break;
        }
      }
    }
    if (listed) {
      cut_back(sh, p.top_k);
    } else {
      // a tournament: the threads' best keys, the best of which is taken and replaced by its thread's next
      __syncthreads();
      unsigned long long mine = 0;
      for (int t = warp * 32; t < warp * 32 + 32; ++t) {
        const unsigned long long k = next_key(x, t, first, last, ~0ull);
        if (t == tid) mine = k;
      }
      for (int k = 0; k < p.top_k; ++k) {
        unsigned long long b = mine;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const unsigned long long u = __shfl_xor_sync(0xFFFFFFFFu, b, o);
          b = u > b ? u : b;
        }
        const unsigned long long warp_best = b;
        if (lane == 0) sh.red[warp] = b;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) b = sh.red[w] > b ? sh.red[w] : b;
        if (tid == 0) sh.best[k] = b;
        if (warp_best == b) {  // this warp's thread holds it: keys are distinct (more than top_k numbers, so none is 0)
          const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, mine == b)) - 1;
          const unsigned long long next = next_key(x, warp * 32 + owner, first, last, b - 1);
          if (lane == owner) mine = next;
        }
        __syncthreads();
      }
      if (tid == 0) sh.count = p.top_k;
      __syncthreads();
    }
  }

  // ---- the block's sums
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
    if (tid < p.top_k) p.keys[at * p.top_k + tid] = tid < sh.count ? sh.best[tid] : 0ull;
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
    if (warp == 0) {  // the parts' sums, by a warp, while the others fetch keys
      Sums a{-INFINITY, 0.f, 0.f};
      for (int i = lane; i < p.splits; i += 32) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.sums + (row * p.splits + i) * 4));
        a = join(a, Sums{v.x, v.y, v.z}, p.c);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1)
        a = join(a, Sums{__shfl_xor_sync(0xFFFFFFFFu, a.r, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o),
                         __shfl_xor_sync(0xFFFFFFFFu, a.t, o)}, p.c);
      if (lane == 0) sh.part[0] = a;
    }
    // The parts' alternatives, each list in descending order.  Of the keys at depth d the m-th largest is reached by m lists
    // with d + 1 keys each, so with m (d + 1) >= top_k nothing below it counts.  Keys are distinct: no more than m lists reach it at
    // depth d, and others have at most d keys above it, which is m top_k + (splits - m) d <= kList in all (d is 0 where there
    // are as many lists as alternatives; all keys are no more than kList where there are fewer).  A part has more than
    // kMaxTop numbers, so none of its keys is missing.
    const int total = p.splits * p.top_k;
    if (total) {
      const int d = (p.top_k + p.splits - 1) / p.splits - 1, m = (p.top_k + d) / (d + 1);
      constexpr int kMine = kMaxSplits * kMaxTop / kThreads;
      unsigned long long key[kMine];
#pragma unroll
      for (int k = 0; k < kMine; ++k) key[k] = tid + k * kThreads < total ? __ldcg(p.keys + row * total + tid + k * kThreads) : 0ull;
      if (tid < p.splits) sh.list[tid] = __ldcg(p.keys + (row * p.splits + tid) * p.top_k + d);
      __syncthreads();
      if (tid < p.splits) {
        const unsigned long long mine = sh.list[tid];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < p.splits; ++j) rank += sh.list[j] > mine;
        if (rank == m - 1) sh.red[0] = mine;
      }
      __syncthreads();
      const unsigned long long from = sh.red[0];
#pragma unroll
      for (int k = 0; k < kMine; ++k)
        if (key[k] >= from && key[k]) sh.list[atomicAdd(&sh.count, 1)] = key[k];
      __syncthreads();
      cut_back(sh, p.top_k);
    }
    if (!total) __syncthreads();
    acc = sh.part[0];
  }

  const float lns = logf(acc.s);
  const bool none = acc.r == -INFINITY;  // no number above minus infinity in the row
  if (tid == 0) {
    p.lse[row] = none ? -INFINITY : acc.r * p.inv_t + lns;
    p.entropy[row] = none ? 0.f : lns - kLn2 * (acc.t / acc.s);
  }
  const auto logprob = [&](float v) { return none ? -INFINITY : __fmaf_rn(v - acc.r, p.inv_t, -lns); };
  if (tid < p.top_k) {
    const unsigned long long key = sh.best[tid];
    p.top_ids[row * p.top_k + tid] = (int32_t)~(uint32_t)key;
    p.top_logprobs[row * p.top_k + tid] = logprob(from_order_bits((uint32_t)(key >> 32)));
  }
  if (tid < p.cands) p.logprobs[row * p.cands + tid] = cand_ok ? logprob(cand) : -INFINITY;
}

// Blocks of a row: as many as the GPU holds at a time over all rows, each thread with one vector at least.  At 256
// rows of 151936 bf16 that is two; three do not all fit at a time.
int splits_of(int n, int vocab, int per_vec) {
  int64_t s = kPerSM * (int64_t)device_sm_count() / n;
  const int64_t most = (vocab + per_vec * kThreads - 1) / (per_vec * kThreads);
  if (s > most) s = most;
  if (s > kMaxSplits) s = kMaxSplits;
  if (n > kCounters) s = 1;
  return s < 1 ? 1 : (int)s;
}

}  // namespace

// Counters (always as many, so that a workspace serves calls of any sizes), sums [n][splits][4], keys
// [n][splits][top_k], for the larger split count of the two types.
size_t logprobs_workspace_bytes(int n, int vocab, int top_k) {
  size_t most = 0;
  // fewer rows have more splits each: a workspace for n rows serves fewer too
  for (int per_vec = 4; per_vec <= 8; per_vec += 4) {
    const int64_t one = splits_of(1, vocab, per_vec);
    const int64_t all = kPerSM * (int64_t)device_sm_count();  // rows * splits, where rows are split at all
    const int64_t parts = one * n < all ? one * n : all;
    const size_t b = (size_t)(kCounters * 4 + parts * 16 + (parts * top_k * 8 + 15) / 16 * 16);
    most = b > most ? b : most;
  }
  return most;
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
  p.splits = splits_of(n, vocab, dtype == TRELLIS_BF16 ? 8 : 4);
  char* w = static_cast<char*>(workspace);
  p.counter = reinterpret_cast<uint32_t*>(w);
  w += kCounters * 4;
  p.sums = reinterpret_cast<float*>(w);
  w += p.splits > 1 ? (int64_t)n * p.splits * 16 : 0;
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

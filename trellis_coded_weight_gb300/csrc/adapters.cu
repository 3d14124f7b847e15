// adapters.cu -- adds low-rank adapters to a projection's output (plan: adapter_plan.cuh).
//
//   h = A x  (fp32),  out = bf16(y + scale B h)
// A cluster of thread blocks takes a tile: up to 64 tokens of one adapter.  Each of its blocks multiplies its part of the inputs with A;
// the parts of h are added up through distributed shared memory, in the order of the blocks, and each block then makes its part of the
// outputs.  x, y and out are touched once, A and B once per tile (where clusters share a tile, x and A by each).  Both products are
// warp-level bf16 MMAs on operands that go from global memory straight into the fragments: a lane loads 16 (or 8) contiguous bytes of a
// row, and the reduction index is permuted alike on both sides so that these are what its fragments hold; likewise the outputs of four
// tiles of 8, so that a lane has 8 contiguous ones.  h enters the second product as the sum of two bf16 numbers.
// Where tiles are fewer than clusters (single tokens), and in the last round, several clusters share a tile: each computes h and makes a
// share of the outputs.
// Bound: 4096 tokens of rank 16, 5120 to 17408: bytes of x, y and out (60 us, 5.4 TB/s).  Higher ranks: the first product of a tile, at
// a few blocks of inputs in flight (4096 tokens, 17408 to 5120, rank 64 84 us, 128 137; A comes again with each tile).  Ranks 17 to 32:
// 4096 tokens, 5120 to 17408, 77 us (4.3 TB/s), in a kernel that spills 35 numbers a thread for two blocks an SM.  64 tokens of 40
// adapters to rank 64: 26 us (1.9 TB/s): a tile of rank 64 takes its cluster 19 whatever the others take, 9 of them before the second
// product, whose blocks of outputs then follow one another in each warp; and there are no more clusters than SMs / 4.  1 token: 5.2 us
// of latency (launch, plan, tokens, x and A, two cluster barriers, B).
// Clusters of 8: 115 us where 4 take 70, since each block reads as many parts of h as there are; of 2: 81.
#include "adapter_plan.cuh"
#include "common.cuh"
#include "devcache.h"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"
#include "tc_ptx.cuh"

namespace trellis {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 4;
constexpr int kCopyLd = 36;                // floats from token to token of a warp's products of 32 ranks: bank conflicts of two
constexpr int kCopy = 64 * kCopyLd;        // floats of a warp's products: 64 tokens by 32 ranks, or 32 by 64
constexpr int kCopyBytes = kWarps / 2 * kCopy * 4;
// A kernel for each bound on the rank: with ranks up to 32 two blocks of 128 registers a thread share an SM, with more one has it (204
// and 210 registers are used; two blocks: 4096 tokens of rank 64, 17408 inputs: 108 us for 97, spilling), which also leaves room for
// more copies in flight.
template <int RMAX>
struct Size {
  static constexpr int Blocks = RMAX <= 32 ? 2 : 1;    // of an SM
  static constexpr int Ring = (RMAX <= 32 ? 64 : 128) * 1024;  // copies in flight
  static constexpr int WarpRing = Ring / kWarps;
  // With more than 64 ranks h takes half of each warp's ring for the second product.
  static constexpr int WideRing = WarpRing / 2;
  static constexpr int Smem = kCopyBytes + Ring + kAdapterTile * 4;
  static_assert(kAdapterTile * kAdapterMaxRank * 4 <= Ring / 2, "h, as fragments");
  static_assert(Blocks * (Smem + 1024) <= 228 * 1024, "fits");
};
static_assert(kAdapterTile * 64 * 4 <= kCopyBytes / 2, "the second half of the products gives way to h");

struct AddParams {
  const uint16_t *x, *y;
  uint16_t* out;
  int64_t x_stride, y_stride, out_stride;
  trellis_adapters_t ad;
  const void* plan;
  int batch, n;
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float2 ld_cluster(const float* p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(tc::mapa_shared(p, rank)) : "memory");
  return v;
}
// The first `n` of the two bf16 numbers of w, the others zero.
__device__ __forceinline__ uint32_t first_of(uint32_t w, int n) { return n >= 2 ? w : n == 1 ? w & 0xFFFFu : 0u; }

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
// The first `bytes` of them, the others zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// How a block's warps share the first product: each has a part of the inputs and, of the tile's tokens and ranks,
//   up to 16 tokens  all tokens, 32 ranks
//   more             64 tokens by 32 ranks, or with more than 32 ranks 32 tokens by 64
// Where the sum over them of h[token][rank] lies: with the products of the first warp that has it.
template <int MT, int NB>
struct Share {
  static constexpr int Tokens = MT == 1 ? 16 : NB == 1 ? 64 : 32, Ranks = MT > 1 && NB > 1 ? 64 : 32;
  static constexpr int Sides = 16 * MT / Tokens, Groups = 32 * NB / Ranks, Splits = kWarps / (Sides * Groups);
  static __device__ __forceinline__ int at(int t, int r) {  // pairs of ranks stay pairs
    return (t / Tokens + Sides * (r / Ranks)) * kCopy + (Ranks == 64 ? (t % Tokens) * 2 + r / 32 % 2 : t % Tokens) * kCopyLd + r % 32;
  }
};

// h of the block's part of the inputs, for 16 MT tokens.  Where tokens are many, a lane copies what it needs of x into its warp's ring,
// some blocks of 32 inputs ahead (x comes from HBM; loads into registers kept half as many bytes in flight), and of A above 32 ranks;
// else A is loaded one block ahead.
template <int RMAX, int MT, bool NARROW, int NB>
__device__ __forceinline__ void shrink(const AddParams& p, const uint16_t* a, int rank, int count, const int* tokens, int rank_of_block,
                                       uint8_t* rings, float* copies) {
  using H = Share<MT, NB>;
  constexpr int kWarpRing = Size<RMAX>::WarpRing;
  constexpr int WT = H::Tokens / 16, NT = NARROW ? 2 : H::Ranks / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int side = warp % H::Sides, group = warp / H::Sides % H::Groups, split = warp / H::Sides / H::Groups;
  const int blocks = (int)((p.ad.in + 31) / 32);
  const int k0 = (int)((int64_t)rank_of_block * blocks / kCluster), k1 = (int)((int64_t)(rank_of_block + 1) * blocks / kCluster);
  const int t0 = side * H::Tokens, r0 = group * H::Ranks;
  const uint16_t* w = a + (int64_t)(r0 + g) * p.ad.in + 8 * q;
  const auto row_of = [&](int i) { return p.x + (int64_t)tokens[t0 + 8 * i + g] * p.x_stride + 8 * q; };
  const auto load_a = [&](int k, uint4 (&v)[NT]) {
    const bool in = k < k1 && 32 * k + 8 * q < p.ad.in;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (in && r0 + 8 * j + g < rank) v[j] = *reinterpret_cast<const uint4*>(w + (int64_t)(8 * j) * p.ad.in + 32 * k);
    }
  };
  float acc[WT][NT][4];
#pragma unroll
  for (int i = 0; i < WT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
  const auto multiply = [&](const uint4 (&u)[2 * WT], const uint4 (&v)[NT]) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < WT; ++i) {
        mma(acc[i][j], u[2 * i].x, u[2 * i + 1].x, u[2 * i].y, u[2 * i + 1].y, v[j].x, v[j].y);
        mma(acc[i][j], u[2 * i].z, u[2 * i + 1].z, u[2 * i].w, u[2 * i + 1].w, v[j].z, v[j].w);
      }
  };
  if (MT > 1) {
    constexpr bool kRingA = NT == 8;  // two sets of so many numbers of A do not fit in registers
    constexpr int kX = 2 * WT * 512, kStage = kX + (kRingA ? NT * 512 : 0), kStages = kWarpRing / kStage < 4 ? kWarpRing / kStage : 4;
    uint8_t* ring = rings + warp * kWarpRing;
    const auto copy = [&](int k, int s) {
      if (k < k1 && 32 * k + 8 * q < p.ad.in)
#pragma unroll
        for (int i = 0; i < 2 * WT; ++i)
          if (t0 + 8 * i + g < count) cp_async16(ring + s * kStage + (i * 32 + lane) * 16, row_of(i) + 32 * k);
      if (kRingA && k < k1 && 32 * k + 8 * q < p.ad.in)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (r0 + 8 * j + g < rank) cp_async16(ring + s * kStage + kX + (j * 32 + lane) * 16, w + (int64_t)(8 * j) * p.ad.in + 32 * k);
      cp_async_commit();
    };
    int k = k0 + split, stage = 0;
#pragma unroll
    for (int s = 0; s < kStages; ++s) copy(k + s * H::Splits, s);
    uint4 v[NT];
    if (!kRingA) load_a(k, v);
#pragma unroll 1
    for (; k < k1; k += H::Splits) {
      uint4 next[NT], u[2 * WT];
      if (!kRingA) load_a(k + H::Splits, next);
      cp_async_wait<kStages - 1>();
      const bool in = 32 * k + 8 * q < p.ad.in;
#pragma unroll
      for (int i = 0; i < 2 * WT; ++i) {
        u[i] = *reinterpret_cast<const uint4*>(ring + stage * kStage + (i * 32 + lane) * 16);
        if (!in || t0 + 8 * i + g >= count) u[i] = make_uint4(0, 0, 0, 0);
      }
      if (kRingA)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          v[j] = *reinterpret_cast<const uint4*>(ring + stage * kStage + kX + (j * 32 + lane) * 16);
          if (!in || r0 + 8 * j + g >= rank) v[j] = make_uint4(0, 0, 0, 0);
        }
      copy(k + kStages * H::Splits, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      multiply(u, v);
      if (!kRingA)
#pragma unroll
        for (int j = 0; j < NT; ++j) v[j] = next[j];
    }
    cp_async_wait<0>();
  } else {
    constexpr int kAhead = 3;  // blocks whose loads are in flight
    for (int k = k0 + split; k < k1; k += H::Splits * kAhead) {
      uint4 u[kAhead][2 * WT], v[kAhead][NT];
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int ks = k + s * H::Splits;
        const bool in = ks < k1 && 32 * ks + 8 * q < p.ad.in;
#pragma unroll
        for (int i = 0; i < 2 * WT; ++i) {
          u[s][i] = make_uint4(0, 0, 0, 0);
          if (in && t0 + 8 * i + g < count) u[s][i] = *reinterpret_cast<const uint4*>(row_of(i) + 32 * ks);
        }
        load_a(ks, v[s]);
      }
#pragma unroll
      for (int s = 0; s < kAhead; ++s) multiply(u[s], v[s]);
    }
  }
  // The sum over the warps that share tokens and ranks: half of those that are left hand theirs to the others.
  const auto at = [&](int i, int half, int j) {
    return (MT > 1 && H::Ranks == 64 ? (16 * i + 8 * half + g) * 2 + j / 4 : 16 * i + 8 * half + g) * kCopyLd + j % 4 * 8 + 2 * q;
  };
  const int mine = side + H::Sides * group;
#pragma unroll 1
  for (int left = H::Splits; left >= 1; left /= 2) {
    const int half = left / 2;  // splits half .. left - 1 write, 0 .. half - 1 add; at last split 0 writes the sum
    float* to = copies + (left == 1 ? mine : mine + H::Sides * H::Groups * (split - half)) * kCopy;
    if (left == 1 ? split == 0 : split >= half && split < left)
#pragma unroll
      for (int i = 0; i < WT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          *reinterpret_cast<float2*>(to + at(i, 0, j)) = make_float2(acc[i][j][0], acc[i][j][1]);
          *reinterpret_cast<float2*>(to + at(i, 1, j)) = make_float2(acc[i][j][2], acc[i][j][3]);
        }
    if (left == 1) break;
    __syncthreads();
    if (split < half) {
      const float* from = copies + (mine + H::Sides * H::Groups * split) * kCopy;
#pragma unroll
      for (int i = 0; i < WT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float2 x = *reinterpret_cast<const float2*>(from + at(i, 0, j)), y = *reinterpret_cast<const float2*>(from + at(i, 1, j));
          acc[i][j][0] += x.x;
          acc[i][j][1] += x.y;
          acc[i][j][2] += y.x;
          acc[i][j][3] += y.y;
        }
    }
    __syncthreads();
  }
}

// The sums over the cluster, as fragments: words of (token tile, block of 32 (NARROW: 16) ranks, step, high or low part), a lane's four
// together.  Blocks of 512 words lie one behind the other, or with more than 64 ranks two in the second half of each warp's ring.
template <int RMAX, bool NARROW, int NB>
__device__ __forceinline__ int fragment(int mt, int kb, int step, int low) {
  constexpr int kWarpRing = Size<RMAX>::WarpRing, kPerWarp = 16 / kWarps;
  if (NARROW) return (mt * 2 + low) * 128;
  const int block = mt * NB + kb;
  return (NB == 4 ? block / kPerWarp * (kWarpRing / 4) + kWarpRing / 8 + block % kPerWarp * 512 : block * 512) + (step * 2 + low) * 128;
}
// The two bf16 numbers (in the upper halves of floats) whose sum h is: cut off (which never overflows), and what that leaves, of the same
// sign.  Neither is zero unless h is: the least bf16 number (2^-133) stands in for it, since zero times an infinite number of B would be
// NaN where h times it is infinite.
__device__ __forceinline__ uint2 split(float h) {
  constexpr uint32_t kLeast = 0x00010000u;
  const uint32_t sign = __float_as_uint(h) & 0x80000000u, size = __float_as_uint(h) & 0x7FFFFFFFu;
  const uint32_t least = size ? kLeast : 0u, high = max(size & 0x7FFF0000u, least);
  const float low = __uint_as_float(size) - __uint_as_float(high);  // NaN where h is infinite
  return make_uint2(sign | high, sign | (low >= __uint_as_float(kLeast) ? __float_as_uint(low) : least));
}
template <int RMAX, int MT, bool NARROW, int NB>
__device__ __forceinline__ void gather(const float* copies, int rank, uint32_t* h) {
  constexpr int wide = NB * (NARROW ? 16 : 32) / 2;  // pairs of ranks
  for (int e = threadIdx.x; e < 16 * MT * wide; e += kThreads) {
    const int t = e / wide, r = (e - t * wide) * 2;
    float2 s = make_float2(0.f, 0.f);
    float2 v[kCluster];
#pragma unroll
    for (int c = 0; c < kCluster; ++c) v[c] = ld_cluster(copies + Share<MT, NB>::at(t, r), c);
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      s.x += v[c].x;
      s.y += v[c].y;
    }
    // ranks that the adapter does not have: zeros, since those of A times an infinite number of x are NaN
    if (r >= rank) s.x = 0.f;
    if (r + 1 >= rank) s.y = 0.f;
    const uint2 x = split(s.x), y = split(s.y);
    const int row = t & 15, kb = NARROW ? 0 : r >> 5;
    const int q = NARROW ? r >> 2 : (r & 31) >> 3, step = NARROW ? 0 : (r & 7) >> 2, pair = (r & 3) >> 1;
    const int word = ((row & 7) * 4 + q) * 4 + (row >> 3) + 2 * pair;
    h[fragment<RMAX, NARROW, NB>(t >> 4, kb, step, 0) + word] = (x.x >> 16) | y.x;
    h[fragment<RMAX, NARROW, NB>(t >> 4, kb, step, 1) + word] = pack_bf16x2(__uint_as_float(x.y), __uint_as_float(y.y));
  }
}

// The second product: outputs of blocks o0 + warp, + kWarps, .. < o1 of 32, for 16 MT tokens.  What a lane needs of y (few tokens: and
// of B) it copies itself into its warp's ring, some blocks ahead; the first ones before h is there.
template <int RMAX, int MT, bool NARROW, int NB>
struct Expand {
  static constexpr int kWarpRing = Size<RMAX>::WarpRing, kWideRing = Size<RMAX>::WideRing;
  static constexpr bool kRingB = MT == 1 && NB <= 2;  // B goes through the ring too, else it is loaded one block ahead
  static constexpr int kY = 2 * MT * 512, kB = kRingB ? 4 * NB * (NARROW ? 256 : 512) : 0, kStage = kY + kB;
  static constexpr int kFit = (NB == 4 ? kWideRing : kWarpRing) / kStage, kStages = kFit < 4 ? kFit : 4;
  static_assert(kStages >= 1, "a block");
  const AddParams& p;
  const uint16_t* b;
  const int* tokens;
  uint8_t* ring;  // the warp's
  const uint16_t* y_row[kRingB ? 2 : 1];  // kRingB: tokens g and 8 + g
  const uint16_t* next_b;  // kRingB: this lane's numbers of the next block to copy, for tile 0 and ranks 0 ..
  int rank, count, o, o1, lane, g, q, left, stage;

  __device__ __forceinline__ Expand(const AddParams& p_, const uint16_t* b_, int rank_, int count_, const int* tokens_, uint8_t* rings, int o0,
                                    int o1_)
      : p(p_), b(b_), tokens(tokens_), rank(rank_), count(count_), o1(o1_), stage(0) {
    const int warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    g = lane >> 2;
    q = lane & 3;
    o = o0 + warp;
    left = rank - (NARROW ? 4 : 8) * q;
    ring = rings + warp * kWarpRing;
    if constexpr (kRingB)
#pragma unroll
      for (int i = 0; i < 2; ++i) y_row[i] = p.y + (8 * i + g < count ? (int64_t)tokens[8 * i + g] * p.y_stride : 0) + 8 * q;
    next_b = b + (32 * (int64_t)o + 8 * (g >> 1) + (g & 1)) * p.ad.max_rank + (left > 0 ? (NARROW ? 4 : 8) * q : 0);
  }
  __device__ __forceinline__ void start() {
#pragma unroll
    for (int s = 0; s < kStages; ++s) copy(o + s * kWarps, s);
  }
  // This lane's numbers of B for tile j of 8 outputs and a block of ranks, where there are any.
  __device__ __forceinline__ const uint16_t* weights(int block, int j, int kb) const {
    const int64_t row = 32 * (int64_t)block + 8 * (g >> 1) + 2 * j + (g & 1);
    return row < p.ad.out && left > 32 * kb ? b + row * p.ad.max_rank + (NARROW ? 4 : 8) * q + 32 * kb : nullptr;
  }
  __device__ __forceinline__ void copy(int block, int s) {
    if (block < o1) {
      const int col = 32 * block + 8 * q;
      uint8_t* to = ring + s * kStage;
      if (col < p.ad.out)
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
          if (8 * i + g < count)
            cp_async16(to + (i * 32 + lane) * 16, kRingB ? y_row[kRingB ? i : 0] + 32 * block : p.y + (int64_t)tokens[8 * i + g] * p.y_stride + col);
      // Ranks that the adapter has not become zeros (the address is one of its own all the same).  Outputs past the end have whatever
      // the ring holds; their results are not stored.
      if constexpr (kRingB) {
        const uint16_t* from = next_b;
        const uint32_t at = tc::smem_u32(to) + kY + lane * (NARROW ? 8 : 16);
        const int rows = (int)p.ad.out - 32 * block - 8 * (g >> 1) - (g & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j, from += 2 * p.ad.max_rank) {
          if (2 * j >= rows) break;
#pragma unroll
          for (int kb = 0; kb < NB; ++kb) {
            if (NARROW) cp_async8(at + j * 256, from, 2 * max(0, min(left, 4)));
            else cp_async16(at + (j * NB + kb) * 512, from + (left > 32 * kb ? 32 * kb : 0), 2 * max(0, min(left - 32 * kb, 8)));
          }
        }
        next_b += (int64_t)kWarps * 32 * p.ad.max_rank;
      }
    }
    cp_async_commit();
  }
  __device__ __forceinline__ void load(int block, uint4 (&v)[4][NB]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int kb = 0; kb < NB; ++kb) {
        v[j][kb] = make_uint4(0, 0, 0, 0);
        const uint16_t* at = block < o1 ? weights(block, j, kb) : nullptr;
        if (!at) continue;
        if (NARROW) {
          const uint2 two = *reinterpret_cast<const uint2*>(at);
          v[j][kb].x = two.x;
          v[j][kb].y = two.y;
        } else {
          v[j][kb] = *reinterpret_cast<const uint4*>(at);
        }
      }
  }
  __device__ __forceinline__ void run(const uint32_t* h, float scale) {
    const uint32_t* hl = h + 4 * lane;
    const bool ragged = rank % (NARROW ? 4 : 8) != 0;
    uint4 v[4][NB], next[4][NB];
    if constexpr (!kRingB && NB < 4) load(o, next);
    // Few tokens: h stays in registers, since reading it again with every block takes as much of shared memory's bandwidth as B does
    // (64 adapters of rank 16: 19 us so, 16).
    constexpr int kSteps = NARROW ? 2 : 4;  // high and low parts of each step
    uint4 held[kRingB ? NB : 1][kSteps];
    if constexpr (kRingB)
#pragma unroll
      for (int kb = 0; kb < NB; ++kb)
#pragma unroll
        for (int f = 0; f < kSteps; ++f) held[kb][f] = *reinterpret_cast<const uint4*>(hl + fragment<RMAX, NARROW, NB>(0, kb, f >> 1, f & 1));
#pragma unroll 1
    for (; o < o1; o += kWarps) {
      cp_async_wait<kStages - 1>();
      const uint8_t* from = ring + stage * kStage;
      uint4 u[2 * MT];
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i)
        u[i] = *reinterpret_cast<const uint4*>(from + (i * 32 + lane) * 16);
      if constexpr (kRingB) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int kb = 0; kb < NB; ++kb) {
            if (NARROW) {
              const uint2 two = *reinterpret_cast<const uint2*>(from + kY + (j * 32 + lane) * 8);
              v[j][kb] = make_uint4(two.x, two.y, 0, 0);
            } else {
              v[j][kb] = *reinterpret_cast<const uint4*>(from + kY + ((j * NB + kb) * 32 + lane) * 16);
            }
          }
      } else if constexpr (NB < 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int kb = 0; kb < NB; ++kb) v[j][kb] = next[j][kb];
        load(o + kWarps, next);
      } else {
        load(o, v);
      }
      copy(o + kStages * kWarps, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if (!kRingB && ragged)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int kb = 0; kb < NB; ++kb) {
            const int n = left - 32 * kb;
            v[j][kb] = make_uint4(first_of(v[j][kb].x, n), first_of(v[j][kb].y, n - 2), first_of(v[j][kb].z, n - 4), first_of(v[j][kb].w, n - 6));
          }
      const int col = 32 * o + 8 * q;
      const bool in = col < p.ad.out;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (16 * i >= count) break;
        float acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
          for (int f = 0; f < kSteps; ++f) {
            uint4 a;
            if constexpr (kRingB) a = held[kb][f];
            else a = *reinterpret_cast<const uint4*>(hl + fragment<RMAX, NARROW, NB>(i, kb, f >> 1, f & 1));
            const bool second = f >= 2;
#pragma unroll
            for (int j = 0; j < 4; ++j) mma(acc[j], a.x, a.y, a.z, a.w, second ? v[j][kb].z : v[j][kb].x, second ? v[j][kb].w : v[j][kb].y);
          }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int t = 16 * i + 8 * half + g;
          if (!in || t >= count) continue;
          const uint4 y = u[2 * i + half];
          const auto add = [&](uint32_t w, int j) {
            return pack_bf16x2(fmaf(scale, acc[j][2 * half], bf16lo_to_f32(w)), fmaf(scale, acc[j][2 * half + 1], bf16hi_to_f32(w)));
          };
          *reinterpret_cast<uint4*>(p.out + (int64_t)tokens[t] * p.out_stride + col) = make_uint4(add(y.x, 0), add(y.y, 1), add(y.z, 2), add(y.w, 3));
        }
      }
    }
    cp_async_wait<0>();
  }
};

template <int RMAX, int MT, bool NARROW, int NB>
__device__ __forceinline__ void tile_of(const AddParams& p, const int4& tile, int rank, float scale, const int* tokens, int o0, int o1,
                                        float* copies, uint8_t* ring) {
  const uint16_t *a = p.ad.a + (int64_t)tile.x * p.ad.max_rank * p.ad.in, *b = p.ad.b + (int64_t)tile.x * p.ad.out * p.ad.max_rank;
  uint32_t* h = reinterpret_cast<uint32_t*>(NB == 4 ? ring : reinterpret_cast<uint8_t*>(copies) + kCopyBytes / 2);
  Expand<RMAX, MT, NARROW, NB> second(p, b, rank, tile.z, tokens, ring, o0, o1);
  if (MT == 1) second.start();
  shrink<RMAX, MT, NARROW, NB>(p, a, rank, tile.z, tokens, (int)tc::cluster_ctarank(), ring, copies);
  if (MT > 1) second.start();  // the ring is free
  cluster_arrive();
  cluster_wait();
  gather<RMAX, MT, NARROW, NB>(copies, rank, h);
  cluster_arrive();  // this block has read the others' sums
  __syncthreads();
  second.run(h, scale);
  cluster_wait();
}
template <int RMAX, int MT>
__device__ __forceinline__ void tile_by_rank(const AddParams& p, const int4& tile, int rank, float scale, const int* tokens, int o0, int o1,
                                             float* copies, uint8_t* ring) {
  if (rank <= 16) return tile_of<RMAX, MT, true, 1>(p, tile, rank, scale, tokens, o0, o1, copies, ring);
  if constexpr (RMAX > 16)
    if (rank <= 32) return tile_of<RMAX, MT, false, 1>(p, tile, rank, scale, tokens, o0, o1, copies, ring);
  if constexpr (RMAX > 32)
    if (rank <= 64) return tile_of<RMAX, MT, false, 2>(p, tile, rank, scale, tokens, o0, o1, copies, ring);
  if constexpr (RMAX > 64) tile_of<RMAX, MT, false, 4>(p, tile, rank, scale, tokens, o0, o1, copies, ring);
}

__device__ __forceinline__ int rank_of(const AddParams& p, int adapter) {
  const bool has = adapter >= 0 && adapter < p.ad.count;
  const int rank = has ? p.ad.ranks ? p.ad.ranks[adapter] : p.ad.max_rank : 0;
  return rank < 0 ? 0 : rank > p.ad.max_rank ? p.ad.max_rank : rank;
}

// The tiles by falling rank, where there are more of them than clusters.  Whether those of the first round differ in rank.
constexpr int kSorted = kThreads;
__device__ __noinline__ bool sort_tiles(const AddParams& p, int tiles, int clusters, int* ranks, uint16_t* order) {
  const int t = threadIdx.x;
  ranks[t] = t < tiles ? rank_of(p, __ldcg(adapter_tiles(p.plan) + t).x) : -1;
  __syncthreads();
  const int mine = ranks[t];
  int place = 0;
  for (int i = 0; i < tiles; ++i) place += ranks[i] > mine || (ranks[i] == mine && i < t);
  if (t < tiles) order[place] = (uint16_t)t;
  __syncthreads();
  const bool differ = ranks[order[0]] != ranks[order[clusters - 1]];
  __syncthreads();  // the ranks' place is used again
  return differ;
}

template <int RMAX>
__global__ void __launch_bounds__(kThreads, Size<RMAX>::Blocks) add_kernel(const __grid_constant__ AddParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  float* copies = reinterpret_cast<float*>(raw);
  uint8_t* ring = raw + kCopyBytes;
  int* tokens = reinterpret_cast<int*>(raw + kCopyBytes + Size<RMAX>::Ring);
  pdl_enter();
  const int4 head = __ldcg(static_cast<const int4*>(p.plan));
  const int tiles = p.out == p.y ? head.y : head.x;  // in place there is nothing to do for tokens without an adapter
  const int32_t* order = adapter_order(p.plan, p.batch, p.n);
  const int cluster = blockIdx.x / kCluster, clusters = gridDim.x / kCluster, rank_of_block = (int)tc::cluster_ctarank();
  const int blocks = (int)((p.ad.out + 31) / 32);
  constexpr bool kSort = RMAX > 32;  // below that tiles cost about the same
  __shared__ uint16_t order_of[kSort ? kSorted : 1];
  const bool sorted = kSort && p.ad.ranks && tiles > clusters && tiles <= kSorted;
  const bool turns = kSort && sorted && sort_tiles(p, tiles, clusters, reinterpret_cast<int*>(raw), order_of);
  bool back = false;  // every other round where ranks differ
  for (int t0 = 0; t0 < tiles; t0 += clusters, back = turns && !back) {
    // The round's tiles; where they are few, as many clusters for each as have a block of outputs per warp.  Back: the clusters whose
    // last tile was least take the first ones, and few tiles are shared by two thirds of the clusters, those that are free first (by
    // all: 31 us for 27, 64 tokens of 40 adapters to rank 64).  With equal ranks all are free at once (50 adapters of rank 64: 40 us,
    // 45 shared by two thirds).
    const int now = min(tiles - t0, clusters);
    const int shares = max(1, min((kSort && back ? clusters * 2 / 3 : clusters) / now, blocks / (kCluster * kWarps)));
    const int me = kSort && back ? clusters - 1 - cluster : cluster;
    if (me >= now * shares) break;
    const int at = t0 + me % now;
    const int4 tile = __ldcg(adapter_tiles(p.plan) + (kSort && sorted ? order_of[at] : at));
    const int share = (me / now) * kCluster + rank_of_block, all = shares * kCluster;
    const int o0 = (int)((int64_t)share * blocks / all), o1 = (int)((int64_t)(share + 1) * blocks / all);
    const int rank = rank_of(p, tile.x);
    __syncthreads();
    if (threadIdx.x < tile.z) tokens[threadIdx.x] = __ldcg(order + tile.y + threadIdx.x);
    __syncthreads();
    if (rank == 0) {
      if (p.out == p.y) continue;
      const int chunks = (min(32 * o1, (int)p.ad.out) - 32 * o0) / 8;
      for (int e = threadIdx.x; e < tile.z * chunks; e += kThreads) {
        const int64_t token = tokens[e / chunks], col = 32 * o0 + 8 * (e % chunks);
        *reinterpret_cast<uint4*>(p.out + token * p.out_stride + col) = *reinterpret_cast<const uint4*>(p.y + token * p.y_stride + col);
      }
      continue;
    }
    const float scale = p.ad.scales ? p.ad.scales[tile.x] : 1.f;
    // in this order: ragged prompts 82 us, and 92 with the code of few tokens in front
    if (tile.z > 16) tile_by_rank<RMAX, 4>(p, tile, rank, scale, tokens, o0, o1, copies, ring);
    else tile_by_rank<RMAX, 1>(p, tile, rank, scale, tokens, o0, o1, copies, ring);
  }
}

}  // namespace

namespace {

template <int RMAX>
int clusters_of(int dev) {
  static PerDevice<int> of;
  return of.get(dev, [] {
    const auto kern = add_kernel<RMAX>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Size<RMAX>::Smem) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Size<RMAX>::Smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
    return n;
  }, 0);
}

template <int RMAX>
cudaError_t launch_rank(const AddParams& p, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const int fit = clusters_of<RMAX>(dev);
  if (fit < 1) return cudaErrorInvalidConfiguration;
  // no more clusters than there can be shares of tiles
  const int64_t shares = (p.ad.out + 31) / 32 / (kCluster * kWarps), most = adapter_max_tiles(p.batch, p.n) * (shares < 1 ? 1 : shares);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < fit ? most : fit) * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Size<RMAX>::Smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, add_kernel<RMAX>, p);
}

}  // namespace

// Clusters that the device runs at once, where two blocks share an SM; half as many where one has it.
int adapter_clusters() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess ? clusters_of<16>(dev) : 0;
}

cudaError_t launch_adapter_add(const uint16_t* x, int64_t x_stride, const uint16_t* y, int64_t y_stride, uint16_t* out,
                               int64_t out_stride, const trellis_adapters_t& ad, const void* plan, int batch, int n,
                               cudaStream_t st) {
  const AddParams p{x, y, out, x_stride, y_stride, out_stride, ad, plan, batch, n};
  return ad.max_rank <= 16 ? launch_rank<16>(p, st) : ad.max_rank <= 32 ? launch_rank<32>(p, st)
       : ad.max_rank <= 64 ? launch_rank<64>(p, st) : launch_rank<128>(p, st);
}

}  // namespace trellis

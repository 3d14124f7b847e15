// prompt_attention.cu -- causal attention of whole prompts over the paged cache, on the 5th-generation tensor cores.
//
// A thread block takes a block of query rows of one key/value head and 128 keys per step; both products are 128-row tcgen05
// MMAs of one issuing warp with accumulators in tensor memory:
//   S = Q K^T    Q and K in shared memory (128-byte swizzle, along the head dim)
//   O += P V     P in tensor memory over the scores it was made of, V in shared memory (swizzled, along the head dim too)
// The softmax is in one pass with a running maximum (tree_tc.cuh).  Heads of 64 and 128: 256 rows, two streams of 128 with an S
// and an O each, so that one's products run while the other's softmax does.  Heads of 256, whose O takes half of tensor memory:
// 128 rows, one stream whose tiles alternate between two S.
// Rows see keys up to their own position: only the last tiles of an item are masked, and streams end where their rows do.
// Keys and values arrive by TMA in a ring of slots in the order of their use.  Of an e4m3 cache the keys are multiplied as they are, as
// in tree_attention_tc1.cu: each row of queries is scaled by a power of two and split into an e4m3 and an e5m2 number, exactly down to
// 2^-13 of the row's largest and within 2^-21 of it below, so S is two 8-bit products at twice the rate.  The values are copied into
// the upper half of a slot and widened in place to fp16 (exact); P is fp16 then, since weights of 4 bits would not do.  (Keys widened
// too: 8192 tokens of heads of 256 took 730 us.)  Values that a product must not meet (rows past the end, numbers that are not finite
// where not every row sees them) are cleared on the way, the latter added back for the rows that see them (rare).
// The warps: one that plans and copies, one that issues, two that bring the queries; two softmax warpgroups (a thread per row); a
// warpgroup that widens and clears (two with e4m3 and heads of 256, whose second softmax warpgroup has nothing else to do).
// Weights are rounded to 16 bits for the product with the values, in their type: an MMA's operands are both bf16 or both fp16.  (Error
// against 64 bits: 0.0021 of the outputs' size with a bf16 cache, 0.0016 from their own rounding alone.)  Their sum is not rounded.
// Bound: the products, and what lies between them.  A tile of a stream is 1024 cycles of products with heads of 128 (512 with 64,
// 2048 with 256) and takes 1480: S at N = 128 needs all of shared memory's bandwidth, which the copies also want, and a commit before
// a wait costs the issuing warp 70 cycles.  16384 tokens, 32/8 heads of 128: 1.43 ms (1.54 PFLOP/s); 8192 tokens, 16/2 of 256: 385 us
// (1.43).  With e4m3 545 (1.01; 4 x 4096 tokens, 32/8 of 128: 525): each block widens the values for its own rows, and tensor pipe, shared
// memory and issue slots are each busy for 40 to 50 % of the time.  Heads of 64: tensor pipe and exponentials are busy for 35 % each; a
// pair of tiles takes 2920 cycles, 1024 in each of them, since a stream has one S and its scores, maximum, weights and product follow one
// another: 8192 tokens, 64/8 661 us (0.83).  Short items pay 5000 cycles each for their end and the first weights of the next: 16 sequences to 2000
// tokens 330 us (1.15).
#include <cstring>
#include <cuda.h>

#include "common.cuh"
#include "devcache.h"
#include "launch.h"
#include "pdl.cuh"
#include "prompt_sched.cuh"
#include "serving.h"
#include "tc_ptx.cuh"
#include "tree_sched.cuh"
#include "tree_tc.cuh"

namespace trellis {
namespace {

using namespace tree;
using prompt::kTile;
using prompt::Work;

__device__ int g_prompt_error = 0;  // set when a bounded wait gives up (trellis_device_error)

constexpr int kThreads = 512;
constexpr int kCopyWarp = 0, kMmaWarp = 1, kQueryWarp = 2, kSoftmaxWarp = 4, kWidenWarp = 12;
constexpr int kSoftmaxRegs = 152, kIssueRegs = 96, kWidenRegs = 112;
static_assert(2 * kSoftmaxRegs + kIssueRegs + kWidenRegs <= 65536 / 128, "what the block was launched with");
constexpr int kWorks = 4;  // stretches that the copying warp has announced
constexpr int kOdd = 8;    // items whose odd values are known at a time: the widening warps are a few ahead of the softmax at the most

template <int D>
struct Cfg {
  static constexpr int Streams = D == 256 ? 1 : 2;
  static constexpr int Rows = 128 * Streams;
  static constexpr int Cols = D < 128 ? D : 128;    // of a slot, which has them for all keys of a tile
  static constexpr int Parts = D / Cols;            // slots of a tile's keys, or values
  static constexpr int Slot = kTile * Cols * 2;
  static constexpr int Slots = D == 64 ? 8 : 4;
  static constexpr int Blocks = Cols / 64;          // 128-byte blocks of a row
  // In a slot 8 rows of a block lie together (1024 bytes), then the blocks of these rows, then the next 8 rows: one copy brings
  // whole pages so.
  static constexpr int Group = Blocks * 1024;
  static __device__ __forceinline__ int at(int row, int chunk) {  // 8 numbers
    return (row >> 3) * Group + (chunk >> 3) * 1024 + (row & 7) * 128 + (((chunk & 7) ^ (row & 7)) << 4);
  }
  static constexpr int QTile = 128 * D * 2;         // bf16, or two 8-bit numbers: the high parts, then the low ones
  static constexpr int QBuffers = D == 64 ? 2 : 1;  // the next stretch's queries are brought early where there is room
  // An 8-bit row of a slot (a block): 128 bytes in the 128-byte swizzle, or 64 in the 64-byte one.
  static __device__ __forceinline__ int at8(int row, int chunk) {  // 16 numbers
    return row * Cols + ((chunk ^ (Cols == 128 ? row & 7 : row >> 1 & 3)) << 4);
  }
  static constexpr int Stage = 32 * 64;             // 32 columns of a warp's rows, on their way out
  static constexpr int Fixed = (int)sizeof(prompt::Map) + kWorks * (int)sizeof(Work) + 4 * Rows * 4 + 1024;
  static constexpr int Smem = 1024 + Slots * Slot + Streams * (QBuffers * QTile + 4 * Stage) + Fixed;
  static_assert(Smem <= 227 * 1024, "fits");
  template <bool F8>
  static constexpr float Lift = F8 ? 7.f : 0.f;     // log2 of a factor of the weights: with it fp16 ones reach 2^15
  // tensor memory columns
  static constexpr int S(int s) { return s * 128; }
  static constexpr int O(int s) { return 256 + s * D; }
};

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Issued by a converged warp with operands that are the warp's, like the products (tree_tc.cuh): copies from lanes of their own are
// taken one lane after the other, some 200 cycles each (8192 tokens, heads of 64, pages of 64: 657 us so).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}"
      ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int block, int group) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%5, %5, %3, %4}], [%2];\n\t}"
      ::"r"(dst), "l"(map), "r"(bar), "r"(block), "r"(group), "r"(0)
      : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
      : "memory");
}

// Two e4m3 numbers as fp16, exactly.
__device__ __forceinline__ uint32_t widen2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// A wait's first look, of a warp: 16 cycles where the phase is complete, as it mostly is (a try with a time limit takes 70).
__device__ __forceinline__ bool is_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return __all_sync(0xFFFFFFFFu, ok != 0);
}

// D[tmem] (+)= A[smem desc] * B[smem desc], 8-bit inputs, each of the kind that the descriptor says, fp32 accumulate.
__device__ __forceinline__ void mma_ss_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
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
// 8 bf16 numbers times f as e4m3 numbers (four in h0, four in h1) and e5m2 ones of what these leave.
__device__ __forceinline__ void split8(const uint4& u, uint32_t flip, float f, uint32_t& h0, uint32_t& h1, uint32_t& l0, uint32_t& l1) {
  const uint32_t x[4] = {u.x ^ flip, u.y ^ flip, u.z ^ flip, u.w ^ flip};
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int z = 0; z < 4; ++z) {
    const float a = bf16lo_to_f32(x[z]) * f, b = bf16hi_to_f32(x[z]) * f;
    hi[z] = e4m3x2(a, b);
    const uint32_t back = widen2((uint16_t)hi[z]);
    lo[z] = e5m2x2(a - f16_to_f32((uint16_t)back), b - f16_to_f32((uint16_t)(back >> 16)));
  }
  h0 = hi[0] | hi[1] << 16;
  h1 = hi[2] | hi[3] << 16;
  l0 = lo[0] | lo[1] << 16;
  l1 = lo[2] | lo[3] << 16;
}
// As desc_mnmajor (tree_tc.cuh), `sbo` bytes from 8 rows to the next 8.
__device__ __forceinline__ uint64_t desc_values(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (desc_mnmajor(saddr, lbo) & ~((uint64_t)0x3FFF << 32)) | (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
}

// The order in which an item's tiles of keys and values are copied and used: place of tile t's keys or values among 2n.
template <int Streams>
__device__ __forceinline__ int place_of(int t, bool value, int n) {
  if (Streams == 2) return 2 * t + (value ? 1 : 0);
  return value ? (t == n - 1 ? 2 * n - 1 : 2 * t + 2) : (t == 0 ? 0 : 2 * t - 1);  // keys of the next tile before a tile's values
}
template <int Streams>
__device__ __forceinline__ int tile_at(int place, int n, bool* value) {
  if (Streams == 2) {
    *value = place & 1;
    return place >> 1;
  }
  if (place < 2 && place < n) { *value = false; return place; }
  if (place == 2 * n - 1) { *value = true; return n - 1; }
  *value = !(place & 1);
  return place & 1 ? (place + 1) / 2 : (place - 2) / 2;
}

// Adds the values that were cleared since they are not finite, times f, to the numbers of a row that sees them (bf16 ones, or floats
// four columns apart by `stride`).  Rare, and out of the way: its code would be in all rows' way else.
template <int D, bool F8>
__device__ __noinline__ void add_odd(const TreeParams& p, int b, int head, int from, int to, float f, uint16_t* out, float* part, int stride) {
  for (int pos = from; pos < to; ++pos) {
    int page = p.table[(int64_t)b * p.width + (pos >> p.page_shift)];
    page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
    const int64_t at = (((((int64_t)page * 2 + 1) * p.hkv + head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1))) * D;
    for (int q = 0; q < D; ++q) {
      float x;
      if (F8) {
        if ((static_cast<const uint8_t*>(p.pool)[at + q] & 0x7F) != 0x7F) continue;
        x = __uint_as_float(0x7FFFFFFFu);
      } else {
        const uint16_t v = static_cast<const uint16_t*>(p.pool)[at + q];
        if ((v & 0x7F80u) != 0x7F80u) continue;
        x = bf16_to_f32(v);
      }
      if (out) out[q] = f32_to_bf16_rn(bf16_to_f32(out[q]) + x * f);
      else part[(int64_t)(q >> 2) * stride + (q & 3)] += x;
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TreeParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = base;
  uint8_t* sq = ring + C::Slots * C::Slot;
  uint8_t* stages = sq + C::QBuffers * C::Streams * C::QTile;
  float* row_up = reinterpret_cast<float*>(stages + C::Streams * 4 * C::Stage);  // e4m3: [stretch % 4][row] log2 of the queries' scale
  prompt::Map& plan = *reinterpret_cast<prompt::Map*>(row_up + 4 * C::Rows);
  Work* works = reinterpret_cast<Work*>(&plan + 1);
  uint64_t* full = reinterpret_cast<uint64_t*>((reinterpret_cast<uintptr_t>(works + kWorks) + 7) & ~(uintptr_t)7);
  uint64_t* raw_full = full + C::Slots;   // of values that are widened, or cleared, first.  A thread that waits for a phase has to have
  uint64_t* empty = raw_full + C::Slots;  // seen the one before, and the widening warps see no others
  uint64_t* ready = empty + C::Slots;   // widened, or clear
  uint64_t* q_full = ready + C::Slots;  // [QBuffers]
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;       // [2] scores there
  uint64_t* p_ready = s_full + 2;       // [2] weights written
  uint64_t* o_full = p_ready + 2;       // [2] the stretch's last product complete
  uint64_t* o_done = o_full + 2;        // one stream: each product with the values
  uint64_t* w_full = o_done + 1;        // [kWorks] a stretch announced
  uint64_t* w_empty = w_full + kWorks;
  uint64_t* drained = w_empty + kWorks;
  volatile int* flags = reinterpret_cast<volatile int*>(drained + 1);  // [0] a wait gave up
  volatile int* odd_of = flags + 4;     // [stretch % kOdd] the stretch, if it has odd values
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(flags) + 4 + kOdd);

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&map);
    for (int i = 0; i < C::Slots; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(raw_full + i, 1);
      tc::mbar_init(empty + i, 1);
      tc::mbar_init(ready + i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(q_full + i, 2);
      tc::mbar_init(q_empty + i, 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(s_full + s, 1);
      tc::mbar_init(p_ready + s, 4);
      tc::mbar_init(o_full + s, 1);
    }
    tc::mbar_init(o_done, 1);
    for (int i = 0; i < kWorks; ++i) {
      tc::mbar_init(w_full + i, 1);
      tc::mbar_init(w_empty + i, 7 + 4 * C::Streams + (F8 && C::Streams == 1 ? 4 : 0));
    }
    tc::mbar_init(drained, 1);
    flags[0] = 0;
    for (int i = 0; i < kOdd; ++i) odd_of[i] = -1;
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  pdl_enter();
  prompt::plan<C::Rows>(p, plan, (int)gridDim.x, reinterpret_cast<int*>(sq));
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(*tmem_slot);
  bool dead = false;
  const auto wait = [&](uint64_t* bar, uint32_t parity) {  // of a converged warp
    if (is_done(bar, parity)) return !dead;
    const bool ok = dead || tc::mbar_wait_short(bar, parity, p.wait_ns);
    if (__any_sync(0xFFFFFFFFu, !ok)) {
      dead = true;
      if (lane == 0) flags[0] = 1;
    }
    return !dead;
  };
  // The k-th stretch, for the warps that are told; false where there is none.
  const auto told = [&](int k, Work& w) {
    const int s = k % kWorks;
    if (!wait(w_full + s, (uint32_t)(k / kWorks & 1))) return false;
    w = works[s];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(w_empty + s);
    return w.more != 0;
  };

  constexpr bool kTwoWiden = F8 && C::Streams == 1;  // the second softmax warpgroup widens too: the odd slots
  if (warp >= kWidenWarp || (kTwoWiden && warp >= kSoftmaxWarp + 4 && warp < kSoftmaxWarp + 8)) {
    // ---- widening and clearing
    if (warp >= kWidenWarp) regs_down<kWidenRegs>();
    else regs_up<kSoftmaxRegs>();
    const int tid = threadIdx.x & 127, group_bar = warp >= kWidenWarp ? 2 : 3;
    Work w;
    int e0 = 0;
    uint32_t f_phase = 0;  // per slot
    // the group's warps meet at barriers, so they leave together
    for (int k = 0; tc::bar_and(told(k, w), group_bar, 128); ++k) {
      const int n = w.tiles;
      const int shared_to = w.shared0;  // keys that every row sees
      for (int e = 0; e < 2 * n && !dead; ++e) {
        bool value;
        const int t = tile_at<C::Streams>(e, n, &value);
        const bool tail = value && (w.tile0 + t + 1) * kTile > shared_to;
        if (!value || (!F8 && !tail)) continue;
        for (int part = 0; part < C::Parts; ++part) {
          const int at = e0 + e * C::Parts + part, slot = at % C::Slots;
          if (kTwoWiden && (slot & 1) != group_bar - 2) continue;
          const int pos0 = (w.tile0 + t) * kTile;
          wait(raw_full + slot, f_phase >> slot & 1u);
          f_phase ^= 1u << slot;
          uint8_t* tile = ring + slot * C::Slot;
          if constexpr (F8) {
            // 64 rows at a time: the first ones go below the copied numbers, the others over them, once all are in registers
            constexpr int Chunks = C::Cols / 16, Each = Chunks / 2;  // 16 numbers; of a row, of a thread
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
            uint4 v[Each];
#pragma unroll
            for (int i = 0; i < Each; ++i)
              v[i] = *reinterpret_cast<const uint4*>(tile + C::Slot / 2 + C::at8(half * 64 + (i * 128 + tid) / Chunks, (i * 128 + tid) % Chunks));
            if (half == 1 && !tc::bar_and(!dead, group_bar, 128)) {
              dead = true;
              break;
            }
#pragma unroll
            for (int i = 0; i < Each; ++i) {
              const int c = i * 128 + tid, row = half * 64 + c / Chunks, ch = c % Chunks * 2;
              uint32_t o[8];
              const uint32_t in[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                o[2 * j] = widen2((uint16_t)in[j]);
                o[2 * j + 1] = widen2((uint16_t)(in[j] >> 16));
              }
              if (tail && pos0 + row >= shared_to) {
                const bool past = pos0 + row >= w.len;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  if (past) {
                    o[j] = 0;
                    continue;
                  }
                  bool odd = false;
                  if ((o[j] & 0x7C00u) == 0x7C00u) { o[j] &= 0xFFFF0000u; odd = true; }
                  if ((o[j] >> 16 & 0x7C00u) == 0x7C00u) { o[j] &= 0xFFFFu; odd = true; }
                  if (odd) {
                    odd_of[k % kOdd] = k;
                    __threadfence_block();
                  }
                }
              }
              // lanes of odd blocks store their second half first: eight lanes then reach all banks
              const bool odd_block = ch >> 3 & 1;
              const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
              *reinterpret_cast<uint4*>(tile + C::at(row, odd_block ? ch + 1 : ch)) = odd_block ? hi : lo;
              *reinterpret_cast<uint4*>(tile + C::at(row, odd_block ? ch : ch + 1)) = odd_block ? lo : hi;
            }
            }
            if (dead) break;
          } else {
            if (dead) break;
            constexpr int Chunks = C::Cols / 8;
            const int from = max(shared_to - pos0, 0), to = min(w.len - pos0, kTile);  // rows that some do not see; their end
            for (int c = max(to, 0) * Chunks + tid; c < kTile * Chunks; c += 128) *reinterpret_cast<uint4*>(tile + C::at(c / Chunks, c % Chunks)) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
            for (int c = from * Chunks + tid; c < to * Chunks; c += 128) {
              uint4* at = reinterpret_cast<uint4*>(tile + C::at(c / Chunks, c % Chunks));
              const uint4 v = *at;
              // an exponent of ones carries into bit 15
              const auto carry = [](uint32_t x) { return (x & 0x7F807F80u) + 0x00800080u; };
              if (((carry(v.x) | carry(v.y) | carry(v.z) | carry(v.w)) & 0x80008000u) == 0) continue;
              const auto clean = [&](uint32_t x) {
                if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
                if ((x >> 16 & 0x7F80u) == 0x7F80u) x &= 0xFFFFu;
                return x;
              };
              *at = make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
              odd_of[k % kOdd] = k;
              __threadfence_block();
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(ready + slot);
        }
      }
      e0 += 2 * n * C::Parts;
    }
  } else if (warp < kSoftmaxWarp) {
    regs_down<kIssueRegs>();
    if (warp == kCopyWarp) {
      // ---- the warp that plans and copies
      const int cta = (int)blockIdx.x;
      const int box = 1 << p.page_shift;  // rows of one copy: a page's
      int at = 0, end = 0, item = cta;
      if (plan.split && cta < plan.ctas) {
        at = (int)((int64_t)cta * plan.total / plan.ctas);
        end = (int)((int64_t)(cta + 1) * plan.total / plan.ctas);
      }
      int e0 = 0, copied = 0;
      uint32_t f_phase = 0, r_phase = 0, is_raw = 0;  // per slot: copies into it, those for the widening warps; what the last one was
      // The next stretch is planned and announced before the tiles of this one are copied, so that its queries are brought meanwhile.
      Work w{}, following;
      for (int k = 0;; ++k) {
        if (plan.split) {
          following = prompt::next_stretch<C::Rows>(p, plan, at, end);
        } else {
          if (k > 0) {
            if (lane == 0) item = (int)gridDim.x + (p.counter ? atomicAdd(p.counter, 1) : item);
            item = __shfl_sync(0xFFFFFFFFu, item, 0);
          }
          following = prompt::whole_item<C::Rows>(p, plan, item);
        }
        const int told_at = k % kWorks;
        if (k >= kWorks && !wait(w_empty + told_at, (uint32_t)(k / kWorks & 1) ^ 1u)) break;
        if (lane == 0) {
          works[told_at] = following;
          tc::mbar_arrive(w_full + told_at);
        }
        __syncwarp();
        if (k == 0) {
          w = following;
          if (!w.more) break;
          continue;
        }
        const int n = w.tiles;
        TreeSegment g;
        g.seq = TreeSeq{w.start, w.len - w.prefix, w.prefix};
        g.b = w.b;
        g.tile0 = w.tile0;
        TreePages<kTile> pages(p, g, lane);
        const int shared_to = w.shared0, to_values = p.hkv << p.page_shift;
        // lane i knows where box i of a tile's keys lies; none past the end
        const auto rows_of = [&](int t) {
          int page = pages.at(t);
          page = page < 0 ? 0 : page >= p.pages ? (int)p.pages - 1 : page;
          return (page * 2 * p.hkv + w.head) << p.page_shift;
        };
        int now = 0, before = 0;  // of the last two tiles of keys
#pragma unroll 1
        for (int e = 0; e < 2 * n && !dead; ++e) {
          bool value;
          const int t = tile_at<C::Streams>(e, n, &value);
          if (!value) {
            before = now;
            now = rows_of(t);
          }
          const int y = value ? (C::Streams == 1 && t + 1 < n ? before : now) + to_values : now;
          const int left = w.len - (w.tile0 + t) * kTile, boxes = min(kTile, left + box - 1) >> p.page_shift;
          const bool through = value && (F8 || (w.tile0 + t + 1) * kTile > shared_to);  // the widening warps
#pragma unroll 1
          for (int part = 0; part < C::Parts; ++part) {
            const int i = e0 + e * C::Parts + part, slot = i % C::Slots, use = i / C::Slots;
            if (use > 0 && !wait(empty + slot, (uint32_t)(use & 1) ^ 1u)) break;
            const uint32_t bar = tc::smem_u32((through ? raw_full : full) + slot),
                           to = tc::smem_u32(ring) + slot * C::Slot + (F8 && value ? C::Slot / 2 : 0);
            (through ? r_phase : f_phase) ^= 1u << slot;
            is_raw = (is_raw & ~(1u << slot)) | (uint32_t)through << slot;
            expect_bytes(bar, (uint32_t)(boxes * box * C::Cols * (F8 ? 1 : 2)));
            copied = i + 1;
#pragma unroll 1
            for (int j = 0; j < boxes; ++j) {
              const int row = __shfl_sync(0xFFFFFFFFu, y, j);
              if constexpr (F8) tma_load_2d(to + j * box * C::Cols, &map, bar, part * C::Cols, row);
              else tma_load_4d(to + (j * box >> 3) * C::Group, &map, bar, part * C::Blocks, row >> 3);
            }
          }
        }
        e0 += 2 * n * C::Parts;
        w = following;
        if (dead || !w.more) break;
      }
      // no copy may land in a block that has left
      for (int i = max(0, copied - C::Slots); i < copied; ++i) {
        const int slot = i % C::Slots;
        const bool was_raw = is_raw >> slot & 1u;
        tc::mbar_wait((was_raw ? raw_full : full) + slot, ((was_raw ? r_phase : f_phase) >> slot & 1u) ^ 1u, kDrainNs);
      }
    } else if (warp == kMmaWarp) {
      // ---- the warp that issues the products.  All it does between two products is on the way of both streams, at 5 to 10 cycles an
      // instruction: so what it needs is carried along, not computed, and there is one copy of the code.
      bool issued = false;
      Work w;
      constexpr uint32_t kNoType = ~((1u << 7) | (1u << 10));  // both operands fp16, or e4m3
      constexpr uint32_t id_s = tc::idesc_bf16_f32(128, kTile) & (F8 ? kNoType : ~0u),
                         id_o = (tc::idesc_bf16_f32(128, C::Cols) & (F8 ? kNoType : ~0u)) | kBMnMajor;
      constexpr uint32_t kSlot = C::Slot >> 4;
      constexpr uint32_t kSwizzle = F8 && C::Cols == 64 ? 4 : 2, kRows8 = F8 ? 8 * C::Cols : 1024;
      const uint64_t q_desc = tc::desc_kmajor(tc::smem_u32(sq), kRows8, kSwizzle), k_desc = tc::desc_kmajor(tc::smem_u32(ring), F8 ? kRows8 : C::Group, kSwizzle),
                     v_desc = desc_values(tc::smem_u32(ring), 1024, C::Group);
      uint32_t p_phase = 0, f_phase = 0, r_phase = 0;  // per S; per slot, of what comes directly, and of the rest
      int e0 = 0;                                      // the slot of the stretch's first copy
      const auto take = [&](int slot, bool through) {  // waits for a slot's tile
        if (through) {
          if (!wait(raw_full + slot, r_phase >> slot & 1u) || !wait(ready + slot, r_phase >> slot & 1u)) return false;
          r_phase ^= 1u << slot;
          return true;
        }
        if (!wait(full + slot, f_phase >> slot & 1u)) return false;
        f_phase ^= 1u << slot;
        return true;
      };
      for (int k = 0; told(k, w); ++k) {
        // Units: a tile of a stream, streams in turn; of one stream every tile.  Unit u has S number u % 2, and its outputs are followed
        // by the scores of unit u + 2.
        const int n = uniform(w.tiles), first_tail = uniform(w.shared0 / kTile - w.tile0);
        const int n0 = uniform(w.n0), n1 = C::Streams == 2 ? uniform(w.n1) : 0;
        const int qb = k % C::QBuffers;
        if (!wait(q_full + qb, (uint32_t)(k / C::QBuffers & 1))) break;
        const uint64_t q_at = q_desc + (uint32_t)(qb * (C::Streams * C::QTile >> 4));
        int t = C::Streams == 2 ? -1 : -2;
        const auto unit = [&](int b) {
          const int mine = C::Streams == 1 ? n : b ? n1 : n0, next = t + (C::Streams == 2 ? 1 : 2);
          if (t >= 0 && t < mine) {
            const int slot = (e0 + place_of<C::Streams>(t, true, n) * C::Parts) % C::Slots;
            if (C::Streams == 1 || b == 0 || n0 <= t)
#pragma unroll
              for (int part = 0; part < C::Parts; ++part)
                if (!take(slot + part, F8 || t >= first_tail)) return;
            if (!wait(p_ready + b, p_phase >> b & 1u)) return;
            p_phase ^= 1u << b;
            tc::fence_after_sync();
            const uint64_t d = v_desc + slot * kSlot;
            const uint32_t o = tmem + (C::Streams == 1 ? C::O(0) : C::O(0) + b * D), a = tmem + C::S(0) + b * 128;
#pragma unroll
            for (int part = 0; part < C::Parts; ++part) {
#pragma unroll
              for (int x = 0; x < kTile / 16; ++x)
                mma_ts(o + part * C::Cols, a + 8 * x, d + part * kSlot + ((x * 2 * C::Group) >> 4), id_o, x > 0 || t > 0);
              if (C::Streams == 1 || b == 1 || n1 <= t) mma_done(empty + slot + part);
            }
            if (C::Streams == 1) mma_done(o_done);
            if (next - (C::Streams == 2 ? 0 : 1) == mine) mma_done(o_full + (C::Streams == 1 ? 0 : b));
          }
          if (next < mine) {
            const int slot = (e0 + place_of<C::Streams>(next, false, n) * C::Parts) % C::Slots;
            if (C::Streams == 1 || b == 0 || n0 <= next) {
#pragma unroll
              for (int part = 0; part < C::Parts; ++part)
                if (!take(slot + part, false)) return;
              tc::fence_after_sync();
            }
            const uint64_t a = q_at + (C::Streams == 1 ? 0 : b * (C::QTile >> 4)), d = k_desc + slot * kSlot;
            const uint32_t to = tmem + C::S(0) + b * 128;
#pragma unroll
            for (int part = 0; part < C::Parts; ++part) {
              if constexpr (F8) {  // [high, low part][block of 128 columns][row]
#pragma unroll
                for (int low = 0; low < 2; ++low)
#pragma unroll
                  for (int x = 0; x < C::Cols / 32; ++x)
                    mma_ss_f8(to, a + ((low * C::QTile / 2 + part * 128 * C::Cols + x * 32) >> 4), d + part * kSlot + (x * 32 >> 4), id_s | (uint32_t)low << 7,
                              part > 0 || low > 0 || x > 0);
              } else
#pragma unroll
              for (int x = 0; x < C::Cols / 16; ++x)
                mma_ss(to, a + ((part * C::Blocks * 128 * 128 + (x >> 2) * (128 * 128) + (x & 3) * 32) >> 4), d + part * kSlot + (((x >> 2) * 1024 + (x & 3) * 32) >> 4),
                       id_s, part > 0 || x > 0);
              if (C::Parts > 1) mma_done(empty + slot + part);
            }
            mma_done(s_full + b);
            if (C::Parts == 1 && (b == 1 || n1 <= next)) mma_done(empty + slot);
            issued = true;
            if (next + 1 == n && (C::Streams == 1 || b == 1 || n1 <= next)) mma_done(q_empty + qb);
          }
        };
        // One copy of it, or two: with heads of 128 in bf16 the products are what bounds, and fewer instructions between them weigh more
        // than their number (8192 tokens 372 us and 397, e4m3 600 and 565).
        constexpr bool kTwice = D == 128 && !F8;
        if (kTwice) {
#pragma unroll 1
          for (; t < n && !dead; ++t) {
            unit(0);
            if (!dead) unit(1);
          }
        } else {
#pragma unroll 1
          for (int b = 0; t < n && !dead; b ^= 1) {
            unit(b);
            t += C::Streams == 2 ? b : 1;
          }
        }
        if (dead) break;
        e0 = (e0 + 2 * n * C::Parts) % C::Slots;
      }
      // tensor memory is given back once every product issued has completed, also where a wait gave up
      if (issued) {
        mma_done(drained);
        tc::mbar_wait(drained, 0, kDrainNs);
      }
    } else {
      // ---- the warps that bring the queries
      const int tid = threadIdx.x - kQueryWarp * 32;
      Work w;
      for (int k = 0; told(k, w); ++k) {
        const float ks = p.scales ? __ldg(p.scales + w.head) : 1.f;
        const uint32_t flip = p.scale_log2 * ks < 0.f ? 0x80008000u : 0u;  // a negative scale goes into the queries' signs
        uint8_t* to = sq + k % C::QBuffers * (C::Streams * C::QTile);
        const auto room = [&] { return k < C::QBuffers || wait(q_empty + k % C::QBuffers, (uint32_t)(k / C::QBuffers & 1) ^ 1u); };
        if constexpr (!F8) {
        constexpr int LPR = D / 8, kRows = 64 / LPR;  // lanes of a row, rows at a time
        const int ch = tid % LPR, r0 = tid / LPR;
        // (token, head of the group) of row r0 + kRows i, without a division each
        int d = prompt::draft(p, w.g0 + r0), hh = w.g0 + r0 - d * p.group;
        const uint16_t* src = p.q + (int64_t)(w.start + w.first + d) * p.q_stride + (int64_t)(w.head * p.group + hh) * D + 8 * ch;
        const int dstep = prompt::draft(p, kRows), hstep = kRows - dstep * p.group;
        const int64_t step = dstep * p.q_stride + hstep * D, wrap = p.q_stride - (int64_t)p.group * D;
        const auto next = [&] {
          hh += hstep;
          src += step;
          if (hh >= p.group) {
            hh -= p.group;
            src += wrap;
          }
        };
          const auto place = [&](int r) { return (r >> 7) * C::QTile + (ch >> 3) * (128 * 128) + (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4); };
          if (!room()) break;
#pragma unroll 4
          for (int r = r0; r < w.rows; r += kRows) {
            cp_async16(tc::smem_u32(to) + place(r), src);
            next();
          }
          cp_async_wait();
          if (flip)
            for (int r = r0; r < w.rows; r += kRows) {
              uint4* at = reinterpret_cast<uint4*>(to + place(r));
              uint4 v = *at;
              *at = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
            }
        } else {
          // A thread per row, 64 numbers at a time: with lanes side by side along a row, its largest number took most of the time (8 x
          // 2000 tokens, 64/8 heads of 64: 542 us for 447).  Larger heads: the scales of all rows first, before there is room.
          const auto row_of = [&](int r) {
            const int dr = prompt::draft(p, w.g0 + r), hr = w.g0 + r - dr * p.group;
            return p.q + (int64_t)(w.start + w.first + dr) * p.q_stride + (int64_t)(w.head * p.group + hr) * D;
          };
          const auto load = [&](const uint16_t* row, uint4 (&u)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = *reinterpret_cast<const uint4*>(row + 8 * i);
          };
          const auto largest = [&](const uint4 (&u)[8], uint32_t big) {  // positive bf16 patterns compare like integers, two at a time
#pragma unroll
            for (int i = 0; i < 8; ++i)
              big = __vmaxu2(big, __vmaxu2(__vmaxu2(u[i].x & 0x7FFF7FFFu, u[i].y & 0x7FFF7FFFu), __vmaxu2(u[i].z & 0x7FFF7FFFu, u[i].w & 0x7FFF7FFFu)));
            return big;
          };
          const auto scale_up = [&](uint32_t big) { return min(134 - (int)(max(big & 0xFFFFu, big >> 16) >> 7), 127); };  // largest to 2^7 .. 2^8
          float* ups = row_up + (k & 3) * C::Rows;
          if (D > 64)
#pragma unroll 1
            for (int r = tid; r < w.rows; r += 64) {
              const uint16_t* row = row_of(r);
              uint32_t big = 0;
#pragma unroll 1
              for (int col = 0; col < D; col += 64) {
                uint4 u[8];
                load(row + col, u);
                big = largest(u, big);
              }
              ups[r] = (float)scale_up(big);
            }
          if (!room()) break;
#pragma unroll 1
          for (int r = tid; r < w.rows; r += 64) {
            const uint16_t* row = row_of(r);
#pragma unroll 1
            for (int col = 0; col < D; col += 64) {
              uint4 u[8];
              load(row + col, u);
              if (D == 64) ups[r] = (float)scale_up(largest(u, 0));
              const float f = __uint_as_float((uint32_t)(127 + (int)ups[r]) << 23);
              uint8_t* at = to + (r >> 7) * C::QTile + col / C::Cols * (128 * C::Cols);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t hi[4], lo[4];
                split8(u[2 * i], flip, f, hi[0], hi[1], lo[0], lo[1]);
                split8(u[2 * i + 1], flip, f, hi[2], hi[3], lo[2], lo[3]);
                const int place = C::at8(r & 127, col % C::Cols / 16 + i);
                *reinterpret_cast<uint4*>(at + place) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(at + C::QTile / 2 + place) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
              }
            }
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(q_full + k % C::QBuffers);
      }
    }
  } else {
    // ---- softmax: stream s, one thread per row; warp i of a group reaches tensor memory lanes 32 i ..
    regs_up<kSoftmaxRegs>();
    const int s = (warp - kSoftmaxWarp) >> 2, r = threadIdx.x - kSoftmaxWarp * 32;  // row of the block
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int cta = (int)blockIdx.x;
    Work w;
    uint32_t s_phase = 0, o_phase = 0;  // s_phase: per S
    int products = 0;                   // one stream: tiles of the stretches before
    int4 shared_item = make_int4(0, 0, 0, 0);  // the item that starts here and ends in a later block
    if (s < C::Streams)
      for (int k = 0; told(k, w); ++k) {
        const bool valid = r < w.rows;
        const int n = s ? w.n1 : w.n0;
        const int d = valid ? prompt::draft(p, w.g0 + r) : 0, hh = w.g0 + r - d * p.group;
        const int seen = valid ? w.prefix + w.first + d + 1 : 0;
        const int masked_from = s ? w.shared1 : w.shared0;  // keys that every row of the stream sees
        float c = score_factor(fabsf(p.scale_log2 * (p.scales ? __ldg(p.scales + w.head) : 1.f)));
        const uint32_t t_o = tmem + C::O(s) + lanes;
        float m = -INFINITY, l = 0.f;  // the maximum in use, the sum
        for (int i = 0; i < n; ++i) {
          const int buf = C::Streams == 1 ? i & 1 : s;
          const uint32_t t_s = tmem + C::S(buf) + lanes;
          if (!wait(s_full + buf, s_phase >> buf & 1u)) break;
          s_phase ^= 1u << buf;
          tc::fence_after_sync();
          if (F8 && i == 0) {  // 2^-up of the row's queries
            const int up = (int)row_up[(k & 3) * C::Rows + r], half = up / 2;
            c *= __uint_as_float((uint32_t)(127 - half) << 23);
            c *= __uint_as_float((uint32_t)(127 - (up - half)) << 23);
            c = c != c ? c : score_factor(fminf(c, 3.402823466e38f));
          }
          const int pos0 = (w.tile0 + i) * kTile;
          // Passes over the scores are loops over 32 or 64 columns: tensor memory is read again for less than what a tile's 128 held in
          // registers cost in code, since the warps of all kinds share the instruction caches.
          if (pos0 + kTile > masked_from) {  // scores that the row does not see become minus infinity, in place
            const int upto = seen - pos0;
#pragma unroll 1
            for (int j = 0; j < kTile; j += 32) {
              const int bits = upto - j;
              if (__all_sync(0xFFFFFFFFu, bits >= 32)) continue;
              const uint32_t keep = bits >= 32 ? 0xFFFFFFFFu : bits > 0 ? (1u << bits) - 1 : 0u;
              uint32_t y[32];
              tc::tmem_ld_32x32b_x32(t_s + j, y);
              tc::tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 32; ++q) y[q] = keep >> q & 1 ? y[q] : 0xFF800000u;
              tmem_st_x32(t_s + j, y);
            }
            tmem_st_wait();
          }
          float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < kTile; j += 64) {
            uint32_t y[2][32];
            tc::tmem_ld_32x32b_x32(t_s + j, y[0]);
            tc::tmem_ld_32x32b_x32(t_s + j + 32, y[1]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 64; q += 8)
#pragma unroll
              for (int z = 0; z < 4; ++z)
                a[z] = fmaxf(fmaxf(a[z], __uint_as_float(y[q >> 5][(q & 31) + 2 * z])), __uint_as_float(y[q >> 5][(q & 31) + 2 * z + 1]));
          }
          const float mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * c;
          const bool move = mx > m + kMove || (m == -INFINITY && mx > -INFINITY);
          if (__any_sync(0xFFFFFFFFu, move)) {
            const float to = move ? mx : m, f = m == to ? 1.f : ex2(m - to);
            l *= f;
            m = to;
            if (i > 0) {
              if (C::Streams == 1) {  // the product of the tile before it
                if (!wait(o_done, (uint32_t)(products + i - 1) & 1u)) break;
                tc::fence_after_sync();
              }
#pragma unroll 1
              for (int col = 0; col < D; col += 16) {
                uint32_t y[16];
                tmem_ld_x16(t_o + col, y);
                tc::tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 16; ++q) y[q] = __float_as_uint(__uint_as_float(y[q]) * f);
                tmem_st_x16(t_o + col, y);
              }
            }
          }
          // ---- weights, over the scores, in the type of the values they are multiplied with
          const float ms = (m == -INFINITY ? 0.f : -m) + C::template Lift<F8>;
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          constexpr int kHalves = F8 ? 1 : 2;  // e4m3: less code for more warps (chunk 557 us with 64 columns at a time, 503)
#pragma unroll 1
          for (int j = 0; j < kTile; j += 32 * kHalves) {
            uint32_t x[kHalves][32];
#pragma unroll
            for (int h = 0; h < kHalves; ++h) tc::tmem_ld_32x32b_x32(t_s + j + 32 * h, x[h]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              uint32_t e[16];
#pragma unroll
              for (int q = 0; q < 32; q += 2) {
                float2 y = __ffma2_rn(make_float2(__uint_as_float(x[h][q]), __uint_as_float(x[h][q + 1])), make_float2(c, c), make_float2(ms, ms));
                y.x = ex2(y.x);
                y.y = ex2(y.y);
                sum[q >> 1 & 1] = __fadd2_rn(sum[q >> 1 & 1], y);
                e[q >> 1] = F8 ? pack_f16x2(y.x, y.y) : pack_bf16x2(y.x, y.y);
              }
              tmem_st_x16(t_s + (j >> 1) + 16 * h, e);
            }
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(p_ready + buf);
        }
        if (dead) break;
        products += n;
        // ---- the stretch's end
        if (n > 0) {
          if (!wait(o_full + s, o_phase)) break;
          o_phase ^= 1u;
          tc::fence_after_sync();
        }
        const bool whole = w.tile0 == 0 && w.tiles == w.last + 1;
        const bool odd = odd_of[k % kOdd] == k;
        const int odd_from = max(w.shared0, w.tile0 * kTile), odd_to = min(seen, (w.tile0 + w.tiles) * kTile);
        const int64_t token = w.start + w.first + d;
        const int head = w.head * p.group + hh;
        const auto fetch = [&](int col, float (&v)[32]) {  // 32 columns of the row
          uint32_t y[32];
#pragma unroll
          for (int q = 0; q < 32; ++q) y[q] = 0;
          if (n > 0) {
            tc::tmem_ld_32x32b_x32(t_o + col, y);
            tc::tmem_ld_wait();
          }
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = __uint_as_float(y[q]);
        };
        if (whole) {
          const float vs = p.scales ? __ldg(p.scales + p.hkv + w.head) : 1.f, f = l == 0.f ? 0.f : vs / l;
          // 32 columns at a time through shared memory, so that 64 bytes of a row are stored by four lanes together (a row per lane:
          // four times as many accesses, the end of an item took 4000 cycles)
          uint8_t* stage = stages + (warp - kSoftmaxWarp) * C::Stage;
          // rows (lane / 4) + 8 i of the warp's 32
          uint16_t* out[4];
          const int q0 = (warp & 3) * 32 + s * 128 + (lane >> 2);
          int dq = prompt::draft(p, w.g0 + q0), hq = w.g0 + q0 - dq * p.group;
          out[0] = p.out + (int64_t)(w.start + w.first + dq) * p.out_stride + (int64_t)(w.head * p.group + hq) * D + 8 * (lane & 3);
          const int dstep = prompt::draft(p, 8), hstep = 8 - dstep * p.group;
          const int64_t step = dstep * p.out_stride + hstep * D, wrap = p.out_stride - (int64_t)p.group * D;
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            hq += hstep;
            out[i] = out[i - 1] + step;
            if (hq >= p.group) {
              hq -= p.group;
              out[i] += wrap;
            }
          }
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            float v[32];
            fetch(col, v);
            if (__any_sync(0xFFFFFFFFu, l == 0.f))  // zeros, also over values that are not finite
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] = l == 0.f ? 0.f : v[q];
            uint32_t e[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float2 y = __fmul2_rn(make_float2(v[2 * q], v[2 * q + 1]), make_float2(f, f));
              e[q] = pack_bf16x2(y.x, y.y);
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4)) = make_uint4(e[4 * q], e[4 * q + 1], e[4 * q + 2], e[4 * q + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int q = 8 * i + (lane >> 2);
              if (q0 + 8 * i < w.rows) *reinterpret_cast<uint4*>(out[i] + col) = *reinterpret_cast<const uint4*>(stage + q * 64 + (((lane & 3) ^ (q >> 1 & 3)) << 4));
            }
          }
          if (odd) {
            __syncwarp();  // the row was stored by other lanes
            if (valid && l != 0.f) add_odd<D, F8>(p, w.b, w.head, odd_from, odd_to, f, p.out + token * p.out_stride + (int64_t)head * D, nullptr, 0);
          }
          if (valid && p.lse) p.lse[token * p.hq + head] = l == 0.f ? -INFINITY : kLn2 * (m + (log2f(l) - C::template Lift<F8>));
        } else {  // a part, for the joining kernel
          float* part = p.part + (int64_t)tree_slot(cta, w.tile0 == 0) * tree_part_floats(C::Rows, D);
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            float v[32];
            fetch(col, v);
            if (valid)
#pragma unroll
              for (int q = 0; q < 32; q += 4)
                *reinterpret_cast<float4*>(part + ((int64_t)(col + q) / 4 * C::Rows + r) * 4) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
          }
          if (odd && valid) add_odd<D, F8>(p, w.b, w.head, odd_from, odd_to, 1.f, nullptr, part + r * 4, C::Rows * 4);
          if (valid) {
            part[(int64_t)C::Rows * D + r] = m;
            part[(int64_t)C::Rows * D + C::Rows + r] = l;
          }
          if (w.tile0 == 0 && r == 0)
            shared_item = make_int4(w.start + w.first, w.head, w.g0, tree_parts_shared(w.until - cta + 1) << 24 | w.rows << 12 | w.until);
        }
        tc::fence_before_sync();  // the accumulator is read before the next stretch's weights are announced
      }
    if (r == 0) p.items[cta] = shared_item;
  }
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && flags[0]) atomicCAS(&g_prompt_error, 0, 4);
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// The counter of items starts at zero whatever the workspace holds: a program may have lent it to other calls.
__global__ void clear_counter(int* counter) {
  pdl_enter();
  *counter = 0;
}

template <int D, bool F8>
cudaError_t launch_d(const CUtensorMap& map, TreeParams p, int ctas, cudaStream_t st) {
  auto kern = prompt_kernel<D, F8>;
  static PerDevice<cudaError_t> attr_of;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const cudaError_t e = attr_of.get(dev, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::Smem);
  }, cudaErrorInvalidDevice);
  if (e != cudaSuccess) return e;
  // Where there is at most an item for each block and none is longer than its parts and their joining would cost, none is split and
  // nobody asks for a second one: neither a counter nor a joining kernel, then (100 tokens: 10.8 us, 12.3 with the latter).
  const int64_t items = (int64_t)p.hkv * ((int64_t)p.n * p.group / Cfg<D>::Rows + p.batch);
  const int64_t most = (((int64_t)p.width << p.page_shift) + kTile - 1) / kTile + prompt::kExtra;
  const bool alone = items <= ctas && most <= prompt::kJoin;
  if (alone) p.counter = nullptr;
  cudaError_t e2 = alone ? cudaSuccess : launch_pdl(clear_counter, dim3(1), dim3(1), 0, st, p.counter);
  if (e2 == cudaSuccess) e2 = launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), Cfg<D>::Smem, st, map, p);
  if (e2 != cudaSuccess || alone) return e2;
  return launch_tree_join(p, D, Cfg<D>::Rows, Cfg<D>::template Lift<F8>, ctas, st);
}

int prompt_ctas() { return device_sm_count() < kTreeMaxCtas ? device_sm_count() : kTreeMaxCtas; }

constexpr size_t kItemBytes = kTreeMaxCtas * sizeof(int4);

}  // namespace

size_t prompt_workspace_bytes(const trellis_cache_t& c, int q_heads) {
  (void)q_heads;  // parts belong to thread blocks, whatever the heads
  const int rows = c.head_dim == 256 ? Cfg<256>::Rows : Cfg<128>::Rows;
  return kItemBytes + 16 + (size_t)tree_part_floats(rows, c.head_dim) * 4 * 2 * prompt_ctas();
}

int read_prompt_error(int reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_prompt_error, sizeof(int)) != cudaSuccess) return -1;
  if (reset && v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

cudaError_t launch_prompt_attention(const uint16_t* q, int64_t q_stride, const trellis_cache_t& c, int layer,
                                    const trellis_drafts_t& d, int q_heads, float scale, uint16_t* out,
                                    int64_t out_stride, float* lse, void* workspace, cudaStream_t st) {
  TreeParams p{};
  p.q = q; p.out = out; p.lse = lse;
  p.table = d.table; p.prefix = d.prefix; p.q_start = d.q_start;
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
  p.counter = reinterpret_cast<int*>(static_cast<char*>(workspace) + kItemBytes);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kItemBytes + 16);

  const auto fn = tensor_map_encoder();
  if (!fn) return cudaErrorNotSupported;
  const bool f8 = c.dtype == TRELLIS_E4M3;
  const int row_bytes = c.head_dim * (int)cache_elem_bytes(c), cols = c.head_dim < 128 ? c.head_dim : 128;
  uint8_t* pool = static_cast<uint8_t*>(c.pool) + (int64_t)layer * c.pages * cache_page_bytes(c);
  CUtensorMap map;
  const cuuint64_t rows = (cuuint64_t)(c.pages * 2 * c.heads * c.page_size);
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult made;
  if (f8) {  // 128 bytes (or 64) of each row, swizzled
    const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, rows}, strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)cols, (cuuint32_t)c.page_size};
    made = fn(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, pool, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {  // (64 numbers, 8 rows, blocks of 64 of a row, groups of 8 rows): what a slot holds, 8 rows of a block swizzled together
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)(c.head_dim / 64), rows / 8},
                     strides[3] = {(cuuint64_t)row_bytes, 128, (cuuint64_t)row_bytes * 8};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)(cols / 64), (cuuint32_t)(c.page_size / 8)};
    made = fn(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (made != CUDA_SUCCESS) return cudaErrorInvalidValue;
  p.pool = pool;
  const int ctas = prompt_ctas();
  if (f8)
    return c.head_dim == 64 ? launch_d<64, true>(map, p, ctas, st) : c.head_dim == 128 ? launch_d<128, true>(map, p, ctas, st)
                                                                                     : launch_d<256, true>(map, p, ctas, st);
  return c.head_dim == 64 ? launch_d<64, false>(map, p, ctas, st) : c.head_dim == 128 ? launch_d<128, false>(map, p, ctas, st)
                                                                                    : launch_d<256, false>(map, p, ctas, st);
}

}  // namespace trellis

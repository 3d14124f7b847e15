// tree_tc.cuh -- what the tree attention kernels on the 5th-generation tensor cores share (tree_attention_tc.cu,
// tree_attention_tc1.cu): the forms of the tensor-memory instructions that only they use, and the order of their copies.
//
// The softmax in one pass with a running maximum is that of Milakov and Gimelshein, "Online normalizer calculation for softmax"
// (2018).  Weights that lie in tensor memory over their scores, and a maximum that is moved only when it has grown far, are
// published too, for attention on this hardware.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "tc_ptx.cuh"
#include "tree_sched.cuh"

namespace trellis {
namespace tree {

constexpr uint64_t kDrainNs = 2000000000ull;  // for copies and products in flight when a block leaves
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kMove = 8.f;                  // log2 of the growth that moves a row's maximum

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void named_sync(int id, int count) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory"); }

// The products are issued by a warp as a whole, one thread of which is elected in the instruction's own block: operands that are
// the warp's then lie in uniform registers.  From a branch of one thread an MMA took no less than 50 cycles to issue, whatever
// its size; so it takes 11 (A in tensor memory, 128 x 16 x 32 bytes), and 34 at N = 64, which is the MMA itself.
// Converged warps only.  D[tmem] (+)= A[smem desc or tmem] * B[smem desc], fp32 accumulate.
#define TRELLIS_TREE_MMA(NAME, KIND, A, ASM_A, REG_A)                                                                     \
  __device__ __forceinline__ void NAME(uint32_t d, A a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {           \
    asm volatile(                                                                                                         \
        "{\n\t.reg .pred p, q;\n\t"                                                                                      \
        "elect.sync _|q, 0xFFFFFFFF;\n\t"                                                                                \
        "setp.ne.b32 p, %4, 0;\n\t"                                                                                      \
        "@q tcgen05.mma.cta_group::1.kind::" KIND " [%0], " ASM_A ", %2, %3, p;\n\t}"                                     \
        ::"r"(d), REG_A(a), "l"(bdesc), "r"(idesc), "r"(accumulate)                                                       \
        : "memory");                                                                                                      \
  }
TRELLIS_TREE_MMA(mma_ss, "f16", uint64_t, "%1", "l")           // 16-bit inputs, both bf16 or both fp16 as the descriptor says
TRELLIS_TREE_MMA(mma_ts, "f16", uint32_t, "[%1]", "r")
TRELLIS_TREE_MMA(mma_ts_f8, "f8f6f4", uint32_t, "[%1]", "r")  // 8-bit inputs, each of the kind that the descriptor says
#undef TRELLIS_TREE_MMA
// The mbarrier receives one arrival once the products issued so far have completed.
__device__ __forceinline__ void mma_done(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar))
      : "memory");
}
// The factor of a row's scores, from its absolute value: a scale of 0 becomes the smallest number instead, times which every
// score that is finite vanishes in a sum, and minus infinity stays what it is.
__device__ __forceinline__ float score_factor(float c) { return c == 0.f ? __uint_as_float(1u) : c; }

// A number that is the same in all lanes, to the compiler too.
template <typename T>
__device__ __forceinline__ T uniform(T v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// This warp's 32 lanes x 16 (32) consecutive columns from registers.
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Operand whose rows are the reduction index (values: [key][head dim]) in the 128-byte swizzle: 64 numbers of a row
// are contiguous; `lbo` bytes from one such block of columns to the next, 1024 bytes from 8 rows to the next 8.
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kBMnMajor = 1u << 16;  // instruction descriptor: B's rows are the reduction index


// The order in which a segment's 2n entries are copied, which is that of their use: entry e is tile at(e)'s keys or
// values.  split_keys: the keys of two tiles come before the first one's values.
struct Order {
  int n;
  bool split_keys;
  __device__ __forceinline__ int at(int e, bool* is_value) const {
    if (!split_keys) {
      *is_value = e & 1;
      return e >> 1;
    }
    if (e < 2 && e < n) { *is_value = false; return e; }
    if (e == 2 * n - 1) { *is_value = true; return n - 1; }
    *is_value = !(e & 1);
    return e & 1 ? (e + 1) / 2 : (e - 2) / 2;
  }
};


}  // namespace tree
}  // namespace trellis

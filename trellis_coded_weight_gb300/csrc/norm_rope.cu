// norm_rope.cu -- norms of queries and keys for each head, the rotation by position and the write of keys and
// values into the pages of a cache, in one launch (trellis_qk_norm_rope_append).
//
// Per token and head, with x the head's D numbers, w its weights and (c, s) the token's row of the rotation table:
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset);   (a, b) -> (a c - b s, b c + a s) on the rotated pairs
// Everything in fp32, one rounding at the end (bf16, or e4m3 of y / scale).
//
// A head lives in D/8 neighbouring lanes, 8 numbers (one 16-byte load) each: the sum of squares is a shuffle over
// those lanes, a pair that spans half a rotation is one shuffle away, an interleaved pair is in one lane.  Nothing is
// staged.  A thread block serves one token (and a share of its heads); its lanes keep their 8 cosines and sines,
// which every head of the token uses.  Bound: launch latency for a few tokens, HBM beyond.
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"

namespace trellis {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // rounds of heads whose loads are in flight

struct Params {
  NormRopeTokens t;
  const uint16_t *wq, *wk;
  const float* rope;
  const float* scales;  // [2][kv_heads] of the layer, or null
  uint8_t* pool;        // the layer's pages
  int64_t max_pos, pages;
  int hq, hkv, rot, page_shift;
  float eps, offset;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  x[0] = bf16lo_to_f32(u.x); x[1] = bf16hi_to_f32(u.x);
  x[2] = bf16lo_to_f32(u.y); x[3] = bf16hi_to_f32(u.y);
  x[4] = bf16lo_to_f32(u.z); x[5] = bf16hi_to_f32(u.z);
  x[6] = bf16lo_to_f32(u.w); x[7] = bf16hi_to_f32(u.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Two fp32 to e4m3 (nearest even; beyond the largest value: clamped), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

template <int D, bool E4M3, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const Params p) {
  pdl_enter();
  constexpr int LPH = D / 8;               // lanes per head
  constexpr int GROUPS = kThreads / LPH;   // heads of a block at a time
  const int lane = threadIdx.x & 31, l = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const int64_t tok = blockIdx.x;
  const int heads = p.hq + 2 * p.hkv;

  const int pos = __ldg(p.t.positions + tok);
  const int64_t slot = __ldg(p.t.slots + tok);
  const bool pos_ok = pos >= 0 && pos < p.max_pos;
  const bool slot_ok = slot >= 0 && slot < p.pages << p.page_shift;
  const bool turned = 8 * l < p.rot;  // rot is a multiple of 16: a lane is rotated as a whole
  const int half = p.rot >> 1;
  const bool second = !INTERLEAVED && 8 * l >= half;  // the b of its pairs
  float c[INTERLEAVED ? 4 : 8], s[INTERLEAVED ? 4 : 8];
  if (turned && pos_ok) {
    const float* row = p.rope + (int64_t)pos * p.rot + (INTERLEAVED ? 4 * l : second ? 8 * l - half : 8 * l);
#pragma unroll
    for (int i = 0; i < (INTERLEAVED ? 4 : 8); i += 4) {
      *reinterpret_cast<float4*>(c + i) = __ldg(reinterpret_cast<const float4*>(row + i));
      *reinterpret_cast<float4*>(s + i) = __ldg(reinterpret_cast<const float4*>(row + half + i));
    }
    if (second)
#pragma unroll
      for (int i = 0; i < (INTERLEAVED ? 4 : 8); ++i) s[i] = -s[i];  // y' = y c - partner s  for both halves
  }
  // the lane that holds the other half of this lane's pairs
  const int partner = (lane - l) + (second ? l - half / 8 : l + half / 8);

  // Every lane of a warp takes part in each round of heads; the loads of kBatch rounds go out together (one at a time
  // measured 25.7 us against 16.5 for 4099 tokens of 20 heads of 256, e4m3: too few bytes in flight).
  for (int h00 = blockIdx.y * GROUPS; h00 < heads; h00 += gridDim.y * GROUPS * kBatch) {
    uint4 us[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = h00 + b * gridDim.y * GROUPS + group;
      us[b] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        const uint16_t* x = h < p.hq ? p.t.q + tok * p.t.q_stride + (int64_t)h * D
                            : h < p.hq + p.hkv ? p.t.k + tok * p.t.k_stride + (int64_t)(h - p.hq) * D
                                               : p.t.v + tok * p.t.v_stride + (int64_t)(h - p.hq - p.hkv) * D;
        us[b] = *reinterpret_cast<const uint4*>(x + 8 * l);
      }
    }
#pragma unroll 1
    for (int b = 0; b < kBatch; ++b) {
      const int h0 = h00 + b * gridDim.y * GROUPS;
      if (h0 >= heads) break;
      const uint4 u = us[0];
#pragma unroll
      for (int i = 1; i < kBatch; ++i) us[i - 1] = us[i];
      const int h = h0 + group;
      const bool is_q = h < p.hq, is_k = !is_q && h < p.hq + p.hkv, active = h < heads;
      const int hk = is_q ? 0 : is_k ? h - p.hq : h - p.hq - p.hkv;
      float x[8];
      unpack8(u, x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
      for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const bool norm = is_q || is_k;
      if (norm) {
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        float w[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>((is_q ? p.wq : p.wk) + 8 * l)), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (w[i] + p.offset);
      }
      if constexpr (INTERLEAVED) {
        if (norm && turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * c[i] - b * s[i];
            x[2 * i + 1] = b * c[i] + a * s[i];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(0xFFFFFFFFu, x[i], partner & 31);
          if (norm && turned) x[i] = x[i] * c[i] - o * s[i];
        }
      }
      if (norm && !pos_ok)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __int_as_float(0x7FC00000);
      if (!active) continue;
      if (is_q) {
        *reinterpret_cast<uint4*>(p.t.q_out + tok * p.t.q_out_stride + (int64_t)h * D + 8 * l) = pack8(x);
      } else if (slot_ok) {
        const int64_t page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
        const int64_t e = ((((page * 2 + (is_k ? 0 : 1)) * p.hkv + hk) << p.page_shift) + off) * D + 8 * l;
        if constexpr (E4M3) {
          const float sc = p.scales ? __ldg(p.scales + (is_k ? 0 : p.hkv) + hk) : 1.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], sc);
          *reinterpret_cast<uint2*>(p.pool + e) = make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16,
                                                             e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
        } else {
          *reinterpret_cast<uint4*>(p.pool + 2 * e) = is_k ? pack8(x) : u;  // values keep their bits
        }
      }
    }
  }
}

template <int D, bool E4M3>
cudaError_t launch_d(const Params& p, int interleaved, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / 8);
  const int heads = p.hq + 2 * p.hkv;
  // A block per token once tokens alone fill the GPU several times over; below that a token's heads are spread
  // over blocks until each group of lanes has one head.
  const int64_t want = 8 * (int64_t)device_sm_count();
  const int rounds = (heads + GROUPS - 1) / GROUPS;
  int64_t split = (want + p.t.n - 1) / p.t.n;
  if (split > rounds) split = rounds;
  const dim3 grid((unsigned)p.t.n, (unsigned)split);
  return interleaved ? launch_pdl(norm_rope_kernel<D, E4M3, true>, grid, dim3(kThreads), 0, st, p)
                     : launch_pdl(norm_rope_kernel<D, E4M3, false>, grid, dim3(kThreads), 0, st, p);
}

template <bool E4M3>
cudaError_t launch_type(const Params& p, int D, int interleaved, cudaStream_t st) {
  if (D == 64) return launch_d<64, E4M3>(p, interleaved, st);
  if (D == 128) return launch_d<128, E4M3>(p, interleaved, st);
  return launch_d<256, E4M3>(p, interleaved, st);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeTokens& t, const trellis_norm_rope_t& nr, const trellis_cache_t& c, int layer,
                             cudaStream_t st) {
  Params p{};
  p.t = t;
  p.wq = nr.q_weight; p.wk = nr.k_weight; p.rope = nr.rope;
  p.scales = c.scales ? c.scales + (int64_t)layer * 2 * c.heads : nullptr;
  p.pool = static_cast<uint8_t*>(c.pool) + (int64_t)layer * c.pages * cache_page_bytes(c);
  p.max_pos = nr.max_pos; p.pages = c.pages;
  p.hq = nr.q_heads; p.hkv = nr.kv_heads; p.rot = nr.rotary_dim;
  p.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  p.eps = nr.eps; p.offset = nr.weight_offset;
  return c.dtype == TRELLIS_E4M3 ? launch_type<true>(p, c.head_dim, nr.interleaved, st)
                                 : launch_type<false>(p, c.head_dim, nr.interleaved, st);
}

}  // namespace trellis

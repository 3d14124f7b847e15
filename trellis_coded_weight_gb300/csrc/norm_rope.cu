// norm_rope.cu -- norms of queries and keys for each head, the rotation by position and the write of keys and
// values into the pages of a cache, in one launch (trellis_qk_norm_rope_append).
//
// Per token and head, with x the head's D numbers, w its weights and (c, s) the token's row of the rotation table:
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset);   (a, b) -> (a c - b s, b c + a s) on the rotated pairs
// Everything in fp32, one rounding at the end (bf16, or e4m3 of y times the reciprocal of its scale).
//
// A head lives in D/8 neighbouring lanes, 8 numbers (one 16-byte load) each: the sum of squares is a shuffle over
// those lanes, a pair that spans half a rotation is one shuffle away, an interleaved pair is in one lane.  Nothing is
// staged.  A group of lanes has a share of one token's heads -- queries, then keys, then values, each in a loop of its own
// with its weights in registers -- and keeps the cosines and sines of its lanes.
// Bound: launch latency for a few tokens (one of 56 heads of 128: 2.2 us); beyond, the latency of loads: 4099 tokens of 20 heads of
// 256 into e4m3 take 21 us, 3.9 TB/s, instructions issue in 42 % of the cycles, and two thirds of the warps' time is spent waiting
// for numbers from memory, two heads of which are in flight (a general loop over all kinds of heads took three times the
// instructions, and 25 us).
#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "serving.h"

namespace trellis {
namespace {

constexpr int kThreads = 256;
// Blocks of an SM at a time (4096 tokens of 56 heads of 128: 28.1 us with 4, 36 with 5 or 6, whose registers spill).
constexpr int kPerSM = 4;

struct Params {
  NormRopeTokens t;
  const uint16_t *wq, *wk;
  const float* rope;
  const float* scales;  // [2][kv_heads] of the layer, or null
  uint8_t* pool;        // the layer's pages
  int64_t max_pos, pages;
  int hq, hkv, rot, page_shift, split;
  float eps, offset;
};

__device__ __forceinline__ void unpack8(const uint4& u, float2 (&x)[4]) {
  x[0] = make_float2(bf16lo_to_f32(u.x), bf16hi_to_f32(u.x));
  x[1] = make_float2(bf16lo_to_f32(u.y), bf16hi_to_f32(u.y));
  x[2] = make_float2(bf16lo_to_f32(u.z), bf16hi_to_f32(u.z));
  x[3] = make_float2(bf16lo_to_f32(u.w), bf16hi_to_f32(u.w));
}
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
}

// Two fp32 to e4m3 (nearest even; beyond the largest value: clamped), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

template <int D, bool E4M3, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kPerSM) norm_rope_kernel(const Params p) {
  pdl_enter();
  constexpr int LPH = D / 8;  // lanes of a head
  const int lane = threadIdx.x & 31, l = lane % LPH;
  constexpr uint32_t kGroup = LPH == 32 ? 0xFFFFFFFFu : (1u << LPH) - 1;
  const uint32_t lanes = kGroup << (lane - l);  // this group's
  const int heads = p.hq + 2 * p.hkv, split = p.split;
  // this group: heads h, h + split, .. of a token
  const uint32_t gid = (blockIdx.x * (uint32_t)kThreads + threadIdx.x) / LPH;
  const uint32_t tok = gid / (uint32_t)split;
  if (tok >= (uint32_t)p.t.n) return;
  int h = (int)(gid - tok * (uint32_t)split);

  const int pos = p.t.positions[tok];
  const int64_t slot = p.t.slots[tok];
  const uint16_t* const qb = p.t.q + tok * p.t.q_stride + 8 * l;
  const uint16_t* const kb = p.t.k + tok * p.t.k_stride + 8 * l;
  const uint16_t* const vb = p.t.v + tok * p.t.v_stride + 8 * l;
  const auto fetch = [&](int at) {
    const uint16_t* from = at < p.hq ? qb + at * D : at < p.hq + p.hkv ? kb + (at - p.hq) * D : vb + (at - p.hq - p.hkv) * D;
    return at < heads ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
  };
  uint4 u = fetch(h), ahead = fetch(h + split);  // two heads in flight, before the position is used

  const bool pos_ok = pos >= 0 && pos < p.max_pos;
  const bool turned = 8 * l < p.rot;  // rot is a multiple of 16: a lane is rotated as a whole
  const int half = p.rot >> 1;
  const bool second = !INTERLEAVED && 8 * l >= half;  // the b of its pairs
  // interleaved: cosines and sines of the lane's four pairs; else of its eight numbers, two by two.  No turn: 1 and 0;
  // positions out of range: NaN.
  float2 c[INTERLEAVED ? 2 : 4], s[INTERLEAVED ? 2 : 4];
  const float one = pos_ok ? 1.f : __int_as_float(0x7FC00000);
#pragma unroll
  for (int i = 0; i < (INTERLEAVED ? 2 : 4); ++i) {
    c[i] = make_float2(one, one);
    s[i] = make_float2(0.f, 0.f);
  }
  if (turned && pos_ok) {
    const float* row = p.rope + (int64_t)pos * p.rot + (INTERLEAVED ? 4 * l : second ? 8 * l - half : 8 * l);
    const float sign = INTERLEAVED || second ? 1.f : -1.f;  // y' = y c + partner s for both halves
#pragma unroll
    for (int i = 0; i < (INTERLEAVED ? 2 : 4); i += 2) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(row + 2 * i)), sv = __ldg(reinterpret_cast<const float4*>(row + half + 2 * i));
      c[i] = make_float2(cv.x, cv.y);
      c[i + 1] = make_float2(cv.z, cv.w);
      s[i] = make_float2(sign * sv.x, sign * sv.y);
      s[i + 1] = make_float2(sign * sv.z, sign * sv.w);
    }
  }
  // the lane that holds the other half of this lane's pairs
  const int partner = turned ? (lane - l) + (second ? l - half / 8 : l + half / 8) : lane;

  float2 w[4];
  const auto weights = [&](const uint16_t* from) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(from + 8 * l)), w);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __fadd2_rn(w[i], make_float2(p.offset, p.offset));
  };
  const auto advance = [&] {
    h += split;
    u = ahead;
    ahead = fetch(h + split);
  };
  // the head in u, normed and rotated
  const auto normed = [&](float2 (&x)[4]) {
    unpack8(u, x);
    float2 sq = __fmul2_rn(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sq = __ffma2_rn(x[i], x[i], sq);
    float ss = sq.x + sq.y;
#pragma unroll
    for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(lanes, ss, o);
    const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __fmul2_rn(__fmul2_rn(x[i], make_float2(r, r)), w[i]);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float cc = i & 1 ? c[i / 2].y : c[i / 2].x, sc = i & 1 ? s[i / 2].y : s[i / 2].x;
        x[i] = make_float2(x[i].x * cc - x[i].y * sc, x[i].y * cc + x[i].x * sc);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 o = make_float2(__shfl_sync(lanes, x[i].x, partner), __shfl_sync(lanes, x[i].y, partner));
        x[i] = __ffma2_rn(o, s[i], __fmul2_rn(x[i], c[i]));
      }
    }
  };

  weights(p.wq);
  uint16_t* const out = p.t.q_out + tok * p.t.q_out_stride + 8 * l;
  while (h < p.hq) {
    float2 x[4];
    normed(x);
    *reinterpret_cast<uint4*>(out + h * D) = pack8(x);
    advance();
  }
  if (slot < 0 || slot >= p.pages << p.page_shift) return;
  // the heads of keys, then those of values, are one after the other in a page
  const int64_t kv_row = ((slot >> p.page_shift) * 2 * p.hkv << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
  uint8_t* const to = p.pool + (kv_row * D + 8 * l) * (E4M3 ? 1 : 2);
  const auto keep = [&](const float2 (&x)[4], int hk, const uint4* same) {
    uint8_t* at = to + ((int64_t)(hk * D) << p.page_shift) * (E4M3 ? 1 : 2);
    if constexpr (E4M3) {
      const float inv = p.scales ? __fdiv_rn(1.f, __ldg(p.scales + hk)) : 1.f;
      *reinterpret_cast<uint2*>(at) = make_uint2(e4m3x2(x[0].x * inv, x[0].y * inv) | e4m3x2(x[1].x * inv, x[1].y * inv) << 16,
                                                 e4m3x2(x[2].x * inv, x[2].y * inv) | e4m3x2(x[3].x * inv, x[3].y * inv) << 16);
    } else {
      *reinterpret_cast<uint4*>(at) = same ? *same : pack8(x);
    }
  };
  weights(p.wk);
  while (h < p.hq + p.hkv) {
    float2 x[4];
    normed(x);
    keep(x, h - p.hq, nullptr);
    advance();
  }
  while (h < heads) {
    float2 x[4];
    unpack8(u, x);
    keep(x, h - p.hq, &u);  // bf16 values keep their bits
    advance();
  }
}

template <int D, bool E4M3>
cudaError_t launch_d(Params p, int interleaved, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / 8);
  const int heads = p.hq + 2 * p.hkv;
  // A token's heads go to as many groups of lanes as fill the GPU once over all tokens: several heads each for many
  // tokens, one for a few.  (Rounding up instead, into a second wave, measured 35 us against 28.)  Rounded down, groups idle just
  // past a whole number of shares, and past one group for each token a second wave begins: 20 heads of 256 into e4m3, 2432 tokens
  // 13.2 us, 2433 19.7, 4864 23.3, 4865 33.8; 56 heads of 128, 4864 tokens 29.9, 4865 45.3.
  const int64_t groups = (int64_t)kPerSM * device_sm_count() * GROUPS;
  const int64_t split = groups / p.t.n;
  p.split = (int)(split < 1 ? 1 : split > heads ? heads : split);
  const dim3 grid((unsigned)(((int64_t)p.t.n * p.split + GROUPS - 1) / GROUPS));
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

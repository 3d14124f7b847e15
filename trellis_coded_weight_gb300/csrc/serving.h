// serving.h -- internal host-side launchers of the calls around a decoding step's projections (norms with
// rotation and cache write, tree attention, cache pages, token log probabilities).  Arguments are validated by
// abi_serving.cu before these are called.
//
// Their kernels are launched as dependents (pdl.cuh): they may have begun before the call ahead has written what they read, so such
// data (lengths, tables, masks, queries, logits, positions) is not read-only while they run.  It is loaded by plain loads or from
// L2, never by the read-only path; that is for the model's constants (norm weights, rotation tables, scales).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "trellis.h"

namespace trellis {

inline int64_t cache_elem_bytes(const trellis_cache_t& c) { return c.dtype == TRELLIS_E4M3 ? 1 : 2; }
// Bytes of one page (keys and values of all heads) in one layer; a multiple of 2048.
inline int64_t cache_page_bytes(const trellis_cache_t& c) {
  return (int64_t)2 * c.heads * c.page_size * c.head_dim * cache_elem_bytes(c);
}

struct NormRopeTokens {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int32_t* positions;
  const int64_t* slots;
  uint16_t* q_out;
  int n;
};
cudaError_t launch_norm_rope(const NormRopeTokens& t, const trellis_norm_rope_t& p, const trellis_cache_t& c, int layer,
                             cudaStream_t st);

cudaError_t launch_tree_attention(const uint16_t* q, int64_t q_stride, const trellis_cache_t& c, int layer,
                                  const trellis_drafts_t& d, int q_heads, float scale, uint16_t* out,
                                  int64_t out_stride, float* lse, void* workspace, cudaStream_t st);
size_t tree_workspace_bytes(const trellis_cache_t& c, int batch, int max_tokens, int q_heads);

cudaError_t launch_cache_copy(const trellis_cache_t& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t st);
cudaError_t launch_cache_fork(const trellis_cache_t& c, int32_t* table, int32_t* lens, int32_t* refs,
                              const int32_t* parent, const int32_t* child, int32_t* status, int pairs, int rows,
                              int width, int room, void* workspace, cudaStream_t st);
cudaError_t launch_cache_compact(const trellis_cache_t& c, const int32_t* table, const int32_t* refs,
                                 int32_t* out_table, int32_t* out_refs, int rows, int width, void* workspace,
                                 cudaStream_t st);
size_t cache_workspace_bytes(const trellis_cache_t& c, int pairs, int width);
cudaError_t launch_cache_commit(const trellis_cache_t& c, const int32_t* table, const int32_t* prefix,
                                const int32_t* path, const int32_t* accepted, int32_t* lens, int batch, int width,
                                int max_tokens, cudaStream_t st);

cudaError_t launch_token_logprobs(const void* logits, int dtype, int64_t row_stride, const int32_t* tokens, int n,
                                  int vocab, int cands, int top_k, float temperature, float* logprobs, float* lse,
                                  float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                                  cudaStream_t st);
size_t logprobs_workspace_bytes(int n, int vocab, int top_k);

constexpr int kTreeMaxTokens = 64;  // a draft mask is one 64-bit word
constexpr int kTreeMaxBatch = 1024;
constexpr int kForkMaxPairs = 1024;
constexpr int kMaxCands = 64;
constexpr int kMaxTop = 32;
constexpr float kLog2e = 1.44269504088896341f;

}  // namespace trellis

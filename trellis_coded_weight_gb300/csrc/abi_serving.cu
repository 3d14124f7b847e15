// abi_serving.cu -- the exported C entry points around a decoding step's projections (declared in
// include/trellis.h): argument validation on the host, then the launches on the caller's stream.  Every failed
// check returns before any launch; nothing here allocates device memory.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "abi_common.h"
#include "serving.h"
#include "trellis.h"

using trellis::aligned16;
using trellis::cuda_status;
using trellis::device_ok;

namespace {

int cache_ok(const trellis_cache_t* c) {
  if (!c || !c->pool) return TRELLIS_ENULL;
  if (c->reserved != 0) return TRELLIS_ESHAPE;
  if (c->pages < 1 || c->pages > (1 << 24) || c->layers < 1 || c->layers > 65535 || c->heads < 1 || c->heads > 1024)
    return TRELLIS_ESHAPE;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return TRELLIS_ESHAPE;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return TRELLIS_ESHAPE;
  if (c->dtype != TRELLIS_BF16 && c->dtype != TRELLIS_E4M3) return TRELLIS_ESHAPE;
  if (c->dtype == TRELLIS_BF16 && c->scales) return TRELLIS_ESHAPE;
  // rows of head_dim numbers in one layer: a tensor map's coordinate is 32 bits
  if (c->pages * 2 * c->heads * c->page_size > INT32_MAX) return TRELLIS_ESHAPE;
  if (!aligned16(c->pool) || !aligned16(c->scales)) return TRELLIS_EALIGN;
  return TRELLIS_OK;
}

bool stride_ok(int64_t stride, int64_t least) { return stride >= least && stride % 8 == 0 && stride <= (int64_t)1 << 40; }

}  // namespace

extern "C" {

int trellis_check_cache(const trellis_cache_t* cache) { return cache_ok(cache); }

int trellis_qk_norm_rope_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                const uint16_t* v, int64_t v_stride, const int32_t* positions, const int64_t* slots,
                                uint16_t* q_out, int64_t q_out_stride, int n, const trellis_norm_rope_t* p,
                                const trellis_cache_t* cache, int layer, trellis_stream_t stream) {
  int st = cache_ok(cache);
  if (st) return st;
  if (!p) return TRELLIS_ENULL;
  if (n < 0 || n > (1 << 20)) return TRELLIS_EM;
  if (p->reserved != 0 || p->q_heads < 1 || p->q_heads > 1024 || p->kv_heads != cache->heads ||
      p->head_dim != cache->head_dim || layer < 0 || layer >= cache->layers)
    return TRELLIS_ESHAPE;
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 16 != 0 || p->max_pos < 0 ||
      (p->interleaved != 0 && p->interleaved != 1) || !(p->eps >= 0.f) || !std::isfinite(p->eps) ||
      !std::isfinite(p->weight_offset))
    return TRELLIS_ESHAPE;
  const int64_t qw = (int64_t)p->q_heads * p->head_dim, kw = (int64_t)p->kv_heads * p->head_dim;
  if (n > 1 && (!stride_ok(q_stride, qw) || !stride_ok(k_stride, kw) || !stride_ok(v_stride, kw) ||
                !stride_ok(q_out_stride, qw)))
    return TRELLIS_ESHAPE;
  if (n == 0) return TRELLIS_OK;
  if (!q || !k || !v || !positions || !slots || !q_out || !p->q_weight || !p->k_weight || (p->rotary_dim && !p->rope))
    return TRELLIS_ENULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(positions) || !aligned16(slots) ||
      !aligned16(q_out) || !aligned16(p->q_weight) || !aligned16(p->k_weight) || !aligned16(p->rope))
    return TRELLIS_EALIGN;
  if ((st = device_ok())) return st;
  const trellis::NormRopeTokens t{q, k, v, q_stride, k_stride, v_stride, q_out_stride, positions, slots, q_out, n};
  return cuda_status(trellis::launch_norm_rope(t, *p, *cache, layer, static_cast<cudaStream_t>(stream)));
}

size_t trellis_tree_workspace_bytes(const trellis_cache_t* cache, int batch, int max_tokens, int q_heads) {
  if (cache_ok(cache) != TRELLIS_OK || batch < 1 || batch > trellis::kTreeMaxBatch || max_tokens < 1 ||
      max_tokens > trellis::kTreeMaxTokens || q_heads < 1 || q_heads > 1024 || q_heads % cache->heads != 0)
    return 0;
  return trellis::tree_workspace_bytes(*cache, batch, max_tokens, q_heads);
}

int trellis_tree_attention(const uint16_t* q, int64_t q_stride, const trellis_cache_t* cache, int layer,
                           const trellis_drafts_t* d, int q_heads, float scale, uint16_t* out, int64_t out_stride,
                           float* lse, void* workspace, size_t workspace_bytes, trellis_stream_t stream) {
  int st = cache_ok(cache);
  if (st) return st;
  if (!d) return TRELLIS_ENULL;
  if (d->batch < 0 || d->batch > trellis::kTreeMaxBatch || d->n < 0 || d->n > (1 << 20)) return TRELLIS_EM;
  if (d->batch == 0 || d->n == 0) return TRELLIS_OK;
  if (d->max_tokens < 1 || d->max_tokens > trellis::kTreeMaxTokens) return TRELLIS_EM;
  if (layer < 0 || layer >= cache->layers || q_heads < 1 || q_heads > 1024 || q_heads % cache->heads != 0 ||
      d->width < 1 || (int64_t)d->width * cache->page_size > (1 << 30) || !std::isfinite(scale))
    return TRELLIS_ESHAPE;
  // steps of all items are counted in 32 bits: 64 keys by 16 rows of a key/value head at the least
  const int64_t tiles = ((int64_t)d->width * cache->page_size + 63) / 64;
  const int64_t blocks = ((int64_t)d->max_tokens * (q_heads / cache->heads) + 15) / 16 * cache->heads;
  if ((double)d->batch * (double)tiles * (double)blocks > (double)(1 << 30)) return TRELLIS_ESHAPE;
  const int64_t w = (int64_t)q_heads * cache->head_dim;
  if (d->n > 1 && (!stride_ok(q_stride, w) || !stride_ok(out_stride, w))) return TRELLIS_ESHAPE;
  if (!q || !out || !d->table || !d->prefix || !d->q_start) return TRELLIS_ENULL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || !aligned16(d->table) || !aligned16(d->prefix) ||
      !aligned16(d->q_start) || !aligned16(d->mask))
    return TRELLIS_EALIGN;
  if ((st = device_ok())) return st;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < trellis::tree_workspace_bytes(*cache, d->batch, d->max_tokens, q_heads))
    return TRELLIS_EWORKSPACE;
  return cuda_status(trellis::launch_tree_attention(q, q_stride, *cache, layer, *d, q_heads, scale, out, out_stride,
                                                    lse, workspace, static_cast<cudaStream_t>(stream)));
}

int trellis_cache_copy(const trellis_cache_t* cache, const int32_t* src, const int32_t* dst, int n,
                       trellis_stream_t stream) {
  int st = cache_ok(cache);
  if (st) return st;
  if (n < 0 || n > (1 << 24)) return TRELLIS_EM;
  if (n == 0) return TRELLIS_OK;
  if (!src || !dst) return TRELLIS_ENULL;
  if (!aligned16(src) || !aligned16(dst)) return TRELLIS_EALIGN;
  if ((st = device_ok())) return st;
  return cuda_status(trellis::launch_cache_copy(*cache, src, dst, n, static_cast<cudaStream_t>(stream)));
}

size_t trellis_cache_workspace_bytes(const trellis_cache_t* cache, int pairs, int width) {
  if (cache_ok(cache) != TRELLIS_OK || pairs < 0 || pairs > trellis::kForkMaxPairs || width < 1 || width > (1 << 20))
    return 0;
  return trellis::cache_workspace_bytes(*cache, pairs, width);
}

int trellis_cache_fork(const trellis_cache_t* cache, int32_t* table, int32_t* lens, int32_t* refs,
                       const int32_t* parent, const int32_t* child, int32_t* status, int pairs, int rows, int width,
                       int room, void* workspace, size_t workspace_bytes, trellis_stream_t stream) {
  int st = cache_ok(cache);
  if (st) return st;
  if (pairs < 0 || pairs > trellis::kForkMaxPairs) return TRELLIS_EM;
  if (rows < 1 || width < 1 || width > (1 << 20) || (int64_t)rows * width > INT32_MAX || room < 0 || room > (1 << 24))
    return TRELLIS_ESHAPE;
  if (pairs == 0) return TRELLIS_OK;
  if (!table || !lens || !refs || !parent || !child || !status) return TRELLIS_ENULL;
  if (!aligned16(table) || !aligned16(lens) || !aligned16(refs) || !aligned16(parent) || !aligned16(child) ||
      !aligned16(status))
    return TRELLIS_EALIGN;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < trellis::cache_workspace_bytes(*cache, pairs, width))
    return TRELLIS_EWORKSPACE;
  if ((st = device_ok())) return st;
  return cuda_status(trellis::launch_cache_fork(*cache, table, lens, refs, parent, child, status, pairs, rows, width,
                                                room, workspace, static_cast<cudaStream_t>(stream)));
}

int trellis_cache_compact(const trellis_cache_t* cache, const int32_t* table, const int32_t* refs, int32_t* out_table,
                          int32_t* out_refs, int rows, int width, void* workspace, size_t workspace_bytes,
                          trellis_stream_t stream) {
  int st = cache_ok(cache);
  if (st) return st;
  if (rows < 1 || width < 1 || width > (1 << 20) || (int64_t)rows * width > INT32_MAX) return TRELLIS_ESHAPE;
  if (!table || !refs || !out_table || !out_refs) return TRELLIS_ENULL;
  if (!aligned16(table) || !aligned16(refs) || !aligned16(out_table) || !aligned16(out_refs)) return TRELLIS_EALIGN;
  if (!workspace || !aligned16(workspace) || workspace_bytes < trellis::cache_workspace_bytes(*cache, 0, width))
    return TRELLIS_EWORKSPACE;
  if ((st = device_ok())) return st;
  return cuda_status(trellis::launch_cache_compact(*cache, table, refs, out_table, out_refs, rows, width, workspace,
                                                   static_cast<cudaStream_t>(stream)));
}

int trellis_cache_commit(const trellis_cache_t* cache, const int32_t* table, const int32_t* prefix,
                         const int32_t* path, const int32_t* accepted, int32_t* lens, int batch, int width,
                         int max_tokens, trellis_stream_t stream) {
  int st = cache_ok(cache);
  if (st) return st;
  if (batch < 0 || batch > (1 << 16)) return TRELLIS_EM;
  if (max_tokens < 1 || max_tokens > trellis::kTreeMaxTokens) return TRELLIS_EM;
  if (width < 1 || (int64_t)width * cache->page_size > (1 << 30)) return TRELLIS_ESHAPE;
  if (batch == 0) return TRELLIS_OK;
  if (!table || !prefix || !path || !accepted || !lens) return TRELLIS_ENULL;
  if (!aligned16(table) || !aligned16(prefix) || !aligned16(path) || !aligned16(accepted) || !aligned16(lens))
    return TRELLIS_EALIGN;
  if ((st = device_ok())) return st;
  return cuda_status(trellis::launch_cache_commit(*cache, table, prefix, path, accepted, lens, batch, width,
                                                  max_tokens, static_cast<cudaStream_t>(stream)));
}

size_t trellis_logprobs_workspace_bytes(int n, int vocab, int top_k) {
  if (n < 1 || n > (1 << 20) || vocab < 1 || vocab > (1 << 24) || top_k < 0 || top_k > trellis::kMaxTop || top_k > vocab)
    return 0;
  return trellis::logprobs_workspace_bytes(n, vocab, top_k);
}

int trellis_token_logprobs(const void* logits, int dtype, int64_t row_stride, const int32_t* tokens, int n, int vocab,
                           int cands, int top_k, float temperature, float* logprobs, float* lse, float* entropy,
                           int32_t* top_ids, float* top_logprobs, void* workspace, size_t workspace_bytes,
                           trellis_stream_t stream) {
  if (n < 0 || n > (1 << 20)) return TRELLIS_EM;
  if (dtype != TRELLIS_BF16 && dtype != TRELLIS_F32) return TRELLIS_ESHAPE;
  if (vocab < 1 || vocab > (1 << 24) || cands < 0 || cands > trellis::kMaxCands || top_k < 0 ||
      top_k > trellis::kMaxTop || top_k > vocab || !(temperature > 0.f) || !std::isfinite(temperature) ||
      !std::isfinite(trellis::kLog2e / temperature))  // the exponentials' factor
    return TRELLIS_ESHAPE;
  if (n > 1 && (row_stride < vocab || row_stride > (int64_t)1 << 40)) return TRELLIS_ESHAPE;
  if (n == 0) return TRELLIS_OK;
  if (!logits || !lse || !entropy || (cands && (!tokens || !logprobs)) || (top_k && (!top_ids || !top_logprobs)))
    return TRELLIS_ENULL;
  if (!aligned16(logits) || !aligned16(tokens) || !aligned16(logprobs) || !aligned16(lse) || !aligned16(entropy) ||
      !aligned16(top_ids) || !aligned16(top_logprobs))
    return TRELLIS_EALIGN;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < trellis::logprobs_workspace_bytes(n, vocab, top_k))
    return TRELLIS_EWORKSPACE;
  int st = device_ok();
  if (st) return st;
  return cuda_status(trellis::launch_token_logprobs(logits, dtype, row_stride, tokens, n, vocab, cands, top_k,
                                                    temperature, logprobs, lse, entropy, top_ids, top_logprobs,
                                                    workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// paged_attn_tree.cu — host side of tree attention: validation, dispatch and
// the C entry points.  The kernel is in paged_attn_tree_kernels.cuh.
#include <math.h>

#include <type_traits>

#include "host_common.h"
#include "paged_attn_tree_kernels.cuh"

namespace pkv {
namespace {

using TreeFn = void (*)(const TreeParams);

template <class DT, class CT>
TreeFn tree_fn(int head_dim) {
  return head_dim == 128 ? paged_attn_tree_kernel<128, DT, CT>
                         : paged_attn_tree_kernel<64, DT, CT>;
}

// Validates and launches; fp8: the caches hold E4M3 codes with per-kv-head
// scales k_scales / v_scales.
pkv_status tree_launch(void* out, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* query_start, const int32_t* parents, float scale,
                       int num_seqs, int num_tokens, int num_heads, int num_kv_heads,
                       int head_dim, int block_size, int max_blocks_per_seq, int max_context_len,
                       int max_query_len, int num_blocks, pkv_dtype dtype, bool fp8,
                       const float* k_scales, const float* v_scales, unsigned* dev_err,
                       void* stream) {
  if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
      max_blocks_per_seq <= 0 || max_context_len < 0 || max_query_len < 0 || num_blocks <= 0 ||
      !dtype_valid(dtype) || num_heads % num_kv_heads != 0 || !isfinite(scale) ||
      max_query_len > max_context_len)
    return PKV_ERR_INVALID_ARG;
  if (!head_dim_supported(head_dim) || !block_size_supported(block_size) ||
      max_query_len > PKV_MAX_TREE_NODES)
    return PKV_ERR_UNSUPPORTED;
  const int group = num_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_context_len) >
      static_cast<long long>(max_blocks_per_seq) * block_size)
    return PKV_ERR_INVALID_ARG;
  if (fp8 && (!k_scales || !v_scales)) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_query_len == 0 || num_tokens == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start ||
      !parents)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  const long long grid =
      (static_cast<long long>(num_seqs) * max_query_len * num_heads + 3) / 4;
  if (grid > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  TreeParams p = {};
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.parents = parents;
  p.qscale = scale * kLog2e;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.max_query_len = max_query_len;
  p.num_blocks = num_blocks;
  p.err = dev_err;
  const TreeFn fn = dtype == PKV_FP16 ? (fp8 ? tree_fn<Fp16, Fp8E4M3>(head_dim)
                                             : tree_fn<Fp16, Fp16>(head_dim))
                                      : (fp8 ? tree_fn<Bf16, Fp8E4M3>(head_dim)
                                             : tree_fn<Bf16, Bf16>(head_dim));
  fn<<<static_cast<unsigned>(grid), 128, 0, as_stream(stream)>>>(p);
  return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_paged_attn_tree(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
    const int32_t* parents, float scale, int num_seqs, int num_tokens, int num_heads,
    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int max_context_len,
    int max_query_len, int num_blocks, pkv_dtype dtype, unsigned* dev_err, void* stream) {
  return pkv::tree_launch(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                          parents, scale, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                          block_size, max_blocks_per_seq, max_context_len, max_query_len,
                          num_blocks, dtype, false, nullptr, nullptr, dev_err, stream);
}

extern "C" pkv_status pkv_paged_attn_tree_fp8(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
    const int32_t* parents, float scale, const float* k_scales, const float* v_scales,
    int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
    int max_blocks_per_seq, int max_context_len, int max_query_len, int num_blocks,
    pkv_dtype dtype, unsigned* dev_err, void* stream) {
  return pkv::tree_launch(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                          parents, scale, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                          block_size, max_blocks_per_seq, max_context_len, max_query_len,
                          num_blocks, dtype, true, k_scales, v_scales, dev_err, stream);
}

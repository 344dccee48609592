// paged_attn_tree.cu — host side of tree attention: validation, dispatch and
// the C entry points.  The kernels are in paged_attn_tree_kernels.cuh.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "host_common.h"
#include "paged_attn_tree_kernels.cuh"

namespace pkv {
namespace {

using TreeFn = void (*)(const TreeParams, const CUtensorMap, const CUtensorMap);
using TreeMergeFn = void (*)(const TreeParams);

struct TreeEntry {
  TreeFn fn;
  TreeMergeFn merge, merge_many;  // for few and for many pieces a unit
  size_t smem;
  int threads, rows, ctas;  // ctas: those resident at once
};

constexpr int kSms = 148;
constexpr int kMergeSlices = 4;

template <int D, class DT, bool FP8, int QT>
TreeEntry tree_entry() {
  using Tr = TreeTraits<D, DT, FP8, QT>;
  return {paged_attn_tree_kernel<Tr>, paged_attn_tree_merge_kernel<D, Tr::ROWS, DT, 1>,
          paged_attn_tree_merge_kernel<D, Tr::ROWS, DT, kMergeSlices>,
          Tr::smem_bytes(), Tr::THREADS, Tr::ROWS, kSms * Tr::MIN_BLOCKS};
}

template <int D, class DT>
TreeEntry tree_entry(bool fp8, int qt) {
  if (fp8) return tree_entry<D, DT, true, 2>();
  return qt == 1 ? tree_entry<D, DT, false, 1>() : tree_entry<D, DT, false, 2>();
}

// Whether units are left whole, which spares the merge kernel and, with no more
// units than CTAs, the scan of the lengths: where a unit has few tiles, and more
// of them the better the units fill the GPU.  Measured on B200 (us, cut / whole;
// GQA of 8 kv heads): 1 sequence of 512 tokens 12.0 / 10.8, of 768 12.6 / 13.5; 4 of
// 768 17.3 / 13.6; 8 of 900 18.8 / 16.3; 32 of 700 26.9 / 21.9, of 1200 40.5 / 34.9.
bool tree_whole(long long units, int max_context_len) {
  const int tiles = (max_context_len + kTreeKeys - 1) / kTreeKeys;
  return tiles <= std::min(11 + units / 12, 20LL);
}

// Two query tiles and two groups of softmax warps a CTA, one CTA an SM: once a unit
// can have more than 128 rows, as its query tiles share each K/V tile; over E4M3,
// whose tiles, held twice, leave room for one CTA an SM; for whole units that are no
// more than the SMs, as the groups take a unit's tiles in turn (1 sequence of 300
// tokens 10.1 -> 8.9 us, 16 of 700 16.8 -> 15.0); and above 64 rows a unit, where the
// deeper ring of tiles outlasts a unit's change (GQA chat batch 69 -> 66).  Else one
// query tile and two CTAs an SM (LLaMA-7B batch, 16 rows a unit: 163 -> 105 us; 64
// sequences of 700 tokens, 32 rows: 59 -> 43).
TreeEntry tree_entry(int head_dim, pkv_dtype dt, bool fp8, int num_seqs, int num_kv_heads,
                     int max_rows, int max_context_len) {
  const long long units = static_cast<long long>(num_seqs) * num_kv_heads;  // of one query tile
  const int qt =
      fp8 || max_rows > 64 || (units <= kSms && tree_whole(units, max_context_len)) ? 2 : 1;
  if (head_dim == 128)
    return dt == PKV_FP16 ? tree_entry<128, Fp16>(fp8, qt) : tree_entry<128, Bf16>(fp8, qt);
  return dt == PKV_FP16 ? tree_entry<64, Fp16>(fp8, qt) : tree_entry<64, Bf16>(fp8, qt);
}

// CTAs of a launch: no more than are resident, nor than the longest batch
// within the bounds has stretches of kTreeMinTiles.
int tree_ctas(int resident, int rows, int num_seqs, int group, int num_kv_heads,
              int max_context_len, int max_query_len) {
  const long long tiles =
      2LL * ((max_context_len + kTreeKeys - 1) / kTreeKeys + tree_unit_cost(rows));  // positions
  const long long units =
      static_cast<long long>(num_seqs) * ((max_query_len * group + rows - 1) / rows);
  // units * kv heads * tiles, without its overflow
  if (units > resident || units * num_kv_heads > resident) return resident;
  if (tree_whole(units * num_kv_heads, max_context_len))
    return static_cast<int>(units * num_kv_heads);
  const long long most = (units * num_kv_heads * tiles + kTreeMinTiles - 1) / kTreeMinTiles;
  return static_cast<int>(std::min<long long>(resident, most));
}

size_t tree_ws_bytes(int ctas, int rows, int head_dim, bool whole) {
  if (whole) return 0;
  return 16 + static_cast<size_t>(ctas) *
                  (sizeof(int4) +
                   2 * static_cast<size_t>(rows) * (8 + 4 * static_cast<size_t>(head_dim)));
}

// Validates and launches; fp8: the caches hold E4M3 codes with per-kv-head
// scales k_scales / v_scales.
pkv_status tree_launch(void* out, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* query_start, const int32_t* parents, float scale,
                       int num_seqs, int num_tokens, int num_heads, int num_kv_heads,
                       int head_dim, int block_size, int max_blocks_per_seq, int max_context_len,
                       int max_query_len, int num_blocks, pkv_dtype dtype, bool fp8,
                       const float* k_scales, const float* v_scales, void* workspace,
                       size_t workspace_bytes, unsigned* dev_err, void* stream) {
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
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(block_tables, context_lens, query_start, parents, k_scales, v_scales, dev_err))
    return PKV_ERR_INVALID_ARG;
  const int max_rows = max_query_len * group;
  const TreeEntry e = tree_entry(head_dim, dtype, fp8, num_seqs, num_kv_heads, max_rows,
                                 max_context_len);
  const int ctas = tree_ctas(e.ctas, e.rows, num_seqs, group, num_kv_heads, max_context_len,
                             max_query_len);
  const int max_rts = (max_rows + e.rows - 1) / e.rows;
  const long long units = static_cast<long long>(num_seqs) * max_rts * num_kv_heads;
  const bool whole = tree_whole(units, max_context_len);
  const size_t need = tree_ws_bytes(ctas, e.rows, head_dim, whole);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return PKV_ERR_WORKSPACE;
  const pkv_dtype cdt = fp8 ? PKV_FP8_E4M3 : dtype;
  CUtensorMap kmap, vmap;
  pkv_status st =
      cache_tensor_map(&kmap, k_cache, num_blocks, num_kv_heads, block_size, head_dim, cdt);
  if (st != PKV_OK) return st;
  st = cache_tensor_map(&vmap, v_cache, num_blocks, num_kv_heads, block_size, head_dim, cdt);
  if (st != PKV_OK) return st;
  TreeParams p = {};
  p.out = out;
  p.q = q;
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
  p.group_shift = group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : 3;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.max_query_len = max_query_len;
  p.num_blocks = num_blocks;
  p.max_rts = max_rts;
  p.whole_units = whole;
  p.direct = whole && units == ctas;
  const bool many = units * 2 * kMergeSlices <= ctas;
  p.by_unit = many;
  p.num_ctas = ctas;
  p.out_aligned32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  p.err = dev_err;
  if (!whole) {
    // the pieces first, on a 32-byte boundary: at most 16 bytes in
    p.ws_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 31) &
                                      ~static_cast<uintptr_t>(31));
    p.ws_ml = reinterpret_cast<float2*>(p.ws_o + static_cast<size_t>(ctas) * 2 * e.rows * head_dim);
    p.ws_meta = reinterpret_cast<int4*>(p.ws_ml + static_cast<size_t>(ctas) * 2 * e.rows);
  }
  st = cuda_status(cudaFuncSetAttribute(e.fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(e.smem)));
  if (st != PKV_OK) return st;
  st = cuda_status(launch_after_previous_smem(e.fn, dim3(ctas), dim3(e.threads), e.smem, stream, p,
                                              kmap, vmap));
  if (st != PKV_OK || ctas == 1 || p.whole_units) return st;
  // Units in eight or more pieces on average are joined by slices of threads, from
  // entries by unit: one sequence of 32000 tokens takes 41.8 us so, 50.1 by one set
  // of threads and entries by CTA, which suit the batches in two or three pieces a
  // unit (GQA chat 72 against 76 us, 8 sequences of 1200 tokens 19.8 against 25.3).
  const int entries = p.by_unit ? static_cast<int>(units) : ctas;
  const int rows = kTreeMergeThreads / (head_dim / 4) / (many ? kMergeSlices : 1);
  // at most about as many blocks as are resident at once
  const dim3 merge(entries, std::min((std::min(max_rows, e.rows) + rows - 1) / rows,
                                     std::max(1, 2400 / entries)));
  return cuda_status(launch_after_previous(many ? e.merge_many : e.merge, merge,
                                           dim3(kTreeMergeThreads), stream, p));
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_paged_attn_tree_workspace_bytes(int num_seqs, int num_heads,
                                                      int num_kv_heads, int head_dim,
                                                      int max_context_len, int max_query_len) {
  using namespace pkv;
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      !head_dim_supported(head_dim) || max_context_len <= 0 || max_query_len <= 0 ||
      max_query_len > PKV_MAX_TREE_NODES || max_query_len > max_context_len)
    return 0;
  const int group = num_heads / num_kv_heads;
  if (group > 8) return 0;
  size_t most = 0;
  for (const bool fp8 : {false, true}) {
    const TreeEntry e = tree_entry(head_dim, PKV_FP16, fp8, num_seqs, num_kv_heads,
                                   max_query_len * group, max_context_len);
    const int ctas = tree_ctas(e.ctas, e.rows, num_seqs, group, num_kv_heads, max_context_len,
                               max_query_len);
    const long long rts = (max_query_len * group + e.rows - 1) / e.rows;
    most = std::max(most, tree_ws_bytes(ctas, e.rows, head_dim,
                                        tree_whole(num_seqs * rts * num_kv_heads,
                                                   max_context_len)));
  }
  return most;
}

extern "C" pkv_status pkv_paged_attn_tree(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
    const int32_t* parents, float scale, int num_seqs, int num_tokens, int num_heads,
    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int max_context_len,
    int max_query_len, int num_blocks, pkv_dtype dtype, void* workspace, size_t workspace_bytes,
    unsigned* dev_err, void* stream) {
  return pkv::tree_launch(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                          parents, scale, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                          block_size, max_blocks_per_seq, max_context_len, max_query_len,
                          num_blocks, dtype, false, nullptr, nullptr, workspace,
                          workspace_bytes, dev_err, stream);
}

extern "C" pkv_status pkv_paged_attn_tree_fp8(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
    const int32_t* parents, float scale, const float* k_scales, const float* v_scales,
    int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
    int max_blocks_per_seq, int max_context_len, int max_query_len, int num_blocks,
    pkv_dtype dtype, void* workspace, size_t workspace_bytes, unsigned* dev_err, void* stream) {
  return pkv::tree_launch(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                          parents, scale, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                          block_size, max_blocks_per_seq, max_context_len, max_query_len,
                          num_blocks, dtype, true, k_scales, v_scales, workspace,
                          workspace_bytes, dev_err, stream);
}

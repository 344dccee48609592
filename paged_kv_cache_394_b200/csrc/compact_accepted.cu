// compact_accepted.cu — moves the K and V of a drafted tree's accepted path to
// the front of the tree's cache positions.
//
// The path's nodes rise, so the d-th of them is at or behind position d, and
// every later source lies behind every earlier destination.  A thread moves
// one 16-byte chunk column (kv head, offset in the row, K or V) of a sequence
// through all its moves in that order, kBatch loads before their stores: a
// store can only hit sources that the same thread has already read, and no
// other thread touches the column.
//
// What bounds it: a serving batch's moves are read and written once (25 MB for 256
// paths of up to 8 nodes over 32 heads: 3.9 us at the copy rate), but they sit behind
// three loads in a row (lengths and path, table entries, rows), which small batches
// consist of.  So the path is loaded beside the lengths, before it is known how
// much of it counts.
#include "common.cuh"
#include "host_common.h"

namespace pkv {

struct CompactParams {
  uint4* k_cache;
  uint4* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const int32_t* accepted;
  const int32_t* num_accepted;
  int max_query_len, num_kv_heads, chunks_per_row, block_size, max_blocks_per_seq, num_blocks;
  unsigned* err;
};

// Grid (sequence, slice of the chunk columns, K or V).
__global__ void __launch_bounds__(256) compact_accepted_kernel(const CompactParams p) {
  __shared__ int64_t src_row[PKV_MAX_TREE_NODES], dst_row[PKV_MAX_TREE_NODES];
  __shared__ int bad;
  const int seq = blockIdx.x;
  grid_dependency_wait();
  trigger_dependents();
  const int32_t* path = p.accepted + static_cast<size_t>(seq) * p.max_query_len;
  int a = -1, before = -1;  // the path's node at this thread's depth, and the one before it
  if (static_cast<int>(threadIdx.x) < p.max_query_len) {
    a = path[threadIdx.x];
    if (threadIdx.x > 0) before = path[threadIdx.x - 1];
  }
  const bool first = blockIdx.y == 0 && blockIdx.z == 0;  // reports for its sequence
  const int ctx = p.context_lens[seq];
  const int q_len = p.query_start[seq + 1] - p.query_start[seq];
  const int n = p.num_accepted[seq];
  if (q_len < 0 || q_len > p.max_query_len || ctx < q_len ||
      ctx > static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size) {
    if (first && threadIdx.x == 0) set_err(p.err, PKV_DEVERR_BAD_CONTEXT);
    return;
  }
  if (n < 0 || n > q_len) {
    if (first && threadIdx.x == 0) set_err(p.err, PKV_DEVERR_BAD_TREE);
    return;
  }
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  const int32_t* table = p.block_tables + static_cast<size_t>(seq) * p.max_blocks_per_seq;
  const int hist = ctx - q_len;
  // at most PKV_MAX_TREE_NODES = blockDim.x nodes: one a thread
  const int d = threadIdx.x;
  if (d < n) {
    if (a < 0 || a >= q_len || (d > 0 && before >= a)) {
      bad = 1;
    } else {
      const int from = hist + a, to = hist + d;
      int64_t s = -1, t = -1;
      if (a != d) {
        const int bf = table[from / p.block_size], bt = table[to / p.block_size];
        if (static_cast<unsigned>(bf) < static_cast<unsigned>(p.num_blocks) &&
            static_cast<unsigned>(bt) < static_cast<unsigned>(p.num_blocks)) {
          s = static_cast<int64_t>(bf) * p.num_kv_heads * p.block_size + from % p.block_size;
          t = static_cast<int64_t>(bt) * p.num_kv_heads * p.block_size + to % p.block_size;
        } else if (first) {
          set_err(p.err, PKV_DEVERR_BAD_BLOCK);
        }
      }
      src_row[d] = s;
      dst_row[d] = t;
    }
  }
  __syncthreads();
  if (bad) {
    if (first && threadIdx.x == 0) set_err(p.err, PKV_DEVERR_BAD_TREE);
    return;
  }
  const int col = blockIdx.y * blockDim.x + threadIdx.x;
  if (col >= p.num_kv_heads * p.chunks_per_row) return;
  const int head = col / p.chunks_per_row, chunk = col % p.chunks_per_row;
  uint4* cache = blockIdx.z == 0 ? p.k_cache : p.v_cache;
  auto at = [&](int64_t row) {
    return (row + static_cast<int64_t>(head) * p.block_size) * p.chunks_per_row + chunk;
  };
  constexpr int kBatch = 8;
  for (int d0 = 0; d0 < n; d0 += kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (d0 + i < n && src_row[d0 + i] >= 0) v[i] = cache[at(src_row[d0 + i])];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (d0 + i < n && src_row[d0 + i] >= 0) cache[at(dst_row[d0 + i])] = v[i];
  }
}

}  // namespace pkv

extern "C" pkv_status pkv_compact_accepted(void* k_cache, void* v_cache,
                                           const int32_t* block_tables,
                                           const int32_t* context_lens,
                                           const int32_t* query_start, const int32_t* accepted,
                                           const int32_t* num_accepted, int num_seqs,
                                           int max_query_len, int num_kv_heads, int head_dim,
                                           int block_size, int max_blocks_per_seq,
                                           int num_blocks, pkv_dtype dtype, unsigned* dev_err,
                                           void* stream) {
  using namespace pkv;
  if (num_seqs < 0 || max_query_len < 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0 || !cache_dtype_valid(dtype))
    return PKV_ERR_INVALID_ARG;
  if (!head_dim_supported(head_dim) || !block_size_supported(block_size) ||
      max_query_len > PKV_MAX_TREE_NODES)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_query_len == 0) return PKV_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !query_start || !accepted ||
      !num_accepted)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(block_tables, context_lens, query_start, accepted, num_accepted, dev_err))
    return PKV_ERR_INVALID_ARG;
  const int chunks = head_dim * cache_elem_bytes(dtype) / 16;
  const int64_t slices = (static_cast<int64_t>(num_kv_heads) * chunks + 255) / 256;
  if (slices > 65535) return PKV_ERR_UNSUPPORTED;
  CompactParams p = {};
  p.k_cache = static_cast<uint4*>(k_cache);
  p.v_cache = static_cast<uint4*>(v_cache);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.accepted = accepted;
  p.num_accepted = num_accepted;
  p.max_query_len = max_query_len;
  p.num_kv_heads = num_kv_heads;
  p.chunks_per_row = chunks;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.err = dev_err;
  const dim3 grid(static_cast<unsigned>(num_seqs), static_cast<unsigned>(slices), 2);
  static_assert(PKV_MAX_TREE_NODES == 256, "a thread per node of a path");
  return cuda_status(
      launch_after_previous(compact_accepted_kernel, grid, dim3(256), stream, p));
}

// paged_attn_tree_kernels.cuh — attention of a tree of drafted tokens over the
// paged cache.
#pragma once

#include <math.h>

#include "common.cuh"

namespace pkv {

struct TreeParams {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const int32_t* parents;
  float qscale;  // scale * log2(e)
  const float* k_scales;  // E4M3 caches
  const float* v_scales;
  int num_seqs, num_tokens, num_heads, num_kv_heads;
  int block_size, max_blocks_per_seq, max_context_len, max_query_len, num_blocks;
  unsigned* err;
};

// Lanes' elements of one cached row: 2 or 4 dims a lane.
template <int D, class CT>
__device__ __forceinline__ void load_row(const void* cache, size_t row, int lane,
                                         float (&f)[D / 32]) {
  if constexpr (std::is_same<CT, Fp8E4M3>::value) {
    const uint8_t* p = static_cast<const uint8_t*>(cache) + row * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; i += 2) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          *reinterpret_cast<const __nv_fp8x2_storage_t*>(p + i), __NV_E4M3);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[i] = x.x;
      f[i + 1] = x.y;
    }
  } else {
    const typename CT::T* p = static_cast<const typename CT::T*>(cache) + row * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) f[i] = static_cast<float>(p[i]);
  }
}

// One warp per (node, head) row: an online softmax in base 2 over the history
// and then over the node's ancestors, found by following its parents.
template <int D, class DT, class CT>
__global__ void __launch_bounds__(128) paged_attn_tree_kernel(const TreeParams p) {
  using T = typename DT::T;
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int head = static_cast<int>(row % p.num_heads);
  const int64_t unit = row / p.num_heads;
  const int seq = static_cast<int>(unit / p.max_query_len);
  const int j = static_cast<int>(unit % p.max_query_len);
  if (seq >= p.num_seqs) return;
  const int ctx = p.context_lens[seq];
  const int q0 = p.query_start[seq];
  const int q_len = p.query_start[seq + 1] - q0;
  if (ctx < 0 || ctx > p.max_context_len || q_len < 0 || q_len > ctx || q_len > p.max_query_len ||
      q0 < 0 || q0 > p.num_tokens - q_len) {
    if (lane == 0 && j == 0 && head == 0) set_err(p.err, PKV_DEVERR_BAD_CONTEXT);
    return;
  }
  if (j >= q_len) return;
  const int kvh = head / (p.num_heads / p.num_kv_heads);
  float ks = 1.f, vs = 1.f;
  if constexpr (std::is_same<CT, Fp8E4M3>::value) {
    ks = p.k_scales[kvh];
    vs = p.v_scales[kvh];
    if (!(ks > 0.f && ks < INFINITY && vs > 0.f && vs < INFINITY) && lane == 0)
      set_err(p.err, PKV_DEVERR_BAD_SCALE);
  }
  const size_t at = (static_cast<size_t>(q0 + j) * p.num_heads + head) * D + lane * N;
  float q[N], acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = static_cast<float>(static_cast<const T*>(p.q)[at + i]);
    acc[i] = 0.f;
  }
  const int32_t* table = p.block_tables + static_cast<size_t>(seq) * p.max_blocks_per_seq;
  float m = -INFINITY, l = 0.f;
  auto take = [&](int pos) {
    const int block = table[pos / p.block_size];
    if (static_cast<unsigned>(block) >= static_cast<unsigned>(p.num_blocks)) {
      if (lane == 0) set_err(p.err, PKV_DEVERR_BAD_BLOCK);
      return;
    }
    const size_t r = (static_cast<size_t>(block) * p.num_kv_heads + kvh) * p.block_size +
                     pos % p.block_size;
    float k[N], v[N];
    load_row<D, CT>(p.k_cache, r, lane, k);
    load_row<D, CT>(p.v_cache, r, lane, v);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
    s *= p.qscale * ks;
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float w = exp2f(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = acc[i] * a + w * v[i];
  };
  const int hist = ctx - q_len;
  for (int k = 0; k < hist; ++k) take(k);
  for (int a = j; a >= 0;) {
    take(hist + a);
    const int up = p.parents[q0 + a];
    if (up < -1 || up >= a) {
      if (lane == 0) set_err(p.err, PKV_DEVERR_BAD_TREE);
      break;
    }
    a = up;
  }
  const float inv = vs / l;
#pragma unroll
  for (int i = 0; i < N; ++i)
    static_cast<T*>(p.out)[at + i] = static_cast<T>(l > 0.f || l != l ? acc[i] * inv : 0.f);
}

}  // namespace pkv

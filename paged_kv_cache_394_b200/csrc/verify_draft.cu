// verify_draft.cu — speculative sampling: which drafted tokens the target
// model accepts, and the token that follows them.
//
// Per sequence: a walk down the tree from gathered probabilities, and for each
// residual r = max(r / Z - q, 0) that a rejection leaves, and for the last
// distribution, one pass over a row of the target (and of the draft): its sum
// and then the first x whose running sum passes the drawn share.  What bounds it
// is reading those rows, vocab_size values each.
//
// A cluster of 1 to 8 CTAs serves a sequence.  Rank 0 gathers what the walk
// needs (each node's parent, token, uniform, and the two probabilities of its
// token at its parent) into every CTA's shared memory, so that all of them walk
// alike; each warp of the cluster has its own contiguous piece of the vocabulary.
// A pass leaves a sum per warp; the CTAs exchange theirs through distributed
// shared memory, and only the warp whose piece holds the next token reads that
// piece again.  All sums are 64-bit and in a fixed order.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "host_common.h"

namespace pkv {

namespace cg = cooperative_groups;

struct VerifyParams {
  int32_t* accepted;
  int32_t* num_accepted;
  int32_t* next_token;
  const void* target;
  const void* draft;  // null: the draft is certain of its tokens
  int64_t target_stride, draft_stride;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* query_start;
  const float* accept_u;
  const float* sample_u;
  int num_seqs, num_tokens, max_query_len, vocab;
  unsigned* err;
};

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;

// Values per 16-byte load.
template <class T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

template <class T>
__device__ __forceinline__ float weight_of(T x) {
  return fmaxf(static_cast<float>(x), 0.f);  // negative and NaN count as 0
}

// Group g of a row: values g * kVec - shift .. + kVec - 1, those outside [0, vocab) as 0.
template <class T>
__device__ __forceinline__ void load_group(const T* row, bool aligned, int x0, int vocab,
                                           float (&f)[kVec<T>]) {
  if (aligned && x0 >= 0 && x0 + kVec<T> <= vocab) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + x0));
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) f[e] = weight_of(t[e]);
  } else {
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
      f[e] = x0 + e >= 0 && x0 + e < vocab ? weight_of(row[x0 + e]) : 0.f;
  }
}

struct VerifyShared {
  int n;
  int parent[PKV_MAX_TREE_NODES], token[PKV_MAX_TREE_NODES];
  float u[PKV_MAX_TREE_NODES];
  float p[PKV_MAX_TREE_NODES], q[PKV_MAX_TREE_NODES];  // of the node's token, at its parent
  double z[PKV_MAX_TREE_NODES + 1];    // Z before each rejection at the current node
  int rejected[PKV_MAX_TREE_NODES];    // the tokens rejected there
  double warp_sum[kVerifyWarps];
  double cta_sum[2][kMaxCluster];      // by parity of the pass
  int cur, nrej, more;
};

// What is left of weight p after nrej rejections of draws from q.
__device__ __forceinline__ double residual(double p, float q, const double* z, int nrej) {
  double r = p;
  for (int k = 0; k < nrej && r > 0.0; ++k)
    r = fmax((k == 0 ? r : r / z[k]) - static_cast<double>(q), 0.0);  // z[0] = 1
  return r;
}

template <class T>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_draft_kernel(const VerifyParams p) {
  __shared__ VerifyShared sh;
  constexpr int V = kVec<T>;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int seq = blockIdx.x / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* acc = p.accepted + static_cast<size_t>(seq) * p.max_query_len;
  const bool certain = p.draft == nullptr;
  const T* target = static_cast<const T*>(p.target);
  const T* draft = static_cast<const T*>(p.draft);
  grid_dependency_wait();
  trigger_dependents();
  const int q0 = p.query_start[seq];  // rank 0's reading decides what is used of it
  if (rank == 0) {
    const int end = p.query_start[seq + 1];
    int n = end < q0 ? -1 : static_cast<int>(static_cast<unsigned>(end) - static_cast<unsigned>(q0));
    if (n < 0 || n > p.max_query_len || q0 < 0 || q0 > p.num_tokens - n) {
      if (tid == 0) set_err(p.err, PKV_DEVERR_BAD_CONTEXT);
      n = 0;
    }
    for (int j = tid; j < n; j += kVerifyThreads) {
      int up = p.parents[q0 + j];
      const int x = p.tokens[q0 + j];
      if (j == 0 ? up != -1 : up < -1 || up >= j) {
        set_err(p.err, PKV_DEVERR_BAD_TREE);
        up = -1;
      }
      float px = 0.f, qx = 0.f;
      if (up >= 0 && static_cast<unsigned>(x) < static_cast<unsigned>(p.vocab)) {
        px = weight_of(target[(q0 + up) * p.target_stride + x]);
        if (!certain) qx = weight_of(draft[(q0 + up) * p.draft_stride + x]);
      }
      const float u = p.accept_u[q0 + j];
      for (int c = 0; c < ranks; ++c) {
        VerifyShared* to = cluster.map_shared_rank(&sh, c);
        to->parent[j] = up;
        to->token[j] = x;
        to->u[j] = u;
        to->p[j] = px;
        to->q[j] = qx;
      }
    }
    if (tid < ranks) cluster.map_shared_rank(&sh, tid)->n = n;
  }
  cluster.sync();
  const int n = sh.n;
  if (n == 0) {
    if (rank == 0) {
      for (int j = tid; j < p.max_query_len; j += kVerifyThreads) acc[j] = -1;
      if (tid == 0) {
        p.num_accepted[seq] = 0;
        p.next_token[seq] = -1;
      }
    }
    return;
  }

  // This warp's piece of a row of node `cur`: 32 groups at a time, in the order of
  // the vocabulary.  f(x0, r) sees a lane's group and its residual weights, and
  // says whether to go on.
  const int gw = rank * kVerifyWarps + warp;
  auto scan = [&](int cur, int nrej, auto&& f) {
    const T* prow = target + (q0 + cur) * p.target_stride;
    const T* qrow = certain ? nullptr : draft + (q0 + cur) * p.draft_stride;
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(prow) / sizeof(T)) % V);
    const bool same =
        !certain && (reinterpret_cast<uintptr_t>(qrow) / sizeof(T)) % V == shift;
    const int groups = static_cast<int>((static_cast<unsigned>(p.vocab) + shift + V - 1) / V);
    const int chunks = (groups + 31) / 32;
    const int per = (chunks + ranks * kVerifyWarps - 1) / (ranks * kVerifyWarps);
    const int c0 = min(chunks, gw * per), c1 = min(chunks, c0 + per);
    const int lo = c0 * 32 * V - shift, hi = c1 * 32 * V - shift;  // this warp's values
    // certain draft: which of the first 32 x 8 rejected tokens lie in this piece
    unsigned hit[PKV_MAX_TREE_NODES / 32] = {};
    if (certain) {
#pragma unroll
      for (int b = 0; b < PKV_MAX_TREE_NODES / 32; ++b) {
        if (b * 32 >= nrej) break;
        const int x = b * 32 + lane < nrej ? sh.rejected[b * 32 + lane] : -1;
        hit[b] = __ballot_sync(kFullMask, x >= 0 && x >= lo && x < hi);
      }
    }
    const bool with_q = !certain && nrej > 0;
#pragma unroll 2
    for (int c = c0; c < c1; ++c) {
      const int x0 = (c * 32 + lane) * V - shift;
      float pf[V], qf[V] = {};
      load_group<T>(prow, true, x0, p.vocab, pf);
      if (with_q) load_group<T>(qrow, same, x0, p.vocab, qf);
      double r[V];
#pragma unroll
      for (int e = 0; e < V; ++e)
        r[e] = with_q ? residual(pf[e], qf[e], sh.z, nrej) : static_cast<double>(pf[e]);
      if (certain) {
#pragma unroll
        for (int b = 0; b < PKV_MAX_TREE_NODES / 32; ++b)
          for (unsigned m = hit[b]; m != 0; m &= m - 1) {
            const int x = sh.rejected[b * 32 + __ffs(m) - 1];
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (x0 + e == x) r[e] = 0.0;
          }
      }
      if (!f(x0, r)) break;
    }
  };
  int passes = 0;
  // The sum of node cur's residual weights, the same in every thread of the
  // cluster; sh.warp_sum and sh.cta_sum[...] hold its parts.
  auto pass = [&](int cur, int nrej) {
    double s = 0.0;
    scan(cur, nrej, [&](int, const double (&r)[V]) {
#pragma unroll
      for (int e = 0; e < V; ++e) s += r[e];
      return true;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
    if (lane == 0) sh.warp_sum[warp] = s;
    __syncthreads();
    const int par = passes++ & 1;
    if (tid < ranks) {
      double t = 0.0;
      for (int w = 0; w < kVerifyWarps; ++w) t += sh.warp_sum[w];
      cluster.map_shared_rank(&sh, tid)->cta_sum[par][rank] = t;
    }
    cluster.sync();
    double t = 0.0;
    for (int c = 0; c < ranks; ++c) t += sh.cta_sum[par][c];
    return t;
  };

  // ---- the walk: warp 0 of every CTA, until it needs a residual's sum ---------------
  int cur = 0, nrej = 0, next = 1, count = 1;
  if (tid == 0) {
    sh.z[0] = 1.0;
    if (rank == 0) acc[0] = 0;
  }
  double total = 0.0;
  bool summed = false;  // total is that of (cur, nrej)
  for (;;) {
    if (warp == 0) {
      __syncwarp();
      bool more = false;
      while (next < n) {
        const int j0 = next + lane;
        const unsigned m = __ballot_sync(kFullMask, j0 < n && sh.parent[j0] == cur);
        if (m == 0) {
          next += 32;
          continue;
        }
        const int j = next + __ffs(m) - 1;
        next = j + 1;
        const int x = sh.token[j];
        if (static_cast<unsigned>(x) >= static_cast<unsigned>(p.vocab)) {
          if (rank == 0 && lane == 0) set_err(p.err, PKV_DEVERR_BAD_DRAFT);
          continue;
        }
        double r = sh.p[j];
        if (certain) {
          bool before = false;
          for (int k = lane; k < nrej; k += 32) before |= sh.rejected[k] == x;
          if (__any_sync(kFullMask, before)) r = 0.0;
        } else {
          r = residual(r, sh.q[j], sh.z, nrej);
        }
        const double q = certain ? 1.0 : static_cast<double>(sh.q[j]);
        if (static_cast<double>(sh.u[j]) * q * sh.z[nrej] < r) {
          cur = j;
          nrej = 0;
          if (rank == 0 && lane == 0) acc[count] = j;
          ++count;
          summed = false;
        } else {
          const double left = sh.z[nrej] - r;
          __syncwarp();
          if (lane == 0) {
            sh.rejected[nrej] = x;
            if (certain) sh.z[nrej + 1] = left;
          }
          __syncwarp();
          ++nrej;
          summed = false;
          if (!certain) {
            more = true;
            break;
          }
        }
      }
      if (lane == 0) {
        sh.cur = cur;
        sh.nrej = nrej;
        // 1: sum and walk on; 0: the end, with the last sum still good; 2: the end
        sh.more = more ? 1 : summed ? 0 : 2;
      }
    }
    __syncthreads();
    const int what = sh.more;
    cur = sh.cur;
    nrej = sh.nrej;
    if (what != 0) total = pass(cur, nrej);
    if (what != 1) break;
    summed = true;
    if (tid == 0) sh.z[nrej] = total;
  }
  if (!(total > 0.0) && nrej > 0) {  // nothing left: the target's own weights again
    nrej = 0;
    total = pass(cur, 0);
  }
  // ---- the next token ------------------------------------------------------------------
  if (rank == 0) {
    if (warp == 0) count = __shfl_sync(kFullMask, count, 0);
    if (tid == 0) {
      sh.n = count;
      p.num_accepted[seq] = count;
    }
    __syncthreads();
    for (int j = sh.n + tid; j < p.max_query_len; j += kVerifyThreads) acc[j] = -1;
  }
  if (!(total > 0.0 && total < INFINITY)) {
    if (rank == 0 && tid == 0) {
      set_err(p.err, PKV_DEVERR_BAD_DRAFT);
      p.next_token[seq] = -1;
    }
    return;
  }
  const double want = static_cast<double>(p.sample_u[seq]) * total;
  const double* sums = sh.cta_sum[(passes - 1) & 1];
  // the CTA, then its warp, whose sums pass the share; the last with any weight
  // where rounding leaves none
  double base = 0.0, at = 0.0, fallback = 0.0;
  int owner = -1, last = 0;
  for (int c = 0; c < ranks && owner < 0; ++c) {
    if (sums[c] > 0.0) last = c, fallback = at;
    if (at + sums[c] > want) owner = c, base = at;
    at += sums[c];
  }
  if (owner < 0) owner = last, base = fallback;
  if (rank != owner) return;
  at = base;
  owner = -1;
  for (int w = 0; w < kVerifyWarps && owner < 0; ++w) {
    if (sh.warp_sum[w] > 0.0) last = w, fallback = at;
    if (at + sh.warp_sum[w] > want) owner = w, base = at;
    at += sh.warp_sum[w];
  }
  if (owner < 0) owner = last, base = fallback;
  if (warp != owner) return;
  int found = -1, positive = -1;
  scan(cur, nrej, [&](int x0, const double (&r)[V]) {
    double s = 0.0;
    int pos = -1;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s += r[e];
      if (r[e] > 0.0) pos = x0 + e;
    }
    double upto = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(kFullMask, upto, o);
      if (lane >= o) upto += y;
    }
    double c = base + (upto - s);
    int mine = -1;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      c += r[e];
      if (mine < 0 && r[e] > 0.0 && c > want) mine = x0 + e;
    }
    const unsigned m = __ballot_sync(kFullMask, mine >= 0);
    const unsigned any = __ballot_sync(kFullMask, pos >= 0);
    if (any != 0) positive = __shfl_sync(kFullMask, pos, 31 - __clz(any));
    if (m != 0) {
      found = __shfl_sync(kFullMask, mine, __ffs(m) - 1);
      return false;
    }
    base += __shfl_sync(kFullMask, upto, 31);
    return true;
  });
  if (lane == 0) p.next_token[seq] = found >= 0 ? found : positive;
}

}  // namespace pkv

extern "C" pkv_status pkv_verify_draft(
    int32_t* accepted, int32_t* num_accepted, int32_t* next_token, const void* target_probs,
    int64_t target_stride, const void* draft_probs, int64_t draft_stride,
    const int32_t* draft_tokens, const int32_t* parents, const int32_t* query_start,
    const float* accept_uniforms, const float* sample_uniforms, int num_seqs, int num_tokens,
    int max_query_len, int vocab_size, pkv_dtype dtype, unsigned* dev_err, void* stream) {
  using namespace pkv;
  const bool f32 = dtype == PKV_FP32;
  if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || vocab_size <= 0 ||
      (!f32 && !dtype_valid(dtype)) || target_stride < vocab_size ||
      (draft_probs != nullptr && draft_stride < vocab_size))
    return PKV_ERR_INVALID_ARG;
  if (max_query_len > PKV_MAX_TREE_NODES || vocab_size > (1 << 30)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!num_accepted || !next_token || !query_start || (max_query_len > 0 && !accepted) ||
      (num_tokens > 0 && (!target_probs || !draft_tokens || !parents || !accept_uniforms)) ||
      !sample_uniforms)
    return PKV_ERR_INVALID_ARG;
  const uintptr_t mask = f32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(target_probs) & mask) ||
      (reinterpret_cast<uintptr_t>(draft_probs) & mask))
    return PKV_ERR_INVALID_ARG;
  VerifyParams p = {};
  p.accepted = accepted;
  p.num_accepted = num_accepted;
  p.next_token = next_token;
  p.target = target_probs;
  p.draft = draft_probs;
  p.target_stride = target_stride;
  p.draft_stride = draft_stride;
  p.tokens = draft_tokens;
  p.parents = parents;
  p.query_start = query_start;
  p.accept_u = accept_uniforms;
  p.sample_u = sample_uniforms;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.max_query_len = max_query_len;
  p.vocab = vocab_size;
  p.err = dev_err;
  auto fn = f32                   ? verify_draft_kernel<float>
            : dtype == PKV_FP16 ? verify_draft_kernel<__half>
                                : verify_draft_kernel<__nv_bfloat16>;
  // As many CTAs a sequence as keep two of them on each of 148 SMs.
  int ranks = kMaxCluster;
  while (ranks > 1 && static_cast<long long>(num_seqs) * ranks > 2 * 148) ranks /= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_seqs) * static_cast<unsigned>(ranks));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = as_stream(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, fn, p));
}

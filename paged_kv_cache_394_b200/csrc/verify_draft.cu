// verify_draft.cu — speculative sampling: which drafted tokens the target
// model accepts, and the token that follows them.
//
// Per sequence: a walk down the tree from gathered probabilities, and for each
// residual that a rejection leaves, and for the last distribution, one pass over
// a row of the target (and of the draft): its sum, and then the first x whose
// running sum passes the drawn share.  What bounds it is reading those rows,
// vocab_size values each.
//
// The residual after k rejections, r_k = max(r_(k-1) / Z_(k-1) - q, 0) with
// Z_k = sum r_k, Z_0 = 1, needs no division and no memory of the steps: with
// c_k = Z_0 ... Z_(k-1), r_k c_k = max(p - (c_1 + ... + c_k) q, 0), as clipping at 0
// between subtractions changes nothing.  So with S_0 = 1 and A_0 = 0
//   A_k = A_(k-1) + S_(k-1),  s_k = max(p - A_k q, 0),  S_k = sum s_k  (= c_(k+1)),
// the next token is drawn from s_k, and u q Z_k < r_k is u q S_k < s_k.
//
// A cluster of 1 to 8 CTAs serves a sequence.  Rank 0 gathers what the walk
// needs (each node's parent, token, uniform, and the two probabilities of its
// token at its parent) into every CTA's shared memory, once all CTAs are known to
// have started (a cluster barrier entered first thing and waited for under those
// loads), so that all of them walk alike; each warp of the cluster has its own
// contiguous piece of the vocabulary.
// A pass leaves a sum per warp; the CTAs exchange theirs through distributed
// shared memory, and only the piece that holds the next token is read again: all
// warps of its CTA sum a share of it, and one scans the share that holds the token.
// All sums are 64-bit and in a fixed order.
#include <cooperative_groups.h>
#include <math.h>

#include <type_traits>

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
  double taken;                        // A of the rejections at the current node
  int rejected[PKV_MAX_TREE_NODES];    // the tokens rejected there
  double warp_sum[kVerifyWarps];
  double cta_sum[2][kMaxCluster];      // by parity of the pass
  int cur, nrej, more;
};

// What is left of weight p of a token that the draft weighs q: max(p - A q, 0).
__device__ __forceinline__ double residual(float p, float q, double taken) {
  return fmax(fma(-taken, static_cast<double>(q), static_cast<double>(p)), 0.0);
}

// The two halves of a cluster barrier that says only that every CTA runs (nothing
// has been written yet, so the arrival orders no memory).  Whole warps call them.
__device__ __forceinline__ void cluster_arrive_started() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_started() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
  // Shared memory of another CTA may be written once that CTA has started: each
  // arrives here, and all wait before rank 0's first remote store.
  if (ranks > 1) cluster_arrive_started();
  grid_dependency_wait();
  trigger_dependents();
  const int q0 = p.query_start[seq];  // rank 0's reading decides what is used of it
  int nodes = 0, up = -1, token = 0;  // rank 0: of the tree; node tid's parent and token
  float px = 0.f, qx = 0.f, u = 0.f;
  static_assert(PKV_MAX_TREE_NODES <= kVerifyThreads, "a thread per node");
  if (rank == 0) {
    const int end = p.query_start[seq + 1];
    nodes = end < q0 ? -1 : static_cast<int>(static_cast<unsigned>(end) - static_cast<unsigned>(q0));
    if (nodes < 0 || nodes > p.max_query_len || q0 < 0 || q0 > p.num_tokens - nodes) {
      if (tid == 0) set_err(p.err, PKV_DEVERR_BAD_CONTEXT);
      nodes = 0;
    }
    if (tid < nodes) {
      up = p.parents[q0 + tid];
      token = p.tokens[q0 + tid];
      if (tid == 0 ? up != -1 : up < -1 || up >= tid) {
        set_err(p.err, PKV_DEVERR_BAD_TREE);
        up = -1;
      }
      if (up >= 0 && static_cast<unsigned>(token) < static_cast<unsigned>(p.vocab)) {
        px = weight_of(target[(q0 + up) * p.target_stride + token]);
        if (!certain) qx = weight_of(draft[(q0 + up) * p.draft_stride + token]);
      }
      u = p.accept_u[q0 + tid];
    }
  }
  if (ranks > 1) {
    __syncwarp();
    cluster_wait_started();
  }
  if (rank == 0) {
    for (int c = 0; c < ranks && tid < nodes; ++c) {
      VerifyShared* to = cluster.map_shared_rank(&sh, c);
      to->parent[tid] = up;
      to->token[tid] = token;
      to->u[tid] = u;
      to->p[tid] = px;
      to->q[tid] = qx;
    }
    if (tid < ranks) cluster.map_shared_rank(&sh, tid)->n = nodes;
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

  // Warp gw's piece of the row of node `cur`: chunks c0 .. c1 - 1 of 32 groups, in
  // the order of the vocabulary; f0 .. f1 - 1 of them lie wholly within the row.
  struct Piece {
    const T *p, *q;
    int shift, c0, c1, f0, f1;
    bool same;                              // q's groups are aligned as p's
    unsigned hit[PKV_MAX_TREE_NODES / 32];  // certain draft: which rejected tokens lie in it
    unsigned hits;
  };
  auto piece_of = [&](int cur, int nrej, int gw) {
    Piece x;
    x.p = target + (q0 + cur) * p.target_stride;
    x.q = certain ? nullptr : draft + (q0 + cur) * p.draft_stride;
    x.shift = static_cast<int>((reinterpret_cast<uintptr_t>(x.p) / sizeof(T)) % V);
    x.same = certain || nrej == 0 ||
             static_cast<int>((reinterpret_cast<uintptr_t>(x.q) / sizeof(T)) % V) == x.shift;
    const int chunks = (p.vocab + x.shift + 32 * V - 1) / (32 * V);
    const int per = (chunks + ranks * kVerifyWarps - 1) / (ranks * kVerifyWarps);
    x.c0 = min(chunks, gw * per);
    x.c1 = min(chunks, x.c0 + per);
    x.f0 = max(x.c0, x.shift > 0 ? 1 : 0);
    x.f1 = x.same ? min(x.c1, (p.vocab + x.shift) / (32 * V)) : x.f0;
    const int lo = x.c0 * 32 * V - x.shift, hi = x.c1 * 32 * V - x.shift;
    x.hits = 0;
#pragma unroll
    for (int b = 0; b < PKV_MAX_TREE_NODES / 32; ++b) {
      x.hit[b] = 0;
      if (certain && b * 32 < nrej) {
        const int t = b * 32 + lane < nrej ? sh.rejected[b * 32 + lane] : -1;
        x.hit[b] = __ballot_sync(kFullMask, t >= 0 && t >= lo && t < hi);
        x.hits |= x.hit[b];
      }
    }
    return x;
  };
  // A lane's residual weights of chunk c, any chunk.
  auto chunk_weights = [&](const Piece& x, int c, double taken, double (&r)[V]) {
    const int x0 = (c * 32 + lane) * V - x.shift;
    float pf[V], qf[V] = {};
    load_group<T>(x.p, true, x0, p.vocab, pf);
    if (taken > 0.0) load_group<T>(x.q, x.same, x0, p.vocab, qf);
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = residual(pf[e], qf[e], taken);
    if (x.hits != 0) {
#pragma unroll
      for (int b = 0; b < PKV_MAX_TREE_NODES / 32; ++b)
        for (unsigned m = x.hit[b]; m != 0; m &= m - 1) {
          const int t = sh.rejected[b * 32 + __ffs(m) - 1];
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (x0 + e == t) r[e] = 0.0;
        }
    }
    return x0;
  };
  int passes = 0;
  // The sum of node cur's residual weights, the same in every thread of the
  // cluster; sh.warp_sum and sh.cta_sum[...] hold its parts.
  auto pass = [&](int cur, int nrej, double taken) {
    const Piece x = piece_of(cur, nrej, rank * kVerifyWarps + warp);
    double s = 0.0;
    int c = x.c0;
    if (x.hits == 0) {
      auto edge = [&](int to) {
        for (; c < to; ++c) {
          double r[V];
          chunk_weights(x, c, taken, r);
#pragma unroll
          for (int e = 0; e < V; ++e) s += r[e];
        }
      };
      edge(min(x.f0, x.c1));
      // whole chunks, kBatch loads of each row under way at once
      constexpr int kBatch = 16 / V;
      auto whole = [&](auto with_q, auto add) {
        for (; c < x.f1; c += kBatch) {
          uint4 pu[kBatch], qu[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            pu[b] = qu[b] = make_uint4(0u, 0u, 0u, 0u);
            if (c + b < x.f1) {
              const int64_t at = static_cast<int64_t>((c + b) * 32 + lane) * V - x.shift;
              pu[b] = __ldg(reinterpret_cast<const uint4*>(x.p + at));
              if constexpr (decltype(with_q)::value) qu[b] = __ldg(reinterpret_cast<const uint4*>(x.q + at));
            }
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const T* pt = reinterpret_cast<const T*>(&pu[b]);
            const T* qt = reinterpret_cast<const T*>(&qu[b]);
#pragma unroll
            for (int e = 0; e < V; ++e) add(weight_of(pt[e]), weight_of(qt[e]));
          }
        }
        c = x.f1;
      };
      if (c < x.f1) {
        if (taken == 0.0) {
          whole(std::false_type(), [&](float a, float) { s += static_cast<double>(a); });
        } else if (taken == 1.0) {  // a node's first rejection: no product
          whole(std::true_type(), [&](float a, float b) {
            const double d = static_cast<double>(a) - static_cast<double>(b);
            if (d > 0.0) s += d;
          });
        } else {
          whole(std::true_type(), [&](float a, float b) { s += residual(a, b, taken); });
        }
      }
      edge(x.c1);
    } else {
      for (; c < x.c1; ++c) {
        double r[V];
        chunk_weights(x, c, taken, r);
#pragma unroll
        for (int e = 0; e < V; ++e) s += r[e];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
    if (lane == 0) sh.warp_sum[warp] = s;
    __syncthreads();
    const int par = passes++ & 1;
    if (warp == 0) {
      double t = lane < kVerifyWarps ? sh.warp_sum[lane] : 0.0;
#pragma unroll
      for (int o = kVerifyWarps / 2; o > 0; o >>= 1) t += __shfl_xor_sync(kFullMask, t, o);
      if (lane < ranks) cluster.map_shared_rank(&sh, lane)->cta_sum[par][rank] = t;
    }
    if (ranks > 1)
      cluster.sync();
    else
      __syncthreads();
    double t = 0.0;
    for (int k = 0; k < ranks; ++k) t += sh.cta_sum[par][k];
    return t;
  };

  // ---- the walk: warp 0 of every CTA, until it needs a residual's sum ---------------
  int cur = 0, nrej = 0, next = 1, count = 1;
  double taken = 0.0, left = 1.0;  // A and S (a certain draft: A stays 0)
  if (rank == 0 && tid == 0) acc[0] = 0;
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
        double r, q = 1.0;
        if (certain) {
          bool before = false;
          for (int k = lane; k < nrej; k += 32) before |= sh.rejected[k] == x;
          r = __any_sync(kFullMask, before) ? 0.0 : static_cast<double>(sh.p[j]);
        } else {
          q = static_cast<double>(sh.q[j]);
          r = residual(sh.p[j], sh.q[j], taken);
        }
        summed = false;
        if (static_cast<double>(sh.u[j]) * q * left < r) {
          cur = j;
          nrej = 0;
          taken = 0.0;
          left = 1.0;
          if (rank == 0 && lane == 0) acc[count] = j;
          ++count;
        } else if (certain) {
          __syncwarp();
          if (lane == 0) sh.rejected[nrej] = x;
          __syncwarp();
          ++nrej;
          left -= r;
        } else {
          ++nrej;
          taken += left;
          more = true;
          break;
        }
      }
      if (lane == 0) {
        sh.cur = cur;
        sh.nrej = nrej;
        sh.taken = taken;
        // 1: sum and walk on; 0: the end, with the last sum still good; 2: the end
        sh.more = more ? 1 : summed ? 0 : 2;
      }
    }
    __syncthreads();
    const int what = sh.more;
    cur = sh.cur;
    nrej = sh.nrej;
    taken = sh.taken;
    if (what != 0) total = pass(cur, nrej, taken);
    if (what != 1) break;
    summed = true;
    left = total;
  }
  if (!(total > 0.0) && nrej > 0) {  // nothing left: the target's own weights again
    nrej = 0;
    taken = 0.0;
    total = pass(cur, 0, 0.0);
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
  // all warps of the CTA sum a part of that warp's piece; the part that passes
  // the share is scanned
  Piece x = piece_of(cur, nrej, rank * kVerifyWarps + owner);
  const int share = (x.c1 - x.c0 + kVerifyWarps - 1) / kVerifyWarps;
  const int first = min(x.c1, x.c0 + warp * share);
  x.c1 = min(x.c1, first + share);
  x.c0 = first;
  double part = 0.0;
  for (int c = x.c0; c < x.c1; ++c) {
    double r[V];
    chunk_weights(x, c, taken, r);
#pragma unroll
    for (int e = 0; e < V; ++e) part += r[e];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kFullMask, part, o);
  __syncthreads();  // everyone has chosen by the sums of the pass
  if (lane == 0) sh.warp_sum[warp] = part;
  __syncthreads();
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
  for (int c = x.c0; c < x.c1; ++c) {
    double r[V];
    const int x0 = chunk_weights(x, c, taken, r);
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
    const unsigned any = __ballot_sync(kFullMask, pos >= 0);
    if (any != 0) positive = __shfl_sync(kFullMask, pos, 31 - __clz(any));
    if (__any_sync(kFullMask, base + upto > want)) {
      double sum = base + (upto - s);
      int mine = -1;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sum += r[e];
        if (mine < 0 && r[e] > 0.0 && sum > want) mine = x0 + e;
      }
      const unsigned m = __ballot_sync(kFullMask, mine >= 0);
      if (m != 0) {
        found = __shfl_sync(kFullMask, mine, __ffs(m) - 1);
        break;
      }
    }
    base += __shfl_sync(kFullMask, upto, 31);
  }
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
  if (!aligned4(accepted, num_accepted, next_token, draft_tokens, parents, query_start,
                accept_uniforms, sample_uniforms, dev_err))
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
  // As many CTAs a sequence as keep two of them on each of 148 SMs, with 2048
  // values each at least (33 chains over 4730 values: 14.1 us in clusters of 8, 9.9
  // of 2; of 8192 at least: 16 trees over 50001 values 20 -> 25 us).
  constexpr int kLeast = 2048;
  int ranks = kMaxCluster;
  while (ranks > 1 && (static_cast<long long>(num_seqs) * ranks > 2 * 148 ||
                       vocab_size < ranks * kLeast))
    ranks /= 2;
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

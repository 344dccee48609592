// verify_draft.cu — speculative sampling: which drafted tokens the target
// model accepts, and the token that follows them.
#include <math.h>

#include "common.cuh"
#include "host_common.h"

namespace pkv {

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

template <class T>
__device__ __forceinline__ double prob(const void* base, int64_t i) {
  return static_cast<double>(fmaxf(static_cast<float>(static_cast<const T*>(base)[i]), 0.f));
}

constexpr int kVerifyThreads = 256;

// One CTA per sequence.  The walk over the nodes is one thread's; what needs a
// whole row (a residual's sum, the next token) is everyone's.  `zs` holds the
// sums Z of the current node's rejections so far, which define its residual.
template <class T>
__global__ void __launch_bounds__(kVerifyThreads) verify_draft_kernel(const VerifyParams p) {
  __shared__ double zs[PKV_MAX_TREE_NODES + 1];
  __shared__ double part[kVerifyThreads];
  __shared__ int s_rejected[PKV_MAX_TREE_NODES];  // certain draft: the tokens rejected at cur
  __shared__ int s_nrej, s_cur, s_j, s_need_sum, s_count;
  const int seq = blockIdx.x, tid = threadIdx.x;
  int32_t* acc = p.accepted + static_cast<size_t>(seq) * p.max_query_len;
  const int q0 = p.query_start[seq];
  int n = p.query_start[seq + 1] - q0;
  if (n < 0 || n > p.max_query_len || q0 < 0 || q0 > p.num_tokens - n) {
    if (tid == 0) set_err(p.err, PKV_DEVERR_BAD_CONTEXT);
    n = 0;
  }
  if (n == 0) {
    for (int j = tid; j < p.max_query_len; j += kVerifyThreads) acc[j] = -1;
    if (tid == 0) {
      p.num_accepted[seq] = 0;
      p.next_token[seq] = -1;
    }
    return;
  }
  if (tid == 0) {
    s_cur = 0;
    s_nrej = 0;
    s_j = 1;
    s_count = 1;
    zs[0] = 1.0;
    acc[0] = 0;
    if (p.parents[q0] != -1) set_err(p.err, PKV_DEVERR_BAD_TREE);
  }
  __syncthreads();
  // r(x) at the current node after its nrej rejections
  auto weight = [&](int cur, int nrej, int x) {
    double r = prob<T>(p.target, (q0 + cur) * p.target_stride + x);
    if (p.draft != nullptr) {
      if (nrej > 0) {
        const double q = prob<T>(p.draft, (q0 + cur) * p.draft_stride + x);
        for (int k = 0; k < nrej; ++k) r = fmax(r / zs[k] - q, 0.0);
      }
    } else {
      for (int k = 0; k < nrej; ++k)
        if (s_rejected[k] == x) r = 0.0;
    }
    return r;
  };
  auto row_sum = [&](int cur, int nrej) {
    double s = 0.0;
    for (int x = tid; x < p.vocab; x += kVerifyThreads) s += weight(cur, nrej, x);
    part[tid] = s;
    __syncthreads();
    for (int h = kVerifyThreads / 2; h > 0; h /= 2) {
      if (tid < h) part[tid] += part[tid + h];
      __syncthreads();
    }
    const double total = part[0];
    __syncthreads();
    return total;
  };
  for (;;) {
    if (tid == 0) {
      s_need_sum = 0;
      int j = s_j;
      for (; j < n; ++j) {
        const int up = p.parents[q0 + j];
        if (up < -1 || up >= j) {
          set_err(p.err, PKV_DEVERR_BAD_TREE);
          continue;
        }
        if (up != s_cur) continue;
        const int x = p.tokens[q0 + j];
        if (static_cast<unsigned>(x) >= static_cast<unsigned>(p.vocab)) {
          set_err(p.err, PKV_DEVERR_BAD_DRAFT);
          continue;
        }
        const double q =
            p.draft ? prob<T>(p.draft, (q0 + s_cur) * p.draft_stride + x) : 1.0;
        const double r = weight(s_cur, s_nrej, x);
        if (static_cast<double>(p.accept_u[q0 + j]) * q * zs[s_nrej] < r) {
          s_cur = j;
          s_nrej = 0;
          acc[s_count++] = j;
        } else {
          s_rejected[s_nrej++] = x;
          if (p.draft == nullptr) {
            zs[s_nrej] = zs[s_nrej - 1] - r;
          } else {
            s_need_sum = 1;
            ++j;
            break;
          }
        }
      }
      s_j = j;
    }
    __syncthreads();
    if (!s_need_sum) break;
    const double z = row_sum(s_cur, s_nrej);
    if (tid == 0) zs[s_nrej] = z;
    __syncthreads();
  }
  for (int j = s_count + tid; j < p.max_query_len; j += kVerifyThreads) acc[j] = -1;
  const int cur = s_cur;
  int nrej = s_nrej;
  double total = row_sum(cur, nrej);
  if (!(total > 0.0) && nrej > 0) {
    nrej = 0;
    total = row_sum(cur, 0);
  }
  if (tid == 0) {
    p.num_accepted[seq] = s_count;
    int next = -1;
    if (total > 0.0 && total < INFINITY) {
      const double want = static_cast<double>(p.sample_u[seq]) * total;
      double c = 0.0;
      for (int x = 0; x < p.vocab; ++x) {
        const double r = weight(cur, nrej, x);
        c += r;
        if (r > 0.0) next = x;
        if (c > want) break;
      }
    } else {
      set_err(p.err, PKV_DEVERR_BAD_DRAFT);
    }
    p.next_token[seq] = next;
  }
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
  if (max_query_len > PKV_MAX_TREE_NODES) return PKV_ERR_UNSUPPORTED;
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
  fn<<<static_cast<unsigned>(num_seqs), kVerifyThreads, 0, as_stream(stream)>>>(p);
  return cuda_status(cudaGetLastError());
}

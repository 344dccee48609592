// paged_attn_tree_kernels.cuh — attention of a tree of drafted tokens over the
// paged cache, on the 5th-generation tensor cores (tcgen05 + TMEM).
//
// Node j of a tree sees its sequence's history (the h = context - q_len tokens
// before the tree) and the nodes on its path up to the history:
//   out = softmax(scale q . K[visible]^T) . V[visible].
// A row is a (node, query head of the kv head) pair, q_len x group of them per
// (sequence, kv head); a unit is up to ROWS = 128 QT of those rows over all the
// sequence's keys in tiles of 64.
//
// What bounds it: K and V are read once per unit, 4 D bytes a key (2 D over
// E4M3), against 4 D multiply-adds per key and row.  At 128 rows the MMAs of a
// 64-key tile take about half the time that HBM needs to bring it to one of 148
// SMs, so up to 128 rows a unit is bound by memory and QT = 1 (one 128-row query
// tile) runs two CTAs an SM, one's softmax under the other's loads.  More rows
// take QT = 2: two query tiles share each K/V tile, one CTA an SM, bound by
// softmax and MMA.
//
// Split: the tiles of all units lie on one line, every sequence's units one
// after the other, and CTA c takes the c-th of gridDim.x equal stretches of it,
// whatever the lengths.  (A unit counts kTreeUnitCost tiles more than it has,
// for its query tile, pipeline fill and output.)  A unit that lies in one
// stretch is written out directly; pieces of a cut unit go to the workspace as
// (max, sum, unnormalised o) and paged_attn_tree_merge_kernel joins them.
//
// A CTA: warp 0 / 2 bring K / V tiles by TMA through the block table into a
// ring of NS stages; warp 1 issues S = Q K^T into one of two TMEM buffers; warp
// 3 issues O += P V with P read from TMEM; 4 softmax warps per query tile, a
// thread per row (online softmax in base 2 in fp32; the reference maximum moves
// only when a logit passes it by 2^8, so O is rarely rescaled).  P is rounded to
// fp16, or split into two bf16 halves for bf16 caches (2^-17 of p), so that it
// costs no accuracy next to the output's rounding.  E4M3 caches: further warps
// widen each tile's codes to fp16 (exact) into the stage that the MMAs read.
//
// The tree's part of the keys: each row's visible nodes are a bit set, made once
// per unit by following the parents.  What a row does not see must not enter
// it, and 0 x NaN would: K is masked in S, and non-finite elements of the
// tree's V are taken out of the tile (and added to the rows that do see them
// when the output is written).  Rows of V past the context are zeroed.
//
// Every wait is bounded; a role that gives up reports PKV_DEVERR_TIMEOUT, and
// TMEM is freed on every path.
#pragma once

#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "paged_prefill_tc_kernels.cuh"

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
  int num_seqs, num_tokens, num_heads, num_kv_heads, group_shift;
  int block_size, max_blocks_per_seq, max_context_len, max_query_len, num_blocks;
  unsigned* err;
  // Workspace: for each CTA one merge entry {first token, kv head, first CTA,
  // rows} (rows = 0: nothing to merge) and two pieces of ROWS rows.
  int4* ws_meta;
  float2* ws_ml;  // (max, sum) of each row of each piece
  float* ws_o;    // [pieces][D / 4][ROWS][4]
};

// What a unit costs beside its tiles, in tiles.  Measured on B200 (us; 2 / 4 / 6 /
// 9): GQA chat batch 86 / 71 / 69 / 70, its E4M3 form 107 / 98 / 89 / 88, the
// LLaMA-7B batch 112 / 111 / 111 / 112.
constexpr int kTreeUnitCost = 6;
constexpr int kTreeMinTiles = 2;  // the shortest stretch worth a CTA
constexpr int kTreeKeys = 64;     // keys per tile

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The lengths of a sequence.
struct TreeSeq {
  int ctx, q0, q_len;
};
struct TreeLens {
  int ctx, q0, end;
};
__device__ __forceinline__ TreeLens tree_lens(const TreeParams& p, int seq) {
  return {p.context_lens[seq], p.query_start[seq], p.query_start[seq + 1]};
}
// False if the sequence has nothing to do.
__device__ __forceinline__ bool tree_seq(const TreeParams& p, const TreeLens& x, TreeSeq& s,
                                         bool report) {
  s.ctx = x.ctx;
  s.q0 = x.q0;
  s.q_len = static_cast<int>(static_cast<unsigned>(x.end) - static_cast<unsigned>(x.q0));
  if (s.ctx < 0 || s.ctx > p.max_context_len || x.end < s.q0 || s.q_len < 0 || s.q_len > s.ctx ||
      s.q_len > p.max_query_len || s.q0 < 0 || s.q0 > p.num_tokens - s.q_len) {
    if (report) set_err(p.err, PKV_DEVERR_BAD_CONTEXT);
    return false;
  }
  return s.q_len > 0;
}

// A CTA's next piece of work: tiles t0 .. t1 - 1 of the nt of a unit.
struct TreeItem {
  int seq, ctx, q0, q_len, kvh, rt, t0, t1, nt;
};

// Walks a CTA's stretch.  Every role walks on its own.  The lengths of the
// sequence after the one at hand are loaded ahead of their use.
template <int ROWS>
struct TreeWalk {
  int seq, unit, at;  // the next sequence, unit of it, and position in the unit
  int left;           // positions left in the stretch
  bool loaded;
  TreeSeq s;
  TreeLens ahead;  // of sequence `seq`, until loaded; then of seq + 1

  __device__ __forceinline__ bool next(const TreeParams& p, TreeItem& it) {
    while (left > 0) {
      if (!loaded) {
        if (seq >= p.num_seqs) return false;
        loaded = tree_seq(p, ahead, s, false);
        if (seq + 1 < p.num_seqs) ahead = tree_lens(p, seq + 1);
        if (!loaded) {
          ++seq;
          continue;
        }
      }
      const int nt = (s.ctx + kTreeKeys - 1) / kTreeKeys;
      const int rts = ((s.q_len << p.group_shift) + ROWS - 1) / ROWS;
      const int span = nt + kTreeUnitCost;
      const int take = min(left, span - at);
      it.seq = seq;
      it.ctx = s.ctx;
      it.q0 = s.q0;
      it.q_len = s.q_len;
      it.kvh = rts == 1 ? unit : unit / rts;
      it.rt = unit - it.kvh * rts;
      it.t0 = max(0, at - kTreeUnitCost);
      it.t1 = max(0, at + take - kTreeUnitCost);
      it.nt = nt;
      left -= take;
      at += take;
      if (at == span) {
        at = 0;
        if (++unit == rts * p.num_kv_heads) {
          unit = 0;
          ++seq;
          loaded = false;
        }
      }
      if (it.t1 > it.t0) return true;
    }
    return false;
  }
};

template <int D_, class DT_, bool FP8_, int QT_>
struct TreeTraits {
  static constexpr int D = D_, QT = QT_, M = 128, ROWS = QT * M, NKEY = kTreeKeys;
  static constexpr bool kFp8 = FP8_;
  using DT = DT_;
  using T = typename DT::T;
  using MT = std::conditional_t<kFp8, Fp16, DT>;  // type of the MMAs and of P
  static constexpr bool kBf16 = std::is_same<MT, Bf16>::value;
  static constexpr bool kQToFp16 = kFp8 && std::is_same<DT, Bf16>::value;
  static constexpr int PIECES = NKEY / 16, HALVES = D / 64;
  // K/V stages, E4M3 staging slots and CTAs an SM: what fits beside the query
  // tiles in 227 KB.  E4M3 tiles are held twice, so one CTA an SM.
  static constexpr int MIN_BLOCKS = QT == 1 && !kFp8 ? 2 : 1;
  static constexpr int NS = kFp8 ? (QT == 1 ? 3 : 2) : QT == 1 ? (D == 128 ? 2 : 4) : 4;
  static constexpr int NSTG = kFp8 ? 4 : 0;
  static constexpr int NWIDEN = kFp8 ? (QT == 1 ? 4 : 2) : 1;  // widening warps for each of K, V
  static constexpr int SOFTMAX_WARP = 4;
  static constexpr int WIDEN_WARP = SOFTMAX_WARP + 4 * QT;
  static constexpr int THREADS = (WIDEN_WARP + (kFp8 ? 2 * NWIDEN : 0)) * 32;
  static constexpr int Q_HALF = M * 128;
  static constexpr int Q_TILE = HALVES * Q_HALF;
  static constexpr int KV_HALF = NKEY * 128;
  static constexpr int KV_TILE = HALVES * KV_HALF;
  static constexpr int STAGE = 2 * KV_TILE;
  static constexpr int STG_TILE = NKEY * D;
  static constexpr int OFF_KV = QT * Q_TILE;
  static constexpr int OFF_STG = OFF_KV + NS * STAGE;
  static constexpr int OFF_SEEN = OFF_STG + 2 * NSTG * STG_TILE;    // [ROWS][8] visible nodes
  static constexpr int OFF_PAR = OFF_SEEN + ROWS * 32;              // [QT][2][256] parents
  static constexpr int OFF_BAR = OFF_PAR + QT * 2 * PKV_MAX_TREE_NODES * 4;
  static constexpr int B_KFULL = 0, B_KEMPTY = NS, B_VFULL = 2 * NS, B_VEMPTY = 3 * NS;
  static constexpr int B_STG = 4 * NS, B_STGEMPTY = B_STG + 2 * NSTG;
  static constexpr int B_Q = B_STGEMPTY + 2 * NSTG;  // per query tile: q, o_free, s[2], p[2], o[2]
  static constexpr int B_GROUP = B_Q + 8 * QT;       // per query tile: its softmax warps meet
  static constexpr int B_DRAIN = B_GROUP + QT;       // per issuer
  static constexpr int NBAR = B_DRAIN + 2;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 64;
  static constexpr int O_COL = 2 * NKEY;
  static constexpr int QCOLS = 256;
  static constexpr uint32_t TMEM_COLS = QT * QCOLS;
  static constexpr float kRescaleThreshold = 8.f;
  static_assert(MIN_BLOCKS * (1024 + 1024 + SMEM) <= 228 * 1024, "shared memory per SM");
  static size_t smem_bytes() { return 1024 + static_cast<size_t>(SMEM); }
};

template <class Tr>
__global__ void __launch_bounds__(Tr::THREADS, Tr::MIN_BLOCKS)
    paged_attn_tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap) {
  using T = typename Tr::T;
  using MT = typename Tr::MT;
  constexpr int D = Tr::D, M = Tr::M, NS = Tr::NS, QT = Tr::QT, NKEY = Tr::NKEY;
  constexpr int PIECES = Tr::PIECES, HALVES = Tr::HALVES, ROWS = Tr::ROWS;
  constexpr uint32_t IDESC_S = tc::idesc_f16(Tr::kBf16, M, NKEY, false);
  constexpr uint32_t IDESC_O = tc::idesc_f16(Tr::kBf16, M, D, true);
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = sbase + Tr::OFF_BAR;
  auto bar = [&](int i) { return bars + 8 * i; };
  auto bar_q = [&](int q) { return bar(Tr::B_Q + 8 * q); };
  auto bar_ofree = [&](int q) { return bar(Tr::B_Q + 8 * q + 1); };
  auto bar_s = [&](int q, int b) { return bar(Tr::B_Q + 8 * q + 2 + b); };
  auto bar_p = [&](int q, int b) { return bar(Tr::B_Q + 8 * q + 4 + b); };
  auto bar_o = [&](int q, int b) { return bar(Tr::B_Q + 8 * q + 6 + b); };
  // behind the barriers: TMEM address, where the stretch starts, the items
  // whose V held non-finite tree elements (by parity: item + 1)
  int* words = reinterpret_cast<int*>(smem + Tr::OFF_BAR + Tr::NBAR * 8);
  int* s_found = words + 1;  // sequence, unit, position, length of the stretch
  int* s_odd = words + 6;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(Tr::B_KFULL + s), Tr::NWIDEN);  // E4M3: each widening warp arrives
      mbar_init(bar(Tr::B_KEMPTY + s), 1);
      mbar_init(bar(Tr::B_VFULL + s), Tr::NWIDEN);
      mbar_init(bar(Tr::B_VEMPTY + s), 1);
    }
    for (int s = 0; s < 2 * Tr::NSTG; ++s) {
      mbar_init(bar(Tr::B_STG + s), 1);
      mbar_init(bar(Tr::B_STGEMPTY + s), Tr::NWIDEN);
    }
    for (int q = 0; q < QT; ++q) {
      mbar_init(bar_q(q), 4);  // one arrival per softmax warp
      mbar_init(bar_ofree(q), 4);
      mbar_init(bar(Tr::B_GROUP + q), 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar_s(q, b), 1);
        mbar_init(bar_p(q, b), 4);
        mbar_init(bar_o(q, b), 1);
      }
    }
    mbar_init(bar(Tr::B_DRAIN), 1);
    mbar_init(bar(Tr::B_DRAIN + 1), 1);
    s_found[3] = 0;
    s_odd[0] = s_odd[1] = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  trigger_dependents();

  // ---- where this CTA's stretch of the line starts -------------------------------
  {
    const int per = (p.num_seqs + Tr::THREADS - 1) / Tr::THREADS;
    const int first = min(p.num_seqs, static_cast<int>(threadIdx.x) * per);
    const int last = min(p.num_seqs, first + per);
    auto weight = [&](int i, bool report) -> long long {
      TreeSeq s;
      if (!tree_seq(p, tree_lens(p, i), s, report)) return 0;
      const int rts = ((s.q_len << p.group_shift) + ROWS - 1) / ROWS;
      return static_cast<long long>(rts) * p.num_kv_heads *
             ((s.ctx + NKEY - 1) / NKEY + kTreeUnitCost);
    };
    long long own = 0;
    for (int i = first; i < last; ++i) own += weight(i, blockIdx.x == 0);
    long long upto = own;  // inclusive scan over the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(kFullMask, upto, o);
      if (lane >= o) upto += x;
    }
    long long* sums = reinterpret_cast<long long*>(smem + Tr::OFF_SEEN);
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < Tr::THREADS / 32; ++w) {
      if (w < warp) upto += sums[w];
      total += sums[w];
    }
    const long long even = (total + gridDim.x - 1) / gridDim.x;
    const long long len = even > kTreeMinTiles ? even : kTreeMinTiles;
    const long long start = len * blockIdx.x;
    if (start < upto && start >= upto - own) {
      long long at = start - (upto - own);
      for (int i = first; i < last; ++i) {
        const long long w = weight(i, false);
        if (at < w) {
          const int span = (p.context_lens[i] + NKEY - 1) / NKEY + kTreeUnitCost;
          s_found[0] = i;
          s_found[1] = static_cast<int>(at / span);
          s_found[2] = static_cast<int>(at % span);
          // the line's end cuts the last stretch by itself
          s_found[3] = static_cast<int>(len < 0x7fffffff ? len : 0x7fffffff);
          break;
        }
        at -= w;
      }
    }
    if (threadIdx.x == 0) p.ws_meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  __syncthreads();
  if (s_found[3] == 0) return;
  TreeWalk<ROWS> walk;
  walk.seq = s_found[0];
  walk.unit = s_found[1];
  walk.at = s_found[2];
  walk.left = s_found[3];
  walk.loaded = false;
  walk.ahead = tree_lens(p, walk.seq);
  const int len = walk.left;

  if (warp == 1) {
    tc::tmem_alloc(smem_addr(words), Tr::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(words[0]);

  // rows of query tile q of an item
  auto rows_of = [&](const TreeItem& it, int q) {
    return min(M, (it.q_len << p.group_shift) - it.rt * ROWS - q * M);
  };
  // the tile holds keys that not every row sees, or none
  auto partial = [&](const TreeItem& it, int t) { return (t + 1) * NKEY > it.ctx - it.q_len; };
  TreeItem it;

  if (warp == 0 || warp == 2) {
    // ---- producers: K (warp 0) and V (warp 2) tiles ----------------------------------
    const bool is_k = warp == 0;
    // the ring that TMA writes: the stages, or (E4M3) the staging slots
    constexpr int RING = Tr::kFp8 ? Tr::NSTG : NS;
    auto full = [&](int s) {
      return bar(Tr::kFp8 ? Tr::B_STG + (is_k ? 0 : Tr::NSTG) + s
                          : (is_k ? Tr::B_KFULL : Tr::B_VFULL) + s);
    };
    auto empty = [&](int s) {
      return bar(Tr::kFp8 ? Tr::B_STGEMPTY + (is_k ? 0 : Tr::NSTG) + s
                          : (is_k ? Tr::B_KEMPTY : Tr::B_VEMPTY) + s);
    };
    const uint32_t ring = Tr::kFp8 ? sbase + Tr::OFF_STG + (is_k ? 0 : Tr::NSTG * Tr::STG_TILE)
                                   : sbase + Tr::OFF_KV + (is_k ? 0 : Tr::KV_TILE);
    constexpr int SLOT = Tr::kFp8 ? Tr::STG_TILE : Tr::STAGE;
    constexpr int BOX = Tr::kFp8 ? 16 * D : 2048;              // bytes of a TMA box: 16 keys
    constexpr int BOXES = Tr::kFp8 ? 1 : HALVES;               // boxes per 16 keys
    constexpr int HALF = Tr::kFp8 ? Tr::STG_TILE : Tr::KV_HALF;
    const int shift = p.block_size == 16 ? 4 : 5;
    int gt = 0;
    bool ok = true;
    // 32 entries of an item's table row at a time, an item's first ones while
    // the item before it is under way
    auto entries = [&](const TreeItem& x, int chunk) {
      const int i = (chunk << 5) + lane;
      return i < (x.ctx + p.block_size - 1) >> shift
                 ? p.block_tables[static_cast<size_t>(x.seq) * p.max_blocks_per_seq + i]
                 : -1;
    };
    auto first_chunk = [&](const TreeItem& x) { return (x.t0 * NKEY) >> (shift + 5); };
    TreeItem nx;
    bool more = walk.next(p, nx);
    int ahead = more ? entries(nx, first_chunk(nx)) : -1;
    while (ok && more) {
      it = nx;
      int chunk = first_chunk(it), entry = ahead;
      more = walk.next(p, nx);
      if (more) ahead = entries(nx, first_chunk(nx));
      for (int t = it.t0; t < it.t1; ++t, ++gt) {
        const int stage = gt % RING;
        if (((t * NKEY) >> (shift + 5)) != chunk) {
          chunk = (t * NKEY) >> (shift + 5);
          entry = entries(it, chunk);
        }
        // this lane's 16 keys
        const int piece = (lane / BOXES) % PIECES;
        const int key = t * NKEY + piece * 16;
        const int pb = __shfl_sync(kFullMask, entry, (key >> shift) & 31);
        const bool mine = lane < PIECES * BOXES && key < it.ctx;
        const bool valid =
            mine && static_cast<unsigned>(pb) < static_cast<unsigned>(p.num_blocks);
        const int boxes = __popc(__ballot_sync(kFullMask, valid));
        if (mine && !valid && is_k) set_err(p.err, PKV_DEVERR_BAD_BLOCK);
        ok = mbar_wait_bounded(empty(stage), ((gt / RING) & 1) ^ 1);
        ok = __all_sync(kFullMask, ok);
        if (!ok) break;
        if (lane == 0) {
          if (boxes > 0)
            mbar_arrive_expect_tx(full(stage), boxes * BOX);
          else
            mbar_arrive(full(stage));
        }
        __syncwarp();
        if (valid) {
          const int half = lane % BOXES;
          const int y = (pb * p.num_kv_heads + it.kvh) * p.block_size +
                        (key & (p.block_size - 1));
          tma_load_2d(ring + stage * SLOT + half * HALF + piece * BOX, is_k ? &kmap : &vmap,
                      half * 64, y, full(stage));
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      set_err(p.err, PKV_DEVERR_TIMEOUT);
      // 16-bit caches: the loads in flight land before the CTA ends
      for (int g = max(0, gt - RING); g < gt; ++g)
        (void)mbar_wait_bounded(full(g % RING), (g / RING) & 1);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ---- MMA issuers: S (warp 1) and P.V (warp 3), one thread each --------------------
    if (lane == 0) {
      bool ok = true;
      const uint64_t d_q = tc::smem_desc_sw128(sbase, 16, 1024);
      const uint64_t d_k = tc::smem_desc_sw128(sbase + Tr::OFF_KV, 16, 1024);
      const uint64_t d_v =
          tc::smem_desc_sw128(sbase + Tr::OFF_KV + Tr::KV_TILE, Tr::KV_HALF, 1024);
      int gt = 0;
      int tq[QT] = {}, iq[QT] = {};  // tiles and items of each query tile so far
      while (ok && walk.next(p, it)) {
        const bool act[2] = {true, QT == 2 && rows_of(it, 1) > 0};
        if (warp == 1) {
#pragma unroll
          for (int q = 0; q < QT; ++q) {
            if (!ok || !act[q]) continue;
            ok = mbar_wait_bounded(bar_q(q), iq[q] & 1);
            ++iq[q];
          }
          for (int t = it.t0; ok && t < it.t1; ++t, ++gt) {
            ok = mbar_wait_bounded(bar(Tr::B_KFULL + gt % NS), (gt / NS) & 1);
            const uint64_t k0 = d_k + static_cast<uint32_t>((gt % NS) * (Tr::STAGE >> 4));
#pragma unroll
            for (int q = 0; q < QT; ++q) {
              if (!ok || !act[q]) continue;
              const int b = tq[q] & 1;
              // the buffer holds P of two tiles ago until P.V has read it
              if (tq[q] >= 2) ok = mbar_wait_bounded(bar_o(q, b), ((tq[q] - 2) >> 1) & 1);
              if (!ok) break;
              tc::tc_fence_after();
              const uint64_t q0d = d_q + q * (Tr::Q_TILE >> 4);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t step = (ks >> 2) * (Tr::Q_HALF >> 4) + (ks & 3) * 2;
                const uint32_t kstep = (ks >> 2) * (Tr::KV_HALF >> 4) + (ks & 3) * 2;
                tc::umma_f16(tmem + q * Tr::QCOLS + b * NKEY, q0d + step, k0 + kstep, IDESC_S,
                             ks > 0 ? 1u : 0u);
              }
              tc::umma_commit(bar_s(q, b));
              ++tq[q];
            }
            if (ok) tc::umma_commit(bar(Tr::B_KEMPTY + gt % NS));
          }
        } else {
          for (int t = it.t0; ok && t < it.t1; ++t, ++gt) {
            // V rows of such a tile are cleared by every query tile's softmax
            const bool all_p = partial(it, t) || t == it.t1 - 1;
            if (all_p) {
#pragma unroll
              for (int q = 0; q < QT; ++q)
                if (ok && act[q]) ok = mbar_wait_bounded(bar_p(q, tq[q] & 1), (tq[q] >> 1) & 1);
            }
            if (ok) ok = mbar_wait_bounded(bar(Tr::B_VFULL + gt % NS), (gt / NS) & 1);
            const uint64_t v0 = d_v + static_cast<uint32_t>((gt % NS) * (Tr::STAGE >> 4));
#pragma unroll
            for (int q = 0; q < QT; ++q) {
              if (!ok || !act[q]) continue;
              const int b = tq[q] & 1;
              if (!all_p) ok = mbar_wait_bounded(bar_p(q, b), (tq[q] >> 1) & 1);
              // the first tile overwrites the O of the item before
              if (ok && t == it.t0 && iq[q] > 0)
                ok = mbar_wait_bounded(bar_ofree(q), (iq[q] - 1) & 1);
              if (!ok) break;
              tc::tc_fence_after();
              const uint32_t ptm = tmem + q * Tr::QCOLS + b * NKEY;
              const uint32_t otm = tmem + q * Tr::QCOLS + Tr::O_COL;
#pragma unroll
              for (int kk = 0; kk < NKEY / 16; ++kk) {
                const uint64_t bdesc = v0 + kk * (2048 >> 4);
                tc::umma_f16_ts(otm, ptm + 8 * kk, bdesc, IDESC_O,
                                (t > it.t0 || kk > 0) ? 1u : 0u);
                if constexpr (Tr::kBf16)
                  tc::umma_f16_ts(otm, ptm + NKEY / 2 + 8 * kk, bdesc, IDESC_O, 1u);
              }
              tc::umma_commit(bar_o(q, b));
              ++tq[q];
            }
            if (ok) tc::umma_commit(bar(Tr::B_VEMPTY + gt % NS));
          }
#pragma unroll
          for (int q = 0; q < QT; ++q)
            if (act[q]) ++iq[q];
        }
      }
      if (!ok) {
        set_err(p.err, PKV_DEVERR_TIMEOUT);
        // what was issued completes before TMEM is freed
        const uint32_t drain = bar(Tr::B_DRAIN + (warp == 1 ? 0 : 1));
        tc::umma_commit(drain);
        (void)mbar_wait_bounded(drain, 0);
      }
    }
    __syncwarp();
  } else if (warp < Tr::WIDEN_WARP) {
    // ---- softmax warps: query tile q, thread <-> row <-> TMEM lane ---------------------
    const int q = (warp - Tr::SOFTMAX_WARP) >> 2;
    const int quarter = warp & 3;  // the TMEM lanes this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t tm = tmem + q * Tr::QCOLS + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t* seen = reinterpret_cast<uint32_t*>(smem + Tr::OFF_SEEN) + (q * M + r) * 8;
    int* par = reinterpret_cast<int*>(smem + Tr::OFF_PAR) + q * 2 * PKV_MAX_TREE_NODES;
    int met = 0;
    // a barrier of the query tile's softmax warps, bounded as every wait
    auto group_sync = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Tr::B_GROUP + q));
      return __all_sync(kFullMask, mbar_wait_bounded(bar(Tr::B_GROUP + q), met++ & 1));
    };
    const int gmask = (1 << p.group_shift) - 1;
    // row `row` of the item's query tile in q and out
    auto row_at = [&](const TreeItem& x, int row) {
      const int c = x.rt * ROWS + q * M + row;
      return static_cast<size_t>(x.q0 + (c >> p.group_shift)) * p.num_heads +
             (static_cast<size_t>(x.kvh) << p.group_shift) + (c & gmask);
    };
    // An item's query rows and its tree's parents come by cp.async, issued once
    // the last S of the item before is complete; rows that do not exist are
    // left as they are (nobody reads their S).
    auto begin_load = [&](const TreeItem& x, int parity) {
      constexpr int CH = D / 8;
      const int n = rows_of(x, q) * CH;
      const uint32_t qt = sbase + q * Tr::Q_TILE;
      for (int i = r; i < n; i += 128) {
        const int row = i / CH, ch = i % CH;
        cp_async16(qt + (ch >> 3) * Tr::Q_HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                   static_cast<const T*>(p.q) + row_at(x, row) * D + ch * 8);
      }
      if (partial(x, x.t1 - 1)) {
        const int nodes = ((x.rt * ROWS + q * M + rows_of(x, q) - 1) >> p.group_shift) + 1;
        for (int i = r; i < nodes; i += 128)
          cp_async4(smem_addr(par + parity * PKV_MAX_TREE_NODES + i), p.parents + x.q0 + i);
      }
    };
    auto end_load = [&](const TreeItem& x) {
      cp_async_wait_all();
      if constexpr (Tr::kQToFp16) {
        constexpr int CH = D / 8;
        const int n = rows_of(x, q) * CH;
        for (int i = r; i < n; i += 128) {
          const int row = i / CH, ch = i % CH;
          uint4* at = reinterpret_cast<uint4*>(smem + q * Tr::Q_TILE + (ch >> 3) * Tr::Q_HALF +
                                               row * 128 + (((ch & 7) ^ (row & 7)) << 4));
          const uint4 u = *at;
          *at = make_uint4(bf16x2_to_f16x2_sat(u.x), bf16x2_to_f16x2_sat(u.y),
                           bf16x2_to_f16x2_sat(u.z), bf16x2_to_f16x2_sat(u.w));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q(q));
    };
    int gt = 0, tq = 0, item = 0;
    bool ok = true;
    TreeItem nx;
    bool more = walk.next(p, nx);
    if (more && rows_of(nx, q) > 0) {
      begin_load(nx, 1);
      end_load(nx);
    }
    while (ok && more) {
      it = nx;
      more = walk.next(p, nx);
      ++item;
      const bool load_next = more && rows_of(nx, q) > 0;
      const int nrows = rows_of(it, q);
      if (nrows <= 0) {  // the second query tile of a unit of few rows
        gt += it.t1 - it.t0;
        if (load_next) {
          begin_load(nx, (item + 1) & 1);
          end_load(nx);
        }
        continue;
      }
      const bool active = r < nrows;
      const bool warp_active = quarter * 32 < nrows;
      const int hist = it.ctx - it.q_len;
      float k_scale = 1.f, v_scale = 1.f;
      if constexpr (Tr::kFp8) {
        k_scale = p.k_scales[it.kvh];
        v_scale = p.v_scales[it.kvh];
        if (!(k_scale > 0.f && k_scale < INFINITY && v_scale > 0.f && v_scale < INFINITY) &&
            r == 0)
          set_err(p.err, PKV_DEVERR_BAD_SCALE);
      }
      if (partial(it, it.t1 - 1)) {
        // the nodes that each row sees: itself, its parent, and so on
        const int node = (it.rt * ROWS + q * M + min(r, nrows - 1)) >> p.group_shift;
        const int* up = par + (item & 1) * PKV_MAX_TREE_NODES;
        ok = group_sync();  // every thread's share of the parents has arrived
        if (!ok) break;
#pragma unroll
        for (int w = 0; w < 8; ++w) seen[w] = 0;
        int at = node >> 5;
        uint32_t bits = 0;
        for (int n = node; n >= 0;) {
          if ((n >> 5) != at) {
            seen[at] = bits;
            at = n >> 5;
            bits = 0;
          }
          bits |= 1u << (n & 31);
          const int x = up[n];
          if (x < -1 || x >= n) {
            set_err(p.err, PKV_DEVERR_BAD_TREE);
            break;
          }
          n = x;
        }
        seen[at] = bits;
      }
      // The row's visible keys of tile t, bit by bit.
      auto window = [&](int t) -> unsigned long long {
        const int k0 = t * NKEY - hist;  // the node at the tile's first key
        if (k0 <= -NKEY) return ~0ull;
        auto word = [&](int w) -> unsigned long long {
          return w < PKV_MAX_TREE_NODES / 32 ? seen[w] : 0u;
        };
        if (k0 <= 0) {
          const unsigned long long lo = word(0) | (word(1) << 32);
          return k0 == 0 ? lo : (lo << -k0) | ((1ull << -k0) - 1);
        }
        const int w = k0 >> 5, sh = k0 & 31;
        const unsigned long long lo = word(w) | (word(w + 1) << 32);
        return sh == 0 ? lo : (lo >> sh) | (word(w + 2) << (64 - sh));
      };
      float m = -INFINITY, l = 0.f;
      // x = s * qscale; for qscale > 0 the row's max of x is (max s) * qscale
      // exactly, so s is masked and reduced unscaled and the scale folds into
      // the exponent's multiply-add
      const float mult0 = p.qscale * k_scale;
      const float mult = mult0 > 0.f ? mult0 : 1.f;
      for (int t = it.t0; t < it.t1; ++t, ++gt, ++tq) {
        const int b = tq & 1;
        ok = mbar_wait_bounded(bar_s(q, b), (tq >> 1) & 1);
        if (!__all_sync(kFullMask, ok)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        // every S of this item is complete: its query tile may be replaced
        if (t == it.t1 - 1 && load_next) begin_load(nx, (item + 1) & 1);
        const bool cut = partial(it, t);
        if (warp_active) {
          const uint32_t sbuf = tm + b * NKEY;
          float s[64];
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            float v[16];
            tc::tmem_ld16(sbuf + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[c + i] = v[i];
          }
          tc::tmem_wait_ld();
          if (!(mult0 > 0.f)) {
#pragma unroll
            for (int c = 0; c < 64; ++c) s[c] *= mult0;
          }
          if (cut) {
            const unsigned long long w = window(t);
            const uint32_t w0 = static_cast<uint32_t>(w), w1 = static_cast<uint32_t>(w >> 32);
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              if (!(w0 & (1u << c))) s[c] = -INFINITY;
              if (!(w1 & (1u << c))) s[32 + c] = -INFINITY;
            }
          }
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 64; c += 8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) mx4[u] = tc::max3(mx4[u], s[c + u], s[c + 4 + u]);
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * mult;
          float alpha = 1.f;
          if (active && mx > m + Tr::kRescaleThreshold) {
            alpha = exp2_approx(m - mx);  // 0 on the first tile (m = -inf)
            m = mx;
          }
          const float neg_m = m == -INFINITY ? 0.f : -m;
          const uint64_t mult2 = tc::f2_pack(mult, mult), neg_m2 = tc::f2_pack(neg_m, neg_m);
          uint64_t sum2[2] = {tc::f2_pack(0.f, 0.f), tc::f2_pack(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x0, x1;
              tc::f2_unpack(
                  tc::f2_fma(tc::f2_pack(s[c + 2 * h], s[c + 2 * h + 1]), mult2, neg_m2), x0, x1);
              s[c + 2 * h] = exp2_approx(x0);
              s[c + 2 * h + 1] = exp2_approx(x1);
              sum2[h] = tc::f2_add(sum2[h], tc::f2_pack(s[c + 2 * h], s[c + 2 * h + 1]));
            }
          }
          // P over the S columns just read: 32 columns, and 32 of low halves for bf16
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t w[16], wl[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float x = s[32 * g + 2 * e], y = s[32 * g + 2 * e + 1];
              w[e] = pack2(x, y, MT());
              if constexpr (Tr::kBf16)
                wl[e] = pack2(x - __uint_as_float(w[e] << 16),
                              y - __uint_as_float(w[e] & 0xffff0000u), Bf16());
            }
            tc::tmem_st16u(sbuf + 16 * g, w);
            if constexpr (Tr::kBf16) tc::tmem_st16u(sbuf + NKEY / 2 + 16 * g, wl);
          }
          tc::tmem_wait_st();
          float a[4];
          tc::f2_unpack(sum2[0], a[0], a[1]);
          tc::f2_unpack(sum2[1], a[2], a[3]);
          l = l * alpha + ((a[0] + a[1]) + (a[2] + a[3]));
          if (t > it.t0 && __any_sync(kFullMask, alpha != 1.f)) {
            // O holds every earlier tile before it is rescaled
            ok = mbar_wait_bounded(bar_o(q, (tq - 1) & 1), ((tq - 1) >> 1) & 1);
            if (!__all_sync(kFullMask, ok)) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float v[16];
              tc::tmem_ld16(tm + Tr::O_COL + c, v);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= alpha;
              tc::tmem_st16(tm + Tr::O_COL + c, v);
            }
            tc::tmem_wait_st();
          }
        }
        if (cut) {
          ok = mbar_wait_bounded(bar(Tr::B_VFULL + gt % NS), (gt / NS) & 1);
          if (!__all_sync(kFullMask, ok)) {
            ok = false;
            break;
          }
          // an element with all exponent bits set is infinite or NaN
          constexpr uint32_t kExp = Tr::kBf16 ? 0x7F807F80u : 0x7C007C00u;
          constexpr uint32_t kOne = Tr::kBf16 ? 0x00800080u : 0x04000400u;
          unsigned char* vt = smem + Tr::OFF_KV + (gt % NS) * Tr::STAGE + Tr::KV_TILE;
          const int from = max(0, hist - t * NKEY), end = it.ctx - t * NKEY;
          for (int i = from * 8 + r; i < NKEY * 8; i += 128) {
            const int row = i >> 3;
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
              uint4* at = reinterpret_cast<uint4*>(vt + h * Tr::KV_HALF + i * 16);
              if (row >= end) {
                *at = make_uint4(0u, 0u, 0u, 0u);
                continue;
              }
              uint4 u = *at;
              auto hit = [&](uint32_t x) { return ((x & kExp) + kOne) & 0x80008000u; };
              if (hit(u.x) | hit(u.y) | hit(u.z) | hit(u.w)) {
                auto clear = [&](uint32_t x) {
                  const uint32_t y = hit(x);
                  return x & ~((y & 0x8000u ? 0xffffu : 0u) | (y >> 16 ? 0xffff0000u : 0u));
                };
                s_odd[item & 1] = item;  // before the elements are cleared
                __threadfence_block();
                *at = make_uint4(clear(u.x), clear(u.y), clear(u.z), clear(u.w));
              }
            }
          }
        }
        fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p(q, b));
      }
      if (!ok) break;
      if (load_next) end_load(nx);
      // ---- output ------------------------------------------------------------------
      ok = mbar_wait_bounded(bar_o(q, (tq - 1) & 1), ((tq - 1) >> 1) & 1);
      if (!__all_sync(kFullMask, ok)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const bool whole = it.t0 == 0 && it.t1 == it.nt;
      const bool odd = *static_cast<volatile int*>(s_odd + (item & 1)) == item;
      if (warp_active) {
        const float inv = l > 0.f || l != l ? v_scale / l : 0.f;
        const size_t row = row_at(it, min(r, nrows - 1));
        // pieces: the one that starts a unit is its CTA's second, any other its first
        const size_t slot =
            (static_cast<size_t>(blockIdx.x) * 2 + (it.t0 == 0 ? 1 : 0)) * ROWS + q * M + r;
        if (!whole && active) p.ws_ml[slot] = make_float2(l != l ? l : m, l);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float v[16];
          tc::tmem_ld16(tm + Tr::O_COL + c, v);
          tc::tmem_wait_ld();
          if (!active) continue;
          if (odd) {
            // infinities and NaN in the V of the nodes that this row sees
            const int32_t* trow =
                p.block_tables + static_cast<size_t>(it.seq) * p.max_blocks_per_seq;
            const int lo = max(0, it.t0 * NKEY - hist), hi = min(it.q_len, it.t1 * NKEY - hist);
            for (int n = lo; n < hi; ++n) {
              if (!(seen[n >> 5] >> (n & 31) & 1u)) continue;
              const int key = hist + n;
              const int pb = trow[key / p.block_size];
              if (static_cast<unsigned>(pb) >= static_cast<unsigned>(p.num_blocks)) continue;
              const size_t at = ((static_cast<size_t>(pb) * p.num_kv_heads + it.kvh) *
                                     p.block_size + key % p.block_size) * D + c;
              for (int i = 0; i < 16; ++i) {
                float x;
                if constexpr (Tr::kFp8)
                  x = (static_cast<const uint8_t*>(p.v_cache)[at + i] & 0x7F) == 0x7F ? NAN : 0.f;
                else
                  x = static_cast<float>(static_cast<const T*>(p.v_cache)[at + i]);
                if (!(fabsf(x) < INFINITY)) v[i] += x;
              }
            }
          }
          if (whole) {
            float a[8], z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              a[i] = v[i] * inv;
              z[i] = v[8 + i] * inv;
            }
            T* o = static_cast<T*>(p.out) + row * D + c;
            *reinterpret_cast<uint4*>(o) = pack8(a, typename Tr::DT());
            *reinterpret_cast<uint4*>(o + 8) = pack8(z, typename Tr::DT());
          } else {
            // [D / 4][ROWS] of 4 floats: a warp's rows side by side
            float4* o = reinterpret_cast<float4*>(p.ws_o) + (slot - q * M - r) * (D / 4) + q * M + r;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[(c / 4 + i) * ROWS] = make_float4(v[4 * i] * v_scale, v[4 * i + 1] * v_scale,
                                 v[4 * i + 2] * v_scale, v[4 * i + 3] * v_scale);
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ofree(q));
      if (q == 0 && r == 0 && it.t0 > 0 && it.t1 == it.nt) {
        // this CTA ends a unit that another began: the one whose stretch holds
        // the unit's first tile, (t0 + kTreeUnitCost) - kTreeUnitCost positions
        // before this stretch's start
        const int before = (it.t0 + len - 1) / len;
        p.ws_meta[blockIdx.x] =
            make_int4(it.q0 + ((it.rt * ROWS) >> p.group_shift), it.kvh,
                      static_cast<int>(blockIdx.x) - before,
                      min(ROWS, (it.q_len << p.group_shift) - it.rt * ROWS));
      }
    }
    if (!ok && lane == 0) set_err(p.err, PKV_DEVERR_TIMEOUT);
    __syncwarp();
  } else if constexpr (Tr::kFp8) {
    // ---- E4M3: NWIDEN warps for each of K and V widen the codes ------------------------
    const int w = warp - Tr::WIDEN_WARP;
    const bool is_k = w < Tr::NWIDEN;
    const int part = is_k ? w : w - Tr::NWIDEN;
    constexpr int CHUNKS = NKEY * D / 16 / Tr::NWIDEN;  // 16 codes each
    const uint32_t stg = sbase + Tr::OFF_STG + (is_k ? 0 : Tr::NSTG * Tr::STG_TILE);
    const int b_stg = Tr::B_STG + (is_k ? 0 : Tr::NSTG);
    const int b_stge = Tr::B_STGEMPTY + (is_k ? 0 : Tr::NSTG);
    int gt = 0;
    bool ok = true;
    while (ok && walk.next(p, it)) {
      for (int t = it.t0; t < it.t1; ++t, ++gt) {
        const int stage = gt % NS, slot = gt % Tr::NSTG;
        ok = mbar_wait_bounded(bar((is_k ? Tr::B_KEMPTY : Tr::B_VEMPTY) + stage),
                               ((gt / NS) & 1) ^ 1) &&
             mbar_wait_bounded(bar(b_stg + slot), (gt / Tr::NSTG) & 1);
        ok = __all_sync(kFullMask, ok);
        if (!ok) break;
        const uint32_t src = stg + slot * Tr::STG_TILE;
        const uint32_t dst =
            sbase + Tr::OFF_KV + stage * Tr::STAGE + (is_k ? 0 : Tr::KV_TILE);
        // Chunk c of key r (dims 16c ..) becomes 16-bit chunks 2(c % 4) and
        // 2(c % 4) + 1 of row r in dim half c / 4, 128-byte swizzled; codes of
        // 128-byte rows come swizzled, of 64-byte rows not.
#pragma unroll 4
        for (int k = 0; k < CHUNKS / 32; ++k) {
          const int i = part * CHUNKS + lane + 32 * k;
          const int row = i / (D / 16), c = i % (D / 16);
          const uint32_t from = D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : i * 16;
          uint32_t x[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                       : "r"(src + from)
                       : "memory");
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[2 * e] = e4m3x2_to(x[e] & 0xffffu, Fp16());
            h[2 * e + 1] = e4m3x2_to(x[e] >> 16, Fp16());
          }
          const uint32_t to = dst + (c >> 2) * Tr::KV_HALF + row * 128;
          const int c0 = (c & 3) * 2;
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                           to + ((c0 ^ (row & 7)) << 4)),
                       "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                           to + (((c0 + 1) ^ (row & 7)) << 4)),
                       "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                       : "memory");
        }
        // the MMAs read the stage, and TMA rewrites the slot, by the async proxy
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar((is_k ? Tr::B_KFULL : Tr::B_VFULL) + stage));
          mbar_arrive(bar(b_stge + slot));
        }
      }
    }
    if (!ok && lane == 0) set_err(p.err, PKV_DEVERR_TIMEOUT);
    __syncwarp();
  }
  // ---- release TMEM (every path reaches here) ---------------------------------------------
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, Tr::TMEM_COLS);
  }
}

// Joins the pieces of the units that lie across CTAs' stretches: with M = max m,
//   out = sum 2^(m - M) o / sum 2^(m - M) l.
// Entry blockIdx.x is of the unit that ended in that CTA; the piece of the unit's
// first CTA is that CTA's second, of every later one its first.  A thread has 4
// dims of a row, a warp 2 rows x 64 dims (whole sectors of the pieces);
// blockIdx.y takes kTreeMergeRows rows.
constexpr int kTreeMergeRows = 8;
template <int D, int ROWS, class DT>
__global__ void __launch_bounds__(kTreeMergeRows * D / 4)
    paged_attn_tree_merge_kernel(const TreeParams p) {
  using T = typename DT::T;
  grid_dependency_wait();
  trigger_dependents();
  const int4 e = p.ws_meta[blockIdx.x];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = static_cast<int>(blockIdx.y) * kTreeMergeRows + (w / (D / 64)) * 2 + (lane & 1);
  const int c4 = (w % (D / 64)) * 16 + (lane >> 1);
  if (r >= e.w) return;
  const int last = static_cast<int>(blockIdx.x);
  auto piece = [&](int c) { return static_cast<size_t>(c) * 2 + (c == e.z ? 1 : 0); };
  // an online sum, so that every load of a piece is under way at once
  float big = -INFINITY, num[4] = {}, den = 0.f;
#pragma unroll 4
  for (int c = e.z; c <= last; ++c) {
    const float2 ml = p.ws_ml[piece(c) * ROWS + r];
    const float4 o = reinterpret_cast<const float4*>(p.ws_o)[(piece(c) * (D / 4) + c4) * ROWS + r];
    const float m = ml.x == -INFINITY ? big : fmaxf(big, ml.x);
    const float a = big == -INFINITY ? 0.f : exp2_approx(big - m);
    const float f = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - m);
    big = m;
    den = den * a + f * ml.y;
    num[0] = num[0] * a + f * o.x;
    num[1] = num[1] * a + f * o.y;
    num[2] = num[2] * a + f * o.z;
    num[3] = num[3] * a + f * o.w;
  }
  const float inv = den > 0.f || den != den ? 1.f / den : 0.f;
  T* out = static_cast<T*>(p.out) +
           (static_cast<size_t>(e.x + (r >> p.group_shift)) * p.num_heads +
            (static_cast<size_t>(e.y) << p.group_shift) + (r & ((1 << p.group_shift) - 1))) * D +
           c4 * 4;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack2(num[0] * inv, num[1] * inv, DT()),
                                              pack2(num[2] * inv, num[3] * inv, DT()));
}

}  // namespace pkv

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
// SMs, so up to 128 rows a unit is bound by memory, and softmax runs under the
// loads: QT = 1 (one 128-row query tile) has two CTAs an SM; QT = 2 one with two
// groups of softmax warps, which take the tiles of such a unit in turn.  More rows
// take QT = 2 with a query tile a group, sharing each K/V tile, bound by softmax and
// MMA.  (paged_attn_tree.cu chooses.)  E4M3 caches take QT = 2 always: their tiles
// lie in shared memory twice, as codes and as fp16, so one CTA fits an SM.  Codes in,
// out and back as fp16, and the MMAs' reads are about 130 KB a tile there, 1024
// cycles at 128 bytes each, where HBM needs 705.
//
// Split: the tiles of all units lie on one line, every sequence's units one
// after the other, and CTA c takes the c-th of gridDim.x equal stretches of it,
// whatever the lengths.  (A unit counts tree_unit_cost() tiles more than it has,
// for its query tile, pipeline fill and output.)  A unit that lies in one
// stretch is written out directly; pieces of a cut unit go to the workspace as
// (max, sum, unnormalised o) and paged_attn_tree_merge_kernel joins them.  Units of
// few tiles are left whole (tree_whole in paged_attn_tree.cu).
//
// A CTA: warp 0 / 2 bring K / V tiles by TMA through the block table into a
// ring of NS stages; warp 1 issues S = Q K^T into one of two TMEM buffers; warp
// 3 issues O += P V with P read from TMEM; 4 softmax warps per query tile, a
// thread per row (online softmax in base 2 in fp32; the reference maximum moves
// only when a logit passes it by 2^8, so O is rarely rescaled).  E4M3 caches:
// further warps widen each tile's codes to fp16 (exact) into the stage that the
// MMAs read.
//
// P in 16 bits, as the MMAs take it.  bf16 caches: two bf16 halves, 2^-17 of p, which
// the output's rounding hides.  fp16 and E4M3 caches: fp16, 2^-12 of p in earnest and
// 2^-11 at most, as much as the output's own rounding where one key dominates and
// less where many errors meet (two halves would double the P V MMAs).  fp16 is
// subnormal below 2^-14, so P = 2^(x - m) with m 7 below the row's reference
// maximum: P is normal down to 2^-21 of that maximum and off by at most 2^-32 of it
// below, that is at most 2^-32 sum |v_k| in the output (without the 7, keys of 2^-25
// and less vanished, however many).  The sum l takes p in fp32 before it is rounded.
//
// The tree's part of the keys: each row's visible nodes are a bit set, made once
// per unit by following the parents.  What a row does not see must not enter
// it, and 0 x NaN would: K is masked in S, and non-finite elements of the
// tree's V are taken out of the tile (and added to the rows that do see them
// when the output is written).  Rows of V past the context are zeroed.  Rows of O that
// hold a NaN are looked at again (tree_non_finite): an infinity stays one.
//
// Every wait is bounded; a role that gives up reports PKV_DEVERR_TIMEOUT, and
// TMEM is freed on every path.
#pragma once

#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "paged_attn_kernels.cuh"
#include "paged_prefill_tc_kernels.cuh"

namespace pkv {

struct TreeParams {
  void* out;
  const void* q;
  const void* v_cache;  // for non-finite elements; K and V come through the tensor maps
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const int32_t* parents;
  float qscale;  // scale * log2(e)
  const float* k_scales;  // E4M3 caches
  const float* v_scales;
  int num_seqs, num_tokens, num_heads, num_kv_heads, group_shift;
  int block_size, max_blocks_per_seq, max_context_len, max_query_len, num_blocks;
  int whole_units;  // units are not cut
  int direct;       // ... and each has its CTA: max_rts for every (sequence, kv head)
  int max_rts, num_ctas;
  int out_aligned32;
  unsigned* err;
  // Workspace: for each CTA one merge entry and two pieces of ROWS rows.  Entry c
  // is of the unit that ended in CTA c, {first token, kv head, first CTA, rows},
  // rows = 0 where none did that another CTA began; or, with at least 8 CTAs a unit
  // (by_unit: units in many pieces), entry u is of unit u (of max_rts for every
  // (sequence, kv head)), {first CTA, last CTA}, the same one where it is not cut.
  int by_unit;
  int4* ws_meta;
  float2* ws_ml;  // (max, sum) of each row of each piece
  float* ws_o;    // [pieces][D / 8][ROWS][8], on a 32-byte boundary
};

// What a unit costs beside its tiles, in tiles, of which a CTA of two query tiles,
// alone on its SM, does nearly twice as many in the time.  Measured on B200 (us):
// LLaMA-7B batch, one query tile, 104.7 / 104.1 / 105.4 at 4 / 5 / 6; two query
// tiles at 5 / 7 / 10: GQA chat 71.7 / 64.5 / 65.8, E4M3 68.3 / 67.2 / 68.9.
__host__ __device__ constexpr int tree_unit_cost(int rows) { return rows > 128 ? 7 : 5; }
// The shortest stretch worth a CTA (2 / 6: one sequence of 1200 tokens 15.3 / 15.9
// us, batches alike).
constexpr int kTreeMinTiles = 2;
constexpr int kTreeKeys = 64;     // keys per tile

// 32 consecutive 32-bit columns of this warp's TMEM lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// 32 bytes to a 32-byte boundary in one store.
__device__ __forceinline__ void store32(void* dst, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

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
// Positions on the line: a unit's cost beside its tiles, then its tiles, each
// of them for every query tile of the unit.  `rows` of a unit, of 128 each.
__device__ __forceinline__ int tree_per(int rows) { return rows > 128 ? 2 : 1; }
template <int ROWS>
__device__ __forceinline__ int tree_span(const TreeParams& p, int ctx, int rows) {
  return p.whole_units ? 1
                       : ((ctx + kTreeKeys - 1) / kTreeKeys + tree_unit_cost(ROWS)) * tree_per(rows);
}
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

// A CTA's next piece of work: tiles t0 .. t1 - 1 of the nt of a unit.  `lead`:
// positions between the unit's first tile and the start of the CTA's stretch.
struct TreeItem {
  int seq, ctx, q0, q_len, kvh, rt, t0, t1, nt, lead;
};

// The units of a sequence, row tile after row tile for each kv head; each kv
// head's take this many positions.
template <int ROWS>
__device__ __forceinline__ int tree_head_span(const TreeParams& p, const TreeSeq& s) {
  const int rows = s.q_len << p.group_shift;
  const int full = rows / ROWS, rest = rows % ROWS;
  return full * tree_span<ROWS>(p, s.ctx, ROWS) + (rest > 0 ? tree_span<ROWS>(p, s.ctx, rest) : 0);
}

// Walks a CTA's stretch.  Every role walks on its own.  The lengths of the
// sequence after the one at hand are loaded ahead of their use.
template <int ROWS>
struct TreeWalk {
  int seq, kvh, rt, at;  // the next sequence, unit of it, and position in the unit
  int left;              // positions left in the stretch
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
      const int rows = (s.q_len << p.group_shift) - rt * ROWS;
      const int per = tree_per(min(rows, ROWS));
      const int span = tree_span<ROWS>(p, s.ctx, min(rows, ROWS));
      const int take = min(left, span - at);
      it.seq = seq;
      it.ctx = s.ctx;
      it.q0 = s.q0;
      it.q_len = s.q_len;
      it.kvh = kvh;
      it.rt = rt;
      it.nt = nt;
      // a tile is the CTA's whose stretch holds its first position
      it.t0 = p.whole_units ? 0 : max(0, (at + per - 1) / per - tree_unit_cost(ROWS));
      it.t1 = p.whole_units ? nt : max(0, (at + take + per - 1) / per - tree_unit_cost(ROWS));
      it.lead = max(0, at - tree_unit_cost(ROWS) * per);
      left -= take;
      at += take;
      if (at == span) {
        at = 0;
        ++rt;
        if (rows <= ROWS) {
          rt = 0;
          if (++kvh == p.num_kv_heads) {
            kvh = 0;
            ++seq;
            loaded = false;
          }
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
  static constexpr int MIN_BLOCKS = QT == 1 ? 2 : 1;
  static constexpr int NS = kFp8 ? 2 : QT == 1 ? (D == 128 ? 2 : 4) : 4;
  static constexpr int NSTG = kFp8 ? 4 : 0;  // (3 stages and 3 slots measured the same)
  static constexpr int NWIDEN = kFp8 ? 2 : 1;  // widening warps for each of K, V
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
  static constexpr int OFF_PAR = OFF_SEEN + ROWS * 32;  // [QT][4 warps][256] parents
  static constexpr int OFF_ML = OFF_PAR + QT * 4 * PKV_MAX_TREE_NODES * 4;  // group 1's (max, sum)
  static constexpr int OFF_BAR = OFF_ML + (QT - 1) * M * 8;
  static constexpr int B_KFULL = 0, B_KEMPTY = NS, B_VFULL = 2 * NS, B_VEMPTY = 3 * NS;
  static constexpr int B_STG = 4 * NS, B_STGEMPTY = B_STG + 2 * NSTG;
  static constexpr int B_Q = B_STGEMPTY + 2 * NSTG;  // q; per group: o_free, s[2], p[2], o[2]
  static constexpr int B_VREADY = B_Q + 8 * QT;     // per group: V of its cut tile is in
  static constexpr int B_BOTH = B_VREADY + QT;       // group 1's share of an item
  static constexpr int B_DRAIN = B_BOTH + 1;         // per issuer
  static constexpr int NBAR = B_DRAIN + 2;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 64;
  static constexpr int O_COL = 2 * NKEY;
  static constexpr int QCOLS = 256;
  static constexpr uint32_t TMEM_COLS = QT * QCOLS;
  static constexpr float kRescaleThreshold = 8.f;
  // log2 of P at the row's reference maximum: P reaches 2^15 in fp16 before a
  // rescale, and is normal down to 2^-21 of that maximum
  static constexpr float kBias = kBf16 ? 0.f : 7.f;
  static_assert(MIN_BLOCKS * (1024 + 1024 + SMEM) <= 228 * 1024, "shared memory per SM");
  static size_t smem_bytes() { return 1024 + static_cast<size_t>(SMEM); }
};

// Infinities and NaN in the V of visible keys k0 .. k1 - 1: where a warp's rows see any,
// their sum is the element's value, whatever the rest is.  Those of the tree (keys from
// `hist`; `seen`: the row's visible nodes, or null) were taken out of the tile; one of the
// history, where its weight, or a bf16 half of it, is 0 or negative, made NaN of O.
// `out`, or the piece `ws`, is this lane's row (or both are null).  For 16-bit caches
// (E4M3 has no infinities); called by whole warps, and not inline: inline it cost the GQA
// chat batch 62.5 -> 74.8 us, so 65.0.  Where there are any it takes 0.3 us a key.
template <class T, int D, int ROWS>
__device__ __noinline__ void tree_non_finite(const void* v_cache, const int32_t* table,
                                             int num_blocks, int num_kv_heads, int kvh,
                                             int block_size, int hist, int k0, int k1,
                                             bool history, const uint32_t* seen, T* out,
                                             float* ws) {
  constexpr int PER = D / 32;  // a lane's dims
  const int lane = threadIdx.x & 31;
  // f(e, value) for the non-finite elements of a key in dims d0 + e, e < dims
  auto odd_of = [&](int key, int d0, int dims, auto f) {
    const int pb = table[key / block_size];
    if (static_cast<unsigned>(pb) >= static_cast<unsigned>(num_blocks)) return;
    const size_t at =
        ((static_cast<size_t>(pb) * num_kv_heads + kvh) * block_size + key % block_size) * D + d0;
#pragma unroll
    for (int e = 0; e < dims; ++e) {
      const float x = static_cast<float>(static_cast<const T*>(v_cache)[at + e]);
      if (!(fabsf(x) < INFINITY)) f(e, x);
    }
  };
  float hsum[PER] = {};  // of the history, which every row sees
  if (history) {
#pragma unroll 8
    for (int key = k0; key < min(hist, k1); ++key)
      odd_of(key, lane * PER, PER, [&](int e, float x) { hsum[e] += x; });
  }
#pragma unroll 1
  for (int src = 0; src < 32; ++src) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int c = src * PER + e;
      float sum = __shfl_sync(kFullMask, hsum[e], src);
      if (seen != nullptr) {
#pragma unroll 1
        for (int n = max(0, k0 - hist); n < k1 - hist; ++n)
          if (seen[n >> 5] >> (n & 31) & 1u)
            odd_of(hist + n, c, 1, [&](int, float x) { sum += x; });
      }
      if (sum == 0.f || (out == nullptr && ws == nullptr)) continue;
      float* to = ws + static_cast<size_t>(c / 8) * ROWS * 8 + c % 8;
      const float o = out != nullptr ? static_cast<float>(out[c]) : *to;
      if (!history && !(fabsf(o) < INFINITY)) sum += o;  // the history's infinity
      if (out != nullptr)
        out[c] = static_cast<T>(sum);
      else
        *to = sum;
    }
  }
}

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
  // behind the barriers: the TMEM address; the items whose V held non-finite tree
  // elements (by parity); where the stretch starts
  int* words = reinterpret_cast<int*>(smem + Tr::OFF_BAR + Tr::NBAR * 8);
  int* s_odd = words + 2;
  struct Found {
    long long at;
    int seq;
    TreeLens lens;
  };
  Found* s_found = reinterpret_cast<Found*>(words + 4);

  const int warp = __shfl_sync(kFullMask, static_cast<int>(threadIdx.x) >> 5, 0);
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
      mbar_init(bar(Tr::B_VREADY + q), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar_s(q, b), 1);
        mbar_init(bar_p(q, b), 4);
        mbar_init(bar_o(q, b), 1);
      }
    }
    mbar_init(bar(Tr::B_BOTH), 4);
    mbar_init(bar(Tr::B_DRAIN), 1);
    mbar_init(bar(Tr::B_DRAIN + 1), 1);
    s_found->seq = -1;
    s_odd[0] = s_odd[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_addr(words), Tr::TMEM_COLS);
    tc::tmem_relinquish();
  }
  grid_dependency_wait();
  trigger_dependents();

  // ---- where this CTA's stretch of the line starts -------------------------------
  TreeWalk<ROWS> walk;
  int len, early = -1;  // early: the first table entries, where the sequence is known at once
  if (p.direct) {
    // a CTA per unit, without the scan
    const int units = p.num_kv_heads * p.max_rts;
    walk.seq = static_cast<int>(blockIdx.x) / units;
    walk.kvh = static_cast<int>(blockIdx.x) % units / p.max_rts;
    walk.rt = static_cast<int>(blockIdx.x) % p.max_rts;
    walk.ahead = tree_lens(p, walk.seq);
    walk.at = 0;
    if ((warp == 0 || warp == 2) && lane < p.max_blocks_per_seq)
      early = p.block_tables[static_cast<size_t>(walk.seq) * p.max_blocks_per_seq + lane];
    TreeSeq s;
    len = tree_seq(p, walk.ahead, s,
                   static_cast<int>(blockIdx.x) % units == 0 && threadIdx.x == 0) &&
          walk.rt * ROWS < s.q_len << p.group_shift;
    tc::tc_fence_before();
    __syncthreads();
  } else {
    auto weight = [&](const TreeLens& x, bool report) -> long long {
      TreeSeq s;
      if (!tree_seq(p, x, s, report)) return 0;
      return static_cast<long long>(tree_head_span<ROWS>(p, s)) * p.num_kv_heads;
    };
    auto scan = [&](long long x) {  // inclusive, over the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o) x += y;
      }
      return x;
    };
    // the stretches' length on a line of `total`; 32-bit divisions are many times as fast
    auto each_of = [&](long long total) {
      const long long even = total + gridDim.x < 0x7fffffff
                                 ? (static_cast<unsigned>(total) + gridDim.x - 1) / gridDim.x
                                 : (total + gridDim.x - 1) / gridDim.x;
      const long long least = p.whole_units ? 1 : kTreeMinTiles;
      return even > least ? even : least;
    };
    if (threadIdx.x == 0 && !p.whole_units && !p.by_unit)
      p.ws_meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    // The sequence that the stretch starts in, and where in it.
    long long at = 0, each = 0;
    if (p.num_seqs <= 32) {  // every warp for itself
      TreeLens x = {};
      long long own = 0;
      if (lane < p.num_seqs) {
        x = tree_lens(p, lane);
        own = weight(x, blockIdx.x == 0 && warp == 0);
      }
      const long long upto = scan(own);
      each = each_of(__shfl_sync(kFullMask, upto, 31));
      const long long start = each * blockIdx.x;
      const unsigned in = __ballot_sync(kFullMask, start < upto && start >= upto - own);
      const int from = in != 0 ? __ffs(in) - 1 : 0;
      walk.seq = from;
      at = start - __shfl_sync(kFullMask, upto - own, from);
      walk.ahead = {__shfl_sync(kFullMask, x.ctx, from), __shfl_sync(kFullMask, x.q0, from),
                    __shfl_sync(kFullMask, x.end, from)};
      if (in == 0) each = 0;
      tc::tc_fence_before();
      __syncthreads();
    } else {
      const int per = (p.num_seqs + Tr::THREADS - 1) / Tr::THREADS;
      const int first = min(p.num_seqs, static_cast<int>(threadIdx.x) * per);
      const int last = min(p.num_seqs, first + per);
      long long own = 0;
      for (int i = first; i < last; ++i) own += weight(tree_lens(p, i), blockIdx.x == 0);
      long long upto = scan(own);
      long long* sums = reinterpret_cast<long long*>(smem + Tr::OFF_SEEN);
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      long long total = 0;
      for (int w = 0; w < Tr::THREADS / 32; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
      }
      each = each_of(total);
      const long long start = each * blockIdx.x;
      if (start < upto && start >= upto - own) {
        at = start - (upto - own);
        for (int i = first; i < last; ++i) {
          const TreeLens x = tree_lens(p, i);
          const long long w = weight(x, false);
          if (at < w) {
            s_found->seq = i;
            s_found->lens = x;
            s_found->at = at;
            break;
          }
          at -= w;
        }
      }
      tc::tc_fence_before();
      __syncthreads();
      walk.seq = s_found->seq;
      walk.ahead = s_found->lens;
      at = s_found->at;
      if (walk.seq < 0) each = 0;
    }
    // the line's end cuts the last stretch by itself
    len = static_cast<int>(each < 0x7fffffff ? each : 0x7fffffff);
    if (len > 0) {
      TreeSeq seq;
      tree_seq(p, walk.ahead, seq, false);
      const int head = tree_head_span<ROWS>(p, seq);
      const int full = tree_span<ROWS>(p, seq.ctx, ROWS);  // every row tile but the last
      walk.kvh = at < 0x7fffffff ? static_cast<int>(at) / head : static_cast<int>(at / head);
      const int in_head = static_cast<int>(at - static_cast<long long>(walk.kvh) * head);
      walk.rt = min(in_head / full, ((seq.q_len << p.group_shift) - 1) / ROWS);
      walk.at = in_head - walk.rt * full;
    }
  }
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFullMask, static_cast<uint32_t>(words[0]), 0);
  if (len == 0) {
    if (warp == 1) tc::tmem_dealloc(tmem, Tr::TMEM_COLS);
    return;
  }
  walk.left = len;
  walk.loaded = false;

  // rows of query tile q of an item
  auto rows_of = [&](const TreeItem& it, int q) {
    return min(M, (it.q_len << p.group_shift) - it.rt * ROWS - q * M);
  };
  // Where a unit has at most 128 rows, the two groups of softmax warps of a QT = 2
  // CTA take its tiles in turn, each with its own S, P and O.
  auto in_turn = [&](const TreeItem& x) { return QT == 2 && rows_of(x, 1) <= 0; };
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
    // 32 entries of an item's table row at a time (those past the context are
    // not used), an item's first ones while the item before it is under way
    auto entries = [&](const TreeItem& x, int chunk) {
      const int i = (chunk << 5) + lane;
      return i < p.max_blocks_per_seq
                 ? p.block_tables[static_cast<size_t>(x.seq) * p.max_blocks_per_seq + i]
                 : -1;
    };
    auto first_chunk = [&](const TreeItem& x) { return (x.t0 * NKEY) >> (shift + 5); };
    TreeItem nx;
    bool more = walk.next(p, nx);
    int ahead = p.direct ? early : more ? entries(nx, first_chunk(nx)) : -1;
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
    // ---- MMA issuers: S (warp 1) and P.V (warp 3) --------------------------------------
    // The whole warp runs the loop and one elected thread issues: with the loop's
    // values the same in all lanes, the descriptors stay in uniform registers,
    // where the MMA wants them.  (One lane alone in the loop moved each of them
    // there anew: 557 cycles for the 8 MMAs of an S, now 403.)
    bool ok = true;
    const uint64_t d_q = tc::smem_desc_sw128(sbase, 16, 1024);
    const uint64_t d_k = tc::smem_desc_sw128(sbase + Tr::OFF_KV, 16, 1024);
    const uint64_t d_v = tc::smem_desc_sw128(sbase + Tr::OFF_KV + Tr::KV_TILE, Tr::KV_HALF, 1024);
    auto wait = [&](uint32_t barrier, int parity) {
      ok = __all_sync(kFullMask, mbar_wait_bounded(barrier, parity & 1));
    };
    int gt = 0;
    int tg[QT] = {}, ig[QT] = {}, iq[QT] = {};  // tiles, items of each group; Q tiles loaded
    while (ok && walk.next(p, it)) {
      const bool alt = __any_sync(kFullMask, in_turn(it));
      const int ntiles = __shfl_sync(kFullMask, it.t1 - it.t0, 0);
      // the first tile with keys that not every row sees
      const int whole = __shfl_sync(kFullMask, max(0, (it.ctx - it.q_len) / NKEY - it.t0), 0);
      if (warp == 1) {
#pragma unroll
        for (int q = 0; q < QT; ++q) {
          if (!ok || (q > 0 && alt)) continue;
          wait(bar_q(q), iq[q]);
          ++iq[q];
        }
        for (int i = 0; ok && i < ntiles; ++i, ++gt) {
          wait(bar(Tr::B_KFULL + gt % NS), gt / NS);
          const uint64_t k0 = d_k + static_cast<uint32_t>((gt % NS) * (Tr::STAGE >> 4));
#pragma unroll
          for (int g = 0; g < QT; ++g) {
            if (!ok || (alt && (i & 1) != g)) continue;
            const int b = tg[g] & 1;
            // the buffer holds P of the group's tile before last until P.V has read it
            if (tg[g] >= 2) wait(bar_o(g, b), (tg[g] - 2) >> 1);
            if (!ok) break;
            tc::tc_fence_after();
            const uint64_t q0d = d_q + (alt ? 0 : g) * (Tr::Q_TILE >> 4);
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t step = (ks >> 2) * (Tr::Q_HALF >> 4) + (ks & 3) * 2;
                const uint32_t kstep = (ks >> 2) * (Tr::KV_HALF >> 4) + (ks & 3) * 2;
                tc::umma_f16(tmem + g * Tr::QCOLS + b * NKEY, q0d + step, k0 + kstep, IDESC_S,
                             ks > 0 ? 1u : 0u);
              }
              tc::umma_commit(bar_s(g, b));
            }
            __syncwarp();
            ++tg[g];
          }
          if (ok && elect_one()) tc::umma_commit(bar(Tr::B_KEMPTY + gt % NS));
          __syncwarp();
        }
      } else {
        for (int i = 0; ok && i < ntiles; ++i, ++gt) {
          wait(bar(Tr::B_VFULL + gt % NS), gt / NS);
          if (!ok) break;
          // The softmax of every group that the tile goes to clears V rows of a
          // cut tile.  It is told here that they are in: this warp alone passes
          // every tile's barrier in turn, and so cannot mistake an earlier phase.
          const bool cut = i >= whole;
          if (cut && lane == 0) {
#pragma unroll
            for (int g = 0; g < QT; ++g)
              if (!alt || (i & 1) == g) mbar_arrive(bar(Tr::B_VREADY + g));
          }
          const bool all_p = !alt && (cut || i == ntiles - 1);
          if (all_p) {
#pragma unroll
            for (int g = 0; g < QT; ++g)
              if (ok) wait(bar_p(g, tg[g] & 1), tg[g] >> 1);
          }
          const uint64_t v0 = d_v + static_cast<uint32_t>((gt % NS) * (Tr::STAGE >> 4));
#pragma unroll
          for (int g = 0; g < QT; ++g) {
            if (!ok || (alt && (i & 1) != g)) continue;
            const int b = tg[g] & 1;
            const bool first = i == (alt ? g : 0);
            if (!all_p) wait(bar_p(g, b), tg[g] >> 1);
            // the first tile overwrites the group's O of the item before
            if (first) {
              if (ok && ig[g] > 0) wait(bar_ofree(g), ig[g] - 1);
              ++ig[g];
            }
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t ptm = tmem + g * Tr::QCOLS + b * NKEY;
            const uint32_t otm = tmem + g * Tr::QCOLS + Tr::O_COL;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < NKEY / 16; ++kk) {
                const uint64_t bdesc = v0 + kk * (2048 >> 4);
                tc::umma_f16_ts(otm, ptm + 8 * kk, bdesc, IDESC_O, (!first || kk > 0) ? 1u : 0u);
                if constexpr (Tr::kBf16)
                  tc::umma_f16_ts(otm, ptm + NKEY / 2 + 8 * kk, bdesc, IDESC_O, 1u);
              }
              tc::umma_commit(bar_o(g, b));
            }
            __syncwarp();
            ++tg[g];
          }
          if (ok && elect_one()) tc::umma_commit(bar(Tr::B_VEMPTY + gt % NS));
          __syncwarp();
        }
      }
    }
    if (!ok && elect_one()) {
      set_err(p.err, PKV_DEVERR_TIMEOUT);
      // what was issued completes before TMEM is freed
      const uint32_t drain = bar(Tr::B_DRAIN + (warp == 1 ? 0 : 1));
      tc::umma_commit(drain);
      (void)mbar_wait_bounded(drain, 0);
    }
    __syncwarp();
  } else if (warp < Tr::WIDEN_WARP) {
    // ---- softmax warps: group g, thread <-> row <-> TMEM lane --------------------------
    const int g = (warp - Tr::SOFTMAX_WARP) >> 2;
    const int quarter = warp & 3;  // the TMEM lanes this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tm = tmem + g * Tr::QCOLS + lanes;
    uint32_t* seen = reinterpret_cast<uint32_t*>(smem + Tr::OFF_SEEN) + (g * M + r) * 8;
    int* par = reinterpret_cast<int*>(smem + Tr::OFF_PAR) + (g * 4 + quarter) * PKV_MAX_TREE_NODES;
    float2* s_ml = reinterpret_cast<float2*>(smem + Tr::OFF_ML);
    const int gmask = (1 << p.group_shift) - 1;
    // row `row` of the item's query tile qt in q and out
    auto row_at = [&](const TreeItem& x, int qt, int row) {
      const int c = x.rt * ROWS + qt * M + row;
      return static_cast<size_t>(x.q0 + (c >> p.group_shift)) * p.num_heads +
             (static_cast<size_t>(x.kvh) << p.group_shift) + (c & gmask);
    };
    // An item's query tiles and its tree's parents come by cp.async, the tiles
    // issued once the last S of the item before is complete; rows that do not
    // exist are left as they are (nobody reads their S).
    auto q_chunks = [&](const TreeItem& x, int qt, auto f) {
      constexpr int CH = D / 8;
      const int n = rows_of(x, qt) * CH;
#pragma unroll 2
      for (int i = r; i < n; i += 128) {
        const int row = i / CH, ch = i % CH;
        f(qt * Tr::Q_TILE + (ch >> 3) * Tr::Q_HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
          row, ch);
      }
    };
    auto begin_q = [&](const TreeItem& x, int qt) {
      q_chunks(x, qt, [&](int at, int row, int ch) {
        cp_async16(sbase + at, static_cast<const T*>(p.q) + row_at(x, qt, row) * D + ch * 8);
      });
    };
    // the parents of the nodes up to this warp's last row
    auto begin_parents = [&](const TreeItem& x) {
      const int qt = in_turn(x) ? 0 : g;
      const int rows = min(rows_of(x, qt), quarter * 32 + 32);
      if (rows <= quarter * 32 || !partial(x, x.t1 - 1)) return;
      const int nodes = ((x.rt * ROWS + qt * M + rows - 1) >> p.group_shift) + 1;
      for (int i = lane; i < nodes; i += 32)
        cp_async4(smem_addr(par + i), p.parents + x.q0 + i);
    };
    auto end_q = [&](const TreeItem& x, int qt) {
      cp_async_wait_all();
      if constexpr (Tr::kQToFp16)
        q_chunks(x, qt, [&](int at, int, int) {
          uint4* c = reinterpret_cast<uint4*>(smem + at);
          const uint4 u = *c;
          *c = make_uint4(bf16x2_to_f16x2_sat(u.x), bf16x2_to_f16x2_sat(u.y),
                          bf16x2_to_f16x2_sat(u.z), bf16x2_to_f16x2_sat(u.w));
        });
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q(qt));
    };
    // tiles of all items before, of this group, of group 1; items, those with an O
    // of this group, those that both groups share; this group's cut tiles
    int gt0 = 0, tg = 0, tg1 = 0, items = 0, ig = 0, shared_items = 0, cuts = 0;
    bool ok = true;
    TreeItem nx;
    bool more = walk.next(p, nx);
    if (more) {
      begin_parents(nx);
      if (g == 0 || !in_turn(nx)) {
        begin_q(nx, g);
        end_q(nx, g);
      }
    }
    while (ok && more) {
      it = nx;
      more = walk.next(p, nx);
      ++items;
      const bool alt = in_turn(it);
      const int qt = alt ? 0 : g, step = alt ? 2 : 1;
      const int ntiles = it.t1 - it.t0;
      const int nrows = rows_of(it, qt);
      const bool active = r < nrows;
      const bool warp_active = quarter * 32 < nrows;
      const int hist = it.ctx - it.q_len;
      // Who brings the next item's query tiles: a group brings its own, but after
      // an item taken in turn the group of the last tile brings both, for its S
      // is the last that reads them.
      const bool mine0 = more && (alt ? ((ntiles - 1) & 1) == g : g == 0);
      const bool mine1 = QT == 2 && more && !in_turn(nx) && (alt ? ((ntiles - 1) & 1) == g : g == 1);
      float k_scale = 1.f, v_scale = 1.f;
      if constexpr (Tr::kFp8) {
        k_scale = p.k_scales[it.kvh];
        v_scale = p.v_scales[it.kvh];
        if (!(k_scale > 0.f && k_scale < INFINITY && v_scale > 0.f && v_scale < INFINITY) &&
            r == 0)
          set_err(p.err, PKV_DEVERR_BAD_SCALE);
      }
      cp_async_wait_all();  // the parents that this thread loads
      __syncwarp();
      if (partial(it, it.t1 - 1)) {
        // the nodes that each row sees: itself, its parent, and so on
        if (active) {
          const int node = (it.rt * ROWS + qt * M + r) >> p.group_shift;
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
            const int x = par[n];
            if (x < -1 || x >= n) {
              set_err(p.err, PKV_DEVERR_BAD_TREE);
              break;
            }
            n = x;
          }
          seen[at] = bits;
        }
        __syncwarp();
        // only an item that ends its unit, and so has tree keys, is followed by another
        if (more) begin_parents(nx);
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
      // rows that do not exist keep a maximum that no value passes
      float m = active ? -INFINITY : INFINITY, l = 0.f;
      // x = s * qscale; for qscale > 0 the row's max of x is (max s) * qscale
      // exactly, so s is masked and reduced unscaled and the scale folds into
      // the exponent's multiply-add
      const float mult0 = p.qscale * k_scale;
      const float mult = mult0 > 0.f ? mult0 : 1.f;
      for (int t = it.t0 + (alt ? g : 0); t < it.t1; t += step, ++tg) {
        const int b = tg & 1, stage = gt0 + t - it.t0;
        ok = mbar_wait_bounded(bar_s(g, b), (tg >> 1) & 1);
        if (!__all_sync(kFullMask, ok)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        if (t == it.t1 - 1) {  // every S of this item is complete
          if (mine0) begin_q(nx, 0);
          if (mine1) begin_q(nx, 1);
        }
        const bool cut = partial(it, t);
        if (warp_active) {
          const uint32_t sbuf = tm + b * NKEY;
          // P of the tile: 2^(s mult - m) in 16 bits, two keys a word, and what
          // that rounds off for bf16; returns the sum
          uint32_t w[32], wl[Tr::kBf16 ? 32 : 1];
          auto weigh = [&](const float (&s)[32], int h, float neg_m, uint64_t (&sum2)[2]) {
            const uint64_t mult2 = tc::f2_pack(mult, mult), neg_m2 = tc::f2_pack(neg_m, neg_m);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float x, y;
              tc::f2_unpack(tc::f2_fma(tc::f2_pack(s[c], s[c + 1]), mult2, neg_m2), x, y);
              x = exp2_approx(x);
              y = exp2_approx(y);
              sum2[(c >> 1) & 1] = tc::f2_add(sum2[(c >> 1) & 1], tc::f2_pack(x, y));
              const uint32_t u = pack2(x, y, MT());
              w[h * 16 + c / 2] = u;
              if constexpr (Tr::kBf16)
                wl[h * 16 + c / 2] = pack2(x - __uint_as_float(u << 16),
                                           y - __uint_as_float(u & 0xffff0000u), Bf16());
            }
          };
          auto total = [&](const uint64_t (&sum2)[2]) {
            float a[4];
            tc::f2_unpack(sum2[0], a[0], a[1]);
            tc::f2_unpack(sum2[1], a[2], a[3]);
            return (a[0] + a[1]) + (a[2] + a[3]);
          };
          float s[2][32];
          tmem_ld32(sbuf, s[0]);
          tmem_ld32(sbuf + 32, s[1]);
          tc::tmem_wait_ld();
          if (cut || !(mult0 > 0.f)) {
            const unsigned long long bits = window(t);
            const uint32_t b0 = static_cast<uint32_t>(bits);
            const uint32_t b1 = static_cast<uint32_t>(bits >> 32);
            const float f = mult0 > 0.f ? 1.f : mult0;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              s[0][c] = b0 & (1u << c) ? s[0][c] * f : -INFINITY;
              s[1][c] = b1 & (1u << c) ? s[1][c] * f : -INFINITY;
            }
          }
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            mx4[0] = tc::max3(mx4[0], s[0][c], s[0][c + 1]);
            mx4[1] = tc::max3(mx4[1], s[0][c + 2], s[0][c + 3]);
            mx4[2] = tc::max3(mx4[2], s[1][c], s[1][c + 1]);
            mx4[3] = tc::max3(mx4[3], s[1][c + 2], s[1][c + 3]);
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * mult;
          float alpha = 1.f;
          if (mx > m + (Tr::kRescaleThreshold + Tr::kBias)) {
            const float top = mx - Tr::kBias;
            alpha = exp2_approx(m - top);  // 0 on the first tile (m = -inf)
            m = top;
          }
          const float neg_m = m == -INFINITY ? 0.f : -m;
          uint64_t sum2[2] = {0, 0};
          weigh(s[0], 0, neg_m, sum2);
          weigh(s[1], 1, neg_m, sum2);
          l = l * alpha + total(sum2);
          // P over S: 32 columns, and 32 of what bf16 rounded off
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = w[16 * h + e];
            tc::tmem_st16u(sbuf + 16 * h, x);
            if constexpr (Tr::kBf16) {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = wl[16 * h + e];
              tc::tmem_st16u(sbuf + NKEY / 2 + 16 * h, x);
            }
          }
          tc::tmem_wait_st();
          if (t - it.t0 >= step && __any_sync(kFullMask, alpha != 1.f)) {
            // O holds every earlier tile before it is rescaled
            ok = mbar_wait_bounded(bar_o(g, (tg - 1) & 1), ((tg - 1) >> 1) & 1);
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
          ok = mbar_wait_bounded(bar(Tr::B_VREADY + g), cuts++ & 1);
          if (!__all_sync(kFullMask, ok)) {
            ok = false;
            break;
          }
          // an element with all exponent bits set is infinite or NaN
          constexpr uint32_t kExp = Tr::kBf16 ? 0x7F807F80u : 0x7C007C00u;
          constexpr uint32_t kOne = Tr::kBf16 ? 0x00800080u : 0x04000400u;
          unsigned char* vt = smem + Tr::OFF_KV + (stage % NS) * Tr::STAGE + Tr::KV_TILE;
          const int from = max(0, hist - t * NKEY), end = it.ctx - t * NKEY;
          auto hit = [&](uint32_t x) { return ((x & kExp) + kOne) & 0x80008000u; };
          // 16-byte chunk k of this thread: row r / 8 + 16 (k / HALVES), half k % HALVES
          constexpr int CHUNKS = NKEY * 8 / 128 * HALVES;
          auto chunk = [&](int k) {
            return reinterpret_cast<uint4*>(vt + (k % HALVES) * Tr::KV_HALF + r * 16 +
                                            (k / HALVES) * 2048);
          };
          uint32_t odd = 0;
#pragma unroll
          for (int k = 0; k < CHUNKS; ++k) {
            const int row = r / 8 + 16 * (k / HALVES);
            const uint4 u = *chunk(k);
            if (row >= end)
              *chunk(k) = make_uint4(0u, 0u, 0u, 0u);
            else if (row >= from)
              odd |= hit(u.x) | hit(u.y) | hit(u.z) | hit(u.w);
          }
          if (odd != 0) {
            s_odd[items & 1] = items;  // before the elements are cleared
            __threadfence_block();
#pragma unroll 1
            for (int k = 0; k < CHUNKS; ++k) {
              const int row = r / 8 + 16 * (k / HALVES);
              uint32_t* at = reinterpret_cast<uint32_t*>(chunk(k));
              for (int e = 0; e < 4 && row >= from && row < end; ++e) {
                const uint32_t y = hit(at[e]);
                at[e] &= ~((y & 0x8000u ? 0xffffu : 0u) | (y >> 16 ? 0xffff0000u : 0u));
              }
            }
          }
          fence_proxy_async_smem();
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p(g, b));
      }
      if (!ok) break;
      if (mine0) end_q(nx, 0);
      if (mine1) end_q(nx, 1);
      const bool both = alt && ntiles > 1;  // the two groups share the item's tiles
      const int other = QT == 1 ? 0 : alt ? ntiles >> 1 : ntiles;
      gt0 += ntiles;
      if (alt && g == 1) {
        if (both) {
          // group 0 takes what this group has; it has read the last such
          if (ig > 0) ok = mbar_wait_bounded(bar_ofree(1), (ig - 1) & 1);
          ok = __all_sync(kFullMask, ok);
          if (!ok) break;
          s_ml[r] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Tr::B_BOTH));
          ++ig;
        }
        continue;
      }
      ++ig;
      tg1 += other;
      // ---- output ------------------------------------------------------------------
      ok = mbar_wait_bounded(bar_o(g, (tg - 1) & 1), ((tg - 1) >> 1) & 1);
      float f0 = 1.f, f1 = 0.f;
      if (both) {
        ok = ok && mbar_wait_bounded(bar(Tr::B_BOTH), shared_items++ & 1) &&
             mbar_wait_bounded(bar_o(1, (tg1 - 1) & 1), ((tg1 - 1) >> 1) & 1);
      }
      if (!__all_sync(kFullMask, ok)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      if (both) {
        const float2 x = s_ml[r];
        const float top = fmaxf(m, x.x);
        f0 = m == -INFINITY ? 0.f : exp2_approx(m - top);
        f1 = x.x == -INFINITY ? 0.f : exp2_approx(x.x - top);
        l = l * f0 + x.y * f1;
        m = top;
      }
      const bool whole = it.t0 == 0 && it.t1 == it.nt;
      const bool odd = *static_cast<volatile int*>(s_odd + (items & 1)) == items;
      const size_t row = row_at(it, qt, min(r, nrows - 1));
      // pieces: the one that starts a unit is its CTA's second, any other its first
      const size_t piece = static_cast<size_t>(blockIdx.x) * 2 + (it.t0 == 0 ? 1 : 0);
      bool from_history = false;
      if (warp_active) {
        const float inv = l > 0.f || l != l ? v_scale / l : 0.f;
        if (!whole && active) p.ws_ml[piece * ROWS + qt * M + r] = make_float2(l != l ? l : m, l);
        float top = 0.f;  // NaN if an element is
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(tm + Tr::O_COL + c, v);
          if (both) {
            float x[32];
            tmem_ld32(tm + Tr::QCOLS + Tr::O_COL + c, x);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = v[i] * f0 + x[i] * f1;
          } else {
            tc::tmem_wait_ld();
          }
          if constexpr (!Tr::kFp8) {
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              asm("max.NaN.f32 %0, %1, %2, %0;" : "+f"(top) : "f"(v[i]), "f"(v[i + 1]));
          }
          if (!active) continue;
          if (whole) {
            T* o = static_cast<T*>(p.out) + row * D + c;
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
              float x[8], y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = v[i + e] * inv, y[e] = v[i + 8 + e] * inv;
              const uint4 a = pack8(x, typename Tr::DT()), b = pack8(y, typename Tr::DT());
              if (p.out_aligned32) {
                store32(o + i, a, b);
              } else {
                *reinterpret_cast<uint4*>(o + i) = a;
                *reinterpret_cast<uint4*>(o + i + 8) = b;
              }
            }
          } else {
            // [D / 8][ROWS] of 8 floats: a warp's rows side by side
            uint4* o = reinterpret_cast<uint4*>(p.ws_o) + (piece * (D / 8) * ROWS + qt * M + r) * 2;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(v[i + e] * v_scale);
              store32(o + (c + i) / 8 * ROWS * 2, make_uint4(x[0], x[1], x[2], x[3]),
                      make_uint4(x[4], x[5], x[6], x[7]));
            }
          }
        }
        if constexpr (!Tr::kFp8) from_history = __any_sync(kFullMask, active && l == l && top != top);
      }
      const int32_t* trow = p.block_tables + static_cast<size_t>(it.seq) * p.max_blocks_per_seq;
      const bool mine = active && l == l;  // a row whose sum is NaN stays NaN
      if constexpr (!Tr::kFp8) {
        if (odd || from_history)
          tree_non_finite<T, D, ROWS>(
              p.v_cache, trow, p.num_blocks, p.num_kv_heads, it.kvh, p.block_size, hist,
              it.t0 * NKEY, min(it.ctx, it.t1 * NKEY), from_history, odd && mine ? seen : nullptr,
              mine && whole ? static_cast<T*>(p.out) + row * D : nullptr,
              mine && !whole ? p.ws_o + (piece * (D / 8) * ROWS + qt * M + r) * 8 : nullptr);
      } else if (odd && mine) {
        // NaN in the V of the nodes that this row sees (the history's is in O)
        const int lo = max(0, it.t0 * NKEY - hist), hi = min(it.q_len, it.t1 * NKEY - hist);
#pragma unroll 1
        for (int c = 0; c < D; ++c) {
          bool nan = false;
#pragma unroll 1
          for (int n = lo; n < hi; ++n) {
            if (!(seen[n >> 5] >> (n & 31) & 1u)) continue;
            const int key = hist + n;
            const int pb = trow[key / p.block_size];
            if (static_cast<unsigned>(pb) >= static_cast<unsigned>(p.num_blocks)) continue;
            const size_t at = ((static_cast<size_t>(pb) * p.num_kv_heads + it.kvh) *
                                   p.block_size + key % p.block_size) * D + c;
            nan |= (static_cast<const uint8_t*>(p.v_cache)[at] & 0x7F) == 0x7F;
          }
          if (!nan) continue;
          if (whole)
            static_cast<T*>(p.out)[row * D + c] = static_cast<T>(NAN);
          else
            p.ws_o[((piece * (D / 8) + c / 8) * ROWS + qt * M + r) * 8 + c % 8] = NAN;
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_ofree(g));
        if (both) mbar_arrive(bar_ofree(1));
      }
      if (g == 0 && r == 0 && it.t1 == it.nt && !p.whole_units) {
        // this CTA ends the unit; the one whose stretch holds the unit's first tile,
        // `lead` positions before this stretch's start, began it
        const int began = static_cast<int>(blockIdx.x) - (it.t0 > 0 ? (it.lead + len - 1) / len : 0);
        if (p.by_unit)
          p.ws_meta[(it.seq * p.num_kv_heads + it.kvh) * p.max_rts + it.rt] =
              make_int4(began, blockIdx.x, 0, 0);
        else if (it.t0 > 0)
          p.ws_meta[blockIdx.x] =
              make_int4(it.q0 + ((it.rt * ROWS) >> p.group_shift), it.kvh, began,
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
        // 128-byte rows come swizzled, of 64-byte rows not.  A step of 32 chunks
        // is 512 bytes of codes and 4 or 8 rows, so that the swizzle of a lane's
        // chunks repeats every second step or every one.
        constexpr int STEPS = CHUNKS / 32, RSTEP = 512 / D;  // rows a step
        const int row0 = part * (CHUNKS * 16 / D) + lane / (D / 16), c = lane % (D / 16);
        uint32_t x[STEPS][4];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
          const int r7 = (row0 + (D == 128 ? (k & 1) * 4 : 0)) & 7;
          const uint32_t from = D == 128 ? row0 * 128 + ((c ^ r7) << 4)
                                         : part * CHUNKS * 16 + lane * 16;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[k][0]), "=r"(x[k][1]), "=r"(x[k][2]), "=r"(x[k][3])
                       : "r"(src + from + k * 512)
                       : "memory");
        }
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
          const int r7 = (row0 + (D == 128 ? (k & 1) * 4 : 0)) & 7;
          const uint32_t to = dst + (c >> 2) * Tr::KV_HALF + row0 * 128 + k * RSTEP * 128;
          // the lanes of the second dim half store their second chunk first, so
          // that the 8 lanes of a row fill all its banks
          const bool swap = c >= 4;
          const uint32_t at = ((((c & 3) * 2) ^ r7) << 4) ^ (swap ? 16 : 0);
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            e4m3x4_to_f16x2(swap ? x[k][e ^ 2] : x[k][e], h[2 * e], h[2 * e + 1]);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + at), "r"(h[0]),
                       "r"(h[1]), "r"(h[2]), "r"(h[3])
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + (at ^ 16)),
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
// The piece of a unit's first CTA is that CTA's second, of every later one its
// first.  A thread has 4 dims of a row, two threads a sector of the pieces, which
// were stored 32 bytes a thread (16 at a time: LLaMA-7B batch 105.0 us instead of
// 103.1, E4M3 66.9 instead of 65.3).  SLICES sets of threads take every SLICES-th
// piece and meet in shared memory.  Block (i, j) takes entry i, of its groups of rows the j-th and
// every gridDim.y-th after.  It is bound by the latency of its loads: N of them
// are under way at once, 8 for units in many pieces, 3 where a unit has two or
// three, which leaves 8 blocks an SM (GQA chat batch 72.9 us with 8, 68.4 with 3).
constexpr int kTreeMergeThreads = 256;
template <int D, int ROWS, class DT, int SLICES>
__global__ void __launch_bounds__(kTreeMergeThreads, SLICES > 1 ? 1 : 8)
    paged_attn_tree_merge_kernel(const TreeParams p) {
  using T = typename DT::T;
  constexpr int PER = kTreeMergeThreads / SLICES;  // threads of a slice
  constexpr int RB = PER / (D / 4);                // rows of a block
  constexpr int N = SLICES > 1 ? 8 : 3;
  __shared__ float part[SLICES > 1 ? SLICES : 1][6][SLICES > 1 ? PER : 1];
  grid_dependency_wait();
  trigger_dependents();
  int4 e = p.ws_meta[blockIdx.x];
  const int slice = threadIdx.x / PER, t = threadIdx.x % PER;
  const int c4 = t % (D / 4);
  int last = static_cast<int>(blockIdx.x);
  if (p.by_unit) {
    const int seq = static_cast<int>(blockIdx.x) / (p.num_kv_heads * p.max_rts);
    const int rt = static_cast<int>(blockIdx.x) % p.max_rts;
    TreeSeq s;
    if (!tree_seq(p, tree_lens(p, seq), s, false)) return;
    last = e.y;
    // only what a CTA that gave up left unwritten is out of range
    if (e.x < 0 || e.x >= last || last >= p.num_ctas) return;
    e = make_int4(s.q0 + ((rt * ROWS) >> p.group_shift),
                  static_cast<int>(blockIdx.x) / p.max_rts % p.num_kv_heads, e.x,
                  min(ROWS, (s.q_len << p.group_shift) - rt * ROWS));
  }
  auto piece_of = [&](int c) { return static_cast<size_t>(c) * 2 + (c == e.z ? 1 : 0); };
  auto output_of = [&](int c, int r) {
    return reinterpret_cast<const float4*>(
        p.ws_o)[((piece_of(c) * (D / 8) + c4 / 2) * ROWS + r) * 2 + c4 % 2];
  };
  for (int r0 = static_cast<int>(blockIdx.y) * RB; r0 < e.w; r0 += RB * gridDim.y) {
    const int r = r0 + t / (D / 4);
    float big = -INFINITY, num[4] = {}, den = 0.f;
    auto add = [&](float m1, float l1, const float4& o) {
      const float m = m1 == -INFINITY ? big : fmaxf(big, m1);
      const float a = big == -INFINITY ? 0.f : exp2_approx(big - m);
      const float f = m1 == -INFINITY ? 0.f : exp2_approx(m1 - m);
      big = m;
      den = den * a + f * l1;
      num[0] = num[0] * a + f * o.x;
      num[1] = num[1] * a + f * o.y;
      num[2] = num[2] * a + f * o.z;
      num[3] = num[3] * a + f * o.w;
    };
    if (r < e.w) {
      for (int c0 = e.z + slice; c0 <= last; c0 += N * SLICES) {
        float2 ml[N];
        float4 o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = min(c0 + i * SLICES, last);
          ml[i] = p.ws_ml[piece_of(c) * ROWS + r];
          o[i] = output_of(c, r);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (c0 + i * SLICES <= last) add(ml[i].x, ml[i].y, o[i]);
      }
    }
    if constexpr (SLICES > 1) {
      __syncthreads();  // the sums of the rows before have been read
      part[slice][0][t] = den != den ? den : big;
      part[slice][1][t] = den;
#pragma unroll
      for (int i = 0; i < 4; ++i) part[slice][2 + i][t] = num[i];
      __syncthreads();
      if (slice > 0) continue;
      for (int k = 1; k < SLICES; ++k)
        add(part[k][0][t], part[k][1][t],
            make_float4(part[k][2][t], part[k][3][t], part[k][4][t], part[k][5][t]));
    }
    if (r >= e.w) continue;
    // A piece's infinity is V's own and stays, however small the piece's weight: where
    // a weight of 0 made it NaN, the element is the sum of the pieces' non-finite ones.
    const float any = (num[0] + num[1]) + (num[2] + num[3]);
    if (any != any && den == den) {
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int c = e.z; c <= last; ++c) {
        const float4 o = output_of(c, r);
        if (!(fabsf(o.x) < INFINITY)) sum.x += o.x;
        if (!(fabsf(o.y) < INFINITY)) sum.y += o.y;
        if (!(fabsf(o.z) < INFINITY)) sum.z += o.z;
        if (!(fabsf(o.w) < INFINITY)) sum.w += o.w;
      }
      if (num[0] != num[0]) num[0] = sum.x;
      if (num[1] != num[1]) num[1] = sum.y;
      if (num[2] != num[2]) num[2] = sum.z;
      if (num[3] != num[3]) num[3] = sum.w;
    }
    const float inv = den > 0.f || den != den ? 1.f / den : 0.f;
    T* out = static_cast<T*>(p.out) +
             (static_cast<size_t>(e.x + (r >> p.group_shift)) * p.num_heads +
              (static_cast<size_t>(e.y) << p.group_shift) + (r & ((1 << p.group_shift) - 1))) * D +
             c4 * 4;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack2(num[0] * inv, num[1] * inv, DT()),
                                                pack2(num[2] * inv, num[3] * inv, DT()));
  }
}

}  // namespace pkv

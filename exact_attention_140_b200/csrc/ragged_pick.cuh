// ragged_pick.cuh -- the sequences of an attention over packed tensors, and the
// work item of a given rank (see ragged_plan.cuh).
#pragma once
#include <cstdint>

#include "tiles.h"

namespace attn {

constexpr int kPlanItem = 8;   // ints of an item
constexpr int kPlanPiece = 12;  // ints of a piece of an item
constexpr int kPieceSeqs = 1024, kPieceItems = 1024;  // sequences and items that are cut into pieces, at most
constexpr int kPickPerLane = 4, kPickSeqs = 32 * kPickPerLane;

struct PlanParams {
  int* plan;           // the list, or nullptr: every block picks its own item
  int max_items;
  int n_seqs, Tq, Tk, max_q, max_kv;
  const int* cu_q;     // or nullptr: sequence s has the rows [s * max_q, (s + 1) * max_q)
  const int* cu_k;     // packed keys; nullptr: paged
  const int* kv_lens;  // paged, or (k_stride > 0) packed with sequence s at k_stride * s
  int k_stride;
  int rows_per_token;  // packed rows of a token (1 or the group size)
  int block_rows, bn;  // powers of two
  bool causal;
  unsigned int* err;
};

// Items of a sequence (nq, nk, nb blocks) that cost at least c key tiles: its last
// ones.  Block qb's last token is min(ceil((qb + 1) R / g), nq) - 1 (R rows a
// block, g a token); it sees more than (c - 1) bn keys iff the token is at least
// L = (c - 1) bn - nk + nq, so the blocks are those from floor(L g / R) on.
// R = 2^shift.
ATTN_HD int ragged_items_from(long long c, int nq, int nk, int nb, int bn, int shift, int g, bool causal) {
  if (c <= 0) return nb;
  const long long below = (c - 1) * bn;
  if (below >= nk) return 0;
  if (!causal) return nb;
  const long long L = below - nk + nq;
  if (L > nq - 1) return 0;
  return L <= 0 ? nb : nb - (int)((L * g) >> shift);
}

// Pieces.  The key tiles of all (item, head) pairs stand in one line, item by item,
// heads within an item, and are cut into runs of `share` tiles.  A pair with the
// tiles [a, a + c) lies in the runs first .. last; the piece in run v holds its tiles
// [lo, hi), and unless it is the whole pair its rows are partial, in slot 2 v where
// the pair ends in the run and 2 v + 1 where it goes on: a run holds one of each
// at most.
// T: long long, or unsigned where a line fits it (its division is much shorter).
template <class T>
struct PieceRuns {
  T first, last;
};
template <class T>
ATTN_HD PieceRuns<T> piece_runs(T a, T c, T share) {
  const T first = a / share;
  return PieceRuns<T>{first, c > 0 ? (a + c - 1) / share : first};
}
template <class T>
struct Piece {
  T lo, hi;
  int slot;  // -1: whole
};
template <class T>
ATTN_HD Piece<T> piece_of(T a, T c, T share, PieceRuns<T> r, T v) {
  Piece<T> x;
  x.lo = (v * share > a ? v * share : a) - a;
  x.hi = ((v + 1) * share < a + c ? (v + 1) * share : a + c) - a;
  x.slot = r.first == r.last ? -1 : (int)(2 * v + (v == r.last ? 0 : 1));
  return x;
}

#ifdef __CUDACC__
// A boundary pair of the device clamped to [0, total].
__device__ __forceinline__ int2 clamped_range(const int* cu, int s, int total, bool& bad) {
  int a = __ldg(cu + s), b = __ldg(cu + s + 1);
  if (a < 0 || b < a || b > total) {
    bad = true;
    a = a < 0 ? 0 : (a > total ? total : a);
    b = b < a ? a : (b > total ? total : b);
  }
  return make_int2(a, b);
}

// Query tokens [q0, q0 + nq) and keys [k0, k0 + nk) of sequence s, clamped to
// their arrays (paged: k0 = 0).
struct RaggedSeq {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ RaggedSeq ragged_seq(const PlanParams& p, int s, bool& bad) {
  RaggedSeq r;
  if (p.cu_q != nullptr) {
    const int2 q = clamped_range(p.cu_q, s, p.Tq, bad);
    r.q0 = q.x;
    r.nq = q.y - q.x;
  } else {
    r.q0 = s * p.max_q;
    r.nq = p.max_q;
  }
  if (r.nq > p.max_q) {
    bad = true;
    r.nq = p.max_q;
  }
  if (p.cu_k != nullptr) {
    const int2 k = clamped_range(p.cu_k, s, p.Tk, bad);
    r.k0 = k.x;
    r.nk = k.y - k.x;
  } else {
    r.k0 = s * p.k_stride;
    r.nk = __ldg(p.kv_lens + s);
    if (r.nk < 0 || r.nk > p.max_kv) {
      bad = true;
      r.nk = r.nk < 0 ? 0 : p.max_kv;
    }
  }
  return r;
}
__device__ __forceinline__ int ragged_blocks(const PlanParams& p, int nq) {
  return (int)(((long long)nq * p.rows_per_token + p.block_rows - 1) >> (31 - __clz(p.block_rows)));
}

// By one converged warp: the item of rank `rank` in falling order of cost, as
// {seq, block, q0, nq}, {k0, nk}; false if there are not that many.  n_seqs <=
// kPickSeqs; lane i holds the sequences i, i + 32, ...
__device__ __forceinline__ bool ragged_pick(const PlanParams& p, int rank, int4& a, int2& b) {
  const int lane = (int)(threadIdx.x & 31);
  RaggedSeq r[kPickPerLane];
  int nb[kPickPerLane];
  bool bad = false;
  int all = 0, most = 0;
#pragma unroll
  for (int i = 0; i < kPickPerLane; ++i) {
    const int s = lane + 32 * i;
    r[i] = RaggedSeq{0, 0, 0, 0};
    if (s < p.n_seqs) r[i] = ragged_seq(p, s, bad);
    nb[i] = ragged_blocks(p, r[i].nq);
    all += nb[i];
    if (nb[i] > 0) most = max(most, (r[i].nk + p.bn - 1) >> (31 - __clz(p.bn)));
  }
  if (bad) atomicOr(p.err, 2u);
  all = __reduce_add_sync(0xffffffffu, all);
  most = __reduce_max_sync(0xffffffffu, most);
  if (rank >= all) return false;
  const int shift = 31 - __clz(p.block_rows);
  auto from = [&](int c, int i) -> int {
    return ragged_items_from(c, r[i].nq, r[i].nk, nb[i], p.bn, shift, p.rows_per_token, p.causal);
  };
  int lo = 0, hi = most;  // the largest c with more than `rank` items of at least c
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPickPerLane; ++i)
      if (32 * i < p.n_seqs) n += from(mid, i);
    n = __reduce_add_sync(0xffffffffu, n);
    if (n > rank) lo = mid; else hi = mid - 1;
  }
  // among the items of cost lo, sequence by sequence
  int above = 0;
#pragma unroll
  for (int i = 0; i < kPickPerLane; ++i) above += from(lo + 1, i);
  int left = rank - __reduce_add_sync(0xffffffffu, above);
#pragma unroll
  for (int i = 0; i < kPickPerLane; ++i) {
    const int f = from(lo, i), e = f - from(lo + 1, i);
    int upto = e;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    if (left < total) {
      const int src = __ffs(__ballot_sync(0xffffffffu, left < upto)) - 1;
      const int qb = nb[i] - f + (left - (upto - e));
      a = make_int4(src + 32 * i, __shfl_sync(0xffffffffu, qb, src), __shfl_sync(0xffffffffu, r[i].q0, src),
                    __shfl_sync(0xffffffffu, r[i].nq, src));
      b = make_int2(__shfl_sync(0xffffffffu, r[i].k0, src), __shfl_sync(0xffffffffu, r[i].nk, src));
      return true;
    }
    left -= total;
  }
  return false;
}
#endif

}  // namespace attn

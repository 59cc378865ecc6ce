// ragged_plan.cuh -- the work items of an attention over packed sequences: one
// item per (sequence, block of query rows), longest first.
//
// The lengths live on the device, so the host cannot list the items.  An item's
// cost is the number of key tiles its last row sees.  One block lists them ahead of
// the attention kernel (whose launch overlaps it) by a counting sort over
// kPlanBuckets levels of cost (the order within a level is arbitrary and does not
// affect any result); that kernel takes 5 us.  In a small call every block of the
// attention kernel finds its own item instead (ragged_pick): within a sequence the
// cost grows with the block, so the number of items that cost at least c has a
// closed form for each sequence, and a bisection over c with a warp's sum over the
// sequences finds the item of a given rank.  That takes every block about 1 us,
// so a call of more blocks than SMs has the list.
//
// Where the blocks are few or the contexts long, whole items would leave SMs
// without work: piece_plan_kernel cuts the key tiles of all of them into one equal
// run per SM, and lists the pieces longest first.  Pieces of an SM's run add up to
// the run, so handing out the longest first fits them together again: the block
// that ends first meets the longest piece left.  The rows of cut items are merged
// by long_combine_kernel.
#pragma once
#include <cstdint>

#include "attn_common.cuh"
#include "ptx.cuh"
#include "tiles.h"

namespace attn {

constexpr int kPlanThreads = 512;
constexpr int kPlanBuckets = 256;

// Exclusive prefix sum over the block's threads; `all` is the total.
template <class T>
__device__ __forceinline__ T block_scan(T mine, T* s_warp, T& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  T front = 0;
  all = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    if (i < warp) front += s_warp[i];
    all += s_warp[i];
  }
  __syncthreads();
  return front + x - mine;
}

// Key tiles that the last row of a sequence's block qb sees.
__device__ __forceinline__ int block_cost(const PlanParams& p, int qb, int nq, int nk) {
  const unsigned end = ((unsigned)(qb + 1) * (unsigned)p.block_rows + p.rows_per_token - 1) / (unsigned)p.rows_per_token;
  return (int)((vis_end((end < (unsigned)nq ? (int)end : nq) - 1, nq, nk, p.causal) + p.bn - 1) >> (31 - __clz(p.bn)));
}
// Counts per level to the places where the levels begin; returns their sum.
__device__ __forceinline__ int level_starts(int* hist, int* s_warp) {
  static_assert(kPlanBuckets <= kPlanThreads, "a thread per level");
  const int i = threadIdx.x;
  int all;
  const int at = block_scan(i < kPlanBuckets ? hist[i] : 0, s_warp, all);
  if (i < kPlanBuckets) hist[i] = at;
  __syncthreads();
  return all;
}

__global__ void __launch_bounds__(kPlanThreads) ragged_plan_kernel(const PlanParams p) {
  __shared__ int s_hist[kPlanBuckets], s_sum[kPlanThreads / 32], s_max;
  ptx::grid_dep_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NW = kPlanThreads / 32;
  for (int i = tid; i < kPlanBuckets; i += kPlanThreads) s_hist[i] = 0;
  if (tid == 0) s_max = 0;
  __syncthreads();
  bool bad = false;
  auto seq = [&](int s, int& q0, int& nq, int& k0, int& nk) {
    const RaggedSeq r = ragged_seq(p, s, bad);
    q0 = r.q0;
    nq = r.nq;
    k0 = r.k0;
    nk = r.nk;
  };
  auto blocks_of = [&](int nq) -> int { return ragged_blocks(p, nq); };
  auto cost = [&](int qb, int nq, int nk) -> int { return block_cost(p, qb, nq, nk); };
  // the largest cost: every sequence's last block
  int mx = 0;
  for (int s = tid; s < p.n_seqs; s += kPlanThreads) {
    int q0, nq, k0, nk;
    seq(s, q0, nq, k0, nk);
    const int nb = blocks_of(nq);
    if (nb > 0) {
      const int c = cost(nb - 1, nq, nk);
      mx = c > mx ? c : mx;
    }
  }
  atomicMax(&s_max, mx);
  __syncthreads();
  const long long top = s_max + 1;
  auto level = [&](int c) -> int { return kPlanBuckets - 1 - (int)((long long)c * kPlanBuckets / top); };
  // two passes over all items: count per level, then place
  for (int s = warp; s < p.n_seqs; s += NW) {
    int q0, nq, k0, nk;
    seq(s, q0, nq, k0, nk);
    const int nb = blocks_of(nq);
    for (int qb = lane; qb < nb; qb += 32) atomicAdd(&s_hist[level(cost(qb, nq, nk))], 1);
  }
  __syncthreads();
  const int count = level_starts(s_hist, s_sum);
  for (int s = warp; s < p.n_seqs; s += NW) {
    int q0, nq, k0, nk;
    seq(s, q0, nq, k0, nk);
    const int nb = blocks_of(nq);
    for (int qb = lane; qb < nb; qb += 32) {
      const int at = atomicAdd(&s_hist[level(cost(qb, nq, nk))], 1);
      if (at < p.max_items) {
        int4* it = reinterpret_cast<int4*>(p.plan + kPlanItem * at);
        it[0] = make_int4(s, qb, q0, nq);
        it[1] = make_int4(k0, nk, 0, 0);
      } else {
        bad = true;  // (boundaries that overlap)
      }
    }
  }
  // the slots behind the last item say so themselves: a block of the attention
  // kernel then needs one look
  for (int i = count + tid; i < p.max_items; i += kPlanThreads) p.plan[kPlanItem * i] = -1;
  if (bad) atomicOr(p.err, kErrIndex);
}

struct PiecePlanParams {
  PlanParams seqs;  // plan: max_pieces pieces of 12 ints: seq (-1: none), block, q0, nq, k0, nk, head, slot, first
                    // and end key tile, 0, 0
  int max_pieces, nh, runs, min_share;
  long long* lin;   // [max_items + 2]: tiles in front of each item (of one head) and of all; [max_items + 1]: a run
  int* first;       // [n_seqs + 1]: items in front of each sequence, and of all
};

__global__ void __launch_bounds__(kPlanThreads) piece_plan_kernel(const PiecePlanParams pp) {
  const PlanParams& p = pp.seqs;
  constexpr int PER = kPieceSeqs / kPlanThreads, IPER = kPieceItems / kPlanThreads;
  __shared__ int4 s_seq[kPieceSeqs];            // q0, nq, k0, nk
  __shared__ int s_first[kPieceSeqs + 1], s_hist[kPlanBuckets], s_warp[kPlanThreads / 32];
  __shared__ short s_of[kPieceItems];           // an item's sequence
  __shared__ long long s_lin[kPieceItems + 1], s_sum[kPlanThreads / 32];
  ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  for (int i = tid; i < kPlanBuckets; i += kPlanThreads) s_hist[i] = 0;
  bool bad = false;
  long long nb[PER], mine = 0, all;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int s = PER * tid + u;
    nb[u] = 0;
    if (s < p.n_seqs) {
      const RaggedSeq r = ragged_seq(p, s, bad);
      s_seq[s] = make_int4(r.q0, r.nq, r.k0, r.nk);
      nb[u] = ragged_blocks(p, r.nq);
    }
    mine += nb[u];
  }
  long long at = block_scan(mine, s_sum, all);
  if (all > p.max_items) bad = true;  // (boundaries that overlap)
  const int n_items = all < p.max_items ? (int)all : p.max_items;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int s = PER * tid + u;
    const int f = at < n_items ? (int)at : n_items;
    if (s < p.n_seqs) s_first[s] = pp.first[s] = f;
    at += nb[u];
  }
  if (tid == 0) s_first[p.n_seqs] = pp.first[p.n_seqs] = n_items;
  __syncthreads();
  auto seq_of = [&](int item) -> int {  // the last s with s_first[s] <= item
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (s_first[mid] <= item) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  long long cost[IPER];
  mine = 0;
#pragma unroll
  for (int u = 0; u < IPER; ++u) {
    const int item = IPER * tid + u;
    cost[u] = 0;
    if (item < n_items) {  // key tiles of the block's last row
      const int s = seq_of(item);
      s_of[item] = (short)s;
      const int4 x = s_seq[s];
      cost[u] = block_cost(p, item - s_first[s], x.y, x.w);
    }
    mine += cost[u];
  }
  at = block_scan(mine, s_sum, all);
#pragma unroll
  for (int u = 0; u < IPER; ++u) {
    const int item = IPER * tid + u;
    if (item < n_items) s_lin[item] = pp.lin[item] = at;
    at += cost[u];
  }
  long long share = (all * pp.nh + pp.runs - 1) / pp.runs;
  share = share < pp.min_share ? pp.min_share : share;
  if (tid == 0) {
    s_lin[n_items] = pp.lin[n_items] = all;
    pp.lin[p.max_items + 1] = share;
  }
  __syncthreads();
  const int pairs = n_items * pp.nh;
  const bool small = all * pp.nh < (1ll << 31) && share < (1ll << 23);
  auto each_in = [&](auto zero, auto&& f) {
    using T = decltype(zero);
    const T sh = (T)share;
    for (int x = tid; x < pairs; x += kPlanThreads) {
      const int item = x / pp.nh, hy = x - item * pp.nh;
      const T front = (T)s_lin[item], c = (T)s_lin[item + 1] - front, a = front * (T)pp.nh + (T)hy * c;
      const PieceRuns<T> r = piece_runs<T>(a, c, sh);
      for (T v = r.first; v <= r.last; ++v) {
        const Piece<T> y = piece_of<T>(a, c, sh, r, v);
        f(item, hy, (int)y.lo, (int)y.hi, y.slot, kPlanBuckets - 1 - (int)((y.hi - y.lo) * kPlanBuckets / (sh + 1)));
      }
    }
  };
  auto each = [&](auto&& f) {
    if (small) each_in(0u, f); else each_in(0ll, f);
  };
  each([&](int, int, int, int, int, int level) { atomicAdd(&s_hist[level], 1); });
  __syncthreads();
  const int count = level_starts(s_hist, s_warp);
  each([&](int item, int hy, int lo, int hi, int slot, int level) {
    const int i = atomicAdd(&s_hist[level], 1);
    if (i >= pp.max_pieces) return;  // (never: at most one more than the pairs for every cut)
    const int s = s_of[item];
    const int4 q = s_seq[s];
    int4* to = reinterpret_cast<int4*>(p.plan + kPlanPiece * i);
    to[0] = make_int4(s, item - s_first[s], q.x, q.y);
    to[1] = make_int4(q.z, q.w, hy, slot);
    to[2] = make_int4(lo, hi, 0, 0);
  });
  for (int i = count + tid; i < pp.max_pieces; i += kPlanThreads) p.plan[kPlanPiece * i] = -1;
  if (bad) atomicOr(p.err, kErrIndex);
}

}  // namespace attn

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
#pragma once
#include <cstdint>

#include "attn_common.cuh"
#include "ptx.cuh"
#include "tiles.h"

namespace attn {

constexpr int kPlanThreads = 512;
constexpr int kPlanBuckets = 256;

__global__ void __launch_bounds__(kPlanThreads) ragged_plan_kernel(const PlanParams p) {
  __shared__ int s_hist[kPlanBuckets], s_max, s_count;
  ptx::grid_dep_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NW = kPlanThreads / 32;
  for (int i = tid; i < kPlanBuckets; i += kPlanThreads) s_hist[i] = 0;
  if (tid == 0) s_max = s_count = 0;
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
  auto cost = [&](int qb, int nq, int nk) -> int {  // key tiles of the block's last row
    const int last = (int)((((long long)(qb + 1) * p.block_rows) + p.rows_per_token - 1) / p.rows_per_token);
    return (int)((vis_end((last < nq ? last : nq) - 1, nq, nk, p.causal) + p.bn - 1) / p.bn);
  };
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
  if (warp == 0) {  // exclusive prefix sums of the levels
    int base = 0;
    for (int i = 0; i < kPlanBuckets; i += 32) {
      const int v = s_hist[i + lane];
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      s_hist[i + lane] = base + x - v;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_count = base;
  }
  __syncthreads();
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
  for (int i = s_count + tid; i < p.max_items; i += kPlanThreads) p.plan[kPlanItem * i] = -1;
  if (bad) atomicOr(p.err, kErrIndex);
}

}  // namespace attn

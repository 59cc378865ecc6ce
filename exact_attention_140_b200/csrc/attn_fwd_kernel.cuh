// attn_fwd_kernel.cuh -- fused exact-attention forward for sm_100a.
//
// One CTA computes NQT query tiles of 128 rows for one (batch, query head).
// It walks the key/value tiles of that head once, keeping the output
// accumulator on chip, so neither the score matrix nor partial outputs ever
// reach HBM (page "FlashAttention (SV)": tiling, online softmax and operator
// fusion; the query-tile-outer loop order is the one page "FlashAttention-4
// 震撼发布" credits to FlashAttention-2's re-partitioned work).
//
// Warp roles (warp specialisation, page "FlashAttention-3 — 闪电注意力-3",
// section 1, recast for tcgen05):
//   warps 0 .. 4*NQT-1  softmax: warp w serves query tile w/4 and TMEM lanes
//                       32*(w%4) .. +31, so thread = one query row;
//   warp 4*NQT          TMA producer: Q tiles once, then K_j and V_j through
//                       KST / VST-stage shared-memory rings (section 2: the
//                       next block is fetched while the current one computes);
//   warp 4*NQT+1        MMA issuer: the warp runs the issue loop and one
//                       elected lane issues every tcgen05.mma; it also
//                       allocates and frees tensor memory;
//   warps 4*NQT+2, +3   idle (they complete the control warpgroup, whose
//                       registers are handed to the softmax warpgroups).
//
// Tensor memory (128 lanes x 512 fp32 columns): per query tile t, SB score
// buffers S of BN columns (P overwrites S in place: BN/2 columns of packed
// bf16, or BN/4 of e4m3) and the output accumulator O of D columns.  With two
// query tiles (NQT = 2) the tensor core alternates between them, so one
// tile's softmax runs under the other's matrix products (the ping-pong idea
// of section 1); with one tile the score buffer is doubled instead (SB = 2)
// so S_{j+1} = Q K_{j+1}^T runs under the softmax of S_j.
//
// Per key tile j and query tile t:
//   S   = Q_t K_j^T                          (tcgen05, SS operands, fp32 in TMEM)
//   m_b = rowmax(scale*log2e * S)            (masked on partial tiles)
//   if m_b > m_ref + TAU: rescale O_t and l by 2^(m_ref - m_b), m_ref = m_b
//   P   = 2^(scale*log2e * S - m_ref);  l += rowsum(P)
//   O_t += P V_j                             (tcgen05, A = P from TMEM)
// The reference max only moves when the block max exceeds it by more than
// TAU (lazy rescaling; page "FlashAttention-4震撼发布", the new online
// softmax that skips most output rescalings).  The result is the same for any
// TAU because the reference cancels in O = acc / l; TAU = 8 bounds P by 2^8.
// Epilogue: O = O_t / l (bf16), LSE = ln2 * (m_ref + log2 l).
//
// Split-KV (launch parameters n_splits, kv_chunk, o_part, lse_part): a block
// then covers one window of the keys (grid z = batch x window; the tile plan
// is shifted so that the causal rule keeps absolute key indices) and writes
// fp32 partials O_s = O_t / l and LSE_s for attn_combine.  With head packing
// (PACK configurations, launch parameter pack = g) the g query heads of one
// key/value head share the query tiles: query row i of head h sits at tile
// row i * g + h % g, and grid y runs over key/value heads.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "attn_common.cuh"
#include "e4m3.cuh"
#include "exp2_soft.cuh"
#include "ptx.cuh"
#include "tiles.h"

namespace attn {



template <class Cfg>
__global__ void __launch_bounds__(Cfg::NTHREADS, Cfg::BPS)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const typename Cfg::Params p) {
  constexpr int BM = Cfg::BM, BN = Cfg::BN, D = Cfg::D, NQT = Cfg::NQT, SB = Cfg::SB;
  static_assert(!Cfg::PSEP, "P overwrites S in this kernel");
  constexpr int KST = Cfg::KST, VST = Cfg::VST;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw_u32);
  auto bar = [&](int i) -> uint32_t { return sbase + Cfg::OFF_BAR + 8u * (uint32_t)i; };
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(sgen + Cfg::OFF_ABORT);
  const WaitCtx wc{abort_flag, p.err, p.timeout_ns};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = Cfg::PACK ? p.pack : 1;  // query heads stacked per tile row group
  int qb, hy, b, split;
  int nq = p.Nq, nk_all = p.Nk;                       // query rows and keys of the item's sequence
  [[maybe_unused]] int q_base = 0, k_base = 0, seq = 0;  // RAGGED: its first query token and key, its index
  [[maybe_unused]] int slot = -1, kv_begin = 0, kv_end = 0;  // RAGGED: its partial rows (-1: none), its keys
  if constexpr (Cfg::RAGGED != 0) {
    // bands of heads as below, the listed items (longest first) within a band
    ptx::grid_dep_launch();
    split = (int)blockIdx.x % p.n_splits;  // (1 with pieces)
    const int L = (int)blockIdx.x / p.n_splits, per = p.band * p.rg.seqs.max_items;
    const int bi = p.rg.pieces ? 0 : L / per, within = L - bi * per;
    const int bsz = p.nh - bi * p.band < p.band ? p.nh - bi * p.band : p.band;
    const int item = within / bsz;
    hy = bi * p.band + within % bsz;
    int4 i0;
    int2 i1;
    if (p.rg.pieces) {
      ptx::grid_dep_wait();
      const int4* it = reinterpret_cast<const int4*>(p.rg.seqs.plan) + 3 * L;
      i0 = __ldcg(it);
      const int4 i2 = __ldcg(it + 1);
      const int2 i3 = __ldcg(reinterpret_cast<const int2*>(it + 2));
      i1 = make_int2(i2.x, i2.y);
      hy = i2.z;
      slot = i2.w;
      kv_begin = i3.x * BN;
      kv_end = i3.y;
    } else if (p.rg.seqs.plan == nullptr) {
      int* s_item = reinterpret_cast<int*>(sgen);  // (nothing has been loaded yet)
      if (warp == 0) {
        const bool there = ragged_pick(p.rg.seqs, item, i0, i1);
        if (lane == 0) {
          s_item[0] = there ? i0.x : -1;
          if (there) {
            s_item[1] = i0.y;
            s_item[2] = i0.z;
            s_item[3] = i0.w;
            s_item[4] = i1.x;
            s_item[5] = i1.y;
          }
        }
      }
      __syncthreads();
      // (all have read it before the first load lands there: the barrier below comes between)
      i0 = make_int4(s_item[0], s_item[1], s_item[2], s_item[3]);
      i1 = make_int2(s_item[4], s_item[5]);
    } else {
      ptx::grid_dep_wait();
      // (from L2: the list was written while this grid was being launched)
      i0 = __ldcg(reinterpret_cast<const int4*>(p.rg.seqs.plan) + 2 * item);
      i1 = __ldcg(reinterpret_cast<const int2*>(p.rg.seqs.plan) + 2 + 4 * item);
    }
    if (i0.x < 0) return;
    b = 0;
    // (a shuffle from lane 0 shows the compiler that the warp agrees on them, so
    // that loops and descriptors stay in uniform registers)
    auto uni = [](int v) -> int { return __shfl_sync(0xffffffffu, v, 0); };
    seq = uni(i0.x);
    qb = uni(i0.y);
    q_base = uni(i0.z);
    nq = uni(i0.w);
    k_base = uni(i1.x);
    nk_all = uni(i1.y);
    if (p.rg.pieces) {
      hy = uni(hy);
      slot = uni(slot);
      kv_begin = uni(kv_begin);
      kv_end = (long long)uni(kv_end) * BN < nk_all ? uni(kv_end) * BN : nk_all;
    } else {
      kv_begin = split * p.kv_chunk;
      if (split > 0 && kv_begin >= nk_all) return;  // no such window
      kv_end = nk_all - kv_begin < p.kv_chunk ? nk_all : kv_begin + p.kv_chunk;
      slot = nk_all > p.kv_chunk ? split : -1;
    }
  } else if (p.band > 0) {
    // longest-first within bands of (batch, head) pairs: a band's K/V stay in
    // L2 while its blocks run, and the hardware hands out blocks in this
    // order as SMs free up, so the long causal blocks do not end up last
    const int L = (int)blockIdx.x, nbh = p.nb * p.nh;
    const int bi = L / (p.band * p.n_qblocks);
    const int within = L - bi * p.band * p.n_qblocks;
    const int bsz = nbh - bi * p.band < p.band ? nbh - bi * p.band : p.band;
    const int r = bi * p.band + within % bsz;
    qb = p.n_qblocks - 1 - within / bsz;
    hy = p.h0 + r % p.nh;
    b = p.b0 + r / p.nh;
    split = 0;
  } else {
    qb = p.n_qblocks - 1 - (int)blockIdx.x;  // longest causal blocks first
    // query head, or key/value head when packed (grid y covers the launch's heads)
    hy = (g > 1 ? p.h0 / g : p.h0) + (int)blockIdx.y;
    b = p.b0 + (int)blockIdx.z / p.n_splits;
    split = (int)blockIdx.z % p.n_splits;
  }
  // key window of this block: [kv0, kv0 + nk), `shift` keys after it
  const int kv0 = Cfg::RAGGED != 0 ? kv_begin : split * p.kv_chunk;
  const int nk = Cfg::RAGGED != 0 ? kv_end - kv_begin : (nk_all - kv0 < p.kv_chunk ? nk_all - kv0 : p.kv_chunk);
  const int shift = nk_all - kv0 - nk;
  const int kh = g > 1 ? hy : hy / p.group;
  const int q0 = qb * BM * NQT;
  int n_kv[NQT];
  int nmax = 0;
  // query rows [ia, ib) of tile t (packed rows r hold query row r / g)
  auto tile_rows = [&](int t, int& ia, int& ib) {
    ia = (q0 + t * BM) / g;
    ib = (q0 + (t + 1) * BM + g - 1) / g;
  };
#pragma unroll
  for (int t = 0; t < NQT; ++t) {
    int ia, ib;
    tile_rows(t, ia, ib);
    n_kv[t] = kv_tile_count(ia, ib, nq, nk, BN, Cfg::CAUSAL, shift);
    nmax = n_kv[t] > nmax ? n_kv[t] : nmax;
  }

  if (threadIdx.x == 0) {
    for (int t = 0; t < NQT; ++t) ptx::mbar_init(bar(Cfg::B_QFULL + t), 1);
    for (int s = 0; s < KST; ++s) {
      ptx::mbar_init(bar(Cfg::B_KFULL + s), Cfg::KV8 ? 32 * Cfg::XP_WARPS : 1);
      ptx::mbar_init(bar(Cfg::B_KEMPTY + s), 1);
    }
    for (int s = 0; s < VST; ++s) {
      ptx::mbar_init(bar(Cfg::B_VFULL + s), Cfg::KV8 ? 32 * Cfg::XP_WARPS : 1);
      ptx::mbar_init(bar(Cfg::B_VEMPTY + s), 1);
    }
    for (int i = 0; i < NQT * SB; ++i) {
      ptx::mbar_init(bar(Cfg::B_SFULL + i), 1);
      ptx::mbar_init(bar(Cfg::B_PFULL + i), 128);
      ptx::mbar_init(bar(Cfg::B_PHALF + i), 128);
    }
    for (int t = 0; t < NQT; ++t) {
      ptx::mbar_init(bar(Cfg::B_ODONE + t), 1);
      ptx::mbar_init(bar(Cfg::B_OFINAL + t), 1);
    }
    if constexpr (Cfg::KV8) {
      for (int i = 0; i < Cfg::RST; ++i) {
        ptx::mbar_init(bar(Cfg::B_RFULL + i), 1);
        ptx::mbar_init(bar(Cfg::B_REMPTY + i), 32 * Cfg::XP_WARPS);
      }
    }
    ptx::mbar_init(bar(Cfg::B_DRAIN), 1);
    *abort_flag = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == Cfg::TMA_WARP && lane == 0) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  if (warp == Cfg::MMA_WARP) {
    ptx::tmem_alloc(sbase + Cfg::OFF_SLOT, Cfg::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sgen + Cfg::OFF_SLOT);

  if (warp < Cfg::SM_WARPS) {
    // ------------------------------------------------------------ softmax
    if constexpr (Cfg::SPLIT_REGS) ptx::setmaxnreg_inc<Cfg::REG_SOFTMAX>();
    const int t = warp >> 2, wq = warp & 3;
    int ia, ib;
    tile_rows(t, ia, ib);
    const int prow_packed = q0 + t * BM + wq * 32 + lane;  // this thread's (packed) tile row
    const int row = prow_packed / g;                         // its query row
    const int h = g > 1 ? kh * g + (prow_packed - row * g) : hy;
    const int nt = n_kv[t];
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t o_taddr = tmem + lane_off + (uint32_t)(Cfg::O_COL0 + t * D);
    float sl2 = p.sl2;
    if constexpr (Cfg::FP8) sl2 *= __ldg(p.dq) * __ldg(p.dk);
    const long long vend = vis_end(row, nq, nk, Cfg::CAUSAL, shift);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      const int si = t * SB + (j % SB);
      ok = wait_bar<kRoleSoftmax>(bar(Cfg::B_SFULL + si), (uint32_t)((j / SB) & 1), wc, kSiteSFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t s_taddr = tmem + lane_off + (uint32_t)(si * BN);
      const bool partial = tile_kind(ia, ib, j, nq, nk, BN, Cfg::CAUSAL, shift) == kTilePartial;
      const int nvis = (int)(vend - (long long)j * BN);  // visible keys of this tile (masks partial tiles)
      // ---- one read of the whole score row per tile, in two halves: the
      // second half's loads are in flight while the first half's maximum is
      // taken (full tiles, scale >= 0)
      uint32_t sr[BN];
      constexpr int NCH = BN / 32, NCH0 = NCH / 2 > 0 ? NCH / 2 : 1;
      const bool fast_max = !partial && sl2 >= 0.f;
      float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
      for (int c = 0; c < NCH0; ++c)
        ptx::tmem_ld32(s_taddr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
#pragma unroll
      for (int c = 0; c < NCH0; ++c) ptx::tmem_wait_ld_dep(*reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
#pragma unroll
      for (int c = NCH0; c < NCH; ++c)
        ptx::tmem_ld32(s_taddr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
      auto fold = [&](int c0, int c1) {  // a0..a3 <- their max with scores [c0, c1)
#pragma unroll
        for (int c = c0; c < c1; c += 8) {
          a0 = ptx::fmax3(a0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
          a1 = ptx::fmax3(a1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
          a2 = ptx::fmax3(a2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
          a3 = ptx::fmax3(a3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
        }
      };
      if (fast_max) fold(0, 32 * NCH0);
#pragma unroll
      for (int c = NCH0; c < NCH; ++c) ptx::tmem_wait_ld_dep(*reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
      float m_blk;
      if (partial) {
        m_blk = masked_max_scaled<BN>(sr, nvis, sl2);
      } else if (sl2 >= 0.f) {
        fold(32 * NCH0, BN);
        m_blk = ptx::fmax3(a0, a1, fmaxf(a2, a3)) * sl2;
      } else {  // a negative scale turns the row max into the row min
        float mn = __uint_as_float(sr[0]);
#pragma unroll
        for (int c = 1; c < BN; ++c) mn = fminf(mn, __uint_as_float(sr[c]));
        m_blk = mn * sl2;
      }
      float alpha = 1.f;
      bool resc = false;
      if (m_blk > m_ref + kTau) {
        alpha = ptx::ex2(m_ref - m_blk);  // 0 when m_ref = -inf
        resc = (m_ref != -INFINITY);
        m_ref = m_blk;
        l *= alpha;
      }
      const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
      const bool resc_any = __any_sync(0xffffffffu, resc);
      // P released in two halves (non-causal: measured faster; with causal
      // masks the extra live state costs more than the overlap gains)
      constexpr bool kHalfP = !Cfg::CAUSAL;
      // ---- exponentiate 32 columns at a time; each chunk's packed P is
      // stored at once (over score columns already read), so the registers of
      // a chunk die before the next chunk is processed
      uint64_t lsum[4] = {ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f), ptx::f2(0.f, 0.f)};
      const uint64_t sl2x2 = ptx::f2(sl2, sl2), negm2 = ptx::f2(-m_use, -m_use);
      constexpr int PW = Cfg::FP8 ? 8 : 16;  // packed P words per 32 scores
      // The tile kind is resolved once, outside the unrolled loop: one loop
      // body per kind, no per-element branches.
      auto exp_row = [&](auto partial_tag) {
        constexpr bool PARTIAL = decltype(partial_tag)::value;
#pragma unroll
        for (int ch = 0; ch < BN / 32; ++ch) {
          uint32_t pk[PW];
          [[maybe_unused]] float hold0 = 0.f, hold1 = 0.f;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int col = 32 * ch + 2 * c;
            const float s0 = __uint_as_float(sr[col]), s1 = __uint_as_float(sr[col + 1]);
            float e0, e1;
            const uint64_t x = ptx::ffma2(ptx::f2(s0, s1), sl2x2, negm2);
            float x0, x1;
            ptx::unf2(x, x0, x1);
            if (((16 * ch + c) % 8) < Cfg::EMU) {
              exp2_soft2(x0, x1, e0, e1);
            } else {
              e0 = ptx::ex2(x0);
              e1 = ptx::ex2(x1);
            }
            if constexpr (PARTIAL) {  // masked keys (a prefix is visible) get exact zeros
              e0 = col < nvis ? e0 : 0.f;
              e1 = col + 1 < nvis ? e1 : 0.f;
            }
            lsum[c % 4] = ptx::fadd2(lsum[c % 4], ptx::f2(e0, e1));
            if constexpr (Cfg::FP8) {
              if (c % 2 == 0) {
                hold0 = e0;
                hold1 = e1;
              } else {
                pk[c / 2] = ptx::pack_e4m3x4(hold0, hold1, e0, e1);
              }
            } else {
              pk[c] = ptx::pack_bf16x2(e0, e1);
            }
          }
          if constexpr (Cfg::FP8)
            ptx::tmem_st8(s_taddr + (uint32_t)(PW * ch), pk);
          else
            ptx::tmem_st16(s_taddr + (uint32_t)(PW * ch), pk);
          if (kHalfP && ch == BN / 64 - 1 && !resc_any) {
            // the first half of P is in tensor memory: the P V over the first
            // half of the keys can start while the second half is
            // exponentiated (a warp that must rescale O first releases it
            // after the rescale instead)
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(Cfg::B_PHALF + si));
          }
        }
      };
      if (partial)
        exp_row(std::true_type{});
      else
        exp_row(std::false_type{});
      {
        float la, lb;
        ptx::unf2(ptx::fadd2(ptx::fadd2(lsum[0], lsum[1]), ptx::fadd2(lsum[2], lsum[3])), la, lb);
        l += la + lb;
      }
      ptx::tmem_wait_st();
      if (resc_any) {
        // O_t must hold exactly the products of key tiles < j: wait for
        // PV(t, j-1).  Whenever S(t, j) is ready, PV(t, j-2) has completed (it
        // was issued before QK(t, j)) and PV(t, j) is not issued yet, so the
        // o_done barrier has completed j-1 or j phases and the parity test
        // for phase j-1 is unambiguous.
        ok = wait_bar<kRoleSoftmax>(bar(Cfg::B_ODONE + t), (uint32_t)((j - 1) & 1), wc, kSiteODone);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const float a = resc ? alpha : 1.f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          ptx::tmem_ld32(o_taddr + 32 * c, r);
          ptx::tmem_wait_ld_dep(r);
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * a);
          ptx::tmem_st32(o_taddr + 32 * c, r);
        }
        ptx::tmem_wait_st();
      }
      ptx::tc_fence_before();
      if (!Cfg::CAUSAL && resc_any) ptx::mbar_arrive(bar(Cfg::B_PHALF + si));
      ptx::mbar_arrive(bar(Cfg::B_PFULL + si));
    }
    // ------------------------------------------------------------ epilogue
    if (ok && nt > 0) {  // o_final completes once, after the tile's last PV
      ok = wait_bar<kRoleSoftmax>(bar(Cfg::B_OFINAL + t), 0u, wc, kSiteODone);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok) {
      ptx::tc_fence_after();
      const bool store = row < nq;
      float inv = l > 0.f ? 1.f / l : 0.f;
      if constexpr (Cfg::FP8) inv *= __ldg(p.dv);
      float lse = l > 0.f ? (m_ref + log2f(l)) * 0.6931471805599453f : -INFINITY;
      if constexpr (Cfg::RAGGED != 0) {
        if (l != l) inv = lse = l;  // a row whose scores hold a NaN
      }
      // first element of the row in [tokens, Hq, D], and its place in lse
      long long tok, lse_at;
      bool final_out;
      if constexpr (Cfg::RAGGED != 0) {
        tok = (long long)q_base + row;
        lse_at = (long long)h * p.rg.seqs.Tq + tok;
        final_out = slot < 0;
      } else {
        tok = (long long)b * p.Nq + row;
        lse_at = ((long long)b * p.Hq + h) * p.Nq + row;
        final_out = p.o_part == nullptr;
      }
      if (final_out) {
        __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(p.o) + (tok * p.Hq + h) * (long long)D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          if (nt > 0) {
            ptx::tmem_ld32(o_taddr + 32 * c, r);
            ptx::tmem_wait_ld_dep(r);
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = nt > 0 ? ptx::pack_bf16x2(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv)
                          : 0u;
          if (store) {
            uint4* dst = reinterpret_cast<uint4*>(orow + 32 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        }
        if (store && p.lse != nullptr) p.lse[lse_at] = lse;
      } else {
        // partial of window `split`, or of a piece: fp32 O_s and LSE_s
        long long prow, plse;
        if constexpr (Cfg::RAGGED != 0) {
          prow = plse = p.rg.pieces ? (long long)slot * (BM * NQT) + (prow_packed - q0)
                                    : ((long long)slot * p.rg.seqs.Tq + tok) * p.Hq + h;
        } else {
          const long long zs = (long long)split * p.B + b;
          prow = (zs * p.Nq + row) * p.Hq + h;
          plse = (zs * p.Hq + h) * p.Nq + row;
        }
        float* orow = p.o_part + prow * (long long)D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          if (nt > 0) {
            ptx::tmem_ld32(o_taddr + 32 * c, r);
            ptx::tmem_wait_ld_dep(r);
          }
          if (store) {
            float4* dst = reinterpret_cast<float4*>(orow + 32 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = nt > 0 ? make_float4(__uint_as_float(r[4 * e]) * inv, __uint_as_float(r[4 * e + 1]) * inv,
                                            __uint_as_float(r[4 * e + 2]) * inv, __uint_as_float(r[4 * e + 3]) * inv)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        if (store) p.lse_part[plse] = lse;
      }
    }
  } else if (warp == Cfg::TMA_WARP) {
    // ------------------------------------------------------------ producer
    if constexpr (Cfg::SPLIT_REGS) ptx::setmaxnreg_dec<Cfg::REG_CONTROL>();
    // (over a paged cache the whole warp runs the loop: lane i fetches the
    // tile's page i and issues its boxes)
    constexpr bool PAGED = Cfg::RAGGED >= 2;
    if (PAGED || lane == 0) {
      int k_issued[KST], v_issued[VST];
#pragma unroll
      for (int s = 0; s < KST; ++s) k_issued[s] = 0;
#pragma unroll
      for (int s = 0; s < VST; ++s) v_issued[s] = 0;
      [[maybe_unused]] int r_issued = 0;  // code tiles
      bool q_issued[NQT];
#pragma unroll
      for (int t = 0; t < NQT; ++t) {
        q_issued[t] = n_kv[t] > 0;
        if (!q_issued[t]) continue;
        if (PAGED && lane != 0) continue;
        const uint32_t fb = bar(Cfg::B_QFULL + t);
        ptx::mbar_arrive_expect_tx(fb, Cfg::QT_BYTES);
#pragma unroll
        for (int c = 0; c < Cfg::NCH; ++c) {
          const uint32_t dst = sbase + Cfg::OFF_Q + t * Cfg::QT_BYTES + c * Cfg::CH_Q;
          if (Cfg::PACK && g > 1)  // box: g heads x BM / g rows of kv head kh
            ptx::tma_load_5d(dst, &tmQ, fb, c * Cfg::BOXE, 0, kh, q_base + (q0 + t * BM) / g, b);
          else
            ptx::tma_load_4d(dst, &tmQ, fb, c * Cfg::BOXE, hy, q_base + q0 + t * BM, b);
        }
      }
      auto wait_empty = [&](uint32_t eb, uint32_t parity, uint32_t site) -> bool {
        if constexpr (PAGED) return wait_bar_warp<kRoleProducer>(eb, parity, wc, site);
        else return wait_bar<kRoleProducer>(eb, parity, wc, site);
      };
      // one operand's key tile: the boxes that make up its BN rows
      auto load_kv = [&](const CUtensorMap* tm, uint32_t dst, uint32_t fb, int j, int page) {
        if constexpr (PAGED) {
          // a row of a box is 128 bytes of bf16, or BOX8 codes
          constexpr int NBOX = Cfg::KV8 ? Cfg::NCH8 : Cfg::NCH, BOXW = Cfg::KV8 ? Cfg::BOX8 : Cfg::BOXE;
          constexpr uint32_t RP = Cfg::KV8 ? Cfg::BOX8 : 128u;
          if (lane == 0) ptx::mbar_arrive_expect_tx(fb, Cfg::KV8 ? Cfg::RAW_BYTES : Cfg::KV_BYTES);
          __syncwarp();
          const int ps = 1 << p.rg.page_shift, rows = ps < BN ? ps : BN;  // rows of a box
          if (lane < BN / rows) {
            const int r0 = ps < BN ? 0 : (kv0 + j * BN) & (ps - 1);
#pragma unroll
            for (int c = 0; c < NBOX; ++c)
              ptx::tma_load_4d(dst + c * (BN * RP) + lane * rows * RP, tm, fb, c * BOXW, kh, r0, page);
          }
        } else {
          ptx::mbar_arrive_expect_tx(fb, Cfg::KV_BYTES);
#pragma unroll
          for (int c = 0; c < Cfg::NCH; ++c)
            ptx::tma_load_4d(dst + c * Cfg::CH_KV, tm, fb, c * Cfg::BOXE, kh, k_base + kv0 + j * BN, b);
        }
      };
      // the page that holds this lane's rows of tile j; the index n_pages (a
      // box outside the map: zeros) behind the sequence and for a bad page
      auto page_of = [&](int j) -> int {
        if constexpr (PAGED) {
          const int ps = 1 << p.rg.page_shift, rows = ps < BN ? ps : BN;
          const int key = kv0 + j * BN + lane * rows;
          if (lane >= BN / rows || j * BN + lane * rows >= nk) return p.rg.n_pages;
          const int pi = key >> p.rg.page_shift;
          const int id = pi < p.rg.table_width ? __ldg(p.rg.table + (long long)seq * p.rg.table_width + pi) : -1;
          if (id >= 0 && id < p.rg.n_pages) return id;
          atomicOr(p.err, kErrIndex);
          return p.rg.n_pages;
        } else {
          return 0;
        }
      };
      [[maybe_unused]] int page = page_of(0);
      for (int j = 0; j < nmax; ++j) {
        [[maybe_unused]] const int page_next = PAGED && j + 1 < nmax ? page_of(j + 1) : 0;
        if constexpr (Cfg::KV8) {  // codes of K_j, then of V_j, through one ring
          bool go = true;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int i = 2 * j + x, rs = i % Cfg::RST;
            go = go && (i < Cfg::RST || wait_empty(bar(Cfg::B_REMPTY + rs), (uint32_t)((i / Cfg::RST - 1) & 1), kSiteKEmpty));
            if (!go) continue;
            load_kv(x == 0 ? &tmK : &tmV, sbase + Cfg::OFF_RAW + rs * Cfg::RAW_BYTES, bar(Cfg::B_RFULL + rs), j, page);
            ++r_issued;
          }
          if (!go) break;
          page = page_next;
          continue;
        }
        const int ks = j % KST;
        if (j >= KST && !wait_empty(bar(Cfg::B_KEMPTY + ks), (uint32_t)(((j / KST) - 1) & 1), kSiteKEmpty)) break;
        {
          load_kv(&tmK, sbase + Cfg::OFF_K + ks * Cfg::KV_BYTES, bar(Cfg::B_KFULL + ks), j, page);
          ++k_issued[ks];
        }
        const int vs = j % VST;
        if (j >= VST && !wait_empty(bar(Cfg::B_VEMPTY + vs), (uint32_t)(((j / VST) - 1) & 1), kSiteVEmpty)) break;
        {
          load_kv(&tmV, sbase + Cfg::OFF_V + vs * Cfg::KV_BYTES, bar(Cfg::B_VFULL + vs), j, page);
          ++v_issued[vs];
        }
        page = page_next;
      }
      // Every issued copy must land before the block may exit (no-op in the
      // normal path, where the consumers have already seen them all).
#pragma unroll
      for (int t = 0; t < NQT; ++t)
        if (q_issued[t]) wait_bar_drain<kRoleProducer>(bar(Cfg::B_QFULL + t), 0u, wc, kSiteQ);
      if constexpr (Cfg::KV8) {
#pragma unroll
        for (int i = 0; i < Cfg::RST; ++i) {
          const int n = (r_issued - i + Cfg::RST - 1) / Cfg::RST;  // fills of stage i
          if (n > 0) wait_bar_drain<kRoleProducer>(bar(Cfg::B_RFULL + i), (uint32_t)((n - 1) & 1), wc, kSiteKFull);
        }
      }
#pragma unroll
      for (int s = 0; s < KST; ++s)
        if (k_issued[s] > 0) wait_bar_drain<kRoleProducer>(bar(Cfg::B_KFULL + s), (uint32_t)((k_issued[s] - 1) & 1), wc, kSiteKFull);
#pragma unroll
      for (int s = 0; s < VST; ++s)
        if (v_issued[s] > 0) wait_bar_drain<kRoleProducer>(bar(Cfg::B_VFULL + s), (uint32_t)((v_issued[s] - 1) & 1), wc, kSiteVFull);
    }
  } else if (Cfg::KV8 && warp >= Cfg::XP_WARP) {
    if constexpr (Cfg::SPLIT_REGS) ptx::setmaxnreg_dec<Cfg::REG_CONTROL>();
    if constexpr (Cfg::KV8) {
      // ---------------------------------------------------------- expanding
      constexpr int RPW = BN / (Cfg::KV8 ? Cfg::XP_WARPS : 1);  // rows of this warp (at most one per lane)
      const int row0 = (warp - Cfg::XP_WARP) * RPW;
      const uint32_t raw0 = sbase + Cfg::OFF_RAW;
      // the page and the exponents of row row0 + lane, fetched two and one
      // tiles ahead (the table, then the bytes behind it)
      struct Facs { uint32_t k, v; };
      auto fetch_id = [&](int j) -> int {
        const int i = j * BN + row0 + lane, pi = (kv0 + i) >> p.rg.page_shift;
        return lane < RPW && j < nmax && i < nk && pi < p.rg.table_width
                   ? __ldg(p.rg.table + (long long)seq * p.rg.table_width + pi) : -1;
      };
      auto fetch_facs = [&](int j, int id) -> Facs {
        const int key = kv0 + j * BN + row0 + lane;
        if (id < 0 || id >= p.rg.n_pages) return Facs{0u, 0u};  // (zeros)
        const long long at = (((long long)id << p.rg.page_shift) + (key & ((1 << p.rg.page_shift) - 1))) * p.Hkv + kh;
        return Facs{__ldg(p.rg.k_exp + at), __ldg(p.rg.v_exp + at)};
      };
      auto expand = [&](uint32_t src, uint32_t dst, uint32_t ex) {
        const bool big = __any_sync(0xffffffffu, ex > 134u);
#pragma unroll 2
        for (int grp = 0; grp < RPW / 8; ++grp) {
          const int r = row0 + grp * 8 + (lane & 7);
          const E4m3Factor f = e4m3_factor(__shfl_sync(0xffffffffu, ex, grp * 8 + (lane & 7)));
#pragma unroll
          for (int it = 0; it < D / 64; ++it) {
            const int pc = (lane >> 3) + 4 * it;  // piece of 16 codes of the row
            // (TMA permutes a row's 16-byte pieces within 128 bytes, or 64 for 64-byte rows)
            const uint32_t pin = D == 64 ? (uint32_t)(pc ^ ((r >> 1) & 3)) : (uint32_t)((pc & 7) ^ (r & 7));
            uint32_t w[4], o[8];
            ptx::ld_shared_v4(src + (uint32_t)(pc * 16 / Cfg::BOX8) * (BN * Cfg::BOX8) + (uint32_t)r * Cfg::BOX8 + pin * 16u, w);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              o[2 * u] = bf16x2_mul(e4m3_hi_bits(__byte_perm(w[u], 0u, 0x1404)), f.m);
              o[2 * u + 1] = bf16x2_mul(e4m3_hi_bits(__byte_perm(w[u], 0u, 0x3424)), f.m);
            }
            if (big) {
#pragma unroll
              for (int u = 0; u < 8; ++u) o[u] = bf16x2_mul(o[u], f.more);
            }
            const uint32_t drow = dst + (uint32_t)(pc / 4) * Cfg::CH_KV + (uint32_t)r * 128u;
            const uint32_t p0 = (uint32_t)(2 * (pc & 3));
            ptx::st_shared_v4(drow + ((p0 ^ (uint32_t)(r & 7)) << 4), o[0], o[1], o[2], o[3]);
            ptx::st_shared_v4(drow + (((p0 + 1) ^ (uint32_t)(r & 7)) << 4), o[4], o[5], o[6], o[7]);
          }
        }
        ptx::fence_proxy_async_smem();
      };
      Facs fac = fetch_facs(0, fetch_id(0));
      int id = fetch_id(1);
      for (int j = 0; j < nmax; ++j) {
        const Facs fac_next = fetch_facs(j + 1, id);
        id = fetch_id(j + 2);
        bool go = true;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = 2 * j + x, rs = i % Cfg::RST, st = x == 0 ? j % KST : j % VST, n_st = x == 0 ? KST : VST;
          go = go && wait_bar_warp<kRoleProducer>(bar(Cfg::B_RFULL + rs), (uint32_t)((i / Cfg::RST) & 1), wc, kSiteKFull);
          go = go && (j < n_st || wait_bar_warp<kRoleProducer>(bar((x == 0 ? Cfg::B_KEMPTY : Cfg::B_VEMPTY) + st),
                                                               (uint32_t)((j / n_st - 1) & 1), wc, kSiteVEmpty));
          if (!go) continue;
          expand(raw0 + rs * Cfg::RAW_BYTES, sbase + (x == 0 ? Cfg::OFF_K : Cfg::OFF_V) + st * Cfg::KV_BYTES,
                 x == 0 ? fac.k : fac.v);
          ptx::mbar_arrive(bar((x == 0 ? Cfg::B_KFULL : Cfg::B_VFULL) + st));
          ptx::mbar_arrive(bar(Cfg::B_REMPTY + rs));
        }
        if (!go) break;
        fac = fac_next;
      }
    }
  } else {
    if constexpr (Cfg::SPLIT_REGS) ptx::setmaxnreg_dec<Cfg::REG_CONTROL>();
  }
  if (warp == Cfg::MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs this loop (waits, counters, descriptors); one
    // elected lane issues the tcgen05 instructions.
    {
      bool ok = true;
#pragma unroll
      for (int t = 0; t < NQT && ok; ++t)
        if (n_kv[t] > 0) ok = wait_bar_warp<kRoleMma>(bar(Cfg::B_QFULL + t), 0u, wc, kSiteQ);
      ptx::tc_fence_after();
      const uint32_t q_s = sbase + Cfg::OFF_Q, k_s = sbase + Cfg::OFF_K, v_s = sbase + Cfg::OFF_V;
      auto issue_qk = [&](int t, int j) {
        const uint32_t d_t = tmem + (uint32_t)((t * SB + j % SB) * BN);
        // descriptors advance by 32 bytes (>> 4 = 2) per K step inside a
        // 128-byte chunk and by one chunk (CH_Q / CH_KV bytes) after four
        const uint64_t ad0 = ptx::sdesc_sw128(q_s + t * Cfg::QT_BYTES, 16u, 1024u);
        const uint64_t bd0 = ptx::sdesc_sw128(k_s + (j % KST) * Cfg::KV_BYTES, 16u, 1024u);
#pragma unroll
        for (int kk = 0; kk < Cfg::QK_STEPS; ++kk) {
          const uint32_t ch = (uint32_t)kk / 4u, in = (uint32_t)kk % 4u;
          const uint64_t ad = ad0 + (uint64_t)((ch * Cfg::CH_Q + in * 32u) >> 4);
          const uint64_t bd = bd0 + (uint64_t)((ch * Cfg::CH_KV + in * 32u) >> 4);
          ptx::warp_mma_ss<Cfg::FP8>(d_t, ad, bd, Cfg::IDESC_QK, kk > 0 ? 1u : 0u);
        }
        ptx::warp_commit(bar(Cfg::B_SFULL + t * SB + j % SB));
      };
      auto issue_pv = [&](int t, int jj) -> bool {
        const int si = t * SB + jj % SB;
        const uint32_t ph = (uint32_t)((jj / SB) & 1);
        const uint32_t d_t = tmem + (uint32_t)(Cfg::O_COL0 + t * D);
        const uint32_t a_t = tmem + (uint32_t)(si * BN);
        const uint64_t bd0 = ptx::sdesc_sw128(v_s + (jj % VST) * Cfg::KV_BYTES, Cfg::CH_KV, 1024u);
        // non-causal: the first half of the keys as soon as their P is
        // written, the rest when the whole P is; causal: all at once
#pragma unroll
        for (int half = Cfg::CAUSAL ? 1 : 0; half < 2; ++half) {
          if (!wait_bar_warp<kRoleMma>(bar((half == 0 ? Cfg::B_PHALF : Cfg::B_PFULL) + si), ph, wc, kSitePFull))
            return false;
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = (Cfg::CAUSAL ? 0 : half * Cfg::PV_STEPS / 2); kk < (half + 1) * Cfg::PV_STEPS / 2; ++kk) {
            const uint64_t bd = bd0 + (uint64_t)(((uint32_t)kk * Cfg::KSTEP * 128u) >> 4);
            ptx::warp_mma_ts<Cfg::FP8>(d_t, a_t + (uint32_t)kk * 8u, bd, Cfg::IDESC_PV,
                                       (jj > 0 || kk > 0) ? 1u : 0u);
          }
        }
        ptx::warp_commit(bar(Cfg::B_ODONE + t));
        if (jj == n_kv[t] - 1) ptx::warp_commit(bar(Cfg::B_OFINAL + t));
        return true;
      };
      // RAGGED: rows of the V tile behind the last key hold what is not this
      // sequence's; a masked weight of zero times a NaN there would reach every
      // row, so they are cleared before the first product reads the tile
      auto clear_tail = [&](int jj) {
        const int valid = nk - jj * BN;
        if (valid >= BN) return;
        const uint32_t v0 = v_s + (jj % VST) * Cfg::KV_BYTES + (uint32_t)lane * 16u;
        for (int r = (valid > 0 ? valid : 0) * 128; r < BN * 128; r += 512) {
          if (r + lane * 16 < BN * 128) {
#pragma unroll
            for (int c = 0; c < Cfg::NCH; ++c) ptx::st_shared_v4(v0 + c * Cfg::CH_KV + r, 0u, 0u, 0u, 0u);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      };
      for (int j = 0; ok && j <= nmax; ++j) {
        const bool has_k = j < nmax, has_v = j >= 1;
        if constexpr (SB == 2) {
          // S is double-buffered: the products for key tile j go first, so
          // they run under the softmax of key tile j-1; then the P V of
          // key tile j-1 as each tile's P is released
          if (has_k) {
            ok = wait_bar_warp<kRoleMma>(bar(Cfg::B_KFULL + j % KST), (uint32_t)((j / KST) & 1), wc, kSiteKFull);
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int t = 0; t < NQT; ++t)
              if (j < n_kv[t]) issue_qk(t, j);
            ptx::warp_commit(bar(Cfg::B_KEMPTY + j % KST));
          }
          if (has_v) {
            ok = wait_bar_warp<kRoleMma>(bar(Cfg::B_VFULL + (j - 1) % VST), (uint32_t)(((j - 1) / VST) & 1),
                                         wc, kSiteVFull);
            if (!ok) break;
            if constexpr (Cfg::RAGGED == 1 || Cfg::RAGGED == 2) clear_tail(j - 1);
            ptx::tc_fence_after();
#pragma unroll
            for (int t = 0; t < NQT && ok; ++t)
              if (j - 1 < n_kv[t]) ok = issue_pv(t, j - 1);
            if (!ok) break;
            ptx::warp_commit(bar(Cfg::B_VEMPTY + (j - 1) % VST));
          }
        } else {
          // P overwrites S in place: PV(t, j-1) must be issued before
          // QK(t, j) reuses the buffer
          if (has_k) {
            ok = wait_bar_warp<kRoleMma>(bar(Cfg::B_KFULL + j % KST), (uint32_t)((j / KST) & 1), wc, kSiteKFull);
            if (!ok) break;
          }
          if (has_v) {
            ok = wait_bar_warp<kRoleMma>(bar(Cfg::B_VFULL + (j - 1) % VST), (uint32_t)(((j - 1) / VST) & 1),
                                         wc, kSiteVFull);
            if (!ok) break;
            if constexpr (Cfg::RAGGED == 1 || Cfg::RAGGED == 2) clear_tail(j - 1);
          }
          ptx::tc_fence_after();
#pragma unroll
          for (int t = 0; t < NQT && ok; ++t) {
            if (has_v && j - 1 < n_kv[t]) ok = issue_pv(t, j - 1);
            if (ok && has_k && j < n_kv[t]) issue_qk(t, j);
          }
          if (!ok) break;
          if (has_k) ptx::warp_commit(bar(Cfg::B_KEMPTY + j % KST));
          if (has_v) ptx::warp_commit(bar(Cfg::B_VEMPTY + (j - 1) % VST));
        }
      }
      // All issued MMAs must finish before tensor memory is freed.
      ptx::warp_commit(bar(Cfg::B_DRAIN));
      wait_bar_warp<kRoleMma>(bar(Cfg::B_DRAIN), 0u, wc, kSiteDrain);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == Cfg::MMA_WARP) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Cfg::TMEM_COLS);
  }
}

}  // namespace attn

// paged_fwd.cuh -- attention of few new tokens over a paged cache, shared out
// along the keys, and the merge of what was shared.
//
// The work is cut into units of 64 or 128 keys of one segment (sequence, tile of packed
// query rows, key/value head); the grid is what the GPU holds at once and every
// block takes an equal run of units, so blocks end together whatever the lengths
// are (windows of fixed size left the longest-working SM at 1.5 times the mean on
// 32 sequences of up to 8192 keys).  A run may end one segment and begin others;
// only a segment that is shared between blocks is written as partial rows, at
// most two per block, and merged by paged_combine_kernel.
//
// The g query heads of a key/value head share a segment: packed row
// r = i * g + h % g of new token i, so a step of decoding reads each cached key
// once per group.  A producer warp streams the units through a ring of stages
// (TMA, one box per page) and runs ahead across segments; four consumer warps run
// on their own, each on 16 keys of a stage at a time, and meet at a segment's end:
//   S^T = K Q^T,   the online softmax of every query row (a column),   O^T += V^T P^T
// on the warp-level matrix instruction (m16n8k16).  The kernel is bound by HBM;
// what it has to spare are instructions.  With the keys as the 16-row operand a
// group of up to 8 rows wastes nothing of the product, the accumulator is half
// as large, and K and V enter as fragments straight from shared memory; only P
// is transposed (movmatrix).  A row's maximum is exchanged between the lanes only
// when a lane sees a score past the threshold over the running reference, so
// most steps exchange nothing.
//
// Orders that are free are chosen for the loads: which reduction index stands
// where in a fragment (both operands agree, so a lane's 16-byte load serves two
// or four instructions), and which of 8 keys is which row (rows r and r + 4 of
// the 128-byte swizzle share no bank, neighbours do).
//
// e4m3 cache: codes become f16 (one conversion instruction per two codes, exact)
// and the products run in f16.  Queries are scaled per row by a power of two so
// that they fit f16 exactly (what falls below its normal range is under 2^-38 of
// the row's largest); the key's power-of-two scale multiplies its scores in fp32.
// The value's scale joins the exponent of its weight: with t = s + log2(scale),
// P = 2^(t - m_t) against a reference m_t of t, kept apart from the reference m of
// s that the row sum uses, and O = 2^(m_t - m) acc / l.  So P is rounded (11 bits)
// relative to the largest contribution to the output, whatever the scales are.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "attn_common.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace attn {

// The sequences of a paged call.
struct PagedSeqs {
  int Tq, n_seqs, max_q, max_kv;
  const int *cu_q, *kv_lens;  // cu_q may be nullptr: max_q tokens each
};

struct PagedParams : PagedSeqs {
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* o;  // [Tq, Hq, D]
  float* lse;        // [Hq, Tq] or nullptr
  int Hq, Hkv, group;
  const int* table;
  int table_width;
  const unsigned char *k_exp, *v_exp;
  int n_pages, page_shift;
  int causal;
  int row_tiles;             // CLUSTER: of a sequence of max_q tokens
  float sl2;                 // scale * log2(e)
  // workspace: units in front of each sequence and the units of a block, then the
  // partial rows [2 * blocks][block rows][D] and their LSE [2 * blocks][block rows]
  long long* base;  // [n_seqs], then the units of a block
  float *o_part, *lse_part;
  unsigned int* err;
  unsigned long long timeout_ns;
};

// The new tokens [q0, q0 + nq) and the cached tokens `len` of sequence s, with
// every value from device memory clamped to its array.
struct SeqRange {
  int q0, nq, len;
  bool bad;
};
__device__ __forceinline__ SeqRange paged_seq(const PagedSeqs& p, int s) {
  SeqRange r;
  r.bad = false;
  if (p.cu_q == nullptr) {
    r.q0 = s * p.max_q;
    r.nq = p.max_q;
  } else {
    int a = __ldg(p.cu_q + s), b = __ldg(p.cu_q + s + 1);
    if (a < 0 || b < a || b > p.Tq || b - a > p.max_q) {
      r.bad = true;
      a = a < 0 ? 0 : (a > p.Tq ? p.Tq : a);
      b = b < a ? a : (b > p.Tq ? p.Tq : b);
      b = b - a > p.max_q ? a + p.max_q : b;
    }
    r.q0 = a;
    r.nq = b - a;
  }
  r.len = __ldg(p.kv_lens + s);
  if (r.len < 0 || r.len > p.max_kv) {
    r.bad = true;
    r.len = r.len < 0 ? 0 : p.max_kv;
  }
  return r;
}
// The sequence that token t belongs to (-1: none).
__device__ __forceinline__ int paged_seq_of(const PagedSeqs& p, int t, SeqRange& r) {
  int s;
  if (p.cu_q == nullptr) {
    s = t / p.max_q;
  } else {
    int lo = 0, hi = p.n_seqs;  // the last s with cu_q[s] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (__ldg(p.cu_q + mid) <= t) lo = mid; else hi = mid - 1;
    }
    s = lo;
  }
  if (s >= p.n_seqs) return -1;
  r = paged_seq(p, s);
  return t >= r.q0 && t < r.q0 + r.nq ? s : -1;
}

// D head size, E4M3 cache type, NT: tiles of 8 packed rows per warp, RW: warps
// along the rows; the other 4 / RW share the keys of a stage, 16 at a time.
template <int D_, bool E4M3_, int NT_, int RW_>
struct PagedCfg {
  static constexpr int D = D_, NT = NT_, RW = RW_, KW = 4 / RW_;
  static constexpr bool E4M3 = E4M3_;
  // SP: groups of 16 keys a warp takes at once, two where a step is short on
  // independent work (one tile of rows, many conversions).  TK: keys of a stage,
  // and of a unit
  static constexpr int SP = E4M3 && NT == 1 && D <= 128 ? 2 : 1, TK = 64 * SP;
  static constexpr int RB = D * (E4M3 ? 1 : 2);        // bytes of a cached row
  static constexpr int CW = RB < 128 ? RB : 128;       // bytes of a box row
  static constexpr int NCHK = RB / CW;                 // boxes across a row
  static constexpr int ROWS = 8 * NT * RW;
  static constexpr uint32_t TILE = TK * RB, STAGE = 2 * TILE;
  // floats of a merge row (the padding spreads the banks; less of it is what lets
  // a third block with SP = 2 fit: 98 -> 91 us on 64 sequences of up to 8192 keys)
  static constexpr int OSTR = D + (SP == 2 ? 4 : 16);
  static constexpr int MROWS = (KW > 1 ? KW / 2 : 1) * ROWS;
  // 2 blocks of three 32 KB stages or 3 of two share an SM (two of the largest
  // stages where the merge rows leave no room for a third)
  static constexpr int NST = STAGE > 32768 && MROWS > 16 ? 2 : (SP == 2 && STAGE == 32768 ? 2 : (STAGE >= 16384 ? 3 : 4));
  static constexpr uint32_t OFF_EXP = NST * STAGE;     // exponent bytes of a stage: its keys', its values'
  static constexpr uint32_t OFF_MRG = OFF_EXP + (E4M3 ? NST * 2 * TK : 0);
  static constexpr uint32_t OFF_ML = OFF_MRG + MROWS * OSTR * 4;  // [KW][ROWS] of m, l, m_t
  static constexpr uint32_t OFF_BAR = OFF_ML + 3 * 4 * 64;        // full[NST], empty[NST]
  static constexpr uint32_t OFF_ABORT = OFF_BAR + 8 * 2 * NST;
  static constexpr uint32_t OFF_SCAN = OFF_ABORT + 8;             // 5 warp sums, then the first sequence and its units
  static constexpr uint32_t SMEM = OFF_SCAN + 8 * 8 + 1024;
  static constexpr int NTHREADS = 160;
  // blocks that share an SM, by shared memory and by the registers of their
  // accumulators and queries
  static constexpr int BY_SMEM = (227 * 1024) / (int)(SMEM + 1024), BY_REGS = NT * D > 128 ? 2 : (NT == 2 ? 3 : 4);
  static constexpr int BPS = BY_SMEM < 1 ? 1 : (BY_SMEM < BY_REGS ? BY_SMEM : BY_REGS);
  static_assert(KW * ROWS <= 64, "the exchange of references");
  static_assert(SMEM <= 227 * 1024, "shared memory per block");
};

// A sequence's row tiles, and the units of each (row tile, head).
struct PagedShape {
  int row_tiles, units;
};
__device__ __forceinline__ PagedShape paged_shape(const SeqRange& r, int group, int block_rows, int unit) {
  PagedShape x;
  x.row_tiles = (int)(((long long)r.nq * group + block_rows - 1) / block_rows);
  x.units = r.len > unit ? (r.len + unit - 1) / unit : 1;
  return x;
}

// CLUSTER: a segment belongs to a cluster of kPagedCluster blocks, which cut its
// units into equal runs and merge their rows through one another's shared memory.
// For calls that small that the second launch of the merge would take as long as
// the attention.
constexpr int kPagedCluster = 8;
template <class Cfg, bool CLUSTER>
__global__ void __launch_bounds__(Cfg::NTHREADS, Cfg::BPS)
    paged_fwd_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const PagedParams p) {
  constexpr int D = Cfg::D, TK = Cfg::TK, SP = Cfg::SP, KW = Cfg::KW, NST = Cfg::NST, NT = Cfg::NT, CW = Cfg::CW;
  constexpr bool E4M3 = Cfg::E4M3;
  constexpr int KS = D / 16;  // reduction steps of K Q^T, 16-row tiles of V^T P^T
  extern __shared__ uint8_t psm_raw[];
  const uint32_t raw_u32 = ptx::smem_u32(psm_raw);
  const uint32_t sb = (raw_u32 + 1023u) & ~1023u;
  uint8_t* psm = psm_raw + (sb - raw_u32);
  float* s_m = reinterpret_cast<float*>(psm + Cfg::OFF_ML);  // [KW][ROWS], 64 in all
  float* s_l = s_m + 64;
  [[maybe_unused]] float* s_t = s_m + 128;
  auto full = [&](int st) -> uint32_t { return sb + Cfg::OFF_BAR + 8u * (uint32_t)st; };
  auto empty = [&](int st) -> uint32_t { return sb + Cfg::OFF_BAR + 8u * (uint32_t)(NST + st); };
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(psm + Cfg::OFF_ABORT);
  const WaitCtx wc{abort_flag, p.err, p.timeout_ns};

  if constexpr (!CLUSTER) ptx::grid_dep_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = p.group;
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      ptx::mbar_init(full(i), E4M3 ? 33 : 1);
      ptx::mbar_init(empty(i), 4);
    }
    *abort_flag = 0u;
    ptx::fence_mbar_init();
  }

  // ---- this block's run of units [u_begin, u_end): of all units, or (CLUSTER) of
  // its segment's
  long long* s_scan = reinterpret_cast<long long*>(psm + Cfg::OFF_SCAN);
  long long u_begin, u_end;
  if constexpr (CLUSTER) {
    const int seg = (int)blockIdx.x / kPagedCluster, per_seq = p.row_tiles * p.Hkv;
    const SeqRange r = paged_seq(p, seg / per_seq);
    if (r.bad && tid == 0) atomicOr(p.err, kErrIndex);
    const PagedShape x = paged_shape(r, g, Cfg::ROWS, TK);
    if (seg % per_seq / p.Hkv >= x.row_tiles) return;  // (the whole cluster)
    const int share = (x.units + kPagedCluster - 1) / kPagedCluster;
    u_begin = (long long)share * ptx::cluster_rank();
    u_end = u_begin + share < x.units ? u_begin + share : x.units;
    __syncthreads();
  } else {
    // a scan over the sequences, each thread taking a contiguous share of them
    const int per = (p.n_seqs + Cfg::NTHREADS - 1) / Cfg::NTHREADS;
    const int sq0 = tid * per, sq1 = sq0 + per < p.n_seqs ? sq0 + per : p.n_seqs;
    auto units_of = [&](int s) -> long long {
      const SeqRange r = paged_seq(p, s);
      if (r.bad) atomicOr(p.err, kErrIndex);
      const PagedShape x = paged_shape(r, g, Cfg::ROWS, TK);
      return (long long)x.row_tiles * p.Hkv * x.units;
    };
    long long mine = 0;
    for (int s = sq0; s < sq1; ++s) mine += units_of(s);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    long long total = 0, front = upto - mine;
#pragma unroll
    for (int i = 0; i < Cfg::NTHREADS / 32; ++i) {
      if (i < warp) front += s_scan[i];
      total += s_scan[i];
    }
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    u_begin = share * blockIdx.x;
    u_end = u_begin + share < total ? u_begin + share : total;
    if (blockIdx.x == 0) {  // for the merge
      long long at = front;
      for (int s = sq0; s < sq1; ++s) {
        p.base[s] = at;
        at += units_of(s);
      }
      if (tid == 0) p.base[p.n_seqs] = share;
    }
    if (u_begin >= u_end) return;
    __syncthreads();  // (the warp sums have been read)
    if (front <= u_begin && u_begin < front + mine) {
      long long at = front;
      int s = sq0;
      for (;; ++s) {
        const long long n = units_of(s);
        if (u_begin < at + n) break;
        at += n;
      }
      s_scan[0] = s;
      s_scan[1] = at;
    }
    __syncthreads();
  }

  // ---- the run as portions: part (from unit `u` on) of a segment (sequence s,
  // row tile rt, head kh), in order; producer and consumers walk it alike
  struct Portion {
    int s, rt, kh;
    SeqRange sr;
    PagedShape sh;
    long long at;    // first unit of the segment
    long long u;     // first unit of the portion
    int k0, n;       // its first key, and the keys that some row of the tile sees
    int n_tiles;
    bool first, last;  // it holds the segment's first, last unit
  };
  auto settle = [&](Portion& x) {
    const long long stop = x.at + x.sh.units < u_end ? x.at + x.sh.units : u_end;  // (CLUSTER: may be no more than x.u)
    x.first = x.u == x.at;
    x.last = x.at + x.sh.units <= u_end;
    x.k0 = (int)(x.u - x.at) * TK;
    const long long k_stop = (stop - x.at) * TK;
    int k1 = k_stop < x.sr.len ? (int)k_stop : x.sr.len;
    if (p.causal) {  // the last row of the tile sees the most
      const long long rows = (long long)x.sr.nq * g, row0 = (long long)x.rt * Cfg::ROWS;
      const long long end = (row0 + Cfg::ROWS < rows ? row0 + Cfg::ROWS : rows) - 1;
      const long long vis = x.sr.len - x.sr.nq + end / g + 1;
      k1 = vis < k1 ? (int)(vis < 0 ? 0 : vis) : k1;
    }
    x.n = k1 > x.k0 ? k1 - x.k0 : 0;
    x.n_tiles = (x.n + TK - 1) / TK;
  };
  auto first_portion = [&]() -> Portion {
    Portion x;
    if constexpr (CLUSTER) {
      const int seg = (int)blockIdx.x / kPagedCluster, in_seq = seg % (p.row_tiles * p.Hkv);
      x.s = seg / (p.row_tiles * p.Hkv);
      x.sr = paged_seq(p, x.s);
      x.sh = paged_shape(x.sr, g, Cfg::ROWS, TK);
      x.rt = in_seq / p.Hkv;
      x.kh = in_seq % p.Hkv;
      x.at = 0;
      x.u = u_begin;
      settle(x);
      return x;
    }
    x.s = (int)s_scan[0];
    x.sr = paged_seq(p, x.s);
    x.sh = paged_shape(x.sr, g, Cfg::ROWS, TK);
    const long long seg = (u_begin - s_scan[1]) / x.sh.units;
    x.rt = (int)(seg / p.Hkv);
    x.kh = (int)(seg % p.Hkv);
    x.at = s_scan[1] + seg * x.sh.units;
    x.u = u_begin;
    settle(x);
    return x;
  };
  auto next_portion = [&](Portion& x) -> bool {  // false at the end of the run
    if constexpr (CLUSTER) return false;
    x.at += x.sh.units;
    if (x.at >= u_end) return false;
    x.u = x.at;
    if (++x.kh == p.Hkv) {
      x.kh = 0;
      if (++x.rt == x.sh.row_tiles) {
        x.rt = 0;
        do {
          x.sr = paged_seq(p, ++x.s);
          x.sh = paged_shape(x.sr, g, Cfg::ROWS, TK);
        } while (x.sh.row_tiles == 0);
      }
    }
    settle(x);
    return true;
  };

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    // Nothing that was just loaded is looked at in the same round: the table is
    // read 32 pages at a time, a block of them ahead, and the exponent bytes two
    // stages ahead (a load's latency is longer than a stage's turn).
    const int ps = 1 << p.page_shift, br = ps < TK ? ps : TK;  // rows of a box
    Portion x = first_portion();
    int issued = 0;  // stages filled
    bool go = true;
    do {
      const int k0 = x.k0, n = x.n, k1 = k0 + n, n_tiles = x.n_tiles, kh = x.kh;
      const int* table = p.table + (long long)x.s * p.table_width;
      const int pg0 = k0 >> p.page_shift;
      auto load_pages = [&](int blk) -> int {  // entries pg0 + 32 blk + lane
        const long long i = (long long)pg0 + 32ll * blk + lane;
        return i < p.table_width && (i << p.page_shift) < k1 ? __ldg(table + i) : -1;
      };
      int blk = 0, pages = load_pages(0), pages_next = load_pages(1);
      // the page of key i (from k0), for tiles in block `blk` or the next; n_pages (a
      // box outside the map: zeros) behind the last key and for a bad page
      auto page_of = [&](int i) -> int {
        const int idx = ((k0 + i) >> p.page_shift) - pg0;
        const int a = __shfl_sync(0xffffffffu, pages, idx & 31), b = __shfl_sync(0xffffffffu, pages_next, idx & 31);
        const int id = (idx >> 5) == blk ? a : b;
        if (i >= n) return p.n_pages;
        if (id >= 0 && id < p.n_pages) return id;
        atomicOr(p.err, kErrIndex);
        return p.n_pages;
      };
      struct Exps { uint32_t k[TK / 32], v[TK / 32]; };  // bytes of keys lane + 32 u of a tile
      auto exps_of = [&](int j) -> Exps {
        Exps r;
#pragma unroll
        for (int u = 0; u < TK / 32; ++u) {
          const int i = j * TK + lane + 32 * u, id = page_of(i);
          const long long at = (((long long)id << p.page_shift) + ((k0 + i) & (ps - 1))) * p.Hkv + kh;
          const bool there = id < p.n_pages;
          r.k[u] = there ? __ldg(p.k_exp + at) : 127u;
          r.v[u] = there ? __ldg(p.v_exp + at) : 127u;
        }
        return r;
      };
      [[maybe_unused]] Exps ex[2];
      if constexpr (E4M3) {
        ex[0] = exps_of(0);
        ex[1] = exps_of(1);
      }
      for (int j0 = 0; go && j0 < n_tiles; j0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = j0 + u;
          if (!go || j >= n_tiles) continue;
          const int b = ((k0 + j * TK) >> p.page_shift) - pg0;
          if ((b >> 5) != blk) {
            blk = b >> 5;
            pages = pages_next;
            pages_next = load_pages(blk + 1);
          }
          const int page = page_of(j * TK + (lane < TK / br ? lane * br : 0));
          const int st = issued % NST;
          if (issued >= NST &&
              !wait_bar_warp<kRoleProducer>(empty(st), (uint32_t)((issued / NST - 1) & 1), wc, kSiteKEmpty)) {
            go = false;
            continue;
          }
          const uint32_t kb = sb + (uint32_t)st * Cfg::STAGE;
          if (lane == 0) ptx::mbar_arrive_expect_tx(full(st), Cfg::STAGE);
          __syncwarp();
          if (lane < TK / br) {
            const int r0 = ps < TK ? 0 : (k0 + j * TK) & (ps - 1);
#pragma unroll
            for (int ch = 0; ch < Cfg::NCHK; ++ch) {
              const uint32_t dst = kb + ch * (TK * CW) + lane * br * CW;
              constexpr int BOXE = CW / (E4M3 ? 1 : 2);
              ptx::tma_load_4d(dst, &tmK, full(st), ch * BOXE, kh, r0, page);
              ptx::tma_load_4d(dst + Cfg::TILE, &tmV, full(st), ch * BOXE, kh, r0, page);
            }
          }
          ++issued;
          if constexpr (E4M3) {
            uint8_t* se = psm + Cfg::OFF_EXP + st * 2 * TK;
#pragma unroll
            for (int e = 0; e < TK / 32; ++e) {
              se[32 * e + lane] = (uint8_t)ex[u].k[e];
              se[TK + 32 * e + lane] = (uint8_t)ex[u].v[e];
            }
            ptx::mbar_arrive(full(st));
            ex[u] = exps_of(j + 2);
          }
        }
      }
    } while (go && next_portion(x));
    // every copy has to land before the block may end
#pragma unroll
    for (int i = 0; i < NST; ++i) {
      const int f = (issued - i + NST - 1) / NST;  // fills of stage i
      if (f > 0) wait_bar_drain<kRoleProducer>(full(i), (uint32_t)((f - 1) & 1), wc, kSiteKFull);
    }
    __syncthreads();
    if constexpr (CLUSTER) {
      ptx::cluster_sync();
      ptx::cluster_sync();
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int rw = warp % Cfg::RW, kw = warp / Cfg::RW;
  const int gr = lane >> 2, c = lane & 3;
  // key of row i of a fragment, among 8
  auto key_of = [](int i) -> int { return CW == 128 ? ((i >> 1) & 3) | ((i & 1) << 2) : i; };
  // byte offset of 16-byte piece pc of row r in a tile, as TMA lays it out
  auto at = [](int r, int pc) -> uint32_t {
    constexpr int PPR = CW / 16;
    const int x = CW == 128 ? r & 7 : (r >> 1) & 3;
    return (uint32_t)((pc / PPR) * (TK * CW) + r * CW + (((pc % PPR) ^ x) << 4));
  };
  Portion x = first_portion();
  int it = 0;  // stages consumed
  bool ok = true;
  do {
    const long long rows = (long long)x.sr.nq * g, row0 = (long long)x.rt * Cfg::ROWS;
    const int n = x.n;
    uint32_t qb[KS][NT][2];
    float rs[NT][2];   // what a raw score of rows 2c, 2c + 1 is multiplied by
    int lim[NT][2];    // keys (from k0) that they see
    int lim_min = n;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const long long r = row0 + rw * 8 * NT + nt * 8 + gr;
      const int i = (int)(r / g);
      const bool live = r < rows;
      const __nv_bfloat16* qr = p.q + (long long)(x.sr.q0 + i) * p.q_stride + (long long)(x.kh * g + (int)(r - (long long)i * g)) * D;
      float scale = p.sl2;
      if constexpr (E4M3) {
        // step 4 ch + t: reduction indexes 64 ch + 16 c + 4 t + {0, 1 | 2, 3}
        uint4 qx[D / 64][2];
        uint32_t top = 0u;  // largest magnitude (bits of bf16, in the upper half of a word)
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            qx[ch][u] = live ? __ldg(reinterpret_cast<const uint4*>(qr + 64 * ch + 16 * c) + u) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t y[4] = {qx[ch][u].x, qx[ch][u].y, qx[ch][u].z, qx[ch][u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              top = max(top, y[e] & 0x7FFF0000u);
              top = max(top, (y[e] << 16) & 0x7FFF0000u);
            }
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest lands in [2^14, 2^15)
        int sh = 141 - (int)(top >> 23);
        sh = top == 0u ? 0 : (sh > 126 ? 126 : sh);
        const float up = __uint_as_float((uint32_t)(sh + 127) << 23);
        scale *= __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t a = t % 2 == 0 ? qx[ch][t / 2].x : qx[ch][t / 2].z, b = t % 2 == 0 ? qx[ch][t / 2].y : qx[ch][t / 2].w;
            qb[4 * ch + t][nt][0] = ptx::pack_f16x2(__uint_as_float(a << 16) * up, __uint_as_float(a & 0xFFFF0000u) * up);
            qb[4 * ch + t][nt][1] = ptx::pack_f16x2(__uint_as_float(b << 16) * up, __uint_as_float(b & 0xFFFF0000u) * up);
          }
      } else {
        // steps 2 ch, 2 ch + 1: reduction indexes 32 ch + 8 c + {0, 1 | 2, 3} and + {4, 5 | 6, 7}
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          const uint4 y = live ? __ldg(reinterpret_cast<const uint4*>(qr + 32 * ch + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
          qb[2 * ch][nt][0] = y.x;
          qb[2 * ch][nt][1] = y.y;
          qb[2 * ch + 1][nt][0] = y.z;
          qb[2 * ch + 1][nt][1] = y.w;
        }
      }
      const long long vis = p.causal ? (long long)x.sr.len - x.sr.nq + i + 1 - x.k0 : n;
      const int my_lim = !live ? n : (vis < 0 ? 0 : (vis > n ? n : (int)vis));
      lim_min = min(lim_min, my_lim);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // from the lanes that hold rows 2c, 2c + 1 as their own
        rs[nt][e] = __shfl_sync(0xffffffffu, scale, (2 * c + e) * 4);
        lim[nt][e] = __shfl_sync(0xffffffffu, my_lim, (2 * c + e) * 4);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));

    // thresholds, log2 units: the references move when a score passes them by
    // TAU; P stays within 2^8, or for e4m3 within 2^15 with a reference 7 below the
    // maximum (f16 then resolves 2^-31 of the largest contribution)
    constexpr float kUp = E4M3 ? 7.f : 0.f;
    float acc[NT][KS][4];
    float m[NT][2], l[NT][2], mt[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = mt[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
    }

    for (int j = 0; j < x.n_tiles; ++j, ++it) {
      const int st = it % NST;
      ok = wait_bar_warp<kRoleSoftmax>(full(st), (uint32_t)((it / NST) & 1), wc, kSiteKFull);
      if (!ok) break;
      const uint32_t kb = sb + (uint32_t)st * Cfg::STAGE, vb = kb + Cfg::TILE;
#pragma unroll 1
      for (int sub = kw * SP; sub < TK / 16; sub += KW * SP) {
        const int key = j * TK + sub * 16;  // first of 16 * SP keys, from k0
        if (key >= n) break;
        const int kr = sub * 16 + key_of(gr);
        // ---- S^T = K Q^T
        float sc[SP][NT][4];
#pragma unroll
        for (int q = 0; q < SP; ++q)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[q][nt][e] = 0.f;
#pragma unroll
        for (int ch = 0; ch < Cfg::RB / 64; ++ch) {
#pragma unroll
          for (int q = 0; q < SP; ++q) {
            uint32_t fx[4], fy[4];
            ptx::ld_shared_v4(kb + at(kr + 16 * q, 4 * ch + c), fx);
            ptx::ld_shared_v4(kb + at(kr + 16 * q + 8, 4 * ch + c), fy);
            if constexpr (E4M3) {
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                uint32_t a[4];
                ptx::e4m3x4_to_f16x4(fx[t], a[0], a[2]);
                ptx::e4m3x4_to_f16x4(fy[t], a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) ptx::mma_f16(sc[q][nt], a, qb[4 * ch + t][nt][0], qb[4 * ch + t][nt][1]);
              }
            } else {
              const uint32_t a0[4] = {fx[0], fy[0], fx[1], fy[1]}, a1[4] = {fx[2], fy[2], fx[3], fy[3]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                ptx::mma_bf16(sc[q][nt], a0, qb[2 * ch][nt][0], qb[2 * ch][nt][1]);
                ptx::mma_bf16(sc[q][nt], a1, qb[2 * ch + 1][nt][0], qb[2 * ch + 1][nt][1]);
              }
            }
          }
        }
        // ---- scale, mask, online softmax (element e: key gr + 8 (e >> 1), row 2c + (e & 1))
        const bool whole = key + 16 * SP <= lim_min;  // every row of the warp sees all the keys
        bool grow = false;
        [[maybe_unused]] float tt[SP][NT][4];
        float sx[NT][2], tx[NT][2];  // this lane's largest
#pragma unroll
        for (int q = 0; q < SP; ++q) {
          float kf[2] = {1.f, 1.f}, kv[2] = {0.f, 0.f};
          if constexpr (E4M3) {
            const uint8_t* se = psm + Cfg::OFF_EXP + st * 2 * TK + kr + 16 * q;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t ke = se[8 * h], ve = se[TK + 8 * h];
              kf[h] = __uint_as_float(ke == kExpNaN ? 0x7FFFFFFFu : ke << 23);
              kv[h] = ve == kExpNaN ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(0x4B000000u | ve) - 8388735.f;
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sc[q][nt][e] *= E4M3 ? rs[nt][e & 1] * kf[e >> 1] : rs[nt][e & 1];
              if constexpr (E4M3) tt[q][nt][e] = sc[q][nt][e] + kv[e >> 1];
            }
            if (!whole) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (key + 16 * q + key_of(gr) + 8 * (e >> 1) >= lim[nt][e & 1]) {
                  sc[q][nt][e] = -INFINITY;
                  if constexpr (E4M3) tt[q][nt][e] = -INFINITY;
                }
              }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = fmaxf(sc[q][nt][e], sc[q][nt][e + 2]), b = E4M3 ? fmaxf(tt[q][nt][e], tt[q][nt][e + 2]) : 0.f;
              sx[nt][e] = q == 0 ? a : fmaxf(sx[nt][e], a);
              tx[nt][e] = q == 0 ? b : fmaxf(tx[nt][e], b);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            grow |= sx[nt][e] > m[nt][e] + kTau;
            if constexpr (E4M3) grow |= tx[nt][e] > mt[nt][e] + (kTau + kUp);
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float a = sx[nt][e], b = tx[nt][e];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                if constexpr (E4M3) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
              }
              float fa = 1.f, fb = 1.f;
              if (a > m[nt][e]) {
                fa = ptx::ex2(m[nt][e] - a);  // 0 from -inf
                m[nt][e] = a;
                l[nt][e] *= fa;
              }
              if constexpr (E4M3) {
                if (b - kUp > mt[nt][e]) {
                  fb = ptx::ex2(mt[nt][e] - (b - kUp));
                  mt[nt][e] = b - kUp;
                }
              } else {
                fb = fa;
              }
#pragma unroll
              for (int i = 0; i < KS; ++i) {
                acc[nt][i][e] *= fb;
                acc[nt][i][e + 2] *= fb;
              }
            }
        }
        uint32_t pb[SP][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float mu[2], mv[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mu[e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
            mv[e] = mt[nt][e] == -INFINITY ? 0.f : mt[nt][e];
          }
#pragma unroll
          for (int q = 0; q < SP; ++q) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pr[e] = ptx::ex2(sc[q][nt][e] - mu[e & 1]);
              l[nt][e & 1] += pr[e];
              if constexpr (E4M3) pr[e] = ptx::ex2(tt[q][nt][e] - mv[e & 1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
              pb[q][nt][h] = ptx::movmatrix_trans(E4M3 ? ptx::pack_f16x2(pr[2 * h], pr[2 * h + 1])
                                                       : ptx::pack_bf16x2(pr[2 * h], pr[2 * h + 1]));
          }
        }
        // ---- O^T += V^T P^T; the last keys' tile: what stands behind them must
        // not be multiplied, not even by zero
        const bool tail = key + 16 * SP > n;
        uint32_t live[SP][2];
        if (tail) {
#pragma unroll
          for (int q = 0; q < SP; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = key + 16 * q + 8 * h;
              live[q][h] = (k + key_of(2 * c) < n ? 0xFFFFu : 0u) | (k + key_of(2 * c + 1) < n ? 0xFFFF0000u : 0u);
            }
        }
        if constexpr (E4M3) {
          // matrices: keys 0-7 and 8-15 of piece d0, the same of piece d0 + 1
          const int vr = sub * 16 + 8 * ((lane >> 3) & 1) + key_of(lane & 7);
#pragma unroll
          for (int d0 = 0; d0 < KS; d0 += 2) {
#pragma unroll
            for (int q = 0; q < SP; ++q) {
              uint32_t fv[4];
              ptx::ldmatrix_x4_trans(vb + at(vr + 16 * q, d0 + (lane >> 4)), fv);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                // a word: columns 2 gr, 2 gr + 1 of two keys; the even column is row gr, the odd one row gr + 8
                uint32_t a[4], lo, hi;
                if (tail) {
                  fv[2 * u] &= live[q][0];
                  fv[2 * u + 1] &= live[q][1];
                }
                ptx::e4m3x4_to_f16x4(fv[2 * u], lo, hi);
                a[0] = __byte_perm(lo, hi, 0x5410);
                a[1] = __byte_perm(lo, hi, 0x7632);
                ptx::e4m3x4_to_f16x4(fv[2 * u + 1], lo, hi);
                a[2] = __byte_perm(lo, hi, 0x5410);
                a[3] = __byte_perm(lo, hi, 0x7632);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) ptx::mma_f16(acc[nt][d0 + u], a, pb[q][nt][0], pb[q][nt][1]);
              }
            }
          }
        } else {
          // matrices: keys 0-7 of pieces 2 i and 2 i + 1, then keys 8-15 of them
          const int vr = sub * 16 + 8 * (lane >> 4) + key_of(lane & 7);
#pragma unroll
          for (int i = 0; i < KS; ++i) {
#pragma unroll
            for (int q = 0; q < SP; ++q) {
              uint32_t fv[4];
              ptx::ldmatrix_x4_trans(vb + at(vr + 16 * q, 2 * i + ((lane >> 3) & 1)), fv);
              if (tail) {
                fv[0] &= live[q][0];
                fv[1] &= live[q][0];
                fv[2] &= live[q][1];
                fv[3] &= live[q][1];
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) ptx::mma_bf16(acc[nt][i], fv, pb[q][nt][0], pb[q][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty(st));
    }

    // ---- merge the key warps: rescale to the common references, sum, divide.
    // (A warp whose wait ran out goes through the same barriers with what it has; all
    // leave together below, the error word set.)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
        if (gr == 0) {
          const int r = kw * Cfg::ROWS + rw * 8 * NT + nt * 8 + 2 * c + e;
          s_m[r] = m[nt][e];
          s_l[r] = l[nt][e];
          if constexpr (E4M3) s_t[r] = mt[nt][e];
        }
      }
    if (KW > 1) ptx::bar_sync(1, 128);
    // acc stands against the reference `ref` of its warp
    const float* s_ref = E4M3 ? s_t : s_m;
    float* so = reinterpret_cast<float*>(psm + Cfg::OFF_MRG);
    auto columns = [&](float* row, int i, float a, float b) {  // this lane's two columns of 16-column piece i
      if constexpr (E4M3) {
        *reinterpret_cast<float2*>(row + 16 * i + 2 * gr) = make_float2(a, b);
      } else {
        row[16 * i + gr] = a;
        row[16 * i + gr + 8] = b;
      }
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (KW == 1) break;
        const int r = rw * 8 * NT + nt * 8 + 2 * c + e;
        float top = s_ref[r];
#pragma unroll
        for (int k = 1; k < KW; ++k) top = fmaxf(top, s_ref[k * Cfg::ROWS + r]);
        const float own = E4M3 ? mt[nt][e] : m[nt][e];
        const float f = own == -INFINITY ? 1.f : ptx::ex2(own - top);  // (without a reference acc is 0, or NaN)
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          acc[nt][i][e] *= f;
          acc[nt][i][e + 2] *= f;
        }
      }
#pragma unroll
    for (int half = KW / 2; half >= 1; half /= 2) {  // the upper half hands its sums to the lower
      if (kw >= half && kw < 2 * half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < KS; ++i)
              columns(so + ((kw - half) * Cfg::ROWS + rw * 8 * NT + nt * 8 + 2 * c + e) * Cfg::OSTR, i, acc[nt][i][e],
                      acc[nt][i][e + 2]);
      }
      ptx::bar_sync(1, 128);
      if (kw < half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float* row = so + (kw * Cfg::ROWS + rw * 8 * NT + nt * 8 + 2 * c + e) * Cfg::OSTR;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              acc[nt][i][e] += row[16 * i + (E4M3 ? 2 * gr : gr)];
              acc[nt][i][e + 2] += row[16 * i + (E4M3 ? 2 * gr + 1 : gr + 8)];
            }
          }
      }
      if (half > 1) ptx::bar_sync(1, 128);
    }
    if (kw == 0) {
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = rw * 8 * NT + nt * 8 + 2 * c + e;
          float mx = s_m[r], tx = s_ref[r];
#pragma unroll
          for (int k = 1; k < KW; ++k) {
            mx = fmaxf(mx, s_m[k * Cfg::ROWS + r]);
            tx = fmaxf(tx, s_ref[k * Cfg::ROWS + r]);
          }
          float lt = 0.f;
#pragma unroll
          for (int k = 0; k < KW; ++k) {
            const float mk = s_m[k * Cfg::ROWS + r], lk = s_l[k * Cfg::ROWS + r];
            lt += mk == -INFINITY ? lk : lk * ptx::ex2(mk - mx);  // (without a reference l is 0, or NaN)
          }
          float inv = lt == 0.f ? 0.f : 1.f / lt;
          if constexpr (E4M3) {
            if (tx != -INFINITY && mx != -INFINITY) inv *= ptx::ex2(tx - mx);
          }
          float* row = so + r * Cfg::OSTR;
#pragma unroll
          for (int i = 0; i < KS; ++i)
            columns(row, i, lt == 0.f ? 0.f : acc[nt][i][e] * inv, lt == 0.f ? 0.f : acc[nt][i][e + 2] * inv);
          // (each lane group writes the same value; the padding behind the row holds it)
          row[D] = lt == 0.f ? -INFINITY : (mx == -INFINITY ? lt : (mx + log2f(lt)) * 0.6931471805599453f);
        }
    }
    ptx::bar_sync(1, 128);
    constexpr int PPR = D / 8;  // 8-column pieces of a row
    for (int i = tid; !CLUSTER && i < Cfg::ROWS * PPR; i += 128) {
      const int r = i / PPR, pc = i % PPR;
      if (row0 + r >= rows) break;
      const float* row = so + r * Cfg::OSTR;
      const float4 a = reinterpret_cast<const float4*>(row)[2 * pc], b = reinterpret_cast<const float4*>(row)[2 * pc + 1];
      if (x.first && x.last) {
        const long long pr = row0 + r;
        const int t = x.sr.q0 + (int)(pr / g), h = x.kh * g + (int)(pr % g);
        const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        reinterpret_cast<uint4*>(p.o + ((long long)t * p.Hq + h) * D)[pc] = pack8(y);
        if (pc == 0 && p.lse != nullptr) p.lse[(long long)h * p.Tq + t] = row[D];
      } else {
        const long long to = (2ll * blockIdx.x + (x.last ? 0 : 1)) * Cfg::ROWS + r;
        float4* dst = reinterpret_cast<float4*>(p.o_part + to * D) + 2 * pc;
        dst[0] = a;
        dst[1] = b;
        if (pc == 0) p.lse_part[to] = row[D];
      }
    }
    if (!ptx::bar_red_and(1, 128, ok)) break;  // (then the merge rows and references are free again)
  } while (next_portion(x));
  __syncthreads();
  if constexpr (CLUSTER) {
    // every block holds its rows and their LSE; block k merges rows k, k + 8, ...
    ptx::cluster_sync();
    const long long rows = (long long)x.sr.nq * g, row0 = (long long)x.rt * Cfg::ROWS;
    for (int r = (int)ptx::cluster_rank(); r < Cfg::ROWS && row0 + r < rows; r += kPagedCluster) {
      const uint32_t row = sb + Cfg::OFF_MRG + (uint32_t)(r * Cfg::OSTR) * 4u;
      float wt[kPagedCluster], mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < kPagedCluster; ++k) {
        wt[k] = ptx::ld_peer_f32(row + D * 4u, (uint32_t)k);
        mx = fmaxf(mx, wt[k]);
      }
      const float mu = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int k = 0; k < kPagedCluster; ++k) {
        wt[k] = expf(wt[k] - mu);
        sum += wt[k];
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const long long pr = row0 + r;
      const int t = x.sr.q0 + (int)(pr / g), h = x.kh * g + (int)(pr % g);
      for (int col = tid; col < D; col += 128) {
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < kPagedCluster; ++k) {
          const float v = ptx::ld_peer_f32(row + (uint32_t)col * 4u, (uint32_t)k);
          y = wt[k] == 0.f ? y : fmaf(wt[k], v, y);
        }
        p.o[((long long)t * p.Hq + h) * D + col] = __float2bfloat16_rn(y * inv);
      }
      if (tid == 0 && p.lse != nullptr) p.lse[(long long)h * p.Tq + t] = sum == 0.f ? -INFINITY : mu + logf(sum);
    }
    ptx::cluster_sync();  // (a block's rows stay until all have read them)
  }
}

// One output row from S partial rows, by a warp: part w is row slot(w) of o_part
// (fp32, normalised by its own sum) with its LSE (natural log) in lse_part.
//   LSE = ln sum_w exp(LSE_w),   O = sum_w exp(LSE_w - LSE) O_w
// (parts without a visible key have O_w = 0, LSE_w = -inf and weigh nothing.)  Bound
// by the latency of one read from L2: the rows of the first AHEAD parts and all
// parts' LSE are requested together, and the row of a lane is one wide load.
template <int D, int AHEAD, class Slot>
__device__ __forceinline__ void merge_parts(const float* o_part, const float* lse_part, int S, Slot slot, int lane,
                                            __nv_bfloat16* o, float* lse) {
  constexpr int PER = D / 32;
  struct Piece { float v[PER]; };
  auto fetch = [&](int w) -> Piece {
    Piece x;
    const float* src = o_part + slot(w) * D + PER * lane;
    if constexpr (PER == 2) {
      const float2 a = __ldcg(reinterpret_cast<const float2*>(src));
      x.v[0] = a.x;
      x.v[1] = a.y;
    } else {
#pragma unroll
      for (int e = 0; e < PER; e += 4) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(src + e));
        x.v[e] = a.x;
        x.v[e + 1] = a.y;
        x.v[e + 2] = a.z;
        x.v[e + 3] = a.w;
      }
    }
    return x;
  };
  Piece y[AHEAD];
  float ls = lane < S ? __ldcg(lse_part + slot(lane)) : -INFINITY;
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
#pragma unroll
    for (int e = 0; e < PER; ++e) y[u].v[e] = 0.f;
    if (u < S) y[u] = fetch(u);
  }
  float mx = ls;
  for (int w = 32 + lane; w < S; w += 32) mx = fmaxf(mx, __ldcg(lse_part + slot(w)));
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
  const float mu = mx == -INFINITY ? 0.f : mx;
  float acc[PER], wsum = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int w0 = 0; w0 < S; w0 += AHEAD) {
    if (w0 > 0) {
      if (w0 % 32 == 0) ls = w0 + lane < S ? __ldcg(lse_part + slot(w0 + lane)) : -INFINITY;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (w0 + u < S) y[u] = fetch(w0 + u);
    }
    const float wl = expf(ls - mu);  // (0 behind the last part)
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const float wt = __shfl_sync(0xffffffffu, wl, (w0 + u) & 31);
      if (w0 + u < S) {
        wsum += wt;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = wt == 0.f ? acc[e] : fmaf(wt, y[u].v[e], acc[e]);
      }
    }
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  uint32_t out[PER / 2];
#pragma unroll
  for (int e = 0; e < PER / 2; ++e) out[e] = ptx::pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  __nv_bfloat16* dst = o + PER * lane;
  if constexpr (PER == 2) *reinterpret_cast<uint32_t*>(dst) = out[0];
  if constexpr (PER == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  if constexpr (PER == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
  if (lane == 0 && lse != nullptr) *lse = wsum == 0.f ? -INFINITY : mu + logf(wsum);
}

// Merge of the segments that several blocks shared: one warp per (token, head).
// The row's segment lies in the units [a, b), so in the blocks a / share ..
// (b - 1) / share; each wrote a partial row (slot 1: its segment goes on in the
// next block, slot 0: it ends here), and one block alone wrote the result itself.
// What the attention kernel was given is looked up while that still runs, the
// units in front of the sequence too where a warp counts them in one step
// (`blocks` blocks shared all units); with more sequences they are read back.
constexpr int kCombineCount = 64;  // sequences that a warp counts itself
template <int D>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams p, int block_rows, int unit, int blocks) {
  const long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int t = (int)(i / p.Hq), h = (int)(i - (long long)t * p.Hq), lane = threadIdx.x & 31;
  SeqRange sr;
  const int s = t < p.Tq ? paged_seq_of(p, t, sr) : -1;
  if (s < 0) {
    ptx::grid_dep_wait();  // (on every path: the grid must not end before the one it follows)
    return;
  }
  const int g = p.group, units = paged_shape(sr, g, block_rows, unit).units;
  const long long pr = (long long)(t - sr.q0) * g + h % g;
  const int r = (int)(pr % block_rows);
  const long long in_seq = ((pr / block_rows) * p.Hkv + h / g) * units;
  long long share, base;
  if (p.n_seqs <= kCombineCount) {
    long long total = 0, front = 0;
    for (int x = lane; x < p.n_seqs; x += 32) {
      const PagedShape sh = paged_shape(paged_seq(p, x), g, block_rows, unit);
      const long long n = (long long)sh.row_tiles * p.Hkv * sh.units;
      total += n;
      front += x < s ? n : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      front += __shfl_xor_sync(0xffffffffu, front, o);
    }
    share = (total + blocks - 1) / blocks;
    base = front;
    ptx::grid_dep_wait();
  } else {
    ptx::grid_dep_wait();
    share = __ldcg(p.base + p.n_seqs);
    base = __ldcg(p.base + s);
  }
  const long long a = base + in_seq, i0 = a / share, i1 = (a + units - 1) / share;
  if (i0 == i1) return;
  const int S = (int)(i1 - i0 + 1);
  merge_parts<D, 8>(p.o_part, p.lse_part, S,
                 [&](int w) -> long long { return (2 * (i0 + w) + (w == S - 1 ? 0 : 1)) * block_rows + r; }, lane,
                 p.o + i * D, p.lse != nullptr ? p.lse + (long long)h * p.Tq + t : nullptr);
}

// Merge of what the tcgen05 kernel left as partial rows: of the key windows of its
// items, parts [window][Tq][Hq] (a sequence of one window is final already), or of
// the items it took in pieces, whose parts are the runs that the pair of item and
// head lies in.  A block takes a token, a warp some of its heads (grid y shares them
// out too): the look-ups (sequence, item, its place in the line) wait for one
// another, so a warp makes them once for its heads (1671 tokens of 32 heads of 128,
// cold caches: 60 us with a warp per head, 30 so).
struct LongParams : PagedSeqs {
  __nv_bfloat16* o;
  float* lse;
  int Hq, window;  // window > 0: windows
  int rows_per_token, block_rows, nh, max_items;
  const long long* lin;
  const int* first;
  const float *o_part, *lse_part;
};
template <int D>
__global__ void __launch_bounds__(256) long_combine_kernel(const LongParams p) {
  const int t = (int)blockIdx.x, lane = threadIdx.x & 31;
  SeqRange sr;
  const int s = paged_seq_of(p, t, sr);
  ptx::grid_dep_wait();
  if (s < 0) return;
  const int h0 = (int)(blockIdx.y * 8 + (threadIdx.x >> 5)), h_step = (int)gridDim.y * 8;
  auto merge = [&](int h, int S, auto slot) {
    merge_parts<D, 4>(p.o_part, p.lse_part, S, slot, lane, p.o + ((long long)t * p.Hq + h) * D,
                   p.lse != nullptr ? p.lse + (long long)h * p.Tq + t : nullptr);
  };
  if (p.window > 0) {
    if (sr.len <= p.window) return;
    const int S = (sr.len - 1) / p.window + 1;
    const long long all = (long long)p.Tq * p.Hq;
    for (int h = h0; h < p.Hq; h += h_step)
      merge(h, S, [&](int w) -> long long { return w * all + (long long)t * p.Hq + h; });
    return;
  }
  const int g = p.rows_per_token, shift = 31 - __clz(p.block_rows);
  const long long r0 = (long long)(t - sr.q0) * g;  // (the g rows of a token are in one block)
  const long long item = __ldcg(p.first + s) + (r0 >> shift);
  if (item >= __ldcg(p.first + p.n_seqs)) return;
  const long long front = __ldcg(p.lin + item), c = __ldcg(p.lin + item + 1) - front;
  const long long share = __ldcg(p.lin + p.max_items + 1);
  const bool small = (front + c) * p.nh < (1ll << 31) && share < (1ll << 31);
  for (int h = h0; h < p.Hq; h += h_step) {
    const int hy = h / g;
    int v0, S;  // the first run, and the runs
    if (small) {
      const PieceRuns<unsigned> x = piece_runs<unsigned>((unsigned)front * (unsigned)p.nh + (unsigned)hy * (unsigned)c,
                                                         (unsigned)c, (unsigned)share);
      v0 = (int)x.first;
      S = (int)(x.last - x.first) + 1;
    } else {
      const PieceRuns<long long> x = piece_runs<long long>(front * p.nh + hy * c, c, share);
      v0 = (int)x.first;
      S = (int)(x.last - x.first) + 1;
    }
    if (S == 1) continue;
    const int row = (int)((r0 + h - hy * g) & (p.block_rows - 1));
    merge(h, S, [&](int w) -> long long { return ((long long)(2 * (v0 + w) + (w == S - 1 ? 0 : 1)) << shift) + row; });
  }
}

}  // namespace attn

// paged_fwd.cuh -- attention of few new tokens over a paged cache, split over
// windows of keys, and the merge of the windows.
//
// One block takes one (sequence, key/value head, tile of packed query rows, key
// window).  The g query heads of a key/value head share the block: packed row
// r = i * g + h % g of new token i, so a step of decoding reads each cached key
// once per group.  The block streams its window through a ring of 64-key
// stages (cp.async, 16 bytes per request, rows gathered through the page table;
// rows behind the last visible key are filled with zeros, so what the cache
// holds there cannot reach the products) and runs, per 16 rows x 16 keys of a
// warp, S = Q K^T, the online softmax and O += P V on the warp-level matrix
// instruction (m16n8k16).  The kernel is bound by HBM: 16 rows of a decoding
// group use a tenth of what that instruction delivers, and a 16-row tile wastes
// far less of the softmax than the 128-row tile of tcgen05.
//
// e4m3 cache: codes are expanded to bf16 in registers (exactly), the key's
// power-of-two scale multiplies its scores in fp32 and the value's its weight
// before that is rounded to bf16, so nothing but the products' operands is
// rounded, as with a bf16 cache.
//
// Which reduction index stands where in a fragment is free as long as both
// operands agree, so the keys are read with 16-byte shared loads: a lane's 16
// bytes are the reduction indexes of two (bf16) or four (e4m3) instructions.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "attn_common.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace attn {

struct PagedParams {
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* o;  // [Tq, Hq, D]
  float* lse;        // [Hq, Tq] or nullptr
  int Tq, n_seqs, max_q, Hq, Hkv, group;
  const int *cu_q, *table, *kv_lens;
  int table_width, max_kv;
  const void *k_pages, *v_pages;
  const unsigned char *k_exp, *v_exp;
  int n_pages, page_shift;
  int causal;
  float sl2;                 // scale * log2(e)
  int n_windows, window;     // key windows of a sequence of max_kv keys; keys per window (a multiple of 64)
  int row_tiles;             // tiles of packed rows of a sequence of max_q tokens
  float *o_part, *lse_part;  // [window][Tq][Hq][D] and [window][Tq][Hq]
  unsigned int* err;
};

// The new tokens [q0, q0 + nq) and the cached tokens `len` of sequence s, with
// every value from device memory clamped to its array.
struct SeqRange {
  int q0, nq, len;
  bool bad;
};
__device__ __forceinline__ SeqRange paged_seq(const PagedParams& p, int s) {
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

// D head size, E4M3 cache type, RW: warps along the packed rows (16 each); the
// other 4 / RW share the keys of a stage, 16 at a time.
template <int D_, bool E4M3_, int RW_>
struct PagedCfg {
  static constexpr int D = D_, RW = RW_, KW = 4 / RW_, TK = 64;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int RB = D * (E4M3 ? 1 : 2);  // bytes of a cached row
  static constexpr int CPR = RB / 16;
  static constexpr int ROWS = 16 * RW;
  static constexpr uint32_t TILE = TK * RB, STAGE = 2 * TILE;
  // stages: about 96 KB of a bf16 ring and 64 KB of an e4m3 one let 2 and 3
  // blocks share an SM at d = 128
  static constexpr int NST = STAGE >= 65536 ? 3 : (STAGE >= 32768 ? 3 : 4);
  static constexpr int MAXW = 2048;               // keys of a window at most
  static constexpr int OSTR = D + 16;             // floats of a merge row (the padding spreads the banks)
  static constexpr uint32_t OFF_PAGE = NST * STAGE;                      // page ids of the window
  static constexpr uint32_t OFF_FAC = OFF_PAGE + 4 * (MAXW / 16 + 4);    // bf16 factors: keys, then values
  static constexpr uint32_t OFF_ML = OFF_FAC + (E4M3 ? 2 * 2 * MAXW : 0);
  static constexpr uint32_t SMEM = OFF_ML + 2 * 4 * 4 * 16;
  static_assert((uint32_t)64 * OSTR * 4 <= NST * STAGE, "the merge rows reuse the ring");
  static_assert(SMEM <= 227 * 1024, "shared memory per block");
};

// Byte offset of 16-byte piece c of row r: pieces are permuted within 128
// bytes so that 8 rows' same piece (ldmatrix) and 2 rows' 4 neighbouring pieces
// (a quarter warp's 16-byte loads) fall into different banks.
template <int RB>
__device__ __forceinline__ uint32_t paged_swz(uint32_t r, uint32_t c) {
  if constexpr (RB == 64) {
    return (r >> 1) * 128u + (((r & 1u) << 2) | (c ^ ((r >> 1) & 3u))) * 16u;
  } else {
    const uint32_t x = ((r & 1u) << 2) | ((r >> 1) & 3u);
    return r * RB + ((c & ~7u) | ((c & 7u) ^ x)) * 16u;
  }
}

template <class Cfg>
__global__ void __launch_bounds__(128) paged_fwd_kernel(const PagedParams p) {
  constexpr int D = Cfg::D, TK = Cfg::TK, KW = Cfg::KW, NST = Cfg::NST, RB = Cfg::RB;
  constexpr bool E4M3 = Cfg::E4M3;
  constexpr int KS = D / 16;  // reduction steps of Q K^T
  extern __shared__ __align__(128) uint8_t psm[];
  const uint32_t sb = ptx::smem_u32(psm);
  int* s_page = reinterpret_cast<int*>(psm + Cfg::OFF_PAGE);
  __nv_bfloat16* s_kf = reinterpret_cast<__nv_bfloat16*>(psm + Cfg::OFF_FAC);
  __nv_bfloat16* s_vf = s_kf + Cfg::MAXW;
  float* s_m = reinterpret_cast<float*>(psm + Cfg::OFF_ML);  // [KW][ROWS], 64 in all
  float* s_l = s_m + 64;

  ptx::grid_dep_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int w = (int)(blockIdx.x % (unsigned)p.n_windows);
  const int rest = (int)(blockIdx.x / (unsigned)p.n_windows);
  const int rt = rest % p.row_tiles;
  const int kh = (rest / p.row_tiles) % p.Hkv;
  const int s = rest / p.row_tiles / p.Hkv;
  const SeqRange sr = paged_seq(p, s);
  if (sr.bad && tid == 0) atomicOr(p.err, kErrIndex);
  const int g = p.group;
  const long long rows = (long long)sr.nq * g;
  const long long row0 = (long long)rt * Cfg::ROWS;
  if (row0 >= rows) return;
  const int nwin = sr.len > p.window ? (sr.len + p.window - 1) / p.window : 1;
  if (w >= nwin) return;
  const int k0 = w * p.window;
  int k1 = sr.len - k0 < p.window ? sr.len : k0 + p.window;
  if (p.causal) {  // the last row of the tile sees the most
    const long long last = (row0 + Cfg::ROWS < rows ? row0 + Cfg::ROWS : rows) - 1;
    const long long vis = sr.len - sr.nq + last / g + 1;
    k1 = vis < k1 ? (int)(vis < k0 ? k0 : vis) : k1;
  }
  const int n = k1 - k0 > 0 ? k1 - k0 : 0;  // keys of this block
  const int n_tiles = (n + TK - 1) / TK;

  // page ids of the window (-1: reads as zeros)
  const int pg0 = k0 >> p.page_shift;
  const int npg = n > 0 ? ((k1 - 1) >> p.page_shift) - pg0 + 1 : 0;
  for (int i = tid; i < npg; i += 128) {
    int id = pg0 + i < p.table_width ? __ldg(p.table + (long long)s * p.table_width + pg0 + i) : -1;
    if (id < 0 || id >= p.n_pages) {
      id = -1;
      atomicOr(p.err, kErrIndex);
    }
    s_page[i] = id;
  }
  __syncthreads();

  // cached row of key k0 + i: index into [slots, Hkv], or -1
  auto cached_row = [&](int i) -> long long {
    const int key = k0 + i;
    const int id = s_page[(key >> p.page_shift) - pg0];
    return id < 0 ? -1 : (((long long)id << p.page_shift) + (key & ((1 << p.page_shift) - 1))) * p.Hkv + kh;
  };
  auto load_tile = [&](int j) {
    const uint32_t kb = sb + (uint32_t)(j % NST) * Cfg::STAGE;
    constexpr int RPI = 128 / Cfg::CPR;  // rows per round of the block (8, 16, 32 or 4)
    const int c = tid % Cfg::CPR;
#pragma unroll
    for (int i = 0; i < TK / RPI; ++i) {
      const int r = i * RPI + tid / Cfg::CPR;
      const int key = j * TK + r;
      const long long row = key < n ? cached_row(key) : -1;
      const long long off = row < 0 ? 0 : row * RB + 16 * c;
      const uint32_t dst = kb + paged_swz<RB>((uint32_t)r, (uint32_t)c);
      ptx::cp_async16(dst, static_cast<const uint8_t*>(p.k_pages) + off, row >= 0);
      ptx::cp_async16(dst + Cfg::TILE, static_cast<const uint8_t*>(p.v_pages) + off, row >= 0);
    }
  };
#pragma unroll
  for (int j = 0; j < NST - 1; ++j) {
    if (j < n_tiles) load_tile(j);
    ptx::cp_async_commit();
  }
  if constexpr (E4M3) {
    for (int i = tid; i < n_tiles * TK; i += 128) {
      const long long row = i < n ? cached_row(i) : -1;
      const uint32_t ke = row < 0 ? 0u : __ldg(p.k_exp + row), ve = row < 0 ? 0u : __ldg(p.v_exp + row);
      s_kf[i] = __ushort_as_bfloat16((unsigned short)(ke == kExpNaN ? 0x7FFFu : ke << 7));
      s_vf[i] = __ushort_as_bfloat16((unsigned short)(ve == kExpNaN ? 0x7FFFu : ve << 7));
    }
  }

  // this warp's 16 rows: the lane holds rows gr and gr + 8
  const int rw = warp % Cfg::RW, kw = warp / Cfg::RW;
  const int gr = lane >> 2, c = lane & 3;
  uint32_t qa[KS][4];
  int lim[2];  // keys (from k0) that the row sees
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const long long r = row0 + rw * 16 + gr + 8 * hf;
    const int i = (int)(r / g);
    const bool live = r < rows;
    const __nv_bfloat16* qr = p.q + (long long)(sr.q0 + i) * p.q_stride + (long long)(kh * g + (int)(r - (long long)i * g)) * D;
    long long vis = p.causal ? (long long)sr.len - sr.nq + i + 1 - k0 : n;
    lim[hf] = vis < 0 ? 0 : (vis > n ? n : (int)vis);
    if constexpr (E4M3) {
      // step 4 ch + t: reduction indexes 64 ch + 16 c + 4 t + {0, 2 | 1, 3}
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch) {
        uint4 x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          x[u] = live ? __ldg(reinterpret_cast<const uint4*>(qr + 64 * ch + 16 * c) + u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t a = t % 2 == 0 ? x[t / 2].x : x[t / 2].z, b = t % 2 == 0 ? x[t / 2].y : x[t / 2].w;
          qa[4 * ch + t][hf] = __byte_perm(a, b, 0x5410);
          qa[4 * ch + t][hf + 2] = __byte_perm(a, b, 0x7632);
        }
      }
    } else {
      // steps 2 ch, 2 ch + 1: reduction indexes 32 ch + 8 c + {0, 1 | 2, 3} and + {4, 5 | 6, 7}
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(qr + 32 * ch + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
        qa[2 * ch][hf] = x.x;
        qa[2 * ch][hf + 2] = x.y;
        qa[2 * ch + 1][hf] = x.z;
        qa[2 * ch + 1][hf + 2] = x.w;
      }
    }
  }
  float acc[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  for (int j = 0; j < n_tiles; ++j) {
    ptx::cp_async_wait<NST - 2>();
    __syncthreads();
    if (j + NST - 1 < n_tiles) load_tile(j + NST - 1);
    ptx::cp_async_commit();
    const uint32_t kb = sb + (uint32_t)(j % NST) * Cfg::STAGE, vb = kb + Cfg::TILE;
#pragma unroll 1
    for (int sub = kw; sub < TK / 16; sub += KW) {
      const int key = j * TK + sub * 16;  // first of 16 keys, from k0
      if (key >= n) break;
      // ---- S = Q K^T, two tiles of 8 keys
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t r = (uint32_t)(sub * 16 + nt * 8 + gr);
#pragma unroll
        for (int ch = 0; ch < Cfg::CPR / 4; ++ch) {
          uint32_t x[4];
          ptx::ld_shared_v4(kb + paged_swz<RB>(r, (uint32_t)(4 * ch + c)), x);
          if constexpr (E4M3) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
              ptx::mma_bf16(sc[nt], qa[4 * ch + t], e4m3_lo_to_bf16x2(x[t]), e4m3_hi_to_bf16x2(x[t]));
          } else {
            ptx::mma_bf16(sc[nt], qa[2 * ch], x[0], x[1]);
            ptx::mma_bf16(sc[nt], qa[2 * ch + 1], x[2], x[3]);
          }
        }
      }
      // ---- scale, mask, online softmax
      float vf[2][2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float f0 = p.sl2, f1 = p.sl2;
        vf[nt][0] = vf[nt][1] = 1.f;
        if constexpr (E4M3) {
          const uint32_t kf = *reinterpret_cast<const uint32_t*>(s_kf + key + nt * 8 + 2 * c);
          const uint32_t vv = *reinterpret_cast<const uint32_t*>(s_vf + key + nt * 8 + 2 * c);
          f0 *= __uint_as_float(kf << 16);
          f1 *= __uint_as_float(kf & 0xFFFF0000u);
          vf[nt][0] = __uint_as_float(vv << 16);
          vf[nt][1] = __uint_as_float(vv & 0xFFFF0000u);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] *= (e & 1) ? f1 : f0;
      }
      const bool whole = key + 16 <= lim[0] && key + 16 <= lim[1];  // (lim is per lane; masks below are per element)
      if (!whole) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key + nt * 8 + 2 * c + (e & 1) >= lim[e >> 1]) sc[nt][e] = -INFINITY;
      }
      float mx[2];
      bool grow = false;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        mx[hf] = fmaxf(fmaxf(sc[0][2 * hf], sc[0][2 * hf + 1]), fmaxf(sc[1][2 * hf], sc[1][2 * hf + 1]));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 2));
        grow |= mx[hf] > m[hf] + kTau;  // the reference moves only past the threshold
      }
      if (__any_sync(0xffffffffu, grow)) {
        float a[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          a[hf] = 1.f;
          if (mx[hf] > m[hf] + kTau) {
            a[hf] = ptx::ex2(m[hf] - mx[hf]);  // 0 from -inf
            m[hf] = mx[hf];
            l[hf] *= a[hf];
          }
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] *= a[e >> 1];
      }
      const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
      uint32_t pa[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = ptx::ex2(sc[nt][e] - mu[e >> 1]);
          l[e >> 1] += pr[e];
          if constexpr (E4M3) {
            // the value's scale, with 2^-8 against the threshold's headroom (put back at the end);
            // a masked key keeps an exact zero whatever its scale
            pr[e] = sc[nt][e] == -INFINITY ? 0.f : pr[e] * (vf[nt][e & 1] * 0.00390625f);
          }
        }
        pa[2 * nt] = ptx::pack_bf16x2(pr[0], pr[1]);
        pa[2 * nt + 1] = ptx::pack_bf16x2(pr[2], pr[3]);
      }
      // ---- O += P V
      const uint32_t vr = (uint32_t)(sub * 16 + (lane & 15));
#pragma unroll
      for (int d0 = 0; d0 < Cfg::CPR; d0 += 2) {
        uint32_t x[4];  // pieces d0, d0 + 1 of keys 0-7 and 8-15
        ptx::ldmatrix_x4_trans(vb + paged_swz<RB>(vr, (uint32_t)(d0 + (lane >> 4))), x);
        if constexpr (E4M3) {  // a piece is 16 columns: the even ones and the odd ones
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            ptx::mma_bf16(acc[2 * (d0 + u)], pa, e4m3_lo_to_bf16x2(x[2 * u]), e4m3_lo_to_bf16x2(x[2 * u + 1]));
            ptx::mma_bf16(acc[2 * (d0 + u) + 1], pa, e4m3_hi_to_bf16x2(x[2 * u]), e4m3_hi_to_bf16x2(x[2 * u + 1]));
          }
        } else {
          ptx::mma_bf16(acc[d0], pa, x[0], x[1]);
          ptx::mma_bf16(acc[d0 + 1], pa, x[2], x[3]);
        }
      }
    }
  }
  ptx::cp_async_wait<0>();

  // ---- merge the key warps: rescale to the common reference, sum, divide
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
    l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
    if (c == 0) {
      s_m[kw * Cfg::ROWS + rw * 16 + gr + 8 * hf] = m[hf];
      s_l[kw * Cfg::ROWS + rw * 16 + gr + 8 * hf] = l[hf];
    }
  }
  __syncthreads();  // (also: every warp is done with the ring)
  float* so = reinterpret_cast<float*>(psm);
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const int r = rw * 16 + gr + 8 * hf;
    float mt = s_m[r];
#pragma unroll
    for (int k = 1; k < KW; ++k) mt = fmaxf(mt, s_m[k * Cfg::ROWS + r]);
    const float f = m[hf] == -INFINITY ? 0.f : ptx::ex2(m[hf] - mt);
    float* row = so + (kw * Cfg::ROWS + r) * Cfg::OSTR;
    if constexpr (E4M3) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        *reinterpret_cast<float4*>(row + 16 * i + 4 * c) =
            make_float4(acc[2 * i][2 * hf] * f, acc[2 * i + 1][2 * hf] * f, acc[2 * i][2 * hf + 1] * f,
                        acc[2 * i + 1][2 * hf + 1] * f);
    } else {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(row + 8 * i + 2 * c) = make_float2(acc[i][2 * hf] * f, acc[i][2 * hf + 1] * f);
    }
  }
  __syncthreads();
  constexpr int PPR = D / 8;  // 8-column pieces of a row
  for (int i = tid; i < Cfg::ROWS * PPR; i += 128) {
    const int r = i / PPR, pc = i % PPR;
    if (row0 + r >= rows) break;
    float mt = s_m[r];
#pragma unroll
    for (int k = 1; k < KW; ++k) mt = fmaxf(mt, s_m[k * Cfg::ROWS + r]);
    float lt = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const float mk = s_m[k * Cfg::ROWS + r];
      if (mk != -INFINITY) lt += s_l[k * Cfg::ROWS + r] * ptx::ex2(mk - mt);
      else lt += s_l[k * Cfg::ROWS + r];  // 0, or NaN from scores that were NaN
      const float4* src = reinterpret_cast<const float4*>(so + (k * Cfg::ROWS + r) * Cfg::OSTR + 8 * pc);
      const float4 a = src[0], b = src[1];
      x[0] += a.x; x[1] += a.y; x[2] += a.z; x[3] += a.w;
      x[4] += b.x; x[5] += b.y; x[6] += b.z; x[7] += b.w;
    }
    const float inv = lt == 0.f ? 0.f : (E4M3 ? 256.f : 1.f) / lt;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = lt == 0.f ? 0.f : x[e] * inv;
    const float lse = lt == 0.f ? -INFINITY : (mt == -INFINITY ? lt : (mt + log2f(lt)) * 0.6931471805599453f);
    const long long pr = row0 + r;
    const int t = sr.q0 + (int)(pr / g), h = kh * g + (int)(pr % g);
    if (nwin == 1) {
      reinterpret_cast<uint4*>(p.o + ((long long)t * p.Hq + h) * D)[pc] = pack8(x);
      if (pc == 0 && p.lse != nullptr) p.lse[(long long)h * p.Tq + t] = lse;
    } else {
      const long long at = ((long long)w * p.Tq + t) * p.Hq + h;
      float4* dst = reinterpret_cast<float4*>(p.o_part + at * D) + 2 * pc;
      dst[0] = make_float4(x[0], x[1], x[2], x[3]);
      dst[1] = make_float4(x[4], x[5], x[6], x[7]);
      if (pc == 0) p.lse_part[at] = lse;
    }
  }
}

// Merge of the windows of each (token, head): one warp per row, as
// attn_combine_kernel, for packed sequences: row t belongs to the sequence
// found by bisection, whose length gives its number of windows (rows of a
// single window are final already).
template <int D>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams p) {
  ptx::grid_dep_wait();
  constexpr int PER = D / 32;
  const long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (i >= (long long)p.Tq * p.Hq) return;
  const int t = (int)(i / p.Hq), h = (int)(i - (long long)t * p.Hq);
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
  if (s >= p.n_seqs) return;
  const SeqRange sr = paged_seq(p, s);
  if (t < sr.q0 || t >= sr.q0 + sr.nq || sr.len <= p.window) return;
  const int S = (sr.len + p.window - 1) / p.window;
  const long long str = (long long)p.Tq * p.Hq;
  float mx = -INFINITY;
  for (int w = lane; w < S; w += 32) mx = fmaxf(mx, p.lse_part[w * str + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float mu = mx == -INFINITY ? 0.f : mx;
  float acc[PER], wsum = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int w0 = 0; w0 < S; w0 += 32) {
    const float wl = w0 + lane < S ? expf(p.lse_part[(w0 + lane) * str + i] - mu) : 0.f;
    const int n = S - w0 < 32 ? S - w0 : 32;
    for (int j0 = 0; j0 < n; j0 += 8) {
      float wt[8], x[8][PER];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        wt[u] = __shfl_sync(0xffffffffu, wl, (j0 + u) & 31);
        const bool live = j0 + u < n && wt[u] != 0.f;  // uniform across the warp
#pragma unroll
        for (int e = 0; e < PER; ++e) x[u][e] = live ? p.o_part[((w0 + j0 + u) * str + i) * D + 32 * e + lane] : 0.f;
        if (!live) wt[u] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        wsum += wt[u];
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = fmaf(wt[u], x[u][e], acc[e]);
      }
    }
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
#pragma unroll
  for (int e = 0; e < PER; ++e) p.o[i * D + 32 * e + lane] = __float2bfloat16_rn(acc[e] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[(long long)h * p.Tq + t] = wsum == 0.f ? -INFINITY : mu + logf(wsum);
}

}  // namespace attn

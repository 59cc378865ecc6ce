// kv_cache.cuh -- the elementwise side of serving: norm and rotation of query
// and key heads, writing keys and values into a paged cache (bf16, or e4m3
// with a power-of-two scale per token and head) and reading them back.
//
// Per head row x of d elements (head_rows_kernel):
//   norm      y = x / sqrt(mean(x^2) + eps) * w          (keys and queries with a weight)
//   rotation  (a, b) -> (a c - b s, b c + a s), c, s = amplitude * (cos, sin)(p * freq)
//   e4m3      e = smallest integer with amax(|y|) <= 448 * 2^e, code = E4M3(y * 2^-e)
// all in fp32, rounded once at the end.  The angle p * freq is taken in fp64
// turns and reduced there (a position of 10^6 leaves an fp32 angle no more than
// a few bits), then sincospi in fp32.
//
// Both kernels are bound by HBM: every row is read once and written once.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "attn_common.cuh"
#include "e4m3.cuh"
#include "ptx.cuh"

namespace attn {

struct HeadRowsParams {
  long long T;
  // inputs: token t of x at x + t * stride (elements), heads contiguous
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  int Hq, Hkv;
  // dense outputs (rows of q always; rows of k unless they go to the cache)
  __nv_bfloat16 *q_out, *k_out;
  long long q_out_stride, k_out_stride;
  // cache modes: pages as [n_slots, Hkv, d]
  const long long* slots;
  long long n_slots;
  void *k_pages, *v_pages;
  unsigned char *k_exp, *v_exp;
  // norm and rotation
  const __nv_bfloat16 *q_weight, *k_weight;
  float eps, amplitude;
  const double* freqs;
  int rot;
  bool interleaved;
  const long long* positions;
  unsigned int* err;
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                    ptx::pack_bf16x2(x[6], x[7]));
}

// The exponent byte of a row, from the bits of its largest magnitude: e + 127
// with the smallest e with amax <= 448 * 2^e = 0.875 * 2^(e + 9), clamped so
// that 2^e, 2^-e and every code * 2^e down to the last subnormal code are exact
// in bf16; 127 for a row of zeros, 255 for a row that holds an infinity or a
// NaN (its bits are the largest).
__device__ __forceinline__ uint32_t e4m3_row_exponent(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return kExpNaN;
  if (amax_bits == 0u) return 127u;
  const int x = (int)(amax_bits >> 23) - 126;  // amax = m * 2^x, m in [0.5, 1) (subnormals end at the lower clamp)
  const int e = (amax_bits & 0x7FFFFFu) <= 0x600000u ? x - 9 : x - 8;
  return (uint32_t)((e < -118 ? -118 : e) + 127);
}

// D / 8 lanes hold one head row, 8 elements each as two groups of four, placed so
// that both members of a rotated pair are in one lane (nothing is exchanged for the
// rotation): in the half layout lane l holds [4l, 4l + 4) of the rotated part's
// first half and the same of its second half, and the lanes behind share the rest
// of the row; interleaved, 8 neighbours.  Either way a lane's pairs are 4l .. 4l + 3.
//
// A block takes `tokens` neighbouring tokens: their cosines and sines once, into
// shared memory, then set after set of rows (one row per lane group), each for all
// the tokens.  Every thread copies its own pieces of the next three steps into a
// ring in shared memory that no other thread touches, so loads go on under the
// arithmetic and across sets, and nothing is waited for but the thread's own
// copies.  A lane group stays with its head for a set, so weights and pointers are
// loop constants.  8192 tokens of 32 + 8 heads of 128 take 35 us (4.8 TB/s); with
// four tokens' loads into registers and no ring 39, with a ring of 8 steps 36.7,
// with more threads a SM 48 (their registers spill).
constexpr int kHeadRowsMaxTokens = 16, kHeadRowsAhead = 4, kHeadRowsBps = 4;
enum : int { kRowsDense = 0, kRowsBf16Cache = 1, kRowsE4m3Cache = 2 };

template <int D, bool INTERLEAVED, int MODE>
__global__ void __launch_bounds__(256, kHeadRowsBps) head_rows_kernel(const HeadRowsParams p, int tokens) {
  constexpr int G = D / 8;           // lanes per row
  constexpr int NG = 256 / G;        // rows of a set
  constexpr int U = kHeadRowsAhead;
  __shared__ __align__(16) float s_cos[kHeadRowsMaxTokens][D / 2], s_sin[kHeadRowsMaxTokens][D / 2];
  __shared__ uint2 s_in[U][2][256];  // (only the thread itself touches its places)
  const int gid = threadIdx.x / G, l = threadIdx.x % G;
  const long long t0 = (long long)blockIdx.x * tokens;
  const int nt = p.T - t0 < tokens ? (int)(p.T - t0) : tokens;
  const int rows = p.Hq + p.Hkv + (MODE != kRowsDense ? p.Hkv : 0);
  const int half = p.rot / 2;
  // this lane's two groups of a row, in elements
  const bool rotated = 4 * l < half;
  const int ea = INTERLEAVED || half == 0 ? 8 * l : (rotated ? 4 * l : p.rot + 8 * (l - half / 4));
  const int eb = !INTERLEAVED && rotated ? half + 4 * l : ea + 4;
  // the warp's steps: set after set, the tokens of each in turn
  const int r_first = (int)blockIdx.y * NG + gid, r_warp = r_first - (int)(threadIdx.x & 31) / G;
  const int r_step = (int)gridDim.y * NG;
  const int steps = r_warp < rows ? ((rows - r_warp + r_step - 1) / r_step) * nt : 0;
  // loads run U - 1 steps ahead of the arithmetic
  const uint32_t slot0 = ptx::smem_u32(&s_in[0][0][threadIdx.x]);
  constexpr uint32_t SLOT = sizeof(uint2) * 2 * 256, SIDE = sizeof(uint2) * 256;
  int lr = r_first - r_step, li = nt, lk = 0;
  const __nv_bfloat16* lp = nullptr;
  long long l_step = 0;
  auto load = [&]() {
    if (lk < steps) {
      if (li == nt) {
        li = 0;
        lr += r_step;
        const bool is_q = lr < p.Hq, is_v = MODE != kRowsDense && lr >= p.Hq + p.Hkv;
        const int h = is_q ? lr : (is_v ? lr - p.Hq - p.Hkv : lr - p.Hq);
        l_step = is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride);
        lp = (is_q ? p.q : (is_v ? p.v : p.k)) + t0 * l_step + (long long)h * D;
      }
      if (lr < rows) {
        const uint32_t at = slot0 + (uint32_t)(lk % U) * SLOT;
        ptx::cp_async8(at, lp + ea);
        ptx::cp_async8(at + SIDE, lp + eb);
      }
      lp += l_step;
      ++li;
      ++lk;
    }
    ptx::cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < U - 1; ++i) load();
  if (half > 0) {
    for (int i = threadIdx.x; i < nt * half; i += 256) {
      const int t = i / half, j = i - t * half;
      const double turns = (double)__ldg(p.positions + t0 + t) * (__ldg(p.freqs + j) * 0.15915494309189533577);
      float s, c;
      sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
      s_cos[t][j] = c * p.amplitude;
      s_sin[t][j] = s * p.amplitude;
    }
    __syncthreads();
  }
  int k = 0;
  for (int r = r_first; k < steps; r += r_step) {
    const bool live = r < rows, is_q = r < p.Hq, is_v = MODE != kRowsDense && r >= p.Hq + p.Hkv;
    const int h = is_q ? r : (is_v ? r - p.Hq - p.Hkv : r - p.Hq);
    // where dense rows go; the cache's rows follow the tokens' slots
    const bool dense = MODE == kRowsDense || is_q;
    const long long out_step = is_q ? p.q_out_stride : p.k_out_stride;
    __nv_bfloat16* out = dense && live ? (is_q ? p.q_out : p.k_out) + t0 * out_step + (long long)h * D : nullptr;
    const __nv_bfloat16* w = is_v || !live ? nullptr : (is_q ? p.q_weight : p.k_weight);
    float wf[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (w != nullptr) {
      const uint2 wa = __ldg(reinterpret_cast<const uint2*>(w + ea)), wb = __ldg(reinterpret_cast<const uint2*>(w + eb));
      unpack8(make_uint4(wa.x, wa.y, wb.x, wb.y), wf);
    }
    const bool turn = rotated && !is_v;
#pragma unroll 1
    for (int i = 0; i < nt; ++i, ++k) {
      load();
      ptx::cp_async_wait<U - 1>();
      const uint2 ra = s_in[k % U][0][threadIdx.x], rb = s_in[k % U][1][threadIdx.x];
      float x[8];
      unpack8(make_uint4(ra.x, ra.y, rb.x, rb.y), x);
      // (the shuffles below run on every lane: all 32 lanes of a warp stay together)
      if (p.q_weight != nullptr || p.k_weight != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = w != nullptr ? rsqrtf(ss * (1.f / D) + p.eps) : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= wf[e] * inv;
      }
      if (turn) {
        const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[i][4 * l]);
        const float4 s4 = *reinterpret_cast<const float4*>(&s_sin[i][4 * l]);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          constexpr int A = INTERLEAVED ? 2 : 1, B = INTERLEAVED ? 1 : 4;  // pair e: elements A e and A e + B
          const float a0 = x[A * e], b0 = x[A * e + B];
          x[A * e] = a0 * c[e] - b0 * s[e];
          x[A * e + B] = b0 * c[e] + a0 * s[e];
        }
      }
      if (dense) {
        if (live) {
          const uint4 y = pack8(x);
          *reinterpret_cast<uint2*>(out + ea) = make_uint2(y.x, y.y);
          *reinterpret_cast<uint2*>(out + eb) = make_uint2(y.z, y.w);
        }
        out += out_step;
      }
      if constexpr (MODE != kRowsDense) {
        long long slot = __ldg(p.slots + t0 + i);
        if (slot >= p.n_slots) {
          if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.err, kErrIndex);
          slot = -1;
        }
        const bool store = live && !is_q && slot >= 0;
        const long long row = slot * p.Hkv + h;
        if constexpr (MODE == kRowsBf16Cache) {
          if (store) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.v_pages : p.k_pages) + row * D;
            const uint4 y = pack8(x);
            *reinterpret_cast<uint2*>(dst + ea) = make_uint2(y.x, y.y);
            *reinterpret_cast<uint2*>(dst + eb) = make_uint2(y.z, y.w);
          }
        } else {
          uint32_t a = 0u;  // the largest magnitude, by its bits
#pragma unroll
          for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
          const uint32_t e = e4m3_row_exponent(a);
          const float m = __uint_as_float((e == kExpNaN ? 127u : 254u - e) << 23);  // 2^-(e - 127)
          if (store) {
            unsigned char* dst = static_cast<unsigned char*>(is_v ? p.v_pages : p.k_pages) + row * D;
            *reinterpret_cast<uint32_t*>(dst + ea) = ptx::pack_e4m3x4(x[0] * m, x[1] * m, x[2] * m, x[3] * m);
            *reinterpret_cast<uint32_t*>(dst + eb) = ptx::pack_e4m3x4(x[4] * m, x[5] * m, x[6] * m, x[7] * m);
            if (l == 0) (is_v ? p.v_exp : p.k_exp)[row] = (unsigned char)e;
          }
        }
      }
    }
  }
}

// Output rows: packed sequences (cu), or sequence s at rows s * stride .. (lens).
struct KvReadParams {
  const int* lens;  // with stride: tokens of each sequence, clamped to it
  int stride;
  const void *k_pages, *v_pages;
  const unsigned char *k_exp, *v_exp;
  int n_pages, page_shift, Hkv, n_seqs, table_width;
  const int *table, *cu;
  __nv_bfloat16 *k, *v;
  long long T;
  unsigned int* err;
};

// One warp per token: its sequence by bisection over the boundaries, its page
// from the table, then the token's Hkv * d contiguous values of K and of V, 16
// bytes read per lane and step.  Bound by HBM (4 tokens a warp, with fewer warps to
// hide the two look-ups: 127 us instead of 100 on 62000 tokens of 8 x 128 e4m3).
template <int D, bool E4M3>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadParams p) {
  constexpr int PE = E4M3 ? 16 : 8;  // elements of a piece
  const long long t = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= p.T) return;
  int lo = 0;  // the token's sequence
  long long start;
  if (p.stride > 0) {
    lo = (int)(t / p.stride);
    start = (long long)lo * p.stride;
    if (t - start >= __ldg(p.lens + lo)) return;
  } else {
    int hi = p.n_seqs;  // the last s with cu[s] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if ((long long)__ldg(p.cu + mid) <= t) lo = mid; else hi = mid - 1;
    }
    start = __ldg(p.cu + lo);
    if (lo >= p.n_seqs || start > t) return;  // behind the last sequence, or in front of the first
  }
  const long long pos = t - start, pi = pos >> p.page_shift;
  int page = -1;
  if (start >= 0 && pi < p.table_width) page = __ldg(p.table + (long long)lo * p.table_width + pi);
  const bool ok = page >= 0 && page < p.n_pages;
  if (!ok && lane == 0) atomicOr(p.err, kErrIndex);
  const long long row = ok ? (((long long)page << p.page_shift) + (pos & ((1 << p.page_shift) - 1))) * p.Hkv : 0;
  const int n = p.Hkv * (D / PE);
  uint4* ko = reinterpret_cast<uint4*>(p.k + t * p.Hkv * D);
  uint4* vo = reinterpret_cast<uint4*>(p.v + t * p.Hkv * D);
  const uint4* ki = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_pages) + row * D * (E4M3 ? 1 : 2));
  const uint4* vi = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v_pages) + row * D * (E4M3 ? 1 : 2));
#pragma unroll 2
  for (int c = lane; c < n; c += 32) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint4* out = x == 0 ? ko : vo;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (ok) w = __ldg((x == 0 ? ki : vi) + c);
      if constexpr (!E4M3) {
        out[c] = w;
      } else {
        const E4m3Factor f = e4m3_factor(ok ? __ldg((x == 0 ? p.k_exp : p.v_exp) + row + c / (D / PE)) : 127u);
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[8];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          o[2 * y] = bf16x2_mul(bf16x2_mul(e4m3_hi_bits(__byte_perm(in[y], 0u, 0x1404)), f.m), f.more);
          o[2 * y + 1] = bf16x2_mul(bf16x2_mul(e4m3_hi_bits(__byte_perm(in[y], 0u, 0x3424)), f.m), f.more);
        }
        out[2 * c] = make_uint4(o[0], o[1], o[2], o[3]);
        out[2 * c + 1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

}  // namespace attn

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
  // inputs: token t of x at x + t * stride (elements), heads contiguous
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  int Hq, Hkv;
  bool has_v;
  // dense outputs (rows of q always; rows of k unless they go to the cache)
  __nv_bfloat16 *q_out, *k_out;
  long long q_out_stride, k_out_stride;
  // cache (to_cache): pages as [n_slots, Hkv, d]
  bool to_cache;
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

// D / 8 lanes hold one head row, 8 elements (16 bytes) each; a group of lanes
// takes UNROLL rows of one token, loaded together.  A block holds the rows
// [blockIdx.y * rows per block, ...) of one token; the cosines and sines of
// the token's position are computed once per block, into shared memory.
template <int D, int UNROLL>
__global__ void __launch_bounds__(256) head_rows_kernel(const HeadRowsParams p) {
  constexpr int G = D / 8;           // lanes per row
  constexpr int NG = 256 / G;        // rows in flight per block and round
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  const long long t = blockIdx.x;
  const int gid = threadIdx.x / G, l = threadIdx.x % G;
  const int rows = p.Hq + p.Hkv + (p.has_v ? p.Hkv : 0);
  const int r0 = blockIdx.y * (NG * UNROLL) + gid;
  uint4 raw[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int r = r0 + u * NG;
    raw[u] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const __nv_bfloat16* src = r < p.Hq ? p.q + t * p.q_stride + (long long)r * D
                                 : r < p.Hq + p.Hkv ? p.k + t * p.k_stride + (long long)(r - p.Hq) * D
                                                    : p.v + t * p.v_stride + (long long)(r - p.Hq - p.Hkv) * D;
      raw[u] = *reinterpret_cast<const uint4*>(src + 8 * l);
    }
  }
  long long slot = -1;
  if (p.to_cache) {
    slot = __ldg(p.slots + t);
    if (slot >= p.n_slots) {
      slot = -1;
      if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.err, kErrIndex);
    }
  }
  const int half = p.rot / 2;
  if (half > 0) {
    if ((int)threadIdx.x < half) {
      const double turns = (double)__ldg(p.positions + t) * __ldg(p.freqs + threadIdx.x) * 0.15915494309189533577;
      float s, c;
      sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
      s_cos[threadIdx.x] = c * p.amplitude;
      s_sin[threadIdx.x] = s * p.amplitude;
    }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int r = r0 + u * NG;
    const bool live = r < rows;
    const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
    float x[8];
    unpack8(raw[u], x);
    const __nv_bfloat16* w = is_v ? nullptr : (is_q ? p.q_weight : p.k_weight);
    // (the shuffles below run on every lane: all 32 lanes of a warp stay together)
    if (p.q_weight != nullptr || p.k_weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (w != nullptr) {
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
        float wf[8];
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * l), wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv * wf[i];
      }
    }
    if (half > 0) {
      if (p.interleaved) {
        if (!is_v && 8 * l < p.rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float c = s_cos[4 * l + i], s = s_sin[4 * l + i];
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * c - b * s;
            x[2 * i + 1] = b * c + a * s;
          }
        }
      } else {
        const int hl = half / 8;  // lanes of one half
        const int partner = l < hl ? l + hl : (l < 2 * hl ? l - hl : l);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner, G);
        if (!is_v && l < 2 * hl) {
          const int c0 = 8 * (l < hl ? l : l - hl);
          const float sign = l < hl ? -1.f : 1.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * s_cos[c0 + i] + sign * (y[i] * s_sin[c0 + i]);
        }
      }
    }
    if (!p.to_cache || is_q) {
      if (live) {
        __nv_bfloat16* dst = is_q ? p.q_out + t * p.q_out_stride + (long long)r * D
                                  : p.k_out + t * p.k_out_stride + (long long)(r - p.Hq) * D;
        *reinterpret_cast<uint4*>(dst + 8 * l) = pack8(x);
      }
    }
    if (p.to_cache) {
      const int h = is_v ? r - p.Hq - p.Hkv : r - p.Hq;
      const bool store = live && !is_q && slot >= 0;
      const long long row = slot * p.Hkv + h;
      if (p.k_exp == nullptr) {
        if (store)
          reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(is_v ? p.v_pages : p.k_pages) + row * D)[l] = pack8(x);
      } else {
        uint32_t a = 0u;  // the largest magnitude, by its bits
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
          a = a > b ? a : b;
        }
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) {
          const uint32_t b = __shfl_xor_sync(0xffffffffu, a, o);
          a = a > b ? a : b;
        }
        const uint32_t e = e4m3_row_exponent(a);
        const float m = __uint_as_float((e == kExpNaN ? 127u : 254u - e) << 23);  // 2^-(e - 127)
        if (store) {
          const uint2 codes = make_uint2(ptx::pack_e4m3x4(x[0] * m, x[1] * m, x[2] * m, x[3] * m),
                                         ptx::pack_e4m3x4(x[4] * m, x[5] * m, x[6] * m, x[7] * m));
          reinterpret_cast<uint2*>(reinterpret_cast<unsigned char*>(is_v ? p.v_pages : p.k_pages) + row * D)[l] = codes;
          if (l == 0) (is_v ? p.v_exp : p.k_exp)[row] = (unsigned char)e;
        }
      }
    }
  }
}

struct KvReadParams {
  const void *k_pages, *v_pages;
  const unsigned char *k_exp, *v_exp;
  int n_pages, page_shift, Hkv, n_seqs, table_width;
  const int *table, *cu;
  __nv_bfloat16 *k, *v;
  long long T;
  unsigned int* err;
};

// One warp per token: its sequence by bisection over the boundaries, its page
// from the table, then Hkv * d contiguous values of K and of V (16 bytes of
// output per lane and step).
template <int D, bool E4M3>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadParams p) {
  const long long t = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= p.T) return;
  int lo = 0, hi = p.n_seqs;  // the last s with cu[s] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if ((long long)__ldg(p.cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  if (lo >= p.n_seqs) return;  // behind the last sequence
  const int start = __ldg(p.cu + lo);
  if (start > t) return;       // in front of the first
  const long long pos = t - start;
  const long long pi = pos >> p.page_shift;
  int page = -1;
  if (start >= 0 && pi < p.table_width) page = __ldg(p.table + (long long)lo * p.table_width + pi);
  const bool ok = page >= 0 && page < p.n_pages;
  if (!ok && lane == 0) atomicOr(p.err, kErrIndex);
  const long long row = ok ? (((long long)page << p.page_shift) + (pos & ((1 << p.page_shift) - 1))) * p.Hkv : 0;
  const int n = p.Hkv * (D / 8);  // 8-element pieces of a token
  for (int c = lane; c < n; c += 32) {
    uint4 w[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const void* src = x == 0 ? p.k_pages : p.v_pages;
      w[x] = make_uint4(0u, 0u, 0u, 0u);
      if (!ok) continue;
      if constexpr (!E4M3) {
        w[x] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(src) + row * D) + c);
      } else {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const unsigned char*>(src) + row * D) + c);
        const uint32_t e = __ldg((x == 0 ? p.k_exp : p.v_exp) + row + c / (D / 8));
        const E4m3Factor f = e4m3_factor(e);
        const uint32_t h[4] = {__byte_perm(q.x, 0u, 0x1404), __byte_perm(q.x, 0u, 0x3424), __byte_perm(q.y, 0u, 0x1404),
                               __byte_perm(q.y, 0u, 0x3424)};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = bf16x2_mul(bf16x2_mul(e4m3_hi_bits(h[i]), f.m), f.more);
        w[x] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    reinterpret_cast<uint4*>(p.k + t * p.Hkv * D)[c] = w[0];
    reinterpret_cast<uint4*>(p.v + t * p.Hkv * D)[c] = w[1];
  }
}

}  // namespace attn

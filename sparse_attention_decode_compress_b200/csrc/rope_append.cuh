// qsa_rope_append: rotary positions on new queries and keys, and the append of
// the new K/V rows to the paged cache, in one pass.
//
// A head's first R dims are R / 2 pairs (x_a, x_b); pair i of the token at
// position p turns by the angle p * f_i:
//   y_a = m (x_a cos - x_b sin),  y_b = m (x_a sin + x_b cos)
// (m: a factor on both, 1 unless the scaling sets it).  "Half" layout: a = i,
// b = i + R/2; interleaved: a = 2i, b = 2i + 1.  The dims behind R and the
// values pass unchanged.
//
// Angles: f_i is kept as a fraction of a turn in 64-bit fixed point, so
// p * f_i in wrapping 64-bit integers is the exact position on the circle for
// any p: no float product whose error grows with the position, and no range
// reduction.  The top 32 bits go to sincospif (float32 rounding: at most
// 2^-24 half turns).
//
// Bound: HBM, each input read and each output written once.  A warp owns a
// token (or a share of its heads): the two angles a lane computes are passed
// around by shuffles, every lane keeps the 8 (cos, sin) pairs of its place in
// the head and applies them to one head after another, 16 bytes at a time.
// Measured (B200): 22,152 tokens of 32 / 4 heads, D 128, bf16: 74.7 us, 6.1 TB/s
// (94 % of the measured copy rate); 4,096 tokens of 16 / 2 heads: 11.3 us (one
// wave of warps, whose chain request -> position -> page -> store is exposed);
// 128 tokens: 2.8 us in a graph.  16,384 tokens of 32 / 4 heads, L2 flushed: bf16
// 59.4 us, from bf16 into fp8 pages 71.7, float32 106.6 (floors 51.9, 49.4, 103.9).
#pragma once
#include "qsa_common.cuh"

namespace qsa {
namespace rope {

struct Params {
  CacheDev c;
  int B, n_tok, Hq;
  const int32_t *pos0, *cu;  // [B], [B + 1]
  const void *q, *k, *v;     // [n_tok, heads, D], token strides below
  long long q_stride, k_stride, v_stride;  // elements
  const uint64_t *freqs;     // [R / 2] turns per token, 2^-64 units
  int R;
  float mscale;
  void *q_out;  // [n_tok, Hq, D]
};

constexpr int kThreads = 128;

// The request of token `tok` (cu[r] <= tok < cu[r + 1]) or -1, by a whole
// warp: 32 offsets are compared at a time.
__device__ __forceinline__ int request_of(const int32_t *cu, int B, int tok, int lane) {
  int lo = 0, n = B;  // the request is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + min(lane * step, n);
    const bool le = lane * step < n && cu[at] <= tok;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0u) return -1;
    const int k = 31 - __clz(m);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return (cu[lo] <= tok && tok < cu[lo + 1]) ? lo : -1;
}

__device__ __forceinline__ void sincos_turns(uint64_t phase, float m, float &s, float &c) {
  const float x = (float)(int32_t)(uint32_t)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31
  sincospif(x, &s, &c);
  s *= m;
  c *= m;
}

// A pair turned by (c, s) = m (cos, sin); the same roundings in every form of
// the kernel.
__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s) {
  const float x = a;
  a = __fmaf_rn(x, c, -__fmul_rn(b, s));
  b = __fmaf_rn(x, s, __fmul_rn(b, c));
}

// 8 consecutive elements as float32 and back.
struct Raw8f {
  float4 a, b;
};
__device__ __forceinline__ Raw8f ld8(const float *p) {
  Raw8f r;
  r.a = *reinterpret_cast<const float4 *>(p);
  r.b = *reinterpret_cast<const float4 *>(p + 4);
  return r;
}
__device__ __forceinline__ uint4 ld8(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void unpack8(const Raw8f &r, float (&x)[8]) {
  x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w;
  x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}
__device__ __forceinline__ void unpack8(const uint4 &r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void st8(float *p, const float (&x)[8], float) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16 *p, const float (&x)[8], float) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// E4M3 codes of x / scale, rounded to nearest even, saturated at 448.
__device__ __forceinline__ uint32_t codes2(float x, float y, float scale) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x, scale), __fdiv_rn(y, scale)),
                                            __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ void st8(__nv_fp8_e4m3 *p, const float (&x)[8], float scale) {
  uint2 w;
  w.x = codes2(x[0], x[1], scale) | codes2(x[2], x[3], scale) << 16;
  w.y = codes2(x[4], x[5], scale) | codes2(x[6], x[7], scale) << 16;
  *reinterpret_cast<uint2 *>(p) = w;
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void st1(float *p, float x, float) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16 *p, float x, float) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void st1(__nv_fp8_e4m3 *p, float x, float scale) {
  p->__x = __nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3);
}

// Where the K/V row of a token goes: cache row (of Hkv heads), or -1.
__device__ __forceinline__ long long cache_row(const Params &p, long long pos, int r, int &page) {
  const long long lp = pos < 0 ? -1 : pos <= 0x7fffffff ? (int)pos / p.c.page_size : pos / p.c.page_size;
  page = physical_page(p.c, r, lp);
  return page < 0 ? -1 : (long long)page * p.c.page_size + (pos - lp * p.c.page_size);
}

// Vector form: R a multiple of 16, rows 16-byte aligned.  Each head is D / 16
// units of two 8-element chunks: unit u < R / 16 holds the pairs 8u .. 8u + 7
// (half: chunks u and u + R/16; interleaved: chunks 2u and 2u + 1), the units
// behind them two unrotated chunks.  A lane stays at one unit and goes
// through the heads, 32 / (D / 16) heads a step; a warp takes NB steps.
template <int D, typename T, typename CT, bool INTERLEAVED, int NB>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(Params p) {
  pdl_open();
  constexpr int kUnits = D / 16;
  constexpr int kHeads = 32 / kUnits;  // heads of one step
  const int lane = threadIdx.x & 31;
  const int heads = p.Hq + 2 * p.c.num_kv_heads;
  const int parts = (heads + kHeads * NB - 1) / (kHeads * NB);
  const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int tok = (int)(w / parts);
  if (tok >= p.n_tok) return;
  const int part = (int)(w - (long long)tok * parts);
  const int u = lane % kUnits, h0 = part * NB * kHeads + lane / kUnits;
  const int ru = p.R / 16;
  const bool turn = u < ru;
  const int c0 = turn ? (INTERLEAVED ? 2 * u : u) : 2 * u;
  const int c1 = turn ? (INTERLEAVED ? 2 * u + 1 : u + ru) : 2 * u + 1;
  const int Hk = p.c.num_kv_heads;
  using Raw = decltype(ld8(static_cast<const T *>(nullptr)));
  Raw x[NB][2];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int h = h0 + j * kHeads;
    if (h < heads) {
      const T *src = h < p.Hq ? static_cast<const T *>(p.q) + tok * p.q_stride + h * D
                     : h < p.Hq + Hk ? static_cast<const T *>(p.k) + tok * p.k_stride + (h - p.Hq) * D
                                     : static_cast<const T *>(p.v) + tok * p.v_stride + (h - p.Hq - Hk) * D;
      x[j][0] = ld8(src + 8 * c0);
      x[j][1] = ld8(src + 8 * c1);
    }
  }
  // lane i: pairs 2i and 2i + 1
  uint64_t fr[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (2 * lane + e < p.R / 2) fr[e] = p.freqs[2 * lane + e];
  const int r = request_of(p.cu, p.B, tok, lane);
  if (r < 0) return;  // a row behind the last request
  const long long pos = (long long)p.pos0[r] + (tok - p.cu[r]);
  int page;
  const long long row = cache_row(p, pos, r, page);
  float sn[2], cs[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) sincos_turns((uint64_t)pos * fr[e], p.mscale, sn[e], cs[e]);
  float s8[8], c8[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s8[i] = __shfl_sync(0xffffffffu, sn[i & 1], (4 * u + (i >> 1)) & 31);
    c8[i] = __shfl_sync(0xffffffffu, cs[i & 1], (4 * u + (i >> 1)) & 31);
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int h = h0 + j * kHeads;
    if (h >= heads) continue;
    float a[8], b[8];
    unpack8(x[j][0], a);
    unpack8(x[j][1], b);
    if (turn && h < p.Hq + Hk) {
      if (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          turn_pair(a[2 * i], a[2 * i + 1], c8[i], s8[i]);
          turn_pair(b[2 * i], b[2 * i + 1], c8[4 + i], s8[4 + i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], c8[i], s8[i]);
      }
    }
    if (h < p.Hq) {
      T *dst = static_cast<T *>(p.q_out) + ((long long)tok * p.Hq + h) * D;
      st8(dst + 8 * c0, a, 1.f);
      st8(dst + 8 * c1, b, 1.f);
    } else if (row >= 0) {
      const bool is_k = h < p.Hq + Hk;
      const int hk = h - p.Hq - (is_k ? 0 : Hk);
      CT *dst = static_cast<CT *>(const_cast<void *>(is_k ? p.c.k_cache : p.c.v_cache)) + (row * Hk + hk) * D;
      const float *sc = is_k ? p.c.k_scale : p.c.v_scale;
      const float scale = sizeof(CT) == 1 ? sc[(long long)page * Hk + hk] : 1.f;
      st8(dst + 8 * c0, a, scale);
      st8(dst + 8 * c1, b, scale);
    }
  }
}

// Any even R and any alignment: one warp per token, one pair or unrotated
// dim of a head per lane.
template <int D, typename T, typename CT>
__global__ void __launch_bounds__(kThreads) rope_append_any_kernel(Params p, int interleaved) {
  pdl_open();
  const int lane = threadIdx.x & 31;
  const int tok = (int)(((long long)blockIdx.x * kThreads + threadIdx.x) >> 5);
  if (tok >= p.n_tok) return;
  const int r = request_of(p.cu, p.B, tok, lane);
  if (r < 0) return;
  const long long pos = (long long)p.pos0[r] + (tok - p.cu[r]);
  int page;
  const long long row = cache_row(p, pos, r, page);
  const int Hk = p.c.num_kv_heads, heads = p.Hq + 2 * Hk, half = p.R / 2;
  for (int e = lane; e < half + (D - p.R); e += 32) {
    const bool pair = e < half;
    float sn = 0.f, cs = 1.f;
    if (pair) sincos_turns((uint64_t)pos * p.freqs[e], p.mscale, sn, cs);
    const int i0 = pair ? (interleaved ? 2 * e : e) : p.R + e - half;
    const int i1 = pair ? (interleaved ? 2 * e + 1 : e + half) : i0;
    for (int h = 0; h < heads; ++h) {
      const T *src = h < p.Hq ? static_cast<const T *>(p.q) + tok * p.q_stride + h * D
                     : h < p.Hq + Hk ? static_cast<const T *>(p.k) + tok * p.k_stride + (h - p.Hq) * D
                                     : static_cast<const T *>(p.v) + tok * p.v_stride + (h - p.Hq - Hk) * D;
      float a = to_f(src[i0]), b = to_f(src[i1]);
      if (pair && h < p.Hq + Hk) turn_pair(a, b, cs, sn);
      if (h < p.Hq) {
        T *dst = static_cast<T *>(p.q_out) + ((long long)tok * p.Hq + h) * D;
        st1(dst + i0, a, 1.f);
        if (pair) st1(dst + i1, b, 1.f);
      } else if (row >= 0) {
        const bool is_k = h < p.Hq + Hk;
        const int hk = h - p.Hq - (is_k ? 0 : Hk);
        CT *dst = static_cast<CT *>(const_cast<void *>(is_k ? p.c.k_cache : p.c.v_cache)) + (row * Hk + hk) * D;
        const float *sc = is_k ? p.c.k_scale : p.c.v_scale;
        const float scale = sizeof(CT) == 1 ? sc[(long long)page * Hk + hk] : 1.f;
        st1(dst + i0, a, scale);
        if (pair) st1(dst + i1, b, scale);
      }
    }
  }
}

}  // namespace rope
}  // namespace qsa

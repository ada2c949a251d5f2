// Attention over key ranges on the CUDA cores, in float32 throughout: the
// kernel of float32 caches.
//
// One CTA of 4 warps takes a tile of 16 query rows of one sequence and kv
// head and one split of its keys.  32 keys at a time are staged in shared
// memory (cp.async, the next tile in flight while one is computed, its pages
// looked up one more tile ahead); a lane owns a key for the scores (its row
// padded against bank conflicts) and a slice of the head dimension for the
// values, a warp owns 4 query rows, and the softmax runs online (running maximum
// and sum).  Measured (B200): one request of 8 / 1 heads, D 64, 1,028 keys: 11.2
// us a call with the merge, and as long in a graph, so the two kernels bound it:
// latency of 17 CTAs of two key tiles, one behind the other, then of the merge
// (alone and cold 11.8 and 6.8 us).  256 tokens of 8 / 1 heads over 4,096 keys,
// D 128: 300 us, 14 TFLOP/s.
#pragma once
#include "attn_common.cuh"

namespace qsa {
namespace attn {

constexpr int kSimpleThreads = 128;
constexpr int kSimpleRows = 16;
constexpr int kSimpleKeys = 32;

template <int D>
struct SimpleSmem {
  float q[kSimpleRows][D];
  float k[2][kSimpleKeys][D + 4];
  float v[2][kSimpleKeys][D];
};

template <int MODE>
__device__ __forceinline__ float4 load4(const void *p, long long at) {
  return ld_mode<MODE>(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at));
}

// Grid (row tiles, Hkv * splits, sequences).
template <int MODE, int D>
__global__ void __launch_bounds__(kSimpleThreads) simple_kernel(Args a) {
  pdl_begin<MODE>();
  constexpr int kVec = D / 4;
  constexpr int kRowsPerWarp = kSimpleRows / 4;
  constexpr int kDims = D / 32;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimpleSmem<D> &sm = *reinterpret_cast<SimpleSmem<D> *>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Seq sq = sequence<MODE>(a, blockIdx.z);
  const int m0 = blockIdx.x * kSimpleRows;
  const int rows = min(kSimpleRows, sq.ntok * a.G - m0);
  if (rows <= 0) {
    pdl_end<MODE>();
    return;
  }
  const int g = blockIdx.y / a.splits, split = blockIdx.y - g * a.splits;
  const Range rg = range_of<MODE>(a, sq, m0 / a.G, (m0 + rows - 1) / a.G + 1);
  const int x0 = split_bound(rg.n, a.splits, split, kSimpleKeys);
  const int x1 = split_bound(rg.n, a.splits, split + 1, kSimpleKeys);

  for (int e = tid; e < kSimpleRows * kVec; e += kSimpleThreads) {
    const int m = e / kVec, d = e % kVec * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m < rows) {
      const int row = m0 + m;
      const long long at = ((long long)(sq.tok0 + row / a.G) * a.Hq + g * a.G + row % a.G) * D;
      v = load4<MODE>(a.q, at + d);
    }
    *reinterpret_cast<float4 *>(&sm.q[m][d]) = v;
  }
  Seen see[kRowsPerWarp];
  float mx[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][kDims];
#pragma unroll
  for (int j = 0; j < kRowsPerWarp; ++j) {
    const int m = warp * kRowsPerWarp + j;
    see[j].hi = see[j].lo = see[j].sink = 0;
    if (m < rows) see[j] = seen_by<MODE>(a, sq, (m0 + m) / a.G);
    mx[j] = -INFINITY;
    l[j] = 0.f;
#pragma unroll
    for (int i = 0; i < kDims; ++i) o[j][i] = 0.f;
  }

  // ---- loads: a warp owns the keys warp, warp + 4, .. of a tile; lane i < 8
  // holds the cache row of the i-th of them (-1: zeros)
  constexpr int kOwn = kSimpleKeys / 4;
  auto lookup = [&](int xt) -> long long {
    const int x = xt + warp + 4 * lane;
    if (lane >= kOwn || x >= x1) return -1;
    const int key = rg.key(x), lp = key / a.c.page_size;
    const int pg = physical_page<MODE == kTail>(a.c, sq.table, lp);
    return pg < 0 ? -1 : (long long)pg * a.c.page_size + (key - lp * a.c.page_size);
  };
  const float *kbase = static_cast<const float *>(a.c.k_cache) + (long long)g * D;
  const float *vbase = static_cast<const float *>(a.c.v_cache) + (long long)g * D;
  auto issue = [&](int buf, long long row) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = warp + 4 * i;
      const long long r = __shfl_sync(0xffffffffu, row, i);
      const long long at = r * a.c.num_kv_heads * D + 4 * (lane % kVec);
      if (lane < kVec) {
        cp_async16_zfill(&sm.k[buf][j][4 * lane], r >= 0 ? kbase + at : kbase, r >= 0);
        cp_async16_zfill(&sm.v[buf][j][4 * lane], r >= 0 ? vbase + at : vbase, r >= 0);
      }
    }
  };
  long long ahead = -1;
  if (x0 < x1) {
    issue(0, lookup(x0));
    ahead = lookup(x0 + kSimpleKeys);
  }
  cp_async_commit();
  int buf = 0;
  for (int xt = x0; xt < x1; xt += kSimpleKeys, buf ^= 1) {
    if (xt + kSimpleKeys < x1) {
      issue(buf ^ 1, ahead);
      ahead = lookup(xt + 2 * kSimpleKeys);
    }
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    float s[kRowsPerWarp];
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) s[j] = 0.f;
#pragma unroll 8
    for (int d = 0; d < D; d += 4) {
      const float4 k = *reinterpret_cast<const float4 *>(&sm.k[buf][lane][d]);
#pragma unroll
      for (int j = 0; j < kRowsPerWarp; ++j) {
        const float4 q = *reinterpret_cast<const float4 *>(&sm.q[warp * kRowsPerWarp + j][d]);
        s[j] += q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
      }
    }
    const int key = rg.key(xt + lane);
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
      const bool ok = xt + lane < x1 && sees(see[j], key);
      const float x = ok ? s[j] * a.scale_log2 : -INFINITY;
      float t = x;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
      const float m_new = fmaxf(mx[j], t);
      const float base = m_new == -INFINITY ? 0.f : m_new;
      const float al = m_new == -INFINITY ? 1.f : ex2(mx[j] - base);
      const float p = ex2(x - base);
      mx[j] = m_new;
      l[j] = l[j] * al + p;
#pragma unroll
      for (int i = 0; i < kDims; ++i) o[j][i] *= al;
      s[j] = p;
    }
#pragma unroll 4
    for (int t = 0; t < kSimpleKeys; ++t) {
      float v[kDims];
#pragma unroll
      for (int i = 0; i < kDims; ++i) v[i] = sm.v[buf][t][lane + 32 * i];
#pragma unroll
      for (int j = 0; j < kRowsPerWarp; ++j) {
        const float p = __shfl_sync(0xffffffffu, s[j], t);
#pragma unroll
        for (int i = 0; i < kDims; ++i) o[j][i] = p != 0.f ? fmaf(p, v[i], o[j][i]) : o[j][i];
      }
    }
    __syncthreads();  // the buffer is read
  }
  cp_async_wait<0>();

#pragma unroll
  for (int j = 0; j < kRowsPerWarp; ++j) {
    const int m = warp * kRowsPerWarp + j;
    if (m >= rows) continue;
    float t = l[j];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    // (a NaN sum stays one)
    const float inv = t != 0.f ? 1.f / t : 0.f;
    const float lse = t != 0.f ? ((mx[j] == -INFINITY ? 0.f : mx[j]) + __log2f(t)) * kLn2 : -INFINITY;
    const int row = m0 + m;
    const long long at = (long long)(sq.tok0 + row / a.G) * a.Hq + g * a.G + row % a.G;
    if (a.slots > 1) {
      const long long slot = at * a.slots + a.slot0 + split;
      if (lane == 0) a.lse_part[slot] = lse;
      // outside every group, or in a refused one: nothing else writes the shared slots
      if (MODE == kTail && split == 0 && !sq.shared)
        for (int k = lane; k < a.slot0; k += 32) a.lse_part[at * a.slots + k] = -INFINITY;
      if (t != 0.f) {
#pragma unroll
        for (int i = 0; i < kDims; ++i) a.o_part[slot * D + lane + 32 * i] = o[j][i] * inv;
      }
    } else {
      if (lane == 0) a.lse[at] = lse;
#pragma unroll
      for (int i = 0; i < kDims; ++i)
        static_cast<float *>(a.o)[at * D + lane + 32 * i] = o[j][i] * inv;
    }
  }
  pdl_end<MODE>();
}

}  // namespace attn
}  // namespace qsa

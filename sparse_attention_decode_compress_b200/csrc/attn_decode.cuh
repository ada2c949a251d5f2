// Attention of few query rows over key ranges, BF16 and FP8 caches: the decode
// form of qsa_window_decode and the tails of qsa_prefix_decode.
//
// At most 32 query rows (T query tokens x G heads) share a kv head's keys, so
// the work is a stream of K/V rows at 8 to 32 multiply-adds a byte: HBM bounds
// it.  Both products put the keys on the wide side of m16n8k16 tiles
// (S^T = K Q^T, O^T = V^T P^T), so 8 query rows fill a tile.  A CTA of 4 warps
// takes a split of one (request, kv head); each warp streams a contiguous part
// of it, 16 keys a stage, through its own cp.async ring with its own running
// maximum and sum (no barriers while it streams), and the four results are
// merged in shared memory.  The splits of a (request, kv head), up to 8, are a
// cluster that merges its results through distributed shared memory (a merge
// kernel behind it cost 4 us a call and the partial results' way to memory);
// only more splits, and tails, whose prefix part comes from another kernel, go
// through the workspace.  fp8 tiles go from shared memory into f16 fragments
// (fp8_frag.cuh).
//
// Weights p = exp(s - max) enter the value product rounded to bf16 (2^-8
// relative; o is rounded to bf16 itself) or, times the V scale, to f16 (2^-11, and
// what f8_ref says about small ones).
//
// Measured (B200): batch 32, 16 / 2 heads, window 4,096 + 64 keys, bf16: 27.4 us,
// 5.0 TB/s (77 % of the measured copy rate; one wave of CTAs starts and ends in
// that); four query tokens, batch 64, window 2,000: 39.5 us, 3.2 TB/s (32 rows a
// kv head: Q fragments come from shared memory at every stage, and 255 registers
// leave 1.7 warps a scheduler, which wait for the instruction before: it issues 34 %
// of the time); fp8, batch 256, 32 / 4 heads: 154 us, 4.5 TB/s (the same wait
// with 2.6 warps a scheduler: issue 54 %, ALU 52 %, and 2.3 waves of CTAs, the SMs
// active for 83 % of the kernel).
#pragma once
#include "attn_common.cuh"
#include "sparse_decode_warp.cuh"

namespace qsa {
namespace attn {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kStageKeys = 16;
constexpr int kMetaKeys = 128;  // keys whose pages a warp looks up at once: 4 a lane

// Growth of a column's scores (log2) over its reference that is left in the
// weights (bf16: below 2^8, which it holds as exactly as 1; f16: kF8Grow): the
// lanes then need not agree on a maximum at every stage.
template <bool FP8>
__host__ __device__ constexpr float dec_lazy() { return FP8 ? kF8Grow : 8.f; }

// Stages of a warp's ring: 96 KB (bf16) or 64 KB (fp8) of shared memory a CTA
// at D = 128, two and three CTAs an SM.
template <bool FP8>
__host__ __device__ constexpr int dec_stages() { return FP8 ? 4 : 3; }

template <int D, bool FP8, int NT>
struct DecSmem {
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kRing = dec_stages<FP8>() * 2 * kStageKeys * kRowBytes;  // per warp
  static constexpr int kOut = NT * 8 * D * 4;
  union {
    uint8_t ring[kDecWarps][kRing];
    float o[kDecWarps][NT * 8][D];
  };
  float m[kDecWarps][NT * 8], l[kDecWarps][NT * 8];
  float cm[NT * 8], cl[NT * 8];  // the CTA's: maximum and sum (its values: o[0])
  // more than 16 rows: their Q fragments (64 registers at 32 rows), by tile,
  // k-step and lane, and the rows' factor on the logits
  uint2 qf[NT > 2 ? NT : 1][NT > 2 ? D / 16 : 1][32];
  float qs[NT * 8];
};

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word or four words at `p` of this CTA's shared memory, in CTA `rank` of
// the cluster.
__device__ __forceinline__ uint32_t peer_at(const void *p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float peer_float(const float *p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_at(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_float4(const float *p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_at(p, rank))
               : "memory");
  return v;
}

// Grid (splits, Hkv, requests).
template <int MODE, int D, bool FP8, int NT>
__global__ void __launch_bounds__(kDecThreads, NT <= 2 ? 2 : 1) decode_kernel(Args a) {
  pdl_begin<MODE>();
  using namespace qsa::dec;
  constexpr int NS = dec_stages<FP8>();
  constexpr int MD = D / 16;
  constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  constexpr int kChunks = kRowBytes / 16;          // 16-byte chunks of a row
  constexpr int kTile = kStageKeys * kRowBytes;
  constexpr int kRowsPerIssue = 32 / kChunks;      // rows one cp.async of the warp covers
  using SM = DecSmem<D, FP8, NT>;
  extern __shared__ uint8_t smem_raw[];
  SM &sm = *reinterpret_cast<SM *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, cq = lane & 3;
  const int g = blockIdx.y, split = blockIdx.x, r = blockIdx.z;
  const Seq sq = sequence<MODE>(a, r);
  const Range rg = range_of<MODE>(a, sq, 0, a.T);
  const int x0 = split_bound(rg.n, a.splits, split, kStageKeys);
  const int x1 = split_bound(rg.n, a.splits, split + 1, kStageKeys);
  const int M = a.T * a.G, Hkv = a.c.num_kv_heads;
  const long long row_stride = (long long)Hkv * kRowBytes;  // bytes between tokens

  float o[MD][NT][4], mcol[NT][2], lcol[NT][2];
#pragma unroll
  for (int i = 0; i < MD; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    mcol[j][0] = mcol[j][1] = -INFINITY;
    lcol[j][0] = lcol[j][1] = 0.f;
  }
  float vsref = 0.f;  // power of two that the V scales are relative to (f8_ref)

  // fragments of rows 8 j .. 8 j + 7; returns row 8 j + gq's factor on the logits
  auto q_frags = [&](int j, uint32_t(&f)[MD][2]) -> float {
    const int m = 8 * j + gq;
    const __nv_bfloat16 *qrow =
        m < M ? static_cast<const __nv_bfloat16 *>(a.q) +
                    ((long long)(sq.tok0 + m / a.G) * a.Hq + g * a.G + m % a.G) * D
              : nullptr;
    if constexpr (FP8) {
      return q_frags_f16<D, MODE == kTail>(qrow, cq, f) * a.scale_log2;
    } else {
#pragma unroll
      for (int kk = 0; kk < MD; ++kk) {
        const uint32_t *at = reinterpret_cast<const uint32_t *>(qrow + 16 * kk + 2 * cq);
        f[kk][0] = qrow ? ld_mode<MODE>(at) : 0u;
        f[kk][1] = qrow ? ld_mode<MODE>(at + 4) : 0u;
      }
      return a.scale_log2;
    }
  };
  constexpr bool kQRegs = NT <= 2;
  if constexpr (!kQRegs) {
    if (warp < NT) {
      uint32_t f[MD][2];
      const float sc = q_frags(warp, f);
#pragma unroll
      for (int kk = 0; kk < MD; ++kk) sm.qf[warp][kk][lane] = make_uint2(f[kk][0], f[kk][1]);
      if (cq == 0) sm.qs[8 * warp + gq] = sc;
    }
    __syncthreads();
  }

  // this warp's part of the split
  const int w0 = x0 + split_bound(x1 - x0, kDecWarps, warp, kStageKeys);
  const int w1 = x0 + split_bound(x1 - x0, kDecWarps, warp + 1, kStageKeys);
  if (w0 < w1) {
    uint8_t *ring = sm.ring[warp];
    const uint8_t *kbase = static_cast<const uint8_t *>(a.c.k_cache) + (long long)g * kRowBytes;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.c.v_cache) + (long long)g * kRowBytes;
    // ---- pages: lane i holds the first token row of the four keys from
    // window start + 4 i on (-1: none), and their scales
    auto lookup = [&](int xw, long long &row, float &ks, float &vs) {
      const int x = xw + 4 * lane;
      row = -1;
      ks = vs = 0.f;
      if (x < w1) {
        const int key = rg.key(x);
        const int lp = key / a.c.page_size;
        const int pg = physical_page<MODE == kTail>(a.c, sq.table, lp);
        if (pg >= 0) {
          row = (long long)pg * a.c.page_size + (key - lp * a.c.page_size);
          if constexpr (FP8) {
            ks = ld_mode<MODE>(a.c.k_scale + (long long)pg * Hkv + g);
            vs = ld_mode<MODE>(a.c.v_scale + (long long)pg * Hkv + g);
          }
        }
      }
    };
    long long row_cur, row_next;
    float ks_cur, vs_cur, ks_next, vs_next;
    lookup(w0, row_cur, ks_cur, vs_cur);
    int win = w0;  // start of the window held in *_cur
    lookup(w0 + kMetaKeys, row_next, ks_next, vs_next);
    // the keys that some query of the request sees are loaded, the others of
    // a group of four (and past the end) are zero
    Seen any = seen_by<MODE>(a, sq, a.T - 1);
    if (MODE == kWindow) any.lo = window_lo(sq.first, a.window);
    // ---- issue of stage s (keys w0 + 16 s ..) into its slot
    auto issue = [&](int s) {
      const int xs = w0 + s * kStageKeys;
      uint8_t *kt = ring + (s % NS) * 2 * kTile, *vt = kt + kTile;
      const bool next = xs >= win + kMetaKeys;  // the prefetch is at most one window ahead
      const int base = (xs - win - (next ? kMetaKeys : 0)) >> 2;
#pragma unroll
      for (int i = 0; i < kStageKeys / kRowsPerIssue; ++i) {
        const int row = i * kRowsPerIssue + lane / kChunks, ch = lane % kChunks;
        const long long r0 = __shfl_sync(0xffffffffu, next ? row_next : row_cur, base + (row >> 2));
        const int x = xs + row;
        const int key = rg.key(x);
        const bool ok = x < w1 && r0 >= 0 && sees(any, key);
        const long long at = (r0 + (row & 3)) * row_stride + ch * 16;
        const int so = FP8 ? fp8_swz<D>(row, ch) : swz<D>(row, ch);
        cp_async16_zfill(kt + so, ok ? kbase + at : kbase, ok);
        cp_async16_zfill(vt + so, ok ? vbase + at : vbase, ok);
      }
    };
    const int nst = (w1 - w0 + kStageKeys - 1) / kStageKeys;
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      if (s < nst) issue(s);
      cp_async_commit();
    }
    // ---- Q as B fragments, rows past M zero
    uint32_t qb[kQRegs ? NT : 1][MD][2];
    float csc[NT][2];
    int rlo[NT][2], rhi[NT][2], rsink = MODE == kWindow ? a.sinks : 0;
    int all_lo = 0, all_hi = 0x7fffffff;  // keys in [all_lo, all_hi) are seen by every row
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if constexpr (kQRegs) {
        const float sc = q_frags(j, qb[j]);
        csc[j][0] = __shfl_sync(0xffffffffu, sc, 4 * (2 * cq));
        csc[j][1] = __shfl_sync(0xffffffffu, sc, 4 * (2 * cq + 1));
      } else {
        csc[j][0] = sm.qs[8 * j + 2 * cq];
        csc[j][1] = sm.qs[8 * j + 2 * cq + 1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int mm = 8 * j + 2 * cq + e;
        rlo[j][e] = rhi[j][e] = 0;
        if (mm < M) {
          const Seen v = seen_by<MODE>(a, sq, mm / a.G);
          rlo[j][e] = v.lo;
          rhi[j][e] = v.hi;
        }
      }
    }
    {
      const Seen first = seen_by<MODE>(a, sq, 0), last = seen_by<MODE>(a, sq, a.T - 1);
      all_hi = first.hi;
      all_lo = last.lo;
    }

    for (int s = 0; s < nst; ++s) {
      const int xs = w0 + s * kStageKeys;
      if (xs >= win + kMetaKeys) {  // the next window's pages
        win += kMetaKeys;
        row_cur = row_next;
        ks_cur = ks_next;
        vs_cur = vs_next;
        lookup(win + kMetaKeys, row_next, ks_next, vs_next);
      }
      if constexpr (FP8) {
        if (xs == win) {
          // the window's largest V scale may raise the reference: what is
          // summed so far goes over to it
          float mx = fabsf(vs_cur);
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          const float ref = f8_ref(mx);
          if (mx > 0.f && ref > vsref) {
            const float f = vsref / ref;
            vsref = ref;
#pragma unroll
            for (int i = 0; i < MD; ++i)
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] *= f;
          }
        }
      }
      if (s + NS - 1 < nst) issue(s + NS - 1);
      cp_async_commit();
      cp_async_wait<NS - 1>();
      __syncwarp();
      const uint8_t *kt = ring + (s % NS) * 2 * kTile, *vt = kt + kTile;
      // ---- S^T = K Q^T
      float sacc[NT][4], sac2[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sacc[j][e] = sac2[j][e] = 0.f;
      if constexpr (FP8) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (kQRegs) {
            qk_fp8<D>(kt, gq, cq, qb[j], sacc[j], sac2[j]);
          } else {
            uint32_t f[MD][2];
#pragma unroll
            for (int kk = 0; kk < MD; ++kk) {
              const uint2 w = sm.qf[j][kk][lane];
              f[kk][0] = w.x;
              f[kk][1] = w.y;
            }
            qk_fp8<D>(kt, gq, cq, f, sacc[j], sac2[j]);
          }
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < MD; ++kk) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4(a0, a1, a2, a3, kt + swz<D>((lane & 7) + 8 * ((lane >> 3) & 1), 2 * kk + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint2 w;
            if constexpr (kQRegs) w = make_uint2(qb[j][kk][0], qb[j][kk][1]);
            else w = sm.qf[j][kk][lane];
            if (kk & 1) mma_bf16(sac2[j], a0, a1, a2, a3, w.x, w.y);
            else mma_bf16(sacc[j], a0, a1, a2, a3, w.x, w.y);
          }
        }
      }
      // ---- softmax; this lane's keys are gq and gq + 8 of the stage
      const int xk = xs + gq, k0 = rg.key(xk), k1 = rg.key(xk + 8);
      const int first = rg.key(xs);
      const bool whole = xs + kStageKeys <= w1 && rg.key(xs + kStageKeys - 1) == first + kStageKeys - 1 &&
                         first + kStageKeys <= all_hi && (first >= all_lo || first + kStageKeys <= rsink);
      float f0 = 1.f, f1 = 1.f, v0 = 1.f, v1 = 1.f;
      if constexpr (FP8) {
        const int at = (xk - win) >> 2;
        f0 = __shfl_sync(0xffffffffu, ks_cur, at);
        f1 = __shfl_sync(0xffffffffu, ks_cur, at + 2);
        const float inv = vsref > 0.f ? 1.f / vsref : 0.f;
        v0 = __shfl_sync(0xffffffffu, vs_cur, at) * inv;
        v1 = __shfl_sync(0xffffffffu, vs_cur, at + 2) * inv;
      }
      uint32_t pb[NT][2];
      float y[NT][4];
      bool grow = false;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          y[j][e] = (sacc[j][e] + sac2[j][e]) * csc[j][e];
          y[j][2 + e] = (sacc[j][2 + e] + sac2[j][2 + e]) * csc[j][e];
          if constexpr (FP8) {
            y[j][e] *= f0;
            y[j][2 + e] *= f1;
          }
          if (!whole) {
            const bool in0 = k0 < rhi[j][e] && (k0 >= rlo[j][e] || k0 < rsink) && xk < w1;
            const bool in1 = k1 < rhi[j][e] && (k1 >= rlo[j][e] || k1 < rsink) && xk + 8 < w1;
            if (!in0) y[j][e] = -INFINITY;
            if (!in1) y[j][2 + e] = -INFINITY;
          }
          grow |= fmaxf(y[j][e], y[j][2 + e]) > mcol[j][e] + dec_lazy<FP8>();
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
        // some column's scores outgrew its reference (its first keys do):
        // the columns' maxima over the lanes, and what is summed follows
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(y[j][e], y[j][2 + e]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float m_new = fmaxf(mcol[j][e], mx);
            alpha[e] = m_new == mcol[j][e] ? 1.f : mcol[j][e] == -INFINITY ? 0.f : attn::ex2(mcol[j][e] - m_new);
            mcol[j][e] = m_new;
            lcol[j][e] *= alpha[e];
          }
#pragma unroll
          for (int i = 0; i < MD; ++i) {
            o[i][j][0] *= alpha[0];
            o[i][j][1] *= alpha[1];
            o[i][j][2] *= alpha[0];
            o[i][j][3] *= alpha[1];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = mcol[j][e] == -INFINITY ? 0.f : mcol[j][e];
          p[e] = attn::ex2(y[j][e] - base);
          p[2 + e] = attn::ex2(y[j][2 + e] - base);
          lcol[j][e] += p[e] + p[2 + e];
        }
        if constexpr (FP8) {
          pb[j][0] = movmatrix_t(pack_f16(p[0] * v0, p[1] * v0));
          pb[j][1] = movmatrix_t(pack_f16(p[2] * v1, p[3] * v1));
        } else {
          pb[j][0] = movmatrix_t(pack_bf16(p[0], p[1]));
          pb[j][1] = movmatrix_t(pack_bf16(p[2], p[3]));
        }
      }
      // ---- O^T += V^T P^T
      if constexpr (FP8) {
        VRaw<D> vr;
        v_raw_fp8<D>(vt, gq, cq, vr);
#pragma unroll
        for (int i = 0; i < MD; ++i) {
          uint32_t a0, a1, a2, a3;
          v_frag_fp8<D>(vr, i, a0, a1, a2, a3);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_f16(o[i][j], a0, a1, a2, a3, pb[j][0], pb[j][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < MD; ++i) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4_t(a0, a1, a2, a3, vt + swz<D>((lane & 7) + 8 * (lane >> 4), 2 * i + ((lane >> 3) & 1)));
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_bf16(o[i][j], a0, a1, a2, a3, pb[j][0], pb[j][1]);
        }
      }
      __syncwarp();  // the slot may be refilled
    }
    cp_async_wait<0>();
  }
  __syncthreads();  // the rings become the four results

#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = lcol[j][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int m = 8 * j + 2 * cq + e;
      float *row = sm.o[warp][m];
      if constexpr (FP8) {
        store_col_fp8<D>(row, [&](int i, int k) { return o[i][j][k]; }, e, gq, vsref);
      } else {
#pragma unroll
        for (int i = 0; i < MD; ++i) {
          row[16 * i + gq] = o[i][j][e];
          row[16 * i + gq + 8] = o[i][j][2 + e];
        }
      }
      if (gq == 0) {
        sm.m[warp][m] = mcol[j][e];
        sm.l[warp][m] = l;
      }
    }
  __syncthreads();
  constexpr int kVec = D / 4;
  for (int e = threadIdx.x; e < M * kVec; e += kDecThreads) {
    const int m = e / kVec, d = e % kVec * 4;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) mx = fmaxf(mx, sm.m[w][m]);
    const float top = mx;
    if (mx == -INFINITY) mx = 0.f;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float f = attn::ex2(sm.m[w][m] - mx);
      const float4 v = *reinterpret_cast<const float4 *>(&sm.o[w][m][d]);
      l += f * sm.l[w][m];
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    if (a.cluster) {
      *reinterpret_cast<float4 *>(&sm.o[0][m][d]) = acc;  // (read by this thread alone)
      if (d == 0) {
        sm.cm[m] = top;
        sm.cl[m] = l;
      }
      continue;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;  // (a NaN sum stays one)
    acc.x *= inv;
    acc.y *= inv;
    acc.z *= inv;
    acc.w *= inv;
    const long long at = (long long)(sq.tok0 + m / a.G) * a.Hq + g * a.G + m % a.G;
    const float lse = l != 0.f ? (mx + __log2f(l)) * attn::kLn2 : -INFINITY;
    if (a.slots > 1) {
      const long long slot = at * a.slots + a.slot0 + split;
      if (l != 0.f) store4(a.o_part + slot * D + d, acc);
      if (d == 0) {
        a.lse_part[slot] = lse;
        if (MODE == kTail && split == 0 && !sq.shared)
          for (int k = 0; k < a.slot0; ++k) a.lse_part[at * a.slots + k] = -INFINITY;
      }
    } else {
      store4(static_cast<__nv_bfloat16 *>(a.o) + at * D + d, acc);
      if (d == 0) a.lse[at] = lse;
    }
  }
  if (a.cluster) {
    cluster_sync_all();  // every CTA's results stand
    for (int e = threadIdx.x + split * kDecThreads; e < M * kVec; e += kDecThreads * a.splits) {
      const int m = e / kVec, d = e % kVec * 4;
      float mx = -INFINITY;
      for (int c = 0; c < a.splits; ++c) mx = fmaxf(mx, peer_float(&sm.cm[m], c));
      if (mx == -INFINITY) mx = 0.f;
      float l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < a.splits; ++c) {
        const float f = attn::ex2(peer_float(&sm.cm[m], c) - mx);
        const float4 v = peer_float4(&sm.o[0][m][d], c);
        l += f * peer_float(&sm.cl[m], c);
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
      const float inv = l != 0.f ? 1.f / l : 0.f;  // (a NaN sum stays one)
      acc.x *= inv;
      acc.y *= inv;
      acc.z *= inv;
      acc.w *= inv;
      const long long at = (long long)(sq.tok0 + m / a.G) * a.Hq + g * a.G + m % a.G;
      store4(static_cast<__nv_bfloat16 *>(a.o) + at * D + d, acc);
      if (d == 0) a.lse[at] = l != 0.f ? (mx + __log2f(l)) * attn::kLn2 : -INFINITY;
    }
    cluster_sync_all();  // until every peer has read
  }
  pdl_end<MODE>();
}

}  // namespace attn
}  // namespace qsa

// Attention of many query rows over key ranges on the tensor cores (tcgen05,
// accumulators in tensor memory), BF16 and FP8 caches: the prefill form of the
// window attention and the shared prefixes of qsa_prefix_decode.
//
// Hundreds of query rows (tokens x heads of a group) read the same keys, so
// the two products, 4 D flops for every (row, key), bound it, and next to them
// one exponential per (row, key): a tile of 128 rows x 128 keys takes the
// tensor core 8 D cycles and the 16-a-cycle exponential unit 1,024, the same
// at D = 128.  Both have to run all the time:
//   - A CTA takes 256 rows as two tiles of 128.  While the exponentials of one
//     tile run, the tensor core works on the other.
//   - warps 0-3, 4-7   softmax of tile 0 / 1, a thread per row: scores from
//     tensor memory, running maximum and sum in registers, weights back to
//     tensor memory as bf16, where the value product reads them as its A
//     operand (they take the place of the scores)
//   - warp 8           one thread issues every product: values of a tile, then
//     the scores of its next keys
//   - warps 9-12       fill the ring of key and value tiles: rows are gathered
//     page by page with 16-byte cp.async (any page size), fp8 rows are
//     converted on the way
// The output accumulators stay in tensor memory.  They are rescaled only when
// a row's maximum has grown by more than 2^8 since the last time (weights up to
// 2^8 lose nothing in bf16 and float32), by the thread that owns the row: the
// scores of step j are issued behind the values of step j - 1, so that thread
// has them to itself between the two.
//
// Rounding: weights to bf16 (2^-9 relative), the error of the output's own
// rounding; fp8 keys are exact in bf16 and their scale multiplies the score in
// float32; fp8 values times their scale are rounded to bf16.
#pragma once
#include "attn_common.cuh"
#include "fp8_frag.cuh"
#include "prefill.cuh"

namespace qsa {
namespace attn {

constexpr int kTileRows = 128;  // rows of one tile (MMA M)
constexpr int kTileKeys = 128;
constexpr int kTileSlots = 4;   // ring: key and value tiles in turn
constexpr int kTileLoaders = 4;  // warps
constexpr int kTileThreads = (8 + 1 + kTileLoaders) * 32;
constexpr uint32_t kTmemCols = 512;  // S0, S1 at 0 and 128, O0, O1 at 256 and 384
constexpr float kLazy = 8.f;    // growth of a row's maximum (log2) that is left in the weights
constexpr unsigned long long kTileWaitNs = 2000000000ull;

template <int D>
struct TileSmem {
  static constexpr int kTile = kTileKeys * D * 2;  // bytes of a key, value or query tile
  uint8_t q[2][kTile];
  uint8_t ring[kTileSlots][kTile];
  float kscale[4][kTileKeys];  // fp8: key scale * sm_scale * log2(e), by key tile
  alignas(8) uint64_t full[kTileSlots], empty[kTileSlots];
  uint64_t qfull, sfull[2], pfull[2], ofull[2];
  uint32_t tmem;
  int dead;  // a wait ran out: every role leaves
};

__device__ __forceinline__ void mbar_init(uint64_t *b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase, at most kTileWaitNs; false when it ran out here or in
// another role.
__device__ __forceinline__ bool mbar_wait_or(uint64_t *b, uint32_t parity, int *dead) {
  if (mbar_try(b, parity)) return true;
  const unsigned long long t0 = pre::globaltimer();
  while (!mbar_try(b, parity)) {
    if (*reinterpret_cast<volatile int *>(dead)) return false;
    if (pre::globaltimer() - t0 > kTileWaitNs) {
      *reinterpret_cast<volatile int *>(dead) = 1;
      record_error(kErrTimeout);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
      :
      : "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
      :
      : "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

#define QSA_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), \
                     "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define QSA_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), \
                     "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : QSA_R8(v, 0), QSA_R8(v, 8), QSA_R8(v, 16), QSA_R8(v, 24)
      : "r"(at));
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::QSA_W8(v, 0),
      QSA_W8(v, 8), QSA_W8(v, 16), QSA_W8(v, 24), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::QSA_W8(v, 0),
      QSA_W8(v, 8), "r"(at)
      : "memory");
}
#undef QSA_R8
#undef QSA_W8
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// kind::f16 with bf16 operands and a float32 accumulator, M = 128; B read
// K-major (keys) or MN-major (values).
__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTileRows >> 4) << 24);
}
// A tile is D / 64 column blocks of 128 rows x 128 bytes, 128-byte swizzled.
constexpr uint32_t kColBlock = kTileKeys * 128;
__device__ __forceinline__ int tile_off(int row, int ch) {
  return (ch >> 3) * (int)kColBlock + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint64_t desc_k(uint32_t at) { return pre::smem_desc<128>(at); }
// Values as the B operand [keys x D], D contiguous: blocks of 64 dims at the
// leading offset, groups of 8 keys (1,024 bytes) at the stride offset.
__device__ __forceinline__ uint64_t desc_v(uint32_t at) {
  return (uint64_t)((at & 0x3FFFFu) >> 4) | (uint64_t)(kColBlock >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Two f16 pairs (from E4M3) times a scale to bf16 pairs.
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h2, float s) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// Grid (row tiles of 256, Hkv * splits, sequences).
template <int MODE, int D, bool FP8>
__global__ void __launch_bounds__(kTileThreads, 1) tile_kernel(Args a) {
  pdl_open();
  using SM = TileSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  SM &sm = *reinterpret_cast<SM *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Seq sq = sequence<MODE>(a, blockIdx.z);
  // the last tiles of a causal chunk see the most keys: they go first
  const int m0 = (int)(gridDim.x - 1 - blockIdx.x) * 2 * kTileRows;
  const int rows = min(2 * kTileRows, sq.ntok * a.G - m0);
  if (rows <= 0) return;
  const int g = blockIdx.y / a.splits, split = blockIdx.y - g * a.splits;
  const int i0 = m0 / a.G, i1 = (m0 + rows - 1) / a.G + 1;
  const Range rg = range_of<MODE>(a, sq, i0, i1);
  const int x0 = split_bound(rg.n, a.splits, split, kTileKeys);
  const int x1 = split_bound(rg.n, a.splits, split + 1, kTileKeys);
  const int nt = (x1 - x0 + kTileKeys - 1) / kTileKeys;
  const int tiles = rows > kTileRows ? 2 : 1;

  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < kTileSlots; ++i) {
      mbar_init(&sm.full[i], kTileLoaders);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.qfull, kTileLoaders);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.sfull[t], 1);
      mbar_init(&sm.pfull[t], 4);
      mbar_init(&sm.ofull[t], 1);
    }
    sm.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pre::tc_fence_before();
  __syncthreads();
  pre::tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax --
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int m = m0 + t * kTileRows + row;
    const bool live = t * kTileRows + row < rows;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * kTileKeys, o_at = tmem + lanes + 256 + t * 128;
    // what the row sees, in virtual keys: x < va or vb <= x < vc
    int va = 0, vb = 0, vc = 0;
    if (live) {
      const Seen v = seen_by<MODE>(a, sq, m / a.G);
      if (rg.sa > 0) va = min(min(v.sink, v.hi), rg.sa);
      else if (rg.b0 == 0) va = min(v.sink, v.hi);
      vb = rg.sa + max(v.lo - rg.b0, 0);
      vc = min(rg.sa + v.hi - rg.b0, rg.n);
    }
    float mx = -INFINITY, l = 0.f;  // maximum (scaled, log2) the weights are relative to, and their sum
    bool ok = true;
    if (t < tiles) {
      for (int j = 0; j < nt; ++j) {
        const int xt = x0 + j * kTileKeys;
        ok = mbar_wait_or(&sm.sfull[t], j & 1, &sm.dead);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        pre::tc_fence_after();
        const bool whole = !live || (xt >= vb && xt + kTileKeys <= vc) || xt + kTileKeys <= va;
        const bool masked = !__all_sync(0xffffffffu, whole);
        const float *ksc = FP8 ? sm.kscale[j & 3] : nullptr;
        auto bits = [&](int c) -> uint32_t {  // keys xt + c .. + 31 that the row sees
          const int x = xt + c;
          auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
          return below(va - x) | (below(vc - x) & ~below(vb - x));
        };
        // ---- the row's maximum
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kTileKeys; c += 32) {
          uint32_t s[32];
          tmem_ld32(s_at + c, s);
          pre::tmem_ld_wait();
          const uint32_t see = masked ? bits(c) : 0xffffffffu;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float y = __uint_as_float(s[e]);
            if (FP8) y *= ksc[c + e];
            if (masked && !((see >> e) & 1u)) y = -INFINITY;
            top = fmaxf(top, y);
          }
        }
        if (!FP8) top *= a.scale_log2;
        const bool grow = top > mx + kLazy || (mx == -INFINITY && top > -INFINITY);
        const float m_new = grow ? top : mx;
        if (__any_sync(0xffffffffu, grow)) {
          const float al = grow ? (mx == -INFINITY ? 0.f : ex2(mx - m_new)) : 1.f;
          l *= al;
          if (j > 0) {
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t v[32];
              tmem_ld32(o_at + c, v);
              pre::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
              tmem_st32(o_at + c, v);
            }
          }
        }
        mx = m_new;
        const float base = mx == -INFINITY ? 0.f : mx;
        // ---- weights, as bf16 in the place of the scores
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int c = 0; c < kTileKeys; c += 32) {
          uint32_t s[32], p[16];
          tmem_ld32(s_at + c, s);
          pre::tmem_ld_wait();
          const uint32_t see = masked ? bits(c) : 0xffffffffu;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0 = ex2(fmaf(__uint_as_float(s[e]), FP8 ? ksc[c + e] : a.scale_log2, -base));
            float p1 = ex2(fmaf(__uint_as_float(s[e + 1]), FP8 ? ksc[c + e + 1] : a.scale_log2, -base));
            if (masked) {
              if (!((see >> e) & 1u)) p0 = 0.f;
              if (!((see >> (e + 1)) & 1u)) p1 = 0.f;
            }
            l0 += p0;
            l1 += p1;
            const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
            p[e / 2] = *reinterpret_cast<const uint32_t *>(&b);
          }
          tmem_st16(s_at + c / 2, p);
        }
        l += l0 + l1;
        tmem_st_wait();
        pre::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pfull[t]);
      }
      // ---- output
      if (ok && nt > 0) ok = mbar_wait_or(&sm.ofull[t], 0, &sm.dead);
      ok = __all_sync(0xffffffffu, ok);
      pre::tc_fence_after();
      const bool some = l != 0.f;  // (a NaN sum stays one)
      const float inv = some ? 1.f / l : 0.f;
      const float lse = some ? ((mx == -INFINITY ? 0.f : mx) + __log2f(l)) * kLn2 : -INFINITY;
      const long long at = (long long)(sq.tok0 + m / a.G) * a.Hq + g * a.G + m % a.G;
      const long long slot = at * a.slots + a.slot0 + split;
      if (ok) {
        if (live) (a.slots > 1 ? a.lse_part[slot] : a.lse[at]) = lse;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          if (nt > 0) {
            tmem_ld32(o_at + c, v);
            pre::tmem_ld_wait();
          }
          if (!live) continue;
          if (a.slots > 1) {
            if (!some) continue;
            float *dst = a.o_part + slot * D + c;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              store4(dst + e, make_float4(__uint_as_float(v[e]) * inv, __uint_as_float(v[e + 1]) * inv,
                                          __uint_as_float(v[e + 2]) * inv, __uint_as_float(v[e + 3]) * inv));
          } else {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.o) + at * D + c;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(some ? __uint_as_float(v[e + 2 * k]) * inv : 0.f,
                                                               some ? __uint_as_float(v[e + 2 * k + 1]) * inv : 0.f);
                w[k] = *reinterpret_cast<const uint32_t *>(&b);
              }
              *reinterpret_cast<uint4 *>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ products --
    if (lane == 0 && nt > 0) {
      const uint32_t idesc_s = idesc_bf16(kTileKeys, false), idesc_o = idesc_bf16(D, true);
      auto scores = [&](int t, int slot) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)(k / 4) * kColBlock + (uint32_t)(k % 4) * 32;
          mma_ss(tmem + t * kTileKeys, desc_k(smem_u32(sm.q[t]) + off), desc_k(smem_u32(sm.ring[slot]) + off),
                 idesc_s, k > 0);
        }
      };
      bool ok = mbar_wait_or(&sm.qfull, 0, &sm.dead) && mbar_wait_or(&sm.full[0], 0, &sm.dead);
      if (ok) {
        pre::tc_fence_after();
        for (int t = 0; t < tiles; ++t) {
          scores(t, 0);
          pre::umma_commit(&sm.sfull[t]);
        }
        pre::umma_commit(&sm.empty[0]);
      }
      for (int j = 0; ok && j < nt; ++j) {
        const int nv = 2 * j + 1, nk = 2 * j + 2;  // this step's values, the next one's keys
        const bool more = j + 1 < nt;
        ok = mbar_wait_or(&sm.full[nv % kTileSlots], (nv / kTileSlots) & 1, &sm.dead);
        if (ok && more) ok = mbar_wait_or(&sm.full[nk % kTileSlots], (nk / kTileSlots) & 1, &sm.dead);
        for (int t = 0; ok && t < tiles; ++t) {
          ok = mbar_wait_or(&sm.pfull[t], j & 1, &sm.dead);
          if (!ok) break;
          pre::tc_fence_after();
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k)
            mma_ts(tmem + 256 + t * 128, tmem + t * kTileKeys + 8 * k,
                   desc_v(smem_u32(sm.ring[nv % kTileSlots]) + k * 2048), idesc_o, j > 0 || k > 0);
          if (more) {
            scores(t, nk % kTileSlots);
            pre::umma_commit(&sm.sfull[t]);
          } else {
            pre::umma_commit(&sm.ofull[t]);
          }
        }
        if (!ok) break;
        pre::umma_commit(&sm.empty[nv % kTileSlots]);
        if (more) pre::umma_commit(&sm.empty[nk % kTileSlots]);
      }
    }
    __syncwarp();
  } else if (nt > 0) {
    // -------------------------------------------------------------- loaders --
    const int wl = warp - 9;
    constexpr int kRowBytes = D * (FP8 ? 1 : 2);
    constexpr int kChunks = kRowBytes / 16;
    constexpr int kRowsPer = 32 / kChunks;          // rows of one load of the warp
    constexpr int kRowsWarp = kTileKeys / kTileLoaders;  // 32 rows of a tile
    constexpr int kLoads = kRowsWarp / kRowsPer;
    const int Hkv = a.c.num_kv_heads;
    const long long row_stride = (long long)Hkv * kRowBytes;
    const uint8_t *base[2] = {static_cast<const uint8_t *>(a.c.k_cache) + (long long)g * kRowBytes,
                              static_cast<const uint8_t *>(a.c.v_cache) + (long long)g * kRowBytes};
    // queries: bf16 rows, 2 D bytes
    {
      constexpr int kQ = D / 8;  // 16-byte chunks
      const __nv_bfloat16 *qg = static_cast<const __nv_bfloat16 *>(a.q);
      for (int e = wl * 32 + lane; e < tiles * kTileRows * kQ; e += kTileLoaders * 32) {
        const int rr = e / kQ, ch = e % kQ, m = m0 + rr;
        const bool ok = rr < rows;
        const __nv_bfloat16 *src =
            ok ? qg + ((long long)(sq.tok0 + m / a.G) * a.Hq + g * a.G + m % a.G) * D + ch * 8 : qg;
        cp_async16_zfill(sm.q[rr / kTileRows] + tile_off(rr % kTileRows, ch), src, ok);
      }
      cp_async_commit();
    }
    // keys that some row of the CTA sees; the others are zero
    Seen any = seen_by<MODE>(a, sq, i1 - 1);
    if (MODE == kWindow) any.lo = max(0, sq.first + i0 + 1 - a.window);
    if (MODE == kShared) any.hi = sq.prefix;
    // lane i < 8: token row of this warp's keys 4 i .. 4 i + 3 of a tile
    auto lookup = [&](int j, long long &row, float &ks, float &vs) {
      row = -1;
      ks = vs = 0.f;
      const int x = x0 + j * kTileKeys + wl * kRowsWarp + 4 * lane;
      if (lane < kRowsWarp / 4 && x < x1) {
        const int key = rg.key(x);
        const int lp = key / a.c.page_size;
        const int pg = physical_page(a.c, sq.table, lp);
        if (pg >= 0) {
          row = (long long)pg * a.c.page_size + (key - lp * a.c.page_size);
          if (FP8) {
            ks = a.c.k_scale[(long long)pg * Hkv + g];
            vs = a.c.v_scale[(long long)pg * Hkv + g];
          }
        }
      }
    };
    // source of load i of tile j (nullptr: zeros)
    auto source = [&](int j, int i, int kv, long long row, int &r) -> const uint8_t * {
      r = i * kRowsPer + lane / kChunks;  // within the warp's 32 rows
      const int ch = lane % kChunks;
      const long long r0 = __shfl_sync(0xffffffffu, row, r >> 2);
      const int x = x0 + j * kTileKeys + wl * kRowsWarp + r;
      const bool ok = x < x1 && r0 >= 0 && sees(any, rg.key(x));
      return ok ? base[kv] + (r0 + (r & 3)) * row_stride + ch * 16 : nullptr;
    };
    long long row_cur, row_next;
    float ks_cur, vs_cur, ks_next, vs_next;
    lookup(0, row_cur, ks_cur, vs_cur);
    lookup(1, row_next, ks_next, vs_next);
    bool ok = true;
    if constexpr (!FP8) {
      // tile n of the ring: keys (n even) or values (n odd) of step n / 2
      auto publish = [&](uint64_t *bar) {
        pre::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      for (int n = 0; n < 2 * nt; ++n) {
        const int j = n >> 1, slot = n % kTileSlots;
        if (n >= 2 && (n & 1) == 0) {
          row_cur = row_next;
          lookup(j + 1, row_next, ks_next, vs_next);
        }
        if (n >= kTileSlots) {
          ok = mbar_wait_or(&sm.empty[slot], ((n / kTileSlots) - 1) & 1, &sm.dead);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          int r;
          const uint8_t *src = source(j, i, n & 1, row_cur, r);
          cp_async16_zfill(sm.ring[slot] + tile_off(wl * kRowsWarp + r, lane % kChunks), src ? src : base[0],
                           src != nullptr);
        }
        cp_async_commit();
        // two tiles stay in flight
        cp_async_wait<2>();
        if (n == 1) publish(&sm.qfull);
        if (n >= 2) publish(&sm.full[(n - 2) % kTileSlots]);
      }
      cp_async_wait<0>();
      for (int n = max(0, 2 * nt - 2); n < 2 * nt; ++n) publish(&sm.full[n % kTileSlots]);
    } else {
      // fp8: raw rows of the next tile are loaded while this one is converted
      uint4 raw[2][kLoads];
      auto fetch = [&](int n, uint4(&v)[kLoads], long long row) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          int r;
          const uint8_t *src = source(n >> 1, i, n & 1, row, r);
          v[i] = src ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0, 0, 0, 0);
        }
      };
      fetch(0, raw[0], row_cur);
      cp_async_wait<0>();
      pre::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.qfull);
      for (int j = 0; j < nt && ok; ++j) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int n = 2 * j + kv, slot = n % kTileSlots;
          const float vs_now = vs_cur, ks_now = ks_cur;
          if (kv == 0) {
            fetch(n + 1, raw[1], row_cur);
          } else {
            row_cur = row_next;
            ks_cur = ks_next;
            vs_cur = vs_next;
            lookup(j + 2, row_next, ks_next, vs_next);
            if (j + 1 < nt) fetch(n + 1, raw[0], row_cur);
          }
          if (n >= kTileSlots) {
            ok = mbar_wait_or(&sm.empty[slot], ((n / kTileSlots) - 1) & 1, &sm.dead);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int r = i * kRowsPer + lane / kChunks, ch = lane % kChunks;
            const float s = kv ? __shfl_sync(0xffffffffu, vs_now, r >> 2) : 1.f;
            const uint4 x = raw[kv][i];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t b[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              b[2 * k] = scaled_bf16x2(dec::e4m3x2_f16x2(w[k]), s);
              b[2 * k + 1] = scaled_bf16x2(dec::e4m3x2_f16x2_hi(w[k]), s);
            }
            uint8_t *tile = sm.ring[slot];
            *reinterpret_cast<uint4 *>(tile + tile_off(wl * kRowsWarp + r, 2 * ch)) = make_uint4(b[0], b[1], b[2], b[3]);
            *reinterpret_cast<uint4 *>(tile + tile_off(wl * kRowsWarp + r, 2 * ch + 1)) = make_uint4(b[4], b[5], b[6], b[7]);
          }
          if (kv == 0) {
            const float s = __shfl_sync(0xffffffffu, ks_now, lane >> 2);
            sm.kscale[j & 3][wl * kRowsWarp + lane] = s * a.scale_log2;
          }
          pre::fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[slot]);
        }
      }
    }
  }
  pre::tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    pre::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace attn
}  // namespace qsa

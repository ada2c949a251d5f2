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
//     tensor memory in 16 bits, where the value product reads them as its A
//     operand (they take the place of the scores)
//   - warps 8-11       fill the ring of key and value tiles, 32 rows each.  bf16
//     rows of whole boxes come by TMA (pages of a multiple of 8 tokens);
//     cp.async gathers the rest and zeroes rows that nothing sees.  (cp.async
//     for everything: its 16-byte writes wait for the tensor core's operand
//     reads, ~110 cycles an instruction, 3,500 a step, and the loaders bound the
//     kernel.)  fp8 rows are converted to f16 on the way.
//   - warp 12          one thread issues every product: values of a tile, then
//     the scores of its next keys (warps 13-15 only complete the warpgroup that
//     gives its registers to the softmax)
// A step's weights are relative to the maximum of the steps BEFORE it: they
// need not wait for their own (which runs beside them), and float32 and bf16
// lose nothing by weights above 1.  When a row's maximum has grown by more than
// 2^8 (f16 weights: 2^4) the next step starts with rescaling its sum and its
// output accumulators, which stay in tensor memory; the scores of step j are
// issued behind the values of step j - 1, so the thread that owns the row has them
// to itself then.  Only growth beyond the weights' range (2^60; f16 weights: 2^4)
// makes 32 keys start again with their own maximum.
//
// Rounding: weights to bf16, the error of the output's own rounding; where 32 keys
// start again, the weights of the step's keys before them follow by a power of two.
// fp8 caches run in f16, which holds every E4M3 code: queries scaled per row by a
// power of two (fp8_frag.cuh says what that keeps), the key scale on the score in
// float32, and the value scale, relative to a power of two that follows the
// largest one seen, on the weight before it is rounded to f16 (2^-11, and what
// f8_ref says about small ones).
//
// Measured (B200): 8,192 tokens of 32 heads over a window of 8,192 in 1.10 ms, call
// after call (1.0 PFLOP/s, 58 % of the measured cuBLAS burst rate and 69 % of its
// sustained one: the power limit holds here too; a first call in 0.97); 4 x 1,024
// tokens of 16 heads over 4,096 in 163 us (855 TFLOP/s, on 1.73 waves of CTAs); from
// an fp8 cache 1.6 and 1.4 times as long (631 and 516 TFLOP/s).  A step of 256 rows
// x 128 keys takes about 3,500 cycles, 2,048 of them products: scores, weights,
// values and next scores follow one another, and with two tiles the tensor core
// waits for softmax.
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
constexpr int kTileThreads = 16 * 32;
constexpr int kLoadWarp = 8, kMmaWarp = 12;
constexpr uint32_t kTmemCols = 512;  // S0, S1 at 0 and 128, O0, O1 at 256 and 384
// growth (log2) of a row's maximum that is left in the weights of later steps, and of
// a step's scores that its own weights hold
template <bool FP8>
__host__ __device__ constexpr float tile_lazy() { return FP8 ? kF8Grow : 8.f; }
template <bool FP8>
__host__ __device__ constexpr float tile_range() { return FP8 ? kF8Grow : 60.f; }
constexpr unsigned long long kTileWaitNs = 2000000000ull;

template <int D>
struct TileSmem {
  static constexpr int kTile = kTileKeys * D * 2;  // bytes of a key, value or query tile
  uint8_t q[2][kTile];
  uint8_t ring[kTileSlots][kTile];
  // fp8: scales of a tile's keys and values by groups of four, the largest |value scale| of each
  // loader's share, and 2^-e of each query row (the row is scaled by 2^e)
  alignas(16) float kscale[4][kTileKeys / 4], vscale[4][kTileKeys / 4], vmax[4][kTileLoaders], qscale[2 * kTileRows];
  alignas(8) uint64_t full[kTileSlots], empty[kTileSlots];
  uint64_t qfull, sfull[2], pfull[2], ofull[2], drain;
  uint32_t tmem;
  int dead;  // a wait ran out: every role leaves
  int announced[kTileLoaders];  // tiles that a loader warp has arrived for
};

template <int D>
__device__ __forceinline__ TileSmem<D> &tile_smem() {
  extern __shared__ uint8_t smem_raw[];
  return *reinterpret_cast<TileSmem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ void mbar_init(uint64_t *b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
// A box of `kBoxCols` dims of one head, some rows, by TMA (128-byte swizzled).
constexpr int kBoxCols = 64;
__device__ __forceinline__ void tma_box(void *dst, const CUtensorMap *map, int col, int head, int row, uint64_t *b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(col), "r"(head), "r"(row), "r"(smem_u32(b))
      : "memory");
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
// Waits for the phase, for about kTileWaitNs at most; false when that ran out
// here or in another role.  (The clock is looked at every 256 tries only: a read
// of the global timer behind the first try put 500 cycles into every hand-over.)
__device__ __forceinline__ bool mbar_wait_or(uint64_t *b, uint32_t parity, int *dead) {
  unsigned long long t0 = 0;
  for (unsigned n = 1; !mbar_try(b, parity); ++n) {
    if (n & 255u) continue;
    if (*reinterpret_cast<volatile int *>(dead)) return false;
    const unsigned long long t = pre::globaltimer();
    if (t0 == 0) t0 = t;
    if (t - t0 > kTileWaitNs) {
      *reinterpret_cast<volatile int *>(dead) = 1;
      record_error(kErrTimeout);
      return false;
    }
  }
  return true;
}

// Products D (+)= A B: A in shared memory (a descriptor) or in tensor memory.
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
      :
      : "r"(d), "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
      :
      : "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// One lane of the warp.  (elect.sync rather than a lane test: the products'
// operands then stay in uniform registers.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
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

// kind::f16 with bf16 or f16 operands and a float32 accumulator, M = 128; B
// read K-major (keys) or MN-major (values).
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, int n, bool b_mn) {
  return (1u << 4) | (bf16 ? 1u << 7 | 1u << 10 : 0u) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
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

// Two float32 in a register pair.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &x, float &y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  if constexpr (BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&b);
  } else {
    return dec::pack_f16(x, y);
  }
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// What a softmax thread keeps of its row: the maximum (scaled, log2) that sum
// and outputs are relative to, the sum, the largest score so far, and (fp8) the
// power of two that the value scales are relative to (f8_ref).
struct RowState {
  float mx, l, seen, vref;
};

// The row's sum and output accumulators over to reference `to` (and vref `ref`).
template <int D, bool FP8>
__device__ __forceinline__ void rebase(RowState &r, float to, float ref, bool first, uint32_t o_at) {
  float al = to > r.mx ? (r.mx == -INFINITY ? 0.f : ex2(r.mx - to)) : 1.f;
  r.l *= al;
  r.mx = fmaxf(r.mx, to);
  if (FP8) {
    al *= ref > r.vref ? r.vref / ref : 1.f;
    r.vref = fmaxf(r.vref, ref);
  }
  if (first) return;
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t v[16];
    pre::tmem_ld16(o_at + c, v);
    pre::tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
    tmem_st16(o_at + c, v);
  }
}

// A row's weights of one step: the scores in tensor memory become weights and
// the row's state follows.  see(c): the keys c .. c + 31 of the tile that the row
// sees, as bits (MASKED).
template <int D, bool FP8, bool MASKED, typename See>
__device__ __forceinline__ void weights(uint32_t s_at, uint32_t o_at, bool first, float scale, const float *ksc,
                                        const float *vsc, const float *vmax, RowState &r, See see) {
  // ---- what the steps before left to do
  float ref = r.vref;
  if (FP8) {
    const float4 w = *reinterpret_cast<const float4 *>(vmax);
    const float v = fmaxf(max3(w.x, w.y, w.z), w.w);
    if (v > 0.f) ref = fmaxf(ref, f8_ref(v));
  }
  const float late = r.seen > r.mx + tile_lazy<FP8>() ? r.seen : r.mx;
  if (__any_sync(0xffffffffu, late > r.mx || ref > r.vref)) rebase<D, FP8>(r, late, ref, first, o_at);

  const f2 sc2 = pack2(scale, scale);
  const float vinv = FP8 && r.vref > 0.f ? 1.f / r.vref : 0.f;
  constexpr float kRange = tile_range<FP8>();
  // the scores of keys c .. c + 31, -inf where the row does not see them
  auto scores = [&](int c, uint32_t(&s)[32]) {
    if (FP8) {
#pragma unroll
      for (int e = 0; e < 32; e += 16) {
        const float4 k = *reinterpret_cast<const float4 *>(ksc + (c + e) / 4);
        const float ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float a, b;
          unpack2(mul2(pack2(__uint_as_float(s[e + i]), __uint_as_float(s[e + i + 1])), pack2(ks[i / 4], ks[i / 4])),
                  a, b);
          s[e + i] = __float_as_uint(a);
          s[e + i + 1] = __float_as_uint(b);
        }
      }
    }
    if (MASKED) {
      const uint32_t bits = see(c);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!((bits >> e) & 1u)) s[e] = 0xff800000u;
    }
  };
  auto largest = [&](const uint32_t(&s)[32]) -> float {
    float t0 = __uint_as_float(s[0]), t1 = __uint_as_float(s[16]);
#pragma unroll
    for (int e = 1; e < 15; e += 2) {
      t0 = max3(t0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
      t1 = max3(t1, __uint_as_float(s[16 + e]), __uint_as_float(s[17 + e]));
    }
    return fmaxf(max3(t0, t1, __uint_as_float(s[15])), __uint_as_float(s[31]));
  };

  float sum;
  uint32_t p[16];
  auto exps = [&](int c, const uint32_t(&s)[32]) {
    const float base = r.mx == -INFINITY ? 0.f : r.mx;
    const f2 nb2 = pack2(-base, -base);
    f2 sum0 = 0, sum1 = 0;  // (0.f, 0.f)
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float x0, x1, x2, x3;
      const f2 y0 = fma2(pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, nb2);
      const f2 y1 = fma2(pack2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), sc2, nb2);
      unpack2(y0, x0, x1);
      x0 = ex2(x0);
      x1 = ex2(x1);
      unpack2(y1, x2, x3);
      x2 = ex2(x2);
      x3 = ex2(x3);
      sum0 = add2(sum0, pack2(x0, x1));
      sum1 = add2(sum1, pack2(x2, x3));
      if (FP8) {
        const float v = vsc[(c + e) / 4] * vinv;
        unpack2(mul2(pack2(x0, x1), pack2(v, v)), x0, x1);
        unpack2(mul2(pack2(x2, x3), pack2(v, v)), x2, x3);
      }
      p[e / 2] = pack16<!FP8>(x0, x1);
      p[e / 2 + 1] = pack16<!FP8>(x2, x3);
    }
    float a, b;
    unpack2(add2(sum0, sum1), a, b);
    sum = a + b;
  };
  uint32_t s[2][32];
  tmem_ld32(s_at, s[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    pre::tmem_ld_wait();
    if (q < 3) tmem_ld32(s_at + 32 * (q + 1), s[(q + 1) & 1]);
    scores(32 * q, s[q & 1]);
    const float top = largest(s[q & 1]) * scale;
    exps(32 * q, s[q & 1]);
    if (__any_sync(0xffffffffu, top > r.mx + kRange)) {
      // out of range (the first keys of every row): once more, relative to
      // these keys' maximum; the weights in place follow
      pre::tmem_ld_wait();
      tmem_st_wait();
      // (rows that are out of range alone, the others' by a factor of one; a power
      // of two where there are weights to follow, so that none is rounded again)
      float to = r.mx, al = 1.f;
      if (top > r.mx + kRange) {
        const float k = floorf(top - r.mx);  // inf: the row's first keys
        to = k < INFINITY ? r.mx + k : top;
        al = k < 126.f ? __int_as_float((127 - (int)k) << 23) : 0.f;
      }
      rebase<D, FP8>(r, to, r.vref, first, o_at);
#pragma unroll 1
      for (int k = 0; k < q; ++k) {
        uint32_t w[16];
        pre::tmem_ld16(s_at + 16 * k, w);
        pre::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float lo, hi;
          if (FP8) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
            lo = f.x, hi = f.y;
          } else {
            lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xffff0000u);
          }
          w[e] = pack16<!FP8>(lo * al, hi * al);
        }
        tmem_st16(s_at + 16 * k, w);
      }
      exps(32 * q, s[q & 1]);
    }
    r.seen = fmaxf(r.seen, top);
    r.l += sum;
    tmem_st16(s_at + 16 * q, p);
  }
  tmem_st_wait();
}

// Ends a CTA of TMA loads, by one warp: if a wait ran out, boxes still in flight
// land first.  The tiles that the farthest loader warp announced get the arrivals of
// the others and are waited for, boundedly; that warp had waited for the slot of the
// tile four ahead, so every warp has announced the tiles before these.  (Out of
// line, and finding the shared memory again: the kernel has no register for it.)
template <int D>
__noinline__ __device__ void land_boxes() {
  TileSmem<D> &sm = tile_smem<D>();
  if ((threadIdx.x & 31) != 0 || !*reinterpret_cast<volatile int *>(&sm.dead)) return;
  int most = 0;
  for (int w = 0; w < kTileLoaders; ++w) most = max(most, sm.announced[w]);
  for (int n = max(0, most - kTileSlots); n < most; ++n) {
    uint64_t *full = &sm.full[n % kTileSlots];
    for (int w = 0; w < kTileLoaders; ++w)
      if (sm.announced[w] <= n) mbar_arrive(full);
    pre::mbar_wait(full, (n / kTileSlots) & 1);
  }
}
// Products in flight, and the arrivals that nobody waits for (the last tiles'
// slots, or all of them when a wait ran out), end before the CTA and its tensor
// memory do.
__noinline__ __device__ void end_products(uint64_t *drain) {
  pre::umma_commit(drain);
  pre::mbar_wait(drain, 0);
}

// The caches as TMA sees them, [token rows][Hkv][D] in boxes of `rows` tokens
// (0: no TMA) that lie within a page.
struct TileMaps {
  CUtensorMap k, v;
  int rows;
};

// Grid (row tiles of 256, Hkv * splits, sequences).
template <int MODE, int D, bool FP8>
__global__ void __launch_bounds__(kTileThreads, 1) tile_kernel(const Args a, const __grid_constant__ TileMaps maps) {
  pdl_begin<MODE>();
  using SM = TileSmem<D>;
  SM &sm = tile_smem<D>();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Seq sq = sequence<MODE>(a, blockIdx.z);
  // the last tiles of a causal chunk see the most keys: they go first
  const int m0 = (int)(gridDim.x - 1 - blockIdx.x) * 2 * kTileRows;
  const int rows = min(2 * kTileRows, sq.ntok * a.G - m0);
  if (rows <= 0) return;
  const int g = blockIdx.y / a.splits, split = blockIdx.y - g * a.splits;
  const int i0 = m0 / a.G, i1 = (m0 + rows - 1) / a.G + 1;
  const Range rg = range_of<MODE>(a, sq, i0, i1, max(maps.rows, 4));
  const int x0 = split_bound(rg.n, a.splits, split, kTileKeys);
  const int x1 = split_bound(rg.n, a.splits, split + 1, kTileKeys);
  const int nt = (x1 - x0 + kTileKeys - 1) / kTileKeys;
  const int tiles = rows > kTileRows ? 2 : 1;

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    // each of the four loader warps arrives once for a tile (its boxes by TMA with
    // the bytes they bring, its own copies when they stand)
    for (int i = 0; i < kTileSlots; ++i) {
      mbar_init(&sm.full[i], kTileLoaders);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.qfull, kLoadWarp);
    mbar_init(&sm.drain, 1);
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

  // registers: 512 threads start with 128 each; the shares add up to that
  constexpr int kRegsSoftmax = FP8 ? 152 : 168, kRegsLoad = FP8 ? 112 : 80, kRegsMma = 96;
  static_assert(2 * kRegsSoftmax + kRegsLoad + kRegsMma <= 4 * 128, "register shares");
  if (warp < kLoadWarp) {
    // ------------------------------------------------------------ softmax --
    regs_up<kRegsSoftmax>();
    // queries: 16 bytes a thread and load, kStep rows a round of the 256 threads
    {
      constexpr int kQ = D / 8, kStep = kLoadWarp * 32 / kQ, kBatch = 8;
      const __nv_bfloat16 *qg = static_cast<const __nv_bfloat16 *>(a.q);
      const int ch = tid % kQ;
      int rr = tid / kQ, tok = (m0 + rr) / a.G, head = (m0 + rr) - tok * a.G;
      const int dtok = kStep / a.G, dhead = kStep - dtok * a.G;
      for (int done = 0; done < tiles * kTileRows; done += kBatch * kStep) {
        uint4 x[kBatch];  // (fp8: a batch of loads in flight, then converted)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const bool ok = rr < rows;
          const __nv_bfloat16 *src = ok ? qg + ((long long)(sq.tok0 + tok) * a.Hq + g * a.G + head) * D + ch * 8 : qg;
          if constexpr (!FP8)
            cp_async16_zfill(sm.q[rr / kTileRows] + tile_off(rr % kTileRows, ch), src, ok);
          else
            x[i] = ok ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
          rr += kStep;
          tok += dtok;
          head += dhead;
          if (head >= a.G) {
            head -= a.G;
            ++tok;
          }
        }
        if constexpr (FP8) {
          // f16, scaled so that 2^14 <= max |q| 2^e < 2^15; kQ lanes hold a row
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int row = done + i * kStep + tid / kQ;
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t mxq = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) mxq = max(mxq, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
#pragma unroll
            for (int off = kQ / 2; off >= 1; off >>= 1) mxq = max(mxq, __shfl_xor_sync(0xffffffffu, mxq, off));
            const int ex = mxq == 0u ? 0 : min(141 - (int)(mxq >> 7), 126);
            const float f = dec::pow2f(ex);
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = dec::pack_f16(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
            *reinterpret_cast<uint4 *>(sm.q[row / kTileRows] + tile_off(row % kTileRows, ch)) =
                make_uint4(h[0], h[1], h[2], h[3]);
            if (ch == 0) sm.qscale[row] = dec::pow2f(-ex);
          }
        }
      }
      if (!FP8) {
        cp_async_commit();
        cp_async_wait<0>();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.qfull);
    }
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
    RowState r = {-INFINITY, 0.f, -INFINITY, 0.f};
    bool ok = true;
    if (t < tiles) {
      float scale = a.scale_log2;
      if (FP8) {
        ok = __all_sync(0xffffffffu, mbar_wait_or(&sm.qfull, 0, &sm.dead));
        scale *= sm.qscale[t * kTileRows + row];
      }
      for (int j = 0; ok && j < nt; ++j) {
        const int xt = x0 + j * kTileKeys;
        ok = mbar_wait_or(&sm.sfull[t], j & 1, &sm.dead);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        pre::tc_fence_after();
        const bool whole = !live || (xt >= vb && xt + kTileKeys <= vc) || xt + kTileKeys <= va;
        const bool masked = !__all_sync(0xffffffffu, whole);
        auto see = [&](int c) -> uint32_t {  // keys xt + c .. + 31 that the row sees
          const int x = xt + c;
          auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
          return below(va - x) | (below(vc - x) & ~below(vb - x));
        };
        if (masked)
          weights<D, FP8, true>(s_at, o_at, j == 0, scale, sm.kscale[j & 3], sm.vscale[j & 3], sm.vmax[j & 3], r, see);
        else
          weights<D, FP8, false>(s_at, o_at, j == 0, scale, sm.kscale[j & 3], sm.vscale[j & 3], sm.vmax[j & 3], r, see);
        pre::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pfull[t]);
      }
      // ---- output
      if (ok && nt > 0) ok = mbar_wait_or(&sm.ofull[t], 0, &sm.dead);
      ok = __all_sync(0xffffffffu, ok);
      pre::tc_fence_after();
      const bool some = r.l != 0.f;  // (a NaN sum stays one)
      const float inv = some ? (FP8 ? r.vref / r.l : 1.f / r.l) : 0.f;
      const float lse = some ? ((r.mx == -INFINITY ? 0.f : r.mx) + __log2f(r.l)) * kLn2 : -INFINITY;
      const long long at = (long long)(sq.tok0 + m / a.G) * a.Hq + g * a.G + m % a.G;
      const long long slot = at * a.slots + a.slot0 + split;
      if (ok) {
        if (live) (a.slots > 1 ? a.lse_part[slot] : a.lse[at]) = lse;
        if (a.slots == 1) {
          // bf16 rows: every thread writes its own
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            if (nt > 0) {
              tmem_ld32(o_at + c, v);
              pre::tmem_ld_wait();
            }
            if (!live) continue;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.o) + at * D + c;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack16<true>(some ? __uint_as_float(v[e + 2 * k]) * inv : 0.f,
                                    some ? __uint_as_float(v[e + 2 * k + 1]) * inv : 0.f);
              *reinterpret_cast<uint4 *>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        } else {
          // float32 parts, rows far apart: by halves of D, a thread puts its half
          // into the warp's quarter of the tile's queries, which nothing reads any
          // more (swizzled by 16 bytes), and the warp writes run after run (a
          // thread writing its own row took 11,000 cycles)
          const unsigned rows_out = __ballot_sync(0xffffffffu, live && some);
          constexpr int kHalf = D / 2, kLanes = kHalf / 4;  // floats, and lanes that write them
          float *stage = reinterpret_cast<float *>(sm.q[t]) + (warp & 3) * 32 * kHalf;
          const int l4 = lane % kLanes;
#pragma unroll 1
          for (int c0 = 0; nt > 0 && c0 < D; c0 += kHalf) {
            __syncwarp();  // the half before is read
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 32) {
              uint32_t v[32];
              tmem_ld32(o_at + c0 + c, v);
              pre::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                store4(stage + lane * kHalf + (((c + e) / 4) ^ (lane & 7)) * 4,
                       make_float4(__uint_as_float(v[e]) * inv, __uint_as_float(v[e + 1]) * inv,
                                   __uint_as_float(v[e + 2]) * inv, __uint_as_float(v[e + 3]) * inv));
            }
            __syncwarp();
#pragma unroll 4
            for (int i = 0; i < kLanes; ++i) {
              const int rr = i * (32 / kLanes) + lane / kLanes;
              const long long dst = __shfl_sync(0xffffffffu, slot, rr) * D + c0 + 4 * l4;
              const float4 v = *reinterpret_cast<const float4 *>(stage + rr * kHalf + ((l4 ^ (rr & 7)) * 4));
              if ((rows_out >> rr) & 1u) store4(a.o_part + dst, v);
            }
          }
        }
      } else if (live) {  // a wait ran out: no result passes for one
        (a.slots > 1 ? a.lse_part[slot] : a.lse[at]) = NAN;
      }
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------ products --
    regs_down<kRegsMma>();
    // (one elected thread runs the whole role: its operands stay in uniform
    // registers, and a wait that is over costs it few cycles)
    if (warp == kMmaWarp && nt > 0 && elect_one()) {
      constexpr uint32_t idesc_s = idesc_16(!FP8, kTileKeys, false), idesc_o = idesc_16(!FP8, D, true);
      const uint64_t q_desc = desc_k(smem_u32(sm.q)), k_desc = desc_k(smem_u32(sm.ring)),
                     v_desc = desc_v(smem_u32(sm.ring));
      constexpr uint32_t kTile16 = SM::kTile / 16;  // descriptors count 16 bytes
      auto scores = [&](int t, int slot) {
        const uint64_t qd = q_desc + t * kTile16, kd = k_desc + slot * kTile16;
        mma_ss<false>(tmem + t * kTileKeys, qd, kd, idesc_s);
#pragma unroll
        for (int k = 1; k < D / 16; ++k) {
          const uint32_t off = ((uint32_t)(k / 4) * kColBlock + (uint32_t)(k % 4) * 32) / 16;
          mma_ss<true>(tmem + t * kTileKeys, qd + off, kd + off, idesc_s);
        }
        pre::umma_commit(&sm.sfull[t]);
      };
      auto filled = [&](int n) { return mbar_wait_or(&sm.full[n % kTileSlots], (n / kTileSlots) & 1, &sm.dead); };
      bool ok = mbar_wait_or(&sm.qfull, 0, &sm.dead) && filled(0);
      if (ok) {
        // what the loaders wrote goes over to the tensor core's view here, where
        // it is waited for: in the loaders the fence would wait for the copies
        // still in flight
        pre::fence_async_smem();
        scores(0, 0);
        if (tiles > 1) scores(1, 0);
        pre::umma_commit(&sm.empty[0]);
        ok = filled(1) && (nt == 1 || filled(2));
        pre::fence_async_smem();
      }
      for (int j = 0; ok && j < nt; ++j) {
        const int nv = 2 * j + 1, nk = 2 * j + 2;  // this step's values, the next one's keys
        const bool more = j + 1 < nt;
        const uint64_t vd = v_desc + (nv % kTileSlots) * kTile16;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= tiles) break;
          ok = mbar_wait_or(&sm.pfull[t], j & 1, &sm.dead);
          if (!ok) break;
          pre::tc_fence_after();
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k)
            mma_ts(tmem + 256 + t * 128, tmem + t * kTileKeys + 8 * k, vd + k * (2048 / 16), idesc_o,
                   k > 0 ? 1u : (uint32_t)(j > 0));
          if (more) scores(t, nk % kTileSlots);
          else pre::umma_commit(&sm.ofull[t]);
        }
        if (!ok) break;
        pre::umma_commit(&sm.empty[nv % kTileSlots]);
        if (more) {
          pre::umma_commit(&sm.empty[nk % kTileSlots]);
          // the next step's tiles, while this one's products run
          ok = filled(nv + 2) && (j + 2 == nt || filled(nk + 2));
          pre::fence_async_smem();
        }
      }
      end_products(&sm.drain);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- loaders --
    regs_down<kRegsLoad>();
    const int wl = warp - kLoadWarp;
    constexpr int kRowBytes = D * (FP8 ? 1 : 2);
    constexpr int kChunks = kRowBytes / 16;
    constexpr int kRowsPer = 32 / kChunks;          // rows of one load of the warp
    constexpr int kRowsWarp = kTileKeys / kTileLoaders;  // 32 rows of a tile
    constexpr int kLoads = kRowsWarp / kRowsPer;
    const int Hkv = a.c.num_kv_heads;
    const long long row_stride = (long long)Hkv * kRowBytes;
    const uint8_t *base[2] = {static_cast<const uint8_t *>(a.c.k_cache) + (long long)g * kRowBytes,
                              static_cast<const uint8_t *>(a.c.v_cache) + (long long)g * kRowBytes};
    // keys that some row of the CTA sees; the others are zero
    Seen any = seen_by<MODE>(a, sq, i1 - 1);
    if (MODE == kWindow) any.lo = window_lo(sq.first + i0, a.window);
    if (MODE == kShared) any.hi = sq.prefix;
    // lane i < 8: the block-table entry of this warp's keys 4 i .. 4 i + 3 of a
    // tile, loaded a step ahead of its use (-1: none is needed)
    const long long table = (long long)sq.table * a.c.max_pages_per_req;
    auto lookup = [&](int j, int &pg, int &in_page) {
      pg = -1;
      in_page = 0;
      const int x = x0 + j * kTileKeys + wl * kRowsWarp + 4 * lane;
      if (lane < kRowsWarp / 4 && x < x1) {
        const int key = rg.key(x);  // below max_pages_per_req * page_size (range_of)
        const int lp = key / a.c.page_size;
        in_page = key - lp * a.c.page_size;
        pg = a.c.block_table[table + lp];
        if (pg < 0) pg = -2;
      }
    };
    // A tile's rows as the lanes load them: load i covers rows kRowsPer i .. of
    // the warp's 32, lane / kChunks picking the row and lane % kChunks its 16
    // bytes.  Four rows share an offset, found once for the keys and the values.
    constexpr int kOffs = kRowsPer == 2 ? kLoads / 2 : kLoads;
    const int lr = lane / kChunks, ch = lane % kChunks;
    const long long in_group = (lr & 3) * row_stride + ch * 16, two_rows = 2 * row_stride;
    long long off[kOffs];
    bool whole = false;  // every row of the warp's share is loaded
    int xw = 0;          // virtual key of its first row
    float ks = 0.f, vs = 0.f;  // fp8: scales of the keys' page
    int tok_row = -1;          // lane i < 8: cache row of keys 4 i .. 4 i + 3
    auto place = [&](int j, int pg, int in_page) {
      long long row = -1;
      ks = vs = 0.f;
      if (pg != -1) {
        if (pg < 0 || pg >= a.c.num_pages) {
          record_error(kErrBounds);
        } else {
          row = ((long long)pg * a.c.page_size + in_page) * row_stride;
          tok_row = pg * a.c.page_size + in_page;  // (TMA: below 2^31)
          if (FP8) {
            ks = a.c.k_scale[(long long)pg * Hkv + g];
            vs = a.c.v_scale[(long long)pg * Hkv + g];
          }
        }
      }
      xw = x0 + j * kTileKeys + wl * kRowsWarp;
      const int k0 = rg.key(xw), k1 = rg.key(xw + kRowsWarp - 1);
      whole = __all_sync(0xffffffffu, lane >= kRowsWarp / 4 || row >= 0) && xw + kRowsWarp <= x1 &&
              k1 - k0 == kRowsWarp - 1 && k1 < any.hi && (k0 >= any.lo || k1 < any.sink);
      if (!FP8 && whole && maps.rows) return;  // TMA
#pragma unroll
      for (int k = 0; k < kOffs; ++k) {
        const int at = kRowsPer == 2 ? k : kRowsPer == 4 ? k : 2 * k + (lr >> 2);
        off[k] = __shfl_sync(0xffffffffu, row, at) + in_group;
      }
      if (!whole) {
        // the rows that nothing sees, or without a page, are marked
#pragma unroll
        for (int k = 0; k < kOffs; ++k) {
          const int at = kRowsPer == 2 ? k : kRowsPer == 4 ? k : 2 * k + (lr >> 2);
          if (__shfl_sync(0xffffffffu, row, at) < 0) off[k] = -1;
        }
      }
    };
    auto source = [&](int i, int kv, bool &ok) -> const uint8_t * {
      const long long o = kRowsPer == 2 ? off[i / 2] + (i & 1) * two_rows : off[i];
      ok = true;
      if (!whole) {
        const int x = xw + i * kRowsPer + lr;
        ok = x < x1 && (kRowsPer == 2 ? off[i / 2] : off[i]) >= 0 && sees(any, rg.key(x));
      }
      return ok ? base[kv] + o : base[kv];
    };
    int pg_next, in_next;
    lookup(0, pg_next, in_next);
    place(0, pg_next, in_next);
    lookup(1, pg_next, in_next);
    bool ok = true;
    if constexpr (!FP8) {
      // tile n of the ring: keys (n even) or values (n odd) of step n / 2
      int behind = -1;  // slot whose copies by this warp are not announced yet
      int n = 0;
      for (; n < 2 * nt; ++n) {
        const int j = n >> 1, slot = n % kTileSlots;
        if (n >= 2 && (n & 1) == 0) {
          place(j, pg_next, in_next);
          lookup(j + 1, pg_next, in_next);
        }
        if (n >= kTileSlots) {
          ok = mbar_wait_or(&sm.empty[slot], ((n / kTileSlots) - 1) & 1, &sm.dead);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        if (whole && maps.rows) {
          if (lane == 0) mbar_arrive_expect(&sm.full[slot], kRowsWarp * D * 2);
          __syncwarp();
          const int per = maps.rows >> 2;  // groups of four rows in a box
          if (lane < kRowsWarp / 4 && (lane & (per - 1)) == 0) {
#pragma unroll
            for (int c = 0; c < D / kBoxCols; ++c)
              tma_box(sm.ring[slot] + c * kColBlock + (wl * kRowsWarp + 4 * lane) * 128, n & 1 ? &maps.v : &maps.k,
                      c * kBoxCols, g, tok_row, &sm.full[slot]);
          }
          if (behind >= 0) {
            cp_async_wait<0>();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.full[behind]);
            behind = -1;
          }
        } else {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            bool ld;
            const uint8_t *src = source(i, n & 1, ld);
            cp_async16_zfill(sm.ring[slot] + tile_off(wl * kRowsWarp + i * kRowsPer + lr, ch), src, ld);
          }
          cp_async_commit();
          if (behind >= 0) {
            cp_async_wait<1>();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.full[behind]);
          }
          behind = slot;
        }
      }
      cp_async_wait<0>();
      __syncwarp();
      if (lane == 0 && behind >= 0) mbar_arrive(&sm.full[behind]);
      if (lane == 0) sm.announced[wl] = n;
    } else {
      // fp8: raw rows of the next tile are loaded while this one is converted
      uint4 raw[2][kLoads];
      auto fetch = [&](int kv, uint4(&v)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          bool ld;
          const uint8_t *src = source(i, kv, ld);
          v[i] = ld ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0, 0, 0, 0);
        }
      };
      if (nt > 0) fetch(0, raw[0]);
      // the 32 bytes of a load are two chunks; half of the lanes write the second
      // one first, so that the rows' halves, a column block apart, miss each
      // other's banks
      const int odd = ch >= kChunks / 2 ? 1 : 0;
      for (int j = 0; j < nt && ok; ++j) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int n = 2 * j + kv, slot = n % kTileSlots;
          const float vs_now = vs, ks_now = ks;
          if (kv == 0) {
            fetch(1, raw[1]);
          } else {
            place(j + 1, pg_next, in_next);
            lookup(j + 2, pg_next, in_next);
            if (j + 1 < nt) fetch(0, raw[0]);
          }
          if (n >= kTileSlots) {
            ok = mbar_wait_or(&sm.empty[slot], ((n / kTileSlots) - 1) & 1, &sm.dead);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          uint8_t *tile = sm.ring[slot];
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int r = wl * kRowsWarp + i * kRowsPer + lr;
            const uint4 x = raw[kv][i];
            const uint4 lo = make_uint4(dec::e4m3x2_f16x2(x.x), dec::e4m3x2_f16x2_hi(x.x), dec::e4m3x2_f16x2(x.y),
                                        dec::e4m3x2_f16x2_hi(x.y));
            const uint4 hi = make_uint4(dec::e4m3x2_f16x2(x.z), dec::e4m3x2_f16x2_hi(x.z), dec::e4m3x2_f16x2(x.w),
                                        dec::e4m3x2_f16x2_hi(x.w));
            *reinterpret_cast<uint4 *>(tile + tile_off(r, 2 * ch + odd)) = odd ? hi : lo;
            *reinterpret_cast<uint4 *>(tile + tile_off(r, 2 * ch + (odd ^ 1))) = odd ? lo : hi;
          }
          if (kv == 0) {  // (the softmax reads both behind the scores of this step)
            if (lane < kRowsWarp / 4) {
              sm.kscale[j & 3][wl * kRowsWarp / 4 + lane] = ks_now;
              sm.vscale[j & 3][wl * kRowsWarp / 4 + lane] = vs_now;
            }
            float v = fabsf(vs_now);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
            if (lane == 0) sm.vmax[j & 3][wl] = v;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[slot]);
        }
      }
    }
  }
  pre::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    if (!FP8) land_boxes<D>();
    __syncwarp();
    pre::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace attn
}  // namespace qsa

// What the attention calls over whole key ranges share (qsa_window_decode,
// qsa_window_prefill, qsa_prefix_decode): which keys a query sees, how query
// rows and keys are numbered, and the merge of partial results.
//
// A call attends SEQUENCES of consecutive query tokens, all of whose keys are
// read through one block-table row:
//   kWindow, cu == NULL   request s: its T newest tokens (decode)
//   kWindow, cu != NULL   request s: tokens cu[s] .. cu[s+1]-1, its newest (chunk)
//   kShared               group s of requests cu[s] .. cu[s+1]-1, T tokens
//                         each, over the first prefix_lens[s] keys that all of
//                         them share (read through the first request's row)
//   kTail                 request s: its T newest tokens over the keys behind
//                         its group's prefix
// A query at position p sees the keys i of
//   kWindow   i <= p and (i > p - window or i < sinks)
//   kShared   i <= p and i < prefix
//   kTail     i <= p and i >= prefix
// so always i < hi and (i >= lo or i < sink) with per-token hi, lo.
//
// The query heads of one kv head are rows of one small matrix: row
// m = token * G + head-in-group of a sequence (G = Hq / Hkv), cut into tiles.
// The keys a tile needs are one or two ranges, [0, sa) and [b0, b1); they are
// walked as one VIRTUAL range [0, sa + b1 - b0).  sa and b0 are multiples of
// `unit`, a power of two that divides the page size (4 at least), so `unit`
// virtual keys from a multiple of it on always lie in one page.
#pragma once
#include "qsa_common.cuh"

namespace qsa {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxT = 4;      // query tokens per request of the decode calls
constexpr int kMaxGroup = 32;  // query heads per kv head (times T in the decode calls)

enum Mode { kWindow = 0, kShared = 1, kTail = 2 };

struct Args {
  CacheDev c;
  const void *q;  // [n_tok, Hq, D]
  void *o;        // [n_tok, Hq, D] of the query type
  float *lse;     // [n_tok, Hq]
  int B, T, Hq, G, n_tok;
  const int32_t *cu;  // sequence offsets (see above) or NULL
  int n_cu;           // sequences that cu describes
  int max_tokens;     // kShared, chunks: host bound of a sequence's tokens (sizes the launch)
  const int32_t *ctx_lens;
  const int32_t *prefix_lens;
  int window, sinks;
  float scale_log2;  // sm_scale * log2(e)
  // partial results: slot k of row (token, head) at (token * Hq + head) * slots + k
  float *o_part;    // [n_tok, Hq, slots, D], normalised
  float *lse_part;  // [n_tok, Hq, slots]
  int slots;        // 1: the kernel writes o / lse itself
  int slot0;        // first slot of this launch
  int splits;       // slots of this launch
  int cluster;      // the splits of a row are the CTAs of a cluster, which merge among themselves
};

// One sequence of query tokens.
struct Seq {
  int tok0, ntok;  // its query tokens are rows tok0 .. tok0 + ntok - 1 of q
  int table;       // its block-table row
  int first;       // kWindow / kTail: position of its first query token
  int prefix;      // kShared / kTail: keys of the shared prefix
  bool shared;     // kTail: the prefixes' kernel writes the request's first slots
};

// A load of what was written before the call; the tails' go to L2 (pdl_begin).
template <int MODE, typename T>
__device__ __forceinline__ T ld_mode(const T *p) {
  if constexpr (MODE == kTail) return __ldcg(p);
  else return *p;
}

// Cached tokens of request r; a negative length counts as none.
template <int MODE>
__device__ __forceinline__ int ctx_len(const Args &a, int r) {
  return max(ld_mode<MODE>(a.ctx_lens + r), 0);
}

// First key in the window of the query at position p.  Positions before 0 (a
// request with fewer cached tokens than query tokens) count as -1, whose window
// ends before key 0: nothing is subtracted from them, so window = INT32_MAX stays
// within 32 bits.
__device__ __forceinline__ int window_lo(int p, int window) { return max(0, max(p + 1, 0) - window); }

// Query tokens t0 .. t1 - 1 as a request of a chunk that the attention kernels take.
__device__ __forceinline__ bool chunk_ok(const Args &a, int t0, int t1) {
  return t0 >= 0 && t1 >= t0 && t1 <= a.n_tok && t1 - t0 <= a.max_tokens;
}

// Requests r0 .. r1 - 1 and a prefix as a group that the prefixes' kernel takes.
// Its tails ask the same, so that a refused group's slots get their empty lse.
__device__ __forceinline__ bool group_ok(const Args &a, int r0, int r1, int prefix) {
  return r0 >= 0 && r1 >= r0 && r1 <= a.B && prefix >= 0 && (r1 - r0) * a.T <= a.max_tokens;
}

// Sequence s; a malformed description (offsets that fall or leave the query
// rows) is recorded and gives an empty sequence.
template <int MODE>
__device__ __forceinline__ Seq sequence(const Args &a, int s) {
  Seq q;
  q.table = s;
  q.prefix = 0;
  q.first = 0;
  q.shared = false;
  if (MODE == kShared) {
    const int r0 = a.cu[s], r1 = a.cu[s + 1];
    q.prefix = a.prefix_lens[s];
    if (!group_ok(a, r0, r1, q.prefix)) {
      record_error(kErrBadInput);
      q.tok0 = q.ntok = 0;
      return q;
    }
    q.tok0 = r0 * a.T;
    q.ntok = (r1 - r0) * a.T;
    q.table = r0;
    return q;
  }
  if (MODE == kWindow && a.cu) {
    const int t0 = a.cu[s], t1 = a.cu[s + 1];
    if (!chunk_ok(a, t0, t1)) {
      record_error(kErrBadInput);
      q.tok0 = q.ntok = 0;
      return q;
    }
    q.tok0 = t0;
    q.ntok = t1 - t0;
    q.first = ctx_len<MODE>(a, s) - q.ntok;
    return q;
  }
  q.tok0 = s * a.T;
  q.ntok = a.T;
  q.first = ctx_len<MODE>(a, s) - a.T;
  if (MODE == kTail) {
    // the group that holds request s: the last one that starts at or before it,
    // by a whole warp, 32 offsets a round (each round waits for L2)
    const int lane = threadIdx.x & 31;
    int lo = 0, n = a.n_cu;
    while (n > 32) {
      const int step = (n + 31) / 32, at = lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, at < n && ld_mode<MODE>(a.cu + lo + min(at, n)) <= s);
      const int k = m ? 31 - __clz(m) : 0;
      lo += k * step;
      n = min(step, n - k * step);
    }
    const int mine = lo + min(lane, n - 1);
    const int c0 = ld_mode<MODE>(a.cu + mine), c1 = ld_mode<MODE>(a.cu + mine + 1);
    const int pre = ld_mode<MODE>(a.prefix_lens + mine);
    const unsigned m = __ballot_sync(0xffffffffu, lane < n && c0 <= s);
    const int k = m ? 31 - __clz(m) : 0;
    const int r0 = __shfl_sync(0xffffffffu, c0, k), r1 = __shfl_sync(0xffffffffu, c1, k);
    const int prefix = __shfl_sync(0xffffffffu, pre, k);
    // a request outside every group shares nothing, one of a refused group loses
    // its prefix
    if (r0 <= s && s < r1) {
      q.prefix = max(prefix, 0);
      q.shared = group_ok(a, r0, r1, prefix);
    }
  }
  return q;
}

// Keys the query token `i` (of the sequence) sees: key < hi and (key >= lo
// or key < sink).
struct Seen {
  int hi, lo, sink;
};
template <int MODE>
__device__ __forceinline__ Seen seen_by(const Args &a, const Seq &q, int i) {
  Seen v;
  v.sink = 0;
  v.lo = 0;
  if (MODE == kShared) {
    const int tok = q.tok0 + i, r = tok / a.T;
    v.hi = min(q.prefix, ctx_len<MODE>(a, r) - a.T + (tok - r * a.T) + 1);
    return v;
  }
  v.hi = q.first + i + 1;
  if (MODE == kTail) {
    v.lo = q.prefix;
  } else {
    v.lo = window_lo(q.first + i, a.window);
    v.sink = a.sinks;
  }
  return v;
}
__device__ __forceinline__ bool sees(const Seen &v, int key) {
  return key < v.hi && (key >= v.lo || key < v.sink);
}

// Programmatic launch of the three kernels of qsa_prefix_decode.  The tails'
// kernel reads nothing that the prefixes' kernel writes, so it starts while that
// one still runs, filling the SMs that run out of prefix work: the prefixes'
// kernel lets it go only behind its own wait (what came before on the stream is
// then complete for both), and the tails' kernel waits for it at its end, so that
// the merge, which waits for the tails, waits for both.
//
// That earlier work is also VISIBLE to the tails, none of whose threads has waited
// yet when they read queries, lengths, tables, scales and caches.  The wait makes
// it visible to the prefixes' kernel, which runs on every SM, so it has reached L2,
// where all SMs meet; one thread of each of its CTAs then has a gpu-scope fence
// ahead of its launch_dependents, and the tails start only when all of them have
// issued that (or ended).  What an SM's L1 may still hold of an earlier call is not
// asked: the tails' loads go to L2 (ld_mode, cp.async.cg).  That costs a short
// tail's CTA the latency of its look-ups: 32 requests behind 28,672 keys took 41.3
// us against 39.5 through L1 (a fence at the start of the tails, which drops the
// SM's L1, 41.6), 128 behind 250,000 nothing.
template <int MODE>
__device__ __forceinline__ void pdl_begin() {
  if (MODE == kShared) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) {
      __threadfence();
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
  } else if (MODE == kWindow) {
    pdl_open();
  }
}
template <int MODE>
__device__ __forceinline__ void pdl_end() {
  if (MODE == kTail) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
}

// The keys that some token of [i0, i1) of the sequence may see, as a virtual
// range: virtual key x is key x below sa, else b0 + x - sa.
struct Range {
  int sa, b0, n;
  __device__ __forceinline__ int key(int x) const { return x < sa ? x : b0 + (x - sa); }
};
template <int MODE>
__device__ __forceinline__ Range range_of(const Args &a, const Seq &q, int i0, int i1, int unit = 4) {
  Range r;
  r.sa = r.b0 = r.n = 0;
  if (i1 <= i0) return r;
  int lo, hi, sink = 0;
  if (MODE == kShared) {
    lo = 0;
    hi = q.prefix;  // a query before the prefix's end masks what it does not see
  } else {
    hi = q.first + i1;
    lo = MODE == kTail ? q.prefix : window_lo(q.first + i0, a.window);
    sink = MODE == kTail ? 0 : a.sinks;
  }
  if (hi <= 0) return r;
  // a length that the block table cannot hold is cut to what it can
  const long long cap = min((long long)a.c.max_pages_per_req * a.c.page_size, 0x7fffff00LL);
  if (hi > cap) {
    record_error(kErrBounds);
    hi = (int)cap;
  }
  sink = (min(sink, hi) + unit - 1) & -unit;
  lo &= -unit;
  if (lo >= hi) lo = hi;
  if (sink >= lo) {  // one range
    r.sa = 0;
    r.b0 = sink > 0 ? 0 : lo;
    r.n = hi - r.b0;
    return r;
  }
  r.sa = sink;
  r.b0 = lo;
  r.n = sink + hi - lo;
  return r;
}

// Split k of n virtual keys in `splits`: bounds at multiples of `unit`, the
// splits alike to one unit.
__device__ __forceinline__ int split_bound(int n, int splits, int k, int unit) {
  const int units = (int)(((unsigned)n + unit - 1) / unit), each = units / splits;
  return min(n, (each * k + min(k, units - each * splits)) * unit);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Weights of an 8-bit cache.  They enter the value product in f16, times their
// page's V scale over a reference: a power of two of 2^-kF8Bias of the largest V
// scale's binade (float32 keeps it from 2^-126 on).  f16 has 11 bits from 2^-14 to
// 2^16, so the bias puts the row's largest weight near the top: a weight may pass
// its row's reference by 2^kF8Grow and the scale its binade by 2, in all 2^15.  A
// weight keeps 2^-11 of itself down to 2^-24 of the row's largest (weight times
// scale), 2^-8 down to 2^-27, and what is below is off by 2^-35 of that at most.
// (Without the bias a flat row behind one key whose logit is 17 above it and whose
// value is zero came out 7 % off, and zero from 18 on.)
constexpr int kF8Bias = 10;
constexpr float kF8Grow = 4.f;
__device__ __forceinline__ float f8_ref(float vs_max) {
  const int E = (__float_as_int(vs_max) >> 23) & 0xff;
  return __int_as_float(max(E - kF8Bias, 1) << 23);
}

__device__ __forceinline__ void store4(float *p, const float4 &v) {
  *reinterpret_cast<float4 *>(p) = v;
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 w;
  w.x = *reinterpret_cast<uint32_t *>(&a);
  w.y = *reinterpret_cast<uint32_t *>(&b);
  *reinterpret_cast<uint2 *>(p) = w;
}

// Merge of the partial results of every (token, head) row:
//   lse = log sum_k exp(lse_k),  o = sum_k exp(lse_k - lse) o_k,
// o = 0 and lse = -inf for a row that saw nothing.  W warps share a row, each
// taking every W-th slot (lane i its i-th): one for up to 16 slots, four, whose
// sums meet in shared memory, for up to 128.  A warp's weights are made lane by
// lane and its rows loaded eight at a time: latency bounds this (one slot after
// the other took 39 us for 65 slots of 512 rows).  Slots are added in a fixed
// order, so a result does not depend on how the work was scheduled.
constexpr int kMergeThreads = 128;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMergeFew = 16;
constexpr int kMaxSlots = 32 * kMergeWarps;

// Whether a request of the chunk that the attention kernels took holds token
// `tok`, by a whole warp, a request a lane: only then were the row's slots
// written.  (Every request is asked, so that any offsets give what the kernels
// did; a chunk has several slots a row only with fewer requests than CTAs of a
// wave or two, so one or a few rounds.)
__device__ __forceinline__ bool in_chunk(const Args &a, int tok, int lane) {
  bool mine = false;
  for (int s = lane; s < a.n_cu; s += 32) {
    const int t0 = a.cu[s], t1 = a.cu[s + 1];
    mine |= t0 <= tok && tok < t1 && chunk_ok(a, t0, t1);
  }
  return __any_sync(0xffffffffu, mine);
}

template <int D, typename OutT, int W>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(Args a) {
  pdl_open();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = W == 1 ? (long long)blockIdx.x * kMergeWarps + warp : (long long)blockIdx.x;
  if (row >= (long long)a.n_tok * a.Hq) return;
  // rows of no request, or of a refused one, stay as they were
  if (a.cu && a.prefix_lens == nullptr && !in_chunk(a, (int)(row / a.Hq), lane)) return;
  const int S = a.slots, w0 = W == 1 ? 0 : warp;
  const int mine = lane * W + w0;  // this lane's slot
  const float l = mine < S ? __ldcg(a.lse_part + row * S + mine) : -INFINITY;
  float mx = l;
  bool nan = l != l;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  nan = __any_sync(0xffffffffu, nan);
  __shared__ float red_mx[kMergeWarps], red_z[kMergeWarps], red_o[W == 1 ? 1 : kMergeWarps][D];
  if (W > 1) {
    if (lane == 0) red_mx[warp] = nan ? NAN : mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) {
      mx = fmaxf(mx, red_mx[i]);
      nan |= red_mx[i] != red_mx[i];
    }
  }
  if (nan) mx = NAN;  // a NaN in any part is one in the result
  const float wt = (l == -INFINITY && !nan) ? 0.f : __expf(l - mx);
  float z = mine < S ? wt : 0.f;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int d = 4 * lane, n = (S - w0 + W - 1) / W;  // slots of this warp
  const float4 *src = reinterpret_cast<const float4 *>(a.o_part + (row * S + w0) * D + d);
  for (int k0 = 0; k0 < n; k0 += 8) {
    float4 v[8];
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = __shfl_sync(0xffffffffu, wt, (k0 + k) & 31);
      // (an empty slot's row was not written)
      v[k] = (k0 + k < n && f[k] != 0.f && d < D) ? __ldcg(src + (long long)(k0 + k) * W * (D / 4))
                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k0 + k >= n || f[k] == 0.f) continue;
      acc.x = __fmaf_rn(f[k], v[k].x, acc.x);
      acc.y = __fmaf_rn(f[k], v[k].y, acc.y);
      acc.z = __fmaf_rn(f[k], v[k].z, acc.z);
      acc.w = __fmaf_rn(f[k], v[k].w, acc.w);
    }
  }
  if (W > 1) {
    if (d < D) *reinterpret_cast<float4 *>(&red_o[warp][d]) = acc;
    if (lane == 0) red_z[warp] = z;
    __syncthreads();
    if (warp > 0) return;
    z = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      z += red_z[i];
      if (d < D) {
        const float4 v = *reinterpret_cast<const float4 *>(&red_o[i][d]);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
    }
  }
  const float inv = z != 0.f ? 1.f / z : 0.f;
  acc.x *= inv;
  acc.y *= inv;
  acc.z *= inv;
  acc.w *= inv;
  if (d < D) store4(static_cast<OutT *>(a.o) + row * D + d, acc);
  if (lane == 0) a.lse[row] = z != 0.f ? mx + __logf(z) : -INFINITY;
}

}  // namespace attn
}  // namespace qsa

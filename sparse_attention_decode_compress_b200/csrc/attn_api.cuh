// Entry points over whole key ranges of the paged caches: qsa_rope_append,
// qsa_window_decode, qsa_window_prefill, qsa_prefix_decode (declared in
// include/qsa.h).  Part of qsa_api.cu, whose launch and validation helpers it
// uses.
#pragma once
#include <cudaTypedefs.h>

#include "attn_common.cuh"
#include "attn_decode.cuh"
#include "attn_simple.cuh"
#include "attn_tile.cuh"
#include "rope_append.cuh"

namespace {

// Splits and workspace sizes are planned for this many SMs (B200), so that
// they depend on the call's shape alone.
constexpr int kPlanSMs = 148;
constexpr int kMaxCluster = 8;  // portable cluster size

// ------------------------------------------------------------------ plan --
// How one launch covers the keys of its rows: `splits` slots each.
struct AttnPlan {
  int splits;       // of this launch
  long long tiles;  // row tiles of a sequence
  bool cluster;     // the splits merge within the launch: no slots
  int slots() const { return cluster ? 1 : splits; }
};

long long ceil_ll(long long a, long long b) { return (a + b - 1) / b; }

// Bound on the keys a tile of `tokens` tokens sees.
long long span_bound(long long window, long long sinks, long long tokens, long long cap) {
  return std::min(cap, std::min(window, cap) + std::min(sinks, cap) + tokens);
}

AttnPlan plan_simple(long long seqs, int Hkv, long long rows, long long span) {
  AttnPlan p = {};
  p.tiles = ceil_ll(std::max(rows, 1LL), qsa::attn::kSimpleRows);
  const long long ctas = std::max(1LL, seqs * Hkv * p.tiles);
  p.splits = (int)std::max(1LL, std::min({4LL * kPlanSMs / ctas, ceil_ll(span, 2 * qsa::attn::kSimpleKeys), 64LL}));
  return p;
}

// Few rows of a 16-bit or 8-bit cache: one CTA of the streaming kernel per
// (request, kv head, split).  `merge`: the splits are all there is to a row.
AttnPlan plan_stream(long long seqs, int Hkv, long long span, bool merge) {
  AttnPlan p = {};
  p.tiles = 1;
  const long long pairs = std::max(1LL, seqs * Hkv);
  if (merge) {
    // two CTAs an SM: batch 32 x 32k, window 4,096 takes 21.1 us in a graph (partly
    // from L2), 33.7 with one and 27.4 with four; 16 x 2,000 keys of 8 kv heads 20.4,
    // 31.5 and 25.8; four query tokens, batch 64, 39.7, 60.4 and 49.6.  Up to 8 of a
    // row form a cluster, also where there is room for more, up to 1,024 keys each.
    // None takes more than 16,384 keys of the longest request that the block table
    // can hold (lengths are on the device), so that one long request does not run on
    // few SMs: dense, a table for 1M tokens, 127 requests of 4,000 and one of 1M
    // take 0.46 ms, 11.1 without this bound.  Short requests pay for such a table:
    // 128 of 2,000 take 227 us, 34 without the bound, 256 of 8,192 586 and 236.
    p.splits = (int)std::max(1LL, std::min({2LL * kPlanSMs / pairs, ceil_ll(span, 128), 64LL}));
    p.splits = (int)std::max<long long>(p.splits, std::min(ceil_ll(span, 16384), 64LL));
    if (p.splits > kMaxCluster && span <= 1024LL * kMaxCluster) p.splits = kMaxCluster;
    p.cluster = p.splits > 1 && p.splits <= kMaxCluster;
  } else {
    // tails of very different lengths: up to eight CTAs an SM (128 tails of 1 to
    // 8,192 keys behind one prefix: 292 us in all against 308 with half as many),
    // of 512 keys, but two from 256 keys on.  A CTA begins with a chain of look-ups
    // in L2: 32 tails of up to 4,096 keys took 36.6 us in all with 512, 41.2 with
    // 256, 40.9 with 1,024; 8 of up to 8,192 19.1, 27.7 and 18.3; but 64 of up to 512
    // 32.0 with one piece and 29.6 with two.
    const long long pieces = std::max(ceil_ll(span, 512), std::min(ceil_ll(span, 256), 2LL));
    p.splits = (int)std::max(1LL, std::min({8LL * kPlanSMs / pairs, pieces, 64LL}));
  }
  return p;
}

// Many rows of a 16-bit or 8-bit cache: one CTA (an SM's) of the tensor-core
// kernel per (sequence, kv head, 256 rows, split).
AttnPlan plan_tiles(long long seqs, int Hkv, long long rows, long long span) {
  AttnPlan p = {};
  p.tiles = ceil_ll(std::max(rows, 1LL), 2 * qsa::attn::kTileRows);
  const long long ctas = std::max(1LL, seqs * Hkv * p.tiles);
  // one wave of CTAs for one sequence; about two for several, whose lengths may
  // differ (eight fp8 prefixes of 3,001 to 16,384 keys: 174 us against 179 with one
  // wave and 196 with three); a split takes four tiles of keys at least (eight:
  // 60 against 54 us for one prefix of 28,672)
  const long long waves = seqs > 1 && ctas < kPlanSMs ? 2 : 1;
  p.splits = (int)std::max(1LL, std::min({waves * kPlanSMs / ctas, ceil_ll(span, 4 * qsa::attn::kTileKeys), 64LL}));
  return p;
}

// Bytes of the partial results of `rows` (token, head) rows.
size_t parts_o_bytes(long long rows, int slots, int D) {
  return align_up((size_t)rows * slots * D * sizeof(float));
}
size_t parts_bytes(long long rows, int slots, int D) {
  return slots > 1 ? parts_o_bytes(rows, slots, D) + align_up((size_t)rows * slots * sizeof(float)) : 0;
}

// -------------------------------------------------------------- validation --
qsa_status check_attn(const qsa_cache *c, int32_t Hq, int32_t T, int32_t q_dtype, float sm_scale) {
  qsa_status st = check_cache(c);
  if (st != QSA_OK) return st;
  if (Hq < 1 || Hq % c->num_kv_heads != 0 || T < 1) return QSA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return QSA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return QSA_ERR_UNSUPPORTED;
  if (T > qsa::attn::kMaxT || Hq / c->num_kv_heads * T > qsa::attn::kMaxGroup) return QSA_ERR_UNSUPPORTED;
  if (c->kv_dtype == QSA_F32 ? q_dtype != QSA_F32
                             : (q_dtype != QSA_BF16 || (c->kv_dtype != QSA_BF16 && c->kv_dtype != QSA_FP8_E4M3)))
    return QSA_ERR_UNSUPPORTED;
  if (!c->k_cache || !c->v_cache || !aligned(c->k_cache, 16) || !aligned(c->v_cache, 16)) return QSA_ERR_INVALID_ARG;
  if (c->kv_dtype == QSA_FP8_E4M3 && (!c->k_scale || !c->v_scale)) return QSA_ERR_INVALID_ARG;
  return QSA_OK;
}

// Keys a request of this cache can hold at most.
long long ctx_cap(const qsa_cache *c) {
  return std::min<long long>((long long)c->max_pages_per_req * c->page_size, 0x7fffffffLL);
}

qsa::attn::Args attn_args(const qsa_cache *c, int32_t B, int32_t T, int32_t Hq, int32_t n_tok, const void *q,
                          const int32_t *ctx_lens, float sm_scale, void *o, float *lse) {
  qsa::attn::Args a = {};
  a.c = to_dev(c);
  if (c->kv_dtype != QSA_FP8_E4M3) a.c.k_scale = a.c.v_scale = nullptr;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.G = Hq / c->num_kv_heads;
  a.n_tok = n_tok;
  a.ctx_lens = ctx_lens;
  a.window = 0x7fffffff;
  a.scale_log2 = sm_scale * qsa::attn::kLog2e;
  return a;
}

void set_parts(qsa::attn::Args &a, int slots, void *workspace) {
  a.slots = slots;
  a.o_part = static_cast<float *>(workspace);
  a.lse_part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                         parts_o_bytes((long long)a.n_tok * a.Hq, slots, a.c.head_dim));
}

// ----------------------------------------------------------------- launch --
template <int MODE, int D>
qsa_status launch_simple(const qsa::attn::Args &a, const AttnPlan &pl, long long seqs, cudaStream_t s) {
  static bool done[kMaxDevices] = {false};
  auto kernel = qsa::attn::simple_kernel<MODE, D>;
  const size_t smem = sizeof(qsa::attn::SimpleSmem<D>);
  {
    std::lock_guard<std::mutex> lk(g_mutex);
    if (prepare_kernel(kernel, smem, done) != cudaSuccess) return QSA_ERR_CUDA;
  }
  const dim3 grid((unsigned)pl.tiles, (unsigned)(a.c.num_kv_heads * pl.splits), (unsigned)seqs);
  return launch(true, kernel, grid, dim3(qsa::attn::kSimpleThreads), smem, s, a);
}

// The K/V caches for TMA: boxes of the largest power of two of rows, up to the
// 32 that a loader warp fills, that divides the page size.  rows = 0 (the
// kernel gathers every row) for fp8 caches, whose rows are converted, for pages
// that are no multiple of 8 tokens, and where a row index passes 31 bits.
qsa_status tile_maps(const qsa::attn::Args &a, qsa::attn::TileMaps &m) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = []() {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  m.rows = 0;
  const int P = a.c.page_size;
  const long long rows = (long long)a.c.num_pages * P;
  if (a.c.kv_dtype != QSA_BF16 || P % 8 != 0 || rows > 0x7fffffffLL) return QSA_OK;
  if (!encode) return QSA_ERR_CUDA;
  m.rows = P % 32 == 0 ? 32 : P % 16 == 0 ? 16 : 8;
  const cuuint64_t D = a.c.head_dim, H = a.c.num_kv_heads;
  const cuuint64_t dims[3] = {D, H, (cuuint64_t)rows}, strides[2] = {2 * D, 2 * D * H};
  const cuuint32_t box[3] = {(cuuint32_t)qsa::attn::kBoxCols, 1, (cuuint32_t)m.rows}, ones[3] = {1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (encode(i ? &m.v : &m.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(i ? a.c.v_cache : a.c.k_cache), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return QSA_ERR_CUDA;
  return QSA_OK;
}

template <int MODE, int D, bool FP8>
qsa_status launch_tile(const qsa::attn::Args &a, const AttnPlan &pl, long long seqs, cudaStream_t s) {
  static bool done[kMaxDevices] = {false};
  auto kernel = qsa::attn::tile_kernel<MODE, D, FP8>;
  const size_t smem = sizeof(qsa::attn::TileSmem<D>) + 1024;
  {
    std::lock_guard<std::mutex> lk(g_mutex);
    if (prepare_kernel(kernel, smem, done) != cudaSuccess) return QSA_ERR_CUDA;
  }
  qsa::attn::TileMaps maps = {};
  const qsa_status st = tile_maps(a, maps);
  if (st != QSA_OK) return st;
  return launch(true, kernel, dim3((unsigned)pl.tiles, (unsigned)(a.c.num_kv_heads * pl.splits), (unsigned)seqs),
                dim3(qsa::attn::kTileThreads), smem, s, a, maps);
}

// The rows of `seqs` sequences, as pl splits them.
template <int MODE>
qsa_status launch_rows(qsa::attn::Args a, const AttnPlan &pl, long long seqs, int slot0, cudaStream_t s) {
  a.slot0 = slot0;
  a.splits = pl.splits;
  if (pl.tiles > 0x7fffffffLL || (long long)a.c.num_kv_heads * pl.splits > 65535 || seqs > 65535)
    return QSA_ERR_UNSUPPORTED;
  if (a.c.kv_dtype == QSA_F32)
    return a.c.head_dim == 64 ? launch_simple<MODE, 64>(a, pl, seqs, s) : launch_simple<MODE, 128>(a, pl, seqs, s);
  if constexpr (MODE != qsa::attn::kTail) {
    const bool fp8 = a.c.kv_dtype == QSA_FP8_E4M3;
    if (a.c.head_dim == 64)
      return fp8 ? launch_tile<MODE, 64, true>(a, pl, seqs, s) : launch_tile<MODE, 64, false>(a, pl, seqs, s);
    return fp8 ? launch_tile<MODE, 128, true>(a, pl, seqs, s) : launch_tile<MODE, 128, false>(a, pl, seqs, s);
  }
  return QSA_ERR_UNSUPPORTED;  // (a 16-bit cache's tails are decode rows)
}

template <int MODE, int D, bool FP8, int NT>
qsa_status launch_stream(const qsa::attn::Args &a, const AttnPlan &pl, cudaStream_t s) {
  static bool done[kMaxDevices] = {false};
  auto kernel = qsa::attn::decode_kernel<MODE, D, FP8, NT>;
  const size_t smem = sizeof(qsa::attn::DecSmem<D, FP8, NT>) + 128;
  {
    std::lock_guard<std::mutex> lk(g_mutex);
    if (prepare_kernel(kernel, smem, done) != cudaSuccess) return QSA_ERR_CUDA;
  }
  return launch_cluster(true, kernel, dim3((unsigned)pl.splits, (unsigned)a.c.num_kv_heads, (unsigned)a.B),
                dim3(qsa::attn::kDecThreads), smem, s, pl.cluster ? pl.splits : 1, a);
}

template <int MODE, int D, bool FP8>
qsa_status launch_stream_nt(const qsa::attn::Args &a, const AttnPlan &pl, cudaStream_t s) {
  const int M = a.T * a.G;
  return M <= 8    ? launch_stream<MODE, D, FP8, 1>(a, pl, s)
         : M <= 16 ? launch_stream<MODE, D, FP8, 2>(a, pl, s)
                   : launch_stream<MODE, D, FP8, 4>(a, pl, s);
}

// T query tokens of each request (kWindow or kTail).
template <int MODE>
qsa_status launch_decode_rows(qsa::attn::Args a, const AttnPlan &pl, int slot0, cudaStream_t s) {
  if (a.c.kv_dtype == QSA_F32) return launch_rows<MODE>(a, pl, a.B, slot0, s);
  a.slot0 = slot0;
  a.splits = pl.splits;
  a.cluster = pl.cluster;
  if (a.c.num_kv_heads > 65535) return QSA_ERR_UNSUPPORTED;
  const bool fp8 = a.c.kv_dtype == QSA_FP8_E4M3;
  if (a.c.head_dim == 64)
    return fp8 ? launch_stream_nt<MODE, 64, true>(a, pl, s) : launch_stream_nt<MODE, 64, false>(a, pl, s);
  return fp8 ? launch_stream_nt<MODE, 128, true>(a, pl, s) : launch_stream_nt<MODE, 128, false>(a, pl, s);
}

template <int W>
qsa_status launch_attn_merge_w(const qsa::attn::Args &a, cudaStream_t s) {
  using namespace qsa::attn;
  const long long rows = (long long)a.n_tok * a.Hq, grid = W == 1 ? ceil_ll(rows, kMergeWarps) : rows;
  if (grid > 0x7fffffffLL) return QSA_ERR_UNSUPPORTED;
  const bool f32 = a.c.kv_dtype == QSA_F32;
  auto k = a.c.head_dim == 64 ? (f32 ? merge_kernel<64, float, W> : merge_kernel<64, __nv_bfloat16, W>)
                              : (f32 ? merge_kernel<128, float, W> : merge_kernel<128, __nv_bfloat16, W>);
  return launch(true, k, dim3((unsigned)grid), dim3(kMergeThreads), 0, s, a);
}

qsa_status launch_attn_merge(const qsa::attn::Args &a, cudaStream_t s) {
  return a.slots <= qsa::attn::kMergeFew ? launch_attn_merge_w<1>(a, s)
                                         : launch_attn_merge_w<qsa::attn::kMergeWarps>(a, s);
}

AttnPlan plan_decode(const qsa_cache *c, int B, int T, int Hq, long long window, long long sinks, bool merge) {
  const long long span = span_bound(window, sinks, T, ctx_cap(c));
  if (c->kv_dtype != QSA_F32) return plan_stream(B, c->num_kv_heads, span, merge);
  return plan_simple(B, c->num_kv_heads, (long long)T * (Hq / c->num_kv_heads), span);
}

AttnPlan plan_chunk(const qsa_cache *c, int B, long long max_q, int Hq, long long window, long long sinks) {
  const long long span = span_bound(window, sinks, max_q, ctx_cap(c));
  if (c->kv_dtype != QSA_F32) return plan_tiles(B, c->num_kv_heads, max_q * (Hq / c->num_kv_heads), span);
  return plan_simple(B, c->num_kv_heads, max_q * (Hq / c->num_kv_heads), span);
}

AttnPlan plan_shared(const qsa_cache *c, int n_groups, long long max_group, int T, int Hq, long long max_prefix) {
  if (c->kv_dtype != QSA_F32)
    return plan_tiles(n_groups, c->num_kv_heads, max_group * T * (Hq / c->num_kv_heads), max_prefix);
  return plan_simple(n_groups, c->num_kv_heads, max_group * T * (Hq / c->num_kv_heads), max_prefix);
}

bool prefix_args_ok(int32_t B, int32_t n_groups, int32_t max_group, int32_t max_prefix, int32_t max_tail) {
  return n_groups >= 1 && n_groups <= std::max(B, 1) && max_group >= 1 && max_group <= B && max_prefix >= 0 &&
         max_tail >= 0;
}

// ------------------------------------------------------------------- rope --
template <int D, typename T, typename CT>
qsa_status launch_rope(const qsa::rope::Params &p, bool vec, int layout, cudaStream_t s) {
  using namespace qsa::rope;
  const int heads = p.Hq + 2 * p.c.num_kv_heads;
  if (!vec) {
    const long long grid = ceil_ll((long long)p.n_tok * 32, kThreads);
    return launch(true, rope_append_any_kernel<D, T, CT>, dim3((unsigned)grid), dim3(kThreads), 0, s, p, layout);
  }
  constexpr int kStep = 32 / (D / 16);
  constexpr int NB = sizeof(T) == 4 ? 2 : 5;
  const long long few = (long long)p.n_tok * ceil_ll(heads, kStep);
  // one step a warp while that leaves the GPU room (128 tokens: latency), NB steps,
  // all loaded at once, for more: 22,000 tokens of 40 heads take 99 us with one,
  // 76, 74, 73 and 72 with two to five (four times the registers from there on).
  // The last warp of a token takes what is left: parts alike in its place were
  // slower for every head count (16,000 tokens: 24 heads 36.9 against 36.0 us, 36
  // 48.3 and 47.5, 44 59.9 and 59.0, 40 52.6 and 52.2).
  const bool one = few <= 16LL * kPlanSMs;
  const long long warps = (long long)p.n_tok * ceil_ll(heads, kStep * (one ? 1 : NB));
  const long long grid = ceil_ll(warps * 32, kThreads);
  if (grid > 0x7fffffffLL) return QSA_ERR_UNSUPPORTED;
  auto k = layout ? (one ? rope_append_kernel<D, T, CT, true, 1> : rope_append_kernel<D, T, CT, true, NB>)
                  : (one ? rope_append_kernel<D, T, CT, false, 1> : rope_append_kernel<D, T, CT, false, NB>);
  return launch(true, k, dim3((unsigned)grid), dim3(kThreads), 0, s, p);
}

template <int D>
qsa_status launch_rope_d(const qsa::rope::Params &p, bool vec, int layout, cudaStream_t s) {
  switch (p.c.kv_dtype) {
    case QSA_F32: return launch_rope<D, float, float>(p, vec, layout, s);
    case QSA_BF16: return launch_rope<D, __nv_bfloat16, __nv_bfloat16>(p, vec, layout, s);
    default: return launch_rope<D, __nv_bfloat16, __nv_fp8_e4m3>(p, vec, layout, s);
  }
}

}  // namespace

extern "C" {

qsa_status qsa_rope_freqs(int32_t rotary_dim, double theta, int32_t scaling, double factor,
                          int32_t original_max_position, double beta_fast, double beta_slow, double *inv_freq,
                          uint64_t *freqs, float *mscale) {
  if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > 128 || !(theta > 1.0) || !std::isfinite(theta))
    return QSA_ERR_INVALID_ARG;
  if (scaling < QSA_ROPE_SCALING_NONE || scaling > QSA_ROPE_SCALING_YARN) return QSA_ERR_INVALID_ARG;
  if (scaling != QSA_ROPE_SCALING_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return QSA_ERR_INVALID_ARG;
  if (scaling == QSA_ROPE_SCALING_NTK && rotary_dim == 2) return QSA_ERR_INVALID_ARG;
  if (scaling == QSA_ROPE_SCALING_YARN &&
      (original_max_position < 1 || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast)))
    return QSA_ERR_INVALID_ARG;
  if (!freqs || !mscale) return QSA_ERR_INVALID_ARG;
  const double kTurn = 6.283185307179586476925286766559;
  const int R = rotary_dim;
  double base = theta, low = 0.0, high = 0.0;
  if (scaling == QSA_ROPE_SCALING_NTK) base = theta * std::pow(factor, (double)R / (R - 2));
  if (scaling == QSA_ROPE_SCALING_YARN) {
    // the (real) pair index that turns `beta` times over the trained length
    auto pair_of = [&](double beta) {
      return R * std::log(original_max_position / (beta * kTurn)) / (2.0 * std::log(base));
    };
    low = std::max(std::floor(pair_of(beta_fast)), 0.0);
    high = std::min(std::ceil(pair_of(beta_slow)), (double)(R - 1));
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R);
    if (scaling == QSA_ROPE_SCALING_LINEAR) f /= factor;
    if (scaling == QSA_ROPE_SCALING_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    if (inv_freq) inv_freq[i] = f;
    // turns per token, below 1, in 2^-64 units
    const double turns = f / kTurn;
    freqs[i] = (uint64_t)std::ldexp(turns - std::floor(turns), 64);
  }
  *mscale = scaling == QSA_ROPE_SCALING_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return QSA_OK;
}

qsa_status qsa_rope_append(const qsa_cache *cache, int32_t B, int32_t n_tokens, const int32_t *pos0,
                           const int32_t *cu_new, const void *q, int64_t q_stride, const void *k,
                           int64_t k_stride, const void *v, int64_t v_stride, int32_t dtype, int32_t Hq,
                           const uint64_t *freqs, int32_t rotary_dim, int32_t layout, float mscale, void *q_out,
                           qsa_stream_t stream) {
  qsa_status st = check_cache(cache);
  if (st != QSA_OK) return st;
  const int D = cache->head_dim;
  if (B < 0 || n_tokens < 0 || Hq < 1) return QSA_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > D) return QSA_ERR_INVALID_ARG;
  if (layout != QSA_ROPE_HALF && layout != QSA_ROPE_INTERLEAVED) return QSA_ERR_INVALID_ARG;
  if (!std::isfinite(mscale)) return QSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return QSA_ERR_UNSUPPORTED;
  if (cache->kv_dtype == QSA_F32 ? dtype != QSA_F32
                                 : (dtype != QSA_BF16 ||
                                    (cache->kv_dtype != QSA_BF16 && cache->kv_dtype != QSA_FP8_E4M3)))
    return QSA_ERR_UNSUPPORTED;
  if (B == 0 || n_tokens == 0) return QSA_OK;
  if (!pos0 || !cu_new || !q || !k || !v || !q_out || (!freqs && rotary_dim > 0) || !cache->k_cache || !cache->v_cache)
    return QSA_ERR_INVALID_ARG;
  if (cache->kv_dtype == QSA_FP8_E4M3 && (!cache->k_scale || !cache->v_scale)) return QSA_ERR_INVALID_ARG;
  const size_t e = dtype == QSA_F32 ? 4 : 2, ce = cache->kv_dtype == QSA_F32 ? 4 : cache->kv_dtype == QSA_BF16 ? 2 : 1;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(q_out, e) || !aligned(freqs, 8) ||
      !aligned(cache->k_cache, ce) || !aligned(cache->v_cache, ce))
    return QSA_ERR_INVALID_ARG;
  const int64_t kv_row = (int64_t)cache->num_kv_heads * D;
  if (q_stride < (int64_t)Hq * D || k_stride < kv_row || v_stride < kv_row) return QSA_ERR_INVALID_ARG;
  // in place only where the rows lie as those of q_out
  if (q_out == q && q_stride != (int64_t)Hq * D) return QSA_ERR_INVALID_ARG;
  if ((long long)n_tokens > 0x7fffffffLL / 4) return QSA_ERR_UNSUPPORTED;
  qsa::rope::Params p = {};
  p.c = to_dev(cache);
  p.B = B;
  p.n_tok = n_tokens;
  p.Hq = Hq;
  p.pos0 = pos0;
  p.cu = cu_new;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.freqs = freqs;
  p.R = rotary_dim;
  p.mscale = mscale;
  p.q_out = q_out;
  const bool vec = rotary_dim % 16 == 0 && aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(q_out, 16) &&
                   aligned(cache->k_cache, 16) && aligned(cache->v_cache, 16) &&
                   (q_stride * e) % 16 == 0 && (k_stride * e) % 16 == 0 && (v_stride * e) % 16 == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return D == 64 ? launch_rope_d<64>(p, vec, layout, s) : launch_rope_d<128>(p, vec, layout, s);
}

size_t qsa_window_decode_workspace_bytes(const qsa_cache *cache, int32_t B, int32_t T, int32_t Hq, int32_t window,
                                         int32_t sinks) {
  if (check_cache(cache) != QSA_OK || B < 1 || T < 1 || Hq < 1 || Hq % cache->num_kv_heads != 0 || window < 1 ||
      sinks < 0)
    return 0;
  return parts_bytes((long long)B * T * Hq, plan_decode(cache, B, T, Hq, window, sinks, true).slots(), cache->head_dim);
}

qsa_status qsa_window_decode(const qsa_cache *cache, int32_t B, int32_t T, int32_t Hq, const void *q, int32_t q_dtype,
                             const int32_t *ctx_lens, int32_t window, int32_t sinks, float sm_scale, void *o,
                             float *lse, void *workspace, size_t workspace_bytes, qsa_stream_t stream) {
  qsa_status st = check_attn(cache, Hq, T, q_dtype, sm_scale);
  if (st != QSA_OK) return st;
  if (B < 0 || window < 1 || sinks < 0) return QSA_ERR_INVALID_ARG;
  if (B == 0) return QSA_OK;
  if (B > 65535) return QSA_ERR_UNSUPPORTED;
  if (!q || !ctx_lens || !o || !lse || !aligned(q, 16) || !aligned(o, 16)) return QSA_ERR_INVALID_ARG;
  const size_t need = qsa_window_decode_workspace_bytes(cache, B, T, Hq, window, sinks);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return QSA_ERR_INVALID_ARG;
  const AttnPlan pl = plan_decode(cache, B, T, Hq, window, sinks, true);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  qsa::attn::Args a = attn_args(cache, B, T, Hq, B * T, q, ctx_lens, sm_scale, o, lse);
  a.window = window;
  a.sinks = sinks;
  set_parts(a, pl.slots(), workspace);
  st = launch_decode_rows<qsa::attn::kWindow>(a, pl, 0, s);
  return st != QSA_OK || pl.slots() == 1 ? st : launch_attn_merge(a, s);
}

size_t qsa_window_prefill_workspace_bytes(const qsa_cache *cache, int32_t B, int32_t n_tokens, int32_t max_q_per_req,
                                          int32_t Hq, int32_t window, int32_t sinks) {
  if (check_cache(cache) != QSA_OK || B < 1 || n_tokens < 1 || max_q_per_req < 1 || Hq < 1 ||
      Hq % cache->num_kv_heads != 0 || window < 1 || sinks < 0)
    return 0;
  max_q_per_req = std::min(max_q_per_req, n_tokens);
  return parts_bytes((long long)n_tokens * Hq, plan_chunk(cache, B, max_q_per_req, Hq, window, sinks).splits,
                     cache->head_dim);
}

qsa_status qsa_window_prefill(const qsa_cache *cache, int32_t B, int32_t n_tokens, int32_t max_q_per_req,
                              const int32_t *cu_q, const int32_t *ctx_lens, const void *q, int32_t q_dtype, int32_t Hq,
                              int32_t window, int32_t sinks, float sm_scale, void *o, float *lse, void *workspace,
                              size_t workspace_bytes, qsa_stream_t stream) {
  qsa_status st = check_attn(cache, Hq, 1, q_dtype, sm_scale);
  if (st != QSA_OK) return st;
  if (B < 0 || n_tokens < 0 || max_q_per_req < 0 || window < 1 || sinks < 0) return QSA_ERR_INVALID_ARG;
  if (B == 0 || n_tokens == 0 || max_q_per_req == 0) return QSA_OK;
  max_q_per_req = std::min(max_q_per_req, n_tokens);
  // rows (tokens x heads of a group) are counted in 31 bits
  if (B > 65535 || (long long)n_tokens * (Hq / cache->num_kv_heads) > 0x7ffffc00LL) return QSA_ERR_UNSUPPORTED;
  if (!cu_q || !q || !ctx_lens || !o || !lse || !aligned(q, 16) || !aligned(o, 16)) return QSA_ERR_INVALID_ARG;
  const size_t need = qsa_window_prefill_workspace_bytes(cache, B, n_tokens, max_q_per_req, Hq, window, sinks);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return QSA_ERR_INVALID_ARG;
  const AttnPlan pl = plan_chunk(cache, B, max_q_per_req, Hq, window, sinks);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  qsa::attn::Args a = attn_args(cache, B, 1, Hq, n_tokens, q, ctx_lens, sm_scale, o, lse);
  a.cu = cu_q;
  a.n_cu = B;
  a.max_tokens = max_q_per_req;
  a.window = window;
  a.sinks = sinks;
  set_parts(a, pl.splits, workspace);
  st = launch_rows<qsa::attn::kWindow>(a, pl, B, 0, s);
  return st != QSA_OK || pl.splits == 1 ? st : launch_attn_merge(a, s);
}

size_t qsa_prefix_decode_workspace_bytes(const qsa_cache *cache, int32_t B, int32_t T, int32_t Hq, int32_t n_groups,
                                         int32_t max_group, int32_t max_prefix, int32_t max_tail) {
  if (check_cache(cache) != QSA_OK || B < 1 || T < 1 || Hq < 1 || Hq % cache->num_kv_heads != 0 ||
      !prefix_args_ok(B, n_groups, max_group, max_prefix, max_tail))
    return 0;
  const int slots = plan_shared(cache, n_groups, max_group, T, Hq, max_prefix).splits +
                    plan_decode(cache, B, T, Hq, std::max(max_tail, 1), 0, false).splits;
  return parts_bytes((long long)B * T * Hq, slots, cache->head_dim);
}

qsa_status qsa_prefix_decode(const qsa_cache *cache, int32_t B, int32_t T, int32_t Hq, const void *q, int32_t q_dtype,
                             const int32_t *ctx_lens, int32_t n_groups, const int32_t *cu_group,
                             const int32_t *prefix_lens, int32_t max_group, int32_t max_prefix, int32_t max_tail,
                             float sm_scale, void *o, float *lse, void *workspace, size_t workspace_bytes,
                             qsa_stream_t stream) {
  qsa_status st = check_attn(cache, Hq, T, q_dtype, sm_scale);
  if (st != QSA_OK) return st;
  if (B < 0) return QSA_ERR_INVALID_ARG;
  if (B == 0) return QSA_OK;
  if (B > 65535) return QSA_ERR_UNSUPPORTED;
  if (!prefix_args_ok(B, n_groups, max_group, max_prefix, max_tail)) return QSA_ERR_INVALID_ARG;
  if (!q || !ctx_lens || !cu_group || !prefix_lens || !o || !lse || !aligned(q, 16) || !aligned(o, 16))
    return QSA_ERR_INVALID_ARG;
  const size_t need = qsa_prefix_decode_workspace_bytes(cache, B, T, Hq, n_groups, max_group, max_prefix, max_tail);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return QSA_ERR_INVALID_ARG;
  const AttnPlan shared = plan_shared(cache, n_groups, max_group, T, Hq, max_prefix);
  const AttnPlan tail = plan_decode(cache, B, T, Hq, std::max(max_tail, 1), 0, false);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  qsa::attn::Args a = attn_args(cache, B, T, Hq, B * T, q, ctx_lens, sm_scale, o, lse);
  a.cu = cu_group;
  a.n_cu = n_groups;
  a.prefix_lens = prefix_lens;
  set_parts(a, shared.splits + tail.splits, workspace);
  a.max_tokens = max_group * T;
  st = launch_rows<qsa::attn::kShared>(a, shared, n_groups, 0, s);
  if (st != QSA_OK) return st;
  st = launch_decode_rows<qsa::attn::kTail>(a, tail, shared.splits, s);
  return st != QSA_OK ? st : launch_attn_merge(a, s);
}

}  // extern "C"

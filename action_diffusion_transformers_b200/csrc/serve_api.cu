// serve_api.cu - host side of the serving calls declared in include/sage.h:
// rotary positions, the quantized KV cache, and attention over packed prompts
// and over the cache.  Validates every argument, picks the kernel variant and
// launches on the caller's stream.  Nothing here allocates device memory or
// synchronises.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "sage.h"
#include "sage_host.h"
#include "serve_prompt.cuh"
#include "serve_rows.cuh"
#include "serve_token.cuh"

namespace {

using sage_host::aligned16;
using sage_host::device_setup;
using sage_host::fail;
using sage_host::launch_check;
using sage_host::pdl_launch;
using sage_host::pdl_launch_clusters;

// Token stride of a call's rows (0 means contiguous).
sage_status check_stride(int64_t stride, int H, int D, const char* name, int64_t* out) {
  const int64_t hd = static_cast<int64_t>(H) * D;
  const int64_t s = stride == 0 ? hd : stride;
  if (s < hd) return fail(SAGE_ERR_INVALID_ARG, "%s %lld < H*D %lld", name, (long long)s, (long long)hd);
  if (s % 8 != 0) return fail(SAGE_ERR_ALIGNMENT, "%s %lld is not a multiple of 8", name, (long long)s);
  if (s >= (int64_t(1) << 37)) return fail(SAGE_ERR_INVALID_ARG, "%s %lld is too large", name, (long long)s);
  *out = s;
  return SAGE_OK;
}

sage_status check_cache(const sage_kv_cache& c, sage::KvCacheView* v) {
  if (c.num_pages < 1 || c.Hk < 1)
    return fail(SAGE_ERR_INVALID_ARG, "num_pages and Hk must be >= 1 (got %d, %d)", c.num_pages, c.Hk);
  if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)))
    return fail(SAGE_ERR_UNSUPPORTED, "page_size must be a power of two in 16 .. 1024 (got %d)", c.page_size);
  if (c.D != 64 && c.D != 128) return fail(SAGE_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", c.D);
  if (c.format != SAGE_KV_INT8 && c.format != SAGE_KV_E4M3)
    return fail(SAGE_ERR_INVALID_ARG, "format must be a sage_kv_format value (got %d)", c.format);
  SAGE_NEED(c.k_codes, "k_codes");
  SAGE_NEED(c.k_scale, "k_scale");
  SAGE_NEED(c.v_codes, "v_codes");
  SAGE_NEED(c.v_scale, "v_scale");
  v->codes[0] = static_cast<uint8_t*>(c.k_codes);
  v->codes[1] = static_cast<uint8_t*>(c.v_codes);
  v->scale[0] = c.k_scale;
  v->scale[1] = c.v_scale;
  v->slots = static_cast<int64_t>(c.num_pages) * c.page_size;
  v->Hk = c.Hk;
  v->page_shift = 0;
  while ((1 << v->page_shift) < c.page_size) ++v->page_shift;
  v->by_heads = sage::FastDiv(static_cast<uint32_t>(c.Hk));
  return SAGE_OK;
}

template <class F>
void with_type(int dtype, F f) {
  if (dtype == SAGE_BF16) f(sage::Bf16T{});
  else if (dtype == SAGE_FP16) f(sage::Fp16T{});
  else f(sage::Fp32T{});
}
template <class F>
void with_flag(bool on, F f) {
  if (on) f(std::true_type{});
  else f(std::false_type{});
}

int ceil_log2(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

sage_status kv_rows_args(const void* k, const void* v, int T, int64_t k_stride, int64_t v_stride, int dtype,
                         const int64_t* slots, const sage_kv_cache& cache, sage::KvRowsParams* p) {
  sage_status st;
  if ((st = check_cache(cache, &p->c)) != SAGE_OK) return st;
  if (T < 0) return fail(SAGE_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
  if (static_cast<int64_t>(T) * cache.Hk >= (int64_t(1) << 31))
    return fail(SAGE_ERR_INVALID_ARG, "T*Hk must stay below 2^31");
  if (dtype != SAGE_BF16 && dtype != SAGE_FP16 && dtype != SAGE_FP32)
    return fail(SAGE_ERR_INVALID_ARG, "dtype must be a sage_dtype value (got %d)", dtype);
  if ((st = check_stride(k_stride, cache.Hk, cache.D, "k_stride", &p->stride[0])) != SAGE_OK) return st;
  if ((st = check_stride(v_stride, cache.Hk, cache.D, "v_stride", &p->stride[1])) != SAGE_OK) return st;
  if (T > 0) {
    SAGE_NEED(k, "k");
    SAGE_NEED(v, "v");
    if (!slots) return fail(SAGE_ERR_INVALID_ARG, "slots is NULL");
    if (reinterpret_cast<uintptr_t>(slots) & 7u) return fail(SAGE_ERR_ALIGNMENT, "slots is not 8-byte aligned");
  }
  p->rows[0] = const_cast<void*>(k);
  p->rows[1] = const_cast<void*>(v);
  p->slot = slots;
  p->T = T;
  return SAGE_OK;
}

// Query heads per CTA of the single-token attention, in blocks of 8.
int token_nt(int G) { return G > 8 ? 2 : 1; }

// Segments of a sequence.
int64_t token_segs(int Hk, int G) { return static_cast<int64_t>(Hk) * ((G + 8 * token_nt(G) - 1) / (8 * token_nt(G))); }
int64_t token_tiles(int max_len) { return (static_cast<int64_t>(max_len) + sage::kTokTile - 1) / sage::kTokTile; }
// Tiles of a chunk: as many chunks as CTAs are resident (three per SM), a tile
// per warp at least, 16 per warp at most, so that uneven sequences spread over
// the SMs.  (8 KV heads, D = 128, E4M3: one sequence of 8192 keys takes 9.9 us
// with 444 chunks wanted and 13.4 with 1776, three of 2000 to 8000 keys 13.9 and
// 20.5; 64 of 300 to 8192 keys 110 us with 4 tiles per warp, 103 with 8, 102 with
// 16.)
constexpr int kTokWant = 148 * sage::kTokPerSm, kTokPerMax = 16;
int token_per(int B, int Hk, int G, int max_len) {
  const int64_t tiles = token_tiles(max_len), w = sage::kTokWarps;
  const int64_t chunks = std::max<int64_t>(1, kTokWant / std::max<int64_t>(1, B * token_segs(Hk, G)));
  const int64_t per = (tiles + chunks - 1) / chunks;
  return static_cast<int>(std::max(w, std::min(kTokPerMax * w, (per + w - 1) / w * w)));
}
int token_chunks(int max_len, int per) {
  return static_cast<int>(std::max<int64_t>(1, (token_tiles(max_len) + per - 1) / per));
}

// Most chunks of all sequences together in any call of up to B sequences and max_len
// keys (0: the chunks' results need no workspace).  Fewer sequences are cut into more
// chunks, and a shorter max_len into as many shorter ones, so this and not the call's
// own number is what a workspace kept for many calls has to hold.  A call of b
// sequences has at most as many chunks each as are wanted or as there are tiles for the
// warps of one, and, where they are as long as may be, one per kTokPerMax tiles a warp;
// from kTokWant sequences on only the latter counts, and grows with b.
int64_t token_chunks_bound(int B, int Hk, int G, int max_len) {
  const int64_t tiles = token_tiles(max_len), w = sage::kTokWarps, segs = token_segs(Hk, G);
  int64_t most = 0;
  auto take = [&](int64_t b) {
    const int64_t wanted = std::max<int64_t>(1, kTokWant / (b * segs));
    const int64_t chunks = std::max(std::min(wanted, (tiles + w - 1) / w), (tiles + kTokPerMax * w - 1) / (kTokPerMax * w));
    if (chunks > 1) most = std::max(most, b * chunks);
  };
  for (int64_t b = 1; b <= std::min<int64_t>(B, kTokWant); ++b) take(b);
  take(B);
  return most;
}

// Workspace of the single-token attention: the chunks' results.
struct TokenWs {
  size_t part_lse, total;
};
TokenWs token_ws(int64_t chunks, int Hq, int D) {              // chunks of all sequences
  if (chunks == 0) return {0, 0};
  const size_t rows = static_cast<size_t>(chunks) * Hq;
  const size_t o = (rows * D * 4 + 255) / 256 * 256;
  return {o, o + (rows * 4 + 255) / 256 * 256};
}

// Shared memory limits of the attention kernels, once per device.
std::atomic<uint64_t> g_attn_ready{0};
std::atomic<int> g_clusters[64][sage::kPrMaxCluster + 1];   // clusters of so many CTAs resident at once, by device

template <class K>
void attr(cudaError_t* e, K kernel, int bytes) {
  if (*e == cudaSuccess) *e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
template <class E, int D>
void attn_attr(cudaError_t* e) {
  attr(e, sage::prompt_attn_kernel<E, D, false>, sage::PrSmem<D>::kAlloc);
  attr(e, sage::prompt_attn_kernel<E, D, true>, sage::PrSmem<D>::kAlloc);
  attr(e, sage::token_attn_kernel<E, D, 1, sage::kKvInt8>, sage::kTokSmem<D, 1>);
  attr(e, sage::token_attn_kernel<E, D, 1, sage::kKvE4m3>, sage::kTokSmem<D, 1>);
  attr(e, sage::token_attn_kernel<E, D, 2, sage::kKvInt8>, sage::kTokSmem<D, 2>);
  attr(e, sage::token_attn_kernel<E, D, 2, sage::kKvE4m3>, sage::kTokSmem<D, 2>);
}

sage_status attn_setup(int dev) {
  const uint64_t bit = uint64_t(1) << dev;
  if (g_attn_ready.load() & bit) return SAGE_OK;
  cudaError_t e = cudaSuccess;
  attn_attr<sage::Bf16T, 128>(&e);
  attn_attr<sage::Bf16T, 64>(&e);
  attn_attr<sage::Fp16T, 128>(&e);
  attn_attr<sage::Fp16T, 64>(&e);
  for (int c = 2; c <= sage::kPrMaxCluster && e == cudaSuccess; ++c) {
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = static_cast<unsigned>(c);
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(c));
    cfg.blockDim = dim3(sage::kPrThreads);
    cfg.dynamicSmemBytes = sage::PrSmem<128>::kAlloc;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, sage::prompt_attn_kernel<sage::Bf16T, 128, true>, &cfg);
    g_clusters[dev][c].store(n);
  }
  if (e != cudaSuccess) return sage_host::cuda_fail(e, "attention setup");
  g_attn_ready.fetch_or(bit);
  return SAGE_OK;
}

// Rows [T, H, D] as a 3-D map; one box is 128 rows x 64 channels of one head.
sage_status encode_rows(CUtensorMap* m, const void* base, int dtype, int64_t T, int H, int D, int64_t stride) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(sage::kPrTile)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = sage_host::encode_tiled()(
      m, dtype == SAGE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
      const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SAGE_ERR_CUDA, "cuTensorMapEncodeTiled (rows) failed (%d)", static_cast<int>(r));
  return SAGE_OK;
}

sage_status check_cu(const int32_t* cu, int n, const char* name) {
  if (!cu) return fail(SAGE_ERR_INVALID_ARG, "%s is NULL", name);
  if (cu[0] != 0) return fail(SAGE_ERR_INVALID_ARG, "%s[0] must be 0", name);
  for (int i = 0; i < n; ++i)
    if (cu[i + 1] < cu[i]) return fail(SAGE_ERR_INVALID_ARG, "%s must be non-decreasing (index %d)", name, i + 1);
  return SAGE_OK;
}

// sm_scale <= 0: 1/sqrt(D) formed in double and rounded once to float.
float scale_log2(float sm_scale, int D) {
  const float s = sm_scale > 0.f ? sm_scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  return static_cast<float>(static_cast<double>(s) * 1.4426950408889634);
}

sage_status check_heads(int Hq, int Hk) {
  if (Hk < 1 || Hq < 1 || Hq % Hk != 0)
    return fail(SAGE_ERR_INVALID_ARG, "Hq must be a positive multiple of Hk (got %d, %d)", Hq, Hk);
  return SAGE_OK;
}

sage_status check_scale(float s) {
  if (!(s < 3.0e38f) || !(s > -3.0e38f)) return fail(SAGE_ERR_INVALID_ARG, "sm_scale must be finite");
  return SAGE_OK;
}

// Row tile of an item (row tile, head) of a sequence.
int64_t prompt_row_tile(const sage::PromptParams& p, int item) { return p.share ? item / p.G : item; }

// Work of one CTA of the prompt kernel, for sorting: its time in halves of a pair's
// step over one key tile (an item alone takes half of them, its key tiles going to
// both tiles of the CTA) plus about one step for its start and end, in front of
// (sequence, which, pair).
uint64_t prompt_key(const sage::PromptParams& p, int i, int pair, uint32_t which) {
  const sage::PromptSeq& sq = p.seq[i];
  int64_t rt = prompt_row_tile(p, 2 * pair + (which == sage::kPrFirst ? 0 : 1));
  bool alone = which != sage::kPrBoth;
  if (!alone && rt * sage::kPrTile >= sq.lq) {
    rt = prompt_row_tile(p, 2 * pair);                             // a pair without its second item
    alone = true;
  }
  const int64_t last = std::min<int64_t>((rt + 1) * sage::kPrTile, sq.lq);
  const int64_t seen = p.causal ? std::max<int64_t>(0, std::min<int64_t>(sq.lk, last + sq.lk - sq.lq)) : sq.lk;
  const int64_t n = (seen + sage::kPrTile - 1) / sage::kPrTile;
  return static_cast<uint64_t>(alone ? n + 3 : 2 * n + 2) << 32 | static_cast<uint64_t>(i) << 24 | which << 20 |
         static_cast<uint64_t>(pair);
}

// End of each entry's last CTA when the CTAs (`lanes` of each entry, in order)
// start one after the other on the SM that is free first; returns the last end.
constexpr int kPrBalance = 128, kPrBalanceSms = 256;
int64_t prompt_ends(const uint64_t* keys, int n, int lanes, int sms, int64_t* ends) {
  struct Group {
    int64_t t;
    int count;
  } heap[kPrBalanceSms];                                 // SMs by the time at which they are free
  auto later = [](const Group& x, const Group& y) { return x.t > y.t; };
  int groups = 1;
  heap[0] = {0, sms};
  int64_t all = 0;
  for (int e = 0; e < n; ++e) {
    const int64_t cost = static_cast<int64_t>(keys[e] >> 32);
    Group done[kPrBalanceSms];
    int nd = 0, need = lanes;
    ends[e] = 0;
    while (need > 0) {
      if (groups == 0) {                                 // more CTAs of an entry than SMs
        for (; nd > 0; --nd) {
          heap[groups++] = done[nd - 1];
          std::push_heap(heap, heap + groups, later);
        }
      }
      std::pop_heap(heap, heap + groups, later);
      Group g = heap[--groups];
      const int take = std::min(g.count, need);
      need -= take;
      done[nd++] = {g.t + cost, take};
      ends[e] = std::max(ends[e], g.t + cost);
      if (g.count > take) {
        heap[groups++] = {g.t, g.count - take};
        std::push_heap(heap, heap + groups, later);
      }
    }
    for (; nd > 0; --nd) {
      heap[groups++] = done[nd - 1];
      std::push_heap(heap, heap + groups, later);
    }
    all = std::max(all, ends[e]);
  }
  return all;
}

// Sorts the entries, the longest first, and parts pairs whose end stands out into
// their two items, as long as that brings the last end forward.  Returns the
// number of entries.  Only for launches of few waves, where it counts.
int prompt_balance(const sage::PromptParams& p, uint64_t* keys, int n, int lanes, int sms) {
  auto larger = [](uint64_t x, uint64_t y) { return x > y; };
  std::sort(keys, keys + n, larger);
  if (n > kPrBalance || sms > kPrBalanceSms || static_cast<int64_t>(n) * lanes > 6 * static_cast<int64_t>(sms)) return n;
  int64_t ends[2 * kPrBalance];
  uint64_t next[2 * kPrBalance];
  int64_t all = prompt_ends(keys, n, lanes, sms, ends);
  for (int pass = 0; pass < 3; ++pass) {
    int64_t work = 0;
    for (int e = 0; e < n; ++e) work += static_cast<int64_t>(keys[e] >> 32) * lanes;
    const int64_t ideal = std::max(work / sms, static_cast<int64_t>(keys[0] >> 32) / 2), limit = ideal + ideal / 16;
    if (all <= limit) break;
    int m = 0;
    for (int e = 0; e < n; ++e) {
      const int seq = static_cast<int>(keys[e] >> 24 & 0xFF), pair = static_cast<int>(keys[e] & 0xFFFFF);
      const bool both = (keys[e] >> 20 & 3) == sage::kPrBoth &&
                        prompt_row_tile(p, 2 * pair + 1) * sage::kPrTile < p.seq[seq].lq;
      if (both && ends[e] > limit && m + n - e < 2 * kPrBalance) {
        next[m++] = prompt_key(p, seq, pair, sage::kPrFirst);
        next[m++] = prompt_key(p, seq, pair, sage::kPrSecond);
      } else {
        next[m++] = keys[e];
      }
    }
    if (m == n) break;
    std::sort(next, next + m, larger);
    const int64_t now = prompt_ends(next, m, lanes, sms, ends);
    if (now >= all) break;
    all = now;
    n = m;
    std::copy(next, next + m, keys);
  }
  return n;
}

// CTAs per item, its keys dealt out among them: the fewest of those whose clusters
// are all resident (15 of 8 CTAs, 33 of 4, 74 of 2 on a B200) that leave the longest
// item the fewest steps, if that saves three, about what the join takes (600 tokens
// x 8 heads 10.9 us alone and 13.3 in clusters, 128 queries over 1024 keys x 16
// heads 18.7 and 12.0).
constexpr int kPrJoinSteps = 3;
int prompt_cluster(const sage::PromptParams& p, int n_seq, int lanes, int dev) {
  if (p.share) return 1;
  int64_t items = 0, longest = 0;
  for (int i = 0; i < n_seq; ++i) {
    items += (static_cast<int64_t>(p.seq[i].lq) + sage::kPrTile - 1) / sage::kPrTile * lanes;
    longest = std::max<int64_t>(longest, (static_cast<int64_t>(p.seq[i].lk) + sage::kPrTile - 1) / sage::kPrTile);
  }
  auto steps = [&](int c) { return (longest + 2 * c - 1) / (2 * c); };
  int best = 1;
  for (int c = 2; c <= sage::kPrMaxCluster; ++c)
    if (items <= g_clusters[dev][c].load() && steps(c) < steps(best)) best = c;
  return steps(1) - steps(best) >= kPrJoinSteps ? best : 1;
}

// Every pair parted into its items.
int prompt_alone(const sage::PromptParams& p, uint64_t* keys, int n) {
  int m = n;
  for (int e = 0; e < n; ++e) {
    const int seq = static_cast<int>(keys[e] >> 24 & 0xFF), pair = static_cast<int>(keys[e] & 0xFFFFF);
    if (prompt_row_tile(p, 2 * pair + 1) * sage::kPrTile < p.seq[seq].lq)
      keys[m++] = prompt_key(p, seq, pair, sage::kPrSecond);
    keys[e] = prompt_key(p, seq, pair, sage::kPrFirst);
  }
  std::sort(keys, keys + m, [](uint64_t x, uint64_t y) { return x > y; });
  return m;
}

}  // namespace

extern "C" {

sage_status sage_rope_plan_init(sage_rope_plan* plan, int rot_dim, int interleaved, double base, int scaling,
                                double factor, int orig_len, double beta_fast, double beta_slow,
                                const unsigned char* axis) {
  if (!plan) return fail(SAGE_ERR_INVALID_ARG, "plan is NULL");
  if (rot_dim < 2 || rot_dim > 2 * SAGE_ROPE_MAX_PAIRS || rot_dim % 2 != 0)
    return fail(SAGE_ERR_INVALID_ARG, "rot_dim must be even, 2 .. %d (got %d)", 2 * SAGE_ROPE_MAX_PAIRS, rot_dim);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(SAGE_ERR_INVALID_ARG, "base must be finite and > 1");
  if (scaling < SAGE_ROPE_NONE || scaling > SAGE_ROPE_YARN)
    return fail(SAGE_ERR_INVALID_ARG, "scaling must be a sage_rope_scaling value (got %d)", scaling);
  if (scaling != SAGE_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(SAGE_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (scaling == SAGE_ROPE_YARN &&
      (orig_len < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return fail(SAGE_ERR_INVALID_ARG, "SAGE_ROPE_YARN needs orig_len >= 1 and finite beta_fast > beta_slow > 0");
  const int n = rot_dim / 2;
  int axes = 1;
  for (int i = 0; axis && i < n; ++i) {
    if (axis[i] >= SAGE_ROPE_MAX_AXES)
      return fail(SAGE_ERR_INVALID_ARG, "axis[%d] = %d must be below %d", i, axis[i], SAGE_ROPE_MAX_AXES);
    axes = std::max(axes, axis[i] + 1);
  }
  std::memset(plan, 0, sizeof(*plan));
  plan->rot_dim = rot_dim;
  plan->interleaved = interleaved ? 1 : 0;
  plan->n_axes = axes;
  plan->mscale = scaling == SAGE_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  const double kTwoPi = 6.283185307179586476925286766559;
  const double b = scaling == SAGE_ROPE_NTK && rot_dim > 2
                       ? base * std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2))
                       : base;
  for (int i = 0; i < n; ++i) {
    double f = std::pow(b, -2.0 * i / rot_dim);
    if (scaling == SAGE_ROPE_LINEAR) f /= factor;
    if (scaling == SAGE_ROPE_YARN) {
      const double g = std::min(1.0, std::max(0.0, (orig_len * f / kTwoPi - beta_slow) / (beta_fast - beta_slow)));
      f = g * f + (1.0 - g) * f / factor;
    }
    plan->turns[i] = f / kTwoPi;
    plan->axis[i] = axis ? axis[i] : 0;
  }
  return SAGE_OK;
}

sage_status sage_rope(sage_rows q, sage_rows k, int T, int D, int dtype, const int64_t* positions,
                      const sage_rope_plan* plan, int transpose, sage_stream_t stream) {
  if (!plan) return fail(SAGE_ERR_INVALID_ARG, "plan is NULL");
  if (T < 0) return fail(SAGE_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
  if (D < 8 || D > 256 || D % 8 != 0)
    return fail(SAGE_ERR_UNSUPPORTED, "D must be a multiple of 8, 8 .. 256 (got %d)", D);
  if (dtype != SAGE_BF16 && dtype != SAGE_FP16 && dtype != SAGE_FP32)
    return fail(SAGE_ERR_INVALID_ARG, "dtype must be a sage_dtype value (got %d)", dtype);
  if (plan->rot_dim < 2 || plan->rot_dim > D || plan->rot_dim % 2 != 0)
    return fail(SAGE_ERR_INVALID_ARG, "plan->rot_dim must be even, 2 .. D = %d (got %d)", D, plan->rot_dim);
  if (plan->n_axes < 1 || plan->n_axes > SAGE_ROPE_MAX_AXES)
    return fail(SAGE_ERR_INVALID_ARG, "plan->n_axes must be 1 .. %d (got %d)", SAGE_ROPE_MAX_AXES, plan->n_axes);
  for (int i = 0; i < plan->rot_dim / 2; ++i) {
    if (plan->axis[i] >= plan->n_axes)
      return fail(SAGE_ERR_INVALID_ARG, "plan->axis[%d] = %d is not below n_axes = %d", i, plan->axis[i],
                  plan->n_axes);
    if (!std::isfinite(plan->turns[i])) return fail(SAGE_ERR_INVALID_ARG, "plan->turns[%d] is not finite", i);
  }
  sage::RopeParams p;
  bool in_place = true;
  sage_rows* rows[2] = {&q, &k};
  const char* names[2][4] = {{"q.in", "q.out", "q.in_stride", "q.out_stride"},
                             {"k.in", "k.out", "k.in_stride", "k.out_stride"}};
  for (int w = 0; w < 2; ++w) {
    const sage_rows& r = *rows[w];
    if (r.H < 0 || r.H > 65535)
      return fail(SAGE_ERR_INVALID_ARG, "heads must be 0 .. 65535 (got %d)", r.H);
    p.heads[w] = r.H;
    p.in[w] = r.in;
    p.out[w] = r.out;
    p.in_stride[w] = p.out_stride[w] = 0;
    if (r.H == 0) continue;
    sage_status st;
    if ((st = check_stride(r.in_stride, r.H, D, names[w][2], &p.in_stride[w])) != SAGE_OK) return st;
    if ((st = check_stride(r.out_stride, r.H, D, names[w][3], &p.out_stride[w])) != SAGE_OK) return st;
    if (T == 0) continue;
    SAGE_NEED(r.in, names[w][0]);
    SAGE_NEED(r.out, names[w][1]);
    if (r.in == r.out && p.in_stride[w] != p.out_stride[w])
      return fail(SAGE_ERR_INVALID_ARG, "in place, %s and %s must be equal", names[w][2], names[w][3]);
    in_place = in_place && r.in == r.out;
  }
  const int H = q.H + k.H;
  if (T == 0 || H == 0) return SAGE_OK;
  if (!positions) return fail(SAGE_ERR_INVALID_ARG, "positions is NULL");
  if (reinterpret_cast<uintptr_t>(positions) & 7u)
    return fail(SAGE_ERR_ALIGNMENT, "positions is not 8-byte aligned");
  int dev, sms = 0;
  int* err;
  sage_status st;
  if ((st = device_setup(&dev, &err, &sms)) != SAGE_OK) return st;

  p.pos = positions;
  p.T = T;
  p.D = D;
  p.pairs = plan->rot_dim / 2;
  p.mscale = plan->mscale;
  p.sign = transpose ? -1.f : 1.f;
  std::memcpy(p.turns, plan->turns, sizeof(p.turns));
  std::memcpy(p.axis, plan->axis, sizeof(p.axis));
  // Channels per piece: 8, or what the half of an odd rotated part allows.
  const bool half = !plan->interleaved;
  const int V = !half ? 8 : p.pairs % 8 == 0 ? 8 : p.pairs % 4 == 0 ? 4 : 1;
  const int rot_units = half ? p.pairs / V : (2 * p.pairs + V - 1) / V;
  const int rest = half ? (D - plan->rot_dim + 2 * V - 1) / (2 * V) : D / V - rot_units;
  p.units = rot_units + (in_place ? 0 : rest);
  p.unit_shift = std::min(ceil_log2(p.units), 5);
  p.pair_stride = (p.pairs + 3) & ~3;
  const int hstep = sage::kRopeThreads >> p.unit_shift;
  // Few tokens: one per CTA, the heads split over grid.y; many: tokens shared by
  // a CTA so that each thread has work behind the angles.
  int parts = 1;
  p.tokens = 1;
  if (T < 4 * sms) {
    parts = std::min((H + hstep - 1) / hstep, std::max(1, 4 * sms / T));
  } else {
    p.tokens = std::max(1, std::min({16 * hstep / H, T / (4 * sms), 4096 / p.pair_stride}));
  }
  p.head_step = (H + parts - 1) / parts;
  p.by_pairs = sage::FastDiv(static_cast<uint32_t>(p.pairs));
  p.by_heads = sage::FastDiv(static_cast<uint32_t>(p.head_step));
  parts = (H + p.head_step - 1) / p.head_step;
  const dim3 grid((T + p.tokens - 1) / p.tokens, parts);
  const size_t smem = static_cast<size_t>(p.tokens) * p.pair_stride * sizeof(float2);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  with_type(dtype, [&](auto e) {
    using E = decltype(e);
    if (!half) pdl_launch(sage::rope_kernel<E, false, 8>, grid, sage::kRopeThreads, smem, cs, p);
    else if (V == 8) pdl_launch(sage::rope_kernel<E, true, 8>, grid, sage::kRopeThreads, smem, cs, p);
    else if (V == 4) pdl_launch(sage::rope_kernel<E, true, 4>, grid, sage::kRopeThreads, smem, cs, p);
    else pdl_launch(sage::rope_kernel<E, true, 1>, grid, sage::kRopeThreads, smem, cs, p);
  });
  return launch_check("sage_rope launch");
}

sage_status sage_kv_write(const void* k, const void* v, int T, int64_t k_stride, int64_t v_stride, int dtype,
                          const int64_t* slots, sage_kv_cache cache, sage_stream_t stream) {
  sage::KvRowsParams p;
  sage_status st;
  if ((st = kv_rows_args(k, v, T, k_stride, v_stride, dtype, slots, cache, &p)) != SAGE_OK) return st;
  if (T == 0) return SAGE_OK;
  int dev;
  int* err;
  if ((st = device_setup(&dev, &err)) != SAGE_OK) return st;
  p.err = err + 1;
  const int64_t per = sage::kKvThreads / (cache.D / sage::kKvPer) * 2;   // rows per CTA
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) * cache.Hk + per - 1) / per), 2);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  with_type(dtype, [&](auto e) {
    with_flag(cache.D == 128, [&](auto wide) {
      with_flag(cache.format == SAGE_KV_E4M3, [&](auto fp8) {
        pdl_launch(sage::kv_write_kernel<decltype(e), wide.value ? 128 : 64,
                                         fp8.value ? sage::kKvE4m3 : sage::kKvInt8>,
                   grid, sage::kKvThreads, 0, cs, p);
      });
    });
  });
  return launch_check("sage_kv_write launch");
}

sage_status sage_kv_read(sage_kv_cache cache, const int64_t* slots, int T, void* k, void* v, int64_t k_stride,
                         int64_t v_stride, int dtype, sage_stream_t stream) {
  sage::KvRowsParams p;
  sage_status st;
  if ((st = kv_rows_args(k, v, T, k_stride, v_stride, dtype, slots, cache, &p)) != SAGE_OK) return st;
  if (T == 0) return SAGE_OK;
  int dev;
  int* err;
  if ((st = device_setup(&dev, &err)) != SAGE_OK) return st;
  p.err = err + 1;
  const int64_t per = sage::kKvThreads / (cache.D / sage::kKvPer) * 2;   // rows per CTA
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) * cache.Hk + per - 1) / per), 2);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  with_type(dtype, [&](auto e) {
    with_flag(cache.D == 128, [&](auto wide) {
      with_flag(cache.format == SAGE_KV_E4M3, [&](auto fp8) {
        pdl_launch(sage::kv_read_kernel<decltype(e), wide.value ? 128 : 64,
                                        fp8.value ? sage::kKvE4m3 : sage::kKvInt8>,
                   grid, sage::kKvThreads, 0, cs, p);
      });
    });
  });
  return launch_check("sage_kv_read launch");
}

sage_status sage_attn_prompt(const void* q, const void* k, const void* v, const sage_prompt* a, void* out, float* lse,
                             sage_stream_t stream) {
  if (!a) return fail(SAGE_ERR_INVALID_ARG, "p is NULL");
  if (a->n_seq < 0) return fail(SAGE_ERR_INVALID_ARG, "n_seq must be >= 0 (got %d)", a->n_seq);
  sage_status st;
  if ((st = check_heads(a->Hq, a->Hk)) != SAGE_OK) return st;
  if (a->D != 64 && a->D != 128) return fail(SAGE_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", a->D);
  if (a->dtype != SAGE_BF16 && a->dtype != SAGE_FP16)
    return fail(SAGE_ERR_UNSUPPORTED, "dtype must be SAGE_BF16 or SAGE_FP16 (got %d)", a->dtype);
  if ((st = check_scale(a->sm_scale)) != SAGE_OK) return st;
  if (a->n_seq == 0) return SAGE_OK;
  const int32_t* cu_q = a->cu_q;
  const int32_t* cu_k = a->cu_k ? a->cu_k : a->cu_q;
  if ((st = check_cu(cu_q, a->n_seq, "cu_q")) != SAGE_OK) return st;
  if ((st = check_cu(cu_k, a->n_seq, "cu_k")) != SAGE_OK) return st;
  const int64_t Tq = cu_q[a->n_seq], Tk = cu_k[a->n_seq];
  sage::PromptParams p;
  if ((st = check_stride(a->q_stride, a->Hq, a->D, "q_stride", &p.q_stride)) != SAGE_OK) return st;
  if ((st = check_stride(a->k_stride, a->Hk, a->D, "k_stride", &p.k_stride)) != SAGE_OK) return st;
  if ((st = check_stride(a->v_stride, a->Hk, a->D, "v_stride", &p.v_stride)) != SAGE_OK) return st;
  if ((st = check_stride(a->out_stride, a->Hq, a->D, "out_stride", &p.out_stride)) != SAGE_OK) return st;
  if (Tq == 0) return SAGE_OK;
  SAGE_NEED(q, "q");
  SAGE_NEED(out, "out");
  if (Tk > 0) {
    SAGE_NEED(k, "k");
    SAGE_NEED(v, "v");
  }
  if (out == q || (Tk > 0 && (out == k || out == v)))
    return fail(SAGE_ERR_INVALID_ARG, "out must not be q, k or v");
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return fail(SAGE_ERR_ALIGNMENT, "lse is not 4-byte aligned");
  int64_t tiles_all = 0;
  for (int i = 0; i < a->n_seq; ++i) tiles_all += (static_cast<int64_t>(cu_q[i + 1]) - cu_q[i] + 255) / 256;
  if (tiles_all * a->Hq >= (int64_t(1) << 30)) return fail(SAGE_ERR_INVALID_ARG, "too many tiles (Tq * Hq too large)");
  int dev, sms = 0;
  int* err;
  if ((st = device_setup(&dev, &err, &sms)) != SAGE_OK) return st;
  if ((st = attn_setup(dev)) != SAGE_OK) return st;

  CUtensorMap tq, tk, tv;
  if ((st = encode_rows(&tq, q, a->dtype, Tq, a->Hq, a->D, p.q_stride)) != SAGE_OK) return st;
  if (Tk > 0) {
    if ((st = encode_rows(&tk, k, a->dtype, Tk, a->Hk, a->D, p.k_stride)) != SAGE_OK) return st;
    if ((st = encode_rows(&tv, v, a->dtype, Tk, a->Hk, a->D, p.v_stride)) != SAGE_OK) return st;
  } else {
    tk = tv = tq;                                        // not read
  }
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.lse = lse;
  p.lse_stride = Tq;
  p.Hq = a->Hq;
  p.G = a->Hq / a->Hk;
  p.share = tiles_all * a->Hq > sms ? 1 : 0;
  p.causal = a->causal ? 1 : 0;
  p.scale_log2 = scale_log2(a->sm_scale, a->D);
  p.err = err;
  p.timeout_ns = sage_host::wait_timeout_ns();
  const int lanes = p.share ? a->Hk : a->Hq;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  for (int base = 0; base < a->n_seq; base += sage::kPrMaxSeq) {
    const int n = std::min(sage::kPrMaxSeq, a->n_seq - base);
    // Longest first: the CTAs with the most keys start first.
    int order[sage::kPrMaxSeq];
    for (int i = 0; i < n; ++i) order[i] = base + i;
    std::sort(order, order + n, [&](int x, int y) {
      const int lx = cu_k[x + 1] - cu_k[x], ly = cu_k[y + 1] - cu_k[y];
      return lx != ly ? lx > ly : x < y;
    });
    int tiles = 0, m = 0;
    for (int i = 0; i < n; ++i) {
      const int s = order[i];
      const sage::PromptSeq sq = {cu_q[s], cu_k[s], cu_q[s + 1] - cu_q[s], cu_k[s + 1] - cu_k[s]};
      if (sq.lq == 0) continue;
      const int64_t row_tiles = (static_cast<int64_t>(sq.lq) + sage::kPrTile - 1) / sage::kPrTile;
      tiles += static_cast<int>(((p.share ? row_tiles * p.G : row_tiles) + 1) / 2);
      p.seq[m] = sq;
      p.tile_end[m] = tiles;
      ++m;
    }
    if (tiles == 0) continue;
    p.n_seq = m;
    p.sorted = tiles <= sage::kPrMaxOrder ? 1 : 0;
    p.cluster = p.sorted ? prompt_cluster(p, m, lanes, dev) : 1;
    if (p.sorted) {
      uint64_t keys[sage::kPrMaxOrder];
      for (int i = 0, t = 0; i < m; ++i)
        for (int pair = 0; t < p.tile_end[i]; ++t, ++pair) keys[t] = prompt_key(p, i, pair, sage::kPrBoth);
      tiles = p.cluster > 1 ? prompt_alone(p, keys, tiles) : prompt_balance(p, keys, tiles, lanes, sms);
      for (int t = 0; t < tiles; ++t) p.order[t] = static_cast<uint32_t>(keys[t]);
    }
    const dim3 grid(static_cast<unsigned>(tiles * lanes * p.cluster));
    with_flag(a->dtype == SAGE_BF16, [&](auto bf) {
      with_flag(a->D == 128, [&](auto wide) {
        using E = std::conditional_t<bf.value, sage::Bf16T, sage::Fp16T>;
        constexpr int D = wide.value ? 128 : 64;
        with_flag(p.cluster > 1, [&](auto shared) {
          pdl_launch_clusters(sage::prompt_attn_kernel<E, D, shared.value>, p.cluster, grid, sage::kPrThreads,
                              sage::PrSmem<D>::kAlloc, cs, tq, tk, tv, p);
        });
      });
    });
  }
  return launch_check("sage_attn_prompt launch");
}

size_t sage_attn_token_workspace_bytes(int B, int Hq, int Hk, int D, int max_len) {
  if (B < 0 || max_len < 0 || (D != 64 && D != 128) || check_heads(Hq, Hk) != SAGE_OK) return 0;
  return B == 0 ? 0 : token_ws(token_chunks_bound(B, Hk, Hq / Hk, max_len), Hq, D).total;
}

sage_status sage_attn_token(const void* q, const sage_token* a, sage_kv_cache cache, void* out, float* lse,
                            void* workspace, size_t ws_bytes, sage_stream_t stream) {
  if (!a) return fail(SAGE_ERR_INVALID_ARG, "p is NULL");
  sage::KvCacheView c;
  sage_status st;
  if ((st = check_cache(cache, &c)) != SAGE_OK) return st;
  if ((st = check_heads(a->Hq, cache.Hk)) != SAGE_OK) return st;
  if (a->B < 0 || a->B > 65535) return fail(SAGE_ERR_INVALID_ARG, "B must be 0 .. 65535 (got %d)", a->B);
  if (a->dtype != SAGE_BF16 && a->dtype != SAGE_FP16)
    return fail(SAGE_ERR_UNSUPPORTED, "dtype must be SAGE_BF16 or SAGE_FP16 (got %d)", a->dtype);
  if ((st = check_scale(a->sm_scale)) != SAGE_OK) return st;
  sage::TokenParams p;
  if ((st = check_stride(a->q_stride, a->Hq, cache.D, "q_stride", &p.q_stride)) != SAGE_OK) return st;
  if ((st = check_stride(a->out_stride, a->Hq, cache.D, "out_stride", &p.out_stride)) != SAGE_OK) return st;
  if (a->table_stride < 0 || a->max_len < 0 || a->max_len > a->table_stride * cache.page_size)
    return fail(SAGE_ERR_INVALID_ARG, "max_len %d must be 0 .. table_stride * page_size = %lld", a->max_len,
                (long long)(a->table_stride * cache.page_size));
  if (a->max_len > (1 << 30)) return fail(SAGE_ERR_INVALID_ARG, "max_len must be at most 2^30");
  if (a->B == 0) return SAGE_OK;
  SAGE_NEED(q, "q");
  SAGE_NEED(out, "out");
  if (q == out && a->B > 1 && p.q_stride != p.out_stride)
    return fail(SAGE_ERR_INVALID_ARG, "in place, q_stride and out_stride must be equal");
  if (!a->lens) return fail(SAGE_ERR_INVALID_ARG, "lens is NULL");
  if (a->max_len > 0 && !a->page_table) return fail(SAGE_ERR_INVALID_ARG, "page_table is NULL");
  if ((reinterpret_cast<uintptr_t>(a->lens) | reinterpret_cast<uintptr_t>(a->page_table) |
       reinterpret_cast<uintptr_t>(lse)) & 3u)
    return fail(SAGE_ERR_ALIGNMENT, "lens, page_table and lse must be 4-byte aligned");
  const int G = a->Hq / cache.Hk;
  p.per = token_per(a->B, cache.Hk, G, a->max_len);
  p.chunks = token_chunks(a->max_len, p.per);
  const TokenWs ws = token_ws(p.chunks > 1 ? static_cast<int64_t>(a->B) * p.chunks : 0, a->Hq, cache.D);
  if (ws.total > 0) {
    if (!workspace) return fail(SAGE_ERR_WORKSPACE, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
      return fail(SAGE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    if (ws_bytes < ws.total)
      return fail(SAGE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, ws.total);
  }
  const int nt = token_nt(G);
  p.head_blocks = (G + 8 * nt - 1) / (8 * nt);
  const int64_t segs = token_segs(cache.Hk, G), tiles = token_tiles(a->max_len);
  if (segs > 65535 || static_cast<int64_t>(a->B) * a->Hq >= (int64_t(1) << 31) ||
      a->B * segs * tiles >= (int64_t(1) << 31))
    return fail(SAGE_ERR_INVALID_ARG, "too much for one call (B = %d, Hq = %d, max_len = %d)", a->B, a->Hq,
                a->max_len);
  int dev, sms = 0;
  int* err;
  if ((st = device_setup(&dev, &err, &sms)) != SAGE_OK) return st;
  if ((st = attn_setup(dev)) != SAGE_OK) return st;

  p.q = q;
  p.out = out;
  p.lse = lse;
  p.k_codes = c.codes[0];
  p.v_codes = c.codes[1];
  p.k_scale = c.scale[0];
  p.v_scale = c.scale[1];
  p.table = a->page_table;
  p.lens = a->lens;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.chunks > 1 ? p.part_o + ws.part_lse / 4 : nullptr;
  p.segs = static_cast<int>(segs);
  p.table_stride = a->table_stride;
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hk = cache.Hk;
  p.G = G;
  p.pages = cache.num_pages;
  p.page_shift = c.page_shift;
  p.max_len = a->max_len;
  p.scale_log2 = scale_log2(a->sm_scale, cache.D);
  p.err = err + 1;
  const dim3 grid(p.chunks, p.segs, a->B);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  with_flag(a->dtype == SAGE_BF16, [&](auto bf) {
    with_flag(cache.D == 128, [&](auto wide) {
      with_flag(nt == 2, [&](auto two) {
        using E = std::conditional_t<bf.value, sage::Bf16T, sage::Fp16T>;
        constexpr int D = wide.value ? 128 : 64, NT = two.value ? 2 : 1;
        with_flag(cache.format == SAGE_KV_E4M3, [&](auto fp8) {
          constexpr int kFmt = fp8.value ? sage::kKvE4m3 : sage::kKvInt8;
          pdl_launch(sage::token_attn_kernel<E, D, NT, kFmt>, grid, sage::kTokThreads, sage::kTokSmem<D, NT>, cs, p);
        });
        if (p.chunks > 1) {
          // Few rows have many parts each: four warps to a row.
          const int64_t rows = static_cast<int64_t>(a->B) * a->Hq;
          with_flag(rows <= 4 * sms, [&](auto few) {
            constexpr int kWarps = few.value ? 4 : 1, kPer = sage::kJoinThreads / 32 / kWarps;
            pdl_launch(sage::token_join_kernel<E, D, kWarps>, dim3(static_cast<unsigned>((rows + kPer - 1) / kPer)),
                       sage::kJoinThreads, 0, cs, p);
          });
        }
      });
    });
  });
  return launch_check("sage_attn_token launch");
}

}  // extern "C"

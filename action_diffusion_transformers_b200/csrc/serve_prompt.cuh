// serve_prompt.cuh - softmax attention over packed prompts on sm_100a tensor
// cores, 16-bit operands:
//   O_i = sum_{j visible} 2^(x_ij - m_i) v_j / sum_j 2^(x_ij - m_i),
//   x_ij = (q_i . k_j) * sm_scale * log2 e,
// key j of a sequence visible to its query i when j <= i + Lk - Lq (causal,
// aligned at the end) or always; grouped heads; sequences packed row after
// row, their bounds given by the host.
//
// One CTA takes two tiles of 128 query rows, A and B, that share a KV head.  The
// (row tile, query head) items of a (sequence, KV head) are paired in order,
// heads running fastest, so that both tiles see about the same keys; where that
// would leave SMs idle (no more CTAs than SMs with a CTA per two row tiles of one
// head) the row tiles of one head are paired instead: 144 against 96 CTAs for
// eight captions x 16 heads, 8.8 against 10.0 us.
//
// An item alone (a pair without its second, or one that the host parts because its
// end would stand out) gives its key tiles to A and B in turn, each with a ring of
// its own, and the two results are joined at the end: 1024 tokens x 24 heads 25.7
// to 19.4 us (16.5 since), chunks of 32 to 1504 tokens behind up to 3000 earlier ones
// x 24 heads 112.5 to 98 in short runs (104 in a long one).  (K of A and B loaded before V of either, 3 slots each: in the
// order K, V of A, K, V of B with 2 slots, A's products held up B's next K; 128
// queries over 8192 keys took 41 instead of 31 us.)
// Where the items are few, each is given to a cluster of 2 to 8 CTAs, its key
// tiles dealt out among all their tiles A and B, and the CTAs' results are joined
// through distributed shared memory in a fixed order (kCluster): 128 queries over
// 8192 keys x 16 heads 119 to 27 us, x 4 heads 20, one head of 6000 tokens 88 to 37.
// (The join is the softmax warps' own: behind a point that all warps share, the
// compiler keeps to the 56 registers of the others, and the chunk took 30 us.)
//
// 384 threads:
//   warps 0-3, 4-7  softmax of tile A, of tile B: thread r owns query row r
//                   (TMEM lane r), reads its 128 scores, writes P back as
//                   16-bit pairs over the first 64 score columns, 64 keys at a
//                   time, rescales its row of O when the reference m moves, and
//                   stores the row.
//   warps 8, 9      MMA of tile A, of tile B: S = Q K^T (shared x shared),
//                   O += P V (P in TMEM).
//   warp 10         TMA loads: Q once, K and V tiles of 128 keys into a ring.
// TMEM (512 columns): S_A, S_B at 0, 128; O_A, O_B at 256, 384 (D = 128: P lies
// over the first half of S) or 256, 320 with P_A, P_B at 384, 448 (D = 64).
// While tile A's softmax runs, the tensor core works on tile B and the other
// way round.  D = 128: S_X(j+1) overwrites the columns that PV_X(j) reads P
// from, so it is issued only after PV_X(j) has completed, and a softmax thread
// that sees S_X(j) knows that O_X holds every product up to j - 1.  D = 64:
// S_X(j+1) is issued as soon as the softmax has read S_X(j), and P_X(j) is
// written once PV_X(j-1) has completed.
//
// The reference m of a row moves only when a score passes the last one it was set by
// by 2^8, so O is rescaled rarely.  P is rounded to the operands' 16-bit type (half a
// step: bf16 2^-8 relative, fp16 2^-11, each weight on its own): the tensor core
// multiplies equal types.  In fp16 the reference lies 2^7 below the score that set it:
// P stays below 2^15 (65504 is the type's end), and the type's fixed step under 2^-14
// costs 2^-32 of such a weight at most, so a long tail of small weights is not lost
// (65535 keys of e^-18 each, a thousandth together, came out as 0 without it).  The
// row sum adds the weights before that rounding; sums, references and O stay in 32
// bits.
//
// Values in masked places: a masked score is replaced, never added to, so K may
// hold anything there.  A masked weight is 0, but 0 times an infinity or a NaN
// in a masked V row (a later token, another sequence's row in the same tile)
// would spread to the row's output; a row whose output is not finite, with a sum
// that is, is therefore looked at again (prompt_rows_again): a NaN or an infinity
// among its visible values stays, what came from masked ones goes.  (A sum that is
// not finite comes from the row's own scores.)
//
// A visible score that is a NaN or +inf, or visible scores that are all -inf, leave
// a row without a softmax: its output and its log-sum-exp are NaN.  The weights
// bring the first two into the row's sum (2^NaN, 2^(inf - inf)), which stays a NaN.
//
// Bound by a row tile's chain (scores, softmax, weights, products) with two tiles
// per SM: 8192 tokens x 32 heads, D = 128, take 529 to 542 us in short runs (1014 to
// 1040 TFLOP/s) and 577 to 593 in long ones under the power cap (927 to 952), the
// tensor pipe 44% and the special-function unit 45% busy; D = 64 390 to 430 us, the
// special-function unit 59%.  Every key visible: 8192 tokens x 16 heads 555 us (991
// TFLOP/s), 4096 x 16 155.
//
// Every wait on a load or a product is bounded (see mbar_wait_bounded), as in
// sage_attn.cuh.  The barriers of the softmax warps, of the CTA and of a cluster have
// no limit of their own: every warp reaches them, after a wait that ran out too, and
// what lies between two of them ends by itself.
#pragma once
#include "serve_rows.cuh"
#include "serve_token.cuh"

namespace sage {

constexpr int kPrTile = 128;
constexpr int kPrThreads = 384;          // 2 x 4 softmax warps, two for MMA, one for loads, one idle
constexpr int kPrWarpMma = 8, kPrWarpLoad = 10;
constexpr int kPrMaxSeq = 256;          // sequences per launch
constexpr int kPrMaxCluster = 8;         // CTAs that share an item at most
constexpr int kPrMaxOrder = 512;        // pairs up to which the host sorts them
constexpr float kPrRaise = 8.f;          // log2: a row's reference moves for a score this far above the last
template <class E>
constexpr float kPrLift = std::is_same<E, Fp16T>::value ? 7.f : 0.f;   // log2: largest weight as the reference moves

template <int D>
struct PrSmem {
  static constexpr int kTileBytes = kPrTile * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kBarSlots = D == 128 ? 6 : 8;          // barriers of slots (see kHalf)
  static constexpr int kQ = 0;                                // A, B
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kBar = kRing + kSlots * kTileBytes;
  static constexpr bool kApart = D == 64;                     // P has TMEM columns of its own
  static constexpr int kColO = 256, kStepO = D, kColP = kApart ? 384 : 0, kStepP = kApart ? 64 : 128;
  // q[2], s_full[2], pv_done[2], p_full[2][2], s_read[2], full[], empty[], drain[2]
  static constexpr int kQFull = 0, kSFull = 2, kPVDone = 4, kPFull = 6, kSRead = 10, kFull = 12,
                       kEmpty = kFull + kBarSlots, kDrain = kEmpty + kBarSlots, kNumBars = kDrain + 2;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kAgain = kMisc + 16;                   // rows to be looked at again, a bit each: 4 words per tile
  static constexpr int kTotal = kAgain + 32;
  static constexpr int kAlloc = kTotal + 1024;
  // An item alone: each of the two tiles has a ring of its own, of kHalf slots
  // (D = 128: Q_B's place is one of them).  At the end of a tile's ring, once it
  // is read, the sums and references of its rows; for a cluster, those of the CTA
  // at the end of B's, and its O from the start of A's.
  static constexpr int kHalf = D == 128 ? 3 : 4;
  static constexpr int kRing2 = kRing + (kSlots - 2 * kHalf) * kTileBytes, kRing2Bytes = kHalf * kTileBytes;
  static constexpr int kStat = kRing2Bytes - 4096, kStatCta = 2 * kRing2Bytes - 2048;
  static constexpr int kPartStride = D + 4;                   // floats from row to row of a CTA's O
  static_assert(kRing2 >= kQ + kTileBytes && kPrTile * kPartStride * 4 <= kStat, "");
};
static_assert(PrSmem<128>::kAlloc <= 232448 && PrSmem<64>::kAlloc <= 232448, "shared memory of one CTA");

// What a CTA takes of a pair of items: both, or one alone, whose key tiles then
// go to the two tiles in turn (see the kernel).
enum PromptWhich : uint32_t { kPrBoth = 0, kPrFirst = 1, kPrSecond = 2 };

struct PromptSeq {
  int q0, k0, lq, lk;       // first rows and lengths
};

struct PromptParams {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;               // [Hq, Tq] or null
  int64_t q_stride, k_stride, v_stride, out_stride;
  int64_t lse_stride;       // Tq
  int Hq, G, n_seq, causal;
  int cluster;              // CTAs that share an item alone, by key tiles: 1 .. kPrMaxCluster
  int share;                // 1: items are paired over the heads of a KV head, 0: over the rows of a head
  float scale_log2;
  int* err;
  int64_t timeout_ns;
  PromptSeq seq[kPrMaxSeq];
  int tile_end[kPrMaxSeq];  // pairs (per KV head, or per head) up to and including a sequence
  int sorted;               // 1: order[] holds the pairs, most key tiles first
  uint32_t order[kPrMaxOrder];   // sequence << 24 | which << 20 | pair (see PromptWhich)
};

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of an operand whose rows (128-byte swizzled, 8-row groups of 1024
// bytes) run along the product's K axis and whose 64-element row pieces lie
// `piece` bytes apart (V: keys are rows, channels are contiguous).
__device__ __forceinline__ uint64_t make_sdesc_mn(uint32_t saddr, uint32_t piece) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((piece & 0x3FFFFu) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// The weights of 64 keys, added up and written in 16-bit pairs to 32 TMEM
// columns.  All of them come from the special-function unit (2^-22 relative): a
// share of two pairs in 16 on the FMA pipe (n + f, 2^f by a polynomial of about that
// accuracy) took 549 to 557 us on 8192 tokens x 32 heads, D = 128, and 420 at D = 64,
// against 541 to 549 and 392 to 405; with a cubic the 32-bit log-sum-exp was off by
// 5e-5.
template <class E>
__device__ __forceinline__ void pr_weights(const uint32_t (&s0)[32], const uint32_t (&s1)[32], f32x2_t sl2,
                                           f32x2_t nref2, uint32_t col, f32x2_t (&sum)[4]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t(&s)[32] = c == 0 ? s0 : s1;
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const f32x2_t t = x2_fma(x2_pack(s[2 * i], s[2 * i + 1]), sl2, nref2);
      const float w0 = ex2_approx(x2_lo(t)), w1 = ex2_approx(x2_hi(t));
      sum[i & 3] = x2_add(sum[i & 3], x2_pack(__float_as_uint(w0), __float_as_uint(w1)));
      pk[i] = E::pack(w0, w1);
    }
    tmem_st16(col + 16 * c, pk);
  }
}

// A softmax warp stays whole in front of its warp-wide TMEM accesses.
__device__ __forceinline__ bool pr_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int64_t tmo) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, tmo));
}

// All warps of the CTA, each whole: from different places in the code, which
// __syncthreads() would not promise.
__device__ __forceinline__ void pr_meet() { asm volatile("bar.sync 0, %0;" ::"n"(kPrThreads) : "memory"); }
// All threads of all CTAs of the cluster, each warp whole.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
  return d;
}
__device__ __forceinline__ float2 peer_ld2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Where a CTA of a cluster leaves its sums and references, and its O.
template <int D>
__device__ __forceinline__ float2* prompt_stat(uint8_t* smem) {
  return reinterpret_cast<float2*>(smem + PrSmem<D>::kRing2 + PrSmem<D>::kStatCta);
}
template <int D>
__device__ __forceinline__ float* prompt_part(uint8_t* smem) {
  return reinterpret_cast<float*>(smem + PrSmem<D>::kRing2);
}

// Row r of tile x is to be looked at again.  What that takes goes where the tile's Q
// was (its products are done), so that no register holds it until then.
struct PromptMark {
  float2 stat[kPrTile];        // reference and 1 / sum of the rows concerned
  PromptSeq seq;
  int row0, head, c0, c1;      // first row of the tile, channels
};
template <int D>
__device__ __forceinline__ PromptMark* prompt_marks(uint8_t* smem, int x) {
  return reinterpret_cast<PromptMark*>(smem + PrSmem<D>::kQ + x * PrSmem<D>::kTileBytes);
}
template <int D>
__device__ __forceinline__ uint32_t* prompt_marked(uint8_t* smem) {
  return reinterpret_cast<uint32_t*>(smem + PrSmem<D>::kAgain);
}
template <int D>
__device__ __forceinline__ void prompt_mark(uint8_t* smem, int x, int r, float m, float rl, const PromptSeq& sq, int row0,
                                            int head, int c0, int c1) {
  PromptMark* mark = prompt_marks<D>(smem, x);
  mark->stat[r] = make_float2(m, rl);
  mark->seq = sq;
  mark->row0 = row0;
  mark->head = head;
  mark->c0 = c0;
  mark->c1 = c1;
  atomicOr(prompt_marked<D>(smem) + 4 * x + r / 32, 1u << (r & 31));
}

// Rows whose stored output is not finite in some of the channels c0 .. c1 - 1 though
// their sum is, by a whole warp: those of the bits of `todo`, in order (each sees no
// fewer keys than the one before).  A NaN or an infinity in a visible row of V
// decides its channel, whatever the weights (all above 0): V is added up, 2^-40 of
// each value, until nothing can change any more, once for all rows of the warp.  Where
// that sum is finite, what spoilt the channel was masked, and the weights are formed
// again, four rows at a time, in 32 bits, a key per lane, and already divided by the
// row's sum (so that finite values near the type's end add up).
// The softmax warps' last act, behind the point where all warps have met: nobody waits
// for them any more, and nothing is held in registers for it before (called where the
// rows are stored, it made 8192 tokens x 32 heads 562 us instead of 535).  2048 tokens
// x 8 heads, clean 38 us: one NaN token in front 76, an infinity in every seventh 120,
// a NaN in the last token, whose row tile is formed again, 2700.
template <class E, int D>
__device__ __forceinline__ void prompt_rows_again(const PromptParams& p, const PromptMark& mark, uint32_t todo) {
  using S = typename E::S;
  constexpr int kBatch = 16, kRows = 4;
  const int lane = threadIdx.x & 31, r0 = threadIdx.x & (kPrTile - 32);
  const PromptSeq sq = mark.seq;
  const int c0 = mark.c0, c1 = mark.c1, head = mark.head, row0 = mark.row0;
  const int pieces = (c1 - c0) / 8, step = 32 / pieces;      // lanes of a row of V, rows that a warp reads at once
  const int sub = lane / pieces, c = c0 + (lane - sub * pieces) * 8;
  const int64_t hk = static_cast<int64_t>(head / p.G) * D, hq = static_cast<int64_t>(head) * D;
  const S* v = static_cast<const S*>(p.v) + sq.k0 * p.v_stride + hk + c;
  const S* k = static_cast<const S*>(p.k) + sq.k0 * p.k_stride + hk;
  const S* q = static_cast<const S*>(p.q) + sq.q0 * p.q_stride + hq;
  S* out = static_cast<S*>(p.out) + sq.q0 * p.out_stride + hq + c;
  float seen[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // of the keys before `at` that this lane reads
  int at = 0;
  auto finite = [](float x) { return fabsf(x) < __int_as_float(0x7F800000); };
  auto bits = [](const float(&x)[8], auto is) {              // a bit per channel
    uint32_t b = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) b |= static_cast<uint32_t>(is(x[e])) << e;
    return b;
  };
  while (todo) {
    // Up to kRows rows whose weights are wanted: the channels concerned, and the row's
    // place, keys, reference and 1 / sum.
    uint32_t want[kRows];
    int r[kRows], vis[kRows], most = 0, n = 0;
    float ref[kRows], part[kRows];
#pragma unroll
    for (int g = 0; g < kRows; ++g) want[g] = r[g] = vis[g] = 0, ref[g] = part[g] = 0.f;
    while (todo && n < kRows) {
      const int src = __ffs(todo) - 1;
      const int ri = row0 + r0 + src, vi = p.causal ? min(sq.lk, max(0, ri + 1 + sq.lk - sq.lq)) : sq.lk;
      todo &= todo - 1;
      Piece<E, 8> got;
      float x[8], all[8];
      got.load(out + ri * p.out_stride);
      got.get(x);
      const uint32_t lost = bits(x, [&](float y) { return !finite(y); });
      while (at < vi) {
        uint32_t done = bits(seen, [](float y) { return y != y; });
        for (int s = pieces; s < 32; s <<= 1) done |= __shfl_xor_sync(0xFFFFFFFFu, done, s);
        if (!__any_sync(0xFFFFFFFFu, lost & ~done)) break;
        Piece<E, 8> a[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int j = at + i * step + sub;
          a[i] = Piece<E, 8>{};
          if (j < vi) a[i].load(v + j * p.v_stride);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          float y[8];
          a[i].get(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) seen[e] = fmaf(y[e], 0x1p-40f, seen[e]);
        }
        at = min(vi, at + kBatch * step);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        all[e] = seen[e];
        for (int s = pieces; s < 32; s <<= 1) all[e] += __shfl_xor_sync(0xFFFFFFFFu, all[e], s);
      }
      const uint32_t own = lost & bits(all, [&](float y) { return !finite(y); });
      if (sub == 0 && own) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (own >> e & 1) x[e] = all[e];
        got.put(x);
        got.store(out + ri * p.out_stride);
      }
      if (__any_sync(0xFFFFFFFFu, lost & ~own)) {
        const float2 st = mark.stat[r0 + src];
        most = vi;
#pragma unroll
        for (int g = 0; g < kRows; ++g)
          if (g == n) want[g] = lost & ~own, r[g] = ri, vis[g] = vi, ref[g] = st.x, part[g] = st.y;
        ++n;
      }
    }
    if (n == 0) break;
    float o[kRows][8];
#pragma unroll
    for (int g = 0; g < kRows; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) o[g][e] = 0.f;
    for (int j0 = 0; j0 < most; j0 += 32) {
      float w[kRows];
      const S* kj = k + min(j0 + lane, most - 1) * p.k_stride;
#pragma unroll
      for (int g = 0; g < kRows; ++g) w[g] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 8) {
        Piece<E, 8> b;
        float y[8];
        b.load(kj + d);
        b.get(y);
#pragma unroll
        for (int g = 0; g < kRows; ++g) {
          Piece<E, 8> a;
          float x[8];
          a.load(q + r[g] * p.q_stride + d);
          a.get(x);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[g] = fmaf(x[e], y[e], w[g]);
        }
      }
#pragma unroll
      for (int g = 0; g < kRows; ++g)
        w[g] = j0 + lane < vis[g] ? ex2_approx(fmaf(w[g], p.scale_log2, -ref[g])) * part[g] : 0.f;
#pragma unroll 4
      for (int i = 0; i < pieces; ++i) {
        const int j = i * step + sub;
        Piece<E, 8> b;
        float y[8];
        b.load(v + min(j0 + j, most - 1) * p.v_stride);
        b.get(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = finite(y[e]) ? y[e] : 0.f;    // masked, or in a channel that is decided
#pragma unroll
        for (int g = 0; g < kRows; ++g) {
          const float wj = __shfl_sync(0xFFFFFFFFu, w[g], j);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[g][e] = fmaf(wj, y[e], o[g][e]);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      for (int s = pieces; s < 32; s <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[g][e] += __shfl_xor_sync(0xFFFFFFFFu, o[g][e], s);
      if (sub == 0 && want[g]) {
        Piece<E, 8> got;
        float x[8];
        got.load(out + r[g] * p.out_stride);
        got.get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (want[g] >> e & 1) x[e] = o[g][e];
        got.put(x);
        got.store(out + r[g] * p.out_stride);
      }
    }
  }
}

// O = sum_c 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c over the CTAs c of the cluster,
// in their order; each CTA takes a share of the rows, a thread 8 channels.  For the
// softmax warps: the others have given their registers away.
template <class E, int D>
__device__ __forceinline__ void prompt_join(const PromptParams& p, const PromptSeq& sq, uint8_t* smem, int rank, int row0,
                                            int head, int off) {
  using S = typename E::S;
  constexpr int kPieces = D / 8;
  const float kNegInf = -__int_as_float(0x7F800000);
  const int share = (kPrTile + p.cluster - 1) / p.cluster;
  for (int i = threadIdx.x; i < share * kPieces; i += 32 * kPrWarpMma) {
    const int r = rank * share + i / kPieces, d = (i % kPieces) * 8, row = row0 + r;
    if (r >= kPrTile || row >= sq.lq) continue;
    const int visible = p.causal ? min(sq.lk, max(0, row + off + 1)) : sq.lk;
    const uint32_t stat = smem_u32(prompt_stat<D>(smem) + r);
    const uint32_t part = smem_u32(prompt_part<D>(smem) + r * PrSmem<D>::kPartStride + d);
    float m = kNegInf, l = 0.f;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float2 st[kPrMaxCluster];
#pragma unroll
    for (int c = 0; c < kPrMaxCluster; ++c) st[c] = c < p.cluster ? peer_ld2(peer_addr(stat, c)) : make_float2(kNegInf, 0.f);
#pragma unroll
    for (int c = 0; c < kPrMaxCluster; ++c) m = fmaxf(m, st[c].x);
#pragma unroll
    for (int c0 = 0; c0 < kPrMaxCluster; c0 += 4) {
      float4 part4[4][2];                                // four peers' pieces under way
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c0 + c < p.cluster) {
          const uint32_t at = peer_addr(part, c0 + c);
          part4[c][0] = peer_ld4(at);
          part4[c][1] = peer_ld4(at + 16);
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c0 + c < p.cluster) {
          const float w = st[c0 + c].x == kNegInf ? 0.f : ex2_approx(st[c0 + c].x - m);
          const float4 a = part4[c][0], b = part4[c][1];
          const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          l = fmaf(st[c0 + c].y, w, l);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = fmaf(f[k], w, o[k]);
        }
      }
    }
    if (visible > 0 && m == kNegInf) l = __int_as_float(0x7FFFFFFF);
    const float rl = visible > 0 ? __fdiv_rn(1.f, l) : 0.f;
    bool finite = true;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      finite = finite && fabsf(o[k]) < __int_as_float(0x7F800000);
      o[k] *= rl;
    }
    Piece<E, 8> pc;
    pc.put(o);
    pc.store(static_cast<S*>(p.out) + static_cast<int64_t>(sq.q0 + row) * p.out_stride +
             static_cast<int64_t>(head) * D + d);
    if (!finite && fabsf(l) < __int_as_float(0x7F800000)) prompt_mark<D>(smem, 0, r, m, rl, sq, row0, head, 0, D);
    if (p.lse && d == 0)
      p.lse[head * p.lse_stride + sq.q0 + row] = visible > 0 ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
  }
}

// The launch gives each of the 384 threads 168 registers; the last four warps
// hand most of theirs to the softmax warps: 2 x 224 + 56 = 3 x 168.
constexpr int kPrRegsSoftmax = 224, kPrRegsOther = 56;
static_assert(2 * kPrRegsSoftmax + kPrRegsOther <= 3 * 168, "register split");
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <class E, int D, bool kCluster>
__global__ void __launch_bounds__(kPrThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PromptParams p) {
  using L = PrSmem<D>;
  using S = typename E::S;
  constexpr int kSlots = L::kSlots, kHalf = L::kHalf;
  constexpr bool kBf16 = std::is_same<E, Bf16T>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t tmo = p.timeout_ns;

  // CTA -> (pair of items, KV head or head): heads run fastest, and the pairs
  // with the most key tiles come first: sorted by the host, or, where they are
  // many, the sequences by length and each from its end to its start.
  const int lanes = p.share ? p.Hq / p.G : p.Hq;
  const int cluster = kCluster ? p.cluster : 1;
  const int cta = blockIdx.x / cluster, rank = blockIdx.x - cta * cluster;
  const int tile = cta / lanes;
  const int hb = cta - tile * lanes;
  int lo = 0, pair;
  uint32_t which = kPrBoth;
  if (p.sorted) {
    lo = p.order[tile] >> 24;
    which = (p.order[tile] >> 20) & 3;
    pair = p.order[tile] & 0xFFFFF;
  } else {
    int hi = p.n_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tile < p.tile_end[mid]) hi = mid;
      else lo = mid + 1;
    }
    pair = p.tile_end[lo] - 1 - tile;
  }
  const PromptSeq sq = p.seq[lo];
  const int off = sq.lk - sq.lq;
  const int hk = p.share ? hb : hb / p.G;
  // First row and head of the two tiles, and the key tiles that the last row of
  // each sees.
  const int first = 2 * pair + (which == kPrSecond ? 1 : 0);
  const bool alone =
      which != kPrBoth || (p.share ? (first + 1) / p.G : first + 1) * static_cast<int64_t>(kPrTile) >= sq.lq;
  int rows[2], heads[2], nt[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int i = alone ? first : first + x;
    const int rt = p.share ? i / p.G : i;
    heads[x] = p.share ? hb * p.G + (i - rt * p.G) : hb;
    rows[x] = rt * kPrTile;
    const int last = min(rows[x] + kPrTile, sq.lq) - 1;
    const int seen = p.causal ? min(sq.lk, last + off + 1) : sq.lk;
    nt[x] = seen > 0 ? (seen + kPrTile - 1) / kPrTile : 0;
  }
  int n = max(nt[0], nt[1]);                              // key tiles that this CTA loads
  // An item alone: its key tiles go round the tiles A and B of its CTAs, each with
  // half of the ring, and the results are joined at the end.
  const int stride = 2 * cluster;
  const bool split = kCluster || (alone && n > 1);
  if (split) {
    const int all = n;
    for (int x = 0; x < 2; ++x) nt[x] = max(0, (all - 2 * rank - x + stride - 1) / stride);
    n = nt[0] + nt[1];
  } else if (alone) {
    nt[1] = 0;
    rows[1] = sq.lq;                                    // no rows
  }

  const int ring = split ? L::kRing2 : L::kRing;

  if (warp == kPrWarpMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < L::kNumBars; ++i)
      // P, S read: one arrival per softmax warp; a ring slot is empty when all tiles that read it have
      mbar_init(&bars[i], i >= L::kPFull && i < L::kFull ? 4 : i >= L::kEmpty && i < L::kDrain && !split ? 2 : 1);
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) prompt_marked<D>(smem)[i] = 0;
    fence_mbar_init();
  }
  if (tid == 32 * kPrWarpLoad) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Up to here nothing of the caller's was read: the set-up above may run beside
  // the kernel before.  (On an SM of its own: this CTA's 384 x 168 registers leave
  // room for no other that wants TMEM, so none of that kernel's can wait for the
  // columns held here while this CTA waits for it.)
  pdl_enter();

  if (warp >= kPrWarpMma) {
   regs_dec<kPrRegsOther>();
   if (warp == kPrWarpLoad) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && n > 0) {
      auto load = [&](uint8_t* dst, const CUtensorMap* tm, int head, int row, uint64_t* bar) {
        mbar_arrive_expect_tx(bar, L::kTileBytes);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * kPrTile * 128, tm, c * 64, head, row, bar);
      };
      uint32_t issued = 0, parity = 0;                  // bit per slot: loaded, parity of its last load
      for (int it = 0; it < 2 * n; ++it) {
        // Split: K of A and B, V of A and B, ... (the last round may be A's alone).
        const bool one = split && (it >> 2) >= nt[1];
        const int x = !split || one ? 0 : it & 1, kv = !split || one ? it & 1 : (it >> 1) & 1;
        const int own = split ? (it >> 2) * 2 + kv : it;
        const int slot = split ? x * kHalf + own % kHalf : own % kSlots;
        const uint32_t use = static_cast<uint32_t>(split ? own / kHalf : own / kSlots);
        if (it == 0 && nt[0] > 0) load(smem + L::kQ, &tm_q, heads[0], sq.q0 + rows[0], &bars[L::kQFull]);
        if (use > 0 && !mbar_wait_bounded(&bars[L::kEmpty + slot], (use - 1) & 1, abort_flag, tmo)) break;
        const int j = split ? (it >> 2) * stride + 2 * rank + x : it >> 1;
        load(smem + ring + slot * L::kTileBytes, kv ? &tm_v : &tm_k, hk, sq.k0 + j * kPrTile,
             &bars[L::kFull + slot]);
        issued |= 1u << slot;
        parity = (parity & ~(1u << slot)) | (use & 1) << slot;
        if (it == 0 && nt[1] > 0 && !split)
          load(smem + L::kQ + L::kTileBytes, &tm_q, heads[1], sq.q0 + rows[1], &bars[L::kQFull + 1]);
      }
      if (*abort_flag) {
        // Wait (bounded) for the loads in flight: Q and the last one of each slot.
        const int64_t drain = 200000000;
        int none = 0;
        volatile int* nf = reinterpret_cast<volatile int*>(&none);
        if (nt[0] > 0) mbar_wait_bounded(&bars[L::kQFull], 0, nf, drain);
        if (nt[1] > 0 && !split) mbar_wait_bounded(&bars[L::kQFull + 1], 0, nf, drain);
        for (int slot = 0; slot < L::kBarSlots; ++slot)
          if (issued >> slot & 1) mbar_wait_bounded(&bars[L::kFull + slot], parity >> slot & 1, nf, drain);
      }
    }
   } else if (warp < kPrWarpLoad) {
    // ------------------------------------------------------------ MMA of tile A, of tile B
    const int x = warp - kPrWarpMma;
    const int ntx = x ? nt[1] : nt[0];
    const int steps = split ? ntx : n;                // key tiles whose slots this tile gives back
    if (lane == 0 && steps > 0) {
      const int qx = split ? 0 : x;
      constexpr uint32_t kFmt = kBf16 ? 1u : 0u;
      constexpr uint32_t kIdescQK = make_idesc(1u, kFmt, 128u, 128u);
      constexpr uint32_t kIdescPV = make_idesc(1u, kFmt, 128u, static_cast<uint32_t>(D)) | (1u << 16);
      auto wait = [&](int bar, int phase) {
        return mbar_wait_bounded(&bars[bar], static_cast<uint32_t>(phase) & 1, abort_flag, tmo);
      };
      auto slot_of = [&](int it) { return split ? x * kHalf + it % kHalf : it % kSlots; };
      auto wait_full = [&](int it) { return wait(L::kFull + slot_of(it), split ? it / kHalf : it / kSlots); };
      auto scores = [&](int j) {                  // S_x(j) = Q_x K_j^T
        const uint64_t qd = make_sdesc(smem_u32(smem + L::kQ + qx * L::kTileBytes), 1024u, 2u);
        const uint64_t kd = make_sdesc(smem_u32(smem + ring + slot_of(2 * j) * L::kTileBytes), 1024u, 2u);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t step = (kk & 3) * 2 + (kk >> 2) * (kPrTile * 128 / 16);
          mma_f16_ss(tmem + x * 128, qd + step, kd + step, kIdescQK, kk > 0 ? 1u : 0u);
        }
        tc_commit(&bars[L::kSFull + x]);
      };
      auto products = [&](int j) {                // O_x += P_x(j) V_j, as its halves come in
        const uint64_t vd =
            make_sdesc_mn(smem_u32(smem + ring + slot_of(2 * j + 1) * L::kTileBytes), kPrTile * 128);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait(L::kPFull + 2 * x + half, j)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = half * 4; kk < half * 4 + 4; ++kk)
            mma_f16_ts(tmem + L::kColO + x * L::kStepO, tmem + L::kColP + x * L::kStepP + kk * 8,
                       vd + kk * (16 * 128 / 16), kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
        }
        tc_commit(&bars[L::kPVDone + x]);
        return true;
      };
      // A commit arrives when all that this thread issued before has completed
      // (at once for a tile without work), so each slot is given back by both.
      bool ok = wait_full(0) && (ntx == 0 || wait(L::kQFull + qx, 0));
      if (ok && ntx > 0) {
        tc_fence_after();
        scores(0);
      }
      if (ok) tc_commit(&bars[L::kEmpty + slot_of(0)]);
      for (int j = 0; ok && j < steps; ++j) {
        if constexpr (L::kApart) {
          if (j + 1 < steps) {
            if (!(ok = wait_full(2 * j + 2) && (j + 1 >= ntx || wait(L::kSRead + x, j)))) break;
            if (j + 1 < ntx) {
              tc_fence_after();
              scores(j + 1);
            }
            tc_commit(&bars[L::kEmpty + slot_of(2 * j + 2)]);
          }
          if (!(ok = wait_full(2 * j + 1) && (j >= ntx || products(j)))) break;
          tc_commit(&bars[L::kEmpty + slot_of(2 * j + 1)]);
        } else {
          // What is on the way from P_x(j) to S_x(j+1) is kept short: K_j+1 is
          // waited for before, V_j given back after (a wait on a completed barrier
          // takes about 120 cycles, a commit behind products up to 300).
          if (!(ok = (j + 1 >= steps || wait_full(2 * j + 2)) && wait_full(2 * j + 1) && (j >= ntx || products(j)))) break;
          if (j + 1 < ntx) {
            // S_x(j+1) takes the columns that hold P_x(j): wait for its products.
            if (!(ok = wait(L::kPVDone + x, j))) break;
            tc_fence_after();
            scores(j + 1);
          }
          tc_commit(&bars[L::kEmpty + slot_of(2 * j + 1)]);
          if (j + 1 < steps) tc_commit(&bars[L::kEmpty + slot_of(2 * j + 2)]);
        }
      }
      tc_commit(&bars[L::kDrain + x]);
      int none = 0;
      mbar_wait_bounded(&bars[L::kDrain + x], 0, reinterpret_cast<volatile int*>(&none), 200000000);
    }
   }
   if constexpr (kCluster) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
   }
   __syncwarp();
   tc_fence_before();
   pr_meet();
   if (warp == kPrWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
   }
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<kPrRegsSoftmax>();
    const int x = warp >> 2;                       // tile A, B
    const int r = tid & 127;
    const int row = (x ? rows[1] : rows[0]) + r;   // of the sequence
    const int head = x ? heads[1] : heads[0];
    const int ntx = x ? nt[1] : nt[0];
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + x * 128 + lane_base;
    const uint32_t to = tmem + L::kColO + x * L::kStepO + lane_base;
    const uint32_t tp = tmem + L::kColP + x * L::kStepP + lane_base;
    const float kNegInf = -__int_as_float(0x7F800000);
    const float sl = p.scale_log2;
    const int visible = p.causal ? min(sq.lk, max(0, row + off + 1)) : sq.lk;
    float m = kNegInf;                             // reference, log2 units
    float l = 0.f;
    bool ok = true;
    for (int j = 0; j < ntx; ++j) {
      if (!(ok = pr_wait(&bars[L::kSFull + x], static_cast<uint32_t>(j) & 1, abort_flag, tmo))) break;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s[c]);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) reg_fence(s[c]);
      if constexpr (L::kApart) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kSRead + x]);
      }
      const int valid = visible - (split ? j * stride + 2 * rank + x : j) * kPrTile;
      const bool masked = __any_sync(0xFFFFFFFFu, valid < kPrTile);
      if (masked) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= valid) s[c][i] = __float_as_uint(kNegInf);
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int i = 1; i < 31; i += 2)
          mx[c] = fmax3(mx[c], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
        mx[c] = fmaxf(mx[c], __uint_as_float(s[c][31]));
      }
      const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
      if (L::kApart && j > 0) {      // P and O: the products of tile j - 1 are done
        if (!(ok = pr_wait(&bars[L::kPVDone + x], static_cast<uint32_t>(j - 1) & 1, abort_flag, tmo))) break;
        tc_fence_after();
      }
      if (__any_sync(0xFFFFFFFFu, tmax > m + (kPrLift<E> + kPrRaise))) {
        const float m1 = fmaxf(m, tmax - kPrLift<E>);
        const float alpha = m == kNegInf ? 0.f : ex2_approx(m - m1);
        l *= alpha;
        m = m1;
        if (j > 0) {
          const f32x2_t a2 = x2_splat(alpha);
#pragma unroll 1
          for (int cb = 0; cb < D; cb += 32) {
            f32x2_t o[16];
            tmem_ld32_pairs(to + cb, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = x2_mul(o[i], a2);
            tmem_st32_pairs(to + cb, o);
          }
        }
      }
      const f32x2_t sl2 = x2_splat(sl), nref2 = x2_splat(m == kNegInf ? 0.f : -m);
      f32x2_t sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        pr_weights<E>(s[2 * half], s[2 * half + 1], sl2, nref2, tp + 32 * half, sum);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kPFull + 2 * x + half]);
      }
      const f32x2_t sum2 = x2_add(x2_add(sum[0], sum[1]), x2_add(sum[2], sum[3]));
      l += x2_lo(sum2) + x2_hi(sum2);
    }
    const bool mine = row < sq.lq;                 // also false for a tile without an item
    S* dst = static_cast<S*>(p.out) + static_cast<int64_t>(sq.q0 + row) * p.out_stride + static_cast<int64_t>(head) * D;
    if (split || ntx > 0) {
      if (ok && ntx > 0) ok = pr_wait(&bars[L::kPVDone + x], static_cast<uint32_t>(ntx - 1) & 1, abort_flag, tmo);
      int cb0 = 0, cb1 = D;                              // channels that this thread stores
      float wa = 1.f, wb = 0.f;                          // split: weights of O_A, O_B
      if (split) {
        // O = (2^(m_A - m) O_A + 2^(m_B - m) O_B) / l, l alike, m the larger of the
        // two: thread r of tile A takes the first half of the channels of row r, of
        // tile B the second; both reach that TMEM lane.  Every softmax warp comes
        // here, after a wait that ran out too.
        float2* stat = reinterpret_cast<float2*>(smem + L::kRing2 + L::kStat);
        stat[x * (L::kRing2Bytes / 8) + r] = make_float2(m, l);
        tc_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float2 a = stat[r], b = stat[L::kRing2Bytes / 8 + r];
        m = fmaxf(a.x, b.x);
        wa = a.x == kNegInf ? 0.f : ex2_approx(a.x - m);
        wb = b.x == kNegInf ? 0.f : ex2_approx(b.x - m);
        l = fmaf(a.y, wa, b.y * wb);
        cb0 = x * (D / 2);
        cb1 = cb0 + D / 2;
      }
      if (kCluster && ok) {
        // For the join of the cluster: sum, reference and O of this CTA's keys to
        // shared memory (the ring is read: both tiles' products are done).
        tc_fence_after();
        if (x == 0) prompt_stat<D>(smem)[r] = make_float2(m, l);
        float* o = prompt_part<D>(smem) + r * L::kPartStride;
#pragma unroll 1
        for (int cb = cb0; cb < cb1; cb += 16) {
          float f[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = 0.f;
          for (int y = 0; y < 2; ++y) {
            if (nt[y] > 0) {                             // or O was never written
              uint32_t t[16];
              tmem_ld16(tmem + L::kColO + y * L::kStepO + lane_base + cb, t);
              tmem_wait_ld();
              reg_fence16(t);
              const float w = y ? wb : wa;
#pragma unroll
              for (int i = 0; i < 16; ++i) f[i] = fmaf(__uint_as_float(t[i]), w, f[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(o + cb + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
        }
      } else if (ok) {
        tc_fence_after();
        // No visible key: nothing was added, the row is zeros.  No score above -inf:
        // no softmax.
        if (visible > 0 && m == kNegInf) l = __int_as_float(0x7FFFFFFF);
        const float rl = visible > 0 ? __fdiv_rn(1.f, l) : 0.f;
        bool finite = true;
        const uint32_t toa = split ? tmem + L::kColO + lane_base : to;
#pragma unroll 1
        for (int cb = cb0; cb < cb1; cb += 32) {
          uint32_t o[32];
          tmem_ld32(toa + cb, o);
          tmem_wait_ld();
          reg_fence(o);
          if (split) {
            uint32_t ob[32];
            tmem_ld32(toa + L::kStepO + cb, ob);
            tmem_wait_ld();
            reg_fence(ob);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(fmaf(__uint_as_float(o[i]), wa, __uint_as_float(ob[i]) * wb));
          }
          if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float f[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float v = __uint_as_float(o[8 * i + k]);
                finite = finite && fabsf(v) < __int_as_float(0x7F800000);
                f[k] = v * rl;
              }
              Piece<E, 8> pc;
              pc.put(f);
              pc.store(dst + cb + 8 * i);
            }
          }
        }
        if (mine && p.lse && (!split || x == 0))
          p.lse[head * p.lse_stride + sq.q0 + row] = visible > 0 ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
        if (mine && !finite && fabsf(l) < __int_as_float(0x7F800000)) prompt_mark<D>(smem, x, r, m, rl, sq, row - r, head, cb0, cb1);
      }
    } else if (mine) {
      Piece<E, 8> z;
#pragma unroll
      for (int i = 0; i < 4; ++i) z.w[i] = 0;
      for (int d = 0; d < D; d += 8) z.store(dst + d);
      if (p.lse) p.lse[head * p.lse_stride + sq.q0 + row] = kNegInf;
    }
    if constexpr (kCluster) {
      // Every warp of the cluster meets twice, after a wait that ran out too: the
      // CTAs' parts are written, and nobody leaves while they are read.
      __syncwarp();
      cluster_sync();
      prompt_join<E, D>(p, sq, smem, rank, rows[0], heads[0], off);
      __syncwarp();
      cluster_sync();
    }
    __syncwarp();
    tc_fence_before();
    pr_meet();
    if (*abort_flag && tid == 0) atomicExch(p.err, 1);
    const uint32_t todo = prompt_marked<D>(smem)[warp];
    if (todo) prompt_rows_again<E, D>(p, *prompt_marks<D>(smem, x), todo);
  }
}

}  // namespace sage

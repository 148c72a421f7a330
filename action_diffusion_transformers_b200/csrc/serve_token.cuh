// serve_token.cuh - attention of one new token per sequence over the quantized
// paged KV cache:
//   x_j = (q . k_j) * sm_scale * log2 e,  O = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
// for the keys j < len of its sequence, with grouped heads (G = Hq / Hk query
// heads share a KV head).
//
// Bound by HBM: every code is read once and used by the G query heads of its
// KV head.  The products run on mma.sync (m16n8k16, f16 operands, f32 sums):
// a query token gives at most G rows, far below a tcgen05 tile, and the codes
// have to pass through registers to become f16 anyway.  Both products take the
// codes as the 16-row operand and the heads as the 8 columns:
//   S^T [16 keys x 8 heads] = K [16 x D] Q^T,   O^T [D x 8] += V^T [D x 16] P^T.
// Which channel or key a lane's fragment element stands for is free as long as
// both operands agree, so each lane takes contiguous pieces of a row:
//   K: lane (g, t) holds keys g, g + 8, channels 16 t .. + 15 of each 64;
//   V: lane (g, t) holds keys 2t, 2t+1, 2t+8, 2t+9, channels g D/8 .. + D/8 - 1.
// P^T's fragment is S^T's transposed 8 x 8 blocks (movmatrix).
// A warp copies its tiles (cp.async, 512 bytes in a row per instruction) into a
// queue of its own in shared memory, one tile ahead, the 16-byte pieces of a row
// in an order that keeps the fragment reads free of bank conflicts.  (Copies of
// each lane's own pieces, 8 rows x 64 bytes per instruction, stayed at 4.9 TB/s
// even without the products; a plain read reaches 6.8.)
//
// Codes are exact in f16 (INT8 and E4M3 both).  q is scaled by a power of two
// per head so that its largest channel lies in [1, 2) and rounded to f16:
// channels above 2^-14 of the largest keep every bit, the others are off by at
// most 2^-25 of it.  P carries the V scale of its key and a power of two per
// head, set by the first weight above 0, that keeps the largest one met so far
// near 1.  Its rounding to f16 is 2^-11 relative, and for weights below 2^-14 of the
// largest 2^-25 of that one: 2^-16 of it over the up to 512 keys that a warp adds
// (16 tiles of a chunk; each warp has a power of its own).  That rounding is
// far below a bf16 output's own (2^-8), but equal to an fp16 output's: there P goes
// in as two f16 parts (kFine), what the first leaves out being the second, which
// takes the error against 64 bits from 1.4 times that of the output's rounding to
// 1.0 times, for 3 to 9% of the time (64 sequences of 300 to 8192 keys 103.1 to 106.5
// us; INT8 codes 110.4 to 120.6).  Sums, row maxima and the output stay in 32 bits.
//
// 64 sequences of 300 to 8192 keys x 8 KV heads (D = 128, E4M3, 583 MB) take 98 to
// 113 us with the join, by the lengths and places of their pages, 5.2 to 5.9 TB/s; ALU
// 52% and issue 51% busy with turning codes into f16.  16 query heads to a KV head
// (NT = 2, 168 registers and up to 64 bytes of spills) take 138 us where 4 take 103:
// twice the softmax and products, the tensor pipe 29%; 32, which read every code once
// per 16, 244.  One sequence of 3999 keys takes 8.5 us, two launches' latency.
//
// A CTA takes one chunk of keys of one segment (a sequence and a KV head with up
// to 8 * NT of its query heads); its warps take 32-key tiles in turn and are
// joined through shared memory; chunks are joined by token_join_kernel in a
// fixed order (no atomics).
#pragma once
#include "serve_rows.cuh"

namespace sage {

constexpr int kTokWarps = 4;
constexpr int kTokThreads = kTokWarps * 32;
constexpr int kTokTile = 32;              // keys per tile: two products of 16
constexpr int kTokStages = 2;             // tiles in a warp's queue
constexpr int kTokPerSm = 3;              // resident CTAs: the queues take 68 KB each at D = 128
constexpr float kTokRaise = 8.f;          // the row max moves only when a score passes it by this (log2)
constexpr float kTokMaxW = 2048.f;        // largest P before its power of two is renewed
// Exponents of that power of two: the largest stands for "no weight above 0 yet", and
// the first such weight passes kTokMaxW by it (or lies below 2^-107, where the V scales
// that the cache write gives end).
constexpr int kTokMaxCf = 118, kTokMinCf = -126;

struct TokenParams {
  const void* q;           // [B, Hq, D], q_stride elements per sequence
  void* out;               // [B, Hq, D], out_stride
  float* lse;              // [B, Hq] or null
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;    // [B, table_stride] pages of each sequence
  const int32_t* lens;     // [B]
  float* part_o;           // [B * Hq, chunks, D] chunk results (chunks > 1)
  float* part_lse;         // [B * Hq, chunks], log2 units
  int64_t q_stride, out_stride, table_stride;
  int B, Hq, Hk, G, pages, page_shift;
  int max_len;             // keys that the table can name
  int per;                 // tiles of a chunk
  int chunks;              // chunks that the longest sequence can have
  int head_blocks;         // blocks of 8 * NT query heads per KV head
  int segs;                // Hk * head_blocks: segments of a sequence
  float scale_log2;        // sm_scale * log2 e
  int* err;
};

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four code bytes -> two f16 pairs (bytes 0, 1 and bytes 2, 3), exactly.
template <int kFmt>
__device__ __forceinline__ void codes_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  if constexpr (kFmt == kKvE4m3) {
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
  } else {
    // 0x64xx is 1024 + xx in f16; xx = code + 128
    const uint32_t b = c ^ 0x80808080u;
    const uint32_t x = __byte_perm(b, 0x64646464u, 0x4140), y = __byte_perm(b, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(0x64806480u));
  }
}

template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A warp's queue.  A stage holds a tile: for each of its two 16-key halves the K
// rows and the V rows, then the K and the V scale of each key.
template <int D>
struct TokQueue {
  static constexpr int kRow = D / 16;                    // 16-byte pieces of a row
  static constexpr int kV = 16 * D, kHalf = 2 * kV;
  static constexpr int kScales = 2 * kHalf, kStage = kScales + 2 * 32 * 4;
  static constexpr int kWarp = kTokStages * kStage, kAll = kTokWarps * kWarp;
  // Place of piece c of row r: the pieces that eight lanes read at once lie in
  // different banks.
  static __device__ __forceinline__ int k_at(int r, int c) { return r * D + (D == 128 ? c ^ ((r & 1) << 2) : c) * 16; }
  static __device__ __forceinline__ int v_at(int r, int c) {
    return r * D + (D == 128 ? c ^ (r & 6) : c ^ ((r >> 1) & 3)) * 16;
  }
};

// Page table entries of the two halves of a tile at `key` of its sequence, as
// read; -1 from key `end` on.  They are looked at only when the tile's copies
// start, a tile later, so that the read is not waited for.
struct TokPages {
  int page[2];
};
__device__ __forceinline__ TokPages tok_pages(const TokenParams& p, const int32_t* table, int key, int end) {
  TokPages r;
#pragma unroll
  for (int h = 0; h < 2; ++h)      // 16-key halves start at multiples of 16, pages hold a multiple of 16 slots
    r.page[h] = key + 16 * h < end ? table[(key + 16 * h) >> p.page_shift] : -1;
  return r;
}
__device__ __forceinline__ void tok_cut(TokPages& r, int key, int end) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (key + 16 * h >= end) r.page[h] = -1;
}

// Starts the copies of the tile at `key` into a stage (one group per tile, empty
// where there is nothing to copy); returns which halves have a page.
template <int D>
__device__ __forceinline__ int tok_issue(uint32_t stage, const TokenParams& p, const TokPages& pages, int key, int end,
                                         int hk, int lane) {
  using Q = TokQueue<D>;
  int have = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (pages.page[h] >= 0 && pages.page[h] < p.pages) {
      have |= 1 << h;
      const int64_t row = ((static_cast<int64_t>(pages.page[h]) * p.Hk + hk) << p.page_shift) +
                          ((key + 16 * h) & ((1 << p.page_shift) - 1));
      const uint32_t dst = stage + h * Q::kHalf;
#pragma unroll
      for (int i = 0; i < Q::kRow / 2; ++i) {
        const int r = (32 * i + lane) / Q::kRow, c = lane % Q::kRow;
        cp_async<16>(dst + Q::k_at(r, c), p.k_codes + (row + r) * D + c * 16);
        cp_async<16>(dst + Q::kV + Q::v_at(r, c), p.v_codes + (row + r) * D + c * 16);
      }
      // lanes 0-15: the K scales of the half, lanes 16-31: its V scales
      cp_async<4>(stage + Q::kScales + ((lane >> 4) * 32 + h * 16 + (lane & 15)) * 4,
                  (lane < 16 ? p.k_scale : p.v_scale) + row + (lane & 15));
    } else if (key + 16 * h < end) {
      atomicExch(p.err, 1);
    }
  }
  cp_async_commit();
  return have;
}

// Running state of the lane's heads 2t, 2t + 1 of each block of 8.
template <int D, int NT>
struct TokState {
  float m[NT][2];            // reference of the exponent, log2 (-inf: nothing seen)
  float l[NT][2];            // sum of 2^(x - m) over this lane's keys
  float w[NT][2];            // largest weight p * vs met, as of the last renewal
  float cf[NT][2];           // power of two on the weights (2^kTokMaxCf: none above 0 yet)
  float o[NT][D / 16][4];
};

// n: keys of the tile that exist; have: bit h is set where the page of half h
// does.  What lies in the other places may be anything: none of it takes part.
template <int D, int NT, int kFmt, bool kFine>
__device__ __forceinline__ void tok_step(const uint8_t* stage, int n, int have, const uint32_t (&q)[NT][D / 16][2],
                                         const float (&qf)[NT][2], TokState<D, NT>& st, int lane) {
  using Q = TokQueue<D>;
  const float kNegInf = -__int_as_float(0x7F800000);
  const int g = lane >> 2, t = lane & 3;
  const bool all = n >= kTokTile && have == 3;          // the same in every lane
  uint32_t a[4];
  float s[NT][2][4];
#pragma unroll
  for (int b = 0; b < NT; ++b)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[b][i >> 2][i & 3] = 0.f;
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    uint32_t k[2][2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 x = *reinterpret_cast<const uint4*>(stage + h * Q::kHalf + Q::k_at(g + 8 * r, 4 * j + t));
        k[h][r][0] = x.x;
        k[h][r][1] = x.y;
        k[h][r][2] = x.z;
        k[h][r][3] = x.w;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        codes_f16<kFmt>(k[h][0][i], a[0], a[2]);
        codes_f16<kFmt>(k[h][1][i], a[1], a[3]);
#pragma unroll
        for (int b = 0; b < NT; ++b) mma_f16_16816(s[b][h], a, q[b][4 * j + i][0], q[b][4 * j + i][1]);
      }
  }
  // Keys 16 h + g and 16 h + g + 8: their scales, and whether they are there.
  float ks[2][2], vs[2][2];
  bool in[2][2];
  const float* sc = reinterpret_cast<const float*>(stage + Q::kScales) + g;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ks[h][r] = sc[16 * h + 8 * r];
      vs[h][r] = sc[32 + 16 * h + 8 * r];
      in[h][r] = all || (16 * h + 8 * r + g < n && ((have >> h) & 1));
      if (!in[h][r]) vs[h][r] = 0.f;
    }
  uint32_t pb[NT][2][2], pl[NT][2][2];         // P in f16; kFine: what that rounding left out, in f16
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    // s[b][h]: (key g, heads 2t, 2t+1), (key g + 8, the same heads)
    float e[2][4], w[2][4];
    bool raise = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[b][h][i] = in[h][i >> 1] ? s[b][h][i] * ks[h][i >> 1] * qf[b][i & 1] : kNegInf;
        raise = raise || s[b][h][i] > st.m[b][i & 1] + kTokRaise;
      }
    auto weights = [&]() {
      float big = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = st.m[b][i & 1];
          e[h][i] = ex2_approx(s[b][h][i] - (m == kNegInf ? 0.f : m));
          w[h][i] = in[h][i >> 1] ? e[h][i] * vs[h][i >> 1] * st.cf[b][i & 1] : 0.f;
          big = fmaxf(big, w[h][i]);
        }
      return big;
    };
    raise = __any_sync(0xFFFFFFFFu, raise);
    if (!raise) raise = __any_sync(0xFFFFFFFFu, weights() > kTokMaxW);
    if (raise) {
      // Renew the reference, and the power of two on the weights, of each head.
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = fmaxf(fmaxf(s[b][0][c], s[b][0][c + 2]), fmaxf(s[b][1][c], s[b][1][c + 2]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const float m0 = st.m[b][c], m1 = fmaxf(m0, mx);
        const float ref = m1 == kNegInf ? 0.f : m1;
        const float alpha = m0 == kNegInf ? 0.f : ex2_approx(m0 - ref);
        float wm = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) wm = fmaxf(wm, ex2_approx(s[b][h][c + 2 * r] - ref) * vs[h][r]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) wm = fmaxf(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, o));
        wm = fmaxf(wm, st.w[b][c] * alpha);
        const int ex = min(max(127 - static_cast<int>(__float_as_uint(wm) >> 23), kTokMinCf), kTokMaxCf);
        const float cf = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
        // cf is a power of two, so dividing by it is exact; the quotient is below
        // 2 / alpha, as wm is at least w * alpha
        const float f = alpha == 0.f ? 0.f : alpha * (cf * (1.f / st.cf[b][c]));
        st.m[b][c] = m1;
        st.w[b][c] = wm;
        st.cf[b][c] = cf;
        st.l[b][c] *= alpha;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.o[b][i][c] *= f;
          st.o[b][i][c + 2] *= f;
        }
      }
      weights();
    }
    st.l[b][0] += (e[0][0] + e[0][2]) + (e[1][0] + e[1][2]);
    st.l[b][1] += (e[0][1] + e[0][3]) + (e[1][1] + e[1][3]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t pk = f16x2_pack(w[h][2 * r], w[h][2 * r + 1]);
        pb[b][h][r] = movmatrix_trans(pk);
        if constexpr (kFine)
          pl[b][h][r] = movmatrix_trans(f16x2_pack(w[h][2 * r] - Fp16T::lo(pk), w[h][2 * r + 1] - Fp16T::hi(pk)));
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 2 * t + (i & 1) + 8 * (i >> 1);
      const uint8_t* src = stage + h * Q::kHalf + Q::kV +
                           (D == 128 ? Q::v_at(r, g) : Q::v_at(r, g >> 1) + (g & 1) * 8);
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(src);
        v[i][0] = x.x;
        v[i][1] = x.y;
        v[i][2] = x.z;
        v[i][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(src);
        v[i][0] = x.x;
        v[i][1] = x.y;
      }
    }
    if (!all) {
      // Keys 16 h + 2t, 2t + 1, 2t + 8, 2t + 9: a code that is not there may be a NaN.
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * h + 2 * t + (i & 1) + 8 * (i >> 1) >= n || !((have >> h) & 1)) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k) v[i][k] = 0;
        }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      // word i of the four keys: channels 4i .. 4i+3 of the lane's D/8
      const uint32_t lo01 = __byte_perm(v[0][i], v[1][i], 0x5140), hi01 = __byte_perm(v[0][i], v[1][i], 0x7362);
      const uint32_t lo23 = __byte_perm(v[2][i], v[3][i], 0x5140), hi23 = __byte_perm(v[2][i], v[3][i], 0x7362);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        codes_f16<kFmt>(c ? hi01 : lo01, a[0], a[1]);
        codes_f16<kFmt>(c ? hi23 : lo23, a[2], a[3]);
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          mma_f16_16816(st.o[b][2 * i + c], a, pb[b][h][0], pb[b][h][1]);
          if constexpr (kFine) mma_f16_16816(st.o[b][2 * i + c], a, pl[b][h][0], pl[b][h][1]);
        }
      }
    }
  }
}

template <int D, int NT>
constexpr int kTokSmem = TokQueue<D>::kAll > kTokWarps * 8 * NT * (D + 4) * 4 ? TokQueue<D>::kAll
                                                                             : kTokWarps * 8 * NT * (D + 4) * 4;

// Tiles of a sequence.
__device__ __forceinline__ int tok_tiles(const TokenParams& p, int b) {
  const int len = min(max(p.lens[b], 0), p.max_len);
  return (len + kTokTile - 1) / kTokTile;
}

// E: type of q and out.  NT: blocks of 8 query heads per warp.
template <class E, int D, int NT, int kFmt>
__global__ void __launch_bounds__(kTokThreads, kTokPerSm) token_attn_kernel(const __grid_constant__ TokenParams p) {
  pdl_enter();
  using S = typename E::S;
  using Q = TokQueue<D>;
  __shared__ float s_m[kTokWarps][8 * NT], s_l[kTokWarps][8 * NT], s_u[kTokWarps][8 * NT];
  // The warps' queues; after the last tile the same bytes join the warps' O.
  extern __shared__ __align__(16) uint8_t tok_smem[];
  float(*s_o)[8 * NT][D + 4] = reinterpret_cast<float(*)[8 * NT][D + 4]>(tok_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const float kNegInf = -__int_as_float(0x7F800000);
  const uint8_t* queue = tok_smem + warp * Q::kWarp;
  const uint32_t qaddr = smem_u32(queue);

  const int b = blockIdx.z, seg = blockIdx.y;
  const int hk = seg / p.head_blocks;
  const int h0 = (seg - hk * p.head_blocks) * 8 * NT;             // first head of the KV head's
  const int nh = min(8 * NT, p.G - h0);
  const int32_t* table = p.table + b * p.table_stride;
  const int tile0 = blockIdx.x * p.per;
  {
    // The length, the pages of the warp's first two tiles and its part of Q are
    // read side by side; pages behind the chunk's keys are dropped once it is there.
    int tile = tile0 + warp;
    const int all = p.lens[b];
    TokPages pg = tok_pages(p, table, tile * kTokTile, warp < p.per ? p.max_len : 0);
    TokPages next = tok_pages(p, table, (tile + kTokWarps) * kTokTile, warp + kTokWarps < p.per ? p.max_len : 0);
    Piece<E, 8> raw[NT][D / 32];
#pragma unroll
    for (int blk = 0; blk < NT; ++blk)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) raw[blk][i].w[k] = 0;
        if (blk * 8 + g < nh)
          raw[blk][i].load(static_cast<const S*>(p.q) + b * p.q_stride +
                           static_cast<int64_t>(hk * p.G + h0 + blk * 8 + g) * D + 64 * (i >> 1) + 16 * t + 8 * (i & 1));
      }
    if (tid == 0 && blockIdx.x == 0 && seg == 0 && all > p.max_len) atomicExch(p.err, 1);
    const int len = min(max(all, 0), p.max_len);
    const int tiles = (len + kTokTile - 1) / kTokTile, tile1 = min(tiles, tile0 + p.per);
    if (tile0 >= tiles && (p.chunks > 1 || blockIdx.x > 0)) return;
    const int end = min(len, tile1 * kTokTile);                   // of the chunk's keys
    tok_cut(pg, tile * kTokTile, end);
    tok_cut(next, (tile + kTokWarps) * kTokTile, end);
    int have = tok_issue<D>(qaddr, p, pg, tile * kTokTile, end, hk, lane);

    // Q fragments (heads g of each block of 8) and the factor of the scores.
    uint32_t q[NT][D / 16][2];
    float qf[NT][2];
#pragma unroll
    for (int blk = 0; blk < NT; ++blk) {
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) bits = max(bits, piece_amax_bits(raw[blk][i]));
      bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 1));
      bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 2));
      // 2^-ex, ex the exponent of the largest channel (no scaling of zeros and non-finite rows)
      int ex = static_cast<int>(bits >> 23) - 127;
      if (ex == 128 || bits == 0) ex = 0;
      ex = max(ex, -126);
      const float dn = __uint_as_float(static_cast<uint32_t>(127 - min(ex, 126)) << 23);
      // An infinity or a NaN in q: every score is one of the two, so the head has no
      // softmax (all scores -inf would pass for a sequence without keys).
      const float up = bits < 0x7F800000u ? __uint_as_float(static_cast<uint32_t>(127 + ex) << 23)
                                          : __uint_as_float(0x7FFFFFFFu);
      const float rest = ex == 127 ? 0.5f : 1.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float f[8];
        raw[blk][i].get(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= dn * rest;
        q[blk][2 * i][0] = f16x2_pack(f[0], f[1]);
        q[blk][2 * i][1] = f16x2_pack(f[2], f[3]);
        q[blk][2 * i + 1][0] = f16x2_pack(f[4], f[5]);
        q[blk][2 * i + 1][1] = f16x2_pack(f[6], f[7]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) qf[blk][k] = __shfl_sync(0xFFFFFFFFu, up, (2 * t + k) * 4) * p.scale_log2;
    }

    TokState<D, NT> st;
#pragma unroll
    for (int blk = 0; blk < NT; ++blk) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        st.m[blk][k] = kNegInf;
        st.l[blk][k] = 0.f;
        st.w[blk][k] = 0.f;
        st.cf[blk][k] = __uint_as_float(static_cast<uint32_t>(127 + kTokMaxCf) << 23);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) st.o[blk][i][k] = 0.f;
    }
    static_assert(kTokStages == 2, "the loop keeps one tile ahead");
    for (int stage = 0; tile < tile1; tile += kTokWarps, stage ^= 1) {
      const int then = tok_issue<D>(qaddr + (stage ^ 1) * Q::kStage, p, next, (tile + kTokWarps) * kTokTile, end, hk,
                                     lane);
      next = tok_pages(p, table, (tile + 2 * kTokWarps) * kTokTile, end);
      cp_async_wait<1>();
      __syncwarp();        // the other lanes' copies too
      if (have)
        tok_step<D, NT, kFmt, std::is_same<E, Fp16T>::value>(queue + stage * Q::kStage, len - tile * kTokTile, have, q, qf, st, lane);
      have = then;
      __syncwarp();        // the stage is free
    }
    __syncthreads();       // every warp has left its queue

    // Join the warps.
#pragma unroll
    for (int blk = 0; blk < NT; ++blk) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = blk * 8 + 2 * t + k;
        float l = st.l[blk][k];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (g == 0) {
          s_m[warp][h] = st.m[blk][k];
          s_l[warp][h] = l;
          s_u[warp][h] = 1.f / st.cf[blk][k];           // exact: a power of two
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(&s_o[warp][h][g * (D / 8) + 2 * i]) =
              make_float2(st.o[blk][i][k], st.o[blk][i][k + 2]);
      }
    }
    __syncthreads();
    constexpr int kPer = D / 4;                          // lanes of 4 channels per head
    for (int i = tid; i < nh * kPer; i += kTokThreads) {
      const int h = i / kPer, d = (i % kPer) * 4;
      float m = s_m[0][h];
#pragma unroll
      for (int w = 1; w < kTokWarps; ++w) m = fmaxf(m, s_m[w][h]);
      const float ref = m == kNegInf ? 0.f : m;
      float l = 0.f, f[kTokWarps];
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kTokWarps; ++w) {
        f[w] = ex2_approx(s_m[w][h] - ref);
        l += f[w] * s_l[w][h];
      }
      const float r = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
      const float lse2 = l == 0.f ? kNegInf : m + log2f(l);
      // Divided by the sum before the weights' power of two goes: values near the end
      // of bf16 would pass that of binary32 otherwise.
#pragma unroll
      for (int w = 0; w < kTokWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(&s_o[w][h][d]);
        const float fr = f[w] * r, up = s_u[w][h];
        o.x += fr * v.x * up;
        o.y += fr * v.y * up;
        o.z += fr * v.z * up;
        o.w += fr * v.w * up;
      }
      const int head = hk * p.G + h0 + h;
      const int64_t at = static_cast<int64_t>(b) * p.Hq + head;
      if (p.chunks == 1) {
        Piece<E, 4> v;
        const float out[4] = {o.x, o.y, o.z, o.w};
        v.put(out);
        v.store(static_cast<S*>(p.out) + b * p.out_stride + static_cast<int64_t>(head) * D + d);
        if (d == 0 && p.lse) p.lse[at] = lse2 * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (at * p.chunks + blockIdx.x) * D + d) = o;
        if (d == 0) p.part_lse[at * p.chunks + blockIdx.x] = lse2;
      }
    }
  }
}

// Joins the chunks of one (sequence, query head), and writes the rows of empty
// sequences: kWarps warps per row, weights 2^(lse - max - 20), each warp its chunks in
// order, then the warps in order.  (2^-20: the sum over the chunks, at most 2^19, of
// values near the end of bf16 stays within binary32.)
constexpr int kJoinThreads = 128;
template <class E, int D, int kWarps>
__global__ void __launch_bounds__(kJoinThreads) token_join_kernel(const __grid_constant__ TokenParams p) {
  pdl_enter();
  constexpr int V = D / 32;
  __shared__ float s_o[kWarps][D];
  __shared__ float s_l[kWarps];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32 / kWarps) + (threadIdx.x >> 5) / kWarps;
  if (row >= static_cast<int64_t>(p.B) * p.Hq) return;
  const int lane = threadIdx.x & 31, way = (threadIdx.x >> 5) % kWarps;
  const int b = static_cast<int>(row / p.Hq), head = static_cast<int>(row - static_cast<int64_t>(b) * p.Hq);
  const int parts = (tok_tiles(p, b) + p.per - 1) / p.per;
  const float kNegInf = -__int_as_float(0x7F800000);
  const float* lse = p.part_lse + row * p.chunks;
  const float* part = p.part_o + row * p.chunks * D + lane * V;
  float m = kNegInf;
  for (int i = lane; i < parts; i += 32) m = fmaxf(m, lse[i]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  m += 20.f;
  const float ref = m == kNegInf ? 0.f : m;
  float l = 0.f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
#pragma unroll 8
  for (int i = way; i < parts; i += kWarps) {
    const float f = ex2_approx(lse[i] - ref);
    l += f;
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] += f * part[static_cast<int64_t>(i) * D + k];
  }
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int k = 0; k < V; ++k) s_o[way][lane * V + k] = o[k];
    if (lane == 0) s_l[way] = l;
    __syncthreads();
    if (way > 0) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      l += s_l[w];
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] += s_o[w][lane * V + k];
    }
  }
  const float r = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] *= r;
  Piece<E, V> v;
  v.put(o);
  v.store(static_cast<typename E::S*>(p.out) + b * p.out_stride + static_cast<int64_t>(head) * D + lane * V);
  if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace sage

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
// Fragments come straight from global memory, without shared memory: which
// channel or key a lane's fragment element stands for is free as long as both
// operands agree, so each lane reads contiguous pieces of a row:
//   K: lane (g, t) holds keys g, g + 8, channels t D/4 .. + D/4 - 1;
//   V: lane (g, t) holds keys 2t, 2t+1, 2t+8, 2t+9, channels g D/8 .. + D/8 - 1.
// P^T's fragment is S^T's transposed 8 x 8 blocks (movmatrix).
//
// Codes are exact in f16 (INT8 and E4M3 both).  q is scaled by a power of two
// per head so that its largest channel lies in [1, 2) and rounded to f16:
// channels above 2^-14 of the largest keep every bit, the others are off by at
// most 2^-25 of it.  P carries the V scale of its key and a power of two per
// head that keeps the largest weight met so far near 1, so its rounding to f16
// (2^-11 relative) is never an underflow of weights that matter.  Sums, row
// maxima and the output stay in 32 bits.
//
// A CTA takes one chunk of keys of one (sequence, KV head); its warps take
// 16-key tiles in turn and are joined through shared memory; chunks are joined
// by token_join_kernel in a fixed order (no atomics).
#pragma once
#include "serve_rows.cuh"

namespace sage {

constexpr int kTokWarps = 4;
constexpr int kTokThreads = kTokWarps * 32;
constexpr int kTokTile = 16;              // keys per tile
constexpr int kTokMaxChunk = 1024;        // keys per CTA
constexpr float kTokRaise = 8.f;          // the row max moves only when a score passes it by this (log2)
constexpr float kTokMaxW = 2048.f;        // largest P before its power of two is renewed

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
  int chunk, chunks;       // keys per CTA (a multiple of 64), CTAs per (sequence, KV head)
  int head_blocks;         // blocks of 8 * NT query heads per KV head
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

// One warp's 16 keys in registers.
template <int D>
struct TokTile {
  uint32_t k[2][D / 16];     // keys g, g + 8: D/4 bytes
  uint32_t v[4][D / 32];     // keys 2t, 2t+1, 2t+8, 2t+9: D/8 bytes
  float ks[2], vs[2];        // scales of keys g, g + 8
  int n;                     // valid keys of the tile (0: none, nothing was read)
};

template <int kWords>
__device__ __forceinline__ void ld_words(uint32_t (&w)[kWords], const uint8_t* p) {
  if constexpr (kWords == 2) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "l"(p + 4 * i));
  }
}

template <int D>
__device__ __forceinline__ void tok_load(TokTile<D>& x, const TokenParams& p, const int* pages, int first, int n,
                                         int key, int hk, int g, int t) {
  x.n = 0;
  if (key < n) {
    // Tiles start at multiples of 16 and pages hold a multiple of 16 slots.
    const int page = pages[((first + key) >> p.page_shift) - (first >> p.page_shift)];
    if (page >= 0) {
      x.n = min(kTokTile, n - key);
      const int off = (first + key) & ((1 << p.page_shift) - 1);
      const int64_t row = ((static_cast<int64_t>(page) * p.Hk + hk) << p.page_shift) + off;
      const uint8_t* kp = p.k_codes + (row + g) * D + t * (D / 4);
      const uint8_t* vp = p.v_codes + (row + 2 * t) * D + g * (D / 8);
      ld_words(x.k[0], kp);
      ld_words(x.k[1], kp + 8 * D);
      x.ks[0] = p.k_scale[row + g];
      x.ks[1] = p.k_scale[row + g + 8];
      ld_words(x.v[0], vp);
      ld_words(x.v[1], vp + D);
      ld_words(x.v[2], vp + 8 * D);
      ld_words(x.v[3], vp + 9 * D);
      x.vs[0] = p.v_scale[row + g];
      x.vs[1] = p.v_scale[row + g + 8];
    }
  }
}

// Running state of the lane's heads 2t, 2t + 1 of each block of 8.
template <int D, int NT>
struct TokState {
  float m[NT][2];            // reference of the exponent, log2 (-inf: nothing seen)
  float l[NT][2];            // sum of 2^(x - m) over this lane's keys
  float w[NT][2];            // largest weight p * vs met, as of the last renewal
  float cf[NT][2];           // power of two on the weights
  float o[NT][D / 16][4];
};

template <int D, int NT, int kFmt>
__device__ __forceinline__ void tok_step(TokTile<D>& x, const uint32_t (&q)[NT][D / 16][2], const float (&qf)[NT][2],
                                         TokState<D, NT>& st, int g, int t) {
  const float kNegInf = -__int_as_float(0x7F800000);
  if (x.n < kTokTile) {
    // Codes and scales behind the last key may be anything: none takes part.
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (2 * t + (i & 1) + 8 * (i >> 1) >= x.n) {
#pragma unroll
        for (int k = 0; k < D / 32; ++k) x.v[i][k] = 0;
      }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (g + 8 * i >= x.n) x.vs[i] = 0.f;
  }
  uint32_t a[4];
  float s[NT][4];
#pragma unroll
  for (int b = 0; b < NT; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[b][i] = 0.f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    codes_f16<kFmt>(x.k[0][i], a[0], a[2]);
    codes_f16<kFmt>(x.k[1][i], a[1], a[3]);
#pragma unroll
    for (int b = 0; b < NT; ++b) mma_f16_16816(s[b], a, q[b][i][0], q[b][i][1]);
  }
  uint32_t pb[NT][2];
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    // s: (key g, head 2t), (key g, head 2t+1), (key g+8, ..), (key g+8, ..)
    float e[4];
    bool raise = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[b][i] = g + 8 * (i >> 1) < x.n ? s[b][i] * x.ks[i >> 1] * qf[b][i & 1] : kNegInf;
      raise = raise || s[b][i] > st.m[b][i & 1] + kTokRaise;
    }
    float w[4];
    auto weights = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float m = st.m[b][i & 1];
        e[i] = ex2_approx(s[b][i] - (m == kNegInf ? 0.f : m));
        w[i] = g + 8 * (i >> 1) < x.n ? e[i] * x.vs[i >> 1] * st.cf[b][i & 1] : 0.f;
      }
    };
    raise = __any_sync(0xFFFFFFFFu, raise);
    if (!raise) {
      weights();
      raise = __any_sync(0xFFFFFFFFu, fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])) > kTokMaxW);
    }
    if (raise) {
      // Renew the reference, and the power of two on the weights, of each head.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(s[b][h], s[b][h + 2]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const float m0 = st.m[b][h], m1 = fmaxf(m0, mx);
        const float ref = m1 == kNegInf ? 0.f : m1;
        const float alpha = m0 == kNegInf ? 0.f : ex2_approx(m0 - ref);
        float wm = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) wm = fmaxf(wm, ex2_approx(s[b][h + 2 * i] - ref) * x.vs[i]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) wm = fmaxf(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, o));
        wm = fmaxf(wm, st.w[b][h] * alpha);
        // exponent of wm in [-100, 100]; wm = 0 keeps the factor
        const int ex = min(max(static_cast<int>(__float_as_uint(wm) >> 23) - 127, -100), 100);
        const float cf = wm > 0.f ? __uint_as_float(static_cast<uint32_t>(127 - ex) << 23) : st.cf[b][h];
        // cf is a power of two, so dividing by it is exact
        const float f = alpha * (cf * (1.f / st.cf[b][h]));
        st.m[b][h] = m1;
        st.w[b][h] = wm;
        st.cf[b][h] = cf;
        st.l[b][h] *= alpha;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.o[b][i][h] *= f;
          st.o[b][i][h + 2] *= f;
        }
      }
      weights();
    }
    st.l[b][0] += e[0] + e[2];
    st.l[b][1] += e[1] + e[3];
    pb[b][0] = movmatrix_trans(f16x2_pack(w[0], w[1]));
    pb[b][1] = movmatrix_trans(f16x2_pack(w[2], w[3]));
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    // word i of the four keys: channels 4i .. 4i+3 of the lane's D/8
    const uint32_t lo01 = __byte_perm(x.v[0][i], x.v[1][i], 0x5140), hi01 = __byte_perm(x.v[0][i], x.v[1][i], 0x7362);
    const uint32_t lo23 = __byte_perm(x.v[2][i], x.v[3][i], 0x5140), hi23 = __byte_perm(x.v[2][i], x.v[3][i], 0x7362);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      codes_f16<kFmt>(h ? hi01 : lo01, a[0], a[1]);
      codes_f16<kFmt>(h ? hi23 : lo23, a[2], a[3]);
#pragma unroll
      for (int b = 0; b < NT; ++b) mma_f16_16816(st.o[b][2 * i + h], a, pb[b][0], pb[b][1]);
    }
  }
}

// E: type of q and out.  NT: blocks of 8 query heads per CTA.
template <class E, int D, int NT, int kFmt>
__global__ void __launch_bounds__(kTokThreads) token_attn_kernel(const __grid_constant__ TokenParams p) {
  pdl_enter();
  using S = typename E::S;
  __shared__ int s_pages[kTokMaxChunk / kTokTile];
  __shared__ float s_m[kTokWarps][8 * NT], s_l[kTokWarps][8 * NT];
  __shared__ float s_o[kTokWarps][8 * NT][D + 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int b = blockIdx.z;
  const int hk = blockIdx.y / p.head_blocks;
  const int h0 = (blockIdx.y - hk * p.head_blocks) * 8 * NT;      // first head of the group
  const int nh = min(8 * NT, p.G - h0);
  int len = p.lens[b];
  if (len > p.max_len) {
    if (tid == 0) atomicExch(p.err, 1);
    len = p.max_len;
  }
  const int first = blockIdx.x * p.chunk;
  const int n = min(p.chunk, len - first);
  if (n <= 0 && (p.chunks > 1 || blockIdx.x > 0)) return;

  const int npg = n > 0 ? ((first + n - 1) >> p.page_shift) - (first >> p.page_shift) + 1 : 0;
  for (int i = tid; i < npg; i += kTokThreads) {
    int page = p.table[b * p.table_stride + (first >> p.page_shift) + i];
    if (page < 0 || page >= p.pages) {
      atomicExch(p.err, 1);
      page = -1;
    }
    s_pages[i] = page;
  }

  // Q fragments (heads g of each block of 8) and the factor of the scores.
  uint32_t q[NT][D / 16][2];
  float qf[NT][2];
#pragma unroll
  for (int blk = 0; blk < NT; ++blk) {
    const int h = blk * 8 + g;
    Piece<E, 8> raw[D / 32];
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) raw[i].w[k] = 0;
      if (h < nh)
        raw[i].load(static_cast<const S*>(p.q) + b * p.q_stride +
                    static_cast<int64_t>(hk * p.G + h0 + h) * D + t * (D / 4) + 8 * i);
      bits = max(bits, piece_amax_bits(raw[i]));
    }
    bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 1));
    bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 2));
    // 2^-e, e the exponent of the largest channel (no scaling of zeros and non-finite rows)
    int ex = static_cast<int>(bits >> 23) - 127;
    if (ex == 128 || bits == 0) ex = 0;
    ex = max(ex, -126);
    const float dn = __uint_as_float(static_cast<uint32_t>(127 - min(ex, 126)) << 23);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
    const float rest = ex == 127 ? 0.5f : 1.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      float f[8];
      raw[i].get(f);
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
  __syncthreads();

  const float kNegInf = -__int_as_float(0x7F800000);
  TokState<D, NT> st;
#pragma unroll
  for (int blk = 0; blk < NT; ++blk) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      st.m[blk][k] = kNegInf;
      st.l[blk][k] = 0.f;
      st.w[blk][k] = 0.f;
      st.cf[blk][k] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) st.o[blk][i][k] = 0.f;
  }
  {
    TokTile<D> x0, x1;
    constexpr int kStep = kTokWarps * kTokTile;
    int key = warp * kTokTile;
    tok_load<D>(x0, p, s_pages, first, n, key, hk, g, t);
    while (key < n) {
      tok_load<D>(x1, p, s_pages, first, n, key + kStep, hk, g, t);
      if (x0.n > 0) tok_step<D, NT, kFmt>(x0, q, qf, st, g, t);
      key += kStep;
      if (key >= n) break;
      tok_load<D>(x0, p, s_pages, first, n, key + kStep, hk, g, t);
      if (x1.n > 0) tok_step<D, NT, kFmt>(x1, q, qf, st, g, t);
      key += kStep;
    }
  }

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
      }
      const float up = 1.f / st.cf[blk][k];           // exact: a power of two
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        *reinterpret_cast<float2*>(&s_o[warp][h][g * (D / 8) + 2 * i]) =
            make_float2(st.o[blk][i][k] * up, st.o[blk][i][k + 2] * up);
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
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kTokWarps; ++w) {
      const float f = ex2_approx(s_m[w][h] - ref);
      const float4 v = *reinterpret_cast<const float4*>(&s_o[w][h][d]);
      l += f * s_l[w][h];
      o.x += f * v.x;
      o.y += f * v.y;
      o.z += f * v.z;
      o.w += f * v.w;
    }
    const float r = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
    const int64_t row = static_cast<int64_t>(b) * p.Hq + hk * p.G + h0 + h;
    const float lse2 = l == 0.f ? kNegInf : m + log2f(l);
    o = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
    if (p.chunks > 1) {
      *reinterpret_cast<float4*>(p.part_o + (row * p.chunks + blockIdx.x) * D + d) = o;
      if (d == 0) p.part_lse[row * p.chunks + blockIdx.x] = lse2;
    } else {
      S* dst = static_cast<S*>(p.out) + b * p.out_stride + static_cast<int64_t>(hk * p.G + h0 + h) * D + d;
      Piece<E, 4> v;
      const float f[4] = {o.x, o.y, o.z, o.w};
      v.put(f);
      v.store(dst);
      if (d == 0 && p.lse) p.lse[row] = lse2 * 0.69314718055994531f;
    }
  }
}

// Joins the chunks of one (sequence, query head): weights 2^(lse_c - max), in
// chunk order within each of the block's kWays interleaved lanes, then the
// lanes in order.
constexpr int kJoinThreads = 128;
template <class E, int D>
__global__ void __launch_bounds__(kJoinThreads) token_join_kernel(const __grid_constant__ TokenParams p) {
  pdl_enter();
  constexpr int kLanes = D / 4, kWays = kJoinThreads / kLanes;
  __shared__ float4 s_o[kWays][kLanes];
  __shared__ float s_l[kWays];
  __shared__ float s_red[kJoinThreads / 32];
  const int64_t row = blockIdx.x;
  const int b = static_cast<int>(row / p.Hq), h = static_cast<int>(row - static_cast<int64_t>(b) * p.Hq);
  const int len = min(p.lens[b], p.max_len);
  const int nc = len > 0 ? (len + p.chunk - 1) / p.chunk : 0;
  const float kNegInf = -__int_as_float(0x7F800000);
  const float* lse = p.part_lse + row * p.chunks;
  const int tid = threadIdx.x, way = tid / kLanes, d = (tid % kLanes) * 4;
  float m = kNegInf;
  bool nan = false;
  for (int c = tid; c < nc; c += kJoinThreads) {
    m = fmaxf(m, lse[c]);
    nan = nan || lse[c] != lse[c];
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((tid & 31) == 0) s_red[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, s_red[w]);
  const float ref = m == kNegInf ? 0.f : m;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int c = way; c < nc; c += kWays) {
    const float f = ex2_approx(lse[c] - ref);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + (row * p.chunks + c) * D + d);
    l += f;
    o.x += f * v.x;
    o.y += f * v.y;
    o.z += f * v.z;
    o.w += f * v.w;
  }
  s_o[way][tid % kLanes] = o;
  if (d == 0) s_l[way] = l;
  __syncthreads();
  if (way == 0) {
#pragma unroll
    for (int w = 1; w < kWays; ++w) {
      const float4 v = s_o[w][tid];
      l += s_l[w];
      o.x += v.x;
      o.y += v.y;
      o.z += v.z;
      o.w += v.w;
    }
    const float r = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
    Piece<E, 4> v;
    const float f[4] = {o.x * r, o.y * r, o.z * r, o.w * r};
    v.put(f);
    v.store(static_cast<typename E::S*>(p.out) + b * p.out_stride + static_cast<int64_t>(h) * D + d);
    if (d == 0 && p.lse) p.lse[row] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace sage

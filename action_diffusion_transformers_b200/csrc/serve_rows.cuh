// serve_rows.cuh - the row-wise serving kernels: rotary positions, and the
// quantized KV cache's write and read.  All three are bound by HBM: each byte
// of a row is read once and each result written once, in 8- or 16-byte pieces
// per lane, several rows in flight per thread.
//
//  rope_kernel      (a, b) -> (a c - b s, a s + b c) for every channel pair of
//                   every head of Q and K, c and s formed once per (token,
//                   pair) in shared memory and used by all heads.
//  kv_write_kernel  row of D channels -> codes and one scale, in the slot of
//                   its token.
//  kv_read_kernel   codes and scale of a slot -> row.
#pragma once
#include <cuda_fp16.h>

#include "sage_ptx.cuh"

namespace sage {

// ---------------------------------------------------------------- elements
struct Bf16T {
  using S = uint16_t;
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
  }
};
struct Fp16T {
  using S = uint16_t;
  static __device__ __forceinline__ float lo(uint32_t w) {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16)));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
  }
};
struct Fp32T {
  using S = float;
};

template <int kBytes>
struct RawOf;
template <>
struct RawOf<2> { using type = uint16_t; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<16> { using type = uint4; };

// V consecutive elements of type E in 32-bit registers (V = 1: one element).
template <class E, int V>
struct Piece {
  static constexpr int kBytes = V * static_cast<int>(sizeof(typename E::S));
  static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const typename E::S* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = a.x;
        w[4 * i + 1] = a.y;
        w[4 * i + 2] = a.z;
        w[4 * i + 3] = a.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x; w[1] = a.y;
    } else {
      w[0] = *reinterpret_cast<const typename RawOf<kBytes>::type*>(p);
    }
  }
  __device__ __forceinline__ void store(typename E::S* p) const {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<typename RawOf<kBytes>::type*>(p) = static_cast<typename RawOf<kBytes>::type>(w[0]);
    }
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
    if constexpr (sizeof(typename E::S) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (V == 1) {
      f[0] = E::lo(w[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        f[2 * i] = E::lo(w[i]);
        f[2 * i + 1] = E::hi(w[i]);
      }
    }
  }
  __device__ __forceinline__ void put(const float (&f)[V]) {
    if constexpr (sizeof(typename E::S) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (V == 1) {
      w[0] = E::pack(f[0], 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = E::pack(f[2 * i], f[2 * i + 1]);
    }
  }
};

// n / d for 32-bit n by a product: q = (t + ((n - t) >> s1)) >> s2, t the high
// word of n * m.  With l = ceil(log2 d): m = floor(2^32 (2^l - d) / d) + 1, s1 =
// min(l, 1), s2 = max(l - 1, 0) (Granlund and Montgomery, division by invariant
// integers).
struct FastDiv {
  uint32_t m, s1, s2, d;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < div) ++l;
    m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << l) - div)) / div + 1);
    s1 = l < 1 ? l : 1;
    s2 = l > 1 ? l - 1 : 0;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    const uint32_t t = __umulhi(n, m);
    return (t + ((n - t) >> s1)) >> s2;
  }
};

// ----------------------------------------------------------------------------
// Rotary positions.
// ----------------------------------------------------------------------------
constexpr int kRopeThreads = 128;
constexpr int kRopeMaxPairs = 128;

struct RopeParams {
  const void* in[2];               // Q, K
  void* out[2];
  int64_t in_stride[2], out_stride[2];   // elements per token
  int heads[2];
  const int64_t* pos;              // [n_axes, T]
  int T, D, pairs;                 // pairs = rot_dim / 2
  int pair_stride;                 // pairs rounded up to 4
  int unit_shift;                  // lanes per head = 1 << unit_shift
  int units;                       // pieces per head (lanes behind it idle)
  int tokens;                      // per CTA
  int head_step;                   // heads per grid.y part
  FastDiv by_pairs, by_heads;      // by pairs, by head_step
  float mscale, sign;              // sign -1: the transposed rotation
  double turns[kRopeMaxPairs];     // revolutions per position, per pair
  uint8_t axis[kRopeMaxPairs];
};

// The angle is reduced in binary64: x = pos * turns is the number of
// revolutions, x - rint(x) in [-1/2, 1/2] its fraction, exact to 2^-53 * |x|
// (a position of a million loses 2^-33 of a revolution); only the fraction is
// rounded to 32 bits.
__device__ __forceinline__ float2 rope_turn(double pos, double turns, float mscale, float sign) {
  const double x = pos * turns;
  const float f = static_cast<float>(2.0 * (x - rint(x)));
  float s, c;
  sincospif(f, &s, &c);
  return make_float2(c * mscale, s * mscale * sign);
}

// kHalf: pair i is channels (i, i + rot/2), a unit is V channels of the first
// half with their V partners; otherwise pair i is (2i, 2i+1) and a unit is V
// channels, V / 2 pairs (V even).  Units past the rotated part copy channels
// that do not turn (only launched when in != out).  The CTA's (token, head)
// pairs are dealt to its lanes in turn, kBatch of them in flight per thread.
// Bound by HBM: 20480 tokens x 48 heads x 128 (504 MB) take 84 to 89 us, 5.7 to 6.0
// TB/s against a copy's 6.5, issue 65%; half of 128 channels of 16381 tokens x 36
// heads 53 to 56 us.  V = 1, for halves that are no multiple of 4 channels: 129 us
// where V = 4 takes 63 (16384 tokens x 40 heads, 18 and 20 pairs; FP32 133 and 115).
template <class E, bool kHalf, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  pdl_enter();
  using S = typename E::S;
  constexpr int kBatch = kHalf ? 2 : 4;
  extern __shared__ __align__(16) float2 cs[];      // [tokens][pair_stride]
  const int t0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  for (int i = threadIdx.x; i < nt * p.pairs; i += kRopeThreads) {
    const int t = p.by_pairs(i), j = i - t * p.pairs;
    const int64_t pos = p.pos[static_cast<int64_t>(p.axis[j]) * p.T + t0 + t];
    cs[t * p.pair_stride + j] = rope_turn(static_cast<double>(pos), p.turns[j], p.mscale, p.sign);
  }
  __syncthreads();
  const int lanes = 1 << p.unit_shift;
  const int step = kRopeThreads >> p.unit_shift;
  const int h0 = blockIdx.y * p.head_step;
  const int nh = min(p.head_step, p.heads[0] + p.heads[1] - h0);
  const int items = nt * p.head_step;
  const int rot_units = kHalf ? p.pairs / V : (2 * p.pairs + V - 1) / V;
  for (int u = threadIdx.x & (lanes - 1); u < p.units; u += lanes) {
    const bool turn = u < rot_units;
    // first channel of the unit, and of its second piece (kHalf)
    const int d0 = kHalf && !turn ? 2 * p.pairs + (u - rot_units) * 2 * V : u * V;
    const int d1 = kHalf ? (turn ? d0 + p.pairs : d0 + V) : d0;
    const bool two = kHalf && d1 < p.D;
    for (int first = threadIdx.x >> p.unit_shift; first < items; first += kBatch * step) {
      Piece<E, V> a[kBatch], b[kBatch];
      S* dst[kBatch];
      int tok[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int it = first + i * step;
        tok[i] = p.by_heads(it);
        const int hh = it - tok[i] * p.head_step;
        dst[i] = nullptr;
        if (it < items && hh < nh) {
          const int h = h0 + hh;
          const int w = h >= p.heads[0];
          const int64_t hd = static_cast<int64_t>(h - (w ? p.heads[0] : 0)) * p.D;
          const S* src = static_cast<const S*>(p.in[w]) + (t0 + tok[i]) * p.in_stride[w] + hd;
          dst[i] = static_cast<S*>(p.out[w]) + (t0 + tok[i]) * p.out_stride[w] + hd;
          a[i].load(src + d0);
          if (two) b[i].load(src + d1);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (dst[i] != nullptr) {
          if (turn) {
            constexpr int P = kHalf ? V : V / 2;
            const float2* cp = cs + tok[i] * p.pair_stride + (kHalf ? d0 : d0 / 2);
            float2 r[P];
            if constexpr (P % 2 == 0) {
#pragma unroll
              for (int k = 0; k < P / 2; ++k) {
                const float4 v = reinterpret_cast<const float4*>(cp)[k];
                r[2 * k] = make_float2(v.x, v.y);
                r[2 * k + 1] = make_float2(v.z, v.w);
              }
            } else {
#pragma unroll
              for (int k = 0; k < P; ++k) r[k] = cp[k];
            }
            float x[V], y[V];
            a[i].get(x);
            if constexpr (kHalf) {
              b[i].get(y);
#pragma unroll
              for (int k = 0; k < V; ++k) {
                const float xa = x[k], xb = y[k];
                x[k] = xa * r[k].x - xb * r[k].y;
                y[k] = xa * r[k].y + xb * r[k].x;
              }
              b[i].put(y);
              a[i].put(x);
            } else {
              // Channels behind the rotated part keep their bits.
              Piece<E, V> o;
#pragma unroll
              for (int k = 0; k < P; ++k) {
                const float xa = x[2 * k], xb = x[2 * k + 1];
                y[2 * k] = xa * r[k].x - xb * r[k].y;
                y[2 * k + 1] = xa * r[k].y + xb * r[k].x;
              }
              o.put(y);
              constexpr int kPairWords = sizeof(S) == 4 ? 2 : 1;
#pragma unroll
              for (int k = 0; k < P; ++k)
                if (d0 / 2 + k < p.pairs) {
#pragma unroll
                  for (int q = 0; q < kPairWords; ++q) a[i].w[k * kPairWords + q] = o.w[k * kPairWords + q];
                }
            }
          }
          a[i].store(dst[i] + d0);
          if (two) b[i].store(dst[i] + d1);
        }
      }
    }
  }
}

// ----------------------------------------------------------------------------
// Quantized KV cache.  Codes [pages, Hk, page_size, D], one byte each; scales
// f32 [pages, Hk, page_size].  A slot is page * page_size + offset.
// ----------------------------------------------------------------------------
constexpr int kKvThreads = 256;
constexpr int kKvInt8 = 0;
constexpr int kKvE4m3 = 1;

struct KvCacheView {
  uint8_t* codes[2];     // K, V
  float* scale[2];
  int64_t slots;         // pages * page_size
  int Hk, page_shift;    // page_size = 1 << page_shift
  FastDiv by_heads;      // by Hk
};

struct KvRowsParams {
  KvCacheView c;
  void* rows[2];         // K, V rows [T, Hk, D]
  int64_t stride[2];     // elements per token
  const int64_t* slot;   // [T]; negative: not in the cache
  int T;
  int* err;              // index error word
};

// Row of the cache that holds head h of a slot (rows are D codes, one scale).
__device__ __forceinline__ int64_t kv_row(const KvCacheView& c, int64_t slot, int h) {
  const int64_t page = slot >> c.page_shift;
  return ((page * c.Hk + h) << c.page_shift) + (slot - (page << c.page_shift));
}

// Largest magnitude of a piece, as the bits of a binary32 number.  Magnitudes
// are compared as integers, so an infinity or a NaN comes out on top.
template <class E, int V>
__device__ __forceinline__ uint32_t piece_amax_bits(const Piece<E, V>& a) {
  if constexpr (sizeof(typename E::S) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, a.w[i] & 0x7FFFFFFFu);
    return m;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) m = __vmaxu2(m, a.w[i] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    return __float_as_uint(E::lo(m));
  }
}

// Four values -> four code bytes.  INT8: the sum with 1.5 * 2^23 holds the
// nearest integer (ties to even) in its low byte; |x| <= 127 (1 + 2^-23)
// rounds to at most 127, so nothing is clamped.
template <int kFmt>
__device__ __forceinline__ uint32_t kv_codes4(float a, float b, float c, float d) {
  if constexpr (kFmt == kKvE4m3) {
    return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
  } else {
    const uint32_t x = __float_as_uint(__fadd_rn(a, 12582912.f)), y = __float_as_uint(__fadd_rn(b, 12582912.f));
    const uint32_t z = __float_as_uint(__fadd_rn(c, 12582912.f)), w = __float_as_uint(__fadd_rn(d, 12582912.f));
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  }
}

// L = D / 16 lanes per row, 16 channels each, kRows rows in flight per thread.
// grid.y: K, V.  One lane of a row divides for the scale and its neighbour for
// the inverse, in one instruction stream, and both are shuffled out.  With 8
// channels per lane the per-row work (index, maximum, division) was issued twice
// as often and bound the kernel (issue 77% busy): 50.9 us for 32768 tokens x 8
// heads of bf16, against 31 us of HBM time; now 35.6 to 37.8 us, 5.4 to 5.7 TB/s,
// issue 72%; FP32 59 us, 5.7 TB/s.
constexpr int kKvPer = 16;
template <class E>
constexpr int kKvPiece = 16 / static_cast<int>(sizeof(typename E::S));   // channels of a piece
template <class E>
constexpr int kKvRows = 2;                                          // rows in flight per thread
template <class E, int D, int kFmt>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const __grid_constant__ KvRowsParams p) {
  pdl_enter();
  using S = typename E::S;
  constexpr int L = D / kKvPer, kRows = kKvRows<E>;
  constexpr float kTop = kFmt == kKvE4m3 ? 448.f : 127.f;
  const int w = blockIdx.y;
  const int lane = threadIdx.x % L;
  const uint32_t total = static_cast<uint32_t>(p.T) * static_cast<uint32_t>(p.c.Hk);   // host: below 2^31
  const uint32_t r0 = blockIdx.x * (kKvThreads / L * kRows) + threadIdx.x / L;
  constexpr int V = kKvPiece<E>, N = kKvPer / V;
  Piece<E, V> x[kRows][N];
  int64_t slot[kRows];
  int head[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t r = r0 + i * (kKvThreads / L);
    slot[i] = -1;
    head[i] = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[i][k].w[q] = 0;
    if (r < total) {
      const int t = static_cast<int>(p.c.by_heads(r));
      head[i] = static_cast<int>(r) - t * p.c.Hk;
      slot[i] = p.slot[t];
      const S* src = static_cast<const S*>(p.rows[w]) + t * p.stride[w] + head[i] * D + lane * kKvPer;
#pragma unroll
      for (int k = 0; k < N; ++k) x[i][k].load(src + k * V);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) bits = max(bits, piece_amax_bits(x[i][k]));
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o));
    const float amax = __uint_as_float(bits);
    // Below 2^-100 the row counts as zero (top / amax must stay finite); with an
    // infinity or NaN in it the scale is NaN, which every reader of it meets.
    const bool finite = bits < 0x7F800000u;
    const bool some = finite && amax >= 7.8886091e-31f;
    const float q = (lane & 1) ? __fdiv_rn(kTop, some ? amax : 1.f) : __fdiv_rn(some ? amax : 0.f, kTop);
    const float inv = __shfl_sync(0xFFFFFFFFu, q, 1, L);
    float scale = q;                                   // lane 0 of the row
    if (!finite) scale = __uint_as_float(0x7FFFFFFFu);
    if (slot[i] >= 0) {
      if (slot[i] < p.c.slots) {
        const int64_t row = kv_row(p.c, slot[i], head[i]);
        uint32_t c[kKvPer / 4];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          float f[V];
          x[i][k].get(f);
#pragma unroll
          for (int q = 0; q < V / 4; ++q)
            c[k * (V / 4) + q] = kv_codes4<kFmt>(__fmul_rn(f[4 * q], inv), __fmul_rn(f[4 * q + 1], inv),
                                                 __fmul_rn(f[4 * q + 2], inv), __fmul_rn(f[4 * q + 3], inv));
        }
        if (!some) c[0] = c[1] = c[2] = c[3] = 0u;
        *reinterpret_cast<uint4*>(p.c.codes[w] + row * D + lane * kKvPer) = make_uint4(c[0], c[1], c[2], c[3]);
        if (lane == 0) p.c.scale[w][row] = scale;
      } else if (lane == 0) {
        atomicExch(p.err, 1);
      }
    }
  }
}

// Four code bytes -> values, exactly.
template <int kFmt>
__device__ __forceinline__ void kv_values4(uint32_t c, float (&f)[4]) {
  if constexpr (kFmt == kKvE4m3) {
    uint32_t h0, h1;
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(h0), "=r"(h1)
        : "r"(c));
    f[0] = Fp16T::lo(h0);
    f[1] = Fp16T::hi(h0);
    f[2] = Fp16T::lo(h1);
    f[3] = Fp16T::hi(h1);
  } else {
    // bytes biased by 128 under the exponent of 2^23: 2^23 + 128 + code
    const uint32_t b = c ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = __fsub_rn(__uint_as_float(__byte_perm(b, 0x4B000000u, 0x7540 + i)), 8388736.f);
  }
}

// L = D / 16 lanes per row, 16 codes each, kRows rows in flight per thread.  A
// lane's channels lie in pieces of 16 result bytes, L pieces side by side, so
// that each store covers whole sectors (16 channels in a run: 42.0 us for 32768
// tokens x 8 heads to bf16, against 34.5 to 36.1, 5.6 to 5.9 TB/s; FP32 57 us).
// grid.y: K, V.
template <class E, int D, int kFmt>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ KvRowsParams p) {
  pdl_enter();
  using S = typename E::S;
  constexpr int L = D / kKvPer, kRows = kKvRows<E>;
  const int w = blockIdx.y;
  const int lane = threadIdx.x % L;
  const uint32_t total = static_cast<uint32_t>(p.T) * static_cast<uint32_t>(p.c.Hk);   // host: below 2^31
  const uint32_t r0 = blockIdx.x * (kKvThreads / L * kRows) + threadIdx.x / L;
  constexpr int V = kKvPiece<E>, N = kKvPer / V;
  uint32_t codes[kRows][N][V / 4];
  float scale[kRows];
  S* dst[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t r = r0 + i * (kKvThreads / L);
    dst[i] = nullptr;
    if (r < total) {
      const int t = static_cast<int>(p.c.by_heads(r));
      const int h = static_cast<int>(r) - t * p.c.Hk;
      const int64_t slot = p.slot[t];
      if (slot >= p.c.slots) {
        if (lane == 0) atomicExch(p.err, 1);
      } else if (slot >= 0) {
        const int64_t row = kv_row(p.c, slot, h);
        const uint8_t* src = p.c.codes[w] + row * D + lane * V;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          if constexpr (V == 8) {
            const uint2 a = *reinterpret_cast<const uint2*>(src + k * L * V);
            codes[i][k][0] = a.x;
            codes[i][k][1] = a.y;
          } else {
            codes[i][k][0] = *reinterpret_cast<const uint32_t*>(src + k * L * V);
          }
        }
        scale[i] = p.c.scale[w][row];
        dst[i] = static_cast<S*>(p.rows[w]) + t * p.stride[w] + h * D + lane * V;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (dst[i] != nullptr) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        float f[V];
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          float v[4];
          kv_values4<kFmt>(codes[i][k][q], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[4 * q + e] = __fmul_rn(v[e], scale[i]);
        }
        Piece<E, V> o;
        o.put(f);
        o.store(dst[i] + k * L * V);
      }
    }
  }
}

}  // namespace sage

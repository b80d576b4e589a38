// Microscaled 4-bit floating point: a matrix to E2M1 codes with a scale per block, and back.
//
//   MXFP4   scale = 2^(floor(log2 max|x|) - 2) over 32 columns;  code = E2M1(x / scale)
//   NVFP4   global = 2^e, scale = E4M3(max|x| / (6 global)) over 16 columns;  code = E2M1(x / (scale global))
//
// Bound by HBM: 2 (or 4) bytes read and 0.53 (0.56) written per element.  A CTA takes a tile of 128 rows x 128
// columns, so that every 128-byte line of the source, every 64-byte piece of a row of codes and
// every 512-byte tile of scales is moved whole.  A lane takes 8 columns, 16 lanes a row: each load and store
// instruction of a warp covers two whole pieces of rows.  The CTAs are persistent and load ahead: a batch
// of rows of the same or the next tile is under way while one is processed.  Four bf16 6144 x 2048
// matrices: to MXFP4 in 21.7 us (127 MB, 5.9 TB/s; instruction issue 0.66 a clock is the next bound: 28.9 us
// before whole tiles lost their bounds checks and bf16 its widening), their values in 22.8 us (0.6 more with a load for each scale).
//
// For the transpose the tile goes through shared memory as 32-bit words, whose place is permuted by
// the 32-row group (word ^ 8 group), so that the four groups of eight columns that a warp reads
// fall into different banks.  8192 x 2048 bf16 to NVFP4: 16.0 us (14.1 plain, MXFP4 8.2 and 7.4), 6.6 of them the pass for
// the largest magnitude, which the matrix's scale needs before the first code.  Instruction issue bounds the other pass
// (16.7 an element and 12.5 us before whole tiles lost their bounds checks and bf16 its fp32 quotients).  Three
// matrices in turn, so that none is in the L2 cache as a whole: bf16 20.8 us (19.0, 11.8, 9.3), fp32 45.0 us (41.1, 16.5,
// 14.1): a quotient of fp32 numbers is divided and corrected to the last bit.
//
// The occupancies below leave some instances a register or two short (4 to 16 bytes spilled: bf16 transposed, fp32 MXFP4).
#include <cuda_runtime.h>

#include <type_traits>

#include "nshb_device.cuh"
#include "nshb_internal.h"

namespace nshb {
namespace {

constexpr int kThreads = 256;
constexpr int kT = 128;            // tile edge

__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float &a, float &b) {
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(h));
}
__device__ __forceinline__ void e2m1x8_to_f32(uint32_t c, float (&x)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int e = 0; e < 4; ++e) f16x2_to_f32(h[e], x[2 * e], x[2 * e + 1]);
}
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)b));
  float lo, hi;
  f16x2_to_f32(h, lo, hi);
  return lo;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // [-126, 127]
__device__ __forceinline__ float from_e8m0(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : b == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(b << 23);
}

// A quotient with a remainder is never exactly a border between two codes, although its fp32
// rounding may be: set the last bit of the truncated quotient ("round to odd"), which no border has,
// so that the next rounding decides as the exact quotient would.
__device__ __forceinline__ float odd(float q, float rem, float x) {
  if (rem == 0.f) return q;
  uint32_t b = __float_as_uint(q);
  if ((rem < 0.f) != (x < 0.f)) b -= 1;
  return __uint_as_float(b | 1u);
}

// a x in fp32 rounded to odd: of the numbers below and above it (the same where it is one) the one with an odd last
// bit.  Rounding that to fewer bits gives the nearest value to the product itself.
__device__ __forceinline__ float odd_product(float a, float x) {
  const float low = __fmul_rd(a, x), high = __fmul_ru(a, x);
  return (__float_as_uint(low) & 1u) ? low : high;
}

// The matrix's scale exponent from its largest finite magnitude (bits): the smallest e >= -126 with max <=
// 2688 2^e; 2688 = 0.65625 x 2^12.
__device__ __forceinline__ int global_exponent(uint32_t top) {
  if (top == 0) return 0;
  const int be = (int)(top >> 23);
  if (be == 0) return -126;                              // below 2^-126
  const int e = be - 126 - 12 + ((top & 0x7fffffu) > 0x280000u ? 1 : 0);   // 0.65625 has the mantissa 1.3125
  return e < -126 ? -126 : e;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Within one unit of the last place.
__device__ __forceinline__ float fast_reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 32 consecutive columns as they were loaded.
template <bool F32>
struct Cols32 {
  static constexpr int NW = F32 ? 32 : 16;
  uint32_t w[NW];
  __device__ __forceinline__ float get(int e) const {
    if (F32) return __uint_as_float(w[e]);
    return (e & 1) ? bf16hi(w[e >> 1]) : bf16lo(w[e >> 1]);
  }
  // Bits of the largest magnitude of columns [c, c + n), NaN and infinity the largest.
  template <int C, int N>
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (F32) {
#pragma unroll
      for (int e = C; e < C + N; ++e) m = max(m, w[e] & 0x7fffffffu);
      return m;
    } else {
#pragma unroll
      for (int e = C / 2; e < (C + N) / 2; ++e) m = max_magnitude(m, w[e]);
      return max(m << 16, m & 0xffff0000u);
    }
  }
};

// 8 consecutive columns as they were loaded.
template <bool F32>
struct Cols8 {
  static constexpr int NW = F32 ? 8 : 4;
  uint32_t w[NW];
  __device__ __forceinline__ float get(int e) const {
    if (F32) return __uint_as_float(w[F32 ? e : 0]);
    return (e & 1) ? bf16hi(w[e >> 1]) : bf16lo(w[e >> 1]);
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, w[e] & 0x7fffffffu);
      return m;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max_magnitude(m, w[e]);
      return max(m << 16, m & 0xffff0000u);
    }
  }
};

// The scale byte of a block whose largest magnitude has the bits `top`, and what its elements are
// multiplied with (MX) or divided by (NV: s, and its reciprocal) to become codes.
template <bool F32, bool NV>
__device__ __forceinline__ uint32_t block_scale(uint32_t top, float down, float &s, float &r) {
  const bool bad = top >= 0x7f800000u;
  if (!NV) {
    const uint32_t be = top >> 23;
    const uint32_t b = be > 2 ? be - 2 : 0;              // biased exponent of the scale, 2^-127 at least
    r = __uint_as_float((254u - b) << 23);               // exact: a power of two
    return bad ? 255u : b;
  }
  const float m = (bad ? 0.f : __uint_as_float(top)) * down;
  uint32_t sb;
  if (F32) {
    const float q6 = __fdiv_rn(m, 6.f);
    sb = to_e4m3(odd(q6, fmaf(-q6, 6.f, m), m));
  } else {
    // A bf16 m (8 bits) is 6 times the border of two scales (5 bits), or differs from it by 2^-8 of itself.
    // So a quotient that is at most 2^-19 too large and then cut to 12 bits is on the border exactly
    // where m / 6 is, and on its side of it elsewhere.
    sb = to_e4m3(__uint_as_float(__float_as_uint(m * (float)((1. + 0x1p-20) / 6.)) & 0xfffff000u));
  }
  s = from_e4m3(sb);
  r = s > 0.f ? (F32 ? __frcp_rn(s) : fast_reciprocal(s)) : 0.f;
  return bad ? 0x7fu : sb;
}
template <bool NV>
__device__ __forceinline__ float scaled(float x, float down, float s, float r) {
  if (!NV) return x * r;
  // x / s correctly rounded: one correction of the product with the correctly rounded
  // reciprocal (P. Markstein, "Computation of elementary functions on the IBM RISC
  // System/6000 processor", 1990).  a is x 2^-eg, exact.
  const float a = x * down;
  float t = a * r;
  t = fmaf(fmaf(-t, s, a), r, t);
  if (s > 0.f) t = odd(t, fmaf(-t, s, a), a);
  return copysignf(t, a);   // the correction of -0 gives +0
}

// The codes of 8 columns (words W .. of v).
template <bool F32, bool NV, class V>
__device__ __forceinline__ uint32_t codes8(const V &v, int first, uint32_t top, float down, float s, float r) {
  float x[8];
  if constexpr (!F32 && !NV) {
    // bf16 times a power of two: exact in bf16 (what underflows is far below half a code)
    const uint32_t r2 = (__float_as_uint(r) >> 16) | (__float_as_uint(r) & 0xffff0000u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t y = mul_bf16x2(v.w[first / 2 + e], r2);
      x[2 * e] = bf16lo(y);
      x[2 * e + 1] = bf16hi(y);
    }
  } else if constexpr (!F32) {
    // A bf16 a (8 bits) is the border of two codes (3 bits) times s (4 bits), or differs from it by 1/254 of
    // itself or more.  So a / s rounded to bf16 is on a border, which is a bf16 value, exactly where a / s
    // is, and on its side of it elsewhere; so is a (rh + rl), 1 / s in two bf16 parts, in two roundings
    // (checked for every a and s).  rl is not negative: -0 stays -0.
    const uint32_t d = __float_as_uint(down), d2 = (d >> 16) | (d & 0xffff0000u);
    const float low = r - __uint_as_float(__float_as_uint(r) & 0xffff0000u);
    const uint32_t rh = __byte_perm(__float_as_uint(r), 0u, 0x3232), rl = pack_bf16(low, low);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a = mul_bf16x2(v.w[first / 2 + e], d2);   // exact: a power of two
      const uint32_t y = fma_bf16x2(a, rh, mul_bf16x2(a, rl));
      x[2 * e] = bf16lo(y);
      x[2 * e + 1] = bf16hi(y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = scaled<NV>(v.get(first + e), down, s, r);
  }
  const uint32_t c = e2m1x8(x);
  return top >= 0x7f800000u ? 0u : c;
}

// Codes (16 bytes) of 32 columns and their scale byte (MX) or two (NV: the second in bits 8-15).
template <bool F32, bool NV>
__device__ __forceinline__ uint32_t quantize32(const Cols32<F32> &v, float down, uint32_t (&codes)[4]) {
  uint32_t scales = 0;
#pragma unroll
  for (int h = 0; h < (NV ? 2 : 1); ++h) {
    const uint32_t top = !NV ? v.template top<0, 32>() : h == 0 ? v.template top<0, 16>() : v.template top<16, 16>();
    float s = 0.f, r;
    scales |= block_scale<F32, NV>(top, down, s, r) << (8 * h);
#pragma unroll
    for (int g = 0; g < (NV ? 2 : 4); ++g) codes[2 * h + g] = codes8<F32, NV>(v, 16 * h + 8 * g, top, down, s, r);
  }
  return scales;
}

template <class P>
__device__ __forceinline__ int find_item(const P &p, int tile) {
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.item[mid].tile_begin <= tile) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Stores what 32 columns from 32 * kc of tile row r became: codes to memory (rows past the matrix
// have none), scale bytes to the staged tile(s).
template <bool NV>
__device__ __forceinline__ void put(const Fp4Item &q, int tr, int tk, int r, int kc, const uint32_t (&codes)[4],
                                    uint32_t scales, uint8_t *stage) {
  const int row = tr * kT + r;
  if (row < q.rows)
    *reinterpret_cast<uint4 *>(q.codes + (int64_t)row * q.ktiles * 64 + tk * 64 + kc * 16) =
        make_uint4(codes[0], codes[1], codes[2], codes[3]);
  const int at = 16 * (r & 31) + 4 * (r >> 5);
  if (NV) *reinterpret_cast<unsigned short *>(stage + (kc >> 1) * 512 + at + 2 * (kc & 1)) = (unsigned short)scales;
  else stage[at + kc] = (uint8_t)scales;
}

template <bool F32>
__device__ __forceinline__ uint32_t load_elem(const void *x, int64_t i) {
  if (F32) return static_cast<const uint32_t *>(x)[i];
  return static_cast<const unsigned short *>(x)[i];
}

// N elements of a row (N * size a multiple of 16) from column c on, zeros from `cols` on.
template <bool F32, int N, int NW>
__device__ __forceinline__ void load_cols(const void *x, int64_t off, int c, int cols, bool vec, bool live, uint32_t (&w)[NW]) {
  static_assert(NW == (F32 ? N : N / 2), "words of N elements");
  const char *b = static_cast<const char *>(x) + (off + c) * (F32 ? 4 : 2);
  if (live && vec && c + N <= cols) {
#pragma unroll
    for (int g = 0; g < NW / 4; ++g) {
      const uint4 u = *reinterpret_cast<const uint4 *>(b + 16 * g);
      w[4 * g] = u.x; w[4 * g + 1] = u.y; w[4 * g + 2] = u.z; w[4 * g + 3] = u.w;
    }
  } else if (live && c < cols) {
#pragma unroll
    for (int e = 0; e < NW; ++e) {
      if (F32) {
        w[e] = c + e < cols ? load_elem<F32>(b, e) : 0u;
      } else {
        const uint32_t lo = c + 2 * e < cols ? load_elem<F32>(b, 2 * e) : 0u;
        const uint32_t hi = c + 2 * e + 1 < cols ? load_elem<F32>(b, 2 * e + 1) : 0u;
        w[e] = lo | (hi << 16);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < NW; ++e) w[e] = 0u;
  }
}

// A tile of the launch's list: its item, its row and column among the item's tiles.
struct Tile {
  int item, l, tr, tk;
};
template <class P>
__device__ __forceinline__ Tile tile_at(const P &p, int t) {
  Tile r;
  r.item = find_item(p, t);
  r.l = t - p.item[r.item].tile_begin;
  r.tr = r.l / p.item[r.item].ktiles;
  r.tk = r.l - r.tr * p.item[r.item].ktiles;
  return r;
}

// NVFP4: 2^-e of an item's scale, from the records of the pass before (every CTA for itself); its first tile's
// CTA writes the scale.
template <class P>
__device__ float down_of(const P &p, const Fp4Item &q, bool write) {
  __shared__ uint32_t tops[kThreads / 32];
  uint32_t top = 0;
  for (int i = threadIdx.x; i < q.n_rec; i += kThreads) top = max(top, (uint32_t)p.rec[q.rec_begin + i]);
  top = __reduce_max_sync(0xffffffffu, top);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, tops[w]);
  const int eg = global_exponent(top);
  if (write && threadIdx.x == 0) *q.global = power_of_two(eg);
  return power_of_two(-eg);
}

template <bool NV>
__device__ __forceinline__ void store_scales(const Fp4Item &q, int l, const uint8_t *stage) {
  constexpr int kBytes = NV ? 1024 : 512;
  if (threadIdx.x * 4 < kBytes)
    reinterpret_cast<uint32_t *>(q.scales + (int64_t)l * kBytes)[threadIdx.x] = reinterpret_cast<const uint32_t *>(stage)[threadIdx.x];
}

template <bool F32, bool NV, int N>
__global__ void __launch_bounds__(kThreads, 4) fp4_quantize_kernel(const __grid_constant__ Fp4Block<N> p) {
  constexpr int kBatch = F32 ? 2 : 4;                    // rows of a lane in a batch: 64 bytes
  __shared__ __align__(16) uint8_t stage[2][1024];
  pdl_trigger();
  pdl_wait();
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  // This thread's first row of a tile: source, codes, and the way to the row 16 below.
  struct Mine {
    const char *src;
    uint8_t *codes;
    int64_t src_step;
    int code_step;
    bool whole;            // the tile has 128 rows and columns and its rows take 16-byte loads
  };
  auto mine = [&](const Tile &t) {
    const Fp4Item &q = p.item[t.item];
    Mine m;
    const int64_t row = t.tr * kT + r0;
    m.src = static_cast<const char *>(q.x) + (row * q.ld + t.tk * kT + 8 * l) * (F32 ? 4 : 2);
    m.src_step = 16 * q.ld * (F32 ? 4 : 2);
    m.codes = q.codes + row * q.ktiles * 64 + t.tk * 64 + 4 * l;
    m.code_step = 16 * 64 * q.ktiles;
    m.whole = (q.flags & kFp4Vec) && t.tr * kT + kT <= q.rows && t.tk * kT + kT <= q.cols;
    return m;
  };
  auto load = [&](const Tile &t, const Mine &m, int b, Cols8<F32> (&v)[kBatch]) {
    if (m.whole) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int g = 0; g < Cols8<F32>::NW / 4; ++g) {
          const uint4 u = *reinterpret_cast<const uint4 *>(m.src + (b + i) * m.src_step + 16 * g);
          v[i].w[4 * g] = u.x; v[i].w[4 * g + 1] = u.y; v[i].w[4 * g + 2] = u.z; v[i].w[4 * g + 3] = u.w;
        }
      return;
    }
    const Fp4Item &q = p.item[t.item];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = t.tr * kT + r0 + 16 * (b + i);
      load_cols<F32, 8>(q.x, (int64_t)row * q.ld, t.tk * kT + 8 * l, q.cols, q.flags & kFp4Vec, row < q.rows, v[i].w);
    }
  };
  int at_tile = blockIdx.x, last_item = -1, turn = 0;
  if (at_tile >= p.total_tiles) return;
  Tile t = tile_at(p, at_tile);
  Mine m = mine(t);
  Cols8<F32> next[kBatch];
  load(t, m, 0, next);
  float down = 1.f;
  for (;;) {
    const Fp4Item &q = p.item[t.item];
    if (NV && (t.item != last_item || t.l == 0)) {
      down = down_of(p, q, t.l == 0);
      last_item = t.item;
    }
    const int next_tile = at_tile + gridDim.x;
    const bool more = next_tile < p.total_tiles;
    const Tile tn = more ? tile_at(p, next_tile) : t;
    const Mine mn = more ? mine(tn) : m;
    // scale (r, b) of the tile is byte 16 (r mod 32) + 4 (r div 32) + b; r = r0 + 16 k
    uint8_t *scale = stage[turn] + 16 * r0 + (NV ? (l >> 3) * 512 + ((l >> 1) & 3) : l >> 2);
    const int rows_left = m.whole ? kT : q.rows - t.tr * kT - r0;
#pragma unroll
    for (int b = 0; b < 8; b += kBatch) {
      Cols8<F32> v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) v[i] = next[i];
      if (b + kBatch < 8) load(t, m, b + kBatch, next);
      else if (more) load(tn, mn, 0, next);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int k = b + i;
        // a block is two lanes (NV) or four
        uint32_t top = v[i].top();
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if (!NV) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float s = 0.f, rc;
        const uint32_t sb = block_scale<F32, NV>(top, down, s, rc);
        const uint32_t c = codes8<F32, NV>(v[i], 0, top, down, s, rc);
        if (16 * k < rows_left) *reinterpret_cast<uint32_t *>(m.codes + (int64_t)k * m.code_step) = c;
        if ((l & (NV ? 1 : 3)) == 0) scale[256 * (k & 1) + 4 * (k >> 1)] = (uint8_t)sb;
      }
    }
    __syncthreads();       // the other half of the stage is free again after this one
    store_scales<NV>(q, t.l, stage[turn]);
    turn ^= 1;
    if (!more) break;
    t = tn;
    m = mn;
    at_tile = next_tile;
  }
}

// The transpose.  A tile of the source: rows tk * 128 .. (the 4-bit matrix's columns), columns tr * 128 ...
template <bool F32, bool NV, int N>
__global__ void __launch_bounds__(kThreads, F32 ? 2 : 3) fp4_quantize_t_kernel(const __grid_constant__ Fp4Block<N> p) {
  extern __shared__ uint32_t tile[];
  __shared__ __align__(16) uint8_t stage[2][1024];
  pdl_trigger();
  pdl_wait();
  constexpr int WPR = F32 ? 128 : 64;            // words per row of the tile
  constexpr int TPR = WPR / 4;                   // threads per row, 16 bytes each
  constexpr int kLoads = kT * TPR / kThreads;
  const int lr = (int)threadIdx.x / TPR, lw = 4 * ((int)threadIdx.x % TPR);
  struct Piece {
    uint32_t w[4];
  };
  auto load = [&](const Tile &t, Piece (&v)[kLoads]) {
    const Fp4Item &q = p.item[t.item];
    if ((q.flags & kFp4Vec) && t.tk * kT + kT <= q.cols && t.tr * kT + kT <= q.rows) {
      const char *src = static_cast<const char *>(q.x) + ((int64_t)(t.tk * kT + lr) * q.ld + t.tr * kT) * (F32 ? 4 : 2) + 4 * lw;
      const int64_t step = (kThreads / TPR) * q.ld * (F32 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint4 u = *reinterpret_cast<const uint4 *>(src + i * step);
        v[i].w[0] = u.x; v[i].w[1] = u.y; v[i].w[2] = u.z; v[i].w[3] = u.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = t.tk * kT + lr + i * (kThreads / TPR);
      load_cols<F32, F32 ? 4 : 8>(q.x, (int64_t)row * q.ld, t.tr * kT + (F32 ? lw : 2 * lw), q.rows, q.flags & kFp4Vec,
                                  row < q.cols, v[i].w);
    }
  };
  int at_tile = blockIdx.x, last_item = -1, turn = 0;
  if (at_tile >= p.total_tiles) return;
  Tile t = tile_at(p, at_tile);
  Piece next[kLoads];
  load(t, next);
  float down = 1.f;
  for (;;) {
    const Fp4Item &q = p.item[t.item];
    if (NV && (t.item != last_item || t.l == 0)) {
      down = down_of(p, q, t.l == 0);
      last_item = t.item;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = lr + i * (kThreads / TPR);
      *reinterpret_cast<uint4 *>(tile + r * WPR + (lw ^ ((r >> 5) << 3))) =
          make_uint4(next[i].w[0], next[i].w[1], next[i].w[2], next[i].w[3]);
    }
    __syncthreads();
    const int next_tile = at_tile + gridDim.x;
    const bool more = next_tile < p.total_tiles;
    const Tile tn = more ? tile_at(p, next_tile) : t;
    if (more) load(tn, next);
    const int kc = threadIdx.x & 3, c0 = threadIdx.x >> 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // fp32: columns c0 and c0 + 64; bf16: the two columns of word c0
      const int c = F32 ? c0 + 64 * i : 2 * c0 + i, word = F32 ? c : c0;
      Cols32<F32> v;
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const uint32_t a = tile[(kc * 32 + e) * WPR + (word ^ (kc << 3))];
        const uint32_t b = tile[(kc * 32 + e + 1) * WPR + (word ^ (kc << 3))];
        if (F32) {
          v.w[F32 ? e : 0] = a;
          v.w[F32 ? e + 1 : 0] = b;
        } else {
          v.w[e / 2] = __byte_perm(a, b, i == 0 ? 0x5410 : 0x7632);
        }
      }
      uint32_t codes[4];
      const uint32_t s = quantize32<F32, NV>(v, down, codes);
      put<NV>(q, t.tr, t.tk, c, kc, codes, s, stage[turn]);
    }
    __syncthreads();       // the tile may be overwritten, the scales are staged
    store_scales<NV>(q, t.l, stage[turn]);
    turn ^= 1;
    if (!more) break;
    t = tn;
    at_tile = next_tile;
  }
}

template <bool F32, bool NV, int N>
__global__ void __launch_bounds__(kThreads, 4) fp4_dequantize_kernel(const __grid_constant__ Fp4Block<N> p) {
  __shared__ __align__(16) float stage[(kThreads / 32) * 2 * kT];
  pdl_trigger();
  pdl_wait();
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4, lane = threadIdx.x & 31;
  struct Codes {
    uint32_t code[8], scale[8];
    float g;
  };
  const int byte = NV ? (l >> 1) & 3 : l >> 2;
  auto load = [&](const Tile &t, Codes &v) {
    const Fp4Item &q = p.item[t.item];
    v.g = NV ? *q.global : 1.f;
    // scale (r, b) of the tile is byte 16 (r mod 32) + 4 (r div 32) + b; r = r0 + 16 i: four rows in 16 bytes
    const uint4 *scale = reinterpret_cast<const uint4 *>(q.scales + (int64_t)t.l * (NV ? 1024 : 512) + (NV ? (l >> 3) * 512 : 0)) + r0;
    const uint4 even = scale[0], uneven = scale[16];
    v.scale[0] = even.x; v.scale[2] = even.y; v.scale[4] = even.z; v.scale[6] = even.w;
    v.scale[1] = uneven.x; v.scale[3] = uneven.y; v.scale[5] = uneven.z; v.scale[7] = uneven.w;
    const uint8_t *codes = q.codes + (int64_t)(t.tr * kT + r0) * q.ktiles * 64 + t.tk * 64 + 4 * l;
    const int step = 1024 * q.ktiles, rows_left = q.rows - t.tr * kT - r0;
    if (q.rows - t.tr * kT >= kT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v.code[i] = *reinterpret_cast<const uint32_t *>(codes + i * step);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v.code[i] = 16 * i < rows_left ? *reinterpret_cast<const uint32_t *>(codes + i * step) : 0u;
    }
  };
  int at_tile = blockIdx.x;
  if (at_tile >= p.total_tiles) return;
  Tile t = tile_at(p, at_tile);
  Codes next;
  load(t, next);
  for (;;) {
    const Codes v = next;
    const Fp4Item &q = p.item[t.item];
    const int next_tile = at_tile + gridDim.x;
    const bool more = next_tile < p.total_tiles;
    const Tile tn = more ? tile_at(p, next_tile) : t;
    if (more) load(tn, next);
    char *d = static_cast<char *>(q.x) + ((int64_t)(t.tr * kT + r0) * q.ld + t.tk * kT + 8 * l) * (F32 ? 4 : 2);
    const int64_t step = 16 * q.ld * (F32 ? 4 : 2);
    auto value = [&](int i, float (&y)[8], auto odd) {
      const uint32_t b = __byte_perm(v.scale[i], 0u, 0x4440 | byte);
      const float s = NV ? from_e4m3(b) : from_e8m0(b);
      e2m1x8_to_f32(v.code[i], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = decltype(odd)::value ? odd_product(y[e] * s, v.g) : y[e] * s * v.g;
    };
    auto store = [&](char *d, const float (&y)[8]) {
      if (F32) {
        float4 *o = reinterpret_cast<float4 *>(d);
        o[0] = make_float4(y[0], y[1], y[2], y[3]);
        o[1] = make_float4(y[4], y[5], y[6], y[7]);
      } else {
        *reinterpret_cast<uint4 *>(d) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      }
    };
    const bool rows_whole = (q.flags & kFp4Vec) && t.tk * kT + kT <= q.cols;
    auto tile = [&](auto odd) {
      if (rows_whole && t.tr * kT + kT <= q.rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float y[8];
          value(i, y, odd);
          store(F32 ? d : d + i * step, y);   // the form that each type has registers for
          if (F32) d += step;
        }
      } else {
        const int rows_left = q.rows - t.tr * kT - r0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float y[8];
          value(i, y, odd);
          if (rows_whole) {
            if (16 * i < rows_left) store(d + i * step, y);
            continue;
          }
          // through shared memory, so that a store instruction covers neighbouring elements
          float *w = stage + (threadIdx.x >> 5) * 2 * kT;
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4 *>(w + (lane >> 4) * kT + 8 * l + 4 * e) =
                make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int rr = e >> 2, cc = 32 * (e & 3) + lane;
            const int to_row = t.tr * kT + (r0 & ~1) + rr + 16 * i, to_col = t.tk * kT + cc;
            if (to_row >= q.rows || to_col >= q.cols) continue;
            const int64_t at = (int64_t)to_row * q.ld + to_col;
            if (F32) static_cast<float *>(q.x)[at] = w[rr * kT + cc];
            else static_cast<__nv_bfloat16 *>(q.x)[at] = __float2bfloat16_rn(w[rr * kT + cc]);
          }
        }
      }
    };
    // The products are exact in fp32, unless the matrix's scale is no power of two: rounding to fp32 would then be one
    // rounding too many for bf16 (2048 x 8192 in 9.5 us instead of 8.5).  Chosen for a whole tile: within `value` the branch
    // costs 0.7 us of a 777 x 333 matrix's 4.5.
    if constexpr (NV && !F32) {
      if (__float_as_uint(v.g) & 0x7fffffu) tile(std::true_type());
      else tile(std::false_type());
    } else {
      tile(std::false_type());
    }
    if (!more) break;
    t = tn;
    at_tile = next_tile;
  }
}

constexpr int kTileBytesT = kT * 128 * 4;   // an fp32 tile of the transposing kernel

int grid_of(int tiles, int per_sm) {
  const int most = per_sm * device_sms();
  return tiles < most ? tiles : most;
}

// The items of a launch are of one dtype and format.
template <bool F32, bool NV, int N>
cudaError_t launch_quantize(const Fp4Params &p, bool transpose, cudaStream_t s) {
  const Fp4Block<N> &b = prefix<Fp4Block<N>>(p);
  if (!transpose)
    return launch_pdl(fp4_quantize_kernel<F32, NV, N>, dim3(grid_of(p.total_tiles, 4)), dim3(kThreads), 0, s, b);
  const int smem = F32 ? kTileBytesT : kTileBytesT / 2;
  static PerDevice attr_set;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!attr_set.get(dev)) {
    e = cudaFuncSetAttribute(fp4_quantize_t_kernel<F32, NV, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_set.set(dev, 1);
  }
  return launch_pdl(fp4_quantize_t_kernel<F32, NV, N>, dim3(grid_of(p.total_tiles, F32 ? 2 : 3)), dim3(kThreads), smem, s, b);
}
template <bool F32, bool NV, int N>
cudaError_t launch_dequantize(const Fp4Params &p, cudaStream_t s) {
  return launch_pdl(fp4_dequantize_kernel<F32, NV, N>, dim3(grid_of(p.total_tiles, 4)), dim3(kThreads), 0, s,
                    prefix<Fp4Block<N>>(p));
}

// Calls f(F32, NV, N) for a launch's dtype, format and the smallest instance that holds its items.
template <class F>
cudaError_t with_kind(const Fp4Params &p, F &&f) {
  const bool f32 = p.item[0].flags & kFp4F32, nv = p.item[0].flags & kFp4Nv;
  auto n = [&](auto a, auto b) {
    return p.n <= kFewFp4 ? f(a, b, std::integral_constant<int, kFewFp4>()) : f(a, b, std::integral_constant<int, kMaxFp4>());
  };
  if (f32) return nv ? n(std::true_type(), std::true_type()) : n(std::true_type(), std::false_type());
  return nv ? n(std::false_type(), std::true_type()) : n(std::false_type(), std::false_type());
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4Params &p, bool transpose, cudaStream_t s) {
  if (p.total_tiles <= 0) return cudaSuccess;
  return with_kind(p, [&](auto f32, auto nv, auto n) {
    return launch_quantize<decltype(f32)::value, decltype(nv)::value, decltype(n)::value>(p, transpose, s);
  });
}

cudaError_t launch_fp4_dequantize(const Fp4Params &p, cudaStream_t s) {
  if (p.total_tiles <= 0) return cudaSuccess;
  return with_kind(p, [&](auto f32, auto nv, auto n) {
    return launch_dequantize<decltype(f32)::value, decltype(nv)::value, decltype(n)::value>(p, s);
  });
}

}  // namespace nshb

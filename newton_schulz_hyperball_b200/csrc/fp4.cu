// Microscaled 4-bit floating point: a matrix to E2M1 codes with a scale per block, and back.
//
//   MXFP4   scale = 2^(floor(log2 max|x|) - 2) over 32 columns;  code = E2M1(x / scale)
//   NVFP4   global = 2^e, scale = E4M3(max|x| / (6 global)) over 16 columns;  code = E2M1(x / (scale global))
//
// Bound by HBM: 2 (or 4) bytes read and 0.53 (0.56) written per element.  A CTA takes a tile of 128 rows x 128
// columns, so that every 128-byte line of the source, every 64-byte piece of a row of codes and
// every 512-byte tile of scales is moved whole; a thread quantises 32 columns of a row at a time.  For the
// transpose the tile goes through shared memory as 32-bit words, whose place is permuted by
// the 32-row group (word ^ 8 group), so that the four groups of eight columns that a warp reads
// fall into different banks.
#include <cuda_runtime.h>

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

// The matrix's scale exponent from its largest finite magnitude (bits): the smallest e >= -126 with max <=
// 2688 2^e; 2688 = 0.65625 x 2^12.
__device__ __forceinline__ int global_exponent(uint32_t top) {
  if (top == 0) return 0;
  const int be = (int)(top >> 23);
  if (be == 0) return -126;                              // below 2^-126
  const int e = be - 126 - 12 + ((top & 0x7fffffu) > 0x280000u ? 1 : 0);   // 0.65625 has the mantissa 1.3125
  return e < -126 ? -126 : e;
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
      for (int e = C / 2; e < (C + N) / 2; ++e) m = __vmaxu2(m, w[e] & 0x7fff7fffu);
      return max(m << 16, m & 0xffff0000u);
    }
  }
};

// Codes (16 bytes) of 32 columns and their scale byte (MX) or two (NV: the second in bits 8-15).
template <bool F32, bool NV>
__device__ __forceinline__ uint32_t quantize32(const Cols32<F32> &v, int eg, uint32_t (&codes)[4]) {
  uint32_t scales = 0;
  if (!NV) {
    const uint32_t top = v.template top<0, 32>();
    const bool bad = top >= 0x7f800000u;
    const uint32_t be = top >> 23;
    const uint32_t s = be > 2 ? be - 2 : 0;            // biased exponent of the scale, 2^-127 at least
    const float inv = __uint_as_float((254u - s) << 23);   // exact: a power of two
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v.get(8 * g + e) * inv;
      const uint32_t c = e2m1x8(x);
      codes[g] = bad ? 0u : c;
    }
    return bad ? 255u : s;
  }
  const float down = power_of_two(-eg);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t top = h == 0 ? v.template top<0, 16>() : v.template top<16, 16>();
    const bool bad = top >= 0x7f800000u;
    const float m = (bad ? 0.f : __uint_as_float(top)) * down;
    const float q6 = __fdiv_rn(m, 6.f);
    const uint32_t sb = to_e4m3(odd(q6, fmaf(-q6, 6.f, m), m));
    const float s = from_e4m3(sb);
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // x / s correctly rounded: one correction of the product with the correctly rounded
        // reciprocal (P. Markstein, "Computation of elementary functions on the IBM RISC
        // System/6000 processor", 1990).  x is x 2^-eg, exact.
        const float a = v.get(16 * h + 8 * g + e) * down;
        float t = a * r;
        t = fmaf(fmaf(-t, s, a), r, t);
        // a bf16 x and its quotient differ from every border or are on it: no remainder can hide
        if (F32 && s > 0.f) t = odd(t, fmaf(-t, s, a), a);
        x[e] = copysignf(t, a);   // the correction of -0 gives +0
      }
      const uint32_t c = e2m1x8(x);
      codes[2 * h + g] = bad ? 0u : c;
    }
    scales |= (bad ? 0x7fu : sb) << (8 * h);
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

template <bool F32, bool NV>
__device__ __forceinline__ void quantize_tile(const Fp4Item &q, int tr, int tk, int eg, uint8_t *stage) {
  const int kc = threadIdx.x & 3, r0 = threadIdx.x >> 2;
  Cols32<F32> v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = tr * kT + r0 + 64 * i;
    load_cols<F32, 32>(q.x, (int64_t)row * q.ld, tk * kT + kc * 32, q.cols, q.flags & kFp4Vec, row < q.rows, v[i].w);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t codes[4];
    const uint32_t s = quantize32<F32, NV>(v[i], eg, codes);
    put<NV>(q, tr, tk, r0 + 64 * i, kc, codes, s, stage);
  }
}

// The tile of the source: rows tk * 128 .. (the 4-bit matrix's columns), columns tr * 128 ...
template <bool F32, bool NV>
__device__ __forceinline__ void quantize_tile_t(const Fp4Item &q, int tr, int tk, int eg, uint8_t *stage, uint32_t *tile) {
  constexpr int WPR = F32 ? 128 : 64;            // words per row of the tile
  constexpr int TPR = WPR / 4;                   // threads per row, 16 bytes each
#pragma unroll
  for (int i = 0; i < kT * TPR / kThreads; ++i) {
    const int r = (int)threadIdx.x / TPR + i * (kThreads / TPR), w = 4 * ((int)threadIdx.x % TPR);
    const int row = tk * kT + r;
    uint32_t v[4];
    load_cols<F32, F32 ? 4 : 8>(q.x, (int64_t)row * q.ld, tr * kT + (F32 ? w : 2 * w), q.rows, q.flags & kFp4Vec,
                                row < q.cols, v);
    *reinterpret_cast<uint4 *>(tile + r * WPR + (w ^ ((r >> 5) << 3))) = make_uint4(v[0], v[1], v[2], v[3]);
  }
  __syncthreads();
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
    const uint32_t s = quantize32<F32, NV>(v, eg, codes);
    put<NV>(q, tr, tk, c, kc, codes, s, stage);
  }
}

template <bool TRANS, int N>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(const __grid_constant__ Fp4Block<N> p) {
  extern __shared__ uint32_t tile[];
  __shared__ __align__(16) uint8_t stage[1024];
  __shared__ uint32_t tops[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const Fp4Item &q = p.item[find_item(p, blockIdx.x)];
  const int l = blockIdx.x - q.tile_begin, tr = l / q.ktiles, tk = l - tr * q.ktiles;
  const bool nv = q.flags & kFp4Nv, f32 = q.flags & kFp4F32;
  int eg = 0;
  if (nv) {
    // the largest magnitude, from the records of the pass before (every CTA for itself)
    uint32_t top = 0;
    for (int i = threadIdx.x; i < q.n_rec; i += kThreads) top = max(top, (uint32_t)p.rec[q.rec_begin + i]);
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, tops[w]);
    eg = global_exponent(top);
    if (l == 0 && threadIdx.x == 0) *q.global = power_of_two(eg);
  }
  if (TRANS) {
    if (nv) f32 ? quantize_tile_t<true, true>(q, tr, tk, eg, stage, tile) : quantize_tile_t<false, true>(q, tr, tk, eg, stage, tile);
    else f32 ? quantize_tile_t<true, false>(q, tr, tk, eg, stage, tile) : quantize_tile_t<false, false>(q, tr, tk, eg, stage, tile);
  } else {
    if (nv) f32 ? quantize_tile<true, true>(q, tr, tk, eg, stage) : quantize_tile<false, true>(q, tr, tk, eg, stage);
    else f32 ? quantize_tile<true, false>(q, tr, tk, eg, stage) : quantize_tile<false, false>(q, tr, tk, eg, stage);
  }
  __syncthreads();
  const int bytes = nv ? 1024 : 512;
  if (threadIdx.x * 4 < bytes)
    reinterpret_cast<uint32_t *>(q.scales + (int64_t)l * bytes)[threadIdx.x] = reinterpret_cast<uint32_t *>(stage)[threadIdx.x];
}

// Values of 32 columns, two rows a thread.
template <int N>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const __grid_constant__ Fp4Block<N> p) {
  pdl_trigger();
  pdl_wait();
  const Fp4Item &q = p.item[find_item(p, blockIdx.x)];
  const int l = blockIdx.x - q.tile_begin, tr = l / q.ktiles, tk = l - tr * q.ktiles;
  const bool nv = q.flags & kFp4Nv, f32 = q.flags & kFp4F32;
  const int kc = threadIdx.x & 3;
  const float g = nv ? *q.global : 1.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (threadIdx.x >> 2) + 64 * i, row = tr * kT + r;
    const int c = tk * kT + kc * 32;
    if (row >= q.rows || c >= q.cols) continue;
    const uint4 u = *reinterpret_cast<const uint4 *>(q.codes + (int64_t)row * q.ktiles * 64 + tk * 64 + kc * 16);
    const int at = 16 * (r & 31) + 4 * (r >> 5);
    float s0, s1;
    if (nv) {
      const uint32_t b = *reinterpret_cast<const unsigned short *>(q.scales + (int64_t)l * 1024 + (kc >> 1) * 512 + at + 2 * (kc & 1));
      s0 = from_e4m3(b & 0xffu);
      s1 = from_e4m3(b >> 8);
    } else {
      s0 = s1 = from_e8m0(q.scales[(int64_t)l * 512 + at + kc]);
    }
    const uint32_t cw[4] = {u.x, u.y, u.z, u.w};
    float y[32];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x[8];
      e2m1x8_to_f32(cw[e], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[8 * e + k] = x[k] * (e < 2 ? s0 : s1) * g;
    }
    const bool whole = (q.flags & kFp4Vec) && c + 32 <= q.cols;
    if (f32) {
      float *d = static_cast<float *>(q.x) + (int64_t)row * q.ld + c;
      if (whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e) reinterpret_cast<float4 *>(d)[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (c + e < q.cols) d[e] = y[e];
      }
    } else {
      __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(q.x) + (int64_t)row * q.ld + c;
      if (whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          reinterpret_cast<uint4 *>(d)[e] = make_uint4(pack_bf16(y[8 * e], y[8 * e + 1]), pack_bf16(y[8 * e + 2], y[8 * e + 3]),
                                                       pack_bf16(y[8 * e + 4], y[8 * e + 5]), pack_bf16(y[8 * e + 6], y[8 * e + 7]));
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (c + e < q.cols) d[e] = __float2bfloat16_rn(y[e]);
      }
    }
  }
}

constexpr int kTileBytesT = kT * 128 * 4;   // an fp32 tile of the transposing kernel

template <int N>
cudaError_t launch_quantize(const Fp4Params &p, bool transpose, cudaStream_t s) {
  const Fp4Block<N> &b = prefix<Fp4Block<N>>(p);
  if (!transpose) return launch_pdl(fp4_quantize_kernel<false, N>, dim3(p.total_tiles), dim3(kThreads), 0, s, b);
  bool f32 = false;
  for (int i = 0; i < p.n; ++i) f32 = f32 || (p.item[i].flags & kFp4F32);
  static PerDevice attr_set;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (f32 && !attr_set.get(dev)) {
    e = cudaFuncSetAttribute(fp4_quantize_kernel<true, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileBytesT);
    if (e != cudaSuccess) return e;
    attr_set.set(dev, 1);
  }
  return launch_pdl(fp4_quantize_kernel<true, N>, dim3(p.total_tiles), dim3(kThreads), f32 ? kTileBytesT : kTileBytesT / 2, s, b);
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4Params &p, bool transpose, cudaStream_t s) {
  if (p.total_tiles <= 0) return cudaSuccess;
  return p.n <= kFewFp4 ? launch_quantize<kFewFp4>(p, transpose, s) : launch_quantize<kMaxFp4>(p, transpose, s);
}

cudaError_t launch_fp4_dequantize(const Fp4Params &p, cudaStream_t s) {
  if (p.total_tiles <= 0) return cudaSuccess;
  if (p.n <= kFewFp4)
    return launch_pdl(fp4_dequantize_kernel<kFewFp4>, dim3(p.total_tiles), dim3(kThreads), 0, s, prefix<Fp4Block<kFewFp4>>(p));
  return launch_pdl(fp4_dequantize_kernel<kMaxFp4>, dim3(p.total_tiles), dim3(kThreads), 0, s, p);
}

}  // namespace nshb

// Norm of a list of tensors taken as one vector, and the list multiplied by a scalar: the
// gradients' global norm and their clipping before an optimizer step.
//
//   norm = sqrt(sum x^2)  or  max |x|;   factor = min(1, max_norm / (norm + 1e-6));   y = factor x
//
// Both are bound by HBM: every element is read once for the norm, and read and written once for
// the scaling.  All tensors of a launch form one line of 16 KB windows, split evenly over the
// CTAs, so that a few vectors and a 12-million-element matrix cost their bytes alone; a CTA
// keeps its sum in registers and reduces it only where its share of a tensor ends.  196 bf16 gradients of
// 1.41 G elements: 396 us (7.1 TB/s of reads); 201 M fp32 elements clipped into bf16: 311 us for the 2.0 GB of
// three passes (6.5 TB/s; the factor is known only when the last element has been read, and 805 MB do not stay
// on the chip).
//
// Short lists are bound by launches: one cluster does all of a call, each CTA as four groups of 256 threads that
// take the place of the CTAs of the long form (tens_small_kernel).
#include <cuda_runtime.h>

#include <type_traits>

#include "nshb_device.cuh"
#include "nshb_internal.h"

namespace nshb {
namespace {

constexpr int kThreads = 256;   // of a group: a CTA of the long form, a quarter of one of the short form

// The threads that work on one share of the line.
struct Group {
  int tid;             // 0 .. 255
  int barrier;         // named barrier of the group
  double *scratch;     // kThreads / 32 doubles
  __device__ __forceinline__ void sync() const { named_barrier(barrier, kThreads); }
};

// The value of one kind over a set: a sum of squares, or the largest magnitude as its bit
// pattern (magnitudes order as their bits; infinity and NaN are the largest).
__device__ __forceinline__ double join(int kind, double a, double b) { return kind == kNormL2 ? a + b : fmax(a, b); }
__device__ __forceinline__ double warp_join(int kind, double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join(kind, v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Every thread gets the value of the whole group (fixed order).
__device__ __forceinline__ double group_join(int kind, double v, const Group &g) {
  v = warp_join(kind, v);
  g.sync();
  if ((g.tid & 31) == 0) g.scratch[g.tid >> 5] = v;
  g.sync();
  double s = g.scratch[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) s = join(kind, s, g.scratch[w]);
  return s;
}

__device__ double join_records(int kind, const double *rec, int n, const Group &g) {
  double v = 0.0;
  for (int i = g.tid; i < n; i += kThreads) v = join(kind, v, rec[i]);
  return group_join(kind, v, g);
}

__device__ __forceinline__ float norm_of(int kind, double v) {
  return kind == kNormL2 ? (float)sqrt(v) : __uint_as_float((uint32_t)v);
}
// Not fminf, which would turn a NaN norm into the factor 1.
__device__ __forceinline__ float factor_of(float norm, float max_norm) {
  if (isinf(norm)) return 0.f;
  const float f = max_norm / (norm + 1e-6f);
  return f > 1.f ? 1.f : f;
}

__device__ __forceinline__ double square(float x) { return (double)x * (double)x; }

// Eight squares are summed in fp32 (four roundings deep) and the sum is carried in fp64; where the
// fp32 sum left the range in which no square can have been lost or have overflowed, the
// eight are summed again in fp64.
struct SumSquares {
  static constexpr bool kOfPairs = false;
  double acc = 0.0;
  __device__ __forceinline__ void add8(const float (&x)[8]) {
    const float a = fmaf(x[0], x[0], x[1] * x[1]), b = fmaf(x[2], x[2], x[3] * x[3]);
    const float c = fmaf(x[4], x[4], x[5] * x[5]), d = fmaf(x[6], x[6], x[7] * x[7]);
    const float s = (a + b) + (c + d);
    if (s > 1e-20f && s < 1e38f) {
      acc += (double)s;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc += square(x[e]);
    }
  }
  __device__ __forceinline__ double value() const { return acc; }
};
template <bool FINITE>
struct LargestBits {
  static constexpr bool kOfPairs = true;
  uint32_t top = 0;
  // Of 32 bf16; false, and nothing done, where one of them is not finite and may not count.
  __device__ __forceinline__ bool add_pairs(const uint32_t (&w)[16]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max_magnitude(m, w[e]);
    m = max(m << 16, m & 0xffff0000u);
    if (FINITE && m >= 0x7f800000u) return false;
    top = top > m ? top : m;
    return true;
  }
  __device__ __forceinline__ void add1(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    if (!FINITE || b < 0x7f800000u) top = top > b ? top : b;
  }
  __device__ __forceinline__ void add8(const float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) add1(x[e]);
  }
  __device__ __forceinline__ double value() const { return (double)top; }
};

template <bool F32>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  if (F32) return static_cast<const float *>(p)[i];
  return bf16lo((uint32_t) static_cast<const unsigned short *>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void store1(void *p, int64_t i, float x) {
  if (F32) static_cast<float *>(p)[i] = x;
  else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

// A thread's share of a window: 64 bytes, E elements.
template <bool F32>
struct Share {
  static constexpr int E = F32 ? 16 : 32;
  uint32_t w[16];
  __device__ __forceinline__ void load(const void *p) {
    uint32_t a[8], b[8];
    ld_global_256(p, a);
    ld_global_256(static_cast<const char *>(p) + 32, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = a[e];
      w[8 + e] = b[e];
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if (F32) return __uint_as_float(w[e]);
    return (e & 1) ? bf16hi(w[e >> 1]) : bf16lo(w[e >> 1]);
  }
};

// Where window `win` of a run puts this thread: the run's row and the first of its E elements
// (negative or past the row's end in the partial windows).
struct Place {
  int row;
  int64_t at;
  bool whole;
};
template <bool F32>
__device__ __forceinline__ Place place(const TensRec &q, int win, int tid) {
  constexpr int E = Share<F32>::E, W = kWinBytes / (F32 ? 4 : 2);
  Place r;
  int k = win;
  r.row = 0;
  if (q.rows > 1) {
    r.row = win / q.per_row;
    k = win - r.row * q.per_row;
  }
  const uintptr_t base = reinterpret_cast<uintptr_t>(q.src) + (uintptr_t)((int64_t)r.row * q.sld * (F32 ? 4 : 2));
  r.at = (int64_t)k * W - (int64_t)((base & 31) / (F32 ? 4 : 2)) + (int64_t)tid * E;
  r.whole = r.at >= 0 && r.at + E <= q.cols;
  return r;
}
template <bool F32>
__device__ __forceinline__ const char *run_ptr(const TensRec &q, const Place &l) {
  return static_cast<const char *>(q.src) + ((int64_t)l.row * q.sld + l.at) * (F32 ? 4 : 2);
}

// A thread's share of a partial window, zeros outside the run: every load under way before the first is used.
template <bool F32>
__device__ __forceinline__ void load_partial(const TensRec &q, const Place &l, float (&x)[Share<F32>::E]) {
  const char *row = static_cast<const char *>(q.src) + (int64_t)l.row * q.sld * (F32 ? 4 : 2);
#pragma unroll
  for (int e = 0; e < Share<F32>::E; ++e)
    x[e] = l.at + e >= 0 && l.at + e < q.cols ? load1<F32>(row, l.at + e) : 0.f;
}

// Walks the elements of a window of short rows, kThreads apart, without a division an element.
struct ShortRows {
  int r, j, dr, dj, cols;
  __device__ __forceinline__ ShortRows(int tid, int cols_)
      : r(tid / cols_), j(tid - tid / cols_ * cols_), dr(kThreads / cols_), dj(kThreads - kThreads / cols_ * cols_), cols(cols_) {}
  __device__ __forceinline__ void next() {
    r += dr;
    j += dj;
    if (j >= cols) {
      j -= cols;
      ++r;
    }
  }
};

template <class V, bool F32, bool TWO>
__device__ __forceinline__ double norm_windows(const TensRec &q, int w, int wend, int tid) {
  V v;
  if (q.flags & kTensRun) {
    auto add = [&](const Share<F32> &s) {
      if constexpr (V::kOfPairs && !F32)
        if (v.add_pairs(s.w)) return;
#pragma unroll
      for (int g = 0; g < Share<F32>::E / 8; ++g) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s.get(8 * g + e);
        v.add8(x);
      }
    };
    auto one = [&](const Place &l) {
      if (l.whole) {
        Share<F32> s;
        s.load(run_ptr<F32>(q, l));
        add(s);
      } else {
        if (l.at + Share<F32>::E <= 0 || l.at >= q.cols) return;
        float x[Share<F32>::E];
        load_partial<F32>(q, l, x);
#pragma unroll
        for (int g = 0; g < Share<F32>::E / 8; ++g) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[8 * g + e];
          v.add8(y);
        }
      }
    };
    // two windows at a time: 128 bytes of each thread in flight
    for (; TWO && w + 1 < wend; w += 2) {
      const Place l0 = place<F32>(q, w, tid), l1 = place<F32>(q, w + 1, tid);
      if (l0.whole && l1.whole) {
        Share<F32> s0, s1;
        s0.load(run_ptr<F32>(q, l0));
        s1.load(run_ptr<F32>(q, l1));
        add(s0);
        add(s1);
      } else {
        one(l0);
        one(l1);
      }
    }
    for (; w < wend; ++w) one(place<F32>(q, w, tid));
  } else {
    for (; w < wend; ++w) {
      const int r0 = w * q.per_row, cols = (int)q.cols;
      const int nr = q.rows - r0 < q.per_row ? q.rows - r0 : q.per_row;
      ShortRows at(tid, cols);
      while (at.r < nr) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e, at.next())
          x[e] = at.r < nr ? load1<F32>(q.src, (int64_t)(r0 + at.r) * q.sld + at.j) : 0.f;
        v.add8(x);
      }
    }
  }
  return v.value();
}

template <class P>
__device__ __forceinline__ int find_tensor(const P &p, int win) {
  int lo = 0, hi = p.ntens - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.t[mid].win_begin <= win) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// CTA c takes windows [c nwin / nctas, (c + 1) nwin / nctas) and writes one record per tensor that
// it meets, at index c + t.  Along the line c + t grows by one at every border of a CTA's share or of a
// tensor; where both borders meet it grows by two, and the record between is set to zero.  So the
// records are a list without gaps in a fixed order, tensor t's are consecutive, and their number does
// not depend on the sizes.
template <class V, bool TWO, class P>
__device__ __forceinline__ void norm_line(const P &p, int c, const Group &g) {
  const int w0 = (int)((int64_t)c * p.nwin / p.nctas), w1 = (int)((int64_t)(c + 1) * p.nwin / p.nctas);
  int t = find_tensor(p, w0);
  for (int w = w0; w < w1; ++t) {
    const TensRec &q = p.t[t];
    const int tend = t + 1 < p.ntens ? p.t[t + 1].win_begin : p.nwin;
    const int wend = tend < w1 ? tend : w1;
    const int a = w - q.win_begin, b = wend - q.win_begin;
    const double v = (q.flags & kTensF32) ? norm_windows<V, true, TWO>(q, a, b, g.tid) : norm_windows<V, false, TWO>(q, a, b, g.tid);
    const double s = group_join(p.kind, v, g);
    if (g.tid == 0) {
      p.rec[c + t] = s;
      if (wend == tend && wend == w1 && t + 1 < p.ntens) p.rec[c + t + 1] = 0.0;
    }
    w = wend;
  }
}

template <bool TWO, class P>
__device__ __forceinline__ void norm_share(const P &p, int c, const Group &g) {
  if (p.kind == kNormL2) norm_line<SumSquares, TWO>(p, c, g);
  else if (p.kind == kNormInf) norm_line<LargestBits<false>, TWO>(p, c, g);
  else norm_line<LargestBits<true>, TWO>(p, c, g);
}

template <int N>
__global__ void __launch_bounds__(kThreads, kTensCtasPerSm) tens_norm_kernel(const __grid_constant__ TensBlock<N> p) {
  __shared__ double scratch[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  norm_share<true>(p, blockIdx.x, Group{(int)threadIdx.x, 1, scratch});
}

// The norms of the tensors, from their records.  A tensor's records are summed by a thread where they are few, by
// a warp otherwise.  at(k): first window and index of tensor k; the last n_empty have no elements.
template <class At>
__device__ __forceinline__ void norms_of_each(int kind, const double *rec, float *each, int ntens, int n_empty, int nwin,
                                              int nctas, int tid, At &&at) {
  const int lane = tid & 31;
  for (int k0 = tid & ~31; k0 < ntens; k0 += kThreads) {
    const int k = k0 + lane;
    int c0 = 0, n = 0;
    if (k < ntens) {
      const int end = k + 1 < ntens ? at(k + 1).win_begin : nwin;
      c0 = win_cta(at(k).win_begin, nwin, nctas);
      n = win_cta(end - 1, nwin, nctas) - c0 + 1;
    }
    double v = 0.0;
    if (n <= 8)
      for (int i = 0; i < n; ++i) v = join(kind, v, rec[c0 + k + i]);
    for (unsigned many = __ballot_sync(0xffffffffu, n > 8); many; many &= many - 1) {
      const int src = __ffs(many) - 1;
      const int first = __shfl_sync(0xffffffffu, c0 + k, src), count = __shfl_sync(0xffffffffu, n, src);
      double s = 0.0;
      for (int i = lane; i < count; i += 32) s = join(kind, s, rec[first + i]);
      s = warp_join(kind, s);
      if (lane == src) v = s;
    }
    if (k < ntens) each[at(k).index] = norm_of(kind, v);
  }
  for (int k = ntens + tid; k < ntens + n_empty; k += kThreads) each[at(k).index] = 0.f;
}

__device__ __forceinline__ float write_total(float *total, uint32_t *status, float norm, float max_norm) {
  const float f = factor_of(norm, max_norm);
  total[0] = norm;
  total[1] = f;
  *status = isfinite(norm) ? 0u : NSHB_DEV_NONFINITE;
  return f;
}

// One CTA: the norms of the tensors (where asked for) and of the whole.
template <int N>
__global__ void __launch_bounds__(kThreads) tens_finalize_kernel(const __grid_constant__ TensFinBlock<N> p) {
  __shared__ double scratch[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  if (p.each)
    norms_of_each(p.kind, p.rec, p.each, p.ntens, p.n_empty, p.nwin, p.nctas, threadIdx.x,
                  [&](int k) -> const TensPlace & { return p.at[k]; });
  double v = join_records(p.kind, p.rec, p.ntens ? p.nctas + p.ntens - 1 : 0, Group{(int)threadIdx.x, 1, scratch});
  if (threadIdx.x == 0) {
    if (!p.first) v = join(p.kind, *p.acc, v);
    if (!p.last) *p.acc = v;
    else write_total(p.total, p.status, norm_of(p.kind, v), p.max_norm);
  }
}

// Stores E = 8 N fp32 values, rounded to the destination's type, with the widest accesses its
// address allows.
template <bool DF32, int E>
__device__ __forceinline__ void store_share(char *d, const float (&y)[E]) {
  constexpr int NW = DF32 ? E : E / 2;
  const uintptr_t a = reinterpret_cast<uintptr_t>(d);
  if ((a & 15) == 0) {
    uint32_t w[NW];
#pragma unroll
    for (int e = 0; e < NW; ++e) w[e] = DF32 ? __float_as_uint(y[e]) : pack_bf16(y[2 * e], y[2 * e + 1]);
    if ((a & 31) == 0) {
#pragma unroll
      for (int g = 0; g < NW / 8; ++g) {
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = w[8 * g + e];
        st_global_256(d + 32 * g, o);
      }
    } else {
#pragma unroll
      for (int g = 0; g < NW / 4; ++g)
        *reinterpret_cast<uint4 *>(d + 16 * g) = make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) store1<DF32>(d, e, y[e]);
  }
}

template <bool F32, bool DF32, bool TWO>
__device__ __forceinline__ void scale_windows(const TensRec &q, int w, int wend, float f, int tid) {
  constexpr int E = Share<F32>::E;
  // backwards: the windows that the norm read last are still in the L2 cache
  if (q.flags & kTensRun) {
    auto out = [&](const Place &l, const Share<F32> &s) {
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = f * s.get(e);
      store_share<DF32, E>(static_cast<char *>(q.dst) + ((int64_t)l.row * q.dld + l.at) * (DF32 ? 4 : 2), y);
    };
    auto one = [&](const Place &l) {
      if (l.whole) {
        Share<F32> s;
        s.load(run_ptr<F32>(q, l));
        out(l, s);
      } else {
        if (l.at + E <= 0 || l.at >= q.cols) return;
        float x[E];
        load_partial<F32>(q, l, x);
        char *drow = static_cast<char *>(q.dst) + (int64_t)l.row * q.dld * (DF32 ? 4 : 2);
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (l.at + e >= 0 && l.at + e < q.cols) store1<DF32>(drow, l.at + e, f * x[e]);
      }
    };
    int u = wend - 1;
    for (; TWO && u > w; u -= 2) {
      const Place l0 = place<F32>(q, u, tid), l1 = place<F32>(q, u - 1, tid);
      if (l0.whole && l1.whole) {
        Share<F32> s0, s1;
        s0.load(run_ptr<F32>(q, l0));
        s1.load(run_ptr<F32>(q, l1));
        out(l0, s0);
        out(l1, s1);
      } else {
        one(l0);
        one(l1);
      }
    }
    for (; u >= w; --u) one(place<F32>(q, u, tid));
  } else {
    for (int u = wend - 1; u >= w; --u) {
      const int r0 = u * q.per_row, cols = (int)q.cols;
      const int nr = q.rows - r0 < q.per_row ? q.rows - r0 : q.per_row;
      ShortRows at(tid, cols);
      while (at.r < nr) {
        float x[8];
        ShortRows to = at;
#pragma unroll
        for (int e = 0; e < 8; ++e, at.next())
          x[e] = at.r < nr ? load1<F32>(q.src, (int64_t)(r0 + at.r) * q.sld + at.j) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e, to.next())
          if (to.r < nr) store1<DF32>(q.dst, (int64_t)(r0 + to.r) * q.dld + to.j, f * x[e]);
      }
    }
  }
}

template <bool TWO, class P>
__device__ __forceinline__ void scale_share(const P &p, int c, float f, int tid) {
  const int w0 = (int)((int64_t)c * p.nwin / p.nctas), w1 = (int)((int64_t)(c + 1) * p.nwin / p.nctas);
  for (int t = find_tensor(p, w1 - 1), w = w1; w > w0; --t) {
    const TensRec &q = p.t[t];
    const int wb = q.win_begin > w0 ? q.win_begin : w0;
    const int a = wb - q.win_begin, b = w - q.win_begin;
    const bool still = f == 1.f && q.src == q.dst;   // in place: the values stay as they are
    if (!still) {
      switch (q.flags & (kTensF32 | kTensDstF32)) {
        case 0: scale_windows<false, false, TWO>(q, a, b, f, tid); break;
        case kTensF32: scale_windows<true, false, TWO>(q, a, b, f, tid); break;
        case kTensDstF32: scale_windows<false, true, TWO>(q, a, b, f, tid); break;
        default: scale_windows<true, true, TWO>(q, a, b, f, tid); break;
      }
    }
    w = wb;
  }
}

// The factor is read, or formed from the norm's records by every CTA for itself (a few KB from L2,
// no launch between the norm and the scaling).
template <int N>
__global__ void __launch_bounds__(kThreads, kTensCtasPerSm) tens_scale_kernel(const __grid_constant__ TensBlock<N> p) {
  __shared__ double scratch[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  float f;
  if (p.coef_rec) {
    const float norm = norm_of(p.kind, join_records(p.kind, p.coef_rec, p.n_rec, Group{(int)threadIdx.x, 1, scratch}));
    f = factor_of(norm, p.max_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) write_total(p.total, p.status, norm, p.max_norm);
  } else {
    f = *p.factor;
  }
  scale_share<true>(p, blockIdx.x, f, threadIdx.x);
}

// All of a call on a short list: one cluster of kSmallCtas CTAs, four groups each.  The records cross between
// the CTAs through the workspace, ordered by the cluster's barrier.
constexpr int kSmallThreads = 4 * kThreads;
__global__ void __launch_bounds__(kSmallThreads, 1) tens_small_kernel(const __grid_constant__ TensSmallParams p) {
  __shared__ double scratch[4][kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int group = threadIdx.x >> 8, c = 4 * (int)cta_rank() + group;
  const Group g{(int)(threadIdx.x & 255), 1 + group, scratch[group]};
  if (c < p.nctas) norm_share<false>(p, c, g);
  cluster_sync();
  const int n_rec = p.ntens ? p.nctas + p.ntens - 1 : 0;
  if (!p.scale) {
    if (c != 0) return;
    if (p.each)
      norms_of_each(p.kind, p.rec, p.each, p.ntens, p.n_empty, p.nwin, p.nctas, g.tid,
                    [&](int k) { return TensPlace{k < p.ntens ? p.t[k].win_begin : p.nwin, p.index[k]}; });
    const double v = join_records(p.kind, p.rec, n_rec, g);
    if (g.tid == 0) write_total(p.total, p.status, norm_of(p.kind, v), p.max_norm);
    return;
  }
  if (c >= p.nctas) return;
  const float norm = norm_of(p.kind, join_records(p.kind, p.rec, n_rec, g));
  if (c == 0 && g.tid == 0) write_total(p.total, p.status, norm, p.max_norm);
  scale_share<false>(p, c, factor_of(norm, p.max_norm), g.tid);
}

}  // namespace

// Calls launch(capacity) with the smallest instance that holds `n` records.
template <class F>
static cudaError_t with_capacity(int n, F &&launch) {
  if (n <= kFewTens) return launch(std::integral_constant<int, kFewTens>());
  if (n <= kSomeTens) return launch(std::integral_constant<int, kSomeTens>());
  return launch(std::integral_constant<int, kMaxTens>());
}

cudaError_t launch_tens_small(const TensSmallParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSmallCtas);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSmallCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tens_small_kernel, p);
}

cudaError_t launch_tens_norm(const TensParams &p, cudaStream_t s) {
  if (p.nwin <= 0) return cudaSuccess;
  return with_capacity(p.ntens, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return launch_pdl(tens_norm_kernel<N>, dim3(p.nctas), dim3(kThreads), 0, s, prefix<TensBlock<N>>(p));
  });
}

cudaError_t launch_tens_finalize(const TensFinParams &p, cudaStream_t s) {
  return with_capacity(p.ntens + p.n_empty, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return launch_pdl(tens_finalize_kernel<N>, dim3(1), dim3(kThreads), 0, s, prefix<TensFinBlock<N>>(p));
  });
}

cudaError_t launch_tens_scale(const TensParams &p, cudaStream_t s) {
  if (p.nwin <= 0) return cudaSuccess;
  return with_capacity(p.ntens, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return launch_pdl(tens_scale_kernel<N>, dim3(p.nctas), dim3(kThreads), 0, s, prefix<TensBlock<N>>(p));
  });
}

}  // namespace nshb

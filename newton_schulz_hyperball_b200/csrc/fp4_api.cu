// C entry points on 4-bit matrices: argument checks and launches.  Host code only.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "../../include/nshb.h"
#include "nshb_internal.h"
#include "tensor_lists.h"

namespace nshb {

nshb_status check_fp4(const nshb_fp4 &q) {
  if (q.rows < 0 || q.cols < 0) return NSHB_ERR_SHAPE;
  if (q.rows > kMaxFp4Dim || q.cols > kMaxFp4Dim) return NSHB_ERR_UNSUPPORTED;
  if (q.format != NSHB_MXFP4 && q.format != NSHB_NVFP4) return NSHB_ERR_DTYPE;
  if (q.reserved != 0) return NSHB_ERR_PARAM;
  if (q.rows == 0 || q.cols == 0) return NSHB_OK;
  if (!q.codes || !q.scales || (q.format == NSHB_NVFP4 && !q.global)) return NSHB_ERR_NULL;
  if ((uintptr_t)q.codes % 16 || (uintptr_t)q.scales % 16) return NSHB_ERR_SHAPE;
  if (q.format == NSHB_NVFP4 && (uintptr_t)q.global % 4) return NSHB_ERR_SHAPE;
  return NSHB_OK;
}

namespace {

// One item; false where the launch would have too many tiles.
bool fill_item(const nshb_fp4 &q, const nshb_tensor &x, int64_t &tiles, Fp4Item &it) {
  const int64_t esz = x.dtype == NSHB_F32 ? 4 : 2, kt = (q.cols + 127) / 128, n = (q.rows + 127) / 128 * kt;
  if (tiles + n > (1LL << 30)) return false;
  it.x = x.data;
  it.codes = static_cast<uint8_t *>(q.codes);
  it.scales = static_cast<uint8_t *>(q.scales);
  it.global = q.global;
  it.ld = x.rows == 1 ? x.cols : x.ld;
  it.rows = (int32_t)q.rows;
  it.cols = (int32_t)q.cols;
  it.ktiles = (int32_t)kt;
  it.tile_begin = (int32_t)tiles;
  const bool vec = (uintptr_t)x.data % 16 == 0 && (x.rows == 1 || (it.ld * esz) % 16 == 0);
  it.flags = (x.dtype == NSHB_F32 ? kFp4F32 : 0) | (q.format == NSHB_NVFP4 ? kFp4Nv : 0) | (vec ? kFp4Vec : 0);
  it.rec_begin = it.n_rec = 0;
  tiles += n;
  return true;
}

// Whether an item's launch has to be another one than `first`'s.
bool another_kind(const nshb_tensor &x, const nshb_fp4 &q, const Fp4Item &first) {
  const int kind = (x.dtype == NSHB_F32 ? kFp4F32 : 0) | (q.format == NSHB_NVFP4 ? kFp4Nv : 0);
  return kind != (first.flags & (kFp4F32 | kFp4Nv));
}

nshb_status check_pairs(const nshb_tensor *x, const nshb_fp4 *q, int32_t n, bool transpose) {
  const nshb_status e = check_tensors(x, n);
  if (e != NSHB_OK) return e;
  if (n > 0 && !q) return NSHB_ERR_NULL;
  for (int32_t i = 0; i < n; ++i) {
    const nshb_status ce = check_fp4(q[i]);
    if (ce != NSHB_OK) return ce;
    if (q[i].rows != (transpose ? x[i].cols : x[i].rows) || q[i].cols != (transpose ? x[i].rows : x[i].cols))
      return NSHB_ERR_SHAPE;
  }
  return NSHB_OK;
}

// The driver's tensor-map encoder, looked up once.
cudaError_t find_encoder(PFN_cuTensorMapEncodeTiled_v12000 *encode) {
  static std::atomic<void *> kept{nullptr};
  void *fn = kept.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    kept.store(fn, std::memory_order_release);
  }
  *encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return cudaSuccess;
}

// Tensor maps of a 4-bit matrix for the products: boxes of `rows` rows of codes and of `row_tiles` row tiles of
// scales, a step of 256 columns wide.
cudaError_t encode_maps(CUtensorMap *codes, CUtensorMap *scales, const nshb_fp4 &q, int rows, int row_tiles) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  const cudaError_t e = find_encoder(&encode);
  if (e != cudaSuccess) return e;
  const cuuint64_t kp = (cuuint64_t)(q.cols + 127) / 128 * 128;
  const bool nv = q.format == NSHB_NVFP4;
  const cuuint32_t ones[3] = {1, 1, 1};
  {
    const cuuint64_t dims[2] = {kp / 2, (cuuint64_t)q.rows};
    const cuuint64_t strides[1] = {kp / 2};
    const cuuint32_t box[2] = {128, (cuuint32_t)rows};
    if (encode(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q.codes, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const cuuint64_t kt = kp / (nv ? 64 : 128), rt = (cuuint64_t)(q.rows + 127) / 128;
  const cuuint64_t dims[3] = {128, kt, rt};
  const cuuint64_t strides[2] = {512, kt * 512};
  const cuuint32_t box[3] = {128, nv ? 4u : 2u, (cuuint32_t)row_tiles};
  if (encode(scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, q.scales, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

// How one product is laid over the GPU.
struct Shape {
  int bn, split;
  bool swap;      // the caller's B takes the accumulator's lanes
  int64_t tiles;
};

// Tiles of bm x bn of a p x q result; of a symmetric one those that reach the diagonal or lie below it.
int64_t count_tiles(int64_t p, int64_t q, int bm, int bn, bool sym) {
  const int64_t pt = (p + bm - 1) / bm, qt = (q + bn - 1) / bn;
  if (!sym) return pt * qt;
  int64_t n = 0;
  for (int64_t i = 0; i < pt; ++i) n += std::min(qt, (i * bm + bm - 1) / bn + 1);
  return n;
}

// pairs: the call has CTA pairs for half of the GPU; narrow: all its tiles, 64 columns wide, fit the GPU at once.
Shape shape_of(int64_t m, int64_t n, int64_t kt, bool sym, bool pairs, bool narrow, int64_t sms) {
  Shape s = {128, 1, false, 0};
  if (pairs && kt > 0 && std::min(m, n) > 128) {
    s.bn = kFp4PairBn;
    s.tiles = count_tiles(m, n, 256, kFp4PairBn, sym);
    return s;
  }
  int64_t p = m, q = n;
  if (!sym && std::min(m, n) <= 64) {
    s.swap = m < n;
    if (s.swap) std::swap(p, q);
    s.bn = q <= 16 ? 16 : q <= 32 ? 32 : 64;
  }
  s.tiles = count_tiles(p, q, 128, s.bn, sym);
  // A step of 256 columns takes a lone CTA 0.3 us, joining the parts of a cluster 2 us (narrow tiles) to 4 us
  // (128 x 128): split long sums of few tiles.  Measured with 1, 2, 4 and 8 CTAs a tile (NVFP4 to bf16, us): 1 x 2048 x 6144
  // 9.5, 7.2, 5.6, 5.4; 64 x 2048 x 6144 11.1, 8.8, 7.0, 7.3; 128 x 2048 x 8192 13.1, 11.8, 8.6, 10.4; but
  // 1 x 6144 x 2048 4.7, 5.2, 5.2, 9.5; 64 x 6144 x 2048 6.3, 6.8, 7.5, 12.5; 1024^3 5.0, 8.2, 9.5, 20.8.
  const bool wide_tile = s.bn == 128;
  if (kt >= (wide_tile ? 32 : 24) && s.tiles * 8 <= (wide_tile ? sms / 2 : sms)) s.split = 8;
  else if (kt >= 16 && s.tiles * 4 <= sms) s.split = 4;
  else if (kt >= (wide_tile ? 32 : 16) && s.tiles * 2 <= sms) s.split = 2;
  // Few tiles without a cluster: half as wide ones spread the epilogue over twice the CTAs.  Measured (128 and 64
  // columns): 1000 x 777 x 1333 to fp32 8.3 and 6.8 us, 768 x 768 x 1000 5.2 and 4.4 us, the Gram matrix of 768 x 1000 7.8 and
  // 5.9 us, 1024^3 to bf16 5.6 and 4.9 us; two CTAs of an SM hide each other's epilogue as well: eight of 512 x 512 x
  // 2048 (256 tiles) 7.9 and 7.0 us, but in two waves 16 of them 9.8 and 14.7 us.
  if (narrow && wide_tile && s.split == 1) {
    s.bn = 64;
    s.tiles = count_tiles(p, q, 128, 64, sym);
  }
  return s;
}

nshb_status check_products(const nshb_fp4 *A, const nshb_fp4 *B, const nshb_tensor *D, int32_t n) {
  const nshb_status e = check_tensors(D, n);
  if (e != NSHB_OK) return e;
  if (n > 0 && !A) return NSHB_ERR_NULL;
  for (int32_t i = 0; i < n; ++i) {
    const nshb_fp4 &a = A[i], &b = B ? B[i] : A[i];
    nshb_status ce = check_fp4(a);
    if (ce == NSHB_OK) ce = check_fp4(b);
    if (ce != NSHB_OK) return ce;
    if (a.format != b.format) return NSHB_ERR_DTYPE;
    if (a.cols != b.cols || D[i].rows != a.rows || D[i].cols != b.rows) return NSHB_ERR_SHAPE;
  }
  return NSHB_OK;
}

}  // namespace

// Products of one launch; `d` as the caller stores it.  See launch_fp4_gemm for what the launches share.
nshb_status run_fp4_products(const nshb_fp4 *A, const nshb_fp4 *B, const nshb_tensor *D, int32_t n, uint32_t *status,
                             bool clear, long long limit, cudaStream_t st) {
  const int64_t sms = device_sms();
  int64_t wide = 0, few = 0;   // tiles of CTA pairs, CTAs with the narrowest tiles in the call
  auto shape = [&](int32_t i, bool pairs, bool narrow) {
    return shape_of(D[i].rows, D[i].cols, (A[i].cols + 255) / 256, !B, pairs, narrow, sms);
  };
  for (int32_t i = 0; i < n; ++i)
    if (D[i].rows && D[i].cols) {
      const Shape s = shape(i, true, false), t = shape(i, false, true);
      wide += s.bn == kFp4PairBn ? s.tiles : 0;
      few += t.tiles * t.split;
    }
  // CTA pairs where their tiles are half as many as the SMs, so that every SM has work.  Measured (single CTAs and pairs):
  // 1024 x 6144 x 2048 (96 pair tiles) 14.6 and 11.9 us, 2304 x 2304 x 2048 (81) 14.0 and 11.4 us, Gram matrices of three
  // 2048 x 8192 inputs (108) 42.4 and 33.6 us; below the border 2048^3 (64) 9.0 and 9.0 us, 1536 x 1536 x 2048 (36) 6.8 and
  // 8.2 us, one such Gram matrix (36) 18.5 and 19.3 us, 1024^3 (16) 4.7 and 7.0 us; but two (72) 24.1 and 21.9 us and
  // 2048 x 2048 x 6144 (64) 17.3 and 14.1 us: for long sums the border is too high.
  const bool pairs = wide >= sms / 2, narrow = few <= 2 * sms;
  // A launch takes the products of one kind (shape and format), wherever they stand in the list: 130 x 140 x 64, 1 x 200 x
  // 300, 40 x 130 x 5000 and 700 x 800 x 256 in turn, eight times, take 23 us, in a launch each 126 us.
  auto log2 = [](int v) {
    int k = 0;
    while (v >>= 1) ++k;
    return k;
  };
  auto kind_of = [&](const Shape &s, int32_t i) {   // bn from 16 to 256, split up to 8
    return 8 * log2(s.bn / 16) + 2 * log2(s.split) + (A[i].format == NSHB_NVFP4);
  };
  uint64_t kinds = 0;
  for (int32_t i = 0; i < n; ++i)
    if (D[i].rows && D[i].cols) kinds |= 1ull << kind_of(shape(i, pairs, narrow), i);
  for (int kind = 0; kinds >> kind; ++kind) {
    if (!(kinds >> kind & 1)) continue;
    for (int32_t i = 0; i < n;) {
      Fp4GemmParams p;
      std::memset(static_cast<Fp4GemmHead *>(&p), 0, sizeof(Fp4GemmHead));
      p.status = status;
      p.wait_limit = limit;
      p.clear_status = clear;
      Shape first = {0, 0, false, 0};
      int32_t format = 0;
      int64_t tiles = 0;
      for (; i < n && p.nprob < kMaxFp4Prob; ++i) {
        const nshb_fp4 &a = A[i], &b = B ? B[i] : A[i];
        if (D[i].rows == 0 || D[i].cols == 0) continue;
        const int64_t kt = (a.cols + 255) / 256;
        const bool sym = !B;
        const Shape s = shape(i, pairs, narrow);
        if (kind_of(s, i) != kind) continue;
        if ((tiles + s.tiles) * s.split > (1LL << 30)) {
          if (p.nprob) break;
          return NSHB_ERR_UNSUPPORTED;
        }
        first = s;
        format = a.format;
        Fp4Prob &q = p.prob[p.nprob++];
        std::memset(&q, 0, sizeof(q));
        const nshb_fp4 &P = s.swap ? b : a, &Q = s.swap ? a : b;
        if (kt) {
          const bool pair = s.bn == kFp4PairBn;
          cudaError_t e = encode_maps(&q.pc, &q.ps, P, 128, 1);
          if (e == cudaSuccess) e = encode_maps(&q.qc, &q.qs, Q, pair ? 128 : s.bn, pair ? 2 : 1);
          if (e != cudaSuccess) {
            record_cuda_error(e);
            return NSHB_ERR_CUDA;
          }
          if (a.format == NSHB_NVFP4) {
            q.pg = P.global;
            q.qg = Q.global;
          }
        }
        const bool f32 = D[i].dtype == NSHB_F32;
        q.d = D[i].data;
        q.ld = D[i].rows == 1 ? D[i].cols : D[i].ld;
        q.np = (int32_t)(s.swap ? D[i].cols : D[i].rows);
        q.nq = (int32_t)(s.swap ? D[i].rows : D[i].cols);
        q.kt = (int32_t)kt;
        q.qtiles = (q.nq + s.bn - 1) / s.bn;
        q.tile_begin = (int32_t)tiles;
        const bool vec = (uintptr_t)D[i].data % 16 == 0 && (D[i].rows == 1 || (q.ld * (f32 ? 4 : 2)) % 16 == 0);
        q.flags = (s.swap ? kFp4DTrans : 0) | (f32 ? kFp4DF32 : 0) | (sym ? kFp4Sym : 0) | (vec ? kFp4DVec : 0);
        tiles += s.tiles;
      }
      if (!p.nprob) break;
      p.total_tiles = (int32_t)tiles;
      NSHB_RUN(NSHB_PROF_FP4, launch_fp4_gemm(p, first.bn, first.split, format == NSHB_NVFP4, st));
      clear = false;
    }
  }
  if (clear) NSHB_RUN(NSHB_PROF_FP4, cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
  return NSHB_OK;
}

}  // namespace nshb

using namespace nshb;

extern "C" {

nshb_status nshb_fp4_size(int64_t rows, int64_t cols, int32_t format, size_t *code_bytes, size_t *scale_bytes) {
  if (!code_bytes || !scale_bytes) return NSHB_ERR_NULL;
  if (rows < 0 || cols < 0) return NSHB_ERR_SHAPE;
  if (rows > kMaxFp4Dim || cols > kMaxFp4Dim) return NSHB_ERR_UNSUPPORTED;
  if (format != NSHB_MXFP4 && format != NSHB_NVFP4) return NSHB_ERR_DTYPE;
  const size_t kp = (size_t)(cols + 127) / 128 * 128, rp = (size_t)(rows + 127) / 128 * 128;
  *code_bytes = (size_t)rows * kp / 2;
  *scale_bytes = rp * kp / (format == NSHB_NVFP4 ? 16 : 32);
  return NSHB_OK;
}

nshb_status nshb_fp4_quantize(const nshb_tensor *X, const nshb_fp4 *Q, int32_t n, int32_t transpose, void *ws,
                              size_t ws_bytes, nshb_stream stream) {
  nshb_status e = check_pairs(X, Q, n, transpose != 0);
  if (e != NSHB_OK) return e;
  bool nv = false;
  for (int32_t i = 0; i < n; ++i) nv = nv || Q[i].format == NSHB_NVFP4;
  if (nv && (e = check_tens_ws(ws, ws_bytes, n)) != NSHB_OK) return e;
  const TensWorkspace w = tens_workspace(ws, n);
  cudaStream_t st = (cudaStream_t)stream;
  for (int32_t i = 0; i < n;) {
    Fp4Params p;
    std::memset(static_cast<Fp4Head *>(&p), 0, sizeof(Fp4Head));
    nshb_tensor src[kMaxFp4];     // the NVFP4 items' sources, whose largest magnitudes come first
    int32_t of[kMaxFp4], n_src = 0;
    int64_t tiles = 0, windows = 0;
    for (; i < n && p.n < kMaxFp4; ++i) {
      if (Q[i].rows == 0 || Q[i].cols == 0) continue;
      if (p.n && another_kind(X[i], Q[i], p.item[0])) break;
      windows += X[i].rows * (X[i].cols / (kWinBytes / 4) + 2);     // of run_largest, at most
      if (p.n && windows > kMaxWindows) break;
      if (!fill_item(Q[i], X[i], tiles, p.item[p.n])) {
        if (p.n == 0) return NSHB_ERR_UNSUPPORTED;
        break;
      }
      if (Q[i].format == NSHB_NVFP4) {
        of[n_src] = p.n;
        src[n_src++] = X[i];
      }
      ++p.n;
    }
    p.total_tiles = (int32_t)tiles;
    p.rec = w.rec;
    if (n_src) {
      int32_t rec_begin[kMaxFp4], n_rec[kMaxFp4];
      e = run_largest(src, n_src, w, st, rec_begin, n_rec);
      if (e != NSHB_OK) return e;
      for (int32_t k = 0; k < n_src; ++k) {
        p.item[of[k]].rec_begin = rec_begin[k];
        p.item[of[k]].n_rec = n_rec[k];
      }
    }
    NSHB_RUN(NSHB_PROF_FP4, launch_fp4_quantize(p, transpose != 0, st));
  }
  return NSHB_OK;
}

nshb_status nshb_fp4_dequantize(const nshb_fp4 *Q, const nshb_tensor *X, int32_t n, nshb_stream stream) {
  const nshb_status e = check_pairs(X, Q, n, false);
  if (e != NSHB_OK) return e;
  cudaStream_t st = (cudaStream_t)stream;
  for (int32_t i = 0; i < n;) {
    Fp4Params p;
    std::memset(static_cast<Fp4Head *>(&p), 0, sizeof(Fp4Head));
    int64_t tiles = 0;
    for (; i < n && p.n < kMaxFp4; ++i) {
      if (Q[i].rows == 0 || Q[i].cols == 0) continue;
      if (p.n && another_kind(X[i], Q[i], p.item[0])) break;
      if (!fill_item(Q[i], X[i], tiles, p.item[p.n])) {
        if (p.n == 0) return NSHB_ERR_UNSUPPORTED;
        break;
      }
      ++p.n;
    }
    p.total_tiles = (int32_t)tiles;
    NSHB_RUN(NSHB_PROF_FP4, launch_fp4_dequantize(p, st));
  }
  return NSHB_OK;
}

nshb_status nshb_fp4_matmul(const nshb_fp4 *A, const nshb_fp4 *B, const nshb_tensor *D, int32_t n, void *ws,
                            size_t ws_bytes, nshb_stream stream) {
  nshb_status e = check_products(A, B, D, n);
  if (e != NSHB_OK) return e;
  e = check_tens_ws(ws, ws_bytes, n);
  if (e != NSHB_OK) return e;
  return run_fp4_products(A, B, D, n, static_cast<uint32_t *>(ws), /*clear=*/true, kFp4WaitLimit, (cudaStream_t)stream);
}

}  // extern "C"

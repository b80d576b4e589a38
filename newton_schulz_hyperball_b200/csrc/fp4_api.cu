// C entry points on 4-bit matrices: argument checks and launches.  Host code only.
#include <cuda_runtime.h>

#include <algorithm>
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

}  // namespace
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
    std::memset(&p, 0, offsetof(Fp4Params, item));
    nshb_tensor src[kMaxFp4];     // the NVFP4 items' sources, whose largest magnitudes come first
    int32_t of[kMaxFp4], n_src = 0;
    int64_t tiles = 0;
    for (; i < n && p.n < kMaxFp4; ++i) {
      if (Q[i].rows == 0 || Q[i].cols == 0) continue;
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
    std::memset(&p, 0, offsetof(Fp4Params, item));
    int64_t tiles = 0;
    for (; i < n && p.n < kMaxFp4; ++i) {
      if (Q[i].rows == 0 || Q[i].cols == 0) continue;
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

}  // extern "C"

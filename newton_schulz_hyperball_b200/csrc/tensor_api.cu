// C entry points on lists of tensors: argument checks, workspace layout and launches.  Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/nshb.h"
#include "nshb_internal.h"
#include "tensor_lists.h"

namespace nshb {

// Sizes, limits, dtype, pointer and alignment of one tensor, in this order.
nshb_status check_tensor(const nshb_tensor &t) {
  if (t.rows < 0 || t.cols < 0 || (t.rows > 1 && t.ld < t.cols)) return NSHB_ERR_SHAPE;
  if (t.rows > (1LL << 40) || t.cols > (1LL << 40) || (t.rows > 1 && t.ld > (1LL << 40))) return NSHB_ERR_UNSUPPORTED;
  if (t.dtype != NSHB_BF16 && t.dtype != NSHB_F32) return NSHB_ERR_DTYPE;
  if (t.reserved != 0) return NSHB_ERR_PARAM;
  if (t.rows == 0 || t.cols == 0) return NSHB_OK;
  // rows * cols and the last element's offset, without overflow: both factors are at most 2^40
  if (t.rows > (1LL << 40) / t.cols) return NSHB_ERR_UNSUPPORTED;
  if (t.rows > 1 && t.rows > (1LL << 44) / t.ld) return NSHB_ERR_UNSUPPORTED;
  if (t.rows > kMaxRuns && t.ld != t.cols) return NSHB_ERR_UNSUPPORTED;
  if (!t.data) return NSHB_ERR_NULL;
  if ((uintptr_t)t.data % (t.dtype == NSHB_F32 ? 4 : 2)) return NSHB_ERR_SHAPE;
  return NSHB_OK;
}

nshb_status check_tensors(const nshb_tensor *t, int32_t n) {
  if (n < 0) return NSHB_ERR_SHAPE;
  if (n > 0 && !t) return NSHB_ERR_NULL;
  for (int32_t i = 0; i < n; ++i) {
    const nshb_status e = check_tensor(t[i]);
    if (e != NSHB_OK) return e;
  }
  return NSHB_OK;
}

TensWorkspace tens_workspace(void *ws, int32_t n) {
  TensWorkspace w;
  char *c = static_cast<char *>(ws);
  w.status = reinterpret_cast<uint32_t *>(c);
  w.acc = reinterpret_cast<double *>(c + 64);
  w.rec = reinterpret_cast<double *>(c + 256);
  const size_t per = std::min<size_t>((size_t)std::max(n, 0), kMaxTens);
  w.bytes = (256 + sizeof(double) * (per + kMaxTensCtas) + 255) / 256 * 256;
  return w;
}

nshb_status check_tens_ws(void *ws, size_t bytes, int32_t n) {
  if (!ws) return NSHB_ERR_NULL;
  if ((uintptr_t)ws % 256 != 0 || bytes < tens_workspace(nullptr, n).bytes) return NSHB_ERR_WORKSPACE;
  return NSHB_OK;
}

int tens_ctas(int nwin) { return std::min(nwin, std::min(kTensCtasPerSm * device_sms(), kMaxTensCtas)); }

namespace {

// One tensor's record: a contiguous tensor is one run whatever its shape.  False where the launch would have too
// many windows; never for its first tensor (up to 2^30 rows of one window, 2^28 of two, and so on).
bool fill(const nshb_tensor &s, const nshb_tensor *d, int64_t &win, TensRec &q) {
  const int64_t esz = s.dtype == NSHB_F32 ? 4 : 2, per = kWinBytes / esz;
  int64_t rows = s.rows, cols = s.cols;
  const bool flat = rows == 1 || (s.ld == cols && (!d || d->ld == cols));
  if (flat) {
    cols *= rows;
    rows = 1;
  }
  q.src = s.data;
  q.dst = d ? d->data : nullptr;
  q.cols = cols;
  q.sld = flat ? cols : s.ld;
  q.dld = flat ? cols : (d ? d->ld : 0);
  q.flags = (s.dtype == NSHB_F32 ? kTensF32 : 0) | (d && d->dtype == NSHB_F32 ? kTensDstF32 : 0);
  q.win_begin = (int32_t)win;
  int64_t n;
  if (rows == 1 || cols >= kLongRow) {
    q.flags |= kTensRun;
    // the alignment of a row decides where its windows begin; several rows take the worst case
    const int64_t lead = rows == 1 ? (int64_t)((uintptr_t)s.data % 32) / esz : 32 / esz - 1;
    q.per_row = (int32_t)((cols + lead + per - 1) / per);
    n = rows * q.per_row;
  } else {
    q.per_row = (int32_t)(per / cols);
    n = (rows + q.per_row - 1) / q.per_row;
  }
  if (win + n > kMaxWindows) return false;
  q.rows = (int32_t)rows;
  win += n;
  return true;
}

// Fills the records of tensors from `i` on, as many as one launch takes; `i` is moved past them.
// index/win_begin/empties (when given) receive what the finalize kernel needs.
void fill_launch(const nshb_tensor *src, const nshb_tensor *dst, int32_t n, int32_t &i, TensParams &p, TensFinParams *fin) {
  int64_t win = 0;
  int32_t seen = 0;
  int32_t empty[kMaxTens];
  int32_t n_empty = 0;
  p.ntens = 0;
  for (; i < n && seen < kMaxTens; ++i, ++seen) {
    if (src[i].rows == 0 || src[i].cols == 0) {
      empty[n_empty++] = i;
      continue;
    }
    if (!fill(src[i], dst ? &dst[i] : nullptr, win, p.t[p.ntens])) break;
    if (fin) {
      fin->at[p.ntens].index = i;
      fin->at[p.ntens].win_begin = p.t[p.ntens].win_begin;
    }
    ++p.ntens;
  }
  p.nwin = (int32_t)win;
  p.nctas = tens_ctas(p.nwin);
  if (fin) {
    for (int32_t k = 0; k < n_empty; ++k) fin->at[p.ntens + k] = {p.nwin, empty[k]};
    fin->ntens = p.ntens;
    fin->n_empty = n_empty;
    fin->nwin = p.nwin;
    fin->nctas = p.nctas;
  }
}

// The whole call in one launch where the list is short.  Otherwise *done stays false and nothing is queued.
nshb_status run_small(const nshb_tensor *src, const nshb_tensor *dst, int32_t n, int32_t kind, float max_norm, float *total,
                      float *each, bool scale, const TensWorkspace &w, cudaStream_t st, bool *done) {
  *done = false;
  if (n > kSmallWindows) return NSHB_OK;
  int64_t bytes = 0;   // windows are of 16 KB at most: a quick bound before the records are made
  for (int32_t i = 0; i < n; ++i) {
    bytes += src[i].rows * src[i].cols * (src[i].dtype == NSHB_F32 ? 4 : 2);
    if (bytes > (int64_t)kSmallWindows * kWinBytes) return NSHB_OK;
  }
  TensSmallParams p;
  static_cast<TensSmallHead &>(p) = TensSmallHead{};
  int64_t win = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (src[i].rows == 0 || src[i].cols == 0) continue;
    const nshb_tensor *d = scale ? (dst ? &dst[i] : &src[i]) : nullptr;
    if (!fill(src[i], d, win, p.t[p.ntens]) || win > (scale ? kSmallClipWindows : kSmallWindows)) return NSHB_OK;
    p.index[p.ntens++] = i;
  }
  for (int32_t i = 0; i < n; ++i)
    if (src[i].rows == 0 || src[i].cols == 0) p.index[p.ntens + p.n_empty++] = i;
  p.nwin = (int32_t)win;
  p.nctas = std::min(p.nwin, 4 * kSmallCtas);
  p.rec = w.rec;
  p.total = total;
  p.status = w.status;
  p.max_norm = max_norm;
  p.kind = kind;
  p.each = each;
  p.scale = scale;
  *done = true;
  NSHB_RUN(NSHB_PROF_GRAD, launch_tens_small(p, st));
  return NSHB_OK;
}

// Norm launches over the whole list.  `one` (optional): where the list fits one launch, its records are left
// for the caller, who forms the norm itself (no finalize kernel).
nshb_status run_norm(const nshb_tensor *g, int32_t n, int32_t kind, float max_norm, float *total, float *each,
                     const TensWorkspace &w, cudaStream_t st, int32_t *n_rec) {
  int32_t i = 0;
  bool first = true;
  do {
    TensParams p;
    std::memset(static_cast<TensHead *>(&p), 0, sizeof(TensHead));
    TensFinParams f;
    std::memset(static_cast<TensFinHead *>(&f), 0, sizeof(TensFinHead));
    fill_launch(g, nullptr, n, i, p, &f);
    p.rec = w.rec;
    p.kind = kind;
    NSHB_RUN(NSHB_PROF_GRAD, launch_tens_norm(p, st));
    if (n_rec && first && i == n) {
      *n_rec = p.ntens ? p.nctas + p.ntens - 1 : 0;
      return NSHB_OK;
    }
    f.rec = w.rec;
    f.acc = w.acc;
    f.total = total;
    f.each = each;
    f.status = w.status;
    f.max_norm = max_norm;
    f.kind = kind;
    f.first = first;
    f.last = i == n;
    NSHB_RUN(NSHB_PROF_GRAD, launch_tens_finalize(f, st));
    first = false;
  } while (i < n);
  if (n_rec) *n_rec = -1;
  return NSHB_OK;
}

nshb_status run_scale(const nshb_tensor *src, const nshb_tensor *dst, int32_t n, const float *factor, int32_t kind,
                      float max_norm, float *total, const TensWorkspace *w, int32_t n_rec, cudaStream_t st) {
  for (int32_t i = 0; i < n;) {
    TensParams p;
    std::memset(static_cast<TensHead *>(&p), 0, sizeof(TensHead));
    fill_launch(src, dst ? dst : src, n, i, p, nullptr);
    p.factor = factor;
    if (w && n_rec >= 0) {
      p.coef_rec = w->rec;
      p.n_rec = n_rec;
      p.total = total;
      p.status = w->status;
    }
    p.kind = kind;
    p.max_norm = max_norm;
    NSHB_RUN(NSHB_PROF_GRAD, launch_tens_scale(p, st));
  }
  return NSHB_OK;
}

}  // namespace

nshb_status run_largest(const nshb_tensor *t, int32_t n, const TensWorkspace &w, cudaStream_t st, int32_t *rec_begin,
                        int32_t *n_rec) {
  int32_t i = 0;
  TensParams p;
  std::memset(static_cast<TensHead *>(&p), 0, sizeof(TensHead));
  fill_launch(t, nullptr, n, i, p, nullptr);
  p.rec = w.rec;
  p.kind = kNormFinite;
  for (int k = 0; k < p.ntens; ++k) {
    const int end = k + 1 < p.ntens ? p.t[k + 1].win_begin : p.nwin;
    const int c0 = win_cta(p.t[k].win_begin, p.nwin, p.nctas), c1 = win_cta(end - 1, p.nwin, p.nctas);
    rec_begin[k] = c0 + k;
    n_rec[k] = c1 - c0 + 1;
  }
  NSHB_RUN(NSHB_PROF_FP4, launch_tens_norm(p, st));
  return NSHB_OK;
}

namespace {

nshb_status check_norm_args(const nshb_tensor *g, int32_t n, int32_t kind, float max_norm, const float *total) {
  const nshb_status e = check_tensors(g, n);
  if (e != NSHB_OK) return e;
  if (!total) return NSHB_ERR_NULL;
  if ((uintptr_t)total % sizeof(float)) return NSHB_ERR_SHAPE;
  if (kind != NSHB_NORM_L2 && kind != NSHB_NORM_INF) return NSHB_ERR_PARAM;
  if (!(max_norm > 0.f)) return NSHB_ERR_PARAM;   // a NaN too
  return NSHB_OK;
}

// dst of a scaling: the sizes of src, and in place only with src's layout.
nshb_status check_dst(const nshb_tensor *src, const nshb_tensor *dst, int32_t n) {
  if (!dst) return NSHB_OK;
  const nshb_status e = check_tensors(dst, n);
  if (e != NSHB_OK) return e;
  for (int32_t i = 0; i < n; ++i) {
    const nshb_tensor &s = src[i], &d = dst[i];
    if (s.rows != d.rows || s.cols != d.cols) return NSHB_ERR_SHAPE;
    if (s.rows == 0 || s.cols == 0 || s.data != d.data) continue;
    if (s.dtype != d.dtype || (s.rows > 1 && s.ld != d.ld)) return NSHB_ERR_PARAM;
  }
  return NSHB_OK;
}

bool has_elements(const nshb_tensor *t, int32_t n) {
  for (int32_t i = 0; i < n; ++i)
    if (t[i].rows > 0 && t[i].cols > 0) return true;
  return false;
}

}  // namespace
}  // namespace nshb

using namespace nshb;

extern "C" {

nshb_status nshb_tensor_workspace_size(const nshb_tensor *t, int32_t n, size_t *bytes) {
  if (!bytes) return NSHB_ERR_NULL;
  const nshb_status e = check_tensors(t, n);
  if (e != NSHB_OK) return e;
  *bytes = tens_workspace(nullptr, n).bytes;
  return NSHB_OK;
}

nshb_status nshb_grad_norm(const nshb_tensor *g, int32_t n, int32_t kind, float max_norm, float *total, float *each,
                           void *ws, size_t ws_bytes, nshb_stream stream) {
  nshb_status e = check_norm_args(g, n, kind, max_norm, total);
  if (e != NSHB_OK) return e;
  if ((uintptr_t)each % sizeof(float)) return NSHB_ERR_SHAPE;
  e = check_tens_ws(ws, ws_bytes, n);
  if (e != NSHB_OK) return e;
  const TensWorkspace w = tens_workspace(ws, n);
  bool done;
  e = run_small(g, nullptr, n, kind, max_norm, total, each, /*scale=*/false, w, (cudaStream_t)stream, &done);
  if (e != NSHB_OK || done) return e;
  return run_norm(g, n, kind, max_norm, total, each, w, (cudaStream_t)stream, nullptr);
}

nshb_status nshb_clip_grads(const nshb_tensor *src, const nshb_tensor *dst, int32_t n, int32_t kind, float max_norm,
                            float *total, void *ws, size_t ws_bytes, nshb_stream stream) {
  nshb_status e = check_norm_args(src, n, kind, max_norm, total);
  if (e != NSHB_OK) return e;
  e = check_dst(src, dst, n);
  if (e != NSHB_OK) return e;
  e = check_tens_ws(ws, ws_bytes, n);
  if (e != NSHB_OK) return e;
  const TensWorkspace w = tens_workspace(ws, n);
  cudaStream_t st = (cudaStream_t)stream;
  bool done;
  e = run_small(src, dst, n, kind, max_norm, total, nullptr, /*scale=*/has_elements(src, n), w, st, &done);
  if (e != NSHB_OK || done) return e;
  if (!has_elements(src, n)) return run_norm(src, n, kind, max_norm, total, nullptr, w, st, nullptr);
  int32_t n_rec = -1;
  e = run_norm(src, n, kind, max_norm, total, nullptr, w, st, &n_rec);
  if (e != NSHB_OK) return e;
  return run_scale(src, dst, n, total + 1, kind, max_norm, total, &w, n_rec, st);
}

nshb_status nshb_scale_grads(const nshb_tensor *src, const nshb_tensor *dst, int32_t n, const float *factor,
                             nshb_stream stream) {
  nshb_status e = check_tensors(src, n);
  if (e != NSHB_OK) return e;
  if (!factor) return NSHB_ERR_NULL;
  if ((uintptr_t)factor % sizeof(float)) return NSHB_ERR_SHAPE;
  e = check_dst(src, dst, n);
  if (e != NSHB_OK) return e;
  return run_scale(src, dst, n, factor, NSHB_NORM_L2, 1.f, nullptr, nullptr, -1, (cudaStream_t)stream);
}

}  // extern "C"

// What the entry points on lists of tensors share (host side).
#pragma once
#include <cstddef>

#include "../../include/nshb.h"
#include "nshb_internal.h"

#define NSHB_RUN(kind, call)                          \
  do {                                                \
    const ::nshb::ProfEvent pe_ = ::nshb::prof_begin(st); \
    const cudaError_t e_ = (call);                    \
    ::nshb::prof_end(pe_, kind, st);                  \
    if (e_ != cudaSuccess) {                          \
      ::nshb::record_cuda_error(e_);                  \
      return NSHB_ERR_CUDA;                           \
    }                                                 \
  } while (0)

namespace nshb {

constexpr int64_t kMaxRuns = 1LL << 30;   // rows that do not follow one another
constexpr int64_t kMaxWindows = 1LL << 30;   // of a launch
constexpr int kMaxTensCtas = 1024;   // records per launch: at most this many CTAs + kMaxTens

// The workspace of a call on a list of tensors: [0, 256) the status word and the running value of
// a norm that takes several launches, then the records of one launch.
struct TensWorkspace {
  uint32_t *status;
  double *acc;
  double *rec;
  size_t bytes;
};
TensWorkspace tens_workspace(void *ws, int32_t n);
nshb_status check_tens_ws(void *ws, size_t bytes, int32_t n);
nshb_status check_tensor(const nshb_tensor &t);
nshb_status check_tensors(const nshb_tensor *t, int32_t n);
int tens_ctas(int nwin);
// The largest finite magnitude of each of up to kMaxTens tensors with elements and kMaxWindows windows, left as
// records: tensor k's are w.rec[rec_begin[k]] .. [+ n_rec[k]), each the bits of a magnitude as a double.
nshb_status run_largest(const nshb_tensor *t, int32_t n, const TensWorkspace &w, cudaStream_t st, int32_t *rec_begin,
                        int32_t *n_rec);
constexpr int64_t kMaxFp4Dim = 1LL << 24;
nshb_status check_fp4(const nshb_fp4 &q);
constexpr long long kFp4WaitLimit = 4000000000LL;   // ~2 s of SM clock per barrier phase
// D[i] = A[i] B[i]^T (B NULL: A[i] A[i]^T) for checked arguments.
nshb_status run_fp4_products(const nshb_fp4 *A, const nshb_fp4 *B, const nshb_tensor *D, int32_t n, uint32_t *status,
                             bool clear, long long limit, cudaStream_t st);

}  // namespace nshb

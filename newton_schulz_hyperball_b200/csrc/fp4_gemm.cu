// Products of microscaled 4-bit matrices on the 5th-generation tensor cores:
//
//   D = gP gQ  sum_k (code_P scale_P)(code_Q scale_Q)      (tcgen05.mma kind::mxf4nvf4, fp32 accumulator)
//
// The codes go from memory to the tensor core as they are stored: one 128-byte box holds 256
// columns of a row.  The scales of a step (512-byte tiles, see nshb_fp4) are loaded next to the
// codes and copied into tensor memory by tcgen05.cp, which the same thread issues ahead of the MMAs that
// read them (the two run in order).  The load and MMA warps stay converged and elect a lane to issue: see
// elect_one.
//
// One CTA computes 128 rows of P x BN rows of Q.  Few rows on one side (single tokens) are bound by
// the bytes of the other operand: that one takes the 128 lanes, BN is as small as the rows allow,
// and a cluster of up to 8 CTAs shares the columns of a tile whose sum is long, each summing its part; the parts are
// joined through distributed shared memory in a fixed order.  One token through 6144 x 2048 NVFP4: 4.8 us for 7.1 MB,
// bound by latency: 48 CTAs, each with 5 of its 8 steps of loads under way at once (a ring of 110 KB, so that larger
// calls have two CTAs on an SM).
//
// Enough 256 x 256 tiles to fill the GPU go to CTA pairs (fp4_pair_kernel): a pair reads 64 bytes of
// codes per clock and SM for the work that single CTAs with 128 x 128 tiles need 128 for.
//
// Roles of the single CTA (320 threads): warp 0 issues the loads of the ring, warp 1 the copies and MMAs, warps
// 2-9 drain the accumulator.  Every wait is bounded.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "nshb_device.cuh"
#include "nshb_internal.h"

namespace nshb {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kTimeoutBit = 0x4u;

template <int BN, bool NV>
struct Cfg {
  static constexpr int kSTiles = NV ? 4 : 2;                 // 512-byte scale tiles of a step and 128 rows
  static constexpr int kPBytes = 128 * 128, kQBytes = BN * 128;
  static constexpr int kPs = kSTiles * 512, kQs = kSTiles * 512;
  static constexpr int kStage = kPBytes + kQBytes + kPs + kQs;   // a multiple of 1024
  // two CTAs on an SM
  static constexpr int kStages = 110 * 1024 / kStage;
  static constexpr int kSmem = kStages * kStage + 1024 + 256;
  static constexpr int kPsCol = BN < 32 ? 32 : BN;           // TMEM columns: accumulator, P's scales, Q's
  static constexpr int kQsCol = kPsCol + 4 * kSTiles;
  static constexpr int kUsed = kQsCol + 4 * kSTiles;
  static constexpr int kTmem = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : 256;
  static_assert(kStage % 1024 == 0, "every stage starts on a swizzle atom");
  static_assert((128 + 64) * (BN + 4) * 4 <= kStages * kStage, "the partial sums and half a tile fit the ring");
};

template <class P>
__device__ __forceinline__ int find_prob(const P &p, int tile) {
  int lo = 0, hi = p.nprob - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.prob[mid].tile_begin <= tile) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tile l of a problem: its P and Q tile; of a symmetric result those that reach the diagonal or lie below it.
template <int BM, int BN>
__device__ __forceinline__ void tile_of(const Fp4Prob &q, int l, int &pt, int &qt) {
  if (q.flags & kFp4Sym) {
    for (pt = 0;; ++pt) {
      const int n = min(q.qtiles, (pt * BM + BM - 1) / BN + 1);
      if (l < n) break;
      l -= n;
    }
    qt = l;
  } else {
    pt = l / q.qtiles;
    qt = l - pt * q.qtiles;
  }
}

// What the accumulator's elements are multiplied with: the product of the matrices' scales, or where that
// leaves fp32's normal range (scales near 2^-77, 2^70) both one after the other, the larger first, so that nothing that
// D can hold is lost and no zero becomes 0 x infinity.  The second is read again where it is needed: the epilogue has no
// register for it.
struct MatrixScales {
  float a = 1.f;
  bool two = false;
  __device__ __forceinline__ explicit MatrixScales(const Fp4Prob &q) {
    if (!q.pg) return;
    const float x = *q.pg, y = *q.qg;
    a = x * y;
    two = !(isfinite(a) && (fabsf(a) >= 0x1p-126f || x == 0.f || y == 0.f));
    if (two) a = fabsf(x) >= fabsf(y) ? x : y;
  }
  template <int N>
  __device__ __forceinline__ void apply(const Fp4Prob &q, float (&v)[N]) const {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] *= a;
    if (two) {
      const float x = *q.pg, y = *q.qg, b = fabsf(x) >= fabsf(y) ? y : x;
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] *= b;
    }
  }
};

// N values of D: row p, columns q0 .. q0 + N - 1 of the tile's orientation.
template <int N>
__device__ __forceinline__ void store_row(const Fp4Prob &q, int64_t p, int64_t q0, const float (&v)[N], bool trans) {
  if (p >= q.np) return;
  const bool f32 = q.flags & kFp4DF32;
  if (trans) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (q0 + e >= q.nq) break;
      const int64_t at = (q0 + e) * q.ld + p;
      if (f32) static_cast<float *>(q.d)[at] = v[e];
      else static_cast<__nv_bfloat16 *>(q.d)[at] = __float2bfloat16_rn(v[e]);
    }
    return;
  }
  const int64_t at = p * q.ld + q0;
  if (N >= 8 && (q.flags & kFp4DVec) && q0 + N <= q.nq) {
    if (f32) {
      float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(q.d) + at);
#pragma unroll
      for (int e = 0; e < N / 4; ++e) d[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
    } else {
      uint4 *d = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(q.d) + at);
#pragma unroll
      for (int e = 0; e < N / 8; ++e)
        d[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                          pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (q0 + e >= q.nq) break;
    if (f32) static_cast<float *>(q.d)[at + e] = v[e];
    else static_cast<__nv_bfloat16 *>(q.d)[at + e] = __float2bfloat16_rn(v[e]);
  }
}

// A warp's 32 rows x 32 columns of D (lane l holds row l) through 2 KB of shared memory, so that a store
// instruction covers whole 64-byte pieces of rows: with a row per lane each of its 32 lines takes the
// load/store unit a turn of its own, and the warps that feed the tensor core wait behind it.
__device__ __forceinline__ void store_block(const Fp4Prob &q, uint8_t *stage, int64_t row0, int64_t c, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  const bool f32 = q.flags & kFp4DF32;
  const int rows = (int)(q.np - row0 < 32 ? q.np - row0 : 32), cols = (int)(q.nq - c < 32 ? q.nq - c : 32);
  if (rows <= 0 || cols <= 0) return;
  const int esz = f32 ? 4 : 2, wide = 64 / esz;      // columns of a pass
  const int64_t pitch = q.ld * esz;
  char *d = static_cast<char *>(q.d) + (row0 * q.ld + c) * esz;
  uint8_t *mine = stage + lane * 64;
  const int turn = (lane >> 1) & 3;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1 && !f32) break;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint4 w;
      if (f32)
        w = make_uint4(__float_as_uint(v[16 * pass + 4 * k]), __float_as_uint(v[16 * pass + 4 * k + 1]),
                       __float_as_uint(v[16 * pass + 4 * k + 2]), __float_as_uint(v[16 * pass + 4 * k + 3]));
      else
        w = make_uint4(pack_bf16(v[8 * k], v[8 * k + 1]), pack_bf16(v[8 * k + 2], v[8 * k + 3]),
                       pack_bf16(v[8 * k + 4], v[8 * k + 5]), pack_bf16(v[8 * k + 6], v[8 * k + 7]));
      *reinterpret_cast<uint4 *>(mine + ((k ^ turn) << 4)) = w;
    }
    __syncwarp();
    const int have = cols - pass * wide < wide ? cols - pass * wide : wide;
    char *dp = d + 64 * pass;
    if ((q.flags & kFp4DVec) && have == wide) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2), k = lane & 3;
        const uint4 w = *reinterpret_cast<const uint4 *>(stage + r * 64 + ((k ^ ((r >> 1) & 3)) << 4));
        if (r < rows) *reinterpret_cast<uint4 *>(dp + r * pitch + 16 * k) = w;
      }
    } else if (f32) {
      // two rows at a time
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4), e = lane & 15;
        if (r < rows && e < have)
          *reinterpret_cast<uint32_t *>(dp + r * pitch + 4 * e) =
              *reinterpret_cast<const uint32_t *>(stage + r * 64 + (((e >> 2) ^ ((r >> 1) & 3)) << 4) + 4 * (e & 3));
      }
    } else {
#pragma unroll 8
      for (int r = 0; r < rows; ++r)
        if (lane < have)
          *reinterpret_cast<unsigned short *>(dp + r * pitch + 2 * lane) =
              *reinterpret_cast<const unsigned short *>(stage + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + 2 * (lane & 7));
    }
  }
}

// Such a block of a symmetric result; row0 and c are multiples of 32.  Blocks below the diagonal are stored with
// their mirror image, those above it not at all, of those on it the elements up to the diagonal with theirs: each
// element of D has one writer, and (i, j) has the bits of (j, i).
__device__ __forceinline__ void store_symmetric(const Fp4Prob &q, uint8_t *stage, int64_t row0, int64_t c, const float (&v)[32]) {
  if (c > row0) return;
  const bool on = c == row0;
  if (!on) store_block(q, stage, row0, c, v);
  const int64_t row = row0 + (threadIdx.x & 31);
  if (row >= q.np) return;
  const int n = on ? (int)(row - c) : 32;              // the elements below the diagonal
  if (q.flags & kFp4DF32) {
    float *d = static_cast<float *>(q.d) + c * q.ld + row, *r = static_cast<float *>(q.d) + row * q.ld + c;
#pragma unroll
    for (int e = 0; e < 32; ++e, d += q.ld) {
      if (e < n) *d = v[e];
      if (on && e <= n) r[e] = v[e];
    }
  } else {
    __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(q.d) + c * q.ld + row, *r = static_cast<__nv_bfloat16 *>(q.d) + row * q.ld + c;
#pragma unroll
    for (int e = 0; e < 32; ++e, d += q.ld) {
      if (e < n) *d = __float2bfloat16_rn(v[e]);
      if (on && e <= n) r[e] = __float2bfloat16_rn(v[e]);
    }
  }
}

template <int BN, bool NV, bool SPLIT, int NP>
__global__ void __launch_bounds__(kThreads, 2) fp4_gemm_kernel(const __grid_constant__ Fp4GemmBlock<NP> p) {
  using C = Cfg<BN, NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kStages * C::kStage);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * C::kStages + 1);
  const uint32_t base = smem_u32(smem), bar_base = smem_u32(bars);
  auto full = [&](int s) { return bar_base + 8u * s; };
  auto empty = [&](int s) { return bar_base + 8u * (C::kStages + s); };
  const uint32_t done = bar_base + 8u * (2 * C::kStages);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = SPLIT ? (int)cta_rank() : 0;
  int parts = 1;
  if (SPLIT) asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
  const int tile = (int)blockIdx.x / parts;
  const Fp4Prob &q = p.prob[find_prob(p, tile)];
  int pt, qt;
  tile_of<128, BN>(q, tile - q.tile_begin, pt, qt);
  const int k0 = (int)((int64_t)part * q.kt / parts), k1 = (int)((int64_t)(part + 1) * q.kt / parts);
  const long long limit = p.wait_limit;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    mbar_fence_init();
    if (q.kt) {
      prefetch_tmap(&q.pc);
      prefetch_tmap(&q.qc);
      prefetch_tmap(&q.ps);
      prefetch_tmap(&q.qs);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();
  // No wait can run out before this: the shortest limit is about a millisecond.
  if (p.clear_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    int last_parity[C::kStages];
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) last_parity[s] = -1;
    for (int kb = k0; kb < k1; ++kb) {
      if (!mbar_wait_warp(empty(stage), phase ^ 1u, limit)) {
        if (lane == 0) set_status(p.status, kTimeoutBit);
        break;
      }
      const uint32_t sp = base + stage * C::kStage, sq = sp + C::kPBytes, ss = sq + C::kQBytes;
      if (elect_one()) {
        mbar_arrive_expect_tx(full(stage), C::kStage);
        tma_load_2d(sp, &q.pc, kb * 128, pt * 128, full(stage));
        tma_load_2d(sq, &q.qc, kb * 128, qt * BN, full(stage));
        tma_load_3d(ss, &q.ps, 0, kb * C::kSTiles, pt, full(stage));
        tma_load_3d(ss + C::kPs, &q.qs, 0, kb * C::kSTiles, qt * BN / 128, full(stage));
      }
      __syncwarp();
#pragma unroll
      for (int s = 0; s < C::kStages; ++s)
        if (s == stage) last_parity[s] = (int)phase;
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // every load that was started must have landed before this CTA leaves
#pragma unroll
    for (int s = 0; s < C::kStages; ++s)
      if (last_parity[s] >= 0 && !mbar_wait_warp(full(s), (uint32_t)last_parity[s], limit) && lane == 0)
        set_status(p.status, kTimeoutBit);
  } else if (warp == 1) {
    const uint32_t qofs = BN < 128 ? (uint32_t)(qt * BN % 128) >> 5 : 0;   // Q's first row within its row tile, in 32s
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = k0; kb < k1; ++kb) {
      if (!mbar_wait_warp(full(stage), phase, limit)) {
        if (lane == 0) set_status(p.status, kTimeoutBit);
        break;
      }
      tc_fence_after();
      const uint32_t sp = base + stage * C::kStage, sq = sp + C::kPBytes, ss = sq + C::kQBytes;
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < C::kSTiles; ++j) {
          tc_cp_scales(tmem + C::kPsCol + 4 * j, smem_desc_scales(ss + 512 * j));
          tc_cp_scales(tmem + C::kQsCol + 4 * j, smem_desc_scales(ss + C::kPs + 512 * j));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // 64 columns: 32 bytes inside the swizzled rows; MX: half of a scale word, NV: a whole one
          const int j = NV ? k : k >> 1, id = NV ? 0 : 2 * (k & 1);
          tc_mma_fp4<NV>(tmem, smem_desc_sw128(sp + 32 * k, 16, 1024), smem_desc_sw128(sq + 32 * k, 16, 1024),
                         idesc_fp4(128, BN, NV, id), tmem + C::kPsCol + 4 * j, tmem + C::kQsCol + 4 * j + qofs,
                         kb != k0 || k != 0);
        }
        tc_commit(empty(stage));
        if (kb + 1 == k1) tc_commit(done);
      }
      __syncwarp();
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  // Warps 2-9: lanes 32 (warp mod 4) .. + 31 of the accumulator, each half of its columns (of narrow tiles
  // warps 2-5 all of them).  The rest waits for them below.
  const int quarter = warp & 3, half = (warp - 2) >> 2;
  constexpr int kHalfBn = BN >= 64 ? BN / 2 : BN;
  const int c_begin = half * kHalfBn, c_end = c_begin + kHalfBn < BN ? c_begin + kHalfBn : BN;
  const int row = quarter * 32 + lane;
  const bool epi = warp >= 2;
  bool have = k1 > k0;
  const MatrixScales g(q);
  const bool trans = q.flags & kFp4DTrans, sym = q.flags & kFp4Sym;
  constexpr int N = BN < 32 ? BN : 32;
  if (epi && have && !mbar_wait_warp(done, 0, limit)) {
    if (lane == 0) set_status(p.status, kTimeoutBit);
    have = false;
  }
  __syncwarp();
  tc_fence_after();
  auto read = [&](int c, float (&v)[N]) {
    uint32_t r[N];
    if constexpr (N == 16) tmem_ld16(tmem + c + ((uint32_t)(quarter * 32) << 16), r);
    else tmem_ld32(tmem + c + ((uint32_t)(quarter * 32) << 16), r);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = __uint_as_float(r[e]);
  };
  auto store = [&](int c, float (&v)[N]) {
    g.apply(q, v);
    const int64_t at = (int64_t)qt * BN + c;
    if constexpr (N == 32) {
      // the ring is free: this CTA's MMAs are done
      uint8_t *stage = smem + 2048 * (warp - 2);
      const int64_t row0 = (int64_t)pt * 128 + 32 * quarter;
      if (sym) store_symmetric(q, stage, row0, at, v);
      else if (!trans) store_block(q, stage, row0, at, v);
      else store_row<N>(q, row0 + lane, at, v, true);
    } else {
      store_row<N>(q, (int64_t)pt * 128 + row, at, v, trans);
    }
  };
  if (!SPLIT) {
    if (epi) {
#pragma unroll 1
      for (int c = c_begin; c < c_end; c += N) {
        float v[N];
        if (have) read(c, v);
        else {
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] = 0.f;
        }
        store(c, v);
      }
    }
  } else {
    // The parts go into this CTA's ring, which its own MMAs have left: rows of kPitch floats, or column by
    // column where D takes the transpose.  Then every CTA sums the rows (columns) that fall to it, part
    // 0 first.
    constexpr int kPitch = BN + 4;
    float *mine = reinterpret_cast<float *>(smem);
    if (epi) {
#pragma unroll 1
      for (int c = c_begin; c < c_end; c += N) {
        float v[N];
        if (have) read(c, v);
        else {
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] = 0.f;
        }
        if (trans) {
#pragma unroll
          for (int e = 0; e < N; ++e) mine[(c + e) * 128 + row] = v[e];
        } else {
#pragma unroll
          for (int e = 0; e < N; e += 4)
            *reinterpret_cast<float4 *>(mine + row * kPitch + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
    }
    cluster_sync();
    if (epi && trans) {
      // BN and parts are powers of two: a CTA takes 2 columns or more
      auto join = [&](int c, auto width) {
        constexpr int W = decltype(width)::value;
        float v[W];
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = 0.f;
        for (int r = 0; r < parts; ++r) {
          const uint32_t from = mapa(base + (uint32_t)((c * 128 + row) * 4), (uint32_t)r);
#pragma unroll
          for (int e = 0; e < W; ++e) v[e] += ld_cluster(from + 512u * e);
        }
        g.apply(q, v);
        store_row<W>(q, (int64_t)pt * 128 + row, (int64_t)qt * BN + c, v, true);
      };
      const int each = BN / parts, c0 = each * part;
      if (each >= 16) {
        for (int c = c0 + 8 * half; c < c0 + each; c += 16) join(c, std::integral_constant<int, 8>());
      } else {
        for (int c = c0 + 2 * half; c < c0 + each; c += 4) join(c, std::integral_constant<int, 2>());
      }
    } else if (epi) {
      constexpr int L = BN / 4, kRows = 32 / L;           // lanes of a row, rows of an instruction
      const int w = warp - 2, n = 128 / parts, r0 = n * part;
      float *sum = mine + 128 * kPitch;                   // n rows, behind the parts
#pragma unroll 4
      for (int i = w * kRows; i < n; i += kEpiWarps * kRows) {
        const int r = i + lane / L, c = 4 * (lane % L);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < parts; ++k) {
          const float4 x = ld_cluster4(mapa(base + (uint32_t)(((r0 + r) * kPitch + c) * 4), (uint32_t)k));
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
        }
        float o[4] = {v.x, v.y, v.z, v.w};
        g.apply(q, o);
        *reinterpret_cast<float4 *>(sum + r * kPitch + c) = make_float4(o[0], o[1], o[2], o[3]);
      }
      named_barrier(1, 32 * kEpiWarps);
      const int64_t p0 = (int64_t)pt * 128 + r0, q0 = (int64_t)qt * BN;
      const int rows = (int)(q.np - p0 < n ? q.np - p0 : n), cols = (int)(q.nq - q0 < BN ? q.nq - q0 : BN);
      const bool f32 = q.flags & kFp4DF32;
      const bool on = sym && pt == qt;                    // a tile on the diagonal: see store_symmetric
      if ((q.flags & kFp4DVec) && cols == BN && !on) {
        for (int i = w * kRows; i < rows; i += kEpiWarps * kRows) {
          const int r = i + lane / L, c = 4 * (lane % L);
          const float4 x = *reinterpret_cast<const float4 *>(sum + r * kPitch + c);
          const int64_t at = (p0 + r) * q.ld + q0 + c;
          if (r >= rows) continue;
          if (f32) *reinterpret_cast<float4 *>(static_cast<float *>(q.d) + at) = x;
          else *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(q.d) + at) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
        }
      } else {
        for (int r = w; r < rows; r += kEpiWarps)
          for (int c = lane; c < (on ? r0 + r + 1 : cols); c += 32) {
            const int64_t at = (p0 + r) * q.ld + q0 + c;
            if (f32) static_cast<float *>(q.d)[at] = sum[r * kPitch + c];
            else static_cast<__nv_bfloat16 *>(q.d)[at] = __float2bfloat16_rn(sum[r * kPitch + c]);
          }
      }
      if (sym) {
        // the mirror image: rows run along D's columns
        for (int c = w; c < cols; c += kEpiWarps)
          for (int r = lane; r < rows; r += 32) {
            if (on && c >= r0 + r) continue;
            const int64_t at = (q0 + c) * q.ld + p0 + r;
            if (f32) static_cast<float *>(q.d)[at] = sum[r * kPitch + c];
            else static_cast<__nv_bfloat16 *>(q.d)[at] = __float2bfloat16_rn(sum[r * kPitch + c]);
          }
      }
    }
    cluster_sync();   // no CTA leaves while another may still read its shared memory
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// 256 x 256 tiles on CTA pairs, persistent.  8192^3: 180 us MXFP4, 186 us NVFP4 (6.1 and 5.9 PFLOP/s, up to 216 us under the
// power cap); 8192 x 6144 x 2048 NVFP4 to bf16: 47 us (57 with operands and result in DRAM), tensor pipe 58 %; four
// 2048 x 8192 Gram matrices MXFP4 to fp32: 36 us.  A step of 256 columns is 513 clocks of MMAs and took 600 to 660 in the
// long sums; what is left is the 870 clocks in which a tile waits for the shared columns below, and the last
// tile's epilogue (2 us in bf16, 7 us for an fp32 block with its mirror image).
//
// Two accumulators of 256 columns and the scales do not fit the 512 columns of tensor memory, so the second
// accumulator starts 192 columns after the first.  The epilogue drains the 64 shared columns
// first and hands them over; the next tile's MMAs run beside the rest of it.
//
// The MMA warp copies a step's scales into tensor memory ahead of its MMAs: 24 (MX) or 48 columns, a third for this
// CTA's rows of P, the others for all rows of Q.  Copies and MMAs of one thread run in order and
// overlap.  (8192 x 6144 x 2048 NVFP4 took 83 us with `lane == 0` code instead of an elected lane.  Under `lane == 0`,
// four more warps for the copies made it 63 us, and 256 x 192 tiles with two whole accumulators 65 us; neither has been
// timed with an elected lane.)
template <bool NV>
struct PairCfg {
  static constexpr int kBn = kFp4PairBn;
  static constexpr int kSTiles = NV ? 4 : 2;                 // scale tiles of a step and row tile
  static constexpr int kHalf = 128 * 128;                    // codes of 128 rows
  static constexpr int kCodes = 2 * kHalf;                   // in one CTA: its rows of P, half of Q's
  static constexpr int kRt = kSTiles * 512;                  // scales of a row tile: P's own, Q's two
  static constexpr int kStage = kCodes + 3 * kRt;
  static constexpr int kStages = 5;
  static constexpr int kOut = 8 * 2048;                      // a block of D for each epilogue warp
  static constexpr int kSmem = kStages * kStage + kOut + 1024 + 256;
  static constexpr int kShared = 64, kShift = 256 - kShared; // between the accumulators
  static constexpr int kPsCol = kShift + 256, kQsCol = kPsCol + 4 * kSTiles;   // a step's scales
  static_assert(kStage % 1024 == 0 && kSmem <= 232448 && kQsCol + 8 * kSTiles <= 512, "fits");
};
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr uint32_t kPeerMask = 0xFEFFFFFFu;                  // clears the CTA-rank bit of a cluster address

template <bool NV, int NP>
__global__ void __launch_bounds__(kPairThreads, 1) fp4_pair_kernel(const __grid_constant__ Fp4GemmBlock<NP> p) {
  using C = PairCfg<NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *out = smem + C::kStages * C::kStage;
  uint64_t *bars = reinterpret_cast<uint64_t *>(out + C::kOut);
  constexpr int kBars = 2 * C::kStages + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
  const uint32_t base = smem_u32(smem), bar_base = smem_u32(bars);
  auto full = [&](int s) { return bar_base + 8u * s; };                       // both CTAs' loads (leader's)
  auto empty = [&](int s) { return bar_base + 8u * (C::kStages + s); };
  const uint32_t tfull = bar_base + 8u * (2 * C::kStages), tfree = tfull + 8u;   // tfree: the leader's

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const bool leader = rank == 0;
  const int cid = (int)cluster_id(), ncl = (int)num_clusters();
  const long long limit = p.wait_limit;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tfree, 2 * kPairEpiWarps);   // one arrival per epilogue warp of both CTAs
    mbar_fence_init();
    const Fp4Prob &q = p.prob[find_prob(p, cid)];
    prefetch_tmap(&q.pc);
    prefetch_tmap(&q.qc);
    prefetch_tmap(&q.ps);
    prefetch_tmap(&q.qs);
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(tmem_slot), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();
  // No wait can run out before this: the shortest limit is about a millisecond.
  if (p.clear_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

  if (warp == 0) {
    // -------------------------------------------------------------- loads (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    int last_parity[C::kStages];
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) last_parity[s] = -1;
    bool ok = true;
    for (int tile = cid; ok && tile < p.total_tiles; tile += ncl) {
      const Fp4Prob &q = p.prob[find_prob(p, tile)];
      int pt, qt;
      tile_of<256, 256>(q, tile - q.tile_begin, pt, qt);
      const int prow = pt * 256 + 128 * (int)rank, qrow = qt * 256 + 128 * (int)rank;
      for (int kb = 0; kb < q.kt; ++kb) {
        ok = mbar_wait_warp(empty(stage), phase ^ 1u, limit);
        if (!ok) break;
        const uint32_t sp = base + stage * C::kStage, sq = sp + C::kHalf, ss = sq + C::kHalf;
        const uint32_t fb = full(stage) & kPeerMask;      // the leader's barrier
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(full(stage), 2 * C::kStage);
          tma_load_2sm(sp, &q.pc, kb * 128, prow, fb);
          tma_load_2sm(sq, &q.qc, kb * 128, qrow, fb);
          tma_load_3d_2sm(ss, &q.ps, 0, kb * C::kSTiles, pt * 2 + (int)rank, fb);
          tma_load_3d_2sm(ss + C::kRt, &q.qs, 0, kb * C::kSTiles, qt * 2, fb);
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s < C::kStages; ++s)
          if (s == stage) last_parity[s] = (int)phase;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) set_status(p.status, kTimeoutBit);
    if (leader) {
      // every load of the pair that was armed must have landed
#pragma unroll
      for (int s = 0; s < C::kStages; ++s)
        if (last_parity[s] >= 0 && !mbar_wait_warp(full(s), (uint32_t)last_parity[s], limit) && lane == 0)
          set_status(p.status, kTimeoutBit);
    }
  } else if (warp == 1) {
    if (leader) {
      // ------------------------------------------------------------ copies and MMAs (leader)
      int stage = 0, tl = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < p.total_tiles; tile += ncl, ++tl) {
        const int kt = p.prob[find_prob(p, tile)].kt;
        // the columns that this tile shares with the one before have been drained, and with them all
        // of the tile before that
        ok = tl == 0 || mbar_wait_warp(tfree, (uint32_t)(tl - 1) & 1u, limit);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)((tl & 1) * C::kShift);
        for (int kb = 0; kb < kt; ++kb) {
          ok = mbar_wait_warp(full(stage), phase, limit);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sp = base + stage * C::kStage, sq = sp + C::kHalf, ss = sq + C::kHalf;
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < C::kSTiles; ++j) {
              tc_cp2_scales(tmem + C::kPsCol + 4 * j, smem_desc_scales(ss + 512 * j));
#pragma unroll
              for (int i = 0; i < 2; ++i)
                tc_cp2_scales(tmem + C::kQsCol + 8 * j + 4 * i, smem_desc_scales(ss + (1 + i) * C::kRt + 512 * j));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // 64 columns: 32 bytes inside the swizzled rows; MX: half of a scale word, NV: a whole one
              const int j = NV ? k : k >> 1, id = NV ? 0 : 2 * (k & 1);
              tc_mma2_fp4<NV>(d, smem_desc_sw128(sp + 32 * k, 16, 1024), smem_desc_sw128(sq + 32 * k, 16, 1024),
                              idesc_fp4(256, C::kBn, NV, id), tmem + C::kPsCol + 4 * j, tmem + C::kQsCol + 8 * j, (kb | k) != 0);
            }
            tc_commit2_mc(empty(stage), 0x3);
            if (kb + 1 == kt) tc_commit2_mc(tfull, 0x3);
          }
          __syncwarp();
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && lane == 0) set_status(p.status, kTimeoutBit);
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    int tl = 0;
    for (int tile = cid; tile < p.total_tiles; tile += ncl, ++tl) {
      const Fp4Prob &q = p.prob[find_prob(p, tile)];
      int pt, qt;
      tile_of<256, 256>(q, tile - q.tile_begin, pt, qt);
      const MatrixScales g(q);
      const int64_t row0 = (int64_t)pt * 256 + 128 * rank + quarter * 32;
      const uint32_t acc = tmem + (uint32_t)((tl & 1) * C::kShift) + ((uint32_t)(quarter * 32) << 16);
      // 32 columns at a time: one of the two shared chunks first, then three others
      const int shared_c = ((tl & 1) ? 0 : C::kShift) + 32 * half, rest_c = ((tl & 1) ? C::kShared : 0) + 96 * half;
      if (!mbar_wait_warp(tfull, (uint32_t)tl & 1u, limit)) {
        set_status(p.status, kTimeoutBit);
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int cc = i == 0 ? shared_c : rest_c + 32 * (i - 1);
        uint32_t r[32];
        tmem_ld32(acc + cc, r);
        tmem_ld_wait();
        if (i == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive_relaxed(mapa(tfree, 0));
        }
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
        g.apply(q, v);
        const int64_t c = (int64_t)qt * 256 + cc;
        if (q.flags & kFp4Sym) store_symmetric(q, out + 2048 * (warp - 2), row0, c, v);
        else store_block(q, out + 2048 * (warp - 2), row0, c, v);
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // no CTA leaves while its partner may still read its shared memory or signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

template <bool NV, int NP>
cudaError_t launch_pair(const Fp4GemmParams &p, cudaStream_t s) {
  using C = PairCfg<NV>;
  static PerDevice pairs;   // pairs that can be resident at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  int most = pairs.get(dev);
  if (!most) {
    e = cudaFuncSetAttribute(fp4_pair_kernel<NV, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int sms = device_sms();
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&most, fp4_pair_kernel<NV, NP>, &cfg) != cudaSuccess || most <= 0) {
      (void)cudaGetLastError();
      most = sms / 2;
    }
    most = most < sms / 2 ? most : sms / 2;
    pairs.set(dev, most);
  }
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(2 * (p.total_tiles < most ? p.total_tiles : most), 1, 1);
  e = cudaLaunchKernelEx(&cfg, fp4_pair_kernel<NV, NP>, prefix<Fp4GemmBlock<NP>>(p));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int BN, bool NV, bool SPLIT, int NP>
cudaError_t launch(const Fp4GemmParams &p, int split, cudaStream_t s) {
  using C = Cfg<BN, NV>;
  static PerDevice attr_set;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!attr_set.get(dev)) {
    e = cudaFuncSetAttribute(fp4_gemm_kernel<BN, NV, SPLIT, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set.set(dev, 1);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.total_tiles * split, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, fp4_gemm_kernel<BN, NV, SPLIT, NP>, prefix<Fp4GemmBlock<NP>>(p));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int BN, bool NV>
cudaError_t launch_bn(const Fp4GemmParams &p, int split, cudaStream_t s) {
  if (p.nprob <= kFewFp4Prob)
    return split > 1 ? launch<BN, NV, true, kFewFp4Prob>(p, split, s) : launch<BN, NV, false, kFewFp4Prob>(p, 1, s);
  return split > 1 ? launch<BN, NV, true, kMaxFp4Prob>(p, split, s) : launch<BN, NV, false, kMaxFp4Prob>(p, 1, s);
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4GemmParams &p, int bn, int split, bool nv, cudaStream_t s) {
  if (p.total_tiles <= 0) return cudaSuccess;
  switch (bn) {
    case kFp4PairBn:
      if (p.nprob <= kFewFp4Prob) return nv ? launch_pair<true, kFewFp4Prob>(p, s) : launch_pair<false, kFewFp4Prob>(p, s);
      return nv ? launch_pair<true, kMaxFp4Prob>(p, s) : launch_pair<false, kMaxFp4Prob>(p, s);
    case 16: return nv ? launch_bn<16, true>(p, split, s) : launch_bn<16, false>(p, split, s);
    case 32: return nv ? launch_bn<32, true>(p, split, s) : launch_bn<32, false>(p, split, s);
    case 64: return nv ? launch_bn<64, true>(p, split, s) : launch_bn<64, false>(p, split, s);
    case 128: return nv ? launch_bn<128, true>(p, split, s) : launch_bn<128, false>(p, split, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace nshb

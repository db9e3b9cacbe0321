// experts.hip -- matrix products grouped by expert with ragged row counts
// (gfx950): the linear layers of a mixture of experts, forward, input
// gradient and weight gradient.
//
//   forward      y[t, o]    = sum_i x[t, i] W_e[o, i]      t in rows(e)
//   input grad   dx[t, i]   = sum_o dy[t, o] W_e[o, i]     t in rows(e)
//   weight grad  dW_e[o, i] = sum_{t in rows(e)} dy[t, o] x[t, i]
//
// The row counts live on the device, so nothing waits for the host: the row
// products launch as many workgroups as the tiles of any split of the rows
// could need (rows / BM + experts, times the column tiles), and each finds its
// tile from the ends with a wave-wide scan; those behind the last tile leave.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kernels.hpp"
#include "operators.hpp"
#include "tiles.hpp"
#include "tiles_f32.hpp"

namespace ar_dev {
namespace {

// Running maximum of the ends, 64 experts at a time: one call gives lane l
// the first and one-past-last row of expert e0 + l (an empty range from the
// last expert on).  carry: the end before expert e0; updated.
__device__ __forceinline__ void scan_ends(const ExpertArgs &a, int e0, int &carry, int &lo, int &hi) {
  const int lane = threadIdx.x & 63, e = e0 + lane;
  int v = e < a.experts ? a.ends[e] : 0;
  v = max(0, min(v, static_cast<int>(a.tokens)));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v = max(v, u);
  }
  v = max(v, carry);
  const int prev = __shfl_up(v, 1);
  lo = lane == 0 ? carry : prev;
  hi = v;
  carry = __shfl(v, 63);
}

__device__ __forceinline__ int wave_sum_to(int v) {  // inclusive prefix sum
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

struct RowTile {
  int e, row, rows, tile_n;  // expert, first row, rows of the tile, column tile
};

// Workgroups go round the 8 XCDs (each with an L2 of its own) in turn, so
// position p of n goes to the place that gives every XCD one run of
// neighbouring tiles.
__device__ __forceinline__ int64_t xcd_run(int64_t p, int64_t n) {
  const int64_t q = n / 8, r = n % 8, x = p % 8;
  return x * q + min(x, r) + p / 8;
}

// Tiles of an mt x nt grid in the order they are worked on: bands of kBand
// row tiles, each swept by columns, so that neighbours share operands.
constexpr int kBand = 4;
__device__ __forceinline__ void band_tile(int l, int mt, int nt, int &m, int &n) {
  const int g = l / (kBand * nt), first = g * kBand, in = min(kBand, mt - first), r = l - g * kBand * nt;
  m = first + r % in;
  n = r / in;
}

template <int BM>
__device__ __forceinline__ bool find_row_tile(const ExpertArgs &a, int nt, RowTile &t) {
  int carry = 0, lo, hi, total = 0;
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    scan_ends(a, e0, carry, lo, hi);
    total += __shfl(wave_sum_to((hi - lo + BM - 1) / BM), 63);
  }
  const int64_t tiles = static_cast<int64_t>(total) * nt;
  if (blockIdx.x >= tiles) return false;
  int64_t want = xcd_run(blockIdx.x, tiles);
  carry = 0;
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    scan_ends(a, e0, carry, lo, hi);
    const int mt = (hi - lo + BM - 1) / BM;
    const int upto = wave_sum_to(mt);
    const int64_t batch = static_cast<int64_t>(__shfl(upto, 63)) * nt;
    if (want >= batch) {
      want -= batch;
      continue;
    }
    const int l = __builtin_ctzll(__ballot(static_cast<int64_t>(upto) * nt > want));
    const int mte = __shfl(mt, l);
    want -= static_cast<int64_t>(__shfl(upto, l) - mte) * nt;
    int m, n;
    band_tile(static_cast<int>(want), mte, nt, m, n);
    const int first = __shfl(lo, l) + m * BM;
    t.e = __builtin_amdgcn_readfirstlane(e0 + l);
    t.row = __builtin_amdgcn_readfirstlane(first);
    t.rows = __builtin_amdgcn_readfirstlane(min(BM, __shfl(hi, l) - first));
    t.tile_n = __builtin_amdgcn_readfirstlane(n);
    return true;
  }
  return false;
}

// Stores v to p[0 .. n) (n in 1 .. 4), rounding once to the output's type.
template <bool BF>
__device__ __forceinline__ void store4(void *base, int64_t at, fx4 v, int n, bool vec) {
  if constexpr (BF) {
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    uint16_t *p = static_cast<uint16_t *>(base) + at;
    if (vec && n >= 4) {
      *reinterpret_cast<ux2 *>(p) = ux2{h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = h[i];
    }
  } else {
    float *p = static_cast<float *>(base) + at;
    if (vec && n >= 4) {
      *reinterpret_cast<fx4 *>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = v[i];
    }
  }
}
template <bool BF>
__device__ __forceinline__ fx4 load4(const void *base, int64_t at, int n, bool vec) {
  fx4 v = {};
  if constexpr (BF) {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at;
    if (vec && n >= 4) {
      const ux2 u = *reinterpret_cast<const ux2 *>(p);
      v = fx4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u), __uint_as_float(u[1] << 16),
              __uint_as_float(u[1] & 0xffff0000u)};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) v[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
    }
  } else {
    const float *p = static_cast<const float *>(base) + at;
    if (vec && n >= 4) {
      v = *reinterpret_cast<const fx4 *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) v[i] = p[i];
    }
  }
  return v;
}

// Forward (GRAD false: A = x, B = W_e as [n][k]) and input gradient (GRAD
// true: A = dy, B = W_e as [k][n]).
template <class P, bool GRAD>
__global__ __launch_bounds__(P::Sh::kThreads) void experts_rows(ExpertArgs a) {
  using S = typename P::Sh;
  using T = typename P::Elem;
  extern __shared__ __align__(16) char lds[];
  const int64_t n = GRAD ? a.in : a.outf, k = GRAD ? a.outf : a.in;
  const int nt = static_cast<int>((n + S::BN - 1) / S::BN);
  RowTile t;
  if (!find_row_tile<S::BM>(a, nt, t)) return;
  const int64_t n0 = static_cast<int64_t>(t.tile_n) * S::BN, ldx = GRAD ? a.dys : a.xs;
  const int validn = static_cast<int>(min(static_cast<int64_t>(S::BN), n - n0));
  const T *x = static_cast<const T *>(GRAD ? a.dy : a.x) + t.row * ldx;
  const T *w = static_cast<const T *>(a.w) + a.offsets[t.e] + (GRAD ? n0 : n0 * a.in);
  P p;
  p.run(lds, x, w, ldx, a.in, t.rows, validn, k);
  p.each([&](int m, int c, fx4 v) {
    if (m < t.rows && c < validn)
      store4<sizeof(T) == 2>(a.out, (t.row + m) * a.outs + n0 + c, v, validn - c, a.vec_out);
  });
}

template <class P, bool GBF>
__global__ __launch_bounds__(P::Sh::kThreads) void experts_weights(ExpertArgs a) {
  using S = typename P::Sh;
  using T = typename P::Elem;
  extern __shared__ __align__(16) char lds[];
  const int mt = static_cast<int>((a.outf + S::BM - 1) / S::BM), nt = static_cast<int>((a.in + S::BN - 1) / S::BN);
  const int64_t id = xcd_run(blockIdx.x, gridDim.x);
  const int per = mt * nt;
  const int e = static_cast<int>(id / per);
  int tm, tn;
  band_tile(static_cast<int>(id % per), mt, nt, tm, tn);
  int carry = 0, lo = 0, hi = 0;
  for (int e0 = 0; e0 <= e; e0 += 64) scan_ends(a, e0, carry, lo, hi);
  const int r0 = __builtin_amdgcn_readfirstlane(__shfl(lo, e & 63));
  const int rows = __builtin_amdgcn_readfirstlane(__shfl(hi, e & 63)) - r0;
  if (a.accumulate && rows == 0) return;
  const int64_t m0 = static_cast<int64_t>(tm) * S::BM, n0 = static_cast<int64_t>(tn) * S::BN;
  const int validm = static_cast<int>(min(static_cast<int64_t>(S::BM), a.outf - m0));
  const int validn = static_cast<int>(min(static_cast<int64_t>(S::BN), a.in - n0));
  const T *dy = static_cast<const T *>(a.dy) + r0 * a.dys + m0;
  const T *x = static_cast<const T *>(a.x) + r0 * a.xs + n0;
  const int64_t out = a.offsets[e] + m0 * a.in + n0;
  P p;
  p.run(lds, dy, x, a.dys, a.xs, validm, validn, rows);
  p.each([&](int m, int c, fx4 v) {
    if (m < validm && c < validn) {
      const int64_t at = out + m * a.in + c;
      if (a.accumulate) {
        const fx4 old = load4<GBF>(a.out, at, validn - c, a.vec_out);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += old[i];
      }
      store4<GBF>(a.out, at, v, validn - c, a.vec_out);
    }
  });
}

template <class K>
hipError_t launch(K kernel, int64_t grid, int threads, int lds, const ExpertArgs &a, hipStream_t s) {
  if (grid == 0) return hipSuccess;
  if (grid * threads > 0x7fffffff) return hipErrorInvalidConfiguration;
  // more than 64 KB of LDS has to be asked for
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  AR_LAUNCH(kernel, dim3(static_cast<uint32_t>(grid)), dim3(threads), lds, s, a);
  return hipGetLastError();
}

using Square = Shape<128, 128, 2, 2>;
using Small = Shape<32, 128, 1, 4>;

template <class S, bool GRAD>
hipError_t launch_rows(const ExpertArgs &a, hipStream_t s) {
  const int64_t n = GRAD ? a.in : a.outf, nt = (n + S::BN - 1) / S::BN;
  const int64_t grid = (a.tokens / S::BM + std::min<int64_t>(a.experts, a.tokens)) * nt;
  constexpr Major B = GRAD ? kMajorMN : kMajorK;
  if (!a.bf16) {
    using P = TileProductF32<S, kMajorK, B, false>;
    return launch(experts_rows<P, GRAD>, grid, S::kThreads, P::kLds, a, s);
  }
  if (a.aligned) {
    using P = TileProduct<kBF16, S, kMajorK, B, true>;
    return launch(experts_rows<P, GRAD>, grid, S::kThreads, P::kLds, a, s);
  }
  using P = TileProduct<kBF16, S, kMajorK, B, false>;
  return launch(experts_rows<P, GRAD>, grid, S::kThreads, P::kLds, a, s);
}

template <bool GRAD>
hipError_t rows(const ExpertArgs &a, hipStream_t s) {
  return a.tokens >= 64 * static_cast<int64_t>(a.experts) ? launch_rows<Square, GRAD>(a, s)
                                                          : launch_rows<Small, GRAD>(a, s);
}

}  // namespace

hipError_t experts_forward(const ExpertArgs &a, hipStream_t s) { return rows<false>(a, s); }
hipError_t experts_input_grad(const ExpertArgs &a, hipStream_t s) { return rows<true>(a, s); }

hipError_t experts_weight_grad(const ExpertArgs &a, hipStream_t s) {
  using S = Square;
  const int64_t grid = ((a.outf + S::BM - 1) / S::BM) * ((a.in + S::BN - 1) / S::BN) * a.experts;
  if (!a.bf16) {
    using P = TileProductF32<S, kMajorMN, kMajorMN, false>;
    return launch(experts_weights<P, false>, grid, S::kThreads, P::kLds, a, s);
  }
  if (a.aligned) {
    using P = TileProduct<kBF16, S, kMajorMN, kMajorMN, true>;
    return a.grad_bf16 ? launch(experts_weights<P, true>, grid, S::kThreads, P::kLds, a, s)
                       : launch(experts_weights<P, false>, grid, S::kThreads, P::kLds, a, s);
  }
  using P = TileProduct<kBF16, S, kMajorMN, kMajorMN, false>;
  return a.grad_bf16 ? launch(experts_weights<P, true>, grid, S::kThreads, P::kLds, a, s)
                     : launch(experts_weights<P, false>, grid, S::kThreads, P::kLds, a, s);
}

}  // namespace ar_dev

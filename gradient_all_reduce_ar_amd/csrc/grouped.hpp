// grouped.hpp -- what the kernels of the products grouped by expert share
// (gfx950): which rows and tiles are whose, and the way into and out of rows
// at any element's address.  A: the call's arguments, with `ends`, `experts`
// and `tokens`.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernels.hpp"
#include "tiles.hpp"

namespace ar_dev {
namespace {

// The value of another lane by a data-parallel primitive, `none` where there is
// no such lane or the masks leave it out.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int lane_moved(int none, int v) {
  return __builtin_amdgcn_update_dpp(none, v, CTRL, ROWS, 0xf, false);
}
// Inclusive scan over the wave: rows of 16 lanes by shifts of 1, 2, 4 and 8,
// then the last lane of a row to the next row, and of the first half to the
// second.  f(identity, v) = v.  (Twelve lane permutations through the LDS instead
// take about a microsecond of every workgroup's start.)
template <class F>
__device__ __forceinline__ int wave_scan(int v, int identity, F f) {
  v = f(lane_moved<0x111>(identity, v), v);
  v = f(lane_moved<0x112>(identity, v), v);
  v = f(lane_moved<0x114>(identity, v), v);
  v = f(lane_moved<0x118>(identity, v), v);
  v = f(lane_moved<0x142, 0xa>(identity, v), v);
  return f(lane_moved<0x143, 0xc>(identity, v), v);
}

// Running maximum of the ends, 64 experts at a time: one call gives lane l
// the first and one-past-last row of expert e0 + l (an empty range from the
// last expert on).  carry: the end before expert e0; updated.
template <class A>
__device__ __forceinline__ void scan_ends(const A &a, int e0, int &carry, int &lo, int &hi) {
  const int lane = threadIdx.x & 63, e = e0 + lane;
  int v = e < a.experts ? a.ends[e] : 0;
  v = max(0, min(v, static_cast<int>(a.tokens)));
  v = max(wave_scan(v, 0, [](int p, int q) { return max(p, q); }), carry);
  lo = lane_moved<0x138>(carry, v);  // the lane before
  hi = v;
  carry = __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ int wave_sum_to(int v) {  // inclusive prefix sum
  return wave_scan(v, 0, [](int p, int q) { return p + q; });
}

struct RowTile {
  int e, row, rows, tile_n;  // expert, first row, rows of the tile, column tile
  int tile_m;                // row tile, of the expert's
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
constexpr int kBand = 8;
__device__ __forceinline__ void band_tile(int l, int mt, int nt, int &m, int &n) {
  const int g = l / (kBand * nt), first = g * kBand, in = min(kBand, mt - first), r = l - g * kBand * nt;
  m = first + r % in;
  n = r / in;
}

// This workgroup's tile: of `nt` column tiles times the row tiles of all
// experts, in runs of neighbours per XCD.
template <int BM, class A>
__device__ __forceinline__ bool find_row_tile(const A &a, int nt, RowTile &t) {
  int carry = 0, lo, hi, total = 0;
  // the tiles up to and of this lane's expert, of the experts from e0 on
  auto scan = [&](int e0, int &mt, int &upto) {
    scan_ends(a, e0, carry, lo, hi);
    mt = (hi - lo + BM - 1) / BM;
    upto = wave_sum_to(mt);
    return __builtin_amdgcn_readlane(upto, 63);
  };
  int mt, upto, batch = 0;
  for (int e0 = 0; e0 < a.experts; e0 += 64) total += batch = scan(e0, mt, upto);
  const int64_t tiles = static_cast<int64_t>(total) * nt;
  if (blockIdx.x >= tiles) return false;
  int64_t want = xcd_run(blockIdx.x, tiles);
  const bool again = a.experts > 64;  // the scan's registers hold the only batch otherwise
  carry = 0;
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    if (again) batch = scan(e0, mt, upto);
    if (want >= static_cast<int64_t>(batch) * nt) {
      want -= static_cast<int64_t>(batch) * nt;
      continue;
    }
    const int l = __builtin_ctzll(__ballot(static_cast<int64_t>(upto) * nt > want));
    const int mte = __builtin_amdgcn_readlane(mt, l);
    want -= static_cast<int64_t>(__builtin_amdgcn_readlane(upto, l) - mte) * nt;
    int m, n;
    band_tile(static_cast<int>(want), mte, nt, m, n);
    const int first = __builtin_amdgcn_readlane(lo, l) + m * BM;
    t.e = __builtin_amdgcn_readfirstlane(e0 + l);
    t.row = __builtin_amdgcn_readfirstlane(first);
    t.rows = __builtin_amdgcn_readfirstlane(min(BM, __builtin_amdgcn_readlane(hi, l) - first));
    t.tile_n = __builtin_amdgcn_readfirstlane(n);
    t.tile_m = __builtin_amdgcn_readfirstlane(m);
    return true;
  }
  return false;
}

// Four elements at any element's address: the hardware takes such 8- and
// 16-byte loads and stores (weight gradients of 515 rows, 24 experts, 1025 x
// 511, bf16: 15.7 us; 20.3 with rows off 8 bytes stored by the element).
typedef ux2 ux2_any __attribute__((aligned(2)));
typedef fx4 fx4_any __attribute__((aligned(4)));

// Stores v to p[0 .. n) (n in 1 .. 4), rounding once to the output's type.
// NT: non-temporal, for what the next kernel will hardly find in a cache.
template <bool BF, bool NT = false>
__device__ __forceinline__ void store4(void *base, int64_t at, fx4 v, int n) {
  if constexpr (BF) {
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    uint16_t *p = static_cast<uint16_t *>(base) + at;
    if (n >= 4) {
      const ux2_any u = {h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16};
      if constexpr (NT) __builtin_nontemporal_store(u, reinterpret_cast<ux2_any *>(p));
      else *reinterpret_cast<ux2_any *>(p) = u;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) p[i] = h[i];
    }
  } else {
    float *p = static_cast<float *>(base) + at;
    if (n >= 4) {
      if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<fx4_any *>(p));
      else *reinterpret_cast<fx4_any *>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) p[i] = v[i];
    }
  }
}
template <bool BF>
__device__ __forceinline__ fx4 load4(const void *base, int64_t at, int n) {
  fx4 v = {};
  if constexpr (BF) {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at;
    if (n >= 4) {
      const ux2 u = *reinterpret_cast<const ux2_any *>(p);
      v = fx4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u), __uint_as_float(u[1] << 16),
              __uint_as_float(u[1] & 0xffff0000u)};
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) v[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
    }
  } else {
    const float *p = static_cast<const float *>(base) + at;
    if (n >= 4) {
      v = *reinterpret_cast<const fx4_any *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) v[i] = p[i];
    }
  }
  return v;
}

template <class K, class... A>
inline hipError_t launch(K kernel, int64_t grid, int parts, int threads, int lds, hipStream_t s, const A &...args) {
  if (grid == 0) return hipSuccess;
  if (grid * threads > 0x7fffffff) return hipErrorInvalidConfiguration;
  // more than 64 KB of LDS has to be asked for
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  AR_LAUNCH(kernel, dim3(static_cast<uint32_t>(grid), parts), dim3(threads), lds, s, args...);
  return hipGetLastError();
}

}  // namespace
}  // namespace ar_dev

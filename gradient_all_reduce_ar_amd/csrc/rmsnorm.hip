// rmsnorm.hip -- RMS norm of rows with the residual's addition and an output
// in 8 bits, its backward pass, and the quantisation of rows (gfx950).
//
//   h = x + r,  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd gain
//   dx = rstd (gain dy - xhat mean(gain dy xhat)) + dh,  dgain = sum dy xhat
//
// Bound by memory.  A team of T threads holds a row in registers between its
// sum and its results, so each row is read once and written once; lane t has
// elements 8 t .. 8 t + 7 of every 8 T.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "grouped.hpp"
#include "kernels.hpp"
#include "operators.hpp"
#include "rows.hpp"

namespace ar_dev {
namespace {

// Teams of a wave share a workgroup of four; larger teams have their own.
template <int T>
constexpr int kTeams = T < 256 ? 256 / T : 1;
template <int T>
constexpr int kRowThreads = T *kTeams<T>;

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sum over the team; `slots` holds a value per wave of the workgroup.  Two
// rows in a row use different slots, so one meeting does for each.
template <int T, class V>
__device__ __forceinline__ V team_sum(V v, V *slots) {
  v = wave_sum(v);
  if constexpr (T == 64) return v;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  V s = slots[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) s += slots[i];
  return s;
}

template <bool BF>
__device__ __forceinline__ void widen(const Raw8<BF> &r, float (&v)[kLane]) {
#pragma unroll
  for (int i = 0; i < kLane; ++i) v[i] = r[i];
}

// 8 elements of the gain (or any vector of a type known at run time).
__device__ __forceinline__ void load_gain(const void *gain, bool bf16, int64_t at, int n, float (&g)[kLane]) {
  if (bf16) widen(load8<true>(gain, at, n), g);
  else widen(load8<false>(gain, at, n), g);
}

template <bool BF, int T, int K>
__global__ __launch_bounds__(kRowThreads<T>) void rms_forward(RmsForward a) {
  __shared__ double slots[T / 64];
  const int t = threadIdx.x % T;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams<T> + threadIdx.x / T;
  if (row >= a.tokens) return;  // whole waves; only teams of one wave, which do not meet
  Raw8<BF> h[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int e = (j * T + t) * kLane;
    h[j] = load8<BF>(a.x, row * a.xs + e, a.features - e);
  }
  if (a.r) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int e = (j * T + t) * kLane;
      const Raw8<BF> r = load8<BF>(a.r, row * a.rs + e, a.features - e);
      float v[kLane];
#pragma unroll
      for (int i = 0; i < kLane; ++i) v[i] = h[j][i] + r[i];
      h[j] = rounded8<BF>(v);
      if constexpr (K >= 8) __builtin_amdgcn_sched_barrier(0);  // one piece of the residual at a time in registers
    }
  }
  // bf16 h, and y where the next product reads the codes, are read much later: non-temporal stores (h, y and codes of
  // 16384 x 4096 105 us, with ordinary stores 109; 16384 x 2048 55 / 59; 4096 x 2048 18 / 21; 512 x 4096 6.2 / 8.2; 64
  // and one row the same; fp32 ones lose 4%).  h beside y alone: 16384 x 4096 98 / 95 by itself, but 493 / 494 with
  // the 16-bit product that reads y behind it; 16384 x 2048 189 / 199 so, 8192 x 4096 246 / 252, 512 x 4096 52.2 / 52.9
  if (a.h) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int e = (j * T + t) * kLane;
      if (e < a.features) store8<BF, true>(a.h, row * a.hs + e, h[j], a.features - e);
    }
  }
  // fp64: an fp32 square overflows from 2^64 on, and is lost below 2^-75
  double s[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      const double d = h[j][i];
      s[i & 1] = __builtin_fma(d, d, s[i & 1]);
    }
  const double sum = team_sum<T>(s[0] + s[1], slots);
  const float rstd = static_cast<float>(1.0 / __builtin_sqrt(sum / a.features + a.eps));
  if (a.rstd && t == 0) a.rstd[row] = rstd;
  if (!a.y && !a.codes) return;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int e = (j * T + t) * kLane, n = a.features - e;
    float v[kLane];
    load_gain(a.gain, a.gain_bf16, e, n, v);
#pragma unroll
    for (int i = 0; i < kLane; ++i) v[i] = (h[j][i] * rstd) * v[i];
    if (a.y && n > 0) {
      if (a.codes) store8<BF, true>(a.y, row * a.ys + e, rounded8<BF>(v), n);
      else store8<BF>(a.y, row * a.ys + e, rounded8<BF>(v), n);
    }
    if (a.codes) {
      const uint32_t byte = scale_byte(row16_max(top_of(v)));
      if (n > 0) {
        store_codes(a.codes + row * a.cs + e, codes8(v, byte), n);
        if ((t & 15) == 0) a.scales[row * a.ss + e / kQBlock8] = static_cast<uint8_t>(byte);
      }
    }
    if constexpr (K >= 8) __builtin_amdgcn_sched_barrier(0);
  }
}

__device__ __forceinline__ void store_gain(const RmsBackward &a, int col, float v) {
  if (a.grad_bf16) {
    uint16_t *p = static_cast<uint16_t *>(a.dgain) + col;
    if (a.accumulate) v += __uint_as_float(static_cast<uint32_t>(*p) << 16);
    *p = static_cast<uint16_t>(bf16_bits(v));
  } else {
    float *p = static_cast<float *>(a.dgain) + col;
    *p = a.accumulate ? *p + v : v;
  }
}

// A team takes every gridDim.x kTeams-th row, the next one's loads under way
// while it works on one, and keeps its sums of dgain in registers; a
// workgroup's sums are one part, and the parts are added by rms_gain.  Rows too
// long for that (kHold false) are read again behind their sum, from the cache.
template <bool BF, int T, int K>
__global__ __launch_bounds__(kRowThreads<T>) void rms_backward(RmsBackward a) {
  constexpr bool kHold = T < 1024;
  constexpr int KH = kHold ? K : 1;
  __shared__ float slots[2][T / 64];
  __shared__ float join[kTeams<T> > 1 ? (kTeams<T> - 1) * T * K * kLane : 1];
  const int t = threadIdx.x % T, team = threadIdx.x / T;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams<T>;
  struct Row {
    Raw8<BF> dy[KH], h[KH], dh[KH];
    float rstd;
  };
  auto load = [&](const void *p, int64_t start, int j) {
    const int e = (j * T + t) * kLane;
    return load8<BF>(p, start + e, a.features - e);
  };
  auto fetch = [&](int64_t row, Row &r) {
    r.rstd = a.rstd[row];
    if constexpr (kHold) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        r.dy[j] = load(a.dy, row * a.dys, j);
        r.h[j] = load(a.h, row * a.hs, j);
        if (a.dh) r.dh[j] = load(a.dh, row * a.dhs, j);
      }
    }
  };
  float acc[K][kLane] = {};
  Row now, next;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams<T> + team;
  if (row < a.tokens) fetch(row, now);
  for (int parity = 0; row < a.tokens; row += step, parity ^= 1) {  // (a team of several waves: all of them)
    if (row + step < a.tokens) fetch(row + step, next);
    auto dy_of = [&](int j) {
      if constexpr (kHold) return now.dy[j];
      else return load(a.dy, row * a.dys, j);
    };
    auto h_of = [&](int j) {
      if constexpr (kHold) return now.h[j];
      else return load(a.h, row * a.hs, j);
    };
    float dot = 0;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int e = (j * T + t) * kLane, n = a.features - e;
      const Raw8<BF> dy = dy_of(j), h = h_of(j);
      float g[kLane];
      load_gain(a.gain, a.gain_bf16, e, n, g);
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        const float xhat = h[i] * now.rstd;
        acc[j][i] = __builtin_fmaf(dy[i], xhat, acc[j][i]);
        dot = __builtin_fmaf(dy[i] * g[i], xhat, dot);
      }
      if constexpr (!kHold) __builtin_amdgcn_sched_barrier(0);
    }
    const float mean = team_sum<T>(dot, slots[parity]) / static_cast<float>(a.features);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int e = (j * T + t) * kLane, n = a.features - e;
      const Raw8<BF> dy = dy_of(j), h = h_of(j);
      float g[kLane], v[kLane];
      load_gain(a.gain, a.gain_bf16, e, n, g);
#pragma unroll
      for (int i = 0; i < kLane; ++i) v[i] = __builtin_fmaf(h[i] * -now.rstd, mean, dy[i] * g[i]) * now.rstd;
      if (a.dh) {
        Raw8<BF> dh;
        if constexpr (kHold) dh = now.dh[j];
        else dh = load(a.dh, row * a.dhs, j);
#pragma unroll
        for (int i = 0; i < kLane; ++i) v[i] += dh[i];
      }
      if (n > 0) store8<BF>(a.dx, row * a.dxs + e, rounded8<BF>(v), n);
      if constexpr (!kHold) __builtin_amdgcn_sched_barrier(0);
    }
    now = next;
  }
  if constexpr (kTeams<T> > 1) {  // the workgroup's teams in their order
    if (team > 0) {
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < kLane; ++i) join[(((team - 1) * K + j) * kLane + i) * T + t] = acc[j][i];
    }
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int o = 0; o < kTeams<T> - 1; ++o)
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < kLane; ++i) acc[j][i] += join[((o * K + j) * kLane + i) * T + t];
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int e = (j * T + t) * kLane, n = a.features - e;
    if (gridDim.x == 1) {
#pragma unroll
      for (int i = 0; i < kLane; ++i)
        if (i < n) store_gain(a, e + i, acc[j][i]);
    } else if (n > 0) {
      store8<false>(a.parts, static_cast<int64_t>(blockIdx.x) * a.features + e, rounded8<false>(acc[j]), n);
    }
  }
}

// dgain of columns 32 b .. 32 b + 31: 8 lanes of four columns, 64 ranges of the
// parts, each added in order, then the ranges in order.  Bound by latency: 512
// parts of 4096 columns (8 MB, from the caches) take 4 us, with sums in fp64 as well.
constexpr int kGainCols = 32, kGainRanges = 64, kGainThreads = kGainCols / 4 * kGainRanges;
__global__ __launch_bounds__(kGainThreads) void rms_gain(RmsBackward a, int parts) {
  __shared__ double sums[kGainRanges][kGainCols];
  const int range = threadIdx.x / (kGainCols / 4), c = threadIdx.x % (kGainCols / 4) * 4;
  const int col = blockIdx.x * kGainCols + c, n = a.features - col;
  double s[4] = {0, 0, 0, 0};
#pragma unroll 8
  for (int p = range; p < parts; p += kGainRanges) {
    const fx4 v = n > 0 ? load4<false>(a.parts, static_cast<int64_t>(p) * a.features + col, n) : fx4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += v[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sums[range][c + i] = s[i];
  __syncthreads();
  const int mine = blockIdx.x * kGainCols + threadIdx.x;
  if (threadIdx.x >= kGainCols || mine >= a.features) return;
  double v = 0;
#pragma unroll 8
  for (int r = 0; r < kGainRanges; ++r) v += sums[r][threadIdx.x];
  store_gain(a, mine, static_cast<float>(v));
}

// Sixteen lanes to a block; a workgroup takes kQuantBlocks blocks of the rows'
// blocks, in their order, all loads first.  Bound by memory: 16384 bf16 rows of 4096
// take 37 us, 5.4 TB/s.
constexpr int kQuantThreads = 256, kQuantDeep = 4, kQuantBlocks = kQuantThreads / 16 * kQuantDeep;
template <bool BF>
__global__ __launch_bounds__(kQuantThreads) void quantize(QuantArgs a) {
  const int64_t blocks = (a.features + kQBlock8 - 1) / kQBlock8, total = blocks * a.tokens;
  const int part = threadIdx.x & 15;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kQuantBlocks; first < total;
       first += static_cast<int64_t>(gridDim.x) * kQuantBlocks) {
    const int64_t row0 = first / blocks;
    const uint32_t col0 = static_cast<uint32_t>(first - row0 * blocks);  // blocks: up to 2^15
    Raw8<BF> x[kQuantDeep];
    int64_t row[kQuantDeep];
    int block[kQuantDeep], n[kQuantDeep];
#pragma unroll
    for (int j = 0; j < kQuantDeep; ++j) {
      const uint32_t i = j * (kQuantThreads / 16) + threadIdx.x / 16, at = col0 + i;
      row[j] = row0 + at / static_cast<uint32_t>(blocks);
      block[j] = static_cast<int>(at % static_cast<uint32_t>(blocks));
      const int e = block[j] * kQBlock8 + part * kLane;
      n[j] = first + i < total ? static_cast<int>(a.features) - e : 0;
      x[j] = load8<BF>(a.x, row[j] * a.xs + e, n[j]);
    }
#pragma unroll
    for (int j = 0; j < kQuantDeep; ++j) {
      float v[kLane];
      widen(x[j], v);
      const uint32_t byte = scale_byte(row16_max(top_of(v)));
      if (n[j] <= 0) continue;
      store_codes(a.codes + row[j] * a.cs + block[j] * kQBlock8 + part * kLane, codes8(v, byte), n[j]);
      if (part == 0) a.scales[row[j] * a.ss + block[j]] = static_cast<uint8_t>(byte);
    }
  }
}

template <bool BF, int T, int K>
hipError_t forward(const RmsForward &a, hipStream_t s) {
  return launch(rms_forward<BF, T, K>, (a.tokens + kTeams<T> - 1) / kTeams<T>, 1, kRowThreads<T>, 0, s, a);
}

// Teams and pieces: few pieces to a thread, so that many rows are under way.
// Microseconds, bf16, residual, h, y and codes, all by ordinary stores (rows x
// features):
//   32768 x 512:   64 threads, 1 piece  33.3;  64, 2  35.5;  256, 1  60.8
//   16384 x 1024:  64, 2  33.9;  64, 4  36.7;  256, 1  39.4
//   16384 x 2048:  256, 1  57.2;  64, 4  62.0;  256, 2  61.3;  512, 1  71.6
//   16384 x 4096:  512, 1  107.6;  256, 2  110.7;  64, 8  124.9;  1024, 1  130.5
//   8192 x 8192:   512, 2  110.4;  256, 4  116.0;  1024, 1  112.3
// (5.6 TB/s; one row of 4096 takes 3.7 in the kernel with any of them.)
template <bool BF>
hipError_t forward_of(const RmsForward &a, hipStream_t s) {
  const int64_t c = (a.features + kLane - 1) / kLane;  // lanes of a row
  if (c <= 64) return forward<BF, 64, 1>(a, s);
  if (c <= 128) return forward<BF, 64, 2>(a, s);
  if (c <= 256) return forward<BF, 256, 1>(a, s);
  if (c <= 512) return forward<BF, 512, 1>(a, s);
  if (c <= 1024) return forward<BF, 512, 2>(a, s);
  if (c <= 2048) return forward<BF, 1024, 2>(a, s);
  if (c <= 4096) return forward<BF, 1024, 4>(a, s);
  return forward<BF, 1024, 8>(a, s);
}

// Workgroups of the backward pass at most, about those that run at once; each
// takes two rows at least (512 rows of 4096: 256 workgroups 13.0 us, 512 of them
// 14.8).
int32_t most_parts(int64_t features, bool bf16) {
  if (features <= 64 * kLane) return 1024;
  if (features <= 128 * kLane) return 512;
  if (features <= 256 * kLane) return bf16 ? 1024 : 512;
  return features <= 512 * kLane ? 512 : 256;
}

template <bool BF, int T, int K>
hipError_t backward(const RmsBackward &a, hipStream_t s) {
  const int64_t rows = 2 * kTeams<T>, teams = (a.tokens + rows - 1) / rows;
  const int64_t grid = std::min<int64_t>(teams, most_parts(a.features, BF));
  const LaunchEvents ev = t_launch_events;  // the call's mark goes on its last kernel
  if (grid > 1) t_launch_events = LaunchEvents{};
  const hipError_t e = launch(rms_backward<BF, T, K>, grid, 1, kRowThreads<T>, 0, s, a);
  t_launch_events = ev;
  if (e != hipSuccess || grid == 1) return e;
  return launch(rms_gain, (a.features + kGainCols - 1) / kGainCols, 1, kGainThreads, 0, s, a, static_cast<int>(grid));
}

// Teams, pieces and workgroups, by microseconds (bf16, with dh):
//   32768 x 512:   64 threads, 1 piece, 1024 workgroups  35.6;  64, 2, 1536  46.7
//   16384 x 1024:  64, 2, 512  40.1;  64, 2, 1024  43.6;  256, 1, 1024  47.5
//   16384 x 2048:  256, 1, 1024  61.9;  256, 1, 512  75.4;  512, 1, 512  74.6
//   16384 x 4096:  512, 1, 512  108.6;  256, 2, 768  113.9;  1024, 1, 256  163.9
//   8192 x 8192:   512, 2, 256  121.4;  256, 4, 512  123.2
//   fp32, 16384 x 2048:  256, 1, 512  100.9;  256, 1, 1024  107.6
template <bool BF>
hipError_t backward_of(const RmsBackward &a, hipStream_t s) {
  const int64_t c = (a.features + kLane - 1) / kLane;
  if (c <= 64) return backward<BF, 64, 1>(a, s);
  if (c <= 128) return backward<BF, 64, 2>(a, s);
  if (c <= 256) return backward<BF, 256, 1>(a, s);
  if (c <= 512) return backward<BF, 512, 1>(a, s);
  if (c <= 1024) return backward<BF, 512, 2>(a, s);
  if (c <= 2048) return backward<BF, 1024, 2>(a, s);
  if (c <= 4096) return backward<BF, 1024, 4>(a, s);
  return backward<BF, 1024, 8>(a, s);
}

}  // namespace

hipError_t quantize_rows(const QuantArgs &a, hipStream_t s) {
  const int64_t blocks = (a.features + kQBlock8 - 1) / kQBlock8;
  const int64_t grid = std::min<int64_t>((blocks * a.tokens + kQuantBlocks - 1) / kQuantBlocks, 1 << 22);
  return a.bf16 ? launch(quantize<true>, grid, 1, kQuantThreads, 0, s, a)
                : launch(quantize<false>, grid, 1, kQuantThreads, 0, s, a);
}

hipError_t rmsnorm_forward(const RmsForward &a, hipStream_t s) {
  return a.bf16 ? forward_of<true>(a, s) : forward_of<false>(a, s);
}

hipError_t rmsnorm_backward(const RmsBackward &a, hipStream_t s) {
  if (a.tokens == 0)
    return launch(rms_gain, (a.features + kGainCols - 1) / kGainCols, 1, kGainThreads, 0, s, a, 0);
  return a.bf16 ? backward_of<true>(a, s) : backward_of<false>(a, s);
}

int32_t rmsnorm_parts(int64_t features, bool bf16) { return most_parts(features, bf16); }

}  // namespace ar_dev

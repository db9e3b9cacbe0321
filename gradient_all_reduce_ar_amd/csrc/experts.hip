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
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kernels.hpp"
#include "operators.hpp"
#include "tiles.hpp"

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
constexpr int kBand = 8;
__device__ __forceinline__ void band_tile(int l, int mt, int nt, int &m, int &n) {
  const int g = l / (kBand * nt), first = g * kBand, in = min(kBand, mt - first), r = l - g * kBand * nt;
  m = first + r % in;
  n = r / in;
}

// This workgroup's tile: of `nt` column tiles times the row tiles of all
// experts, in runs of neighbours per XCD.
template <int BM>
__device__ __forceinline__ bool find_row_tile(const ExpertArgs &a, int nt, RowTile &t) {
  int carry = 0, lo, hi, total = 0;
  // the tiles up to and of this lane's expert, of the experts from e0 on
  auto scan = [&](int e0, int &mt, int &upto) {
    scan_ends(a, e0, carry, lo, hi);
    mt = (hi - lo + BM - 1) / BM;
    upto = wave_sum_to(mt);
    return __shfl(upto, 63);
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

// Forward (GRAD false: A = x, B = W_e as [n][k]) and input gradient (GRAD
// true: A = dy, B = W_e as [k][n]).
template <class P, bool GRAD>
__global__ __launch_bounds__(P::Sh::kThreads) void experts_rows(ExpertArgs a) {
  using S = typename P::Sh;
  using T = typename P::T;
  extern __shared__ __align__(16) char lds[];
  const int64_t n = GRAD ? a.in : a.outf, k = GRAD ? a.outf : a.in;
  const int nt = static_cast<int>((n + S::BN - 1) / S::BN);
  RowTile t;
  if (!find_row_tile<S::BM>(a, nt, t)) return;
  const int64_t n0 = static_cast<int64_t>(t.tile_n) * S::BN, ldx = GRAD ? a.dys : a.xs;
  const int validn = static_cast<int>(min(static_cast<int64_t>(S::BN), n - n0));
  const T *x = static_cast<const T *>(GRAD ? a.dy : a.x) + t.row * ldx;
  const T *w = static_cast<const T *>(a.w) + table_entry(a.offsets + t.e) + (GRAD ? n0 : n0 * a.in);
  P p;
  p.run(lds, x, w, ldx, a.in, t.rows, validn, static_cast<int>(k));
  using Out = TileOut<S, P::kLds>;
  Out::all(lds, p.acc, [&](int pass, int tid) {
    Out::rows(lds, pass, tid, [&](int m, int c, fx4 v) {
      if (m < t.rows && c < validn)
        store4<sizeof(T) == 2>(a.out, (t.row + m) * a.outs + n0 + c, v, validn - c);
    });
  });
}

// Forward for few rows per expert (decoding): the time is that of reading
// each active expert's weights once.  A workgroup takes 16 columns of one
// expert and up to 32 of its rows; its 8 waves take turns at 128-byte pieces
// of the weights' rows, so that the workgroup reads 1 KiB of each of the 16
// rows at a time, straight into the registers that feed the matrix
// instructions (lane l holds 32 bytes of weight row l % 16: any order of the
// contraction will do as long as x comes in the same), and the waves' sums
// are added in LDS in a fixed order.
constexpr int kFewWaves = 8, kFewRows = 32, kFewCols = 16;
template <bool BF>
struct Few {
  using T = std::conditional_t<BF, uint16_t, float>;
  static constexpr int kVec = 16 / sizeof(T);  // elements of a 16-byte load
  static constexpr int kPiece = 8 * kVec;      // of 128 bytes
  struct Piece {
    ux4 v[2];
  };
  // The lane's two loads of the piece at p (its own 32 bytes), of which the
  // first `n` elements exist.
  template <bool WHOLE>
  static __device__ __forceinline__ Piece load(const T *p, int64_t n) {
    Piece f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      f.v[c] = ux4{0, 0, 0, 0};
      if (WHOLE || n >= (c + 1) * kVec) {
        __builtin_memcpy(&f.v[c], p + c * kVec, 16);
      } else {
        T h[kVec] = {};
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (c * kVec + i < n) h[i] = p[c * kVec + i];
        __builtin_memcpy(&f.v[c], h, 16);
      }
    }
    return f;
  }
  static __device__ __forceinline__ fx4 add(const Piece &w, const Piece &x, fx4 acc) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      constexpr Elem E = BF ? kBF16 : kF32;
      acc = mfma16<E>(__builtin_bit_cast(Frag<E>, w.v[c]), __builtin_bit_cast(Frag<E>, x.v[c]), acc);
    }
    return acc;
  }
};

template <bool BF>
__global__ __launch_bounds__(64 * kFewWaves) void experts_few(ExpertArgs a) {
  using F = Few<BF>;
  using T = typename F::T;
  __shared__ fx4 part[kFewWaves][kFewRows / 16][64];
  RowTile t;
  if (!find_row_tile<kFewRows>(a, static_cast<int>((a.outf + kFewCols - 1) / kFewCols), t)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15;
  const int64_t n0 = static_cast<int64_t>(t.tile_n) * kFewCols, own = (lane >> 4) * 2 * F::kVec;
  // rows and columns that do not exist repeat the last one; not stored
  const T *w = static_cast<const T *>(a.w) + table_entry(a.offsets + t.e) + min(n0 + r, a.outf - 1) * a.in + own;
  const T *x0 = static_cast<const T *>(a.x) + (t.row + min(r, t.rows - 1)) * a.xs + own;
  const T *x1 = static_cast<const T *>(a.x) + (t.row + min(r + 16, t.rows - 1)) * a.xs + own;
  const bool two = t.rows > 16;
  fx4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  const int64_t whole = a.in / F::kPiece;
  constexpr int kBatch = 4;  // pieces in flight per wave
  int64_t b = wave;
  auto work = [&](auto n) {
    constexpr int N = decltype(n)::value;
    typename F::Piece fw[N], f0[N], f1[N];
#pragma unroll
    for (int i = 0; i < N; ++i) fw[i] = F::template load<true>(w + (b + i * kFewWaves) * F::kPiece, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) f0[i] = F::template load<true>(x0 + (b + i * kFewWaves) * F::kPiece, 0);
    if (two) {
#pragma unroll
      for (int i = 0; i < N; ++i) f1[i] = F::template load<true>(x1 + (b + i * kFewWaves) * F::kPiece, 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) acc[0] = F::add(fw[i], f0[i], acc[0]);
    if (two) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[1] = F::add(fw[i], f1[i], acc[1]);
    }
    b += N * kFewWaves;
  };
  while (b + (kBatch - 1) * kFewWaves < whole) work(std::integral_constant<int, kBatch>{});
  while (b < whole) work(std::integral_constant<int, 1>{});
  if (b == whole && a.in % F::kPiece != 0) {  // the piece that the rows end in
    const int64_t at = whole * F::kPiece, left = a.in - at - own;
    const typename F::Piece fw = F::template load<false>(w + at, left);
    acc[0] = F::add(fw, F::template load<false>(x0 + at, left), acc[0]);
    if (two) acc[1] = F::add(fw, F::template load<false>(x1 + at, left), acc[1]);
  }
  part[wave][0][lane] = acc[0];
  part[wave][1][lane] = acc[1];
  __syncthreads();
  if (wave > 1) return;
  fx4 v = part[0][wave][lane];
#pragma unroll
  for (int i = 1; i < kFewWaves; ++i) {
    const fx4 u = part[i][wave][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += u[e];
  }
  const int m = wave * 16 + r, left = static_cast<int>(min(static_cast<int64_t>(4), a.outf - n0 - (lane >> 4) * 4));
  if (m < t.rows && left > 0) store4<BF>(a.out, (t.row + m) * a.outs + n0 + (lane >> 4) * 4, v, left);
}

// One tile of one expert's weight gradient.
struct WeightTile {
  int e, row, rows;  // expert, its first row and number of rows
  int64_t m0, n0;
  int validm, validn;
};
template <class S>
__device__ __forceinline__ WeightTile weight_tile(const ExpertArgs &a, int64_t id) {
  WeightTile t;
  const int mt = static_cast<int>((a.outf + S::BM - 1) / S::BM), nt = static_cast<int>((a.in + S::BN - 1) / S::BN);
  const int per = mt * nt;
  int tm, tn;
  t.e = static_cast<int>(id / per);
  band_tile(static_cast<int>(id % per), mt, nt, tm, tn);
  int carry = 0, lo = 0, hi = 0;
  for (int e0 = 0; e0 <= t.e; e0 += 64) scan_ends(a, e0, carry, lo, hi);
  t.row = __builtin_amdgcn_readfirstlane(__shfl(lo, t.e & 63));
  t.rows = __builtin_amdgcn_readfirstlane(__shfl(hi, t.e & 63)) - t.row;
  t.m0 = static_cast<int64_t>(tm) * S::BM;
  t.n0 = static_cast<int64_t>(tn) * S::BN;
  t.validm = static_cast<int>(min(static_cast<int64_t>(S::BM), a.outf - t.m0));
  t.validn = static_cast<int>(min(static_cast<int64_t>(S::BN), a.in - t.n0));
  return t;
}

// One pass of the tile's way into the arena.
template <class Out, bool GBF>
__device__ __forceinline__ void store_weights(const ExpertArgs &a, const WeightTile &t, char *lds, int pass, int tid) {
  const int64_t out = table_entry(a.offsets + t.e) + t.m0 * a.in + t.n0;
  Out::rows(lds, pass, tid, [&](int m, int c, fx4 v) {
    if (m >= t.validm || c >= t.validn) return;
    const int64_t at = out + m * a.in + c;
    if (a.accumulate) {
      const fx4 old = load4<GBF>(a.out, at, t.validn - c);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += old[i];
    }
    store4<GBF, true>(a.out, at, v, t.validn - c);
  });
}

// Rows of one of `parts` parts of an expert's rows: whole stages.
__device__ __forceinline__ int part_rows(int rows, int parts) { return ((rows + parts - 1) / parts + 63) & ~63; }

// gridDim.y > 1: the expert's rows are cut into as many parts, whose sums go to
// slots (in the order that the threads hold them) for experts_join.
template <class P, bool GBF>
__global__ __launch_bounds__(P::Sh::kThreads) void experts_weights(ExpertArgs a) {
  using S = typename P::Sh;
  using T = typename P::T;
  extern __shared__ __align__(16) char lds[];
  // Tiles in the order of the workgroups, which go round the XCDs: all of the
  // device then writes one neighbourhood of the arena at a time (16384 rows,
  // 64 experts, 2048 x 1408: 227 us; 231 with a run of tiles per XCD).
  WeightTile t = weight_tile<S>(a, blockIdx.x);
  if (a.accumulate && t.rows == 0) return;
  const bool split = gridDim.y > 1;
  int row = t.row, rows = t.rows;
  if (split) {
    const int part = part_rows(t.rows, gridDim.y), at = part * static_cast<int>(blockIdx.y);
    if (at >= t.rows) return;
    row += at;
    rows = min(part, t.rows - at);
  }
  P p;
  p.run(lds, static_cast<const T *>(a.dy) + row * a.dys + t.m0, static_cast<const T *>(a.x) + row * a.xs + t.n0, a.dys,
        a.xs, t.validm, t.validn, rows);
  if constexpr (S::BM * S::BN == kExpertSlot) {
    if (split) {
      fx4 *slot = reinterpret_cast<fx4 *>(a.slots + (static_cast<int64_t>(blockIdx.x) * gridDim.y + blockIdx.y) * kExpertSlot) +
                  threadIdx.x;
#pragma unroll
      for (int i = 0; i < S::FM; ++i)
#pragma unroll
        for (int j = 0; j < S::FN; ++j) slot[(i * S::FN + j) * S::kThreads] = p.acc[i][j];
      return;
    }
  }
  using Out = TileOut<S, P::kLds>;
  Out::all(lds, p.acc, [&](int pass, int tid) { store_weights<Out, GBF>(a, t, lds, pass, tid); });
}

// Adds the parts of each tile in their order; one row of fragments of a tile
// per workgroup.
template <class S, bool GBF>
__global__ __launch_bounds__(S::kThreads) void experts_join(ExpertArgs a, int parts) {
  constexpr int kLds = 16 * S::WM * S::BN * 4;
  using Out = TileOut<S, kLds>;
  static_assert(Out::IP == 1, "one row of fragments");
  __shared__ __align__(16) char lds[kLds];
  const int64_t id = blockIdx.x / S::FM;
  const int pass = blockIdx.x % S::FM;
  const WeightTile t = weight_tile<S>(a, id);
  if (a.accumulate && t.rows == 0) return;
  const fx4 *slot = reinterpret_cast<const fx4 *>(a.slots + id * parts * kExpertSlot) +
                    static_cast<int64_t>(pass) * S::FN * S::kThreads + threadIdx.x;
  fx4 v[1][S::FN];
#pragma unroll
  for (int j = 0; j < S::FN; ++j) v[0][j] = fx4{0, 0, 0, 0};
  const int part = part_rows(t.rows, parts);
  for (int at = 0; at < t.rows; at += part) {
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
      const fx4 u = slot[j * S::kThreads];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][j][e] += u[e];
    }
    slot += kExpertSlot / 4;
  }
  Out::put(lds, v, threadIdx.x);
  __syncthreads();
  store_weights<Out, GBF>(a, t, lds, pass, threadIdx.x);
}

template <class K, class... A>
hipError_t launch(K kernel, int64_t grid, int parts, int threads, int lds, hipStream_t s, const A &...args) {
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

// Tiles.  Big runs one workgroup on a CU at 1.2 to 1.4 PFLOP/s, the others
// several.
using Big = Shape<256, 256, 2, 4>;
using Square = Shape<128, 128, 2, 2>;
using Half = Shape<64, 128, 2, 2>;
using Small = Shape<32, 64, 1, 4, 4>;

template <class S, bool GRAD>
int64_t row_tiles(const ExpertArgs &a) {
  const int64_t n = GRAD ? a.in : a.outf;
  return (a.tokens / S::BM + std::min<int64_t>(a.experts, a.tokens)) * ((n + S::BN - 1) / S::BN);
}

template <Elem E, class S, bool GRAD, bool ALIGNED>
hipError_t launch_rows(const ExpertArgs &a, hipStream_t s) {
  using P = TileProduct<E, S, kMajorK, GRAD ? kMajorMN : kMajorK, ALIGNED>;
  return launch(experts_rows<P, GRAD>, row_tiles<S, GRAD>(a), 1, S::kThreads, P::kLds, s, a);
}

template <class S, bool GRAD>
hipError_t launch_rows(const ExpertArgs &a, hipStream_t s) {
  if constexpr (S::BM >= 256) {  // aligned bf16 alone
    return launch_rows<kBF16, S, GRAD, true>(a, s);
  } else {
    if (a.aligned)
      return a.bf16 ? launch_rows<kBF16, S, GRAD, true>(a, s) : launch_rows<kF32, S, GRAD, true>(a, s);
    return a.bf16 ? launch_rows<kBF16, S, GRAD, false>(a, s) : launch_rows<kF32, S, GRAD, false>(a, s);
  }
}

// Which tile: the least of modelled times.  A tile's time is that of its
// contraction steps (of 64) and a rest; `slots` tiles run at once.  One
// workgroup on a CU goes faster than several (`alone`, launches of up to 256
// tiles).  The model against measured times, bf16 (rows, experts, in x out:
// Big / Square / Half / Small, microseconds):
//   16384, 8, 4096 x 12288:  1362 / 1823 / 2206 / 4184   measured 1403 / 1777 / 2227 / 4196
//   16384, 4, 2048 x 2048:    175 /  176 /  209 /  395             159 /  162 /  176 /  324
//   8192, 32, 2048 x 2048:    117 /  116 /  124 /  212             118 /  120 /  124 /  192
//   4096, 8, 1024 x 1024:      33 /   22 /   20 /   35              32 /   21 /   20 /   30
//   64, 32, 4096 x 1536:       95 /   72 /   67 /   32             106 /   93 /   91 /   77
// fp32 (Big, the matrix instructions' rate being a sixteenth, only lost: 4690
// in the first of these):
//   16384, 8, 4096 x 4096:       - / 4468 / 4180 / 5720   measured 4187 / 4120 / 5129
//   8192, 4, 2048 x 2048:        - /  661 /  598 /  759             632 /  574 /  678
//   3001, 8, 1024 x 1536:        - /  131 /   95 /  126             130 /  102 /  112
//   500, 4, 1000 x 1000:         - /   77 /   44 /   36              72 /   42 /   27
// The fp32 input gradients of these sizes by the tile that is chosen: 3782,
// 508, 111 and 20.
struct TileCost {
  double slots, alone, full, rest;
};
constexpr TileCost kBF16Cost[4] = {{256, 1.3, 1.45, 12}, {512, 0.65, 1.05, 5}, {768, 0.55, 0.98, 4}, {768, 0.4, 0.45, 3.5}};
constexpr TileCost kF32Cost[4] = {{}, {512, 4.5, 7.9, 5}, {768, 2.5, 5.7, 4}, {768, 0.9, 2.0, 3.5}};

template <class S, bool GRAD>
double rows_time(const ExpertArgs &a, const TileCost &c) {
  const double n = static_cast<double>(GRAD ? a.in : a.outf), steps = static_cast<double>(GRAD ? a.outf : a.in) / 64;
  const double e = static_cast<double>(std::min<int64_t>(a.experts, a.tokens)), t = static_cast<double>(a.tokens);
  // every expert ends inside a tile, half of it unused on average
  const double tiles = std::max(e, t / S::BM + e / 2) * std::ceil(n / S::BN);
  double rounds = tiles / c.slots;
  // short launches end with a round that is not full; in long ones with
  // several workgroups on a CU these end at different times
  rounds = rounds < 2 || c.slots <= 256 ? std::ceil(rounds) : rounds + 0.5;
  return rounds * (std::ceil(steps) * (tiles <= 256 ? c.alone : c.full) + c.rest);
}

// What a call launches: the tiles above, or experts_few.
enum Choice { kBig, kSquare, kHalf, kSmall, kFew };

template <bool GRAD>
Choice rows_choice(const ExpertArgs &a) {
  if constexpr (!GRAD) {
    // Short decoding calls, where latency counts: up to 16 MiB of weights, as
    // counted here.  Microseconds with experts_few / Small, bf16, weights from
    // memory (rows, active of experts, in x out: MiB):
    //   1, 1 of 8, 1024 x 512: 1          4.7 /  7.7
    //   8, 8 of 8, 1024 x 512: 8          5.8 /  8.4
    //   4, 4 of 8, 2048 x 1024: 16        7.7 / 13.1
    //   8, 8 of 8, 1024 x 1024: 16        9.8 /  8.5
    //   16, 8 of 8, 2048 x 1024: 32      13.7 / 15.1
    //   8, 8 of 8, 2048 x 2048: 64       25.3 / 19.0
    //   32, 20 of 32, 2048 x 1536: 192   45.9 / 31.3
    //   32, 20 of 32, 4096 x 1536: 384   65.1 / 56.9
    // Long rows of few experts (2 of 8, 4096 x 4096: 64 MiB) take 17.4 / 23.2;
    // fp32 meets at 128 MiB (8 of 8, 2048 x 2048: 37.1 / 36.8).
    const int64_t e = a.experts, bytes = std::min(e, a.tokens) * a.in * a.outf * (a.bf16 ? 2 : 4);
    if (a.tokens <= 16 * e && bytes <= 16 << 20) return kFew;
  }
  const TileCost *c = a.bf16 ? kBF16Cost : kF32Cost;
  const double big = a.aligned && a.bf16 ? rows_time<Big, GRAD>(a, c[0]) : 1e300;
  const double square = rows_time<Square, GRAD>(a, c[1]), half = rows_time<Half, GRAD>(a, c[2]);
  const double small = rows_time<Small, GRAD>(a, c[3]);
  if (big <= std::min({square, half, small})) return kBig;
  if (square <= std::min(half, small)) return kSquare;
  return half <= small ? kHalf : kSmall;
}

template <bool GRAD>
hipError_t rows(const ExpertArgs &a, hipStream_t s) {
  switch (rows_choice<GRAD>(a)) {
    case kBig: return launch_rows<Big, GRAD>(a, s);
    case kSquare: return launch_rows<Square, GRAD>(a, s);
    case kHalf: return launch_rows<Half, GRAD>(a, s);
    case kSmall: return launch_rows<Small, GRAD>(a, s);
    case kFew: break;
  }
  if constexpr (GRAD) return hipErrorInvalidValue;  // not chosen
  const int64_t grid = (a.tokens / kFewRows + std::min<int64_t>(a.experts, a.tokens)) * ((a.outf + kFewCols - 1) / kFewCols);
  return a.bf16 ? launch(experts_few<true>, grid, 1, 64 * kFewWaves, 0, s, a)
                : launch(experts_few<false>, grid, 1, 64 * kFewWaves, 0, s, a);
}

template <class S>
int64_t weight_tiles(const ExpertArgs &a) {
  return ((a.outf + S::BM - 1) / S::BM) * ((a.in + S::BN - 1) / S::BN) * a.experts;
}

// A split launch of few tiles: parts per expert, at least kPartRows rows each
// on average, and partial tiles for at most kMaxSlots workgroups.
constexpr int64_t kMaxSlots = 512, kMaxParts = 16, kPartRows = 256;
int64_t most_parts(int64_t tiles) { return tiles <= 0 ? 1 : std::clamp<int64_t>(kMaxSlots / tiles, 1, kMaxParts); }

// Parts of the rows of a launch of Half's tiles: 8001 rows of one expert, 512 x
// 768 (48 tiles): 73 us whole, 26 us in parts; 16000, 2, 1024 x 1024 (256
// tiles): 96 and 71.
int64_t weight_parts(const ExpertArgs &a) {
  return a.slots ? std::max<int64_t>(1, std::min(most_parts(weight_tiles<Half>(a)), a.tokens / a.experts / kPartRows)) : 1;
}

template <Elem E, class S, bool GBF, bool ALIGNED>
hipError_t launch_weights(const ExpertArgs &a, hipStream_t s) {
  using P = TileProduct<E, S, kMajorMN, kMajorMN, ALIGNED>;
  const int64_t tiles = weight_tiles<S>(a);
  if constexpr (S::BM * S::BN == kExpertSlot) {
    const int64_t parts = weight_parts(a);
    if (parts > 1) {
      const LaunchEvents ev = t_launch_events;  // the call's mark goes on its last kernel
      t_launch_events = LaunchEvents{};
      const hipError_t e =
          launch(experts_weights<P, GBF>, tiles, static_cast<int>(parts), S::kThreads, P::kLds, s, a);
      t_launch_events = ev;
      if (e != hipSuccess) return e;
      return launch(experts_join<S, GBF>, tiles * S::FM, 1, S::kThreads, 0, s, a, static_cast<int>(parts));
    }
  }
  return launch(experts_weights<P, GBF>, tiles, 1, S::kThreads, P::kLds, s, a);
}

template <Elem E, class S, bool ALIGNED>
hipError_t launch_weights_of(const ExpertArgs &a, hipStream_t s) {
  if constexpr (E == kF32) return launch_weights<E, S, false, ALIGNED>(a, s);
  else return a.grad_bf16 ? launch_weights<E, S, true, ALIGNED>(a, s) : launch_weights<E, S, false, ALIGNED>(a, s);
}

// Big where its tiles give every CU one and an expert's rows fill a few
// steps; Half where Square's would leave CUs idle, for fp32, and for operands
// that are not aligned if the rows are few.  Microseconds Big / Square / Half
// (rows, experts, in x out):
//   16384, 64, 2048 x 1408:         228 / 226 / 232
//   16384, 8, 4096 x 2048:          285 / 338 / 616
//   4096, 32, 2048 x 1024 (128 rows each, bf16 gradients): 68 / 64 / 66
//   16384, 2, 512 x 512 (32 square tiles):  212 / 118 / 36 (in parts)
//   8192, 8, 2047 x 2047:             - / 147 / 175
//   515, 24, 1025 x 511:              - / 18.6 / 16.6
//   fp32, 8192, 4, 2048 x 2048:       - / 505 / 508
//   fp32, 8192, 4, 2047 x 2047:       - / 600 / 608
// Adding to the arena reads it as well: the first of these takes 487 us instead
// of 255 (bf16 gradients 434 for 222), the fp32 one of 2048 x 2048 495 for 491.
// The choice knows the rows of all experts together: with all of 16384 rows
// going to one of 8 experts, 4096 x 2048 takes 329 us instead of 254, and 1024
// x 512, whose 32 tiles of that expert leave the other CUs idle, 159 for 33.
Choice weight_choice(const ExpertArgs &a) {
  const bool fill = a.tokens >= 256 * static_cast<int64_t>(a.experts);
  if (!a.bf16) return kHalf;
  if (a.aligned && fill && weight_tiles<Big>(a) >= 256) return kBig;
  return weight_tiles<Square>(a) < 256 || (!a.aligned && !fill) ? kHalf : kSquare;
}

template <class S>
ExpertShape shape_of(int64_t parts = 1) {
  return {S::BM, S::BN, static_cast<int32_t>(parts)};
}

}  // namespace

hipError_t experts_forward(const ExpertArgs &a, hipStream_t s) { return rows<false>(a, s); }
hipError_t experts_input_grad(const ExpertArgs &a, hipStream_t s) { return rows<true>(a, s); }

hipError_t experts_weight_grad(const ExpertArgs &a, hipStream_t s) {
  const Choice c = weight_choice(a);
  if (!a.bf16) return a.aligned ? launch_weights_of<kF32, Half, true>(a, s) : launch_weights_of<kF32, Half, false>(a, s);
  if (c == kBig) return launch_weights_of<kBF16, Big, true>(a, s);
  if (c == kHalf)
    return a.aligned ? launch_weights_of<kBF16, Half, true>(a, s) : launch_weights_of<kBF16, Half, false>(a, s);
  return a.aligned ? launch_weights_of<kBF16, Square, true>(a, s) : launch_weights_of<kBF16, Square, false>(a, s);
}

ExpertShape experts_shape(const ExpertArgs &a, ExpertProduct product) {
  const Choice c = product == kExpertsForward     ? rows_choice<false>(a)
                   : product == kExpertsInputGrad ? rows_choice<true>(a)
                                                  : weight_choice(a);
  switch (c) {
    case kBig: return shape_of<Big>();
    case kSquare: return shape_of<Square>();
    case kHalf: return shape_of<Half>(product == kExpertsWeightGrad ? weight_parts(a) : 1);
    case kSmall: return shape_of<Small>();
    case kFew: break;
  }
  return {kFewRows, kFewCols, 1};
}

int64_t experts_weight_slots(int64_t experts, int64_t in, int64_t outf) {
  static_assert(Half::BM * Half::BN == kExpertSlot, "Half's tiles are the ones that are split");
  ExpertArgs a{};
  a.experts = static_cast<int32_t>(experts);
  a.in = in;
  a.outf = outf;
  const int64_t tiles = weight_tiles<Half>(a), parts = most_parts(tiles);
  return parts > 1 ? tiles * parts : 0;
}

}  // namespace ar_dev

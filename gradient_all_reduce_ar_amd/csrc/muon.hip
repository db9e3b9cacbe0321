// muon.hip -- Newton-Schulz orthogonalisation and the Muon step (gfx950).
//
// Per matrix (m <= n; a tall one is worked on transposed):
//   U  = the gradient, or s G + mu M' with M' = mu M + s G
//   X  = U / (||U||_F + 1e-7)
//   A  = X X^T,  B = a I + b A + c A A,  X <- B X        (each step)
//   out = X, or W' = keep W - lr scale X
// All matrices of the plan share every launch: a workgroup takes one tile of
// a list that the host made once.  A and B are symmetric: only the tiles on
// and above the diagonal are computed, and each is stored twice.
//
// Numbers.  X, A and B are kept as fp16 or as a sum of two (hi + lo, 22
// bits), scaled by a power of two.  Singular values stay inside a bound that
// the host follows through the steps (X_0 has Frobenius norm at most 1), and
// no element of a matrix exceeds its largest singular value, so the scale
// that puts the bound under 2^15 puts every element inside fp16's range, and
// leaves elements 2^-29 of it still normal numbers.  A product of two sums is
// three products (hi hi + hi lo + lo hi; lo lo lies 2^-22 below), added into
// one fp32 sum.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernels.hpp"
#include "operators.hpp"
#include "tiles.hpp"

namespace ar_dev {
namespace {

constexpr double kEps = 1e-7;
constexpr int kThreads = 256;

template <bool BF>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  if constexpr (BF) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
  else return static_cast<const float *>(p)[i];
}
template <bool BF>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
  if constexpr (BF) static_cast<uint16_t *>(p)[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else static_cast<float *>(p)[i] = v;
}
// Four consecutive elements at any alignment (the hardware takes 8- and
// 16-byte loads and stores at any element's address).
template <bool BF>
__device__ __forceinline__ fx4 load4(const void *p, int64_t i) {
  if constexpr (BF) {
    ux2 u;
    __builtin_memcpy(&u, static_cast<const uint16_t *>(p) + i, 8);
    return fx4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u), __uint_as_float(u[1] << 16),
               __uint_as_float(u[1] & 0xffff0000u)};
  } else {
    fx4 v;
    __builtin_memcpy(&v, static_cast<const float *>(p) + i, 16);
    return v;
  }
}
template <bool BF>
__device__ __forceinline__ void store4(void *p, int64_t i, fx4 v) {
  if constexpr (BF) {
    uint16_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[k]));
    __builtin_memcpy(static_cast<uint16_t *>(p) + i, h, 8);
  } else {
    __builtin_memcpy(static_cast<float *>(p) + i, &v, 16);
  }
}

// M' and U of one element.
__device__ __forceinline__ float momentum_of(const MuonArgs &a, float g, float m) {
  return a.mu * m + a.gscale * g;
}
__device__ __forceinline__ float update_of(const MuonArgs &a, float g, float m1) {
  return a.nesterov ? a.gscale * g + a.mu * m1 : m1;
}

// Momentum, and the sum of squares of U over one part of a matrix (fp64).
template <bool GBF, bool STEP>
__global__ __launch_bounds__(kThreads) void muon_norm(MuonArgs a) {
  const MuonTile t = a.parts[blockIdx.x];
  const MuonMat &mat = a.mats[t.mat];
  const int64_t size = static_cast<int64_t>(mat.rows) * mat.cols;
  const int64_t lo = static_cast<int64_t>(t.m) * mat.chunk, hi = min(lo + mat.chunk, size);
  double sum = 0;
  auto one = [&](float g, float m, float &m1) {
    float u = g;
    if constexpr (STEP) {
      m1 = momentum_of(a, g, m);
      u = update_of(a, g, m1);
    }
    sum += static_cast<double>(u) * u;
  };
  for (int64_t i = lo + threadIdx.x * 4; i < hi; i += kThreads * 4) {
    const int64_t at = mat.at + i;
    if (i + 4 <= hi) {
      const fx4 g = load4<GBF>(a.g, at);
      fx4 m = {}, m1 = {};
      if constexpr (STEP) m = load4<false>(a.mom, at);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float r = 0;
        one(g[k], m[k], r);
        m1[k] = r;
      }
      if constexpr (STEP) store4<false>(a.mom_out, at, m1);
    } else {
      for (int k = 0; k < hi - i; ++k) {
        float r = 0;
        one(load1<GBF>(a.g, at + k), STEP ? a.mom[at + k] : 0.0f, r);
        if constexpr (STEP) a.mom_out[at + k] = r;
      }
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_down(sum, d);
  __shared__ double waves[kThreads / 64];
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0;
    for (int w = 0; w < kThreads / 64; ++w) s += waves[w];
    a.partials[mat.part0 + t.m] = s;
  }
}

// hi + lo of a number already scaled into fp16's range.
__device__ __forceinline__ void split(float v, _Float16 &hi, _Float16 &lo) {
  hi = static_cast<_Float16>(v);
  lo = static_cast<_Float16>(v - static_cast<float>(hi));
}
__device__ __forceinline__ void store_pair4(uint16_t *hi, uint16_t *lo, fx4 v, bool pair) {
  _Float16 h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(v[i], h[i], l[i]);
  __builtin_memcpy(__builtin_assume_aligned(hi, 8), h, 8);
  if (pair) __builtin_memcpy(__builtin_assume_aligned(lo, 8), l, 8);
}

// X_0: one 64 x 64 block of U, divided by the norm, scaled by 2^ex, turned if
// the matrix is tall, zeros in the padding.
template <bool GBF, bool STEP>
__global__ __launch_bounds__(kThreads) void muon_scale(MuonArgs a, int ex, bool pair) {
  const MuonTile t = a.blocks[blockIdx.x];
  const MuonMat &mat = a.mats[t.mat];
  double sum = 0;
  for (int i = threadIdx.x; i < mat.parts; i += kThreads) sum += a.partials[mat.part0 + i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  __shared__ double waves[kThreads / 64];
  __shared__ float turn[64][65];
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < kThreads / 64; ++w) sum += waves[w];
  const double inv = ldexp(1.0, ex) / (sqrt(sum) + kEps);
  const int r0 = (mat.tall ? t.n : t.m) * 64, c0 = (mat.tall ? t.m : t.n) * 64;  // of the matrix as given
  const int col = threadIdx.x % 16 * 4, row = threadIdx.x / 16;
  uint16_t *const x = a.ws + mat.x[0];
  const int64_t plane = static_cast<int64_t>(mat.mp) * mat.np;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = r0 + row + 16 * p, c = c0 + col;
    fx4 u = {};
    if (r < mat.rows && c < mat.cols) {
      const int64_t at = mat.at + static_cast<int64_t>(r) * mat.cols + c;
      fx4 g = {}, m1 = {};
      if (c + 4 <= mat.cols) {
        g = load4<GBF>(a.g, at);
        if constexpr (STEP) m1 = load4<false>(a.mom_out, at);
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (c + k < mat.cols) {
            g[k] = load1<GBF>(a.g, at + k);
            if constexpr (STEP) m1[k] = a.mom_out[at + k];
          }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = STEP ? update_of(a, g[k], m1[k]) : g[k];
        u[k] = c + k < mat.cols ? static_cast<float>(v * inv) : 0.0f;
      }
    }
    if (mat.tall) {
#pragma unroll
      for (int k = 0; k < 4; ++k) turn[col + k][row + 16 * p] = u[k];
    } else {
      const int64_t at = static_cast<int64_t>(r) * mat.np + c;
      store_pair4(x + at, x + plane + at, u, pair);
    }
  }
  if (!mat.tall) return;
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int m = row + 16 * p;
    fx4 u;
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = turn[m][col + k];
    const int64_t at = static_cast<int64_t>(c0 + m) * mat.np + r0 + col;
    store_pair4(x + at, x + plane + at, u, pair);
  }
}

// Workgroups go round the 8 XCDs (each with an L2 of its own) in turn; this
// gives every XCD one run of neighbouring tiles.
__device__ __forceinline__ int xcd_run(int p, int n) {
  const int q = n / 8, r = n % 8, x = p % 8;
  return x * q + min(x, r) + p / 8;
}

__device__ __forceinline__ float pow2(int e) { return ldexpf(1.0f, e); }

__device__ __forceinline__ fx4 times(fx4 v, float f) { return fx4{v[0] * f, v[1] * f, v[2] * f, v[3] * f}; }

// Stores C[m][n .. n+3] and, off the diagonal tiles, C[n .. n+3][m].
__device__ __forceinline__ void store_sym(uint16_t *c, int ld, int m, int n, fx4 v, bool pair, bool mirror) {
  const int64_t plane = static_cast<int64_t>(ld) * ld;
  const int64_t at = static_cast<int64_t>(m) * ld + n;
  store_pair4(c + at, c + plane + at, v, pair);
  if (!mirror) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    _Float16 h, l;
    split(v[i], h, l);
    const int64_t to = static_cast<int64_t>(n + i) * ld + m;
    c[to] = __builtin_bit_cast(uint16_t, h);
    if (pair) c[plane + to] = __builtin_bit_cast(uint16_t, l);
  }
}

// A = X X^T (POLY false) and B = a I + b A + c A A (POLY true).
template <class S, bool POLY>
__global__ __launch_bounds__(S::kThreads) void muon_sym(MuonArgs a, MuonStep k) {
  static_assert(S::BM == S::BN, "square tiles");
  extern __shared__ __align__(16) char lds[];
  const MuonTile t = a.sym[xcd_run(blockIdx.x, gridDim.x)];
  const MuonMat &mat = a.mats[t.mat];
  const int mp = mat.mp, m0 = t.m * S::BM, n0 = t.n * S::BN;
  const int64_t ld = POLY ? mp : mat.np;
  const uint16_t *src = a.ws + (POLY ? mat.a : mat.x[k.from]);
  const int64_t plane = mp * ld;
  const bool pair = k.pair_ab;  // then X is a pair too
  const uint16_t *hm = src + m0 * ld, *hn = src + n0 * ld;
  const uint16_t *sa[3] = {hm, hm, hm + plane}, *sb[3] = {hn, hn + plane, hn};
  using P = TileProduct<kF16, S, kMajorK, kMajorK, true>;
  P p;
  p.run(lds, sa, sb, pair ? 3 : 1, ld, ld, min(S::BM, mp - m0), min(S::BN, mp - n0), ld);
  const bool mirror = t.m != t.n;
  uint16_t *out = a.ws + (POLY ? mat.b : mat.a);
  if constexpr (!POLY) {
    const float f = pow2(k.ea - 2 * k.ex);
    p.each([&](int m, int n, fx4 v) {
      m += m0;
      n += n0;
      if (m < mp && n < mp) store_sym(out, mp, m, n, times(v, f), pair, mirror);
    });
  } else {
    const float fa = k.coef_a * pow2(k.eb), fb = k.coef_b * pow2(k.eb - k.ea), fc = k.coef_c * pow2(k.eb - 2 * k.ea);
    p.each([&](int m, int n, fx4 v) {
      m += m0;
      n += n0;
      if (m >= mp || n >= mp) return;
      const int64_t at = static_cast<int64_t>(m) * mp + n;
      _Float16 h[4], l[4] = {0, 0, 0, 0};
      __builtin_memcpy(h, __builtin_assume_aligned(src + at, 8), 8);
      if (pair) __builtin_memcpy(l, __builtin_assume_aligned(src + plane + at, 8), 8);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = fc * v[i] + fb * (static_cast<float>(h[i]) + static_cast<float>(l[i])) + (m == n + i ? fa : 0.0f);
      store_sym(out, mp, m, n, v, pair, mirror);
    });
  }
}

// X <- B X, or after the last step the result.
template <class S, bool LAST, bool WBF>
__global__ __launch_bounds__(S::kThreads) void muon_mul(MuonArgs a, MuonStep k) {
  extern __shared__ __align__(16) char lds[];
  const MuonTile t = a.full[xcd_run(blockIdx.x, gridDim.x)];
  const MuonMat &mat = a.mats[t.mat];
  const int mp = mat.mp, np = mat.np, m0 = t.m * S::BM, n0 = t.n * S::BN;
  const int64_t xplane = static_cast<int64_t>(mp) * np, bplane = static_cast<int64_t>(mp) * mp;
  const uint16_t *b = a.ws + mat.b + static_cast<int64_t>(m0) * mp, *x = a.ws + mat.x[k.from] + n0;
  const uint16_t *sa[3] = {b, b, b + bplane}, *sb[3] = {x, x + xplane, x};
  using P = TileProduct<kF16, S, kMajorK, kMajorMN, true>;
  P p;
  p.run(lds, sa, sb, k.pair_ab ? 3 : k.pair_x ? 2 : 1, mp, np, min(S::BM, mp - m0), min(S::BN, np - n0), mp);
  if constexpr (!LAST) {
    const float f = pow2(k.ex_next - k.eb - k.ex);
    uint16_t *out = a.ws + mat.x[k.from ^ 1];
    p.each([&](int m, int n, fx4 v) {
      m += m0;
      n += n0;
      if (m >= mp || n >= np) return;
      const int64_t at = static_cast<int64_t>(m) * np + n;
      store_pair4(out + at, out + xplane + at, times(v, f), k.pair_next);
    });
  } else {
    const float f = pow2(-k.eb - k.ex), lr = a.lr * mat.scale;
    p.each([&](int m, int n, fx4 v) {
      m += m0;
      n += n0;
      if (m >= mat.m || n >= mat.n) return;
      const int64_t stride = mat.tall ? mat.cols : 1;
      const int64_t at = mat.at + (mat.tall ? static_cast<int64_t>(n) * mat.cols + m
                                            : static_cast<int64_t>(m) * mat.cols + n);
      v = times(v, f);
      const int left = mat.n - n;
      if (!mat.tall && left >= 4) {
        if (a.step) {
          const fx4 w = load4<WBF>(a.w, at);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = a.keep * w[i] - lr * v[i];
        }
        store4<WBF>(a.w_out, at, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < left) {
            const int64_t to = at + i * stride;
            store1<WBF>(a.w_out, to, a.step ? a.keep * load1<WBF>(a.w, to) - lr * v[i] : v[i]);
          }
      }
    });
  }
}

using Shape0 = Shape<128, 128, 2, 2>;
using Shape1 = Shape<64, 64, 2, 2>;

template <class K, class... A>
hipError_t go(K kernel, int grid, int threads, int lds, hipStream_t s, const A &...args) {
  if (grid == 0) return hipSuccess;
  AR_LAUNCH(kernel, dim3(grid), dim3(threads), lds, s, args...);
  return hipGetLastError();
}

template <class S>
constexpr int lds_of() {
  return TileProduct<kF16, S, kMajorK, kMajorK, true>::kLds;
}

template <class S>
hipError_t mul(const MuonArgs &a, const MuonStep &k, hipStream_t s) {
  if (!k.last) return go(muon_mul<S, false, false>, a.nfull, S::kThreads, lds_of<S>(), s, a, k);
  return a.w_bf16 ? go(muon_mul<S, true, true>, a.nfull, S::kThreads, lds_of<S>(), s, a, k)
                  : go(muon_mul<S, true, false>, a.nfull, S::kThreads, lds_of<S>(), s, a, k);
}

}  // namespace

int muon_tile(int shape) { return shape == 0 ? Shape0::BM : Shape1::BM; }

hipError_t muon_begin(const MuonArgs &a, int32_t ex0, bool pair, hipStream_t s) {
  hipError_t e;
  if (a.step)
    e = a.g_bf16 ? go(muon_norm<true, true>, a.nparts, kThreads, 0, s, a)
                 : go(muon_norm<false, true>, a.nparts, kThreads, 0, s, a);
  else
    e = a.g_bf16 ? go(muon_norm<true, false>, a.nparts, kThreads, 0, s, a)
                 : go(muon_norm<false, false>, a.nparts, kThreads, 0, s, a);
  if (e != hipSuccess) return e;
  const int ex = ex0;
  if (a.step)
    return a.g_bf16 ? go(muon_scale<true, true>, a.nblocks, kThreads, 0, s, a, ex, pair)
                    : go(muon_scale<false, true>, a.nblocks, kThreads, 0, s, a, ex, pair);
  return a.g_bf16 ? go(muon_scale<true, false>, a.nblocks, kThreads, 0, s, a, ex, pair)
                  : go(muon_scale<false, false>, a.nblocks, kThreads, 0, s, a, ex, pair);
}

hipError_t muon_gram(const MuonArgs &a, const MuonStep &k, hipStream_t s) {
  if (a.shape_sym == 0) return go(muon_sym<Shape0, false>, a.nsym, Shape0::kThreads, lds_of<Shape0>(), s, a, k);
  return go(muon_sym<Shape1, false>, a.nsym, Shape1::kThreads, lds_of<Shape1>(), s, a, k);
}

hipError_t muon_poly(const MuonArgs &a, const MuonStep &k, hipStream_t s) {
  if (a.shape_sym == 0) return go(muon_sym<Shape0, true>, a.nsym, Shape0::kThreads, lds_of<Shape0>(), s, a, k);
  return go(muon_sym<Shape1, true>, a.nsym, Shape1::kThreads, lds_of<Shape1>(), s, a, k);
}

hipError_t muon_apply(const MuonArgs &a, const MuonStep &k, hipStream_t s) {
  return a.shape_full == 0 ? mul<Shape0>(a, k, s) : mul<Shape1>(a, k, s);
}

}  // namespace ar_dev

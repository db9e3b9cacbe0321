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
// Numbers.  X, A and B are kept as a sum of two fp16 (hi + lo, 22 bits),
// scaled by a power of two.  Singular values stay inside a bound that
// the host follows through the steps (X_0 has Frobenius norm at most 1), and
// no element of a matrix exceeds its largest singular value, so the scale
// that puts the bound under 2^15 puts every element inside fp16's range, and
// leaves elements 2^-29 of it still normal numbers.  (A matrix whose norm is
// below the constant beside it has a power of two of its own on top, from
// that norm: MuonStep.)  A product of two sums is
// three products (hi hi + hi lo + lo hi; lo lo lies 2^-22 below), added into
// one fp32 sum.  bf16 weights take the same: with A and B as one fp16, whose
// rounding (2^-12 at most) each step amplifies, and X as one in the last step,
// four 64 x 64 matrices came out 2.05e-3 off, 1.67e-3 being bf16's rounding.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernels.hpp"
#include "operators.hpp"
#include "tiles.hpp"

namespace ar_dev {
namespace {

constexpr double kEps = 1e-7;
constexpr int kThreads = 256;
constexpr int kJoinLds = 65536;  // of a join's workgroup: two to a CU

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
  const MuonTile t = table_entry(a.parts + blockIdx.x);
  const MuonMat mat = table_entry(a.mats + t.mat);
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

// d_0 of a matrix (MuonStep): 0 where the norm is zero, infinite or NaN.
__device__ __forceinline__ int first_shift(double norm) {
  const double r = norm / (norm + kEps);
  return r > 0 && r < 0.5 ? -ilogb(r) - 1 : 0;
}
__device__ __forceinline__ int next_shift(int d, const MuonStep &k) { return max(0, d - k.drop); }

// hi + lo of a number already scaled into fp16's range.
__device__ __forceinline__ void split(float v, _Float16 &hi, _Float16 &lo) {
  hi = static_cast<_Float16>(v);
  lo = static_cast<_Float16>(v - static_cast<float>(hi));
}
__device__ __forceinline__ void store_pair4(uint16_t *hi, uint16_t *lo, fx4 v) {
  _Float16 h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(v[i], h[i], l[i]);
  __builtin_memcpy(__builtin_assume_aligned(hi, 8), h, 8);
  __builtin_memcpy(__builtin_assume_aligned(lo, 8), l, 8);
}

// X_0: one 64 x 64 block of U, divided by the norm, scaled by 2^(ex0 + d_0),
// turned if the matrix is tall, zeros in the padding; and every step's d.
template <bool GBF, bool STEP>
__global__ __launch_bounds__(kThreads) void muon_scale(MuonArgs a, MuonSteps st) {
  const MuonTile t = table_entry(a.blocks + blockIdx.x);
  const MuonMat mat = table_entry(a.mats + t.mat);
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
  const double norm = sqrt(sum);
  int d = first_shift(norm);
  const double inv = ldexp(1.0, st.ex0 + d) / (norm + kEps);
  if (t.m == 0 && t.n == 0 && threadIdx.x == 0)
    for (int i = 0; i < st.n; ++i) {
      a.shifts[t.mat * kMuonMaxSteps + i] = d;
      d = next_shift(d, st.k[i]);
    }
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
      store_pair4(x + at, x + plane + at, u);
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
    store_pair4(x + at, x + plane + at, u);
  }
}

__device__ __forceinline__ float pow2(int e) { return ldexpf(1.0f, e); }

__device__ __forceinline__ fx4 times(fx4 v, float f) { return fx4{v[0] * f, v[1] * f, v[2] * f, v[3] * f}; }
__device__ __forceinline__ fx4 shifted(fx4 v, int e) {
  return fx4{ldexpf(v[0], e), ldexpf(v[1], e), ldexpf(v[2], e), ldexpf(v[3], e)};
}

// Where the sums of a tile go: row(m, n, v) takes C[m][n .. n + 3], column(m,
// n, v) takes C[m .. m + 3][n].  A and B are stored along rows, and off the
// diagonal tiles along columns too, as the transposed tile; a tall matrix's
// result, which is held transposed, along columns only.  d: the matrix's d_k
// (MuonStep), which A's factor does not need, as X's and A's cancel.
enum Product { kGram, kPoly, kMul, kLast };

// A = X X^T
struct FinishGram {
  uint16_t *out;
  int64_t plane;
  float f;
  int mp, ld;
  bool mirror;
  __device__ __forceinline__ FinishGram(const MuonArgs &a, const MuonStep &k, const MuonMat &mat, int, bool mir)
      : out(a.ws + mat.a), plane(static_cast<int64_t>(mat.mp) * mat.mp), f(pow2(k.ea - 2 * k.ex)), mp(mat.mp),
        ld(mat.mp), mirror(mir) {}
  __device__ __forceinline__ bool along_rows() const { return true; }
  __device__ __forceinline__ bool along_columns() const { return mirror; }
  __device__ __forceinline__ void put(int r, int c, fx4 v) const {
    if (r >= mp || c >= mp) return;
    const int64_t at = static_cast<int64_t>(r) * ld + c;
    store_pair4(out + at, out + plane + at, times(v, f));
  }
  __device__ __forceinline__ void row(int m, int n, fx4 v) const { put(m, n, v); }
  __device__ __forceinline__ void column(int m, int n, fx4 v) const { put(n, m, v); }
};

// B = a I + b A + c A A
struct FinishPoly {
  uint16_t *out;
  const uint16_t *src;
  int64_t plane;
  float fa, fb, fc;
  int mp, ld;
  bool mirror;
  __device__ __forceinline__ FinishPoly(const MuonArgs &a, const MuonStep &k, const MuonMat &mat, int d, bool mir)
      : out(a.ws + mat.b), src(a.ws + mat.a), plane(static_cast<int64_t>(mat.mp) * mat.mp),
        fa(k.coef_a * pow2(k.eb)), fb(k.coef_b * pow2(k.eb - k.ea - 2 * d)),
        fc(k.coef_c * pow2(k.eb - 2 * k.ea - 4 * d)), mp(mat.mp), ld(mat.mp), mirror(mir) {}
  __device__ __forceinline__ bool along_rows() const { return true; }
  __device__ __forceinline__ bool along_columns() const { return mirror; }
  // B[r][c .. c + 3]: A is as symmetric as its tiles were stored, so the
  // transposed tile reads it where it will lie itself
  __device__ __forceinline__ void put(int r, int c, fx4 v) const {
    if (r >= mp || c >= mp) return;
    const int64_t at = static_cast<int64_t>(r) * ld + c;
    _Float16 h[4], l[4];
    __builtin_memcpy(h, __builtin_assume_aligned(src + at, 8), 8);
    __builtin_memcpy(l, __builtin_assume_aligned(src + plane + at, 8), 8);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = fc * v[i] + fb * (static_cast<float>(h[i]) + static_cast<float>(l[i])) + (r == c + i ? fa : 0.0f);
    store_pair4(out + at, out + plane + at, v);
  }
  __device__ __forceinline__ void row(int m, int n, fx4 v) const { put(m, n, v); }
  __device__ __forceinline__ void column(int m, int n, fx4 v) const { put(n, m, v); }
};

// X <- B X
struct FinishMul {
  uint16_t *out;
  int64_t plane;
  float f;
  int mp, np, ld;
  __device__ __forceinline__ FinishMul(const MuonArgs &a, const MuonStep &k, const MuonMat &mat, int d, bool)
      : out(a.ws + (k.from ? mat.x[0] : mat.x[1])), plane(static_cast<int64_t>(mat.mp) * mat.np),
        f(pow2(k.ex_next + next_shift(d, k) - k.eb - k.ex - d)), mp(mat.mp), np(mat.np), ld(mat.np) {}
  __device__ __forceinline__ bool along_rows() const { return true; }
  __device__ __forceinline__ bool along_columns() const { return false; }
  __device__ __forceinline__ void row(int m, int n, fx4 v) const {
    if (m >= mp || n >= np) return;
    const int64_t at = static_cast<int64_t>(m) * ld + n;
    store_pair4(out + at, out + plane + at, times(v, f));
  }
  __device__ __forceinline__ void column(int, int, fx4) const {}
};

// The result: X, or the new weights.
template <bool WBF>
struct FinishLast {
  const void *w;
  void *w_out;
  int64_t at;
  float keep, lr;
  int e, m_, n_, cols;
  bool step, tall;
  __device__ __forceinline__ FinishLast(const MuonArgs &a, const MuonStep &k, const MuonMat &mat, int d, bool)
      : w(a.w), w_out(a.w_out), at(mat.at), keep(a.keep), lr(a.lr * mat.scale), e(-k.eb - k.ex - d), m_(mat.m),
        n_(mat.n), cols(mat.cols), step(a.step), tall(mat.tall) {}
  __device__ __forceinline__ bool along_rows() const { return !tall; }
  __device__ __forceinline__ bool along_columns() const { return tall; }
  // W[r][c .. c + 3] of the matrix as given, `left` columns from c on
  __device__ __forceinline__ void put(int r, int c, int left, fx4 v) const {
    v = shifted(v, e);
    const int64_t to = at + static_cast<int64_t>(r) * cols + c;
    if (left >= 4) {
      if (step) {
        const fx4 o = load4<WBF>(w, to);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = keep * o[i] - lr * v[i];
      }
      store4<WBF>(w_out, to, v);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) store1<WBF>(w_out, to + i, step ? keep * load1<WBF>(w, to + i) - lr * v[i] : v[i]);
    }
  }
  __device__ __forceinline__ void row(int m, int n, fx4 v) const {
    if (m < m_ && n < n_) put(m, n, n_ - n, v);
  }
  __device__ __forceinline__ void column(int m, int n, fx4 v) const {
    if (m < m_ && n < n_) put(n, m, m_ - m, v);
  }
};

template <class Out, class F>
__device__ __forceinline__ void leave(char *lds, int pass, int tid, int m0, int n0, const F &f) {
  if (f.along_rows()) Out::rows(lds, pass, tid, [&](int m, int n, fx4 v) { f.row(m0 + m, n0 + n, v); });
  if (f.along_columns()) Out::columns(lds, pass, tid, [&](int m, int n, fx4 v) { f.column(m0 + m, n0 + n, v); });
}

template <Product PR, bool WBF>
struct FinishOf {
  using type = FinishLast<WBF>;
};
template <>
struct FinishOf<kGram, false> {
  using type = FinishGram;
};
template <>
struct FinishOf<kPoly, false> {
  using type = FinishPoly;
};
template <>
struct FinishOf<kMul, false> {
  using type = FinishMul;
};

template <Product PR>
__device__ __forceinline__ const MuonWork &work_of(const MuonArgs &a) {
  return PR == kGram ? a.gram : PR == kPoly ? a.poly : a.mul;
}

__device__ __forceinline__ int shift_of(const MuonArgs &a, int mat, const MuonStep &k) {
  return table_entry(a.shifts + mat * kMuonMaxSteps + k.index);
}

// The products of one step: each workgroup works through its items.  A split
// item's sums are stored in the order that the threads hold them.
template <class S, Product PR, bool WBF>
__global__ __launch_bounds__(S::kThreads) void muon_product(MuonArgs a, MuonStep k) {
  constexpr bool kSym = PR == kGram || PR == kPoly;
  static_assert(S::BM == S::BN, "square tiles");
  extern __shared__ __align__(16) char lds[];
  const MuonWork &w = work_of<PR>(a);
  const int last = table_entry(w.first + blockIdx.x + 1);
  for (int it = table_entry(w.first + blockIdx.x); it < last; ++it) {
    const MuonItem t = table_entry(w.items + it);
    const MuonMat mat = table_entry(a.mats + t.mat);
    const int mp = mat.mp, cols = kSym ? mp : mat.np, m0 = t.m * S::BM, n0 = t.n * S::BN;
    const int64_t lda = PR == kGram ? mat.np : mat.mp, ldb = PR == kPoly ? mat.mp : mat.np;
    const uint16_t *x = a.ws + (k.from ? mat.x[1] : mat.x[0]) + t.k0 * (kSym ? 1 : ldb), *sq = a.ws + (PR == kPoly ? mat.a : mat.b) + t.k0;
    const uint16_t *pa = (PR == kGram ? x : sq) + m0 * lda;
    const uint16_t *pb = PR == kPoly ? sq + n0 * ldb : PR == kGram ? x + n0 * ldb : x + n0;
    using P = TileProduct<kF16, S, kMajorK, kSym ? kMajorK : kMajorMN, true>;
    P p;
    p.run(lds, pa, pb, lda, ldb, min(S::BM, mp - m0), min(S::BN, cols - n0), t.k1 - t.k0, 3, mp * lda, mp * ldb);
    if constexpr (S::BM * S::BN == kMuonSlot) {
      if (t.slot >= 0) {
        fx4 *slot = reinterpret_cast<fx4 *>(a.slots + static_cast<int64_t>(t.slot) * kMuonSlot) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < S::FM; ++i)
#pragma unroll
          for (int j = 0; j < S::FN; ++j) slot[(i * S::FN + j) * S::kThreads] = p.acc[i][j];
        continue;
      }
    }
    const typename FinishOf<PR, WBF>::type f(a, k, mat, shift_of(a, t.mat, k), t.m != t.n);
    using Out = TileOut<S, P::kLds>;
    Out::all(lds, p.acc, [&](int pass, int tid) { leave<Out>(lds, pass, tid, m0, n0, f); });
  }
}

// Split tiles: one pass of one tile's way out per workgroup.
template <class S, Product PR, bool WBF>
__global__ __launch_bounds__(S::kThreads) void muon_join(MuonArgs a, MuonStep k) {
  using Out = TileOut<S, kJoinLds>;
  extern __shared__ __align__(16) char lds[];
  const MuonWork &w = work_of<PR>(a);
  const MuonJoin t = table_entry(w.joins + blockIdx.x / Out::kPasses);
  const int pass = blockIdx.x % Out::kPasses;
  const MuonMat mat = table_entry(a.mats + t.mat);
  const fx4 *slot = reinterpret_cast<const fx4 *>(a.slots + static_cast<int64_t>(t.slot) * kMuonSlot) +
                    static_cast<int64_t>(pass) * Out::IP * S::FN * S::kThreads + threadIdx.x;
  fx4 v[Out::IP][S::FN];
#pragma unroll
  for (int i = 0; i < Out::IP; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j) v[i][j] = slot[(i * S::FN + j) * S::kThreads];
  for (int c = 1; c < t.count; ++c) {
    slot += kMuonSlot / 4;
#pragma unroll
    for (int i = 0; i < Out::IP; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const fx4 u = slot[(i * S::FN + j) * S::kThreads];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][j][e] += u[e];
      }
  }
  Out::put(lds, v, threadIdx.x);
  __syncthreads();
  const typename FinishOf<PR, WBF>::type f(a, k, mat, shift_of(a, t.mat, k), t.m != t.n);
  leave<Out>(lds, pass, threadIdx.x, t.m * S::BM, t.n * S::BN, f);
}

// ---- Small matrices: everything in one launch
//
// A matrix whose X (hi and lo) and A or B fit into the LDS is worked on by one
// workgroup from the gradient to the result.  The work is tens of matrix
// instructions per wave and step; what a step costs is the LDS's latency and
// five meetings, where a launch per product costs 4 to 6 us: four 64 x 64
// matrices took 65 us in 17 launches and take 18 us here.  Each wave has
// one block of every product, so that A can be overwritten by B and X by B X
// after a meeting; the code is kept short (loops, not unrolled), since most of
// it runs once and comes from memory.  m and n are padded with zeros to
// multiples of 32; rows have 32 bytes more than their elements, so that eight
// neighbouring rows start in different banks.
__host__ __device__ constexpr int64_t pad32(int64_t v) { return (v + 31) / 32 * 32; }
// Blocks of kRows x 32, one per wave: up to 64 x 64 in 8 waves of 16-row
// blocks, up to 16 of 32 x 32 (128 x 128, 64 x 256) in 16 waves.
template <bool TINY>
struct Small {
  static constexpr int kWaves = TINY ? 8 : 16, TX = TINY ? 1 : 2, kRows = 16 * TX, kThreads = 64 * kWaves;
};

template <int TX>  // 16-row fragments of the block: 1 or 2
struct SmallTask {
  static constexpr int kRows = 16 * TX;
  fx4 acc[TX][2];
  // kRows x 32 block at (i, j) of P Q over k, a multiple of 32.  P: rows of
  // `pp` bytes along k; Q: the same with QT (Q^T in memory), else rows along
  // the columns.  lo planes lie lp and lq bytes behind.
  template <bool QT>
  __device__ __forceinline__ void run(const char *p, int pp, int lp, const char *q, int pq, int lq, int i, int j, int k) {
    const int lane = threadIdx.x & 63;
    fx4 low[TX][2];  // hi lo + lo hi, added at the end (see TileProduct)
#pragma unroll
    for (int x = 0; x < TX; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) acc[x][y] = low[x][y] = fx4{0, 0, 0, 0};
    const char *pr = p + (i + (lane & 15)) * pp + (lane >> 4) * 16;
    const char *qr = QT ? q + (j + (lane & 15)) * pq + (lane >> 4) * 16
                        : q + ((lane >> 4) * 8 + ((lane & 15) >> 2)) * pq + j * 2 + (lane & 3) * 8;
    auto left = [&](int plane, int x, int ks) {
      return *reinterpret_cast<const s16x8 *>(pr + plane * lp + x * 16 * pp + ks * 64);
    };
    auto right = [&](int plane, int y, int ks) {
      if constexpr (QT) {
        return *reinterpret_cast<const s16x8 *>(qr + plane * lq + y * 16 * pq + ks * 64);
      } else {
        s16x4 h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          h[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)const_cast<char *>(
              qr + plane * lq + (ks * 32 + e * 4) * pq + y * 32));
        return s16x8(__builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
      }
    };
    for (int ks = 0; ks < k / 32; ++ks) {
      s16x8 ph[TX], qh[2], pl[TX], ql[2];
#pragma unroll
      for (int x = 0; x < TX; ++x) {
        ph[x] = left(0, x, ks);
        pl[x] = left(1, x, ks);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        qh[y] = right(0, y, ks);
        ql[y] = right(1, y, ks);
      }
#pragma unroll
      for (int x = 0; x < TX; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          acc[x][y] = mfma16<kF16>(qh[y], ph[x], acc[x][y]);
          low[x][y] = mfma16<kF16>(ql[y], ph[x], low[x][y]);
          low[x][y] = mfma16<kF16>(qh[y], pl[x], low[x][y]);
        }
    }
#pragma unroll
    for (int x = 0; x < TX; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[x][y][e] += low[x][y][e];
  }
  // f(m, n, v): v holds [m][n .. n + 3] of the product.
  template <class F>
  __device__ __forceinline__ void each(int i, int j, F f) const {
    const_cast<SmallTask *>(this)->change(i, j, [&](int m, int n, const fx4 &v) { f(m, n, v); });
  }
  template <class F>
  __device__ __forceinline__ void change(int i, int j, F f) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int x = 0; x < TX; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) f(i + x * 16 + (lane & 15), j + y * 16 + (lane >> 4) * 4, acc[x][y]);
  }
};

template <bool GBF, bool WBF, bool STEP, bool TINY>
__global__ __launch_bounds__(Small<TINY>::kThreads) void muon_small_kernel(MuonArgs a, MuonSteps st) {
  using Sm = Small<TINY>;
  extern __shared__ __align__(16) char lds[];
  __shared__ double sums[Sm::kWaves];
  const MuonMat mat = table_entry(a.mats + blockIdx.x);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mp = static_cast<int>(pad32(mat.m)), np = static_cast<int>(pad32(mat.n));
  const int px = np * 2 + 32, pq = mp * 2 + 32, lx = mp * px, lq = mp * pq;
  char *const x = lds, *const q = lds + 2 * lx;
  const int cols = mat.cols, size = mat.rows * cols, whole = size & ~3;
  // momentum and norm; the last size % 4 elements one by one
  double sum = 0;
#pragma unroll 2
  for (int i = tid * 4; i < whole; i += Sm::kThreads * 4) {
    const int64_t at = mat.at + i;
    fx4 u = load4<GBF>(a.g, at);
    if constexpr (STEP) {
      fx4 m = load4<false>(a.mom, at);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[e] = momentum_of(a, u[e], m[e]);
        u[e] = update_of(a, u[e], m[e]);
      }
      store4<false>(a.mom_out, at, m);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += static_cast<double>(u[e]) * u[e];
  }
  if (whole + tid < size) {
    const int64_t at = mat.at + whole + tid;
    float u = load1<GBF>(a.g, at);
    if constexpr (STEP) {
      const float m1 = momentum_of(a, u, a.mom[at]);
      a.mom_out[at] = m1;
      u = update_of(a, u, m1);
    }
    sum += static_cast<double>(u) * u;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((tid & 63) == 0) sums[wave] = sum;
  for (int i = tid * 16; i < 2 * lx; i += Sm::kThreads * 16) *reinterpret_cast<ux4 *>(x + i) = ux4{0, 0, 0, 0};
  __syncthreads();  // also: the new momentum can be read back
  sum = 0;
  for (int w = 0; w < Sm::kWaves; ++w) sum += sums[w];
  const double norm = sqrt(sum);
  int d = first_shift(norm);
  const double inv = ldexp(1.0, st.ex0 + d) / (norm + kEps);
  auto fill = [&](int r, int c, float u) {
    _Float16 hi, lo;
    split(static_cast<float>(u * inv), hi, lo);
    char *to = mat.tall ? x + c * px + r * 2 : x + r * px + c * 2;
    *reinterpret_cast<_Float16 *>(to) = hi;
    *reinterpret_cast<_Float16 *>(to + lx) = lo;
  };
  for (int i = tid * 4; i < whole; i += Sm::kThreads * 4) {
    const int64_t at = mat.at + i;
    fx4 u = load4<GBF>(a.g, at);
    if constexpr (STEP) {
      const fx4 m1 = load4<false>(a.mom_out, at);
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = update_of(a, u[e], m1[e]);
    }
    int r = i / cols, c = i - r * cols;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      fill(r, c, u[e]);
      if (++c == cols) {
        c = 0;
        ++r;
      }
    }
  }
  if (whole + tid < size) {
    const int i = whole + tid;
    const float g = load1<GBF>(a.g, mat.at + i);
    fill(i / cols, i % cols, STEP ? update_of(a, g, a.mom_out[mat.at + i]) : g);
  }
  __syncthreads();

  // the wave's blocks of A and B (i, ja) and of X (i2, jx)
  const int nb = mp / Sm::kRows, nm = mp / 32, nn = np / 32;
  const bool square = wave < nb * nm, wide = wave < nb * nn;
  const int i = wave / nm * Sm::kRows, j = wave % nm * 32, ix = wave / nn * Sm::kRows, jx = wave % nn * 32;
  auto put = [&](char *base, int pitch, int plane, int m, int n, fx4 v) {
    char *to = base + m * pitch + n * 2;
    store_pair4(reinterpret_cast<uint16_t *>(to), reinterpret_cast<uint16_t *>(to + plane), v);
  };
  SmallTask<Sm::TX> task;
  for (int step = 0; step < st.n; ++step) {
    const MuonStep &k = st.k[step];
    if (square) {  // A = X X^T
      const float f = pow2(k.ea - 2 * k.ex);
      task.template run<true>(x, px, lx, x, px, lx, i, j, np);
      task.each(i, j, [&](int m, int n, fx4 v) { put(q, pq, lq, m, n, times(v, f)); });
    }
    __syncthreads();
    if (square) {  // B = a I + b A + c A A
      const float fa = k.coef_a * pow2(k.eb), fb = k.coef_b * pow2(k.eb - k.ea - 2 * d);
      const float fc = k.coef_c * pow2(k.eb - 2 * k.ea - 4 * d);
      task.template run<true>(q, pq, lq, q, pq, lq, i, j, mp);
      task.change(i, j, [&](int m, int n, fx4 &v) {
        const char *p = q + m * pq + n * 2;
        _Float16 h[4], l[4];
        __builtin_memcpy(h, __builtin_assume_aligned(p, 8), 8);
        __builtin_memcpy(l, __builtin_assume_aligned(p + lq, 8), 8);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = fc * v[e] + fb * (static_cast<float>(h[e]) + static_cast<float>(l[e])) + (m == n + e ? fa : 0.0f);
      });
    }
    __syncthreads();
    if (square) task.each(i, j, [&](int m, int n, fx4 v) { put(q, pq, lq, m, n, v); });
    __syncthreads();
    if (wide) task.template run<false>(q, pq, lq, x, px, lx, ix, jx, mp);
    if (k.last) break;
    __syncthreads();
    const int next = next_shift(d, k);
    if (wide) {  // X <- B X
      const float f = pow2(k.ex_next + next - k.eb - k.ex - d);
      task.each(ix, jx, [&](int m, int n, fx4 v) { put(x, px, lx, m, n, times(v, f)); });
    }
    d = next;
    __syncthreads();
  }
  if (!wide) return;
  const FinishLast<WBF> f(a, st.k[st.n - 1], mat, d, false);
  task.each(ix, jx, [&](int m, int n, fx4 v) {
    if (!mat.tall) {
      f.row(m, n, v);
    } else if (m < mat.m) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < mat.n) f.put(n + e, m, 1, fx4{v[e], 0, 0, 0});
    }
  });
}

using Shape0 = Shape<256, 256, 2, 4>;
using Shape1 = Shape<128, 128, 2, 2>;
using Shape2 = Shape<64, 64, 2, 2, 4>;

template <class K, class... A>
hipError_t go(K kernel, int grid, int threads, int lds, hipStream_t s, const A &...args) {
  if (grid == 0) return hipSuccess;
  if (lds > 65536) {  // more than 64 KB of LDS has to be asked for
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  AR_LAUNCH(kernel, dim3(grid), dim3(threads), lds, s, args...);
  return hipGetLastError();
}

template <class S>
constexpr int lds_of() {
  return TileProduct<kF16, S, kMajorK, kMajorK, true>::kLds;
}

template <class S, Product PR, bool WBF>
hipError_t product_of(const MuonArgs &a, const MuonWork &w, const MuonStep &k, hipStream_t s) {
  // the call's mark goes on its last kernel
  const LaunchEvents ev = t_launch_events;
  if (w.njoins > 0) t_launch_events = LaunchEvents{};
  const hipError_t e = go(muon_product<S, PR, WBF>, w.groups, S::kThreads, lds_of<S>(), s, a, k);
  t_launch_events = ev;
  if (e != hipSuccess || w.njoins == 0) return e;
  if constexpr (S::BM * S::BN == kMuonSlot)
    return go(muon_join<S, PR, WBF>, w.njoins * TileOut<S, kJoinLds>::kPasses, S::kThreads, kJoinLds, s, a, k);
  else
    return hipErrorInvalidValue;  // only the largest tiles are split
}

template <Product PR, bool WBF>
hipError_t product(const MuonArgs &a, const MuonWork &w, const MuonStep &k, hipStream_t s) {
  return w.shape == 0   ? product_of<Shape0, PR, WBF>(a, w, k, s)
         : w.shape == 1 ? product_of<Shape1, PR, WBF>(a, w, k, s)
                        : product_of<Shape2, PR, WBF>(a, w, k, s);
}

}  // namespace

int muon_tile(int shape) { return shape == 0 ? Shape0::BM : shape == 1 ? Shape1::BM : Shape2::BM; }

int64_t muon_small_lds(int64_t m, int64_t n) {
  const int64_t mp = pad32(m), np = pad32(n);
  // one block for each of the 16 waves; then the LDS holds it
  return mp / 32 * (np / 32) <= Small<false>::kWaves ? 2 * mp * (np * 2 + 32 + mp * 2 + 32) : 0;
}

namespace {

template <bool TINY>
hipError_t small(const MuonArgs &a, const MuonSteps &k, int32_t nmats, int32_t lds, hipStream_t s) {
  constexpr int t = Small<TINY>::kThreads;
  if (a.step)
    return a.g_bf16 ? (a.w_bf16 ? go(muon_small_kernel<true, true, true, TINY>, nmats, t, lds, s, a, k)
                                : go(muon_small_kernel<true, false, true, TINY>, nmats, t, lds, s, a, k))
                    : (a.w_bf16 ? go(muon_small_kernel<false, true, true, TINY>, nmats, t, lds, s, a, k)
                                : go(muon_small_kernel<false, false, true, TINY>, nmats, t, lds, s, a, k));
  return a.g_bf16 ? (a.w_bf16 ? go(muon_small_kernel<true, true, false, TINY>, nmats, t, lds, s, a, k)
                              : go(muon_small_kernel<true, false, false, TINY>, nmats, t, lds, s, a, k))
                  : (a.w_bf16 ? go(muon_small_kernel<false, true, false, TINY>, nmats, t, lds, s, a, k)
                              : go(muon_small_kernel<false, false, false, TINY>, nmats, t, lds, s, a, k));
}

}  // namespace

hipError_t muon_small(const MuonArgs &a, const MuonSteps &k, int32_t nmats, int32_t lds, bool tiny, hipStream_t s) {
  return tiny ? small<true>(a, k, nmats, lds, s) : small<false>(a, k, nmats, lds, s);
}

hipError_t muon_begin(const MuonArgs &a, const MuonSteps &k, hipStream_t s) {
  hipError_t e;
  if (a.step)
    e = a.g_bf16 ? go(muon_norm<true, true>, a.nparts, kThreads, 0, s, a)
                 : go(muon_norm<false, true>, a.nparts, kThreads, 0, s, a);
  else
    e = a.g_bf16 ? go(muon_norm<true, false>, a.nparts, kThreads, 0, s, a)
                 : go(muon_norm<false, false>, a.nparts, kThreads, 0, s, a);
  if (e != hipSuccess) return e;
  if (a.step)
    return a.g_bf16 ? go(muon_scale<true, true>, a.nblocks, kThreads, 0, s, a, k)
                    : go(muon_scale<false, true>, a.nblocks, kThreads, 0, s, a, k);
  return a.g_bf16 ? go(muon_scale<true, false>, a.nblocks, kThreads, 0, s, a, k)
                  : go(muon_scale<false, false>, a.nblocks, kThreads, 0, s, a, k);
}

hipError_t muon_gram(const MuonArgs &a, const MuonStep &k, hipStream_t s) {
  return product<kGram, false>(a, a.gram, k, s);
}

hipError_t muon_poly(const MuonArgs &a, const MuonStep &k, hipStream_t s) {
  return product<kPoly, false>(a, a.poly, k, s);
}

hipError_t muon_apply(const MuonArgs &a, const MuonStep &k, hipStream_t s) {
  if (!k.last) return product<kMul, false>(a, a.mul, k, s);
  return a.w_bf16 ? product<kLast, true>(a, a.mul, k, s) : product<kLast, false>(a, a.mul, k, s);
}

}  // namespace ar_dev

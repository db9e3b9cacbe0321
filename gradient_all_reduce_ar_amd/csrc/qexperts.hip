// qexperts.hip -- matrix products grouped by expert on 8-bit rows and weights
// with a power of two for each block of 128 (gfx950): forward and input
// gradient of a mixture of experts' linear layers, and the quantisation of the
// weights.
//
//   forward      y[t, o]  = sum over blocks b of 2^(sx[t,b] + sw[o/128,b] - 254) sum_{i in b} qx[t,i] qw[o,i]
//   input grad   dx[t, i] = the same over o, with sw[b,i/128]
//
// A stage of the contraction is one block of 128: one matrix instruction
// (16x16x128) of two fragments, which takes each lane's scale byte of either
// operand with it, so the scales cost no arithmetic.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "grouped.hpp"
#include "kernels.hpp"
#include "operators.hpp"
#include "rows.hpp"
#include "tiles.hpp"

namespace ar_dev {
namespace {

// 32 codes of one row or column: contraction elements 16 g .. and 64 + 16 g ..
// (g: the lane's group of 16), in this order in both operands.
struct Frag8 {
  ux4 v[2];
};

// Sums of 128 products and c.  The 8-bit instruction adds 8 neighbours of the
// contraction at a time (8 bytes of a lane), and of each product cuts off, towards
// zero, what is below 2^-13 of 2^E, E the largest sum of two codes' exponents
// among the 8: less than 7 2^(E - 13) of each eight.  The eights' sums and c are
// added in fp32.  That is 1.2e-5 of the result on normal inputs and 5.8e-5 where
// one row element is 448 among ones; rounding to bf16 takes 1.7e-3, and the codes
// themselves are off by up to 2^-4.  It runs at twice the rate of the 16-bit
// instructions, which lose nothing: fp32 results take those.
__device__ __forceinline__ fx4 mfma8(const Frag8 &a, const Frag8 &b, fx4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(ix8, a), __builtin_bit_cast(ix8, b), c, 0,
                                                          0, 0, sa, 0, sb);
}

// fp32 results: the codes as bf16, which holds them exactly, so that the
// products are exact and their sums fp32; a block's sum takes its scales then.
struct Wide8 {
  s16x8 v[4];
};
__device__ __forceinline__ Wide8 widen8(const Frag8 &f) {
  Wide8 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t q = f.v[i >> 1][(i & 1) * 2 + j];
      u[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, 1.0f, false));
      u[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, 1.0f, true));
    }
    __builtin_memcpy(&w.v[i], u, 16);
  }
  return w;
}
__device__ __forceinline__ fx4 mfma_wide(const Wide8 &a, const Wide8 &b, fx4 c, int sa, int sb) {
  fx4 z = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) z = mfma16<kBF16>(a.v[i], b.v[i], z);
  const bool nan = sa == 255 || sb == 255;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] += nan ? __builtin_nanf("") : __builtin_ldexpf(z[i], sa + sb - 254);
  return c;
}

// A matrix of scales: byte (row, block) at base + row * by_row + block * by_block.
struct Scales {
  const uint8_t *base;
  int64_t by_row, by_block;
  int rows;    // that exist (those beyond take the last one's)
  int blocks;  // of the contraction
};

// The scales of 32 blocks of a tile, in the LDS: rows of 32 bytes, 36 apart, so
// that 16 rows' bytes lie in different banks; the tile's rows, then its blocks
// of columns.
constexpr int kScaleChunk = 32, kScalePitch = 36;
template <int BM, int BN, int NT>
struct ScaleChunk {
  static constexpr int kColBlocks = (BN + 127) / 128, kUnits = BM * (kScaleChunk / 4);
  static constexpr int kBytes = ((BM + kColBlocks) * kScalePitch + 15) / 16 * 16;

  // Those of blocks b0 .. b0 + 31 that exist.
  static __device__ __forceinline__ void move(char *lds, const Scales &sa, const Scales &sb, int b0) {
    const int n = min(kScaleChunk, sa.blocks - b0);
#pragma unroll
    for (int u0 = 0; u0 < kUnits; u0 += NT) {
      const int u = u0 + static_cast<int>(threadIdx.x), row = u / (kScaleChunk / 4), b = u % (kScaleChunk / 4) * 4;
      if (b >= n || row >= BM) continue;
      const uint8_t *p = sa.base + min(row, sa.rows - 1) * sa.by_row + b0 + b;
      uint32_t v = 0;
      if (b + 4 <= n) {
        __builtin_memcpy(&v, p, 4);
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (b + i < n) v |= static_cast<uint32_t>(p[i]) << (8 * i);
      }
      *reinterpret_cast<uint32_t *>(lds + row * kScalePitch + b) = v;
    }
    const int c = threadIdx.x / kScaleChunk, b = threadIdx.x % kScaleChunk;
    if (c < kColBlocks && b < n)
      lds[(BM + c) * kScalePitch + b] = static_cast<char>(sb.base[min(c, sb.rows - 1) * sb.by_row + (b0 + b) * sb.by_block]);
  }
};

// The tile product of 8-bit operands: Operand's stages, in one loop (of the
// loops that TileProduct has, those of smaller tiles), with the scales of 32
// blocks at a time beside them in the LDS.
template <bool EXACT, class S, Major BMJ, bool ALIGNED>
struct TileProduct8 {
  using Sh = S;
  using OpA = Operand<kF8, kMajorK, S::BM, S::kThreads, ALIGNED>;
  using OpB = Operand<kF8, BMJ, S::BN, S::kThreads, ALIGNED>;
  static constexpr int kStep = 128;
  static constexpr int kStage = OpA::kBytes + OpB::kBytes;
  static constexpr int kStages = ALIGNED ? S::kStages : 2;
  using Chunk = ScaleChunk<S::BM, S::BN, S::kThreads>;
  static constexpr int kChunk = kScaleChunk, kPitch = kScalePitch, kScales = Chunk::kBytes;
  static constexpr int kLds = kStages * kStage + kScales;
  fx4 acc[S::FM][S::FN];
  OpA oa;
  OpB ob;
  int k, at, per;  // stage `at` of `per` is loaded next

  __device__ __forceinline__ void next_stage() {
    if (++at < per) {
      oa.advance();
      ob.advance();
    }
  }
  __device__ __forceinline__ void load(uint32_t stage) {
    const int n = k - at * kStep;
    if (n < kStep) {
      oa.cut(n);
      ob.cut(n);
    }
    oa.load(stage);
    ob.load(stage + OpA::kBytes);
    next_stage();
  }
  __device__ __forceinline__ void fetch(int set) {
    oa.fetch(set, k - at * kStep);
    ob.fetch(set, k - at * kStep);
    next_stage();
  }
  __device__ __forceinline__ void land(int set, char *stage) {
    oa.land(set, stage);
    ob.land(set, stage + OpA::kBytes);
  }

  // The products of the stage at sa, block b of the chunk.
  __device__ __forceinline__ void multiply(const char *sa, const char *scales, int b, int rm, int rn) {
    const char *sb = sa + OpA::kBytes;
    const int lane = threadIdx.x & 63;
    const int colscale = static_cast<uint8_t>(scales[(S::BM + rn / 128) * kPitch + b]);
    auto a_of = [&](int i) { return Frag8{{OpA::fragment(sa, rm + i * 16, 0), OpA::fragment(sa, rm + i * 16, 1)}}; };
    auto scale_of = [&](int i) { return static_cast<int>(static_cast<uint8_t>(scales[(rm + i * 16 + (lane & 15)) * kPitch + b])); };
    if constexpr (EXACT) {
      Wide8 fb[S::FN];
#pragma unroll
      for (int j = 0; j < S::FN; ++j)
        fb[j] = widen8(Frag8{{OpB::fragment(sb, rn + j * 16, 0), OpB::fragment(sb, rn + j * 16, 1)}});
#pragma unroll
      for (int i = 0; i < S::FM; ++i) {
        const Wide8 fa = widen8(a_of(i));
        const int s = scale_of(i);
#pragma unroll
        for (int j = 0; j < S::FN; ++j) acc[i][j] = mfma_wide(fb[j], fa, acc[i][j], colscale, s);
      }
    } else {
      Frag8 fa[S::FM], fb[S::FN];
      int s[S::FM];
#pragma unroll
      for (int j = 0; j < S::FN; ++j) fb[j] = Frag8{{OpB::fragment(sb, rn + j * 16, 0), OpB::fragment(sb, rn + j * 16, 1)}};
#pragma unroll
      for (int i = 0; i < S::FM; ++i) {
        fa[i] = a_of(i);
        s[i] = scale_of(i);
      }
#pragma unroll
      for (int i = 0; i < S::FM; ++i)
#pragma unroll
        for (int j = 0; j < S::FN; ++j) acc[i][j] = mfma8(fb[j], fa[i], acc[i][j], colscale, s[i]);
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < S::FM; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) acc[i][j] = fx4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void init(const uint8_t *a, const uint8_t *b, int64_t lda, int64_t ldb, int validm, int validn,
                                       int length) {
    k = length;
    at = 0;
    per = (k + kStep - 1) / kStep;
    oa.init(a, lda, validm);
    ob.init(b, ldb, validn);
  }
  __device__ __forceinline__ void run(char *lds, const Scales &sa, const Scales &sb) {
    clear();
    if constexpr (ALIGNED) direct(lds, per, sa, sb);
    else through_registers(lds, per, sa, sb);
  }

  __device__ __forceinline__ void direct(char *lds, int steps, const Scales &sa, const Scales &sb) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rm = wave / S::WN * (S::BM / S::WM), rn = wave % S::WN * (S::BN / S::WN);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    char *scales = lds + kStages * kStage;
    constexpr int kAhead = kStages - 1;  // stages in flight when a step begins
    constexpr int kLoads = OpA::kPer + OpB::kPer;
    for (int i = 0; i < kAhead && i < steps; ++i) load(lds0 + i * kStage);
    Chunk::move(scales, sa, sb, 0);
    int buf = 0, to = kAhead;  // stage read, stage loaded
    for (int t = 0; t < steps; ++t) {
      if (kAhead > 1 && t + kAhead <= steps) {  // all but the newest kAhead - 1 stages have landed
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kAhead - 1) * kLoads) : "memory");
      } else {
        loads_done_and_meet();
      }
      if (t + kAhead < steps) load(lds0 + to * kStage);
      if (t > 0 && t % kChunk == 0) {
        Chunk::move(scales, sa, sb, t);
        __syncthreads();
      }
      multiply(lds + buf * kStage, scales, t % kChunk, rm, rn);
      buf = buf + 1 == kStages ? 0 : buf + 1;
      to = to + 1 == kStages ? 0 : to + 1;
    }
    __syncthreads();
  }

  // Operands that are not aligned: as TileProduct's.
  __device__ __forceinline__ void through_registers(char *lds, int steps, const Scales &sa, const Scales &sb) {
    constexpr int kSets = OpA::kSets < OpB::kSets ? OpA::kSets : OpB::kSets;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rm = wave / S::WN * (S::BM / S::WM), rn = wave % S::WN * (S::BN / S::WN);
    char *scales = lds + kStages * kStage;
#pragma unroll
    for (int i = 0; i < kSets; ++i)
      if (i < steps) fetch(i);
    Chunk::move(scales, sa, sb, 0);
    land(0, lds);
    auto step = [&](int t, auto set) {
      constexpr int cur = decltype(set)::value, nxt = (cur + 1) % kSets;
      __syncthreads();
      if (t > 0 && t % kChunk == 0) {
        Chunk::move(scales, sa, sb, t);
        __syncthreads();
      }
      if (t + kSets < steps) fetch(cur);
      multiply(lds + (t & 1) * kStage, scales, t % kChunk, rm, rn);
      if (t + 1 < steps) land(nxt, lds + (t + 1 & 1) * kStage);
    };
    for (int t = 0; t < steps; t += kSets) {
      step(t, std::integral_constant<int, 0>{});
      if constexpr (kSets == 3) {
        if (t + 1 < steps) step(t + 1, std::integral_constant<int, 1>{});
        if (t + 2 < steps) step(t + 2, std::integral_constant<int, 2>{});
      }
    }
    __syncthreads();
  }
};

__device__ __forceinline__ int64_t blocks_of(int64_t n) { return (n + kQBlock8 - 1) / kQBlock8; }

// The way out of a tile of bf16 results: as TileOut's, but rounded before they
// pass through the LDS, and 16 bytes to a lane.  16-byte chunk c of row r is
// kept at c ^ (r & 15) (fewer where a row has fewer): 16 rows' writes of one
// column lie in different banks.
template <class S, int LDS>
struct TileOut16 {
  static constexpr int kRowBytes = S::BN * 2, kChunks = kRowBytes / 16, kMask = kChunks < 16 ? kChunks - 1 : 15;
  static constexpr int fit(int ip) { return ip * 16 * S::WM * kRowBytes <= LDS ? ip : fit(ip / 2); }
  static constexpr int IP = fit(S::FM), kPasses = S::FM / IP, kRows = IP * 16 * S::WM;

  // f(m, n, v): v holds C[m][n .. n + 7] of the tile.
  template <class F>
  static __device__ __forceinline__ void all(char *lds, const fx4 (&acc)[S::FM][S::FN], F f) {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // (see TileOut)
    const int wave = tid >> 6, lane = tid & 63;
    const int row0 = wave / S::WN * (IP * 16) + (lane & 15), col0 = wave % S::WN * (S::BN / S::WN) * 2 + (lane >> 4) * 8;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      if (pass > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < IP; ++i)
#pragma unroll
        for (int j = 0; j < S::FN; ++j) {
          const fx4 v = acc[pass * IP + i][j];
          const int row = row0 + i * 16, col = col0 + j * 32;
          *reinterpret_cast<ux2 *>(lds + row * kRowBytes + (((col >> 4) ^ (row & kMask)) << 4) + (col & 8)) =
              ux2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        }
      __syncthreads();
      constexpr int kAll = kRows * kChunks;
      static_assert(kAll % S::kThreads == 0, "whole rounds");
#pragma unroll 4
      for (int r = 0; r < kAll / S::kThreads; ++r) {
        const int c = r * S::kThreads + tid, row = c / kChunks, chunk = c % kChunks;
        const ux4 v = *reinterpret_cast<const ux4 *>(lds + row * kRowBytes + ((chunk ^ (row & kMask)) << 4));
        f(row / (IP * 16) * (S::BM / S::WM) + pass * IP * 16 + row % (IP * 16), chunk * 8, v);
      }
    }
    __syncthreads();
  }
};

// Stores v to out[0 .. n) (n in 1 .. 8).
__device__ __forceinline__ void store8_bf16(uint16_t *out, const ux4 &v, int n) {
  Raw8<true> r;
  r.v[0] = v;
  store8<true>(out, 0, r, n);
}

// A tile's operands and scales.
template <class S, bool GRAD>
struct QTile {
  RowTile t;
  int64_t n0;
  int validn, k;
  const uint8_t *x, *w;
  Scales sa, sb;

  __device__ __forceinline__ QTile(const QExpertArgs &a, const RowTile &tile) : t(tile) {
    const int64_t n = GRAD ? a.in : a.outf, in_blocks = blocks_of(a.in);
    n0 = static_cast<int64_t>(t.tile_n) * S::BN;
    k = static_cast<int>(GRAD ? a.outf : a.in);
    validn = static_cast<int>(min(static_cast<int64_t>(S::BN), n - n0));
    x = a.x + t.row * a.xs;
    w = a.w + table_entry(a.offsets + t.e) + (GRAD ? n0 : n0 * a.in);
    const int64_t first = n0 / kQBlock8;  // block of columns
    const uint8_t *ws = a.w_scales + t.e * (blocks_of(a.outf) * in_blocks) + (GRAD ? first : first * in_blocks);
    const int kb = static_cast<int>(blocks_of(k));
    sa = Scales{a.x_scales + t.row * a.xss, a.xss, 1, t.rows, kb};
    sb = Scales{ws, GRAD ? 1 : in_blocks, GRAD ? in_blocks : 1, static_cast<int>(blocks_of(n) - first), kb};
  }
  template <class P, bool BF, int LDS>
  __device__ __forceinline__ void store(const QExpertArgs &a, const P &p, char *lds) const {
    if constexpr (BF) {
      TileOut16<S, LDS>::all(lds, p.acc, [&](int m, int c, const ux4 &v) {
        if (m < t.rows && c < validn) store8_bf16(static_cast<uint16_t *>(a.out) + (t.row + m) * a.outs + n0 + c, v, validn - c);
      });
    } else {
      using Out = TileOut<S, LDS>;
      Out::all(lds, p.acc, [&](int pass, int tid) {
        Out::rows(lds, pass, tid, [&](int m, int c, fx4 v) {
          if (m < t.rows && c < validn) store4<false>(a.out, (t.row + m) * a.outs + n0 + c, v, validn - c);
        });
      });
    }
  }
};

__device__ __forceinline__ int column_tiles(int64_t n, int bn) { return static_cast<int>((n + bn - 1) / bn); }

// Forward (GRAD false: W_e as [n][k]) and input gradient (GRAD true: as [k][n]).
template <class P, bool GRAD, bool BF>
__global__ __launch_bounds__(P::Sh::kThreads) void qexperts_rows(QExpertArgs a) {
  using S = typename P::Sh;
  extern __shared__ __align__(16) char lds[];
  RowTile t;
  if (!find_row_tile<S::BM>(a, column_tiles(GRAD ? a.in : a.outf, S::BN), t)) return;
  const QTile<S, GRAD> q(a, t);
  P p;
  p.init(q.x, q.w, a.xs, a.in, q.t.rows, q.validn, q.k);
  p.run(lds, q.sa, q.sb);
  q.template store<P, BF, P::kLds>(a, p, lds);
}

using Big = Shape<256, 256, 2, 2>;

// Tiles of 256 x 256 for long products (aligned, 16-bit results).  The LDS holds
// two stages; fragments are read half a stage ahead of their instructions, and
// between a stage's halves the workgroup meets: the next stage has landed, and
// this one's LDS is free for the loads of the next but one.
//
// Bound by the matrix units: 16384 rows, 8 experts, 4096 x 12288 take 750 us (2.2
// PFLOP/s; 58% of the cycles in matrix instructions at the 1.97 GHz that power
// leaves).  Four waves, one to a SIMD, of 128 x 128 and 512 registers: 8 of 128 x
// 64 take 5% more, and TileProduct8's loop on this tile 836.  Instructions of
// 32x32x64: alone on its SIMD a wave issues them at 4.05 PFLOP/s, 16x16x128 at 3.7.
template <bool GRAD>
struct Long8 {
  static constexpr int kThreads = Big::kThreads, kStep = 128;
  static constexpr int NJ = Big::BN / Big::WN / 32, kSlots = 2 * NJ;
  using OpA = Operand<kF8, kMajorK, Big::BM, kThreads, true>;
  using OpB = Operand<kF8, GRAD ? kMajorMN : kMajorK, Big::BN, kThreads, true>;
  using Chunk = ScaleChunk<Big::BM, Big::BN, kThreads>;
  static constexpr int kStage = OpA::kBytes + OpB::kBytes;
  static constexpr int kLds = 2 * kStage + 2 * Chunk::kBytes + 4 * kThreads;
  typedef float fx16 __attribute__((ext_vector_type(16)));

  fx16 acc[4][NJ];
  Frag8 fa[2][2][2], fb[NJ][2];  // [rows 64 s ..][32 rows][half], [32 columns][half]
  int sa[2][2], sb;
  OpA oa;
  OpB ob;
  Chunk chunk;
  char *lds;
  uint32_t lds0;
  int rm, rn;  // the wave's first row and column

  // What the L2 is told to fetch one stage before the LDS is: one 128-byte line
  // to a lane, by loads of 4 bytes to a place in the LDS that nobody reads (16384 x
  // 4096 x 12288 in even rows: 729 us without, 680 with; two stages ahead more).  The tiles that an XCD
  // works on at once are mostly 8 row tiles by 4 column tiles, so a workgroup
  // asks for a quarter of its rows' lines and an eighth of its columns'.
  const uint8_t *soon_a, *soon_b;
  int64_t by_stage;          // bytes from a stage's columns to the next one's
  uint32_t line_a, line_b;   // bytes from there; kOutOfRange: nothing
  uint32_t unread;           // LDS, 256 bytes to a wave

  __device__ __forceinline__ void aim_ahead(const QTile<Big, GRAD> &q, int64_t lda, int64_t ldb, int last) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int kWaves = kThreads / 64, kA = 64 / kWaves, kB = 32 / kWaves;
    const int row = (wave * kA + lane) * 4 + (q.t.tile_n & 3), line = (wave * kB + lane) * 8 + (q.t.tile_m & 7);
    soon_a = q.x;
    soon_b = q.w;
    by_stage = GRAD ? kStep * ldb : kStep;
    line_a = lane < kA ? static_cast<uint32_t>(min(row, q.t.rows - 1)) * static_cast<uint32_t>(lda) : kOutOfRange;
    // columns: 256 rows of a line, or 128 contraction steps (of the last stage `last`) of two lines
    const uint32_t at = GRAD ? static_cast<uint32_t>(min(line >> 1, last - 1)) * static_cast<uint32_t>(ldb) +
                                   min((line & 1) * 128, (q.validn - 1) & ~15)
                             : static_cast<uint32_t>(min(line, q.validn - 1)) * static_cast<uint32_t>(ldb);
    line_b = lane < kB ? at : kOutOfRange;
    unread = lds0 + 2 * kStage + 2 * Chunk::kBytes + uniform(static_cast<int32_t>(wave)) * 256;
  }
  __device__ __forceinline__ void touch(const uint8_t *base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(unread), "v"(off),
                 "s"(resource(base))
                 : "memory", "m0");
  }

  // The 32 bytes of half h of the stage (contraction elements 64 h + 32 (lane / 32) ..) of row/column r + lane % 32.
  static __device__ __forceinline__ Frag8 rows32(const char *stage, int r, int h) {
    const int lane = threadIdx.x & 63, row = r + (lane & 31), c = h * 4 + (lane >> 5) * 2;
    Frag8 f;
#pragma unroll
    for (int i = 0; i < 2; ++i) f.v[i] = *reinterpret_cast<const ux4 *>(stage + row * 128 + (((c + i) ^ k_swizzle<kF8, 256>(row)) << 4));
    return f;
  }
  static __device__ __forceinline__ Frag8 columns32(const char *stage, int r, int h) {
    const int lane = threadIdx.x & 63;
    Frag8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 8 contraction elements each: a block of 8 x 16 bytes per 16 lanes
      const int k = h * 64 + (lane >> 5) * 32 + 8 * i + ((lane & 15) >> 1);
      const char *p = stage + k * Big::BN + ((((r >> 4) + ((lane >> 4) & 1)) ^ mn_swizzle8<Big::BN>(k)) << 4) + (lane & 1) * 8;
      const ux2 v = __builtin_bit_cast(
          ux2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) ix2 *)const_cast<char *>(p)));
      f.v[i >> 1][2 * (i & 1)] = v[0];
      f.v[i >> 1][2 * (i & 1) + 1] = v[1];
    }
    return f;
  }
  __device__ __forceinline__ void read_a(int set, int i, int h, const char *stage) {
    fa[set][i][h] = rows32(stage, rm + set * 64 + i * 32, h);
  }
  __device__ __forceinline__ void read_b(int j, int h, const char *stage) {
    const char *p = stage + OpA::kBytes;
    fb[j][h] = GRAD ? columns32(p, rn + j * 32, h) : rows32(p, rn + j * 32, h);
  }
  __device__ __forceinline__ const uint8_t *scales(int at) const {  // at: chunk's buffer and block
    return reinterpret_cast<const uint8_t *>(lds) + 2 * kStage + at;
  }
  __device__ __forceinline__ void read_row_scales(int set, int at) {
#pragma unroll
    for (int i = 0; i < 2; ++i) sa[set][i] = scales(at)[(rm + set * 64 + i * 32 + (threadIdx.x & 31)) * kScalePitch];
  }
  __device__ __forceinline__ int col_scale(int at) const { return scales(at)[(Big::BM + rn / 128) * kScalePitch]; }
  static __device__ __forceinline__ fx16 mfma(const Frag8 &a, const Frag8 &b, fx16 c, int s, int t) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(__builtin_bit_cast(ix8, a), __builtin_bit_cast(ix8, b), c, 0,
                                                           0, 0, s, 0, t);
  }

  // One stage, the one in buffer `buf`; now, next: where its scales and the next stage's are.  The code is free of
  // branches: behind one, the compiler would gather all products of the stage.
  __device__ __forceinline__ void step(int buf, int now, int next, int ahead) {
    const char *mine = lds + buf * kStage, *other = lds + (buf ^ 1) * kStage;
    const uint32_t to = lds0 + buf * kStage;
    read_row_scales(1, now);
    touch(soon_a + static_cast<int64_t>(ahead) * kStep, line_a);
    touch(soon_b + ahead * by_stage, line_b);
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
      const int h = n / NJ, j = n % NJ;
      if (n < 4) read_a(1, n & 1, n >> 1, mine);
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i][j] = mfma(fb[j][h], fa[0][i][h], acc[i][j], sb, sa[0][i]);
      __builtin_amdgcn_sched_barrier(0);  // keeps the reads spread among the products
    }
    // all loads to the LDS have landed: only the two above, the youngest, may be under way
    asm volatile("s_waitcnt vmcnt(2) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const int next_sb = col_scale(next);
    read_row_scales(0, next);
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
      const int h = n / NJ, j = n % NJ;
      static_assert(OpA::kPer == kSlots && OpB::kPer == kSlots, "one load of each operand");
      oa.load_one(n, to);
      ob.load_one(n, to + OpA::kBytes);
      if (n < 4) read_a(0, n & 1, n >> 1, other);
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[2 + i][j] = mfma(fb[j][h], fa[1][i][h], acc[2 + i][j], sb, sa[1][i]);
      read_b(j, h, other);
      __builtin_amdgcn_sched_barrier(0);
    }
    sb = next_sb;
    oa.advance();
    ob.advance();
  }

  __device__ __forceinline__ void run(char *l, const QTile<Big, GRAD> &q, int64_t lda, int64_t ldb) {
    const int wave = uniform(static_cast<int32_t>(threadIdx.x >> 6));
    const int per = (q.k + kStep - 1) / kStep;
    lds = l;
    lds0 = uniform(static_cast<int32_t>(lds_offset(l)));
    rm = wave / Big::WN * (Big::BM / Big::WM);
    rn = wave % Big::WN * (Big::BN / Big::WN);
    oa.init(q.x, lda, q.t.rows);
    ob.init(q.w, ldb, q.validn);
    int left = q.k;  // contraction elements from the stage on that is loaded next
    const auto aim = [&] {  // the last stage may be short; behind it, zeros
      if (left < kStep) {
        oa.cut(max(left, 0));
        ob.cut(max(left, 0));
      }
      left -= kStep;
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      aim();
      oa.load(lds0 + i * kStage);
      ob.load(lds0 + i * kStage + OpA::kBytes);
      oa.advance();
      ob.advance();
    }
    aim_ahead(q, lda, ldb, q.k - (per - 1) * kStep);
    char *chunks = lds + 2 * kStage;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = fx16{};
    Chunk::move(chunks, q.sa, q.sb, 0);
    loads_done_and_meet();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 2; ++i) read_a(0, i, h, lds);
#pragma unroll
      for (int j = 0; j < NJ; ++j) read_b(j, h, lds);
    }
    read_row_scales(0, 0);
    sb = col_scale(0);
    int now = 0, then = Chunk::kBytes;  // the chunks' places
    for (int t = 0; t < per;) {
      if (t + kScaleChunk < per) Chunk::move(chunks + then, q.sa, q.sb, t + kScaleChunk);
      const int end = min(per, t + kScaleChunk), last = end - 1 - t;
      for (int b = 0; t < end; ++t, ++b) {
        aim();
        step(t & 1, now + b, b < last ? now + b + 1 : then, min(t + 3, per - 1));
      }
      const int s = now;
      now = then;
      then = s;
    }
    loads_done_and_meet();
  }

  // A lane has, of each 32 columns, 8 q + 4 (lane / 32) .. + 3 of row lane % 32.  Rounded, they pass through the LDS,
  // all of the tile at once, and leave in whole lines: 16-byte chunk c of row r is kept at c ^ (r & 31).
  __device__ __forceinline__ void store(const QExpertArgs &a, const QTile<Big, GRAD> &q) const {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // (see TileOut)
    const int lane = tid & 63;
    constexpr int kRowBytes = Big::BN * 2, kChunks = kRowBytes / 16;
    static_assert(Big::BM * kRowBytes <= 2 * kStage, "the tile fits");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = rm + i * 32 + (lane & 31);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<ux2 *>(lds + row * kRowBytes + (((rn / 8 + j * 4 + c) ^ (row & 31)) << 4) + (lane >> 5) * 8) =
              ux2{bf16_pair(acc[i][j][4 * c], acc[i][j][4 * c + 1]), bf16_pair(acc[i][j][4 * c + 2], acc[i][j][4 * c + 3])};
    }
    __syncthreads();
    const int chunk = tid % kChunks, c = chunk * 8;
    uint16_t *out = static_cast<uint16_t *>(a.out) + q.t.row * a.outs + q.n0 + c;
    if (c >= q.validn) return;  // (whole vectors: the columns are a multiple of 16)
#pragma unroll 8
    for (int row = tid / kChunks; row < q.t.rows; row += kThreads / kChunks)
      *reinterpret_cast<ux4_at2 *>(out + row * a.outs) =
          *reinterpret_cast<const ux4 *>(lds + row * kRowBytes + ((chunk ^ (row & 31)) << 4));
  }
};

template <bool GRAD>
__global__ __launch_bounds__(Big::kThreads) void qexperts_long(QExpertArgs a) {
  extern __shared__ __align__(16) char lds[];
  RowTile t;
  if (!find_row_tile<Big::BM>(a, column_tiles(GRAD ? a.in : a.outf, Big::BN), t)) return;
  const QTile<Big, GRAD> q(a, t);
  Long8<GRAD> p;
  p.run(lds, q, a.xs, a.in);
  p.store(a, q);
}

// Forward for few rows per expert (decoding): the time is that of reading each
// active expert's weights once.  A workgroup takes 16 columns of one expert and
// up to 32 of its rows; its 8 waves take turns at blocks of the contraction,
// so that the workgroup reads 1 KiB of each of the 16 weight rows at a time,
// straight into the registers that feed the matrix instructions (lane l holds
// 32 bytes of row l % 16), and the waves' sums are added in LDS in a fixed
// order.
constexpr int kFewWaves8 = 8, kFewRows8 = 32, kFewCols8 = 16;

// The lane's 32 codes at p, of which the first n exist.
template <bool WHOLE>
__device__ __forceinline__ Frag8 load_codes(const uint8_t *p, int64_t n) {
  Frag8 f;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    f.v[c] = ux4{0, 0, 0, 0};
    if (WHOLE || n >= (c + 1) * 16) {
      __builtin_memcpy(&f.v[c], p + c * 16, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c * 16 + i < n) f.v[c][i >> 2] |= static_cast<uint32_t>(p[c * 16 + i]) << (8 * (i & 3));
    }
  }
  return f;
}

template <bool EXACT>
__device__ __forceinline__ fx4 add_block(const Frag8 &w, const Frag8 &x, fx4 c, int sw, int sx) {
  if constexpr (EXACT) return mfma_wide(widen8(w), widen8(x), c, sw, sx);
  else return mfma8(w, x, c, sw, sx);
}

template <bool EXACT>
__global__ __launch_bounds__(64 * kFewWaves8) void qexperts_few(QExpertArgs a) {
  __shared__ fx4 part[kFewWaves8][kFewRows8 / 16][64];
  RowTile t;
  if (!find_row_tile<kFewRows8>(a, static_cast<int>((a.outf + kFewCols8 - 1) / kFewCols8), t)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15;
  const int64_t n0 = static_cast<int64_t>(t.tile_n) * kFewCols8, own = (lane >> 4) * 32;
  const int64_t blocks = blocks_of(a.in);
  // rows and columns that do not exist repeat the last one; not stored
  const uint8_t *w = a.w + table_entry(a.offsets + t.e) + min(n0 + r, a.outf - 1) * a.in + own;
  const uint8_t *ws = a.w_scales + (t.e * blocks_of(a.outf) + n0 / kQBlock8) * blocks;
  const int64_t row0 = t.row + min(r, t.rows - 1), row1 = t.row + min(r + 16, t.rows - 1);
  const uint8_t *x0 = a.x + row0 * a.xs + own, *x1 = a.x + row1 * a.xs + own;
  const uint8_t *s0 = a.x_scales + row0 * a.xss, *s1 = a.x_scales + row1 * a.xss;
  const bool two = t.rows > 16;
  fx4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  const int64_t whole = a.in / kQBlock8;
  constexpr int kBatch = 4;  // blocks in flight per wave
  int64_t b = wave;
  auto work = [&](auto n) {
    constexpr int N = decltype(n)::value;
    Frag8 fw[N], f0[N], f1[N];
    int sw[N], sx0[N], sx1[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t at = b + i * kFewWaves8;
      fw[i] = load_codes<true>(w + at * kQBlock8, 0);
      sw[i] = ws[at];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t at = b + i * kFewWaves8;
      f0[i] = load_codes<true>(x0 + at * kQBlock8, 0);
      sx0[i] = s0[at];
    }
    if (two) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t at = b + i * kFewWaves8;
        f1[i] = load_codes<true>(x1 + at * kQBlock8, 0);
        sx1[i] = s1[at];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) acc[0] = add_block<EXACT>(fw[i], f0[i], acc[0], sw[i], sx0[i]);
    if (two) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[1] = add_block<EXACT>(fw[i], f1[i], acc[1], sw[i], sx1[i]);
    }
    b += N * kFewWaves8;
  };
  while (b + (kBatch - 1) * kFewWaves8 < whole) work(std::integral_constant<int, kBatch>{});
  while (b < whole) work(std::integral_constant<int, 1>{});
  if (b == whole && whole < blocks) {  // the block that the rows end in
    const int64_t at = whole * kQBlock8, left = a.in - at - own;
    const Frag8 fw = load_codes<false>(w + at, left);
    acc[0] = add_block<EXACT>(fw, load_codes<false>(x0 + at, left), acc[0], ws[whole], s0[whole]);
    if (two) acc[1] = add_block<EXACT>(fw, load_codes<false>(x1 + at, left), acc[1], ws[whole], s1[whole]);
  }
  part[wave][0][lane] = acc[0];
  part[wave][1][lane] = acc[1];
  __syncthreads();
  if (wave > 1) return;
  fx4 v = part[0][wave][lane];
#pragma unroll
  for (int i = 1; i < kFewWaves8; ++i) {
    const fx4 u = part[i][wave][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += u[e];
  }
  const int m = wave * 16 + r, left = static_cast<int>(min(static_cast<int64_t>(4), a.outf - n0 - (lane >> 4) * 4));
  if (m < t.rows && left > 0) store4<!EXACT>(a.out, (t.row + m) * a.outs + n0 + (lane >> 4) * 4, v, left);
}

// A workgroup takes one 128 x 128 block at a time: 16 lanes to a row, 16 rows
// to a pass, all of it in registers between its maximum and its codes.  Bound by
// memory: 64 fp32 matrices of 1408 x 2048 take 160 us, 5.8 TB/s (ordinary stores of
// the codes 170; 8 bf16 ones of 2048 x 2048 16.3 / 21.6, with non-temporal loads too 19.9).
constexpr int kQuantThreads8 = 256, kPasses8 = kQBlock8 / (kQuantThreads8 / 16);
template <bool BF>
__global__ __launch_bounds__(kQuantThreads8) void quantize_weights(QWeightArgs a) {
  __shared__ uint32_t tops[2][kQuantThreads8 / 64];
  const int64_t ib = blocks_of(a.in), per = ib * blocks_of(a.outf), total = per * a.experts;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = (threadIdx.x & 15) * kLane, r0 = threadIdx.x >> 4;
  int parity = 0;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x, parity ^= 1) {
    const int64_t e = id / per, bo = (id - e * per) / ib, bi = id - e * per - bo * ib;
    const int64_t start = table_entry(a.offsets + e) + bo * kQBlock8 * a.in + bi * kQBlock8 + c;
    const int n = static_cast<int>(min(static_cast<int64_t>(kQBlock8), a.in - bi * kQBlock8)) - c;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kQBlock8), a.outf - bo * kQBlock8));
    Raw8<BF> x[kPasses8];
#pragma unroll
    for (int p = 0; p < kPasses8; ++p) {
      const int r = p * (kQuantThreads8 / 16) + r0;
      x[p] = load8<BF>(a.w, start + r * a.in, r < rows ? n : 0);
    }
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < kPasses8; ++p) {
      float v[kLane];
#pragma unroll
      for (int i = 0; i < kLane; ++i) v[i] = x[p][i];
      top = max(top, top_of(v));
    }
    top = row16_max(top);
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
    if (lane == 0) tops[parity][wave] = top;
    __syncthreads();  // (two blocks in a row use different slots)
#pragma unroll
    for (int i = 0; i < kQuantThreads8 / 64; ++i) top = max(top, tops[parity][i]);
    const uint32_t byte = scale_byte(top);
    if (threadIdx.x == 0) a.scales[id] = static_cast<uint8_t>(byte);
#pragma unroll
    for (int p = 0; p < kPasses8; ++p) {
      const int r = p * (kQuantThreads8 / 16) + r0;
      float v[kLane];
#pragma unroll
      for (int i = 0; i < kLane; ++i) v[i] = x[p][i];
      if (r < rows && n > 0) store_codes<true>(a.codes + start + r * a.in, codes8(v, byte), n);
    }
  }
}

// Tiles.  Big (aligned, 16-bit results) is qexperts_long's.
using Square = Shape<128, 128, 2, 2>;
using Half = Shape<64, 128, 2, 2>;
using Small = Shape<32, 64, 1, 4, 4>;

template <class S, bool GRAD>
int64_t row_tiles(const QExpertArgs &a) {
  const int64_t n = GRAD ? a.in : a.outf;
  return (a.tokens / S::BM + std::min<int64_t>(a.experts, a.tokens)) * ((n + S::BN - 1) / S::BN);
}

template <bool EXACT, class S, bool GRAD, bool ALIGNED>
hipError_t launch_rows(const QExpertArgs &a, hipStream_t s) {
  using P = TileProduct8<EXACT, S, GRAD ? kMajorMN : kMajorK, ALIGNED>;
  return launch(qexperts_rows<P, GRAD, !EXACT>, row_tiles<S, GRAD>(a), 1, S::kThreads, P::kLds, s, a);
}

template <class S, bool GRAD>
hipError_t launch_rows(const QExpertArgs &a, hipStream_t s) {
  if (a.bf16) return a.aligned ? launch_rows<false, S, GRAD, true>(a, s) : launch_rows<false, S, GRAD, false>(a, s);
  if constexpr (S::BM < 128) {  // fp32 results take the smaller tiles
    return a.aligned ? launch_rows<true, S, GRAD, true>(a, s) : launch_rows<true, S, GRAD, false>(a, s);
  } else {
    return hipErrorInvalidValue;  // not chosen
  }
}

// Which tile: the least of modelled times.  A tile's time is that of its blocks
// of the contraction and a rest; `slots` tiles run at once, one workgroup on a
// CU or several, whose rounds overlap.  `alone`: launches of up to 256 tiles.
// The model against measured times, bf16 results, rows spread over the experts
// as a router does (rows, experts, in x out: Big / Square / Half / Small,
// microseconds):
//   16384, 8, 4096 x 12288:  723 / 983 / 1172 / 2111   measured 833 / 945 / 1132 / 2258
//   16384, 4, 2048 x 2048:   104 / 100 / 115 / 217               94 / 85 / 91 / 202
//   8192, 32, 2048 x 2048:    70 / 66 / 68 / 117                 70 / 66 / 76 / 122
//   2048, 8, 4096 x 4096:     59 / 68 / 71 / 101                 65 / 77 / 76 / 111
//   4096, 8, 1024 x 1024:     25 / 14 / 14 / 22                  20 / 14 / 13 / 20
//   300, 2, 3968 x 3968:      57 / 34 / 27 / 21                  44 / 27 / 21 / 18
// (28 such calls of both products take 2% more than with the best tile for
// each.)  fp32 results (Square only lost, 920 and 37 in these):
//   16384, 8, 4096 x 4096:      - / - / 831 / 1173   measured 807 / 1131
//   3001, 8, 1024 x 1536:       - / - / 27 / 34                26 / 30
struct TileCost {
  double slots, alone, full, rest;
};
constexpr TileCost kBF16Cost[4] = {{256, 1.4, 1.3, 14}, {512, 0.95, 1.06, 5}, {768, 0.75, 1.0, 3.5}, {768, 0.36, 0.4, 3.5}};
constexpr TileCost kF32Cost[4] = {{}, {}, {768, 2.1, 2.1, 4}, {768, 0.6, 0.71, 3.5}};

template <class S, bool GRAD>
double rows_time(const QExpertArgs &a, const TileCost &c) {
  const double n = static_cast<double>(GRAD ? a.in : a.outf), steps = static_cast<double>(GRAD ? a.outf : a.in) / 128;
  const double e = static_cast<double>(std::min<int64_t>(a.experts, a.tokens)), t = static_cast<double>(a.tokens);
  // one of several experts ends inside a tile, half of it unused on average
  const double tiles = (e > 1 ? std::max(e, t / S::BM + e / 2) : std::ceil(t / S::BM)) * std::ceil(n / S::BN);
  const double rounds = tiles / c.slots;
  return (c.slots <= 256 ? std::ceil(rounds) : std::max(1.0, rounds + 0.5)) *
         (std::ceil(steps) * (tiles <= 256 ? c.alone : c.full) + c.rest);
}

enum Choice { kBig, kSquare, kHalf, kSmall, kFew };

template <bool GRAD>
Choice rows_choice(const QExpertArgs &a) {
  if constexpr (!GRAD) {
    // Short decoding calls, where latency counts: up to 512 workgroups of
    // qexperts_few, two to a CU.  Microseconds with it / Small, weights from
    // memory (rows, active of experts, in x out):
    //   2, 2 of 8, 1024 x 512         7.4 /  7.1
    //   1, 1 of 1, 4096 x 4096        7.3 / 13.4
    //   4, 4 of 8, 2048 x 1024        6.9 /  8.5
    //   2, 2 of 8, 4096 x 4096       11.0 / 13.9
    //   16, 8 of 8, 2048 x 1024       8.4 /  8.6
    //   8, 8 of 8, 2048 x 2048       14.5 /  9.6
    //   1, 1 of 1, 4096 x 12288      15.6 / 14.2
    //   32, 20 of 32, 4096 x 1536    43.9 / 30.4
    const int64_t e = a.experts;
    if (a.tokens <= 16 * e && std::min(e, a.tokens) * ((a.outf + kFewCols8 - 1) / kFewCols8) <= 512) return kFew;
  }
  const TileCost *c = a.bf16 ? kBF16Cost : kF32Cost;
  const double big = a.aligned && a.bf16 ? rows_time<Big, GRAD>(a, c[0]) : 1e300;
  const double square = a.bf16 ? rows_time<Square, GRAD>(a, c[1]) : 1e300;
  const double half = rows_time<Half, GRAD>(a, c[2]);
  const double small = rows_time<Small, GRAD>(a, c[3]);
  if (big <= std::min({square, half, small})) return kBig;
  if (square <= std::min(half, small)) return kSquare;
  return half <= small ? kHalf : kSmall;
}

template <bool GRAD>
hipError_t rows(const QExpertArgs &a, hipStream_t s) {
  switch (rows_choice<GRAD>(a)) {
    case kBig:
      return launch(qexperts_long<GRAD>, row_tiles<Big, GRAD>(a), 1, Big::kThreads, Long8<GRAD>::kLds, s, a);
    case kSquare: return launch_rows<Square, GRAD>(a, s);
    case kHalf: return launch_rows<Half, GRAD>(a, s);
    case kSmall: return launch_rows<Small, GRAD>(a, s);
    case kFew: break;
  }
  if constexpr (GRAD) return hipErrorInvalidValue;  // not chosen
  const int64_t grid = (a.tokens / kFewRows8 + std::min<int64_t>(a.experts, a.tokens)) * ((a.outf + kFewCols8 - 1) / kFewCols8);
  return a.bf16 ? launch(qexperts_few<false>, grid, 1, 64 * kFewWaves8, 0, s, a)
                : launch(qexperts_few<true>, grid, 1, 64 * kFewWaves8, 0, s, a);
}

}  // namespace

hipError_t qexperts_forward(const QExpertArgs &a, hipStream_t s) { return rows<false>(a, s); }
hipError_t qexperts_input_grad(const QExpertArgs &a, hipStream_t s) { return rows<true>(a, s); }

ExpertShape qexperts_shape(const QExpertArgs &a, ExpertProduct product) {
  switch (product == kExpertsForward ? rows_choice<false>(a) : rows_choice<true>(a)) {
    case kBig: return {Big::BM, Big::BN, 1};
    case kSquare: return {Square::BM, Square::BN, 1};
    case kHalf: return {Half::BM, Half::BN, 1};
    case kSmall: return {Small::BM, Small::BN, 1};
    case kFew: break;
  }
  return {kFewRows8, kFewCols8, 1};
}

hipError_t qexperts_quantize(const QWeightArgs &a, hipStream_t s) {
  const int64_t blocks = ((a.in + kQBlock8 - 1) / kQBlock8) * ((a.outf + kQBlock8 - 1) / kQBlock8) * a.experts;
  const int64_t grid = std::min<int64_t>(blocks, 1 << 22);
  return a.bf16 ? launch(quantize_weights<true>, grid, 1, kQuantThreads8, 0, s, a)
                : launch(quantize_weights<false>, grid, 1, kQuantThreads8, 0, s, a);
}

}  // namespace ar_dev

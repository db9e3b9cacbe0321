// tiles.hpp -- the matrix-product tile that the expert products and the
// Newton-Schulz products share (gfx950, device code).
//
// One workgroup computes a BM x BN tile of C = A B over a contraction of
// length k, both operands 16-bit floats (bf16 or fp16), sums in fp32.  Each
// operand lies in memory in one of two orders:
//   kMajorK   row r of the tile is contiguous along the contraction
//             (A[r][k]; for B: B given as its transpose, [n][k])
//   kMajorMN  step k of the contraction is contiguous along the tile
//             (A given as [k][m]; B as [k][n])
// and is staged in LDS in that order, kStepK = 64 contraction elements at a
// time, in two stages: the loads of one stage are in flight while the matrix
// instructions read the other.  MFMA wants 8 consecutive contraction elements
// of one row in each lane: a kMajorK tile gives them with one 16-byte LDS
// read, a kMajorMN tile with two transposing reads (ds_read_b64_tr_b16, which
// hands each lane of a group of 16 one column of a 4 x 16 block).
//
// LDS banks.  A kMajorK row holds 128 bytes, so 16 lanes that read the same
// 16-byte column of 16 rows would meet in 4 banks: column c of row r is kept
// at c ^ (r & 7).  A kMajorMN row holds 2 BN bytes and half a wave reads one
// 32-byte block of 8 rows (k, k+1, k+2, k+3 and the same plus 8): block b of
// row k is kept at b ^ mn_swizzle(k), which takes 8 values over these rows.
//
// Aligned operands (16-byte rows and starts) go from memory to LDS without
// passing through registers (buffer_load ... lds: lane l of the wave writes
// the 16 bytes at its base + 16 l, so the swizzle is applied to the address
// that the lane reads); others are loaded into registers, masked element by
// element at the ends of a row, and written to LDS from there.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

namespace ar_dev {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float fx4 __attribute__((ext_vector_type(4)));
typedef uint32_t ux4 __attribute__((ext_vector_type(4)));
typedef uint32_t ux2 __attribute__((ext_vector_type(2)));

enum Elem16 { kBF16, kF16 };
enum Major { kMajorK, kMajorMN };
constexpr int kStepK = 64;

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)static_cast<const char *>(p)));
}

// 64 lanes x 16 bytes from base + off (per lane) to LDS at lds_base + 16 lane;
// a lane whose off is at or over 2^31 - 1 writes zeros (the buffer's range
// check).  Asynchronous: loads_done() waits.  In asm because the compiler
// would wait for every such load before each transposing LDS read; the
// instruction has no output register.  s_nop 4: the wait states that a
// scalar register written by the vector unit needs before a buffer load.
constexpr uint32_t kOutOfRange = 0x80000000u;
__device__ __forceinline__ void load_to_lds(const void *base, uint32_t off, uint32_t lds_base) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  // a buffer resource in scalar registers: 48-bit base, 2^31 - 1 bytes, 32-bit data format
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32)) & 0xffffu;
  const ux4 r = {lo, hi, 0x7fffffffu, 0x00020000u};
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds_base), "v"(off),
               "s"(r)
               : "memory");
}

// Every load_to_lds of this wave has landed and its LDS reads are done, then
// the workgroup meets.
__device__ __forceinline__ void loads_done_and_meet() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int W>  // tile width in elements
__device__ __forceinline__ constexpr int mn_swizzle(int k) {
  return W >= 128 ? ((k & 3) | ((k >> 3) & 1) << 2) : (((k >> 1) & 1) | ((k >> 3) & 1) << 1);
}

// Byte of the 16-byte chunk that holds, in a kMajorK tile, contraction
// elements 8 c .. 8 c + 7 of row r.
__device__ __forceinline__ constexpr int chunk_k(int r, int c) { return r * (kStepK * 2) + ((c ^ (r & 7)) << 4); }

template <Elem16 E>
__device__ __forceinline__ fx4 mfma16(s16x8 a, s16x8 b, fx4 c) {
  if constexpr (E == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// One operand of a tile: W rows (kMajorK) or columns (kMajorMN) of it, loaded
// by NT threads.
//   base    first element of the tile's first row/column at contraction 0
//   ld      elements between rows (kMajorK) or contraction steps (kMajorMN)
//   valid   rows/columns of the tile that exist (>= 1); what lies beyond is
//           loaded from the last one that exists (its products are not stored)
template <Major MJ, int W, int NT, bool ALIGNED>
struct Operand {
  static constexpr int kChunks = W * kStepK / 8;  // 16-byte chunks of a stage
  static constexpr int kPer = kChunks / NT;       // per thread
  static constexpr int kBytes = W * kStepK * 2;
  static_assert(kPer * NT == kChunks, "whole chunks per thread");

  const uint16_t *base;
  int64_t ld;
  int valid;
  uint32_t off[ALIGNED ? kPer : 1];  // bytes from base, contraction step 0
  s16x8 reg[ALIGNED ? 1 : kPer];

  // Chunk j of this thread: its row in LDS, and which 16 bytes of that row
  // in memory land there.
  __device__ __forceinline__ void where(int j, int &row, int &col) const {
    const int c = (threadIdx.x >> 6) * (64 * kPer) + j * 64 + (threadIdx.x & 63);
    if constexpr (MJ == kMajorK) {
      row = c >> 3;
      col = (c & 7) ^ (row & 7);
    } else {
      constexpr int kRow = W / 8;  // chunks of a row
      row = c / kRow;
      const int p = c % kRow;
      col = (((p >> 1) ^ mn_swizzle<W>(row)) << 1) | (p & 1);
    }
  }

  __device__ __forceinline__ void init(const uint16_t *b, int64_t l, int v) {
    base = b;
    ld = l;
    valid = v;
    if constexpr (ALIGNED) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        int row, col;
        where(j, row, col);
        if constexpr (MJ == kMajorK)
          off[j] = static_cast<uint32_t>(min(row, valid - 1)) * static_cast<uint32_t>(ld * 2) + col * 16;
        else
          off[j] = static_cast<uint32_t>(row) * static_cast<uint32_t>(ld * 2) + min(col * 8, (valid - 1) & ~7) * 2;
      }
    }
  }

  __device__ __forceinline__ void advance() { base += MJ == kMajorK ? kStepK : kStepK * ld; }

  // Starts the loads of the stage at `base`, of whose contraction elements
  // the first `left` exist (the rest are zeros).
  __device__ __forceinline__ void load(int left, uint32_t lds) {
    if constexpr (ALIGNED) {
      const uint32_t wave = lds + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (1024 * kPer);
      if (left >= kStepK) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) load_to_lds(base, off[j], wave + j * 1024);
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          int row, col;
          where(j, row, col);
          const bool in = (MJ == kMajorK ? col * 8 : row) < left;
          load_to_lds(base, in ? off[j] : kOutOfRange, wave + j * 1024);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        int row, col;
        where(j, row, col);
        const uint16_t *p;
        int n;  // elements that exist
        if constexpr (MJ == kMajorK) {
          p = base + static_cast<int64_t>(min(row, valid - 1)) * ld + col * 8;
          n = left - col * 8;
        } else {
          p = base + static_cast<int64_t>(row) * ld + col * 8;
          n = row < left ? valid - col * 8 : 0;
        }
        s16x8 v = {};
        if (n >= 8) {
          __builtin_memcpy(&v, p, 16);
        } else if (n > 0) {
#pragma unroll
          for (int i = 0; i < 7; ++i)
            if (i < n) v[i] = static_cast<short>(p[i]);
        }
        reg[j] = v;
      }
    }
  }

  // The register path's second half: what load() read goes to LDS.
  __device__ __forceinline__ void land(char *stage) {
    if constexpr (!ALIGNED) {
      char *w = stage + (threadIdx.x >> 6) * (1024 * kPer) + (threadIdx.x & 63) * 16;
#pragma unroll
      for (int j = 0; j < kPer; ++j) *reinterpret_cast<s16x8 *>(w + j * 1024) = reg[j];
    }
  }

  // The 8 contraction elements 32 ks + 8 (lane / 16) .. of row/column
  // r + lane % 16 of the stage.
  static __device__ __forceinline__ s16x8 fragment(const char *stage, int r, int ks) {
    const int lane = threadIdx.x & 63;
    if constexpr (MJ == kMajorK) {
      return *reinterpret_cast<const s16x8 *>(stage + chunk_k(r + (lane & 15), ks * 4 + (lane >> 4)));
    } else {
      const int k = ks * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2);
      s16x4 h[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const char *p = stage + (k + 4 * i) * (W * 2) + (((r >> 4) ^ mn_swizzle<W>(k + 4 * i)) << 5) + (lane & 3) * 8;
        h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4 *)const_cast<char *>(p));
      }
      return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Tile shape: BM x BN by WM x WN waves, each wave 16-row fragments.
template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments of a wave
};

// The contraction: nseg pairs (A_s, B_s) of length k each, added into one sum
// (a product of numbers held as sums of 16-bit parts is such a list).
// Finishes with all LDS reads done.
template <Elem16 E, class S, Major AM, Major BMJ, bool ALIGNED>
struct TileProduct {
  using Elem = uint16_t;
  using Sh = S;
  using OpA = Operand<AM, S::BM, S::kThreads, ALIGNED>;
  using OpB = Operand<BMJ, S::BN, S::kThreads, ALIGNED>;
  static constexpr int kStage = OpA::kBytes + OpB::kBytes;
  static constexpr int kLds = 2 * kStage;
  fx4 acc[S::FM][S::FN];

  __device__ __forceinline__ void run(char *lds, const uint16_t *const *a, const uint16_t *const *b, int nseg,
                                      int64_t lda, int64_t ldb, int validm, int validn, int64_t k) {
#pragma unroll
    for (int i = 0; i < S::FM; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) acc[i][j] = fx4{0, 0, 0, 0};
    if (k <= 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rm = wave / S::WN * (S::BM / S::WM), rn = wave % S::WN * (S::BN / S::WN);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    OpA oa;
    OpB ob;
    oa.init(a[0], lda, validm);
    ob.init(b[0], ldb, validn);
    const int64_t per = (k + kStepK - 1) / kStepK;
    int seg = 0;
    int64_t at = 0;  // stage of the segment that is loaded next
    auto load = [&](int buf) {
      const int left = static_cast<int>(min(k - at * kStepK, static_cast<int64_t>(kStepK)));
      oa.load(left, lds0 + buf * kStage);
      ob.load(left, lds0 + buf * kStage + OpA::kBytes);
      if (++at < per) {
        oa.advance();
        ob.advance();
      } else if (++seg < nseg) {
        at = 0;
        oa.base = a[seg];
        ob.base = b[seg];
      }
    };
    auto land = [&](int buf) {
      oa.land(lds + buf * kStage);
      ob.land(lds + buf * kStage + OpA::kBytes);
    };
    const int64_t steps = per * nseg;
    load(0);
    land(0);
    for (int64_t t = 0; t < steps; ++t) {
      const int buf = static_cast<int>(t & 1);
      if constexpr (ALIGNED) loads_done_and_meet();
      else __syncthreads();
      if (t + 1 < steps) load(buf ^ 1);
      const char *sa = lds + buf * kStage, *sb = sa + OpA::kBytes;
#pragma unroll
      for (int ks = 0; ks < kStepK / 32; ++ks) {
        s16x8 fa[S::FM], fb[S::FN];
#pragma unroll
        for (int i = 0; i < S::FM; ++i) fa[i] = OpA::fragment(sa, rm + i * 16, ks);
#pragma unroll
        for (int j = 0; j < S::FN; ++j) fb[j] = OpB::fragment(sb, rn + j * 16, ks);
#pragma unroll
        for (int i = 0; i < S::FM; ++i)
#pragma unroll
          for (int j = 0; j < S::FN; ++j) acc[i][j] = mfma16<E>(fb[j], fa[i], acc[i][j]);
      }
      if (t + 1 < steps) land(buf ^ 1);
    }
    __syncthreads();
  }

  __device__ __forceinline__ void run(char *lds, const uint16_t *a, const uint16_t *b, int64_t lda, int64_t ldb,
                                      int validm, int validn, int64_t k) {
    run(lds, &a, &b, 1, lda, ldb, validm, validn, k);
  }

  // f(m, n, v): v holds C[m][n .. n + 3] of the tile.
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int rm = wave / S::WN * (S::BM / S::WM) + (lane & 15), rn = wave % S::WN * (S::BN / S::WN) + (lane >> 4) * 4;
#pragma unroll
    for (int i = 0; i < S::FM; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) f(rm + i * 16, rn + j * 16, acc[i][j]);
  }
};

}  // namespace ar_dev

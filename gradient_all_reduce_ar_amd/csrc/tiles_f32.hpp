// tiles_f32.hpp -- the fp32 counterpart of tiles.hpp's product tile (gfx950).
//
// v_mfma_f32_16x16x4_f32 takes one float per lane and operand, so a tile is
// kept in LDS in the order it has in memory, kStepKF32 = 32 contraction elements
// at a time in two stages, and needs no transposing read.  A matrix
// instruction of 32 cycles per pair of 4-byte LDS reads leaves the LDS far
// from its limit: the tile is bound by the fp32 matrix rate (256 operations
// per cycle and CU).  Rows are padded so that the 64 lanes of one read (16
// rows or columns x 4 contraction elements) fall into 64 different banks.
#pragma once
#include "tiles.hpp"

namespace ar_dev {

constexpr int kStepKF32 = 32;

template <Major MJ, int W, int NT, bool ALIGNED>
struct OperandF32 {
  static constexpr int kRows = MJ == kMajorK ? W : kStepKF32;        // rows of the stage
  static constexpr int kRow = MJ == kMajorK ? kStepKF32 : W;         // floats of a row
  static constexpr int kPitch = MJ == kMajorK ? kRow + 4 : kRow + 16;
  static constexpr int kBytes = kRows * kPitch * 4;
  static constexpr int kPer = kRows * kRow / 4 / NT;
  static_assert(kPer * NT * 4 == kRows * kRow, "whole chunks per thread");

  const float *base;
  int64_t ld;
  int valid;
  fx4 reg[kPer];

  __device__ __forceinline__ void init(const float *b, int64_t l, int v) {
    base = b;
    ld = l;
    valid = v;
  }
  __device__ __forceinline__ void advance() { base += MJ == kMajorK ? kStepKF32 : kStepKF32 * ld; }
  __device__ __forceinline__ void load(int left) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int c = j * NT + threadIdx.x, row = c / (kRow / 4), col = c % (kRow / 4) * 4;
      const float *p;
      int n;
      if constexpr (MJ == kMajorK) {
        p = base + static_cast<int64_t>(min(row, valid - 1)) * ld + col;
        n = left - col;
      } else {
        p = base + static_cast<int64_t>(row) * ld + col;
        n = row < left ? valid - col : 0;
      }
      fx4 v = {};
      if (n >= 4) {
        if constexpr (ALIGNED) v = *reinterpret_cast<const fx4 *>(p);
        else __builtin_memcpy(&v, p, 16);
      } else if (n > 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < n) v[i] = p[i];
      }
      reg[j] = v;
    }
  }
  __device__ __forceinline__ void land(char *stage) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int c = j * NT + threadIdx.x, row = c / (kRow / 4), col = c % (kRow / 4) * 4;
      *reinterpret_cast<fx4 *>(stage + (row * kPitch + col) * 4) = reg[j];
    }
  }
  // contraction element 4 ks + lane / 16 of row/column r + lane % 16
  static __device__ __forceinline__ float fragment(const char *stage, int r, int ks) {
    const int lane = threadIdx.x & 63, i = r + (lane & 15), k = ks * 4 + (lane >> 4);
    return reinterpret_cast<const float *>(stage)[MJ == kMajorK ? i * kPitch + k : k * kPitch + i];
  }
};

template <class S, Major AM, Major BMJ, bool ALIGNED>
struct TileProductF32 {
  using Elem = float;
  using Sh = S;
  using OpA = OperandF32<AM, S::BM, S::kThreads, ALIGNED>;
  using OpB = OperandF32<BMJ, S::BN, S::kThreads, ALIGNED>;
  static constexpr int kStage = OpA::kBytes + OpB::kBytes;
  static constexpr int kLds = 2 * kStage;
  fx4 acc[S::FM][S::FN];

  __device__ __forceinline__ void run(char *lds, const float *a, const float *b, int64_t lda, int64_t ldb, int validm,
                                      int validn, int64_t k) {
#pragma unroll
    for (int i = 0; i < S::FM; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) acc[i][j] = fx4{0, 0, 0, 0};
    if (k <= 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rm = wave / S::WN * (S::BM / S::WM), rn = wave % S::WN * (S::BN / S::WN);
    OpA oa;
    OpB ob;
    oa.init(a, lda, validm);
    ob.init(b, ldb, validn);
    const int64_t steps = (k + kStepKF32 - 1) / kStepKF32;
    auto load = [&](int64_t t) {
      const int left = static_cast<int>(min(k - t * kStepKF32, static_cast<int64_t>(kStepKF32)));
      oa.load(left);
      ob.load(left);
      oa.advance();
      ob.advance();
    };
    auto land = [&](int buf) {
      oa.land(lds + buf * kStage);
      ob.land(lds + buf * kStage + OpA::kBytes);
    };
    load(0);
    land(0);
    for (int64_t t = 0; t < steps; ++t) {
      const int buf = static_cast<int>(t & 1);
      __syncthreads();
      if (t + 1 < steps) load(t + 1);
      const char *sa = lds + buf * kStage, *sb = sa + OpA::kBytes;
#pragma unroll
      for (int ks = 0; ks < kStepKF32 / 4; ++ks) {
        float fa[S::FM], fb[S::FN];
#pragma unroll
        for (int i = 0; i < S::FM; ++i) fa[i] = OpA::fragment(sa, rm + i * 16, ks);
#pragma unroll
        for (int j = 0; j < S::FN; ++j) fb[j] = OpB::fragment(sb, rn + j * 16, ks);
#pragma unroll
        for (int i = 0; i < S::FM; ++i)
#pragma unroll
          for (int j = 0; j < S::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
      if (t + 1 < steps) land(buf ^ 1);
    }
    __syncthreads();
  }
};

}  // namespace ar_dev

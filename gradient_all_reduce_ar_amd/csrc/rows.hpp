// rows.hpp -- eight elements of a row to a lane, and 8-bit blocks of 128
// (gfx950, device code of the RMS norm and of the quantisers).
//
// A lane takes 8 consecutive elements, so a scale block is the 16 lanes of one
// DPP row.  Rows may start at any element's address: the hardware takes such
// 16-byte loads and stores.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "tiles.hpp"

namespace ar_dev {

constexpr int kLane = 8;  // elements of a lane

typedef ux4 ux4_at2 __attribute__((aligned(2)));
typedef ux4 ux4_at4 __attribute__((aligned(4)));
typedef ux2 ux2_at1 __attribute__((aligned(1)));

// 8 elements as they lie in memory.
template <bool BF>
struct Raw8 {
  ux4 v[BF ? 1 : 2];
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (BF) return __uint_as_float(i & 1 ? v[0][i >> 1] & 0xffff0000u : v[0][i >> 1] << 16);
    else return __uint_as_float(v[i >> 2][i & 3]);
  }
};

// p[0 .. n), zeros beyond; n <= 0: nothing is read.
template <bool BF>
__device__ __forceinline__ Raw8<BF> load8(const void *base, int64_t at, int n) {
  Raw8<BF> r = {};
  if constexpr (BF) {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at;
    if (n >= kLane) {
      r.v[0] = *reinterpret_cast<const ux4_at2 *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < kLane - 1; ++i)
        if (i < n) r.v[0][i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    }
  } else {
    const uint32_t *p = static_cast<const uint32_t *>(base) + at;
    if (n >= kLane) {
      r.v[0] = *reinterpret_cast<const ux4_at4 *>(p);
      r.v[1] = *reinterpret_cast<const ux4_at4 *>(p + 4);
    } else {
#pragma unroll
      for (int i = 0; i < kLane - 1; ++i)
        if (i < n) r.v[i >> 2][i & 3] = p[i];
    }
  }
  return r;
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {  // nearest, ties to even
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// Two of them in a word, in one instruction.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float fx2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(fx2{lo, hi}, bf16x2));
}

// v rounded once to the rows' type.
template <bool BF>
__device__ __forceinline__ Raw8<BF> rounded8(const float (&v)[kLane]) {
  Raw8<BF> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      r.v[0][i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    } else {
      r.v[0][i] = __float_as_uint(v[i]);
      r.v[1][i] = __float_as_uint(v[4 + i]);
    }
  }
  return r;
}

// NT: non-temporal (whole pieces of 16 bits).
template <bool BF, bool NT = false>
__device__ __forceinline__ void store8(void *base, int64_t at, const Raw8<BF> &r, int n) {
  if constexpr (BF) {
    uint16_t *p = static_cast<uint16_t *>(base) + at;
    if (n >= kLane) {
      if constexpr (NT) __builtin_nontemporal_store(r.v[0], reinterpret_cast<ux4_at2 *>(p));
      else *reinterpret_cast<ux4_at2 *>(p) = r.v[0];
    } else {
#pragma unroll
      for (int i = 0; i < kLane - 1; ++i)
        if (i < n) p[i] = static_cast<uint16_t>(r.v[0][i >> 1] >> (16 * (i & 1)));
    }
  } else {
    uint32_t *p = static_cast<uint32_t *>(base) + at;
    if (n >= kLane) {
      *reinterpret_cast<ux4_at4 *>(p) = r.v[0];
      *reinterpret_cast<ux4_at4 *>(p + 4) = r.v[1];
    } else {
#pragma unroll
      for (int i = 0; i < kLane - 1; ++i)
        if (i < n) p[i] = r.v[i >> 2][i & 3];
    }
  }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
}
// The largest over the 16 lanes of a DPP row: lanes 1 and 2 apart, then the
// halves mirrored (quads agree by then), then the row.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, dpp<0xb1>(v));
  v = max(v, dpp<0x4e>(v));
  v = max(v, dpp<0x141>(v));
  return max(v, dpp<0x140>(v));
}

// Magnitudes are compared by their bits: infinities and NaN are the largest.
__device__ __forceinline__ uint32_t top_of(const float (&v)[kLane]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kLane; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// The scale's byte for a block whose largest magnitude has the bits `top`:
// top = 1.m 2^(E - 127) is at most 448 2^e = 1.75 2^(8 + e) from e = E - 135
// on, one more if 1.m is over 1.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  const int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}

// e4m3 codes of v 2^(127 - byte): the product is exact (or below what a code
// holds), so each element is rounded once.
__device__ __forceinline__ ux2 codes8(const float (&v)[kLane], uint32_t byte) {
  if (byte == 255) return ux2{0x7f7f7f7fu, 0x7f7f7f7fu};
  const float inv = __uint_as_float((254 - byte) << 23);
  ux2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
    r[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, w, true));
  }
  return r;
}

template <bool NT = false>
__device__ __forceinline__ void store_codes(uint8_t *p, ux2 c, int n) {
  if (n >= kLane) {
    if constexpr (NT) __builtin_nontemporal_store(c, reinterpret_cast<ux2_at1 *>(p));
    else *reinterpret_cast<ux2_at1 *>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < kLane - 1; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(c[i >> 2] >> (8 * (i & 3)));
  }
}

}  // namespace ar_dev

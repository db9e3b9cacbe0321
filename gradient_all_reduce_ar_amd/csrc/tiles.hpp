// tiles.hpp -- the matrix-product tile that the expert products and the
// Newton-Schulz products share (gfx950, device code).
//
// One workgroup computes a BM x BN tile of C = A B over a contraction of
// length k, both operands bf16, fp16 or fp32, sums in fp32 (operands of 8 bits,
// whose products qexperts.hip forms, are staged in the same way: 128 elements
// to a stage, which transposing reads of 8 x 16 bytes take across).  Each operand lies
// in memory in one of two orders:
//   kMajorK   row r of the tile is contiguous along the contraction
//             (A[r][k]; for B: B given as its transpose, [n][k])
//   kMajorMN  step k of the contraction is contiguous along the tile
//             (A given as [k][m]; B as [k][n])
// and is staged in LDS in that order, 128 bytes of contraction elements at a
// time (64 of 16 bits, 32 of fp32), in two or more stages: the loads of a
// stage are in flight while the matrix instructions read another.  A lane
// takes 16 bytes of consecutive contraction elements of one row: 8 of 16 bits
// are one operand of a 16x16x32 matrix instruction, 4 of fp32 those of four
// 16x16x4 (element j of every lane to the j-th: which contraction element
// meets which lane does not matter as long as both operands agree).  A kMajorK
// tile gives them with one 16-byte LDS read; a kMajorMN tile of 16-bit
// elements with two transposing reads (ds_read_b64_tr_b16, which hands each
// lane of a group of 16 one column of a 4 x 16 block), of fp32 with four
// 4-byte reads.
//
// LDS banks.  A kMajorK row holds 128 bytes, so 16 lanes that read the same
// 16-byte column of 16 rows would meet in 4 banks: column c of row r is kept
// at c ^ (r & 7).  A kMajorMN row holds W elements.  16 bits: half a wave
// reads one 32-byte block of 8 rows (k, k+1, k+2, k+3 and the same plus 8);
// block b of row k is kept at b ^ mn_swizzle(k), which takes 8 values over
// these rows.  fp32: half a wave reads 64 bytes of rows k and k + 4, which are
// kept 64 bytes apart (16-byte column c at c ^ (k & 4)).
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
#include <type_traits>

namespace ar_dev {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float fx4 __attribute__((ext_vector_type(4)));
typedef uint32_t ux4 __attribute__((ext_vector_type(4)));
typedef uint32_t ux2 __attribute__((ext_vector_type(2)));
typedef int32_t ix2 __attribute__((ext_vector_type(2)));
typedef int32_t ix8 __attribute__((ext_vector_type(8)));

enum Elem { kBF16, kF16, kF32, kF8 };
enum Major { kMajorK, kMajorMN };
template <Elem E>
using ElemOf = std::conditional_t<E == kF32, float, std::conditional_t<E == kF8, uint8_t, uint16_t>>;
// 16 bytes of contraction elements.
template <Elem E>
using Frag = std::conditional_t<E == kF32, fx4, std::conditional_t<E == kF8, ux4, s16x8>>;
constexpr int kStepK = 64;  // contraction elements of a stage, 16 bits

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)static_cast<const char *>(p)));
}

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(v >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// An entry of a plan's table, which nothing writes while a kernel runs, at a
// uniform address: read with scalar loads, so that what is computed from it
// (a contraction's addresses and loop counts) stays in the scalar unit.  The
// compiler would read it into vector registers, since the kernel stores.
template <class T>
__device__ __forceinline__ T table_entry(const T *p) {
  static_assert(sizeof(T) % 4 == 0, "whole words");
  const auto *w = (const __attribute__((address_space(4))) uint32_t *)reinterpret_cast<uintptr_t>(p);
  uint32_t h[sizeof(T) / 4];
#pragma unroll
  for (size_t i = 0; i < sizeof(T) / 4; ++i) h[i] = w[i];
  T v;
  __builtin_memcpy(&v, h, sizeof(T));
  return v;
}

// A buffer resource at a uniform address: 48-bit base, 2^31 - 1 bytes, 32-bit
// data format.  s_nop 4: the wait states between a scalar register that the
// vector unit wrote and a buffer load, which asm hides from the compiler.
__device__ __forceinline__ ux4 resource(const void *base) {
  const uint64_t b = static_cast<uint64_t>(uniform(static_cast<int64_t>(reinterpret_cast<uintptr_t>(base))));
  ux4 r = {static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32) & 0xffffu, 0x7fffffffu, 0x00020000u};
  asm volatile("s_nop 4" : "+s"(r));
  return r;
}

// 64 lanes x 16 bytes from the resource's base + off (per lane) to LDS at
// lds_base + 16 lane; a lane whose off is at or over 2^31 - 1 writes zeros
// (the buffer's range check).  Asynchronous: loads_done_and_meet() waits.  In
// asm because the compiler would wait for every such load before each
// transposing LDS read; the instruction has no output register.
constexpr uint32_t kOutOfRange = 0x80000000u;
__device__ __forceinline__ void load_to_lds(ux4 r, uint32_t off, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds_base), "v"(off),
               "s"(r)
               : "memory", "m0");
}

// Every load_to_lds of this wave has landed and its LDS reads are done, then
// the workgroup meets.
__device__ __forceinline__ void loads_done_and_meet() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int W>  // tile width in 16-bit elements
__device__ __forceinline__ constexpr int mn_swizzle(int k) {
  return W >= 128 ? ((k & 3) | ((k >> 3) & 1) << 2) : (((k >> 1) & 1) | ((k >> 3) & 1) << 1);
}

// Where a kMajorK row keeps its 16-byte column c: at c ^ k_swizzle(row).  A read
// of 16 bytes takes the wave in quarters, lanes l .. l + 7 with l + 16 .. l + 23:
// these are eight rows of two columns where 16 rows make a fragment, and rows r
// .. r + 7 and r + 16 .. r + 23 of one column where 32 do (of 8 bits, 256 rows:
// half of the LDS's cycles were conflicts with r & 7).
template <Elem E, int W>
__device__ __forceinline__ constexpr int k_swizzle(int row) {
  return E == kF8 && W >= 256 ? (row & 6) | ((row >> 4) & 1) : row & 7;
}

// mn_swizzle for bytes, in 16-byte columns.  Half a wave reads one column of rows
// k .. k + 7 and k + 16 .. k + 23 (rows of 64 and 128 bytes go round the banks
// faster, so fewer columns have to differ), or, of 256 columns, two
// neighbouring columns of rows k .. k + 7.
template <int W>
__device__ __forceinline__ constexpr int mn_swizzle8(int k) {
  const int far = (k >> 4) & 1;
  return W >= 256 ? (k & 7) << 1 : W >= 128 ? (((k >> 1) & 3) | far << 2) : (((k >> 2) & 1) | far << 1);
}

template <Elem E>
__device__ __forceinline__ fx4 mfma16(Frag<E> a, Frag<E> b, fx4 c) {
  if constexpr (E == kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  } else if constexpr (E == kF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
}

// One operand of a tile: W rows (kMajorK) or columns (kMajorMN) of it, loaded
// by NT threads.
//   base    first element of the tile's first row/column at contraction 0
//   ld      elements between rows (kMajorK) or contraction steps (kMajorMN)
//   valid   rows/columns of the tile that exist (>= 1); what lies beyond is
//           loaded from the last one that exists (its products are not stored)
template <Elem E, Major MJ, int W, int NT, bool ALIGNED>
struct Operand {
  using T = ElemOf<E>;
  static constexpr int ES = sizeof(T), kVec = 16 / ES, kStep = 128 / ES;
  static constexpr int kChunks = W * 8;      // 16-byte chunks of a stage
  static constexpr int kPer = kChunks / NT;  // per thread
  static constexpr int kBytes = W * 128;
  static constexpr int kRow = W * ES / 16;   // chunks of a kMajorMN row
  static_assert(kPer * NT == kChunks, "whole chunks per thread");
  // Unaligned: stages on their way in registers.  Three for small tiles (64 rows,
  // 8 experts, 2047 -> 1023: 24 us, with one 28), one for those whose workgroups
  // share a CU (weight gradients of 8192 rows, 8 experts, 2047 x 2047: 207 us,
  // with three 229).
  static constexpr int kSets = ALIGNED ? 0 : kPer <= 2 ? 3 : 1;

  const T *base;
  int64_t ld;
  int valid;
  uint32_t off[ALIGNED ? kPer : 1];  // bytes from base, contraction step 0
  ux4 res;                           // resource at base
  uint32_t mine;                     // LDS bytes of a stage before this wave's
  ux4 reg[ALIGNED ? 1 : 3][ALIGNED ? 1 : kPer];

  __device__ __forceinline__ void point(const T *b) {
    base = b;
    if constexpr (ALIGNED) res = resource(base);
  }

  // Chunk j of this thread: its row in LDS, and which 16 bytes of that row
  // in memory land there.
  __device__ __forceinline__ void where(int j, int &row, int &col) const {
    const int c = ALIGNED ? (threadIdx.x >> 6) * (64 * kPer) + j * 64 + (threadIdx.x & 63) : j * NT + threadIdx.x;
    if constexpr (MJ == kMajorK) {
      row = c >> 3;
      col = (c & 7) ^ k_swizzle<E, W>(row);
    } else {
      row = c / kRow;
      const int p = c % kRow;
      if constexpr (E == kF32) col = p ^ (row & 4);
      else if constexpr (E == kF8) col = p ^ mn_swizzle8<W>(row);
      else col = (((p >> 1) ^ mn_swizzle<W>(row)) << 1) | (p & 1);
    }
  }

  __device__ __forceinline__ void init(const T *b, int64_t l, int v) {
    point(b);
    ld = l;
    valid = v;
    mine = uniform(static_cast<int32_t>(threadIdx.x >> 6)) * (1024 * kPer);
    if constexpr (ALIGNED) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        int row, col;
        where(j, row, col);
        if constexpr (MJ == kMajorK)
          off[j] = static_cast<uint32_t>(min(row, valid - 1)) * static_cast<uint32_t>(ld * ES) + col * 16;
        else
          off[j] = static_cast<uint32_t>(row) * static_cast<uint32_t>(ld * ES) +
                   min(col * kVec, (valid - 1) & ~(kVec - 1)) * ES;
      }
    }
  }

  __device__ __forceinline__ void advance() { point(base + (MJ == kMajorK ? kStep : kStep * ld)); }

  // For the last stage, of whose contraction elements the first `left` exist:
  // the loads of the others give zeros.
  __device__ __forceinline__ void cut(int left) {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        int row, col;
        where(j, row, col);
        if ((MJ == kMajorK ? col * kVec : row) >= left) off[j] = kOutOfRange;
      }
    }
  }

  // Aligned: starts load j of the stage at `base`.
  __device__ __forceinline__ void load_one(int j, uint32_t lds) {
    load_to_lds(res, off[j], lds + mine + j * 1024);
  }
  __device__ __forceinline__ void load(uint32_t lds) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) load_one(j, lds);
  }

  // Unaligned: starts the loads of the stage at `base`, from where on `rest`
  // contraction elements exist, into register set `set`; land() takes them to
  // the LDS.  What lies beyond the contraction's end is zero.  Beyond the last
  // row/column anything will do, so a kMajorMN piece that ends there is read
  // whole, into the rows that follow, where these exist: element by element,
  // the tiles at the edge would be slower than all others together (weight
  // gradients of 8192 rows, 8 experts, 2047 x 2047: 459 us, so 207).
  __device__ __forceinline__ void fetch(int set, int rest) {
    const int left = min(rest, kStep), follow = ld >= kVec ? 1 : kVec;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      int row, col;
      where(j, row, col);
      const T *p;
      int n;  // elements that exist
      if constexpr (MJ == kMajorK) {
        p = base + static_cast<int64_t>(min(row, valid - 1)) * ld + col * kVec;
        n = left - col * kVec;
      } else {
        p = base + static_cast<int64_t>(row) * ld + col * kVec;
        n = row < left ? valid - col * kVec : 0;
        if (n > 0 && row + follow < rest) n = kVec;
      }
      ux4 v = {};
      if (n >= kVec) {
        __builtin_memcpy(&v, p, 16);
      } else if (n > 0) {
        T h[kVec] = {};
#pragma unroll
        for (int i = 0; i < kVec - 1; ++i)
          if (i < n) h[i] = p[i];
        __builtin_memcpy(&v, h, 16);
      }
      reg[set][j] = v;
    }
  }
  __device__ __forceinline__ void land(int set, char *stage) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) *reinterpret_cast<ux4 *>(stage + (j * NT + threadIdx.x) * 16) = reg[set][j];
  }

  // The 16 bytes of contraction elements from (ks * 4 + lane / 16) kVec on, of
  // row/column r + lane % 16 of the stage.
  static __device__ __forceinline__ Frag<E> fragment(const char *stage, int r, int ks) {
    const int lane = threadIdx.x & 63;
    if constexpr (MJ == kMajorK) {
      const int row = r + (lane & 15), c = ks * 4 + (lane >> 4);
      return *reinterpret_cast<const Frag<E> *>(stage + row * 128 + ((c ^ k_swizzle<E, W>(row)) << 4));
    } else if constexpr (E == kF32) {
      const int i = r + (lane & 15);
      const char *p = stage + (ks * 16 + (lane >> 4) * 4) * (W * 4) + (((i >> 2) ^ (lane >> 2 & 4)) << 4) + (i & 3) * 4;
      fx4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float *>(p + j * (W * 4));
      return v;
    } else if constexpr (E == kF8) {
      ux4 v;
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // 8 contraction elements each: a block of 8 x 16 bytes per 16 lanes
        const int k = ks * 64 + (lane >> 4) * 16 + 8 * i + ((lane & 15) >> 1);
        const char *p = stage + k * W + (((r >> 4) ^ mn_swizzle8<W>(k)) << 4) + (lane & 1) * 8;
        const ux2 h = __builtin_bit_cast(
            ux2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) ix2 *)const_cast<char *>(p)));
        v[2 * i] = h[0];
        v[2 * i + 1] = h[1];
      }
      return v;
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

// Tile shape: BM x BN by WM x WN waves, each wave 16-row fragments; the LDS
// holds kStages stages (of aligned operands; of others two).
template <int BM_, int BN_, int WM_, int WN_, int STAGES = 2>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kStages = STAGES;
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments of a wave
};

// The way out of a tile.  A lane's four sums lie in one row, 16 rows to an
// instruction: stored from there, memory would see 32- or 64-byte pieces (a
// weight gradient of 64 experts, 738 MB of fp32: 346 us; with whole lines 270,
// with non-temporal stores of them 227).  So the sums pass through the LDS, which the
// contraction no longer needs, IP rows of fragments of each wave at a time,
// and leave it along rows or along columns, four sums to a lane.
// Banks: 16-byte chunk c of row r is kept at c ^ ((r >> 2 ^ r << 2) & 15),
// which takes 8 values over 8 neighbouring rows (the writes) and 16 over 16
// neighbouring groups of four rows (the reads along columns).
template <class S, int LDS>
struct TileOut {
  static constexpr int kRowBytes = S::BN * 4;
  // rows of fragments of a wave that fit, a power of two
  static constexpr int fit(int ip) { return ip * 16 * S::WM * kRowBytes <= LDS ? ip : fit(ip / 2); }
  static constexpr int IP = fit(S::FM), kPasses = S::FM / IP, kRows = IP * 16 * S::WM;
  static_assert(S::BN >= 64 && IP >= 1, "16 chunks to a row, and room for one row of fragments");

  static __device__ __forceinline__ char *at(char *lds, int row, int chunk) {
    return lds + row * kRowBytes + ((chunk ^ (((row >> 2) ^ (row << 2)) & 15)) << 4);
  }
  // Tile row of the pass's row r.
  static __device__ __forceinline__ int tile_row(int pass, int r) {
    return r / (IP * 16) * (S::BM / S::WM) + pass * IP * 16 + r % (IP * 16);
  }
  // v: this thread's sums of fragment rows pass * IP ..
  static __device__ __forceinline__ void put(char *lds, const fx4 (&v)[IP][S::FN], int tid) {
    const int wave = tid >> 6, lane = tid & 63;
    const int row = wave / S::WN * (IP * 16) + (lane & 15), chunk = wave % S::WN * (S::BN / S::WN / 4) + (lane >> 4);
#pragma unroll
    for (int i = 0; i < IP; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) *reinterpret_cast<fx4 *>(at(lds, row + i * 16, chunk + j * 4)) = v[i][j];
  }
  // f(m, n, v): v holds C[m][n .. n + 3] of the tile, neighbouring lanes along n.
  template <class F>
  static __device__ __forceinline__ void rows(char *lds, int pass, int tid, F f) {
    constexpr int kAll = kRows * S::BN / 4;
    static_assert(kAll % S::kThreads == 0, "whole rounds");
#pragma unroll 4
    for (int r = 0; r < kAll / S::kThreads; ++r) {
      const int c = r * S::kThreads + tid, row = c / (S::BN / 4), chunk = c % (S::BN / 4);
      f(tile_row(pass, row), chunk * 4, *reinterpret_cast<const fx4 *>(at(lds, row, chunk)));
    }
  }
  // f(m, n, v): v holds C[m .. m + 3][n], neighbouring lanes along m.
  template <class F>
  static __device__ __forceinline__ void columns(char *lds, int pass, int tid, F f) {
    constexpr int kAll = kRows / 4 * S::BN;
#pragma unroll 4
    for (int r = 0; r < kAll / S::kThreads; ++r) {
      const int c = r * S::kThreads + tid, row = c % (kRows / 4) * 4, n = c / (kRows / 4);
      fx4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const float *>(at(lds, row + i, n >> 2))[n & 3];
      f(tile_row(pass, row), n, v);
    }
  }
  // All of acc through f(pass, thread), called when the pass's sums are in
  // the LDS.  The thread number is hidden from the compiler, which would
  // compute the addresses of the way out before the contraction and hold them
  // in registers through it.
  template <class F>
  static __device__ __forceinline__ void all(char *lds, const fx4 (&acc)[S::FM][S::FN], F f) {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      fx4 v[IP][S::FN];
#pragma unroll
      for (int i = 0; i < IP; ++i)
#pragma unroll
        for (int j = 0; j < S::FN; ++j) v[i][j] = acc[pass * IP + i][j];
      if (pass > 0) __syncthreads();
      put(lds, v, tid);
      __syncthreads();
      f(pass, tid);
    }
    __syncthreads();
  }
};

// The contraction over k, or over three pairs of planes of length k (a
// multiple of kStepK then) added into one sum: numbers held as the sum of two
// 16-bit planes, hi and lo, give hi lo + lo hi + hi hi.  The small products
// come first:
// every addition to a sum is off by a part of the sum (the matrix instruction
// cuts), and with hi hi first the other two pairs would add to the full sum
// (X X^T of 64 x 2432: 4.9e-6 off, in this order 2.1e-6).  Finishes with all
// LDS reads done.
//
// Two loops.  Tiles of 256 x 256 with 8 waves (two per SIMD) hold their
// fragments in two register sets: while the matrix instructions work on one
// half of a stage, the other half's LDS reads and the next stage but one's
// loads are issued between them, so that a stage costs one meeting and no
// wait for the LDS.  Smaller tiles leave room for several workgroups on a CU,
// which cover each other's waits, and read each fragment right before its
// use.  bf16, 8192^3, both operands kMajorK: 1.40 PFLOP/s with the first loop
// and this tile (a large library product: 1.44), 1.22 with the second; 128 x
// 128 tiles of 4 waves 1.08 with the second; a bucket of 1024-sized matrices,
// whose launches these share, takes 1178 us with the second for them and 1214
// with the first.  (16 waves with the second loop: 1.27; 4 waves of 128 x 128
// with the first: 0.96; two wave groups that alternate between LDS reads and
// matrix instructions: 1.24; stages of 32 elements, five of them in the LDS: 9%
// slower, its loads being half lines.)
template <Elem E, class S, Major AM, Major BMJ, bool ALIGNED>
struct TileProduct {
  using T = ElemOf<E>;
  using Sh = S;
  using OpA = Operand<E, AM, S::BM, S::kThreads, ALIGNED>;
  using OpB = Operand<E, BMJ, S::BN, S::kThreads, ALIGNED>;
  static constexpr int kStep = OpA::kStep;
  static constexpr int kStage = OpA::kBytes + OpB::kBytes;
  static constexpr int kStages = ALIGNED ? S::kStages : 2;
  static constexpr bool kTwoSets = ALIGNED && S::BM * S::BN >= 256 * 256;
  static constexpr int kLds = kTwoSets ? kStage * 5 / 2 : kStages * kStage;
  static_assert(!kTwoSets || OpA::kBytes == OpB::kBytes, "a ring of operand stages");
  fx4 acc[S::FM][S::FN];
  OpA oa;
  OpB ob;
  // what is loaded next: stage `at` of `per` of pair `pair`
  const T *a0, *b0;
  int64_t lo_a, lo_b;  // elements from a hi plane to its lo plane
  // (32 bits: ordered 64-bit comparisons would go to the vector unit)
  int k, at, per;
  int pair, pairs;

  __device__ __forceinline__ int left() const {
    return min(k - at * kStep, kStep);
  }
  __device__ __forceinline__ void next() {
    if (++at < per) {
      oa.advance();
      ob.advance();
    } else if (++pair < pairs) {
      at = 0;
      oa.point(a0 + (pair + 2 == pairs ? lo_a : 0));
      ob.point(b0);
    }
  }
  // Only a list of one pair may end inside a stage: the masks of cut() stay.
  __device__ __forceinline__ void existing() {
    const int n = left();
    if (n < kStep) {
      oa.cut(n);
      ob.cut(n);
    }
  }
  __device__ __forceinline__ void load(uint32_t stage) {
    existing();
    oa.load(stage);
    ob.load(stage + OpA::kBytes);
    next();
  }
  __device__ __forceinline__ void fetch(int set) {
    oa.fetch(set, k - at * kStep);
    ob.fetch(set, k - at * kStep);
    next();
  }
  __device__ __forceinline__ void land(int set, char *stage) {
    oa.land(set, stage);
    ob.land(set, stage + OpA::kBytes);
  }

  __device__ __forceinline__ void run(char *lds, const T *a, const T *b, int64_t lda, int64_t ldb,
                                      int validm, int validn, int length, int npairs = 1, int64_t plane_a = 0,
                                      int64_t plane_b = 0) {
#pragma unroll
    for (int i = 0; i < S::FM; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) acc[i][j] = fx4{0, 0, 0, 0};
    if (length <= 0) return;
    a0 = a;
    b0 = b;
    lo_a = plane_a;
    lo_b = plane_b;
    pairs = npairs;
    k = length;
    pair = 0;
    at = 0;
    per = k / kStep + (k % kStep != 0);
    oa.init(a, lda, validm);
    ob.init(b + (pairs > 1 ? lo_b : 0), ldb, validn);
    if constexpr (kTwoSets) two_sets(lds, per * pairs);
    else if constexpr (ALIGNED) one_set(lds, per * pairs);
    else through_registers(lds, per * pairs);
  }

  // The products of the stage at sa.
  __device__ __forceinline__ void multiply(const char *sa, int rm, int rn) {
    const char *sb = sa + OpA::kBytes;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      Frag<E> fa[S::FM], fb[S::FN];
#pragma unroll
      for (int i = 0; i < S::FM; ++i) fa[i] = OpA::fragment(sa, rm + i * 16, ks);
#pragma unroll
      for (int j = 0; j < S::FN; ++j) fb[j] = OpB::fragment(sb, rn + j * 16, ks);
#pragma unroll
      for (int i = 0; i < S::FM; ++i)
#pragma unroll
        for (int j = 0; j < S::FN; ++j) acc[i][j] = mfma16<E>(fb[j], fa[i], acc[i][j]);
    }
  }

  __device__ __forceinline__ void one_set(char *lds, int steps) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rm = wave / S::WN * (S::BM / S::WM), rn = wave % S::WN * (S::BN / S::WN);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    constexpr int kAhead = kStages - 1;  // stages in flight when a step begins
    constexpr int kLoads = OpA::kPer + OpB::kPer;
    for (int i = 0; i < kAhead && i < steps; ++i) load(lds0 + i * kStage);
    int buf = 0, to = kAhead;  // stage read, stage loaded
    for (int t = 0; t < steps; ++t) {
      if (kAhead > 1 && t + kAhead <= steps) {  // all but the newest kAhead - 1 stages have landed
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kAhead - 1) * kLoads) : "memory");
      } else {
        loads_done_and_meet();
      }
      if (t + kAhead < steps) load(lds0 + to * kStage);
      multiply(lds + buf * kStage, rm, rn);
      buf = buf + 1 == kStages ? 0 : buf + 1;
      to = to + 1 == kStages ? 0 : to + 1;
    }
    __syncthreads();
  }

  // Operands that are not aligned.  Step t: stage t + kSets starts on its way
  // to the registers that stage t left for the LDS; after the products stage
  // t + 1, whose loads began kSets - 1 steps ago, goes to the LDS's other half.
  __device__ __forceinline__ void through_registers(char *lds, int steps) {
    constexpr int kSets = OpA::kSets < OpB::kSets ? OpA::kSets : OpB::kSets;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rm = wave / S::WN * (S::BM / S::WM), rn = wave % S::WN * (S::BN / S::WN);
#pragma unroll
    for (int i = 0; i < kSets; ++i)
      if (i < steps) fetch(i);
    land(0, lds);
    auto step = [&](int t, auto set) {
      constexpr int cur = decltype(set)::value, nxt = (cur + 1) % kSets;
      __syncthreads();
      if (t + kSets < steps) fetch(cur);
      multiply(lds + (t & 1) * kStage, rm, rn);
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

  // The LDS is a ring of five parts, each one operand's stage: A of stage t in
  // part 2t % 5, B in the next.  The first half of stage t's contraction
  // elements is in register set 0 when step t begins.  Step t: matrix
  // instructions on set 0 while set 1 reads the stage's other half and A of
  // stage t + 2 starts on its way to the part that B of stage t - 1 left; then
  // every wave is done with stage t, and stage t + 1 has landed (its loads
  // began a step ago): matrix instructions on set 1 while set 0 reads stage
  // t + 1 and B of stage t + 2 starts into the part of A of stage t.  So one
  // load goes out for every two rows of fragments: all in the second half of
  // the step (two stages of LDS do for that), they take 2% longer, and in its
  // first quarter 8%.  The steps without such loads, and the one before them,
  // whose stage may be cut, are apart, so that the others are free of branches.
  __device__ __forceinline__ void two_sets(char *lds, int steps) {
    enum { kWhole, kLast, kNone };
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rm = wave / S::WN * (S::BM / S::WM), rn = wave % S::WN * (S::BN / S::WN);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    constexpr int kReads = S::FM + S::FN, kLoads = OpA::kPer + OpB::kPer;
    Frag<E> fa[2][S::FM], fb[2][S::FN];
    auto read = [&](int set, const char *sa, const char *sb, int ks, int r) {
      if (r < S::FN) fb[set][r] = OpB::fragment(sb, rn + r * 16, ks);
      else fa[set][r - S::FN] = OpA::fragment(sa, rm + (r - S::FN) * 16, ks);
    };
    load(lds0);
    if (steps > 1) {
      load(lds0 + kStage);  // (parts 2 and 3)
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
    } else {
      loads_done_and_meet();
    }
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(0, lds, lds + OpA::kBytes, 0, r);
    // kind: kWhole / kLast where a stage t + 2 exists and is whole / may be cut
    constexpr int kPart = OpA::kBytes;
    const auto part = [](int p) { return p >= 5 * kPart ? p - 5 * kPart : p; };
    int at_a = 0;  // where A of stage t is
    auto step = [&](auto kind) {
      constexpr bool more = decltype(kind)::value != kNone;
      const char *sa = lds + at_a, *sb = lds + part(at_a + kPart);
      const char *na = lds + part(at_a + 2 * kPart), *nb = lds + part(at_a + 3 * kPart);
      const uint32_t da = lds0 + part(at_a + 4 * kPart), db = lds0 + at_a;
      if constexpr (decltype(kind)::value == kLast) existing();
#pragma unroll
      for (int i = 0; i < S::FM; ++i) {
        if constexpr (more) {
#pragma unroll
          for (int r = i * OpA::kPer / S::FM; r < (i + 1) * OpA::kPer / S::FM; ++r) oa.load_one(r, da);
        }
#pragma unroll
        for (int r = i * kReads / S::FM; r < (i + 1) * kReads / S::FM; ++r) read(1, sa, sb, 1, r);
#pragma unroll
        for (int j = 0; j < S::FN; ++j) acc[i][j] = mfma16<E>(fb[0][j], fa[0][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);  // keeps the reads spread among the products
      }
      // A of stage t + 2 may still be on its way
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(more ? OpA::kPer : 0) : "memory");
#pragma unroll
      for (int i = 0; i < S::FM; ++i) {
        if constexpr (more) {
#pragma unroll
          for (int r = i * OpB::kPer / S::FM; r < (i + 1) * OpB::kPer / S::FM; ++r) ob.load_one(r, db);
        }
        // (behind the last stage: what another tile or stage left, not used)
#pragma unroll
        for (int r = i * kReads / S::FM; r < (i + 1) * kReads / S::FM; ++r) read(0, na, nb, 0, r);
#pragma unroll
        for (int j = 0; j < S::FN; ++j) acc[i][j] = mfma16<E>(fb[1][j], fa[1][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (more) next();
      at_a = part(at_a + 2 * kPart);
    };
    int t = 0;
    for (; t + 3 < steps; ++t) step(std::integral_constant<int, kWhole>{});
    if (t + 2 < steps) step(std::integral_constant<int, kLast>{}), ++t;
    for (; t < steps; ++t) step(std::integral_constant<int, kNone>{});
    loads_done_and_meet();
  }
};

}  // namespace ar_dev

// clip.hip -- the norm of all gradients of an arena, and their scaling to a
// largest norm (gfx950).
//
//   norm = scale sqrt(sum g^2),   c = min(1, max_norm / (norm + 1e-6)),   g' = c g
//
// The host cuts the tensors into chunks, a wave's work each, so a kernel never
// looks for the tensor that an element is of, and elements between tensors
// are not touched.  Bound by memory: the norm reads every gradient, and the
// scaling, which needs the whole norm first, reads it again and writes it.  The
// squares in fp64 cost nothing beside that (fp32 ones take the same time).
// The norm's loads are ordinary ones, and the scaling finds part of what they
// left; its own loads and its stores are non-temporal (norm and scaling of 174 M
// bf16 gradients to another arena 167 us; with non-temporal loads in the norm too
// 183, with ordinary stores 206; going backwards over the chunks 170).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "grouped.hpp"
#include "kernels.hpp"
#include "operators.hpp"

namespace ar_dev {
namespace {

constexpr int kNormThreads = 64 * kNormWaves;

template <bool BF>
struct Grad {
  using T = std::conditional_t<BF, uint16_t, float>;
  static constexpr int kVec = 16 / sizeof(T);
  static __device__ __forceinline__ float wide(T v) {
    if constexpr (BF) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else return v;
  }
  static __device__ __forceinline__ T narrow(float v) {
    if constexpr (BF) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    else return v;
  }
  static __device__ __forceinline__ void split(ux4 v, float (&f)[kVec]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      } else {
        f[i] = __uint_as_float(v[i]);
      }
    }
  }
};

// A chunk's elements before its 16-byte pieces: those up to the next multiple of
// kVec elements of the arena, for the norm, whose order is the plan's then, at
// any address (174 M bf16 gradients in 300 tensors of an arena off 16 bytes: 76 us;
// on them 64); for the scaling, which has none, up to a boundary of what is
// written.
template <bool BF>
__device__ __forceinline__ int lead_of(uint64_t at, int n) {
  constexpr int kVec = Grad<BF>::kVec;
  return min(n, static_cast<int>(-at & (kVec - 1)));
}

// 16 bytes at any element's address: the hardware takes such loads.
typedef uint32_t ux4_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ double wave_total(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Squares in fp64 (exact of an fp32 number), so neither a large gradient's
// square overflows nor a small one's is lost.
template <bool BF>
__device__ __forceinline__ double chunk_squares(const NormArgs &a, const NormChunk &c) {
  using G = Grad<BF>;
  using T = typename G::T;
  const int lane = threadIdx.x & 63;
  const T *p = static_cast<const T *>(a.g) + c.at;
  const int lead = lead_of<BF>(static_cast<uint64_t>(c.at), c.count), pieces = (c.count - lead) / G::kVec;
  const int tail = lead + pieces * G::kVec;
  double s[2] = {0, 0};
  if (lane < lead) {
    const double d = G::wide(p[lane]);
    s[0] = d * d;
  }
  if (tail + lane < c.count) {
    const double d = G::wide(p[tail + lane]);
    s[1] = d * d;
  }
  const ux4_any *v = reinterpret_cast<const ux4_any *>(p + lead);
  auto add = [&](ux4 u) {
    float f[G::kVec];
    G::split(u, f);
#pragma unroll
    for (int i = 0; i < G::kVec; ++i) s[i & 1] = __builtin_fma(static_cast<double>(f[i]), static_cast<double>(f[i]), s[i & 1]);
  };
  constexpr int kBatch = 8;  // loads in flight
  int i = lane;
  for (; i + 64 * (kBatch - 1) < pieces; i += 64 * kBatch) {
    ux4 u[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) u[j] = v[i + 64 * j];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) add(u[j]);
  }
  for (; i < pieces; i += 64) add(v[i]);
  return wave_total(s[0] + s[1]);
}

// A workgroup's sum over its chunks; a launch of one workgroup has the norm then.
template <bool BF>
__global__ __launch_bounds__(kNormThreads) void norm_sums(NormArgs a) {
  __shared__ double part[kNormWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = uniform(static_cast<int32_t>(blockIdx.x * kNormWaves + wave));
  double s = 0;
  if (c < a.nchunks) {
    const NormChunk chunk = table_entry(a.chunks + c);
    s = chunk_squares<BF>(a, chunk);
    if (a.tensor_norms && lane == 0) a.chunk_sums[c] = s;
  }
  if (lane == 0) part[wave] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double sum = 0;
#pragma unroll
  for (int i = 0; i < kNormWaves; ++i) sum += part[i];
  if (gridDim.x == 1) a.norm[0] = static_cast<float>(__builtin_sqrt(sum) * a.scale);
  else a.group_sums[blockIdx.x] = sum;
}

// The workgroups' sums, added in a fixed order.  A launch of its own: that the
// last workgroup of norm_sums does it needs each of them to write its L2 back
// before it counts itself (174 M bf16 gradients: 120 us; so 60, 5.8 TB/s).
__global__ __launch_bounds__(kNormThreads) void norm_total(NormArgs a, int groups) {
  __shared__ double part[kNormWaves];
  double sum = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < groups; i += kNormThreads) sum += a.group_sums[i];
  sum = wave_total(sum);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  sum = 0;
#pragma unroll
  for (int i = 0; i < kNormWaves; ++i) sum += part[i];
  a.norm[0] = static_cast<float>(__builtin_sqrt(sum) * a.scale);
}

// The tensors' own norms: a wave adds the sums of its tensor's chunks.
__global__ __launch_bounds__(kNormThreads) void norm_tensors(NormArgs a) {
  const int t = blockIdx.x * kNormWaves + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= a.ntensors) return;
  double s = 0;
  for (int c = a.first[t] + lane; c < a.first[t + 1]; c += 64) s += a.chunk_sums[c];
  s = wave_total(s);
  if (lane == 0) a.tensor_norms[t] = static_cast<float>(__builtin_sqrt(s) * a.scale);
}

template <bool BF>
__global__ __launch_bounds__(kNormThreads) void clip_chunks(NormArgs a) {
  using G = Grad<BF>;
  using T = typename G::T;
  const int lane = threadIdx.x & 63;
  const int id = uniform(static_cast<int32_t>(blockIdx.x * kNormWaves + (threadIdx.x >> 6)));
  if (id >= a.nchunks) return;
  const float ratio = static_cast<float>(a.max_norm / (static_cast<double>(a.norm[0]) + 1e-6));
  const float c = ratio >= 1.0f ? 1.0f : ratio;  // NaN stays
  if (c == 1.0f && a.out == a.g) return;
  const NormChunk chunk = table_entry(a.chunks + id);
  const T *p = static_cast<const T *>(a.g) + chunk.at;
  T *q = static_cast<T *>(a.out) + chunk.at;
  const int lead = lead_of<BF>(reinterpret_cast<uintptr_t>(q) / sizeof(T), chunk.count);
  const int pieces = (chunk.count - lead) / G::kVec;
  const int tail = lead + pieces * G::kVec;
  if (lane < lead) q[lane] = G::narrow(G::wide(p[lane]) * c);
  if (tail + lane < chunk.count) q[tail + lane] = G::narrow(G::wide(p[tail + lane]) * c);
  const ux4_any *v = reinterpret_cast<const ux4_any *>(p + lead);
  ux4 *w = reinterpret_cast<ux4 *>(q + lead);
  auto scaled = [&](ux4 u) {
    float f[G::kVec];
    G::split(u, f);
    T h[G::kVec];
#pragma unroll
    for (int i = 0; i < G::kVec; ++i) h[i] = G::narrow(f[i] * c);
    ux4 r;
    __builtin_memcpy(&r, h, 16);
    return r;
  };
  constexpr int kBatch = 4;
  int i = lane;
  for (; i + 64 * (kBatch - 1) < pieces; i += 64 * kBatch) {
    ux4 u[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) u[j] = __builtin_nontemporal_load(v + i + 64 * j);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) __builtin_nontemporal_store(scaled(u[j]), w + i + 64 * j);
  }
  for (; i < pieces; i += 64) __builtin_nontemporal_store(scaled(__builtin_nontemporal_load(v + i)), w + i);
}

int64_t groups(int64_t n) { return (n + kNormWaves - 1) / kNormWaves; }

}  // namespace

hipError_t grad_norm(const NormArgs &a, hipStream_t s) {
  const LaunchEvents ev = t_launch_events;  // the call's mark goes on its last kernel
  const bool each = a.tensor_norms && a.ntensors > 0;
  const int64_t grid = std::max<int64_t>(1, groups(a.nchunks));
  if (each || grid > 1) t_launch_events = LaunchEvents{};
  hipError_t e = a.bf16 ? launch(norm_sums<true>, grid, 1, kNormThreads, 0, s, a)
                        : launch(norm_sums<false>, grid, 1, kNormThreads, 0, s, a);
  if (!each) t_launch_events = ev;
  if (e == hipSuccess && grid > 1) e = launch(norm_total, 1, 1, kNormThreads, 0, s, a, static_cast<int>(grid));
  t_launch_events = ev;
  if (e != hipSuccess || !each) return e;
  return launch(norm_tensors, groups(a.ntensors), 1, kNormThreads, 0, s, a);
}

hipError_t grad_clip(const NormArgs &a, hipStream_t s) {
  return a.bf16 ? launch(clip_chunks<true>, groups(a.nchunks), 1, kNormThreads, 0, s, a)
                : launch(clip_chunks<false>, groups(a.nchunks), 1, kNormThreads, 0, s, a);
}

}  // namespace ar_dev

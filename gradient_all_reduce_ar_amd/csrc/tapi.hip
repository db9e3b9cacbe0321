// tapi.hip -- C ABI (include/ar.h) of gradient clipping, of the RMS norm and of
// the 8-bit rows and expert products: argument checks, the plans' device
// tables, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>
#include <utility>
#include <vector>

#include "../../include/ar.h"
#include "host.hpp"
#include "kernels.hpp"
#include "operators.hpp"

using ar_host::check_rows;
using ar_host::fail;
using ar_host::float_type;
using ar_host::guarded;
using ar_host::hip_fail;
using ar_host::on;
using ar_host::overlap;
using ar_host::raw_enum;
using ar_host::RowsArg;

namespace {

// rows are counted in int32, rounded up to whole tiles
constexpr size_t kMaxTokens = (size_t{1} << 31) - 65536;
constexpr int64_t kMaxFeatures = 1 << 22;

int64_t blocks_of(int64_t n) { return (n + ar_dev::kQBlock8 - 1) / ar_dev::kQBlock8; }

// What a call reads or writes: `bytes` from p on.
struct Range {
  const void *p;
  int64_t bytes;
  const char *name;
};

// No output shares a byte with an input or another output.  `may`: an output
// and an input of the same pointer that were found to be the same rows.
ar_status_t check_apart(const std::vector<Range> &outs, const std::vector<Range> &ins,
                        const std::vector<std::pair<int, int>> &may = {}) {
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
        return fail(AR_ERR_INVALID_ARG, std::string(outs[i].name) + " and " + outs[j].name + " overlap");
    for (size_t j = 0; j < ins.size(); ++j) {
      if (!overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) continue;
      if (std::find(may.begin(), may.end(), std::pair<int, int>(static_cast<int>(i), static_cast<int>(j))) != may.end())
        continue;
      return fail(AR_ERR_INVALID_ARG, std::string(outs[i].name) + " and " + ins[j].name + " overlap");
    }
  }
  return AR_OK;
}

ar_status_t check_pointer(const void *p, uintptr_t elem, const char *name) {
  if (!p) return fail(AR_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (!on(p, elem)) return fail(AR_ERR_INVALID_ARG, std::string(name) + " is not aligned to its elements");
  return AR_OK;
}

ar_status_t launched(hipError_t e, const char *what) {
  if (e == hipErrorInvalidConfiguration)
    return fail(AR_ERR_UNSUPPORTED, std::string(what) + " larger than one launch grid");
  return e == hipSuccess ? AR_OK : hip_fail(e, "kernel launch");
}

// Launches f on s and marks the call's end.
template <class F>
ar_status_t run_marked(ar_host::CallMarks &marks, hipStream_t s, const char *what, F f) {
  hipEvent_t mark = nullptr;
  const ar_status_t st = marks.of(s, &mark);
  if (st != AR_OK) return st;
  ar_dev::t_launch_events = ar_dev::LaunchEvents{nullptr, mark};
  const hipError_t e = f();
  ar_dev::t_launch_events = ar_dev::LaunchEvents{};
  return launched(e, what);
}

// Where a plan is prepared, its device has to be the current one.
template <class P>
ar_status_t check_device(const P *p, const char *what) {
  if (p->device < 0) return AR_OK;
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  return dev == p->device ? AR_OK : fail(AR_ERR_INVALID_ARG, std::string(what) + " plan was prepared on another device");
}

// Allocates a plan's device memory with f on the current device, once.
template <class P, class F>
ar_status_t prepare_on(P *p, const char *what, F f) {
  if (p->device >= 0) return check_device(p, what);
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  e = f();
  if (e != hipSuccess) {
    p->release();
    const std::string name = std::string(what) + " workspace";
    return e == hipErrorOutOfMemory ? fail(AR_ERR_OOM, name + " allocation") : hip_fail(e, name.c_str());
  }
  p->device = dev;
  return AR_OK;
}

// prepare for a call on `stream`.
template <class P>
ar_status_t prepare_for(P *p, void *stream) {
  const ar_status_t st = p->device >= 0 ? AR_OK : ar_host::refuse_capture(static_cast<hipStream_t>(stream));
  return st == AR_OK ? p->prepare() : st;
}

void free_all(std::initializer_list<void **> all) {
  for (void **p : all) {
    if (*p) (void)hipFree(*p);
    *p = nullptr;
  }
}

}  // namespace

// ------------------------------------------------------- norm and clipping

struct ar_norm_plan {
  bool bf16 = false;
  int32_t ntensors = 0;
  int64_t count = 0, arena = 0;
  std::vector<ar_dev::NormChunk> chunks;
  std::vector<int32_t> first;  // [ntensors + 1]
  int device = -1;
  void *d_chunks = nullptr, *d_first = nullptr, *d_sums = nullptr;
  ar_host::CallMarks marks;

  int64_t groups() const {
    return std::max<int64_t>(1, (static_cast<int64_t>(chunks.size()) + ar_dev::kNormWaves - 1) / ar_dev::kNormWaves);
  }
  // the workgroups' sums, the chunks'
  size_t sum_bytes() const { return 8 * (static_cast<size_t>(groups()) + chunks.size()); }
  size_t table_bytes() const { return chunks.size() * sizeof(ar_dev::NormChunk) + first.size() * 4; }

  ar_status_t prepare() {
    return prepare_on(this, "norm", [&] {
      hipError_t e = ar_host::device_table(&d_sums, nullptr, sum_bytes());
      if (e == hipSuccess && !chunks.empty())
        e = ar_host::device_table(&d_chunks, chunks.data(), chunks.size() * sizeof(ar_dev::NormChunk));
      if (e == hipSuccess) e = ar_host::device_table(&d_first, first.data(), first.size() * 4);
      return e;
    });
  }
  void release() {
    marks.release();
    free_all({&d_chunks, &d_first, &d_sums});
    device = -1;
  }
};

namespace {

// Elements of a chunk: whole 64 x 16 bytes, so that chunks of an aligned tensor
// stay aligned; few gradients in one workgroup, which saves a launch, more of
// them in enough chunks to fill the device, of 16 KiB at most (norm and
// scaling of 174 M bf16 gradients 167 us; with 32 KiB 171, with 8 KiB 164, but 184 M
// fp32 ones then take 371 instead of 356).  Over 2^36 gradients again more: 2^24
// chunks and two for each tensor's ends are less than one launch takes.
int64_t chunk_elements(int64_t count, bool bf16) {
  const int64_t piece = bf16 ? 512 : 256;
  if (count <= ar_dev::kNormWaves * 8 * piece)
    return std::max(piece, (count / ar_dev::kNormWaves + piece - 1) / piece * piece);
  const int64_t even = (count / (256 * 16) + piece - 1) / piece * piece;
  return std::max(std::clamp<int64_t>(even, piece, 16 * piece), ((count >> 24) + piece - 1) / piece * piece);
}

ar_dev::NormArgs norm_args(const ar_norm_plan *p) {
  ar_dev::NormArgs a{};
  a.chunks = static_cast<const ar_dev::NormChunk *>(p->d_chunks);
  a.first = static_cast<const int32_t *>(p->d_first);
  a.group_sums = static_cast<double *>(p->d_sums);
  a.chunk_sums = a.group_sums + p->groups();
  a.nchunks = static_cast<int32_t>(p->chunks.size());
  a.ntensors = p->ntensors;
  a.bf16 = p->bf16;
  return a;
}

}  // namespace

// ---------------------------------------------------------------- RMS norm

struct ar_rmsnorm {
  int64_t features = 0;
  bool bf16 = false, gain_bf16 = false, grad_bf16 = false;
  double eps = 0;
  int32_t parts = 0;
  int device = -1;
  void *d_parts = nullptr;
  ar_host::CallMarks marks;

  int64_t elem() const { return bf16 ? 2 : 4; }
  int64_t gain_bytes() const { return features * (gain_bf16 ? 2 : 4); }
  int64_t grad_bytes() const { return features * (grad_bf16 ? 2 : 4); }
  size_t part_bytes() const { return static_cast<size_t>(parts) * static_cast<size_t>(features) * 4; }
  ar_status_t prepare() {
    return prepare_on(this, "RMS norm", [&] { return ar_host::device_table(&d_parts, nullptr, part_bytes()); });
  }
  void release() {
    marks.release();
    free_all({&d_parts});
    device = -1;
  }
};

namespace {

ar_status_t forward(ar_rmsnorm *p, const ar_rmsnorm_forward_t &q, size_t ntokens, void *stream) {
  if (ntokens > kMaxTokens) return fail(AR_ERR_INVALID_ARG, "more than 2^31 - 65536 tokens");
  const int64_t t = static_cast<int64_t>(ntokens), f = p->features, b = blocks_of(f);
  if ((q.codes != nullptr) != (q.scales != nullptr)) return fail(AR_ERR_INVALID_ARG, "codes and scales come together");
  int64_t bx = 0, br = 0, bh = 0, by = 0, bc = 0, bs = 0;
  ar_status_t st = check_rows({q.x, q.x_stride, f, "x"}, t, p->elem(), &bx);
  if (st == AR_OK && q.residual) st = check_rows({q.residual, q.residual_stride, f, "residual"}, t, p->elem(), &br);
  if (st == AR_OK && q.h) st = check_rows({q.h, q.h_stride, f, "h"}, t, p->elem(), &bh);
  if (st == AR_OK && q.y) st = check_rows({q.y, q.y_stride, f, "y"}, t, p->elem(), &by);
  if (st == AR_OK && q.codes) st = check_rows({q.codes, q.codes_stride, f, "codes"}, t, 1, &bc);
  if (st == AR_OK && q.scales) st = check_rows({q.scales, q.scales_stride, b, "scales"}, t, 1, &bs);
  if (st == AR_OK && t > 0) st = check_pointer(q.gain, p->gain_bf16 ? 2 : 4, "gain");
  if (st == AR_OK && t > 0 && q.rstd) st = check_pointer(q.rstd, 4, "rstd");
  if (st != AR_OK) return st;
  if (t > 0) {
    std::vector<std::pair<int, int>> may;  // h (0) or y (1) is x (0) or residual (1)
    auto same = [&](const void *o, size_t os, const void *i, size_t is) { return o && o == i && (os == is || t == 1); };
    if (same(q.h, q.h_stride, q.x, q.x_stride)) may.push_back({0, 0});
    if (same(q.h, q.h_stride, q.residual, q.residual_stride)) may.push_back({0, 1});
    if (same(q.y, q.y_stride, q.x, q.x_stride)) may.push_back({1, 0});
    if (same(q.y, q.y_stride, q.residual, q.residual_stride)) may.push_back({1, 1});
    st = check_apart({{q.h, bh, "h"}, {q.y, by, "y"}, {q.codes, bc, "codes"}, {q.scales, bs, "scales"},
                      {q.rstd, q.rstd ? 4 * t : 0, "rstd"}},
                     {{q.x, bx, "x"}, {q.residual, br, "residual"}, {q.gain, p->gain_bytes(), "gain"}}, may);
    if (st != AR_OK) return st;
  }
  // the kernel uses nothing of the plan's: no workspace for it, which a program that only runs forward would never
  // touch, and no mark, since destroying the plan need not wait
  st = check_device(p, "RMS norm");
  if (st != AR_OK || t == 0) return st;
  ar_dev::RmsForward a{};
  a.x = q.x;
  a.r = q.residual;
  a.gain = q.gain;
  a.h = q.h;
  a.y = q.y;
  a.codes = static_cast<uint8_t *>(q.codes);
  a.scales = static_cast<uint8_t *>(q.scales);
  a.rstd = q.rstd;
  a.xs = static_cast<int64_t>(q.x_stride);
  a.rs = static_cast<int64_t>(q.residual_stride);
  a.hs = static_cast<int64_t>(q.h_stride);
  a.ys = static_cast<int64_t>(q.y_stride);
  a.cs = static_cast<int64_t>(q.codes_stride);
  a.ss = static_cast<int64_t>(q.scales_stride);
  a.tokens = t;
  a.features = static_cast<int32_t>(f);
  a.eps = p->eps;
  a.bf16 = p->bf16;
  a.gain_bf16 = p->gain_bf16;
  return launched(ar_dev::rmsnorm_forward(a, static_cast<hipStream_t>(stream)), "RMS norm");
}

ar_status_t backward(ar_rmsnorm *p, const ar_rmsnorm_backward_t &q, size_t ntokens, void *stream) {
  if (ntokens > kMaxTokens) return fail(AR_ERR_INVALID_ARG, "more than 2^31 - 65536 tokens");
  const int64_t t = static_cast<int64_t>(ntokens), f = p->features;
  int64_t bdy = 0, bh = 0, bdh = 0, bdx = 0;
  ar_status_t st = check_rows({q.dy, q.dy_stride, f, "dy"}, t, p->elem(), &bdy);
  if (st == AR_OK) st = check_rows({q.h, q.h_stride, f, "h"}, t, p->elem(), &bh);
  if (st == AR_OK && q.dh) st = check_rows({q.dh, q.dh_stride, f, "dh"}, t, p->elem(), &bdh);
  if (st == AR_OK) st = check_rows({q.dx, q.dx_stride, f, "dx"}, t, p->elem(), &bdx);
  if (st == AR_OK) st = check_pointer(q.dgain, p->grad_bf16 ? 2 : 4, "dgain");
  if (st == AR_OK && t > 0) st = check_pointer(q.gain, p->gain_bf16 ? 2 : 4, "gain");
  if (st == AR_OK && t > 0) st = check_pointer(q.rstd, 4, "rstd");
  if (st != AR_OK) return st;
  if (t > 0) {
    std::vector<std::pair<int, int>> may;  // dx (0) is dy (0), h (1) or dh (2)
    auto same = [&](const void *i, size_t is) { return q.dx == i && (q.dx_stride == is || t == 1); };
    if (same(q.dy, q.dy_stride)) may.push_back({0, 0});
    if (same(q.h, q.h_stride)) may.push_back({0, 1});
    if (same(q.dh, q.dh_stride)) may.push_back({0, 2});
    st = check_apart({{q.dx, bdx, "dx"}, {q.dgain, p->grad_bytes(), "dgain"}},
                     {{q.dy, bdy, "dy"}, {q.h, bh, "h"}, {q.dh, bdh, "dh"}, {q.gain, p->gain_bytes(), "gain"},
                      {q.rstd, 4 * t, "rstd"}}, may);
    if (st != AR_OK) return st;
  }
  st = prepare_for(p, stream);
  if (st != AR_OK || (t == 0 && q.accumulate)) return st;
  ar_dev::RmsBackward a{};
  a.dy = q.dy;
  a.h = q.h;
  a.dh = q.dh;
  a.gain = q.gain;
  a.rstd = q.rstd;
  a.dx = q.dx;
  a.dgain = q.dgain;
  a.parts = static_cast<float *>(p->d_parts);
  a.dys = static_cast<int64_t>(q.dy_stride);
  a.hs = static_cast<int64_t>(q.h_stride);
  a.dhs = static_cast<int64_t>(q.dh_stride);
  a.dxs = static_cast<int64_t>(q.dx_stride);
  a.tokens = t;
  a.features = static_cast<int32_t>(f);
  a.bf16 = p->bf16;
  a.gain_bf16 = p->gain_bf16;
  a.grad_bf16 = p->grad_bf16;
  a.accumulate = q.accumulate != 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run_marked(p->marks, s, "RMS norm", [&] { return ar_dev::rmsnorm_backward(a, s); });
}

}  // namespace

// ----------------------------------------------------- 8-bit expert products

struct ar_qexperts {
  int32_t nexperts = 0;
  int64_t in = 0, out = 0;
  bool bf16 = false;
  std::vector<int64_t> offsets;
  int64_t arena = 0;          // elements an arena holds at least
  bool offsets_by_16 = true;  // every matrix starts on a multiple of 16 elements
  int device = -1;
  void *d_offsets = nullptr;
  ar_host::CallMarks marks;

  int64_t scale_count() const { return nexperts * blocks_of(in) * blocks_of(out); }
  ar_status_t prepare() {
    return prepare_on(this, "8-bit expert",
                      [&] { return ar_host::device_table(&d_offsets, offsets.data(), offsets.size() * sizeof(int64_t)); });
  }
  void release() {
    marks.release();
    free_all({&d_offsets});
    device = -1;
  }
};

namespace {

ar_dev::QExpertArgs call_args(const ar_qexperts *p, int64_t tokens) {
  ar_dev::QExpertArgs a{};
  a.tokens = tokens;
  a.in = p->in;
  a.outf = p->out;
  a.experts = p->nexperts;
  a.bf16 = p->bf16;
  a.aligned = p->in % 16 == 0 && p->out % 16 == 0 && p->offsets_by_16;
  return a;
}

ar_status_t product(ar_qexperts *p, bool grad, const RowsArg &x, const RowsArg &xs, const void *weights,
                    const void *weight_scales, const RowsArg &y, const int32_t *ends, size_t ntokens, void *stream) {
  if (ntokens > kMaxTokens) return fail(AR_ERR_INVALID_ARG, "more than 2^31 - 65536 tokens");
  const int64_t t = static_cast<int64_t>(ntokens), elem = p->bf16 ? 2 : 4;
  int64_t bx = 0, bs = 0, by = 0;
  ar_status_t st = check_rows(x, t, 1, &bx);
  if (st == AR_OK) st = check_rows(xs, t, 1, &bs);
  if (st == AR_OK) st = check_rows(y, t, elem, &by);
  if (st == AR_OK && t > 0) st = check_pointer(ends, 4, "ends");
  if (st == AR_OK && t > 0) st = check_pointer(weights, 1, "the weight arena");
  if (st == AR_OK && t > 0) st = check_pointer(weight_scales, 1, "weight_scales");
  if (st == AR_OK && t > 0)
    st = check_apart({{y.p, by, y.name}},
                     {{x.p, bx, x.name}, {xs.p, bs, xs.name}, {weights, p->arena, "the weight arena"},
                      {weight_scales, p->scale_count(), "weight_scales"}, {ends, 4 * static_cast<int64_t>(p->nexperts), "ends"}});
  if (st == AR_OK) st = prepare_for(p, stream);
  if (st != AR_OK || t == 0) return st;
  ar_dev::QExpertArgs a = call_args(p, t);
  a.x = static_cast<const uint8_t *>(x.p);
  a.w = static_cast<const uint8_t *>(weights);
  a.x_scales = static_cast<const uint8_t *>(xs.p);
  a.w_scales = static_cast<const uint8_t *>(weight_scales);
  a.out = const_cast<void *>(y.p);
  a.offsets = static_cast<const int64_t *>(p->d_offsets);
  a.ends = ends;
  a.xs = static_cast<int64_t>(x.stride);
  a.xss = static_cast<int64_t>(xs.stride);
  a.outs = static_cast<int64_t>(y.stride);
  a.aligned = a.aligned && on(x.p, 16) && x.stride % 16 == 0 && on(weights, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run_marked(p->marks, s, "expert product",
                    [&] { return grad ? ar_dev::qexperts_input_grad(a, s) : ar_dev::qexperts_forward(a, s); });
}

}  // namespace

extern "C" {

ar_norm_plan_t *ar_norm_plan_create(int ntensors, const size_t *counts, const size_t *offsets, ar_dtype_t grad_dtype) {
  ar_norm_plan *p = nullptr;
  const ar_status_t st = guarded([&]() -> ar_status_t {
    const int32_t g = raw_enum(grad_dtype);
    if (ntensors < 0 || ntensors > 1 << 20) return fail(AR_ERR_INVALID_ARG, "ntensors must be from 0 to 2^20");
    if (ntensors > 0 && !counts) return fail(AR_ERR_INVALID_ARG, "counts is NULL");
    if (!float_type(g)) return fail(AR_ERR_INVALID_ARG, "norm plans take AR_FLOAT32 or AR_BFLOAT16");
    p = new ar_norm_plan;
    p->bf16 = g == AR_BFLOAT16;
    p->ntensors = ntensors;
    constexpr int64_t kMost = int64_t{1} << 40;
    std::vector<std::pair<int64_t, int64_t>> ranges;
    int64_t next = 0;
    for (int i = 0; i < ntensors; ++i) {
      const std::string name = "tensor " + std::to_string(i);
      if (counts[i] > static_cast<size_t>(kMost)) return fail(AR_ERR_INVALID_ARG, name + " is too large");
      if (offsets && offsets[i] > static_cast<size_t>(INT64_MAX / 16))
        return fail(AR_ERR_INVALID_ARG, name + ": offset too large");
      const int64_t at = offsets ? static_cast<int64_t>(offsets[i]) : next;
      next = at + static_cast<int64_t>(counts[i]);
      p->count += static_cast<int64_t>(counts[i]);
      if (p->count > kMost) return fail(AR_ERR_INVALID_ARG, "the tensors hold more than 2^40 elements");
      ranges.push_back({at, next});
      if (next > at) p->arena = std::max(p->arena, next);
    }
    std::vector<std::pair<int64_t, int64_t>> sorted = ranges;
    std::sort(sorted.begin(), sorted.end());
    int64_t end = 0;
    for (const auto &r : sorted) {
      if (r.second == r.first) continue;
      if (r.first < end) return fail(AR_ERR_INVALID_ARG, "tensors overlap");
      end = r.second;
    }
    const int64_t size = chunk_elements(p->count, p->bf16);
    size_t chunks = 0;
    for (const auto &r : ranges)
      if (r.second > r.first) chunks += static_cast<size_t>((r.second - 1) / size - r.first / size + 1);
    p->chunks.reserve(chunks);
    for (int i = 0; i < ntensors; ++i) {
      p->first.push_back(static_cast<int32_t>(p->chunks.size()));
      // the first cut of a tensor falls where the following ones are multiples of the chunks' size in the arena
      for (int64_t at = ranges[i].first, last = ranges[i].second; at < last;) {
        const int64_t to = std::min(last, at / size * size + size);
        p->chunks.push_back({at, static_cast<int32_t>(to - at), 0});
        at = to;
      }
    }
    p->first.push_back(static_cast<int32_t>(p->chunks.size()));
    return AR_OK;
  });
  if (st != AR_OK) {
    delete p;
    return nullptr;
  }
  return p;
}

ar_status_t ar_norm_plan_prepare(ar_norm_plan_t *p) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "norm plan is NULL");
  return guarded([&] { return p->prepare(); });
}

ar_norm_stats_t ar_norm_plan_stats(const ar_norm_plan_t *p) {
  ar_norm_stats_t s{};
  if (!p) {
    fail(AR_ERR_INVALID_ARG, "norm plan is NULL");
    return s;
  }
  s.ntensors = p->ntensors;
  s.device = p->device;
  s.grad_bytes = p->bf16 ? 2 : 4;
  s.count = static_cast<uint64_t>(p->count);
  s.arena_count = static_cast<uint64_t>(p->arena);
  s.workspace_bytes = p->table_bytes() + p->sum_bytes();
  return s;
}

ar_status_t ar_grad_norm(ar_norm_plan_t *p, const void *grads, double scale, float *norm, float *tensor_norms,
                         void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "norm plan is NULL");
  return guarded([&]() -> ar_status_t {
    const uintptr_t elem = p->bf16 ? 2 : 4;
    if (!std::isfinite(scale) || scale < 0) return fail(AR_ERR_INVALID_ARG, "scale must be finite and not negative");
    ar_status_t st = check_pointer(norm, 4, "norm");
    if (st == AR_OK && p->arena > 0) st = check_pointer(grads, elem, "grads");
    if (st == AR_OK && tensor_norms) st = check_pointer(tensor_norms, 4, "tensor_norms");
    if (st == AR_OK)
      st = check_apart({{norm, 4, "norm"}, {tensor_norms, tensor_norms ? 4 * static_cast<int64_t>(p->ntensors) : 0, "tensor_norms"}},
                       {{grads, p->arena * static_cast<int64_t>(elem), "grads"}});
    if (st == AR_OK) st = prepare_for(p, stream);
    if (st != AR_OK) return st;
    ar_dev::NormArgs a = norm_args(p);
    a.g = grads;
    a.scale = scale;
    a.norm = norm;
    a.tensor_norms = tensor_norms;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return run_marked(p->marks, s, "gradient norm", [&] { return ar_dev::grad_norm(a, s); });
  });
}

ar_status_t ar_grad_clip(ar_norm_plan_t *p, const void *grads, void *grads_out, const float *norm, double max_norm,
                         void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "norm plan is NULL");
  return guarded([&]() -> ar_status_t {
    const uintptr_t elem = p->bf16 ? 2 : 4;
    void *out = grads_out ? grads_out : const_cast<void *>(grads);
    const float most = static_cast<float>(max_norm);
    if (!std::isfinite(most) || !(most > 0)) return fail(AR_ERR_INVALID_ARG, "max_norm must be a finite fp32 number above zero");
    ar_status_t st = check_pointer(norm, 4, "norm");
    if (st == AR_OK && p->arena > 0) st = check_pointer(grads, elem, "grads");
    if (st == AR_OK && p->arena > 0) st = check_pointer(out, elem, "grads_out");
    const int64_t bytes = p->arena * static_cast<int64_t>(elem);
    if (st == AR_OK) {
      std::vector<std::pair<int, int>> may;
      if (out == grads) may.push_back({0, 0});
      st = check_apart({{out, bytes, "grads_out"}}, {{grads, bytes, "grads"}, {norm, 4, "norm"}}, may);
    }
    if (st == AR_OK) st = prepare_for(p, stream);
    if (st != AR_OK || p->chunks.empty()) return st;
    ar_dev::NormArgs a = norm_args(p);
    a.g = grads;
    a.out = out;
    a.norm = const_cast<float *>(norm);
    a.max_norm = max_norm;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return run_marked(p->marks, s, "gradient clipping", [&] { return ar_dev::grad_clip(a, s); });
  });
}

void ar_norm_plan_destroy(ar_norm_plan_t *p) {
  if (!p) return;
  p->release();
  delete p;
}

ar_status_t ar_quantize_rows(const void *x, ar_dtype_t dtype, size_t x_stride, void *codes, size_t codes_stride,
                             void *scales, size_t scales_stride, size_t features, size_t ntokens, void *stream) {
  return guarded([&]() -> ar_status_t {
    const int32_t d = raw_enum(dtype);
    if (!float_type(d)) return fail(AR_ERR_INVALID_ARG, "rows to quantise are AR_FLOAT32 or AR_BFLOAT16");
    if (features < 1 || features > kMaxFeatures) return fail(AR_ERR_INVALID_ARG, "features must be from 1 to 2^22");
    if (ntokens > kMaxTokens) return fail(AR_ERR_INVALID_ARG, "more than 2^31 - 65536 tokens");
    const int64_t t = static_cast<int64_t>(ntokens), f = static_cast<int64_t>(features), b = blocks_of(f);
    int64_t bx = 0, bc = 0, bs = 0;
    ar_status_t st = check_rows({x, x_stride, f, "x"}, t, d == AR_BFLOAT16 ? 2 : 4, &bx);
    if (st == AR_OK) st = check_rows({codes, codes_stride, f, "codes"}, t, 1, &bc);
    if (st == AR_OK) st = check_rows({scales, scales_stride, b, "scales"}, t, 1, &bs);
    if (st == AR_OK) st = check_apart({{codes, bc, "codes"}, {scales, bs, "scales"}}, {{x, bx, "x"}});
    if (st != AR_OK || t == 0) return st;
    ar_dev::QuantArgs a{};
    a.x = x;
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = static_cast<uint8_t *>(scales);
    a.features = f;
    a.tokens = t;
    a.xs = static_cast<int64_t>(x_stride);
    a.cs = static_cast<int64_t>(codes_stride);
    a.ss = static_cast<int64_t>(scales_stride);
    a.bf16 = d == AR_BFLOAT16;
    const hipError_t e = ar_dev::quantize_rows(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? AR_OK : hip_fail(e, "kernel launch");
  });
}

ar_rmsnorm_t *ar_rmsnorm_create(size_t features, ar_dtype_t dtype, ar_dtype_t gain_dtype, ar_dtype_t grad_dtype,
                                double eps) {
  ar_rmsnorm *p = nullptr;
  const ar_status_t st = guarded([&]() -> ar_status_t {
    const int32_t d = raw_enum(dtype), w = raw_enum(gain_dtype), g = raw_enum(grad_dtype);
    if (features < 1 || features > 65536) return fail(AR_ERR_INVALID_ARG, "features must be from 1 to 65536");
    if (!float_type(d) || !float_type(w) || !float_type(g))
      return fail(AR_ERR_INVALID_ARG, "RMS norms take AR_FLOAT32 or AR_BFLOAT16");
    if (!std::isfinite(eps) || !(eps >= 1e-75))  // 1 / sqrt(eps) is an fp32 number
      return fail(AR_ERR_INVALID_ARG, "eps must be finite and at least 1e-75");
    p = new ar_rmsnorm;
    p->features = static_cast<int64_t>(features);
    p->bf16 = d == AR_BFLOAT16;
    p->gain_bf16 = w == AR_BFLOAT16;
    p->grad_bf16 = g == AR_BFLOAT16;
    p->eps = eps;
    p->parts = ar_dev::rmsnorm_parts(p->features, p->bf16);
    return AR_OK;
  });
  return st == AR_OK ? p : nullptr;
}

ar_status_t ar_rmsnorm_prepare(ar_rmsnorm_t *p) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "RMS norm plan is NULL");
  return guarded([&] { return p->prepare(); });
}

ar_rmsnorm_stats_t ar_rmsnorm_stats(const ar_rmsnorm_t *p) {
  ar_rmsnorm_stats_t s{};
  if (!p) {
    fail(AR_ERR_INVALID_ARG, "RMS norm plan is NULL");
    return s;
  }
  s.device = p->device;
  s.features = static_cast<uint64_t>(p->features);
  s.elem_bytes = static_cast<uint64_t>(p->elem());
  s.gain_bytes = p->gain_bf16 ? 2 : 4;
  s.grad_bytes = p->grad_bf16 ? 2 : 4;
  s.workspace_bytes = p->part_bytes();
  return s;
}

ar_status_t ar_rmsnorm_forward(ar_rmsnorm_t *p, const ar_rmsnorm_forward_t *args, size_t ntokens, void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "RMS norm plan is NULL");
  if (!args) return fail(AR_ERR_INVALID_ARG, "args is NULL");
  return guarded([&] { return forward(p, *args, ntokens, stream); });
}

ar_status_t ar_rmsnorm_backward(ar_rmsnorm_t *p, const ar_rmsnorm_backward_t *args, size_t ntokens, void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "RMS norm plan is NULL");
  if (!args) return fail(AR_ERR_INVALID_ARG, "args is NULL");
  return guarded([&] { return backward(p, *args, ntokens, stream); });
}

void ar_rmsnorm_destroy(ar_rmsnorm_t *p) {
  if (!p) return;
  p->release();
  delete p;
}

ar_qexperts_t *ar_qexperts_create(int nexperts, size_t in_features, size_t out_features, ar_dtype_t dtype,
                                  const size_t *weight_offsets) {
  ar_qexperts *p = nullptr;
  const ar_status_t st = guarded([&]() -> ar_status_t {
    const int32_t d = raw_enum(dtype);
    if (nexperts < 1 || nexperts > 65536) return fail(AR_ERR_INVALID_ARG, "nexperts must be from 1 to 65536");
    if (in_features < 1 || out_features < 1 || in_features > kMaxFeatures || out_features > kMaxFeatures)
      return fail(AR_ERR_INVALID_ARG, "features must be from 1 to 2^22");
    if (!float_type(d)) return fail(AR_ERR_INVALID_ARG, "8-bit expert products give AR_FLOAT32 or AR_BFLOAT16");
    p = new ar_qexperts;
    p->nexperts = nexperts;
    p->in = static_cast<int64_t>(in_features);
    p->out = static_cast<int64_t>(out_features);
    p->bf16 = d == AR_BFLOAT16;
    const int64_t size = p->in * p->out;
    for (int e = 0; e < nexperts; ++e) {
      if (weight_offsets && weight_offsets[e] > static_cast<size_t>(INT64_MAX / 16))
        return fail(AR_ERR_INVALID_ARG, "weight offset of expert " + std::to_string(e) + " is too large");
      const int64_t at = weight_offsets ? static_cast<int64_t>(weight_offsets[e]) : e * size;
      p->offsets.push_back(at);
      p->arena = std::max(p->arena, at + size);
      p->offsets_by_16 = p->offsets_by_16 && at % 16 == 0;
    }
    std::vector<int64_t> sorted = p->offsets;
    std::sort(sorted.begin(), sorted.end());
    for (int e = 1; e < nexperts; ++e)
      if (sorted[e] - sorted[e - 1] < size) return fail(AR_ERR_INVALID_ARG, "the experts' matrices overlap");
    return AR_OK;
  });
  if (st != AR_OK) {
    delete p;
    return nullptr;
  }
  return p;
}

ar_status_t ar_qexperts_prepare(ar_qexperts_t *p) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "8-bit expert plan is NULL");
  return guarded([&] { return p->prepare(); });
}

ar_qexperts_stats_t ar_qexperts_stats(const ar_qexperts_t *p) {
  ar_qexperts_stats_t s{};
  if (!p) {
    fail(AR_ERR_INVALID_ARG, "8-bit expert plan is NULL");
    return s;
  }
  s.nexperts = p->nexperts;
  s.device = p->device;
  s.in_features = static_cast<uint64_t>(p->in);
  s.out_features = static_cast<uint64_t>(p->out);
  s.elem_bytes = p->bf16 ? 2 : 4;
  s.arena_count = static_cast<uint64_t>(p->arena);
  s.scale_count = static_cast<uint64_t>(p->scale_count());
  s.workspace_bytes = p->offsets.size() * sizeof(int64_t);
  return s;
}

ar_status_t ar_qexperts_launch_shape(const ar_qexperts_t *p, int product, size_t ntokens, int aligned,
                                     int32_t *tile_rows, int32_t *tile_cols) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "8-bit expert plan is NULL");
  if (product < ar_dev::kExpertsForward || product > ar_dev::kExpertsInputGrad)
    return fail(AR_ERR_INVALID_ARG, "product must be 0 or 1");
  if (ntokens > kMaxTokens) return fail(AR_ERR_INVALID_ARG, "more than 2^31 - 65536 tokens");
  ar_dev::ExpertShape s{0, 0, 0};
  if (ntokens > 0) {
    ar_dev::QExpertArgs a = call_args(p, static_cast<int64_t>(ntokens));
    a.aligned = a.aligned && aligned;
    s = ar_dev::qexperts_shape(a, static_cast<ar_dev::ExpertProduct>(product));
  }
  if (tile_rows) *tile_rows = s.rows;
  if (tile_cols) *tile_cols = s.cols;
  return AR_OK;
}

ar_status_t ar_qexperts_quantize(ar_qexperts_t *p, const void *weights, ar_dtype_t weight_dtype, void *codes,
                                 void *scales, void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "8-bit expert plan is NULL");
  return guarded([&]() -> ar_status_t {
    const int32_t d = raw_enum(weight_dtype);
    if (!float_type(d)) return fail(AR_ERR_INVALID_ARG, "weights to quantise are AR_FLOAT32 or AR_BFLOAT16");
    const int64_t elem = d == AR_BFLOAT16 ? 2 : 4;
    ar_status_t st = check_pointer(weights, static_cast<uintptr_t>(elem), "the weight arena");
    if (st == AR_OK) st = check_pointer(codes, 1, "codes");
    if (st == AR_OK) st = check_pointer(scales, 1, "scales");
    if (st == AR_OK)
      st = check_apart({{codes, p->arena, "codes"}, {scales, p->scale_count(), "scales"}},
                       {{weights, p->arena * elem, "the weight arena"}});
    if (st == AR_OK) st = prepare_for(p, stream);
    if (st != AR_OK) return st;
    ar_dev::QWeightArgs a{};
    a.w = weights;
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = static_cast<uint8_t *>(scales);
    a.offsets = static_cast<const int64_t *>(p->d_offsets);
    a.in = p->in;
    a.outf = p->out;
    a.experts = p->nexperts;
    a.bf16 = d == AR_BFLOAT16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return run_marked(p->marks, s, "quantisation", [&] { return ar_dev::qexperts_quantize(a, s); });
  });
}

ar_status_t ar_qexperts_forward(ar_qexperts_t *p, const void *x, size_t x_stride, const void *x_scales,
                                size_t x_scales_stride, const void *weights, const void *weight_scales, void *y,
                                size_t y_stride, const int32_t *ends, size_t ntokens, void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "8-bit expert plan is NULL");
  return guarded([&] {
    return product(p, false, {x, x_stride, p->in, "x"}, {x_scales, x_scales_stride, blocks_of(p->in), "x_scales"}, weights,
                   weight_scales, {y, y_stride, p->out, "y"}, ends, ntokens, stream);
  });
}

ar_status_t ar_qexperts_input_grad(ar_qexperts_t *p, const void *dy, size_t dy_stride, const void *dy_scales,
                                   size_t dy_scales_stride, const void *weights, const void *weight_scales, void *dx,
                                   size_t dx_stride, const int32_t *ends, size_t ntokens, void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "8-bit expert plan is NULL");
  return guarded([&] {
    return product(p, true, {dy, dy_stride, p->out, "dy"}, {dy_scales, dy_scales_stride, blocks_of(p->out), "dy_scales"},
                   weights, weight_scales, {dx, dx_stride, p->in, "dx"}, ends, ntokens, stream);
  });
}

void ar_qexperts_destroy(ar_qexperts_t *p) {
  if (!p) return;
  p->release();
  delete p;
}

}  // extern "C"

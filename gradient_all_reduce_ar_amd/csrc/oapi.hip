// oapi.hip -- C ABI (include/ar.h) of the expert products and of the Muon
// update: argument checks, the plans' device tables, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <string>
#include <vector>

#include "../../include/ar.h"
#include "host.hpp"
#include "kernels.hpp"
#include "operators.hpp"

using ar_host::fail;
using ar_host::hip_fail;
using ar_host::raw_enum;

namespace ar_host {

ar_status_t CallMarks::of(hipStream_t s, hipEvent_t *ev) {
  *ev = nullptr;
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  hipError_t e = hipStreamIsCapturing(s, &cs);
  if (e != hipSuccess) return hip_fail(e, "hipStreamIsCapturing");
  if (cs != hipStreamCaptureStatusNone) return AR_OK;
  for (const Mark &m : marks_)
    if (m.stream == s) {
      *ev = m.event;
      return AR_OK;
    }
  if (marks_.size() >= kMax) {  // retire the oldest stream's mark
    (void)hipEventSynchronize(marks_.front().event);
    (void)hipEventDestroy(marks_.front().event);
    marks_.erase(marks_.begin());
  }
  marks_.reserve(kMax);
  e = hipEventCreate(ev);  // with timing: a dispatch can record it
  if (e != hipSuccess) {
    *ev = nullptr;
    return hip_fail(e, "hipEventCreate");
  }
  marks_.push_back({s, *ev});
  return AR_OK;
}

void CallMarks::wait() const {
  for (const Mark &m : marks_) (void)hipEventSynchronize(m.event);
}

void CallMarks::release() {
  wait();
  for (const Mark &m : marks_) (void)hipEventDestroy(m.event);
  marks_.clear();
}

ar_status_t refuse_capture(hipStream_t s) {
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  const hipError_t e = hipStreamIsCapturing(s, &cs);
  if (e != hipSuccess) return hip_fail(e, "hipStreamIsCapturing");
  return cs == hipStreamCaptureStatusNone ? AR_OK
                                          : fail(AR_ERR_INVALID_ARG, "the plan has to be prepared before it is captured");
}

hipError_t upload(void *dst, const void *src, size_t bytes) {
  // a non-blocking stream and an event: a synchronous copy would go through
  // the default stream, which ends a capture that another thread has open
  hipStream_t s = nullptr;
  hipEvent_t done = nullptr;
  hipError_t e = hipStreamCreateWithFlags(&s, hipStreamNonBlocking);
  if (e == hipSuccess) e = hipEventCreateWithFlags(&done, hipEventDisableTiming);
  if (e == hipSuccess) e = hipMemcpyAsync(dst, src, bytes, hipMemcpyHostToDevice, s);
  if (e == hipSuccess) e = hipEventRecord(done, s);
  if (e == hipSuccess) e = hipEventSynchronize(done);
  if (done) (void)hipEventDestroy(done);
  if (s) (void)hipStreamDestroy(s);
  return e;
}

hipError_t device_table(void **dst, const void *src, size_t bytes) {
  hipError_t e = hipMalloc(dst, bytes);
  if (e != hipSuccess) {
    (void)hipGetLastError();  // clear the sticky allocation error
    *dst = nullptr;
    return e;
  }
  if (!src) return hipSuccess;
  e = upload(*dst, src, bytes);
  if (e != hipSuccess) {
    (void)hipFree(*dst);
    *dst = nullptr;
  }
  return e;
}

}  // namespace ar_host

struct ar_experts {
  int32_t nexperts = 0;
  int64_t in = 0, out = 0;
  bool bf16 = false, grad_bf16 = false;
  std::vector<int64_t> offsets;
  int64_t arena = 0;         // elements an arena holds at least
  bool offsets_by_8 = true;  // every matrix starts on a multiple of 8 elements
  int device = -1;
  void *d_offsets = nullptr;
  size_t slot_bytes = 0;     // partial tiles of split weight gradients
  void *d_slots = nullptr;
  ar_host::CallMarks marks;

  void release() {
    marks.release();
    for (void **p : {&d_offsets, &d_slots}) {
      if (*p) (void)hipFree(*p);
      *p = nullptr;
    }
    device = -1;
  }
};

namespace {

constexpr int64_t kMaxFeatures = 1 << 22, kMaxStride = 1 << 22;
// rows are counted in int32, rounded up to whole tiles and parts
constexpr size_t kMaxTokens = (size_t{1} << 31) - 65536;

// [p, p + n) and [q, q + m) share a byte.
bool overlap(const void *p, int64_t n, const void *q, int64_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return n > 0 && m > 0 && a < b + static_cast<uint64_t>(m) && b < a + static_cast<uint64_t>(n);
}

bool on(const void *p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

ar_status_t prepare(ar_experts *ex) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (ex->d_offsets) {
    if (dev != ex->device) return fail(AR_ERR_INVALID_ARG, "expert plan was prepared on another device");
    return AR_OK;
  }
  e = ar_host::device_table(&ex->d_offsets, ex->offsets.data(), ex->offsets.size() * sizeof(int64_t));
  if (e == hipSuccess && ex->slot_bytes > 0) e = ar_host::device_table(&ex->d_slots, nullptr, ex->slot_bytes);
  if (e != hipSuccess) {
    ex->release();
    return e == hipErrorOutOfMemory ? fail(AR_ERR_OOM, "expert workspace allocation") : hip_fail(e, "expert tables");
  }
  ex->device = dev;
  return AR_OK;
}

// A matrix of `rows` rows of `features` elements, `stride` apart.
struct RowsArg {
  const void *p;
  size_t stride;
  int64_t features;
  const char *name;
};

ar_status_t check_rows(const RowsArg &r, int64_t rows, int64_t elem, int64_t *bytes) {
  *bytes = 0;
  if (r.stride < static_cast<size_t>(r.features) || r.stride > static_cast<size_t>(kMaxStride))
    return fail(AR_ERR_INVALID_ARG, std::string(r.name) + ": row stride must be from its features to 2^22");
  if (rows == 0) return AR_OK;
  if (!r.p) return fail(AR_ERR_INVALID_ARG, std::string(r.name) + " is NULL");
  if (!on(r.p, elem)) return fail(AR_ERR_INVALID_ARG, std::string(r.name) + " is not aligned to its elements");
  *bytes = ((rows - 1) * static_cast<int64_t>(r.stride) + r.features) * elem;
  return AR_OK;
}

using ar_dev::ExpertProduct;
using ar_dev::kExpertsForward;
using ar_dev::kExpertsInputGrad;
using ar_dev::kExpertsWeightGrad;

// What every call of a plan has, and whether its rows and (in the products
// that read the weights) matrices let it read 16 bytes at a time if all
// pointers and strides do: 16-byte rows; and offsets inside a tile of 256 rows
// fit into 31 bits.
size_t far_stride(const ar_experts *ex) { return (size_t{1} << 23) / (ex->bf16 ? 2 : 4); }
ar_dev::ExpertArgs call_args(const ar_experts *ex, ExpertProduct which, int64_t tokens) {
  ar_dev::ExpertArgs a{};
  a.tokens = tokens;
  a.in = ex->in;
  a.outf = ex->out;
  a.experts = ex->nexperts;
  a.bf16 = ex->bf16;
  a.grad_bf16 = ex->grad_bf16;
  const int64_t vec = ex->bf16 ? 8 : 4;
  a.aligned = ex->in % vec == 0 && ex->out % vec == 0 && static_cast<size_t>(ex->in) <= far_stride(ex) &&
              (which == kExpertsWeightGrad || ex->offsets_by_8);
  return a;
}

ar_status_t run(ar_experts *ex, ExpertProduct which, const RowsArg &r1, const RowsArg &r2, const void *arena, bool out_is_rows,
                bool accumulate, const int32_t *ends, size_t ntokens, void *stream) {
  if (ntokens > kMaxTokens) return fail(AR_ERR_INVALID_ARG, "more than 2^31 - 65536 tokens");
  const int64_t t = static_cast<int64_t>(ntokens), elem = ex->bf16 ? 2 : 4;
  int64_t b1 = 0, b2 = 0;
  ar_status_t st = check_rows(r1, t, elem, &b1);
  if (st == AR_OK) st = check_rows(r2, t, elem, &b2);
  if (st != AR_OK) return st;
  const int64_t aelem = which == kExpertsWeightGrad ? (ex->grad_bf16 ? 2 : 4) : elem;
  if (t > 0 || which == kExpertsWeightGrad) {
    if (!ends) return fail(AR_ERR_INVALID_ARG, "ends is NULL");
    if (!on(ends, 4)) return fail(AR_ERR_INVALID_ARG, "ends is not aligned to its elements");
    if (!arena) return fail(AR_ERR_INVALID_ARG, "the weight arena is NULL");
    if (!on(arena, aelem)) return fail(AR_ERR_INVALID_ARG, "the weight arena is not aligned to its elements");
  }
  const int64_t ab = ex->arena * aelem, eb = 4 * static_cast<int64_t>(ex->nexperts);
  if (out_is_rows ? overlap(r2.p, b2, r1.p, b1) || overlap(r2.p, b2, arena, ab) || overlap(r2.p, b2, ends, eb)
                  : overlap(arena, ab, r1.p, b1) || overlap(arena, ab, r2.p, b2) || overlap(arena, ab, ends, eb))
    return fail(AR_ERR_INVALID_ARG, "the output overlaps an input");
  if (!ex->d_offsets) st = ar_host::refuse_capture(static_cast<hipStream_t>(stream));
  if (st == AR_OK) st = prepare(ex);
  if (st != AR_OK) return st;
  if (t == 0 && which != kExpertsWeightGrad) return AR_OK;
  ar_dev::ExpertArgs a = call_args(ex, which, t);
  a.offsets = static_cast<const int64_t *>(ex->d_offsets);
  a.slots = static_cast<float *>(ex->d_slots);
  a.ends = ends;
  a.accumulate = accumulate;
  const size_t vec = static_cast<size_t>(16 / elem), far = far_stride(ex);
  auto rows16 = [&](const RowsArg &r) { return on(r.p, 16) && r.stride % vec == 0 && r.stride <= far; };
  if (which == kExpertsWeightGrad) {
    a.x = r1.p;
    a.xs = static_cast<int64_t>(r1.stride);
    a.dy = r2.p;
    a.dys = static_cast<int64_t>(r2.stride);
    a.out = const_cast<void *>(arena);
    a.aligned = a.aligned && rows16(r1) && rows16(r2);
  } else {
    a.w = arena;
    a.out = const_cast<void *>(r2.p);
    a.outs = static_cast<int64_t>(r2.stride);
    (which == kExpertsForward ? a.x : a.dy) = r1.p;
    (which == kExpertsForward ? a.xs : a.dys) = static_cast<int64_t>(r1.stride);
    a.aligned = a.aligned && rows16(r1) && on(arena, 16);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipEvent_t mark = nullptr;
  st = ex->marks.of(s, &mark);
  if (st != AR_OK) return st;
  ar_dev::t_launch_events = ar_dev::LaunchEvents{nullptr, mark};
  const hipError_t e = which == kExpertsForward     ? ar_dev::experts_forward(a, s)
                       : which == kExpertsInputGrad ? ar_dev::experts_input_grad(a, s)
                                                    : ar_dev::experts_weight_grad(a, s);
  ar_dev::t_launch_events = ar_dev::LaunchEvents{};
  if (e == hipErrorInvalidConfiguration)
    return fail(AR_ERR_UNSUPPORTED, "expert product larger than one launch grid");
  return e == hipSuccess ? AR_OK : hip_fail(e, "kernel launch");
}

// Runs f, turning a failed host allocation into a status.
template <class F>
ar_status_t guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc &) {
    return fail(AR_ERR_OOM, "host allocation failed");
  }
}

bool float_type(int32_t d) { return d == AR_FLOAT32 || d == AR_BFLOAT16; }

}  // namespace

struct ar_muon_plan {
  bool g_bf16 = false, w_bf16 = false;
  int32_t nmatrices = 0;
  std::vector<ar_dev::MuonMat> mats;  // those with elements; scale from scales
  std::vector<int32_t> index;         // their numbers
  int64_t arena = 0;                  // elements an arena holds at least
  std::vector<ar_dev::MuonStep> steps;
  int32_t ex0 = 0;
  int32_t small_lds = 0;  // > 0: one launch, a workgroup per matrix (muon_small)
  bool tiny = true;       // then: every matrix is up to 64 x 64
  // Work lists.  table holds them all for the device, one after another (see
  // fill_table): the offsets are in bytes.
  std::vector<ar_dev::MuonTile> parts, blocks;
  struct Work {
    std::vector<ar_dev::MuonItem> items;
    std::vector<int32_t> first;
    std::vector<ar_dev::MuonJoin> joins;
    int32_t shape = 0;
    size_t at_items = 0, at_first = 0, at_joins = 0;
  } gram, poly, mul;
  std::vector<char> table;
  size_t at_parts = 0, at_blocks = 0;
  // workspace: sums of squares, shifts, partial tiles, then X, A and B
  size_t partial_bytes = 0, shift_bytes = 0, slot_bytes = 0, ws_bytes = 0;
  size_t work_bytes() const { return partial_bytes + shift_bytes + slot_bytes + ws_bytes; }
  int device = -1;
  void *d_table = nullptr, *d_work = nullptr;
  ar_host::CallMarks marks;

  void release() {
    marks.release();
    for (void **p : {&d_table, &d_work}) {
      if (*p) (void)hipFree(*p);
      *p = nullptr;
    }
    device = -1;
  }
};

namespace {

using ar_dev::MuonMat;
using ar_dev::MuonStep;
using ar_dev::MuonTile;

constexpr double kNsA = 3.4445, kNsB = -4.7750, kNsC = 2.0315;
constexpr int kNsSteps = 5;

// The largest |f| of f(t) = a + b t + c t^2 over [0, s].
double quad_bound(double a, double b, double c, double s) {
  double m = std::max(std::fabs(a), std::fabs(a + b * s + c * s * s));
  if (c != 0) {
    const double t = -b / (2 * c);
    if (t > 0 && t < s) m = std::max(m, std::fabs(a + b * t + c * t * t));
  }
  return m;
}

// The largest |sigma f(sigma^2)| over [0, s].
double step_bound(double a, double b, double c, double s) {
  auto p = [&](double x) { return std::fabs(x * (a + x * x * (b + x * x * c))); };
  double m = p(s);
  // extremes: a + 3 b t + 5 c t^2 = 0 in t = sigma^2
  double roots[2];
  int n = 0;
  if (c == 0) {
    if (b != 0) roots[n++] = -a / (3 * b);
  } else {
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
      roots[n++] = (-3 * b + std::sqrt(d)) / (10 * c);
      roots[n++] = (-3 * b - std::sqrt(d)) / (10 * c);
    }
  }
  for (int i = 0; i < n; ++i)
    if (roots[i] > 0 && roots[i] < s * s) m = std::max(m, p(std::sqrt(roots[i])));
  return m;
}

// The power of two that takes a number of at most `bound` (and 1/16 more, for
// what rounding adds) to at most 2^15.
constexpr double kLeast = 1e-6;  // smaller bounds are taken for this
int32_t scale_exp(double bound) { return 15 - static_cast<int32_t>(std::ceil(std::log2(std::max(bound, kLeast) * 1.0625))); }

// The steps' factors; false where a bound is passed.
bool make_steps(int n, const double *abc, std::vector<MuonStep> &steps, int32_t &ex0) {
  steps.clear();
  double s = 1;  // largest singular value; X_0's Frobenius norm is at most 1
  ex0 = scale_exp(s);
  for (int i = 0; i < n; ++i) {
    const double a = abc ? abc[3 * i] : kNsA, b = abc ? abc[3 * i + 1] : kNsB, c = abc ? abc[3 * i + 2] : kNsC;
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    MuonStep k{};
    k.coef_a = static_cast<float>(a);
    k.coef_b = static_cast<float>(b);
    k.coef_c = static_cast<float>(c);
    k.ex = scale_exp(s);
    k.ea = scale_exp(s * s);
    const double q = quad_bound(a, b, c, s * s);
    const double next = step_bound(a, b, c, s);
    // the terms of B are formed before they are added
    const double terms = std::fabs(a) + std::fabs(b) * s * s + std::fabs(c) * s * s * s * s;
    if (!(terms <= 1 << 14) || !(next <= 1 << 10)) return false;
    k.eb = scale_exp(q);
    // |B X| <= q |X|, which is below `next` too once d is zero
    k.drop = static_cast<int32_t>(std::ceil(std::log2(std::max(1.0, q * s / std::max(next, kLeast)))));
    s = std::max(next, kLeast);
    k.ex_next = scale_exp(s);
    k.index = i;
    k.last = i + 1 == n;
    k.from = i & 1;
    steps.push_back(k);
  }
  return true;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// One product over all matrices: a tile's row, column and contraction steps
// (of kStep elements).
constexpr int kStep = 64;
struct Tile {
  int32_t mat, m, n, steps;
};

// Tile shapes: workgroups that run at once, and the microseconds of a tile's
// contraction step where every CU has one workgroup at most (`alone`, a launch
// of up to 256 tiles) and where the launch is full, of the rest of a tile's
// work, and of that which a square product adds (`mirror`: its tiles leave
// twice).  Measured with the three shapes: the product with X of
// 512 x 2048 (alone) 37, 21 and 12 us, of 12288 x 4096 (full) 891, 1123 and
// 2022; X X^T of 512 x 2048 65 and 33 with the smaller two, of eight matrices
// of 1024 x 1024 and 1024 x 2048 84 (split) and 107 with the largest and the
// smallest.
struct ShapeCost {
  int32_t slots;
  double alone, full, rest, mirror;
};
constexpr ShapeCost kCost[ar_dev::kMuonShapes] = {
    {256, 1.15, 1.48, 12.0, 17.0}, {512, 0.6, 0.97, 5.0, 8.0}, {512, 0.31, 0.6, 3.5, 1.5}};
// A split launch also writes and reads its partial tiles (256 KiB each; 5.5
// TB/s, 402 pieces of a 4096 x 4096 and a 1024 x 4096 matrix 42 us with the
// launch) and launches the join.
constexpr double kJoinLaunch = 6.0, kJoinSlot = 2 * 262144 / 5.5e6;
constexpr int32_t kMinPiece = 4;  // steps of a piece at least
constexpr int kPairs = 3;         // planes' products of a step (TileProduct)

// The time until the last tile is done if each goes, in order, to the
// workgroup with the least to do.
double list_time(const std::vector<Tile> &tiles, const ShapeCost &c, double rest) {
  std::vector<double> heap(c.slots, 0.0);  // the least on top
  const auto more = [](double x, double y) { return x > y; };
  const double step = kPairs * (tiles.size() <= 256 ? c.alone : c.full);
  double last = 0;
  for (const Tile &t : tiles) {
    std::pop_heap(heap.begin(), heap.end(), more);
    heap.back() += t.steps * step + rest;
    last = std::max(last, heap.back());
    std::push_heap(heap.begin(), heap.end(), more);
  }
  return last;
}

// Splits a launch of the largest tiles over its workgroups: each gets whole
// tiles while they fit into an equal share of the steps; the other tiles are
// cut along the contraction to fill what is left of the shares.  Returns the
// time until the joined tiles are out.
double split_tiles(const std::vector<Tile> &tiles, const ShapeCost &c, double rest_time, ar_muon_plan::Work &w) {
  const int32_t groups = c.slots;
  int64_t total = 0;
  for (const Tile &t : tiles) total += t.steps;
  const int64_t share = (total + groups - 1) / groups + kMinPiece;
  std::vector<std::vector<ar_dev::MuonItem>> of(groups);
  std::vector<std::pair<int64_t, int32_t>> heap;  // (steps, workgroup), the least on top
  for (int32_t g = 0; g < groups; ++g) heap.push_back({0, g});
  const auto more = [](const auto &x, const auto &y) { return x > y; };
  std::make_heap(heap.begin(), heap.end(), more);
  std::vector<Tile> rest;
  for (const Tile &t : tiles) {
    if (heap.front().first + t.steps > share) {
      rest.push_back(t);
      continue;
    }
    std::pop_heap(heap.begin(), heap.end(), more);
    heap.back().first += t.steps;
    of[heap.back().second].push_back({t.mat, t.m, t.n, 0, t.steps * kStep, -1});
    std::push_heap(heap.begin(), heap.end(), more);
  }
  // The first piece of each tile starts at the contraction's beginning, so
  // that the workgroups that do these read the same columns of the operands
  // at the same time; what is left of the tiles is dealt out in order.
  struct Piece {
    int32_t group, k0, k1;
  };
  std::vector<std::vector<Piece>> pieces(rest.size());
  std::vector<int64_t> left(groups);
  for (const auto &h : heap) left[h.second] = share - h.first;
  std::vector<int32_t> room;
  for (int32_t g = 0; g < groups; ++g)
    if (left[g] >= kMinPiece) room.push_back(g);
  auto give = [&](size_t i, int32_t g, int32_t from, int64_t n) {
    const int32_t all = rest[i].steps;
    if (all - from - n < kMinPiece) n = all - from;
    pieces[i].push_back({g, from, static_cast<int32_t>(from + n)});
    left[g] -= n;
    return static_cast<int32_t>(from + n);
  };
  std::vector<int32_t> done(rest.size(), 0);
  for (size_t i = 0; i < rest.size() && i < room.size(); ++i)
    done[i] = give(i, room[i], 0, std::min<int64_t>(rest[i].steps, left[room[i]]));
  int32_t g = 0;
  for (size_t i = 0; i < rest.size(); ++i)
    while (done[i] < rest[i].steps) {
      while (g + 1 < groups && left[g] < kMinPiece) ++g;
      const int64_t need = rest[i].steps - done[i];
      done[i] = give(i, g, done[i], g + 1 == groups ? need : std::min(need, left[g]));
    }
  int32_t slot = 0;
  for (size_t i = 0; i < rest.size(); ++i) {
    const Tile &t = rest[i];
    const int32_t n = static_cast<int32_t>(pieces[i].size());
    if (n > 1) w.joins.push_back({t.mat, t.m, t.n, slot, n});
    for (const Piece &x : pieces[i])
      of[x.group].push_back({t.mat, t.m, t.n, x.k0 * kStep, x.k1 * kStep, n > 1 ? slot++ : -1});
  }
  double last = 0;
  for (const auto &items : of) {
    double time = 0;
    for (const ar_dev::MuonItem &x : items)
      time += (x.k1 - x.k0) / kStep * (kPairs * c.full) + (x.slot >= 0 ? c.rest : rest_time);
    last = std::max(last, time);
  }
  // workgroup b runs on XCD b % 8: neighbouring shares go to one XCD, whose
  // L2 then holds the operands that their tiles share
  for (int32_t b = 0; b < groups; ++b) {
    const int32_t s = groups % 8 ? b : b % 8 * (groups / 8) + b / 8;
    w.first.push_back(static_cast<int32_t>(w.items.size()));
    w.items.insert(w.items.end(), of[s].begin(), of[s].end());
  }
  w.first.push_back(static_cast<int32_t>(w.items.size()));
  return last + (slot > 0 ? kJoinLaunch + slot * kJoinSlot : 0);
}

// Chooses the tile shape, whole or split, with the least modelled time, and
// makes the launch's lists.
template <class List>
void plan_product(List list, bool sym, ar_muon_plan::Work &w) {
  double best = 0;
  bool split = false;
  std::vector<Tile> tiles;
  for (int i = 0; i < ar_dev::kMuonShapes; ++i) {
    std::vector<Tile> t = list(ar_dev::muon_tile(i));
    const ShapeCost &c = kCost[i];
    const double rest = c.rest + (sym ? c.mirror : 0), whole = list_time(t, c, rest);
    if (i == 0) {
      ar_muon_plan::Work cut;
      const double even = split_tiles(t, c, rest, cut);
      if (even < whole) {
        best = even;
        split = true;
        w = std::move(cut);
        continue;
      }
    }
    if (i == 0 || whole < best) {
      best = whole;
      split = false;
      w = ar_muon_plan::Work{};
      w.shape = i;
      tiles = std::move(t);
    }
  }
  if (split) return;
  // one workgroup per tile, neighbours on one XCD
  const int32_t n = static_cast<int32_t>(tiles.size()), q = n / 8, r = n % 8;
  for (int32_t b = 0; b < n; ++b) {
    const int32_t x = b % 8;
    const Tile &t = tiles[x * q + std::min(x, r) + b / 8];
    w.first.push_back(b);
    w.items.push_back({t.mat, t.m, t.n, 0, t.steps * kStep, -1});
  }
  w.first.push_back(n);
}

// Work lists and workspace layout.
void lay_out(ar_muon_plan *p) {
  int64_t lds = 0;
  for (const MuonMat &m : p->mats) {
    const int64_t n = ar_dev::muon_small_lds(m.m, m.n);
    if (n == 0) lds = INT64_MAX;
    lds = std::max(lds, n);
    p->tiny = p->tiny && m.n <= 64;
  }
  if (lds > 0 && lds < INT64_MAX) {
    p->small_lds = static_cast<int32_t>(lds);
    return;
  }
  int64_t ws = 0, part0 = 0;
  auto take = [&](int64_t n) {
    const int64_t at = ws;
    ws += n;
    return at;
  };
  const int32_t nm = static_cast<int32_t>(p->mats.size());
  for (int32_t i = 0; i < nm; ++i) {
    MuonMat &m = p->mats[i];
    const int64_t size = static_cast<int64_t>(m.rows) * m.cols;
    const int64_t x = static_cast<int64_t>(m.mp) * m.np;
    const int64_t sq = static_cast<int64_t>(m.mp) * m.mp;
    for (int b = 0; b < 2; ++b) m.x[b] = take(2 * x);
    m.a = take(2 * sq);
    m.b = take(2 * sq);
    // parts: of 4096 elements, larger where a matrix would have more than 1024
    m.chunk = static_cast<int32_t>(up(std::max<int64_t>(4096, (size + 1023) / 1024), 1024));
    m.parts = static_cast<int32_t>((size + m.chunk - 1) / m.chunk);
    m.part0 = static_cast<int32_t>(part0);
    part0 += m.parts;
    for (int32_t k = 0; k < m.parts; ++k) p->parts.push_back({i, k, 0});
    for (int32_t r = 0; r < m.mp / 64; ++r)
      for (int32_t c = 0; c < m.np / 64; ++c) p->blocks.push_back({i, r, c});
  }
  // product tiles: the matrices of the longest contraction first, so that
  // what is left at a launch's end is short; bands of kBand row tiles are
  // swept together, so that neighbours share operands
  constexpr int32_t kBand = 8;
  std::vector<int32_t> order(nm);
  for (int32_t i = 0; i < nm; ++i) order[i] = i;
  auto longest = [&](auto key) {
    std::stable_sort(order.begin(), order.end(),
                     [&](int32_t a, int32_t b) { return key(p->mats[a]) > key(p->mats[b]); });
  };
  auto tiles = [&](int64_t bt, bool sym, bool wide) {  // wide: contracted over n, not m
    std::vector<Tile> t;
    for (int32_t i : order) {
      const MuonMat &m = p->mats[i];
      const int32_t r = static_cast<int32_t>(up(m.mp, bt) / bt), c = sym ? r : static_cast<int32_t>(up(m.np, bt) / bt);
      const int32_t steps = (wide ? m.np : m.mp) / kStep;
      for (int32_t m0 = 0; m0 < r; m0 += kBand)
        for (int32_t n = sym ? m0 : 0; n < c; ++n)
          for (int32_t k = m0; k < std::min(r, m0 + kBand); ++k)
            if (!sym || n >= k) t.push_back({i, k, n, steps});
    }
    return t;
  };
  longest([](const MuonMat &m) { return m.np; });
  plan_product([&](int64_t bt) { return tiles(bt, true, true); }, true, p->gram);
  longest([](const MuonMat &m) { return m.mp; });
  plan_product([&](int64_t bt) { return tiles(bt, true, false); }, true, p->poly);
  plan_product([&](int64_t bt) { return tiles(bt, false, false); }, false, p->mul);
  int64_t slots = 0;
  for (const ar_muon_plan::Work *w : {&p->gram, &p->poly, &p->mul})
    for (const ar_dev::MuonJoin &j : w->joins) slots = std::max<int64_t>(slots, j.slot + j.count);
  p->partial_bytes = static_cast<size_t>(up(part0 * 8, 256));
  p->shift_bytes = static_cast<size_t>(up(static_cast<int64_t>(nm) * ar_dev::kMuonMaxSteps * 4, 256));
  p->slot_bytes = static_cast<size_t>(slots) * ar_dev::kMuonSlot * 4;
  p->ws_bytes = static_cast<size_t>(ws) * 2;
}

// The device table's contents: the matrices, then every list.
void fill_table(ar_muon_plan *p) {
  p->table.clear();
  auto put = [&](const auto &v) {
    const size_t at = p->table.size(), bytes = v.size() * sizeof(v[0]);
    p->table.resize(static_cast<size_t>(up(static_cast<int64_t>(at + bytes), 256)));
    if (bytes) std::memcpy(p->table.data() + at, v.data(), bytes);
    return at;
  };
  (void)put(p->mats);
  p->at_parts = put(p->parts);
  p->at_blocks = put(p->blocks);
  for (ar_muon_plan::Work *w : {&p->gram, &p->poly, &p->mul}) {
    w->at_items = put(w->items);
    w->at_first = put(w->first);
    w->at_joins = put(w->joins);
  }
}

void default_scales(ar_muon_plan *p) {
  for (MuonMat &m : p->mats)
    m.scale = static_cast<float>(std::sqrt(std::max(1.0, static_cast<double>(m.rows) / m.cols)));
}

ar_status_t prepare(ar_muon_plan *p) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (p->device >= 0) {
    if (dev != p->device) return fail(AR_ERR_INVALID_ARG, "Muon plan was prepared on another device");
    return AR_OK;
  }
  if (!p->mats.empty()) {
    fill_table(p);
    e = ar_host::device_table(&p->d_table, p->table.data(), p->table.size());
    if (e == hipSuccess && p->small_lds == 0)
      e = ar_host::device_table(&p->d_work, nullptr, p->work_bytes());
    if (e != hipSuccess) {
      p->release();
      return e == hipErrorOutOfMemory ? fail(AR_ERR_OOM, "Muon workspace allocation") : hip_fail(e, "Muon tables");
    }
  }
  p->device = dev;
  return AR_OK;
}

struct MuonCall {
  const void *g;
  const float *mom;
  float *mom_out;
  const void *w;
  void *w_out;
  const ar_muon_params_t *params;  // NULL: orthogonalisation only
};

ar_status_t run(ar_muon_plan *p, const MuonCall &c, void *stream) {
  const int64_t gb = p->arena * (p->g_bf16 ? 2 : 4), wb = p->arena * (p->w_bf16 ? 2 : 4), mb = p->arena * 4;
  struct Arena {
    const void *p;
    int64_t bytes;
    uintptr_t elem;
    const char *name;
    bool out;
  };
  const Arena all[5] = {{c.g, gb, p->g_bf16 ? 2u : 4u, "grads", false},
                        {c.w_out, wb, p->w_bf16 ? 2u : 4u, c.params ? "weights_out" : "out", true},
                        {c.mom, mb, 4, "momentum", false},
                        {c.mom_out, mb, 4, "momentum_out", true},
                        {c.w, wb, p->w_bf16 ? 2u : 4u, "weights", false}};
  const int n = c.params ? 5 : 2;
  if (p->arena > 0)
    for (int i = 0; i < n; ++i) {
      if (!all[i].p) return fail(AR_ERR_INVALID_ARG, std::string(all[i].name) + " is NULL");
      if (!on(all[i].p, all[i].elem))
        return fail(AR_ERR_INVALID_ARG, std::string(all[i].name) + " is not aligned to its elements");
      for (int j = 0; j < i; ++j) {
        if ((!all[i].out && !all[j].out) || !overlap(all[i].p, all[i].bytes, all[j].p, all[j].bytes)) continue;
        // an output may be its own input: weights_out and weights (1, 4),
        // momentum_out and momentum (3, 2), out and grads of one type (1, 0)
        const bool own = (i == 4 && j == 1) || (i == 3 && j == 2) || (!c.params && p->g_bf16 == p->w_bf16);
        if (!own || all[i].p != all[j].p)
          return fail(AR_ERR_INVALID_ARG, std::string(all[i].name) + " and " + all[j].name + " overlap");
      }
    }
  ar_dev::MuonArgs a{};
  if (c.params) {
    const ar_muon_params_t &q = *c.params;
    const float f[4] = {static_cast<float>(q.momentum), static_cast<float>(q.grad_scale),
                        static_cast<float>(1.0 - q.lr * q.weight_decay), static_cast<float>(q.lr)};
    for (float v : f)
      if (!std::isfinite(v)) return fail(AR_ERR_INVALID_ARG, "a Muon parameter is not a finite fp32 number");
    a.step = true;
    a.nesterov = q.nesterov != 0;
    a.mu = f[0];
    a.gscale = f[1];
    a.keep = f[2];
    a.lr = f[3];
  }
  ar_status_t st = p->device >= 0 ? AR_OK : ar_host::refuse_capture(static_cast<hipStream_t>(stream));
  if (st == AR_OK) st = prepare(p);
  if (st != AR_OK || p->mats.empty()) return st;
  const char *t = static_cast<const char *>(p->d_table);
  a.mats = reinterpret_cast<const MuonMat *>(t);
  a.parts = reinterpret_cast<const MuonTile *>(t + p->at_parts);
  a.blocks = reinterpret_cast<const MuonTile *>(t + p->at_blocks);
  a.nparts = static_cast<int32_t>(p->parts.size());
  a.nblocks = static_cast<int32_t>(p->blocks.size());
  auto work = [t](const ar_muon_plan::Work &w) {
    return ar_dev::MuonWork{reinterpret_cast<const ar_dev::MuonItem *>(t + w.at_items),
                            reinterpret_cast<const int32_t *>(t + w.at_first),
                            reinterpret_cast<const ar_dev::MuonJoin *>(t + w.at_joins),
                            static_cast<int32_t>(w.first.size()) - 1, static_cast<int32_t>(w.joins.size()), w.shape};
  };
  a.gram = work(p->gram);
  a.poly = work(p->poly);
  a.mul = work(p->mul);
  char *dw = static_cast<char *>(p->d_work);
  a.partials = reinterpret_cast<double *>(dw);
  a.shifts = reinterpret_cast<int32_t *>(dw + p->partial_bytes);
  a.slots = reinterpret_cast<float *>(dw + p->partial_bytes + p->shift_bytes);
  a.ws = reinterpret_cast<uint16_t *>(dw + p->partial_bytes + p->shift_bytes + p->slot_bytes);
  a.g = c.g;
  a.mom = c.mom;
  a.mom_out = c.mom_out;
  a.w = c.w;
  a.w_out = c.w_out;
  a.g_bf16 = p->g_bf16;
  a.w_bf16 = p->w_bf16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipEvent_t mark = nullptr;
  st = p->marks.of(s, &mark);
  if (st != AR_OK) return st;
  ar_dev::MuonSteps steps{};
  steps.n = static_cast<int32_t>(p->steps.size());
  steps.ex0 = p->ex0;
  std::copy(p->steps.begin(), p->steps.end(), steps.k);
  if (p->small_lds > 0) {
    ar_dev::t_launch_events = ar_dev::LaunchEvents{nullptr, mark};
    const hipError_t e = ar_dev::muon_small(a, steps, static_cast<int32_t>(p->mats.size()), p->small_lds, p->tiny, s);
    ar_dev::t_launch_events = ar_dev::LaunchEvents{};
    return e == hipSuccess ? AR_OK : hip_fail(e, "kernel launch");
  }
  hipError_t e = ar_dev::muon_begin(a, steps, s);
  for (const MuonStep &k : p->steps) {
    if (e == hipSuccess) e = ar_dev::muon_gram(a, k, s);
    if (e == hipSuccess) e = ar_dev::muon_poly(a, k, s);
    if (k.last) ar_dev::t_launch_events = ar_dev::LaunchEvents{nullptr, mark};
    if (e == hipSuccess) e = ar_dev::muon_apply(a, k, s);
  }
  ar_dev::t_launch_events = ar_dev::LaunchEvents{};
  return e == hipSuccess ? AR_OK : hip_fail(e, "kernel launch");
}

}  // namespace

extern "C" {

ar_experts_t *ar_experts_create(int nexperts, size_t in_features, size_t out_features, ar_dtype_t dtype,
                                ar_dtype_t grad_dtype, const size_t *weight_offsets) {
  ar_experts *ex = nullptr;
  const ar_status_t st = guarded([&]() -> ar_status_t {
    const int32_t d = raw_enum(dtype), g = raw_enum(grad_dtype);
    if (nexperts < 1 || nexperts > 65536) return fail(AR_ERR_INVALID_ARG, "nexperts must be from 1 to 65536");
    if (in_features < 1 || out_features < 1 || in_features > kMaxFeatures || out_features > kMaxFeatures)
      return fail(AR_ERR_INVALID_ARG, "features must be from 1 to 2^22");
    if (!float_type(d) || !float_type(g))
      return fail(AR_ERR_INVALID_ARG, "expert products take AR_FLOAT32 or AR_BFLOAT16");
    if (d == AR_FLOAT32 && g != AR_FLOAT32)
      return fail(AR_ERR_UNSUPPORTED, "AR_FLOAT32 expert products give AR_FLOAT32 weight gradients");
    ex = new ar_experts;
    ex->nexperts = nexperts;
    ex->in = static_cast<int64_t>(in_features);
    ex->out = static_cast<int64_t>(out_features);
    ex->bf16 = d == AR_BFLOAT16;
    ex->grad_bf16 = g == AR_BFLOAT16;
    const int64_t size = ex->in * ex->out;
    for (int e = 0; e < nexperts; ++e) {
      if (weight_offsets && weight_offsets[e] > static_cast<size_t>(INT64_MAX / 16))
        return fail(AR_ERR_INVALID_ARG, "weight offset of expert " + std::to_string(e) + " is too large");
      const int64_t at = weight_offsets ? static_cast<int64_t>(weight_offsets[e]) : e * size;
      ex->offsets.push_back(at);
      ex->arena = std::max(ex->arena, at + size);
      ex->offsets_by_8 = ex->offsets_by_8 && at % 8 == 0;
    }
    ex->slot_bytes =
        static_cast<size_t>(ar_dev::experts_weight_slots(nexperts, ex->in, ex->out)) * ar_dev::kExpertSlot * 4;
    std::vector<int64_t> sorted = ex->offsets;
    std::sort(sorted.begin(), sorted.end());
    for (int e = 1; e < nexperts; ++e)
      if (sorted[e] - sorted[e - 1] < size) return fail(AR_ERR_INVALID_ARG, "the experts' matrices overlap");
    return AR_OK;
  });
  if (st != AR_OK) {
    delete ex;
    return nullptr;
  }
  return ex;
}

ar_status_t ar_experts_prepare(ar_experts_t *ex) {
  if (!ex) return fail(AR_ERR_INVALID_ARG, "expert plan is NULL");
  return guarded([&] { return prepare(ex); });
}

ar_experts_stats_t ar_experts_stats(const ar_experts_t *ex) {
  ar_experts_stats_t s{};
  if (!ex) {
    fail(AR_ERR_INVALID_ARG, "expert plan is NULL");
    return s;
  }
  s.nexperts = ex->nexperts;
  s.device = ex->device;
  s.in_features = static_cast<uint64_t>(ex->in);
  s.out_features = static_cast<uint64_t>(ex->out);
  s.elem_bytes = ex->bf16 ? 2 : 4;
  s.grad_bytes = ex->grad_bf16 ? 2 : 4;
  s.arena_count = static_cast<uint64_t>(ex->arena);
  s.workspace_bytes = ex->offsets.size() * sizeof(int64_t) + ex->slot_bytes;
  return s;
}

ar_status_t ar_experts_launch_shape(const ar_experts_t *ex, int product, size_t ntokens, int aligned,
                                    int32_t *tile_rows, int32_t *tile_cols, int32_t *parts) {
  if (!ex) return fail(AR_ERR_INVALID_ARG, "expert plan is NULL");
  if (product < kExpertsForward || product > kExpertsWeightGrad)
    return fail(AR_ERR_INVALID_ARG, "product must be from 0 to 2");
  if (ntokens > kMaxTokens) return fail(AR_ERR_INVALID_ARG, "more than 2^31 - 65536 tokens");
  const ExpertProduct which = static_cast<ExpertProduct>(product);
  ar_dev::ExpertShape s{0, 0, 0};
  if (ntokens > 0 || which == kExpertsWeightGrad) {
    float any = 0;
    ar_dev::ExpertArgs a = call_args(ex, which, static_cast<int64_t>(ntokens));
    a.aligned = a.aligned && aligned;
    a.slots = ex->slot_bytes > 0 ? &any : nullptr;  // is there a workspace
    s = ar_dev::experts_shape(a, which);
  }
  if (tile_rows) *tile_rows = s.rows;
  if (tile_cols) *tile_cols = s.cols;
  if (parts) *parts = s.parts;
  return AR_OK;
}

ar_status_t ar_experts_forward(ar_experts_t *ex, const void *x, size_t x_stride, const void *weights, void *y,
                               size_t y_stride, const int32_t *ends, size_t ntokens, void *stream) {
  if (!ex) return fail(AR_ERR_INVALID_ARG, "expert plan is NULL");
  return guarded([&] {
    return run(ex, kExpertsForward, {x, x_stride, ex->in, "x"}, {y, y_stride, ex->out, "y"}, weights, true, false, ends,
               ntokens, stream);
  });
}

ar_status_t ar_experts_input_grad(ar_experts_t *ex, const void *dy, size_t dy_stride, const void *weights, void *dx,
                                  size_t dx_stride, const int32_t *ends, size_t ntokens, void *stream) {
  if (!ex) return fail(AR_ERR_INVALID_ARG, "expert plan is NULL");
  return guarded([&] {
    return run(ex, kExpertsInputGrad, {dy, dy_stride, ex->out, "dy"}, {dx, dx_stride, ex->in, "dx"}, weights, true, false,
               ends, ntokens, stream);
  });
}

ar_status_t ar_experts_weight_grad(ar_experts_t *ex, const void *x, size_t x_stride, const void *dy, size_t dy_stride,
                                   void *grads, int accumulate, const int32_t *ends, size_t ntokens, void *stream) {
  if (!ex) return fail(AR_ERR_INVALID_ARG, "expert plan is NULL");
  return guarded([&] {
    return run(ex, kExpertsWeightGrad, {x, x_stride, ex->in, "x"}, {dy, dy_stride, ex->out, "dy"}, grads, false,
               accumulate != 0, ends, ntokens, stream);
  });
}

void ar_experts_destroy(ar_experts_t *ex) {
  if (!ex) return;
  ex->release();
  delete ex;
}

ar_muon_plan_t *ar_muon_plan_create(int nmatrices, const size_t *rows, const size_t *cols, const size_t *offsets,
                                    ar_dtype_t grad_dtype, ar_dtype_t weight_dtype) {
  ar_muon_plan *p = nullptr;
  const ar_status_t st = guarded([&]() -> ar_status_t {
    const int32_t g = raw_enum(grad_dtype), w = raw_enum(weight_dtype);
    if (nmatrices < 0 || nmatrices > 65536) return fail(AR_ERR_INVALID_ARG, "nmatrices must be from 0 to 65536");
    if (nmatrices > 0 && (!rows || !cols)) return fail(AR_ERR_INVALID_ARG, "rows or cols is NULL");
    if (!float_type(g) || !float_type(w))
      return fail(AR_ERR_INVALID_ARG, "Muon plans take AR_FLOAT32 or AR_BFLOAT16");
    p = new ar_muon_plan;
    p->nmatrices = nmatrices;
    p->g_bf16 = g == AR_BFLOAT16;
    p->w_bf16 = w == AR_BFLOAT16;
    int64_t next = 0;
    double work = 0;
    std::vector<std::pair<int64_t, int64_t>> ranges;
    for (int i = 0; i < nmatrices; ++i) {
      const std::string name = "matrix " + std::to_string(i);
      if (rows[i] > 1u << 20 || cols[i] > 1u << 20) return fail(AR_ERR_INVALID_ARG, name + " has a side over 2^20");
      if (offsets && offsets[i] > static_cast<size_t>(INT64_MAX / 16))
        return fail(AR_ERR_INVALID_ARG, name + ": offset too large");
      const int64_t at = offsets ? static_cast<int64_t>(offsets[i]) : next;
      const int64_t size = static_cast<int64_t>(rows[i]) * static_cast<int64_t>(cols[i]);
      next = at + size;
      if (size == 0) continue;
      MuonMat m{};
      m.at = at;
      m.rows = static_cast<int32_t>(rows[i]);
      m.cols = static_cast<int32_t>(cols[i]);
      m.tall = m.rows > m.cols;
      m.m = std::min(m.rows, m.cols);
      m.n = std::max(m.rows, m.cols);
      m.mp = static_cast<int32_t>(up(m.m, ar_dev::kMuonPad));
      m.np = static_cast<int32_t>(up(m.n, ar_dev::kMuonPad));
      work += static_cast<double>(m.mp) * (4.0 * m.np + 4.0 * m.mp);
      p->mats.push_back(m);
      p->index.push_back(i);
      ranges.push_back({at, next});
      p->arena = std::max(p->arena, next);
    }
    // tiles are counted in int32 and the workspace in bytes
    if (work > 2e11) return fail(AR_ERR_INVALID_ARG, "the matrices are too large for one plan");
    std::sort(ranges.begin(), ranges.end());
    for (size_t i = 1; i < ranges.size(); ++i)
      if (ranges[i].first < ranges[i - 1].second) return fail(AR_ERR_INVALID_ARG, "matrices overlap");
    default_scales(p);
    (void)make_steps(kNsSteps, nullptr, p->steps, p->ex0);
    lay_out(p);
    fill_table(p);
    return AR_OK;
  });
  if (st != AR_OK) {
    delete p;
    return nullptr;
  }
  return p;
}

ar_status_t ar_muon_plan_set_iterations(ar_muon_plan_t *p, int n, const double *abc) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "Muon plan is NULL");
  return guarded([&]() -> ar_status_t {
    if (n < 1 || n > ar_dev::kMuonMaxSteps) return fail(AR_ERR_INVALID_ARG, "iterations must be from 1 to 32");
    std::vector<MuonStep> steps;
    int32_t ex0 = 0;
    if (!make_steps(n, abc, steps, ex0))
      return fail(AR_ERR_INVALID_ARG, "the coefficients let singular values or a factor grow beyond bounds");
    p->steps = std::move(steps);
    p->ex0 = ex0;
    return AR_OK;
  });
}

ar_status_t ar_muon_plan_set_scales(ar_muon_plan_t *p, const double *scales) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "Muon plan is NULL");
  if (scales)
    for (int i = 0; i < p->nmatrices; ++i)
      if (!std::isfinite(static_cast<float>(scales[i])))
        return fail(AR_ERR_INVALID_ARG, "scale of matrix " + std::to_string(i) + " is not a finite fp32 number");
  const bool held = p->d_table != nullptr;
  int dev = 0;
  if (held) {
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    if (dev != p->device) return fail(AR_ERR_INVALID_ARG, "Muon plan was prepared on another device");
  }
  if (!scales) default_scales(p);
  else
    for (size_t i = 0; i < p->mats.size(); ++i) p->mats[i].scale = static_cast<float>(scales[p->index[i]]);
  if (!held) return AR_OK;
  // in place: captured graphs hold the table's address
  p->marks.wait();
  const hipError_t e = ar_host::upload(p->d_table, p->mats.data(), p->mats.size() * sizeof(MuonMat));
  return e == hipSuccess ? AR_OK : hip_fail(e, "Muon tables");
}

ar_status_t ar_muon_plan_prepare(ar_muon_plan_t *p) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "Muon plan is NULL");
  return guarded([&] { return prepare(p); });
}

ar_muon_stats_t ar_muon_plan_stats(const ar_muon_plan_t *p) {
  ar_muon_stats_t s{};
  if (!p) {
    fail(AR_ERR_INVALID_ARG, "Muon plan is NULL");
    return s;
  }
  s.nmatrices = p->nmatrices;
  s.device = p->device;
  s.iterations = static_cast<int32_t>(p->steps.size());
  const int32_t joins = !p->gram.joins.empty() + !p->poly.joins.empty() + !p->mul.joins.empty();
  s.launches = p->mats.empty() ? 0 : p->small_lds > 0 ? 1 : 2 + (3 + joins) * s.iterations;
  s.grad_bytes = p->g_bf16 ? 2 : 4;
  s.weight_bytes = p->w_bf16 ? 2 : 4;
  s.arena_count = static_cast<uint64_t>(p->arena);
  s.workspace_bytes = p->mats.empty() ? 0 : p->table.size() + p->work_bytes();
  return s;
}

int64_t ar_muon_plan_work(const ar_muon_plan_t *p, int product, int32_t *tile, int32_t *group, int32_t *matrix,
                          int32_t *row, int32_t *col, int32_t *k0, int32_t *k1, int32_t *slot, int64_t cap) {
  if (!p) {
    fail(AR_ERR_INVALID_ARG, "Muon plan is NULL");
    return -1;
  }
  if (product < 0 || product > 2) {
    fail(AR_ERR_INVALID_ARG, "product must be from 0 to 2");
    return -1;
  }
  const ar_muon_plan::Work &w = product == 0 ? p->gram : product == 1 ? p->poly : p->mul;
  if (tile) *tile = w.items.empty() ? 0 : ar_dev::muon_tile(w.shape);
  auto put = [](int32_t *to, int64_t i, int32_t v) {
    if (to) to[i] = v;
  };
  for (size_t g = 0; g + 1 < w.first.size(); ++g)
    for (int64_t i = w.first[g]; i < w.first[g + 1] && i < cap; ++i) {
      const ar_dev::MuonItem &t = w.items[static_cast<size_t>(i)];
      put(group, i, static_cast<int32_t>(g));
      put(matrix, i, p->index[static_cast<size_t>(t.mat)]);
      put(row, i, t.m);
      put(col, i, t.n);
      put(k0, i, t.k0);
      put(k1, i, t.k1);
      put(slot, i, t.slot);
    }
  return static_cast<int64_t>(w.items.size());
}

ar_status_t ar_orthogonalize(ar_muon_plan_t *p, const void *grads, void *out, void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "Muon plan is NULL");
  return guarded([&] { return run(p, MuonCall{grads, nullptr, nullptr, nullptr, out, nullptr}, stream); });
}

ar_status_t ar_muon_step(ar_muon_plan_t *p, const void *grads, float *momentum, void *weights, float *momentum_out,
                         void *weights_out, const ar_muon_params_t *params, void *stream) {
  if (!p) return fail(AR_ERR_INVALID_ARG, "Muon plan is NULL");
  if (!params) return fail(AR_ERR_INVALID_ARG, "params is NULL");
  return guarded([&] {
    return run(p, MuonCall{grads, momentum, momentum_out ? momentum_out : momentum, weights,
                           weights_out ? weights_out : weights, params}, stream);
  });
}

void ar_muon_plan_destroy(ar_muon_plan_t *p) {
  if (!p) return;
  p->release();
  delete p;
}

}  // extern "C"

// operators.hpp -- interface between the C ABI and the kernels of the expert
// products (in their own types and in 8 bits), of the RMS norm, of gradient
// clipping and of the Muon update.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ar_dev {

// ---- Products grouped by expert (experts.hip)

// Rows of expert e: [end of e - 1, end of e), where the ends are the running
// maximum of ends[0 .. e], clamped to [0, tokens].
struct ExpertArgs {
  const void *x, *w, *dy;  // which are set depends on the product
  void *out;
  const int64_t *offsets;  // [experts] first element of expert e's matrix
  const int32_t *ends;     // [experts]
  int64_t tokens, in, outf;
  int64_t xs, dys, outs;   // elements between rows of x, dy (y for the forward product's out) and out
  int32_t experts;
  bool bf16;               // element type of x, w, dy, y and dx
  bool grad_bf16;          // element type of the weight gradients
  bool accumulate;
  bool aligned;            // every row and matrix starts on 16 bytes
  float *slots;            // weight gradient: partial tiles (experts_weight_slots)
};

hipError_t experts_forward(const ExpertArgs &a, hipStream_t s);
hipError_t experts_input_grad(const ExpertArgs &a, hipStream_t s);
hipError_t experts_weight_grad(const ExpertArgs &a, hipStream_t s);
// Rows and columns of the tiles of the product that such a call launches, and
// the parts that a weight gradient's rows are cut into.
enum ExpertProduct { kExpertsForward, kExpertsInputGrad, kExpertsWeightGrad };
struct ExpertShape {
  int32_t rows, cols, parts;
};
ExpertShape experts_shape(const ExpertArgs &a, ExpertProduct product);
// Partial tiles, of kExpertSlot sums, that the weight gradient of such experts
// may use: 0 where its tiles are enough for the device.
int64_t experts_weight_slots(int64_t experts, int64_t in, int64_t outf);
constexpr int kExpertSlot = 64 * 128;

// ---- Newton-Schulz and Muon (muon.hip)

// One matrix.  m <= n: its smaller and larger side; tall: rows > cols, worked
// on transposed.  mp, np: m and n rounded up to kMuonPad.  x, a, b: first
// element (16-bit) of its buffers in the workspace: two X buffers of two
// planes (hi, lo) of mp x np, A and B of two planes of mp x mp.
struct MuonMat {
  int64_t at;  // first element in the arenas
  int64_t x[2], a, b;
  int32_t rows, cols, m, n, mp, np;
  int32_t tall;
  int32_t part0, parts;  // its partial sums of squares
  int32_t chunk;         // elements of a part
  float scale;
};
constexpr int kMuonPad = 64;

struct MuonTile {
  int32_t mat, m, n;  // tile row and column; a part's number in m
};

// A product tile's contraction range [k0, k1) that one workgroup works on.
// slot >= 0: the tile is split; the range's sums go to that slot of the
// partial tiles, and a join adds the slots and finishes the tile.
struct MuonItem {
  int32_t mat, m, n, k0, k1, slot;
};
// A split tile: its slots are slot .. slot + count - 1.
struct MuonJoin {
  int32_t mat, m, n, slot, count;
};
// One launch's work: workgroup b does items first[b] .. first[b + 1] - 1.
struct MuonWork {
  const MuonItem *items;
  const int32_t *first;
  const MuonJoin *joins;
  int32_t groups, njoins, shape;  // shape: of the tiles (muon_tile)
};

struct MuonArgs {
  const MuonMat *mats;
  const MuonTile *parts, *blocks;  // work lists
  int32_t nparts, nblocks;
  MuonWork gram, poly, mul;  // X X^T, A A, B X
  double *partials;
  int32_t *shifts;  // [matrix][kMuonMaxSteps]: see MuonStep::drop
  float *slots;     // partial tiles
  uint16_t *ws;
  const void *g;
  const float *mom;
  float *mom_out;
  const void *w;
  void *w_out;
  bool g_bf16, w_bf16;
  bool step, nesterov;
  float mu, gscale, keep, lr;  // keep: 1 - lr * weight decay
};

// One step's factors: powers of two that the stored X, A and B and the next
// X carry, and the polynomial.
//
// A matrix whose norm is not far above the constant that is added to it
// starts with an X_0 far below 1.  Its X carries 2^d more, and its A 2^(2 d):
// d_0 from the norm, so that ||X_0||_F 2^d_0 is in [1/2, 1), and d_k+1 =
// max(0, d_k - drop_k), where 2^drop_k is what the step can make of a small X
// beyond what the bound on the singular values grows by.
struct MuonStep {
  float coef_a, coef_b, coef_c;
  int32_t ex, ea, eb, ex_next;
  int32_t drop;
  int32_t index;     // of the step
  bool last;
  int32_t from;      // X buffer read
};

constexpr int kMuonMaxSteps = 32;
struct MuonSteps {
  int32_t n, ex0;
  MuonStep k[kMuonMaxSteps];
};

// Plans whose matrices all fit into the LDS of one CU run in one launch, a
// workgroup per matrix: LDS bytes of an m x n matrix there (m <= n), 0 if it
// does not fit.
int64_t muon_small_lds(int64_t m, int64_t n);
// tiny: all matrices are up to 64 x 64.
hipError_t muon_small(const MuonArgs &a, const MuonSteps &k, int32_t nmats, int32_t lds, bool tiny, hipStream_t s);

// Rows and columns of tile shape i (0: the largest, the one that can be
// split into partial tiles of kMuonSlot sums).
int muon_tile(int shape);
constexpr int kMuonShapes = 3;
constexpr int kMuonSlot = 256 * 256;

hipError_t muon_begin(const MuonArgs &a, const MuonSteps &k, hipStream_t s);
hipError_t muon_gram(const MuonArgs &a, const MuonStep &k, hipStream_t s);
hipError_t muon_poly(const MuonArgs &a, const MuonStep &k, hipStream_t s);
hipError_t muon_apply(const MuonArgs &a, const MuonStep &k, hipStream_t s);

// ---- The global gradient norm and clipping (clip.hip)

// A run of one tensor's elements, which one wave works on.
struct NormChunk {
  int64_t at;
  int32_t count, unused;  // (16 bytes)
};
constexpr int kNormWaves = 8;  // chunks, a wave each, of a workgroup

struct NormArgs {
  const void *g;
  void *out;
  const NormChunk *chunks;
  const int32_t *first;   // [tensors + 1] first chunk of each tensor
  double *chunk_sums;     // [chunks] sums of squares
  double *group_sums;     // [workgroups]
  float *norm;
  float *tensor_norms;    // or NULL
  double scale, max_norm;
  int32_t nchunks, ntensors;
  bool bf16;
};
hipError_t grad_norm(const NormArgs &a, hipStream_t s);
hipError_t grad_clip(const NormArgs &a, hipStream_t s);

// ---- 8-bit rows and the RMS norm (rmsnorm.hip)

constexpr int kQBlock8 = 128;  // elements of a scale

struct QuantArgs {
  const void *x;
  uint8_t *codes, *scales;
  int64_t features, tokens, xs, cs, ss;  // strides of x, codes and scales
  bool bf16;
};
hipError_t quantize_rows(const QuantArgs &a, hipStream_t s);

struct RmsForward {
  const void *x, *r, *gain;
  void *h, *y;
  uint8_t *codes, *scales;
  float *rstd;
  int64_t xs, rs, hs, ys, cs, ss, tokens;
  int32_t features;
  double eps;
  bool bf16, gain_bf16;
};
hipError_t rmsnorm_forward(const RmsForward &a, hipStream_t s);

struct RmsBackward {
  const void *dy, *h, *dh, *gain;
  const float *rstd;
  void *dx, *dgain;
  float *parts;  // [parts][features] sums of dgain
  int64_t dys, hs, dhs, dxs, tokens;
  int32_t features;
  bool bf16, gain_bf16, grad_bf16, accumulate;
};
hipError_t rmsnorm_backward(const RmsBackward &a, hipStream_t s);
// Parts that such rows are summed in at most.
int32_t rmsnorm_parts(int64_t features, bool bf16);

// ---- 8-bit products grouped by expert (qexperts.hip)

struct QExpertArgs {
  const uint8_t *x, *w;         // codes: rows, weights
  const uint8_t *x_scales, *w_scales;
  void *out;
  const int64_t *offsets;       // [experts] first element of expert e's matrix
  const int32_t *ends;          // [experts]
  int64_t tokens, in, outf;
  int64_t xs, xss, outs;        // elements between rows of x, of its scales, of out
  int32_t experts;
  bool bf16;                    // element type of out
  bool aligned;                 // every row and matrix of codes starts on 16 bytes
};
hipError_t qexperts_forward(const QExpertArgs &a, hipStream_t s);
hipError_t qexperts_input_grad(const QExpertArgs &a, hipStream_t s);
ExpertShape qexperts_shape(const QExpertArgs &a, ExpertProduct product);

struct QWeightArgs {
  const void *w;
  uint8_t *codes, *scales;
  const int64_t *offsets;
  int64_t in, outf;
  int32_t experts;
  bool bf16;
};
hipError_t qexperts_quantize(const QWeightArgs &a, hipStream_t s);

}  // namespace ar_dev

// vocab_gemm.hpp -- the three products of the losses over a vocabulary.
#pragma once

#include <algorithm>

#include "mss_train.hpp"

namespace mss {

// bf16 losses keep a logit as its distance below its tile's ceiling in 16 bits:
// steps of 2^-10, so that a probability is off by at most 2^-11, an eighth of
// what its rounding to bf16 takes; one 64 below (1e-28 of its tile's largest) is 0.
constexpr float kCodeSteps = 1024.0f;

// Columns of dz's panels, and where its elements and those of the probabilities lie.
constexpr int kZPanel = 32;
__device__ inline int64_t z_index(const LossArgs& a, int i, int v) {
  return (static_cast<int64_t>(v / kZPanel) * a.piece + i) * kZPanel + v % kZPanel;
}

// How many parts of the vocabulary the dx product is cut into, for `tiles` tiles
// of its rows and columns: the least time, in steps of about a microsecond, of the
// rounds that the parts' workgroups make (256 of large tiles at a time, 768 of
// small ones), each with some steps besides its own, and of writing and adding
// the parts.  Host and device agree on it.
__host__ __device__ inline int dx_splits(const LossArgs& a, int tiles) {
  const float slots = a.small_dx ? 768.0f : 256.0f, steps = static_cast<float>((a.vocab + 63) / 64 * (a.planes == 1 ? 1 : 6));
  const float part = a.small_dx ? 0.016f : 0.13f;
  int best = 1;
  float least = 3e38f;
  for (int s = 1; s <= a.splits; s += s < 8 ? 1 : s / 4) {
    const float n = static_cast<float>(tiles) * s, t = ceilf(n / slots) * (steps / s + 6.0f) + n * part;
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

// Tiles of the dx product for this many rows.
__host__ __device__ inline int dx_tiles(const LossArgs& a, int rows) {
  return a.small_dx ? (rows + 63) / 64 * ((a.dim + 127) / 128) : (rows + 255) / 256 * ((a.dim + 255) / 256);
}

// logits of the piece's rows: stats, and with `keep` the codes or logits
hipError_t launch_logits(const LossArgs& a, int first, bool io_bf16, bool keep, hipStream_t stream);
// The products of dz that are wanted: part = dz weight, by splits of the vocabulary;
// dweight = dz^T x, or its sum over the pieces so far.
hipError_t launch_gradients(const LossArgs& a, int first, bool io_bf16, hipStream_t stream);

}  // namespace mss

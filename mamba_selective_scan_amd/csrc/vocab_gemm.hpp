// vocab_gemm.hpp -- the three products of the losses over a vocabulary.
#pragma once

#include <algorithm>

#include "mss_train.hpp"

namespace mss {

// bf16 losses keep a logit as its distance below its tile's maximum in 16 bits:
// steps of 2^-10, so that a probability is off by at most 2^-11, an eighth of
// what its rounding to bf16 takes; one 64 below (1e-28 of its tile's largest) is 0.
constexpr float kCodeSteps = 1024.0f;

// Where the elements of dz and of the probabilities lie: blocks of 64 rows, in them
// panels of 32 columns.
constexpr int kZPanel = 32;
__device__ inline int64_t z_index(const LossArgs& a, int i, int v) {
  return (i / 64 * (a.vpad / kZPanel) + v / kZPanel) * (64 * kZPanel) + i % 64 * kZPanel + v % kZPanel;
}

// Tiles of the products: rows and columns, how many a CU holds, and in nanoseconds
// the time of 64 of the summed axis where it holds as many, the least it gets to
// where it holds fewer, and the time of the rest (measured; those of fp32 are of
// three planes).  Large and small ones.
struct TileShape {
  int m, n, per_cu, step, least, rest;
};
__host__ __device__ constexpr TileShape logits_shape(bool f32, bool small) {
  if (f32) return small ? TileShape{128, 64, 2, 2000, 1100, 6000} : TileShape{256, 128, 1, 3800, 3800, 10000};
  return small ? TileShape{128, 64, 3, 930, 600, 5600} : TileShape{256, 256, 1, 1770, 1770, 12800};
}
__host__ __device__ constexpr TileShape dx_shape(bool f32, bool small) {
  if (f32) return small ? TileShape{64, 128, 2, 2000, 1100, 6000} : TileShape{128, 256, 1, 3800, 3800, 10000};
  return small ? TileShape{64, 128, 4, 1800, 640, 6000} : TileShape{256, 256, 1, 1700, 1700, 9000};
}
__host__ __device__ constexpr TileShape dw_shape(bool f32, bool small) {
  if (f32) return small ? TileShape{128, 64, 2, 2000, 1100, 6000} : TileShape{256, 128, 1, 3800, 3800, 10000};
  return small ? TileShape{128, 64, 4, 1350, 700, 4500} : TileShape{256, 256, 1, 1700, 1700, 10000};
}
__host__ __device__ inline int64_t tiles_of(TileShape t, int64_t m, int64_t n) {
  return (m + t.m - 1) / t.m * ((n + t.n - 1) / t.n);
}

// About the time of `tiles` tiles, each cut into `splits` parts along a summed axis
// of `steps` times 64: the rounds that the workgroups make, and writing and adding
// the parts.
__host__ __device__ inline float product_time(TileShape t, float tiles, float splits, float steps) {
  const float n = tiles * splits, cus = ceilf(n * (1.0f / 256.0f)), full = static_cast<float>(t.per_cu);
  const float step = fmaxf(static_cast<float>(t.step) * fminf(cus / full, 1.0f), static_cast<float>(t.least));
  return ceilf(cus / full) * (ceilf(steps / splits) * step + static_cast<float>(t.rest)) + (splits > 1.0f ? n * static_cast<float>(t.m * t.n) * 2e-3f : 0.0f);
}

// Workgroups of the dx product: its tiles cut into as many parts of the vocabulary
// as suit the rows that count, which the device alone knows.
constexpr int kDxBlocks = 2048;
inline int64_t dx_blocks(const LossArgs& a, int64_t rows) {
  const int64_t n = tiles_of(dx_shape(a.planes == 3, a.small_dx), rows, a.dim);
  return std::max<int64_t>((n + 7) / 8 * 8, kDxBlocks);
}
// The parts for this many rows: one wave's work, each lane tries one count.
__device__ inline int dx_cuts(const LossArgs& a, int rows) {
  const TileShape t = dx_shape(a.planes == 3, a.small_dx);
  const int n = static_cast<int>(tiles_of(t, max(rows, 1), a.dim)), s = static_cast<int>(threadIdx.x & 63) + 1;
  float time = s == 1 || (s <= a.splits && s * n <= kDxBlocks)
                   ? product_time(t, static_cast<float>(n), static_cast<float>(s), static_cast<float>((a.vocab + 63) / 64))
                   : INFINITY;
  int best = s;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float other = __shfl_xor(time, o, 64);
    const int from = __shfl_xor(best, o, 64);
    if (other < time || (other == time && from < best)) {
      time = other;
      best = from;
    }
  }
  return best;
}

// Up to so many rows of fp32, with gradients and without, take their products from
// the matrix as it is, not from planes of it (20000 x 2560, 60 rows with gradients:
// 259 us, 382 from planes; without, 72 rows: 133 us, 226 from planes; 129 rows: 216).
constexpr int kDirectRows = 64, kDirectLossRows = 128;

// logits of the piece's rows: stats, and with `keep` the codes or logits
hipError_t launch_logits(const LossArgs& a, int first, bool keep, hipStream_t stream);
// The products of dz that are wanted: part = dz weight, by splits of the vocabulary;
// dweight = dz^T x, or its sums over parts of the rows, or over the pieces so far.
hipError_t launch_gradients(const LossArgs& a, int first, hipStream_t stream);
// The same of few rows of fp32.
hipError_t launch_few_logits(const LossArgs& a, hipStream_t stream);
hipError_t launch_few_gradients(const LossArgs& a, hipStream_t stream);

}  // namespace mss

// vocab_gemm.hip -- the three products of the losses over a vocabulary, gfx950:
//   logits  z2[i, v]    = scale2 sum_d x[i, d] w[v, d], with each tile's softmax sums
//   dx      part[i, d]  = sum_v dz[i, v] w[v, d], cut over v
//   dweight dw[v, d]    = sum_i dz[i, v] x[i, d]
//
// Operands are bf16 planes: one, or three whose sum is an fp32 value.  The
// product of two values in three planes takes the six products of planes whose
// orders sum to at most two; what is left out is below 2^-24 of it.
#include "mss.h"
#include "vocab_gemm.hpp"

namespace mss {
namespace {

__device__ constexpr int kPlaneA[6] = {0, 0, 1, 0, 1, 2}, kPlaneB[6] = {0, 1, 0, 2, 1, 0};

struct Gemm {
  const uint16_t* a;  // element (m, k) at m * am + k * ak, a plane every `ap`
  const uint16_t* b;
  int64_t am, ak, ap, bn, bk, bp;
  int m, n, k, pairs;
};

__device__ inline float as_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// 64 x 64 of the product over k in [k0, k1): acc[i][j] of row ty + 16 i and
// column tx + 16 j of the tile.
__device__ inline void tile(const Gemm& g, int m0, int n0, int k0, int k1, float (&acc)[4][4]) {
  __shared__ float sa[16][65], sb[16][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int pr = 0; pr < g.pairs; ++pr) {
    const uint16_t* a = g.a + kPlaneA[pr] * g.ap;
    const uint16_t* b = g.b + kPlaneB[pr] * g.bp;
    for (int k = k0; k < k1; k += 16) {
      for (int e = threadIdx.x; e < 1024; e += 256) {
        const int kk = e >> 6, r = e & 63;
        sa[kk][r] = m0 + r < g.m && k + kk < k1 ? as_float(a[(m0 + r) * g.am + (k + kk) * g.ak]) : 0.0f;
        sb[kk][r] = n0 + r < g.n && k + kk < k1 ? as_float(b[(n0 + r) * g.bn + (k + kk) * g.bk]) : 0.0f;
      }
      __syncthreads();
      for (int kk = 0; kk < 16; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[kk][ty + 16 * i], sb[kk][tx + 16 * j], acc[i][j]);
      __syncthreads();
    }
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void logits_kernel(LossArgs a, int first, bool keep) {
  const int rows = min(a.piece, *a.live - first), i0 = blockIdx.y * 64, v0 = blockIdx.x * 64;
  if (i0 >= rows) return;
  const Gemm g{a.xp + first * a.dpad, a.wp, a.dpad, 1, a.rows * a.dpad, a.wp_stride, 1, a.wp_plane,
               rows, a.vocab, a.dim, a.planes == 1 ? 1 : 6};
  float acc[4][4];
  tile(g, i0, v0, 0, a.dim, acc);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i0 + ty + 16 * i;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[i][j] = v0 + tx + 16 * j < a.vocab ? acc[i][j] * a.scale2 : -INFINITY;
      top = fmaxf(top, acc[i][j]);
    }
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 16));
    top = ceilf(top);
    const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += exp2f(acc[i][j] - from);
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 16);
    if (r >= rows) continue;
    if (tx == 0) a.stats[static_cast<int64_t>(r) * a.tiles + blockIdx.x] = make_float2(top, sum);
    if (keep)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = v0 + tx + 16 * j;
        if (v >= a.vocab) continue;
        if constexpr (BF16)
          static_cast<uint16_t*>(a.probs)[r * a.vpad + v] =
              static_cast<uint16_t>(fminf(rintf((top - acc[i][j]) * 1024.0f), 65535.0f));
        else
          static_cast<float*>(a.probs)[r * a.vpad + v] = acc[i][j];
      }
  }
}

__global__ __launch_bounds__(256) void dx_part_kernel(LossArgs a, int first) {
  const int rows = min(a.piece, *a.live - first), i0 = blockIdx.y * 64, d0 = blockIdx.x * 64;
  if (i0 >= rows) return;
  const int per = (a.vocab + a.splits - 1) / a.splits, v0 = blockIdx.z * per, v1 = min(v0 + per, a.vocab);
  const Gemm g{a.dz, a.wp, a.vpad, 1, a.piece * a.vpad, 1, a.wp_stride, a.wp_plane, rows, a.dim, a.vocab,
               a.planes == 1 ? 1 : 6};
  float acc[4][4];
  tile(g, i0, d0, v0, v1, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = i0 + (threadIdx.x >> 4) + 16 * i, c = d0 + (threadIdx.x & 15) + 16 * j;
      if (r < rows && c < a.dim) a.part[(static_cast<int64_t>(blockIdx.z) * a.piece + r) * a.dpad + c] = acc[i][j];
    }
}

template <typename IO>
__global__ __launch_bounds__(256) void dw_tile_kernel(LossArgs a, int first) {
  const int rows = max(min(a.piece, *a.live - first), 0), v0 = blockIdx.x * 64, d0 = blockIdx.y * 64;
  if (first > 0 && rows == 0) return;
  const Gemm g{a.dz, a.xp + first * a.dpad, 1, a.vpad, a.piece * a.vpad, 1, a.dpad, a.rows * a.dpad, a.vocab,
               a.dim, rows, a.planes == 1 ? 1 : 6};
  float acc[4][4];
  tile(g, v0, d0, 0, rows, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + (threadIdx.x >> 4) + 16 * i, c = d0 + (threadIdx.x & 15) + 16 * j;
      if (v >= a.vocab || c >= a.dim) continue;
      if (a.pieces == 1)
        io_traits<IO>::store(static_cast<IO*>(a.dweight) + v * a.sdw + c, acc[i][j]);
      else
        a.dw_sum[v * a.dpad + c] = acc[i][j] + (first > 0 ? a.dw_sum[v * a.dpad + c] : 0.0f);
    }
}

}  // namespace

hipError_t launch_logits(const LossArgs& a, int first, bool io_bf16, bool keep, hipStream_t stream) {
  const dim3 g(static_cast<unsigned>(a.tiles), static_cast<unsigned>(std::min(a.piece, a.rows - first) + 63) / 64);
  if (io_bf16) logits_kernel<true><<<g, 256, 0, stream>>>(a, first, keep);
  else logits_kernel<false><<<g, 256, 0, stream>>>(a, first, keep);
  return hipGetLastError();
}

hipError_t launch_dx(const LossArgs& a, int first, hipStream_t stream) {
  const dim3 g(static_cast<unsigned>(a.dim + 63) / 64, static_cast<unsigned>(std::min(a.piece, a.rows - first) + 63) / 64,
               static_cast<unsigned>(a.splits));
  dx_part_kernel<<<g, 256, 0, stream>>>(a, first);
  return hipGetLastError();
}

hipError_t launch_dw(const LossArgs& a, int first, bool io_bf16, hipStream_t stream) {
  const dim3 g(static_cast<unsigned>(a.vocab + 63) / 64, static_cast<unsigned>(a.dim + 63) / 64);
  if (io_bf16) dw_tile_kernel<bf16_t><<<g, 256, 0, stream>>>(a, first);
  else dw_tile_kernel<float><<<g, 256, 0, stream>>>(a, first);
  return hipGetLastError();
}

}  // namespace mss

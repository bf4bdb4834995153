// rms_norm.hip -- root-mean-square norm with the residual's addition and an
// output in the input's type or in 8 bits with scales, gfx950.
//
//   r = x + residual;  y = r / sqrt(mean(r^2) + eps) * weight
//   scale = max |y| / 448 over the row or 128 columns;  out = e4m3(y / scale)
//
// A stream: every input is read once and every output written once, so it is
// bound by HBM bandwidth.  A row stays in registers between its two sums (the
// squares, the largest |y|) and its output: one wave a row up to 2048 columns,
// 256 threads up to 8192, 1024 above.  A lane owns 8 adjacent columns (16 bytes
// of bf16), so a block's 128 columns are the 16 lanes of a DPP row.  32768 rows of
// 5120 with an fp32 residual and 8-bit blocks: 346 us, 5.3 TB/s, past a copy's 5.1
// (part of the residual stays in the last-level cache); one row of 1536: 3.1 us,
// a launch and one trip to memory.
#include "mss.h"
#include "mss_head.hpp"

namespace mss {
namespace {

constexpr int kV = 8;
constexpr float kE4m3Max = 448.0f;
// A mean square below kFewBits may have lost addends.  2^75 takes the smallest
// normal value to 2^-51 and its inverse the largest to 2^53, whose squares, and
// sums of 32768 of them, are in the normal range.
constexpr float kFewBits = 0x1p-80f, kScaleUp = 0x1p75f;

template <int OFF>
__device__ inline uint32_t row_ror(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x120 + OFF, 0xF, 0xF, true));
}
// |y| is compared as bits: the order of non-negative floats, with a NaN above
// everything, so a NaN reaches the scale.
__device__ inline uint32_t row_max16(uint32_t v) {
  v = max(v, row_ror<8>(v));
  v = max(v, row_ror<4>(v));
  v = max(v, row_ror<2>(v));
  v = max(v, row_ror<1>(v));
  return v;
}
__device__ inline uint32_t wave_max(uint32_t v) {
  v = row_max16(v);
  v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 16, 64)));
  return max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 32, 64)));
}
__device__ inline float wave_sum(float v) {
  v = row_sum16(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// The scale for a largest |y| (as bits): 1 where max / 448 is zero, below the
// normal range, or not a number.
__device__ inline float scale_of(uint32_t top) {
  const float s = __uint_as_float(top) / kE4m3Max;
  return s >= 1.17549435e-38f ? s : 1.0f;
}

// 8 values divided by their scale, in e4m3.  A NaN stays one.
__device__ inline void to_e4m3(const float* y, float inv, uint32_t* out) {
  float q[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const float v = y[i] * inv;
    q[i] = v != v ? v : fminf(fmaxf(v, -kE4m3Max), kE4m3Max);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true);
    out[i] = static_cast<uint32_t>(w);
  }
}
typedef uint32_t __attribute__((ext_vector_type(2), aligned(1))) bytes8;

// TPR threads a row, K vectors a thread.  Rows of 1024 threads with two vectors stay
// at 64 registers, so that a CU holds two of them (8192 rows of 16384: 274 us, 295 us
// with more).
template <typename IO, typename RES, int QUANT, int TPR, int K>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, TPR == 1024 && K == 2 ? 8 : 1) void norm_kernel(NormArgs a) {
  constexpr int kBlock = TPR < 256 ? 256 : TPR;
  constexpr int kWavesRow = TPR / 64;
  __shared__ float sums[kWavesRow > 1 ? kWavesRow : 1];
  __shared__ uint32_t tops[kWavesRow > 1 ? kWavesRow : 1];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kBlock / TPR) + threadIdx.x / TPR;
  if (kWavesRow == 1 && row >= a.rows) return;  // (whole waves; never with barriers)
  const int tid = threadIdx.x % TPR;
  const IO* x = static_cast<const IO*>(a.x) + row * a.sx;
  const RES* res = static_cast<const RES*>(a.res) + row * a.sr;
  float r[K][kV], w[K][kV];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + tid) * kV;
    load_part<IO, kV>(x + c, a.dim - c, r[k]);
  }
  if (a.res != nullptr) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + tid) * kV;
      float q[kV];
      load_part<RES, kV>(res + c, a.dim - c, q);
#pragma unroll
      for (int i = 0; i < kV; ++i) r[k][i] += q[i];
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + tid) * kV;
    load_part<float, kV>(a.weight + c, a.dim - c, w[k]);
  }
  auto squares = [&]() __attribute__((always_inline)) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < kV; ++i) sum = fmaf(r[k][i], r[k][i], sum);
    sum = wave_sum(sum);
    if constexpr (kWavesRow > 1) {
      if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
      __syncthreads();
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kWavesRow; ++i) sum += sums[i];
    }
    return sum;
  };
  float mean = squares() / static_cast<float>(a.dim) + a.eps;
  if (a.res_out != nullptr) {
    RES* ro = static_cast<RES*>(a.res_out) + row * a.sro;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + tid) * kV;
      store_part<RES, kV>(ro + c, a.dim - c, r[k]);
    }
  }
  if (!(mean < INFINITY) || mean < kFewBits) {
    // squares past fp32, or lost below it: those of the row scaled towards 1
    const float by = mean < 1.0f ? kScaleUp : 1.0f / kScaleUp;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < kV; ++i) r[k][i] *= by;
    if constexpr (kWavesRow > 1) __syncthreads();  // (the sums have been read)
    mean = squares() / static_cast<float>(a.dim) + a.eps * by * by;
  }
  const float inv = 1.0f / sqrtf(mean);
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      r[k][i] = r[k][i] * inv * w[k][i];
      if constexpr (QUANT == MSS_QUANT_ROW) top = max(top, __float_as_uint(fabsf(r[k][i])));
    }
  if constexpr (QUANT == MSS_QUANT_NONE) {
    IO* out = static_cast<IO*>(a.out) + row * a.so;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + tid) * kV;
      store_part<IO, kV>(out + c, a.dim - c, r[k]);
    }
    return;
  }
  float scale = 1.0f;
  if constexpr (QUANT == MSS_QUANT_ROW) {
    top = wave_max(top);
    if constexpr (kWavesRow > 1) {
      if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
      __syncthreads();
      top = 0;
#pragma unroll
      for (int i = 0; i < kWavesRow; ++i) top = max(top, tops[i]);
    }
    scale = scale_of(top);
    if (tid == 0) a.scale[row] = scale;
  }
  uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.so;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + tid) * kV;
    if constexpr (QUANT == MSS_QUANT_BLOCK) {
      top = 0;
#pragma unroll
      for (int i = 0; i < kV; ++i) top = max(top, __float_as_uint(fabsf(r[k][i])));
      scale = scale_of(row_max16(top));
      if (c < a.dim && (threadIdx.x & 15) == 0) a.scale[row * (a.dim / kScaleBlock) + c / kScaleBlock] = scale;
    }
    uint32_t q[2];
    to_e4m3(r[k], 1.0f / scale, q);
    if (c + kV <= a.dim) {
      *reinterpret_cast<bytes8*>(out + c) = bytes8{q[0], q[1]};
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (c + i < a.dim) out[c + i] = static_cast<uint8_t>(q[i / 4] >> (8 * (i % 4)));
    }
  }
}

template <typename IO, typename RES, int QUANT>
hipError_t launch_q(const NormArgs& a, hipStream_t stream) {
  const int d = a.dim;
  const unsigned by4 = static_cast<unsigned>((a.rows + 3) / 4), by1 = static_cast<unsigned>(a.rows);
  if (d <= 512) norm_kernel<IO, RES, QUANT, 64, 1><<<by4, 256, 0, stream>>>(a);
  else if (d <= 1024) norm_kernel<IO, RES, QUANT, 64, 2><<<by4, 256, 0, stream>>>(a);
  else if (d <= 1536) norm_kernel<IO, RES, QUANT, 64, 3><<<by4, 256, 0, stream>>>(a);
  else if (d <= 2048) norm_kernel<IO, RES, QUANT, 64, 4><<<by4, 256, 0, stream>>>(a);
  else if (d <= 4096) norm_kernel<IO, RES, QUANT, 256, 2><<<by1, 256, 0, stream>>>(a);
  else if (d <= 6144) norm_kernel<IO, RES, QUANT, 256, 3><<<by1, 256, 0, stream>>>(a);
  else if (d <= 8192) norm_kernel<IO, RES, QUANT, 256, 4><<<by1, 256, 0, stream>>>(a);
  else if (d <= 16384) norm_kernel<IO, RES, QUANT, 1024, 2><<<by1, 1024, 0, stream>>>(a);
  else norm_kernel<IO, RES, QUANT, 1024, 4><<<by1, 1024, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename IO, typename RES>
hipError_t launch_r(const NormArgs& a, int quant, hipStream_t stream) {
  if (quant == MSS_QUANT_ROW) return launch_q<IO, RES, MSS_QUANT_ROW>(a, stream);
  if (quant == MSS_QUANT_BLOCK) return launch_q<IO, RES, MSS_QUANT_BLOCK>(a, stream);
  return launch_q<IO, RES, MSS_QUANT_NONE>(a, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool io_bf16, bool res_bf16, int quant, hipStream_t stream) {
  if (io_bf16)
    return res_bf16 ? launch_r<bf16_t, bf16_t>(a, quant, stream) : launch_r<bf16_t, float>(a, quant, stream);
  return res_bf16 ? launch_r<float, bf16_t>(a, quant, stream) : launch_r<float, float>(a, quant, stream);
}

}  // namespace mss

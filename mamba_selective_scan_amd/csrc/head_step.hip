// head_step.hip -- one token a row through the conv step and the head-wise
// scan step, on caches of windows and states by slot, gfx950.
//
//   u     = silu(bias + sum_k w[k] * line[k]),  line = window followed by the sample
//   delta = softplus(dt_raw + dt_bias)
//   S     <- exp(-delta exp(A_log)) S + delta * x * B      (in place, x, B, C parts of u)
//   out   = (sum_n C[n] S[n] + D x) * silu(z)
//
// Bound by the states, read and written once (8 P N bytes a head; everything
// else is two orders smaller).  Two launches: the first filters every channel,
// slides its window and leaves u in fp32, since the windows of B and C are read
// by all heads of a group and may only slide once; the second walks the states.
#include "mss_head.hpp"

namespace mss {
namespace {

template <typename IO, int W>
__global__ __launch_bounds__(256) void head_step_conv_kernel(HeadStepArgs a, int chans) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.rows) * chans) return;
  const int b = static_cast<int>(i / chans);
  const int c = static_cast<int>(i % chans);
  const int slot = slot_of(a.slots, a.cache_slots, b);
  if (slot < 0) return;
  IO* st = static_cast<IO*>(a.window) + slot * a.swin + static_cast<int64_t>(c) * (W - 1);
  float line[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) line[k] = io_traits<IO>::load(st + k);
  line[W - 1] = io_traits<IO>::load(static_cast<const IO*>(a.xbc) + b * a.sx[0] + c * a.sx[1]);
  float acc = a.bias != nullptr ? a.bias[c] : 0.0f;
#pragma unroll
  for (int k = 0; k < W; ++k) acc = fmaf(a.weight[c * a.sw[0] + k * a.sw[1]], line[k], acc);
  a.u[i] = silu(acc);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) io_traits<IO>::store(st + k, line[k + 1]);
}

// Sum over groups of LPR adjacent lanes, left in every lane of the group: quad
// permutations, then mirrors (which reach across once quads and halves agree).
template <int LPR>
__device__ inline float group_sum(float v) {
  auto dpp = [&](auto ctrl) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v += dpp(std::integral_constant<int, 0xB1>{});  // quad_perm [1,0,3,2]
  v += dpp(std::integral_constant<int, 0x4E>{});  // quad_perm [2,3,0,1]
  if constexpr (LPR >= 8) v += dpp(std::integral_constant<int, 0x141>{});   // row_half_mirror
  if constexpr (LPR >= 16) v += dpp(std::integral_constant<int, 0x140>{});  // row_mirror
  if constexpr (LPR >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

// One workgroup per (row, head, tile of columns p).  LPR lanes hold one column's
// states, four per lane; a thread holds NP columns, all loaded before the first
// is used.
template <typename IO, int LPR, int NP>
__global__ __launch_bounds__(256) void head_step_kernel(HeadStepArgs a, int chans, int ptiles) {
  constexpr int RP = 256 / LPR;  // columns per pass
  int64_t id = blockIdx.x;
  const int tile = static_cast<int>(id % ptiles);
  id /= ptiles;
  const int h = static_cast<int>(id % a.heads);
  const int b = static_cast<int>(id / a.heads);
  const int slot = slot_of(a.slots, a.cache_slots, b);
  if (slot < 0) return;
  const int l = threadIdx.x % LPR;
  const int p0 = tile * RP * NP + threadIdx.x / LPR;
  const int n0 = 4 * l;
  const int nn = a.dstate - n0;
  float* st = a.state + slot * a.sstate + (static_cast<int64_t>(h) * a.headdim + p0) * a.dstate + n0;
  float s[NP][4];
#pragma unroll
  for (int k = 0; k < NP; ++k)
    load_part<float, 4>(st + static_cast<int64_t>(k) * RP * a.dstate, p0 + k * RP < a.headdim ? nn : 0, s[k]);
  const float* u = a.u + static_cast<int64_t>(b) * chans;
  const int g = h / (a.heads / a.groups);
  const int hp = a.heads * a.headdim;
  float bn[4], cn[4];
  load_part<float, 4>(u + hp + g * a.dstate + n0, nn, bn);
  load_part<float, 4>(u + hp + (a.groups + g) * a.dstate + n0, nn, cn);
  const float xr = io_traits<IO>::load(static_cast<const IO*>(a.dt) + b * a.sdt[0] + h * a.sdt[1]) +
                   (a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f);
  const float dl = a.softplus ? softplus(xr) : xr;
  const float decay = fast_exp2(dl * (-expf(a.A_log[h]) * kLog2e));
  const float skip = a.D != nullptr ? a.D[h] : 0.0f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int p = p0 + k * RP;
    if (p - static_cast<int>(threadIdx.x / LPR) >= a.headdim) break;  // the whole pass lies past the head
    const bool valid = p < a.headdim;
    const float x = valid ? u[h * a.headdim + p] : 0.0f;
    const float v = dl * x;
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[k][i] = fmaf(decay, s[k][i], v * bn[i]);
      y = fmaf(cn[i], s[k][i], y);
    }
    store_part<float, 4>(st + static_cast<int64_t>(k) * RP * a.dstate, valid ? nn : 0, s[k]);
    y = group_sum<LPR>(y);
    if (valid && l == 0) {
      y = fmaf(skip, x, y);
      if (a.z != nullptr)
        y *= silu(io_traits<IO>::load(static_cast<const IO*>(a.z) + b * a.sz[0] + h * a.sz[1] + p * a.sz[2]));
      io_traits<IO>::store(static_cast<IO*>(a.out) + b * a.so[0] + h * a.so[1] + p * a.so[2], y);
    }
  }
}

template <typename IO, int LPR>
hipError_t launch_lpr(const HeadStepArgs& a, int chans, hipStream_t stream) {
  constexpr int RP = 256 / LPR;
  const int passes = (a.headdim + RP - 1) / RP;
  const int np = passes >= 8 ? 8 : passes >= 4 ? 4 : passes >= 2 ? 2 : 1;
  const int ptiles = (passes + np - 1) / np;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.rows) * a.heads * ptiles)), block(256);
  switch (np) {
    case 1: head_step_kernel<IO, LPR, 1><<<grid, block, 0, stream>>>(a, chans, ptiles); break;
    case 2: head_step_kernel<IO, LPR, 2><<<grid, block, 0, stream>>>(a, chans, ptiles); break;
    case 4: head_step_kernel<IO, LPR, 4><<<grid, block, 0, stream>>>(a, chans, ptiles); break;
    default: head_step_kernel<IO, LPR, 8><<<grid, block, 0, stream>>>(a, chans, ptiles); break;
  }
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_t(const HeadStepArgs& a, hipStream_t stream) {
  const int chans = a.heads * a.headdim + 2 * a.groups * a.dstate;
  const int64_t n = static_cast<int64_t>(a.rows) * chans;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256)), block(256);
  switch (a.width) {
    case 1: head_step_conv_kernel<IO, 1><<<grid, block, 0, stream>>>(a, chans); break;
    case 2: head_step_conv_kernel<IO, 2><<<grid, block, 0, stream>>>(a, chans); break;
    case 3: head_step_conv_kernel<IO, 3><<<grid, block, 0, stream>>>(a, chans); break;
    default: head_step_conv_kernel<IO, 4><<<grid, block, 0, stream>>>(a, chans); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.dstate <= 16) return launch_lpr<IO, 4>(a, chans, stream);
  if (a.dstate <= 32) return launch_lpr<IO, 8>(a, chans, stream);
  if (a.dstate <= 64) return launch_lpr<IO, 16>(a, chans, stream);
  return launch_lpr<IO, 32>(a, chans, stream);
}

}  // namespace

hipError_t launch_head_step(const HeadStepArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_t<bf16_t>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace mss

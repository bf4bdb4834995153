// head_step.hip -- one token a row through the conv step and the head-wise
// scan step, on caches of windows and states by slot, gfx950.
//
//   u     = silu(bias + sum_k w[k] * line[k]),  line = window followed by the sample
//   delta = softplus(dt_raw + dt_bias)
//   S     <- exp(-delta exp(A_log)) S + delta * x * B      (in place, x, B, C parts of u)
//   out   = (sum_n C[n] S[n] + D x) * silu(z)
//
// Bound by the states, read and written once (8 P N bytes a head; everything
// else is two orders smaller).  A workgroup has a tile of one head's columns: it
// starts the loads of the tile's states, filters the tile's x channels and its
// group's B and C while they are on their way, and walks the states.  The windows
// of x slide there, where they have their only reader; those of B and C, which
// every head of the group reads, in a second small launch.  (Filtering B and C
// once for all heads, in a launch before, took a workspace and the same time.)
// The new states leave past the caches: nobody reads them before the next token,
// and what they would push out is read (128 rows of 80 heads: 136 -> 121 us; 64
// rows of two layers, 336 MB: 80 -> 66; 32 rows of 24 heads, eight layers that fit
// the last-level cache: 15.0 -> 14.5).  What the conv, the scan and the norm write
// is read by the operation behind them: there the same stores gain up to 5% alone
// and lose 1.5% over the three (32768 tokens of 80 heads: 1069 -> 1086 us).
// 128 rows of 80 heads of 64 x 128 in bf16: 5.4 TB/s, past a copy's 5.1, as part of
// the states stays in the last-level cache; one row of 24 heads: 6.6 us, bound by
// the two launches and the chain from the windows to the outputs.
#include "mss_head.hpp"

namespace mss {
namespace {

// One channel's window followed by its new sample, at the end of `line`.
template <typename IO>
__device__ inline void conv_line(const HeadStepArgs& a, int b, int slot, int c, IO (&line)[4]) {
  const int H = a.width - 1;
  const IO* st = static_cast<const IO*>(a.window) + slot * a.swin + static_cast<int64_t>(c) * H;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k >= 3 - H) line[k] = st[k - (3 - H)];
  line[3] = static_cast<const IO*>(a.xbc)[b * a.sx[0] + c * a.sx[1]];
}
template <typename IO>
__device__ inline float conv_filter(const HeadStepArgs& a, int c, const IO (&line)[4]) {
  const int H = a.width - 1;
  float acc = a.bias != nullptr ? a.bias[c] : 0.0f;
  if (H == 3 && a.sw[1] == 1) {  // taps that lie together, as layers hold them
    float w[4];
    vecio<float, 4>::load(a.weight + c * a.sw[0], w);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc = fmaf(w[k], io_traits<IO>::load(&line[k]), acc);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k >= 3 - H) acc = fmaf(a.weight[c * a.sw[0] + (k - (3 - H)) * a.sw[1]], io_traits<IO>::load(&line[k]), acc);
  }
  return silu(acc);
}
template <typename IO>
__device__ inline void conv_slide(const HeadStepArgs& a, int slot, int c, const IO (&line)[4]) {
  const int H = a.width - 1;
  IO* st = static_cast<IO*>(a.window) + slot * a.swin + static_cast<int64_t>(c) * H;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k >= 3 - H) st[k - (3 - H)] = line[k + 1];
}

// Slides the windows of B and C.
template <typename IO>
__global__ __launch_bounds__(256) void head_step_slide_kernel(HeadStepArgs a, int bc) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.rows) * bc) return;
  const int b = static_cast<int>(i / bc);
  const int slot = slot_of(a.slots, a.cache_slots, b);
  if (slot < 0) return;
  const int c = a.heads * a.headdim + static_cast<int>(i % bc);
  IO line[4];
  conv_line(a, b, slot, c, line);
  conv_slide(a, slot, c, line);
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
__global__ __launch_bounds__(256) void head_step_kernel(HeadStepArgs a, int ptiles) {
  constexpr int RP = 256 / LPR;  // columns per pass
  constexpr int kCols = RP * NP;
  __shared__ float xs[kCols], ys[kCols];
  __shared__ __attribute__((aligned(16))) float bc[2][kMaxHeadState];  // the group's B and C
  int64_t id = blockIdx.x;
  const int tile = static_cast<int>(id % ptiles);
  id /= ptiles;
  const int h = static_cast<int>(id % a.heads);
  const int b = static_cast<int>(id / a.heads);
  const int slot = slot_of(a.slots, a.cache_slots, b);
  if (slot < 0) return;
  const int l = threadIdx.x % LPR;
  const int pl = threadIdx.x / LPR;          // this thread's first column in the tile
  const int cols = min(kCols, a.headdim - tile * kCols);
  const int n0 = 4 * l;
  const int nn = a.dstate - n0;
  float* st = a.state + slot * a.sstate + (static_cast<int64_t>(h) * a.headdim + tile * kCols + pl) * a.dstate + n0;
  float s[NP][4];
#pragma unroll
  for (int k = 0; k < NP; ++k)
    load_part<float, 4>(st + static_cast<int64_t>(k) * RP * a.dstate, pl + k * RP < cols ? nn : 0, s[k]);
  const int g = h / (a.heads / a.groups);
  const float xr = io_traits<IO>::load(static_cast<const IO*>(a.dt) + b * a.sdt[0] + h * a.sdt[1]) +
                   (a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f);
  const float dl = a.softplus ? softplus(xr) : xr;
  const float decay = fast_exp2(dl * (-expf(a.A_log[h]) * kLog2e));
  // a channel of B or C (2 N <= 256 of them) and the first of x a thread, with
  // both on their way before either is filtered
  const int k = threadIdx.x, which = k >= a.dstate ? 1 : 0;
  const int cb = a.heads * a.headdim + (which * a.groups + g) * a.dstate + k - which * a.dstate;
  const int cx = h * a.headdim + tile * kCols + k;
  IO lb[4], lx[4];
  if (k < 2 * a.dstate) conv_line(a, b, slot, cb, lb);
  if (k < cols) conv_line(a, b, slot, cx, lx);
  if (k < 2 * a.dstate) bc[which][k - which * a.dstate] = conv_filter(a, cb, lb);
  if (k < cols) {
    xs[k] = conv_filter(a, cx, lx);
    conv_slide(a, slot, cx, lx);
  }
  if constexpr (kCols > 256) {
    for (int p = k + 256; p < cols; p += 256) {
      conv_line(a, b, slot, cx + p - k, lx);
      xs[p] = conv_filter(a, cx + p - k, lx);
      conv_slide(a, slot, cx + p - k, lx);
    }
  }
  __syncthreads();
  float bn[4], cn[4];
  load_part<float, 4>(&bc[0][min(n0, kMaxHeadState - 4)], nn, bn);
  load_part<float, 4>(&bc[1][min(n0, kMaxHeadState - 4)], nn, cn);
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int p = pl + k * RP;
    if (k * RP >= cols) break;  // the whole pass lies past the head
    const bool valid = p < cols;
    const float v = valid ? dl * xs[p] : 0.0f;
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[k][i] = fmaf(decay, s[k][i], v * bn[i]);
      y = fmaf(cn[i], s[k][i], y);
    }
    store_part<float, 4, true>(st + static_cast<int64_t>(k) * RP * a.dstate, valid ? nn : 0, s[k]);
    y = group_sum<LPR>(y);
    if (valid && l == 0) ys[p] = y;
  }
  __syncthreads();
  const float skip = a.D != nullptr ? a.D[h] : 0.0f;
  for (int p = threadIdx.x; p < cols; p += 256) {
    const int64_t at = tile * kCols + p;
    float y = fmaf(skip, xs[p], ys[p]);
    if (a.z != nullptr)
      y *= silu(io_traits<IO>::load(static_cast<const IO*>(a.z) + b * a.sz[0] + h * a.sz[1] + at * a.sz[2]));
    io_traits<IO>::store(static_cast<IO*>(a.out) + b * a.so[0] + h * a.so[1] + at * a.so[2], y);
  }
}

template <typename IO, int LPR>
hipError_t launch_lpr(const HeadStepArgs& a, hipStream_t stream) {
  constexpr int RP = 256 / LPR;
  const int passes = (a.headdim + RP - 1) / RP;
  int np = passes >= 8 ? 8 : passes >= 4 ? 4 : passes >= 2 ? 2 : 1;
  // fewer workgroups than CUs: smaller tiles, so that the states come through more
  // of them (one row of 24 heads of 64 x 128 in a graph: 6.6 us, 7.5 us at eight
  // columns a thread); more workgroups than that only filter B and C more often
  // (8 rows of 80 heads: 10.9 us at 640 workgroups, 11.3 us at 1280)
  while (np > 1 && static_cast<int64_t>(a.rows) * a.heads * ((passes + np - 1) / np) < 256) np /= 2;
  const int ptiles = (passes + np - 1) / np;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.rows) * a.heads * ptiles)), block(256);
  switch (np) {
    case 1: head_step_kernel<IO, LPR, 1><<<grid, block, 0, stream>>>(a, ptiles); break;
    case 2: head_step_kernel<IO, LPR, 2><<<grid, block, 0, stream>>>(a, ptiles); break;
    case 4: head_step_kernel<IO, LPR, 4><<<grid, block, 0, stream>>>(a, ptiles); break;
    default: head_step_kernel<IO, LPR, 8><<<grid, block, 0, stream>>>(a, ptiles); break;
  }
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_t(const HeadStepArgs& a, hipStream_t stream) {
  hipError_t e;
  if (a.dstate <= 16) e = launch_lpr<IO, 4>(a, stream);
  else if (a.dstate <= 32) e = launch_lpr<IO, 8>(a, stream);
  else if (a.dstate <= 64) e = launch_lpr<IO, 16>(a, stream);
  else e = launch_lpr<IO, 32>(a, stream);
  if (e != hipSuccess || a.width == 1) return e;
  const int bc = 2 * a.groups * a.dstate;
  const int64_t n = static_cast<int64_t>(a.rows) * bc;
  head_step_slide_kernel<IO><<<dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, stream>>>(a, bc);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_head_step(const HeadStepArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_t<bf16_t>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace mss

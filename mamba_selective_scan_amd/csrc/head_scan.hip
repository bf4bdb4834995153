// head_scan.hip -- head-wise selective scan over packed prompts, gfx950.
#include "mss_head.hpp"

namespace mss {
namespace {

// One wave per four columns of a head of one prompt, walking it token by token:
// 16 lanes hold a column's states.
template <typename IO>
__global__ __launch_bounds__(256) void head_scan_walk_kernel(HeadScanArgs a, int ptiles) {
  constexpr int K = kMaxHeadState / 16;
  int64_t id = blockIdx.x;
  const int tile = static_cast<int>(id % ptiles);
  id /= ptiles;
  const int h = static_cast<int>(id % a.heads);
  const int s = static_cast<int>(id / a.heads);
  const int slot = slot_of(a.q.slots, a.q.cache_slots, s);
  if (slot < 0) return;
  const Span sp = prompt_span(a.q, s);
  const bool from_cache = resumes(a.q, s);
  const int l = threadIdx.x & 15;
  const int p = tile * 16 + threadIdx.x / 16;
  const bool valid = p < a.headdim;
  const int pp = valid ? p : 0;
  const int g = h / (a.heads / a.groups);
  float* cache = a.state + slot * a.sstate + (static_cast<int64_t>(h) * a.headdim + pp) * a.dstate;
  float st[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int n = l + 16 * k;
    st[k] = from_cache && n < a.dstate ? cache[n] : 0.0f;
  }
  const float a2 = -expf(a.A_log[h]) * kLog2e;
  const float bias = a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f;
  const float skip = a.D != nullptr ? a.D[h] : 0.0f;
  for (int64_t t = sp.begin; t < sp.end; ++t) {
    const float xr = io_traits<IO>::load(static_cast<const IO*>(a.dt) + t * a.sdt[0] + h * a.sdt[1]) + bias;
    const float dl = a.softplus ? softplus(xr) : xr;
    const float decay = fast_exp2(dl * a2);
    const float x = io_traits<IO>::load(static_cast<const IO*>(a.x) + t * a.sx[0] + h * a.sx[1] + pp);
    const IO* B = static_cast<const IO*>(a.B) + t * a.sB[0] + g * a.sB[1];
    const IO* C = static_cast<const IO*>(a.C) + t * a.sC[0] + g * a.sC[1];
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int n = l + 16 * k;
      const float bn = n < a.dstate ? io_traits<IO>::load(B + n) : 0.0f;
      const float cn = n < a.dstate ? io_traits<IO>::load(C + n) : 0.0f;
      st[k] = fmaf(decay, st[k], dl * x * bn);
      y = fmaf(cn, st[k], y);
    }
    y = row_sum16(y);
    if (valid && l == 0) {
      y = fmaf(skip, x, y);
      if (a.z != nullptr)
        y *= silu(io_traits<IO>::load(static_cast<const IO*>(a.z) + t * a.sz[0] + h * a.sz[1] + p));
      io_traits<IO>::store(static_cast<IO*>(a.out) + t * a.so[0] + h * a.so[1] + p, y);
    }
  }
  if (sp.end == sp.begin && from_cache) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int n = l + 16 * k;
    if (valid && n < a.dstate) cache[n] = st[k];
  }
}

}  // namespace

hipError_t launch_head_scan(const HeadScanArgs& a, bool io_bf16, hipStream_t stream) {
  const int ptiles = (a.headdim + 15) / 16;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.q.seqs) * a.heads * ptiles)), block(256);
  if (io_bf16)
    head_scan_walk_kernel<bf16_t><<<grid, block, 0, stream>>>(a, ptiles);
  else
    head_scan_walk_kernel<float><<<grid, block, 0, stream>>>(a, ptiles);
  return hipGetLastError();
}

}  // namespace mss

// head_api.hip -- the C ABI of the head-wise operations: argument checks,
// launch planning and stream-ordered enqueue.  As in mss_api.hip, every check
// runs on the host before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "mss.h"
#include "mss_checks.hpp"
#include "mss_head.hpp"

namespace {

using mss::Extent;
using mss::aligned;
using mss::extent_of;
using mss::non_overlapping;
using mss::overlaps;
using mss::strides_nonneg;

constexpr int64_t kMaxInt = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1;  // of a launch
constexpr int64_t kMaxGroups = kMaxThreads / 256;        // workgroups of 256
constexpr int64_t kMaxTokens = int64_t{1} << 30;
constexpr int64_t kMaxSeqs = int64_t{1} << 20;
constexpr int64_t kMaxNormDim = 32768;
const int64_t kOne[1] = {1};

bool bad_dtype(int32_t t) { return t != MSS_F32 && t != MSS_BF16; }
int64_t elem(int32_t t) { return t == MSS_BF16 ? 2 : 4; }

Extent vec(const void* p, int64_t n, int64_t es) { return extent_of(p, &n, kOne, 1, es); }

// [slot][inner] with contiguous inner entries.
Extent cache_extent(const void* p, int64_t slots, int64_t inner, int64_t stride, int64_t es) {
  const int64_t sz[2] = {slots, inner}, st[2] = {stride, 1};
  return extent_of(p, sz, st, 2, es);
}
bool cache_stride_ok(int64_t slots, int64_t inner, int64_t stride) {
  return slots == 1 ? stride >= 0 : stride >= inner;
}

template <size_t N>
bool any_overlap(const Extent& e, const Extent (&ins)[N]) {
  for (const Extent& i : ins)
    if (overlaps(e, i)) return true;
  return false;
}

// Waves along the rows: short runs while they keep the grid small, so that a
// short prompt's rows are read in parallel, and runs of kConvRun rows otherwise.
constexpr int64_t kConvRun = 32;
constexpr int64_t kConvShortRun = 4;
constexpr int64_t kConvWaves = 4096;

mss_status check_head_shape(int64_t heads, int64_t headdim, int64_t dstate, int64_t groups) {
  if (heads < 1 || headdim < 1 || groups < 1 || heads > kMaxInt || headdim > kMaxInt ||
      groups > heads || heads % groups != 0)
    return MSS_ERR_BAD_SHAPE;
  if (dstate < 1 || dstate > MSS_MAX_HEAD_DSTATE) return MSS_ERR_UNSUPPORTED_DSTATE;
  if (heads * headdim > kMaxInt / 4 || groups * dstate > kMaxInt / 4) return MSS_ERR_BAD_SHAPE;
  return MSS_OK;
}

// How a head-wise scan is cut over time and over columns: prompts longer than
// seg_len run as segments, so that a few long prompts still fill the card, and
// tiles of 16 columns take the place of 32 while there are too few of those.
// From the sizes alone: the prompts' lengths stay on the device.
//
// One long prompt wants as many segments as workgroups can run at once and not
// one more (24 heads of 64 x 128, 32768 tokens in bf16: 220 us at 480 workgroups
// of 512, 249 us at 516; a prompt's last segment counts as half a one).  A cut
// call makes three passes: it takes more than five chunks to be worth it (320
// tokens: 32.1 us whole, 32.3 us cut; 512: 48 and 35), on the average of the
// prompts, as the lengths are not known here; then segments may be as short as
// two chunks (2048 tokens: 46 us at 128 tokens a segment, 51 us at 256).  Longer
// than kSegMax, a batch of equal prompts does not care (8 x 4096 tokens of 80
// heads: 629 us whole, 615 us at 1024) while one of unequal prompts would wait for
// its longest (24 prompts, 32768 tokens: 664 us at 1024, 737 us at 2560).
//
// Tiles of 16 columns do a chunk in three quarters of the time but form its decays
// twice: for calls that leave a quarter of the workgroup slots empty at 32 (200
// tokens of 24 heads: 27.2 us, 35.4 us at 32; 1000 tokens of 80 heads: 55 and 60;
// 2000 tokens of 80 heads, over that line: 82 and 77) and still run at once (8 x 200
// tokens of 80 heads, which do not: 62 and 58).
struct HeadScanPlan {
  bool narrow = false;
  int64_t ptiles, tiles, seg_len = 0, cut_slots = 0, cut_prompts = 0;
  size_t parts = 0, workspace = 0;
};
constexpr int64_t kCus = 256;
constexpr int64_t kSegMax = 1024;

HeadScanPlan head_scan_plan(const mss_head_scan_args* a) {
  HeadScanPlan p;
  const bool f32 = a->io_dtype == MSS_F32;
  const int64_t chunk = f32 ? 32 : 64;
  // workgroups a CU holds (by LDS and registers): three of the small fp32 kernels
  const int64_t slots = kCus * (f32 && a->dstate <= 64 ? 3 : 2);
  int64_t seg = 0;
  // the tiles of `cols` columns and their segments; returns the workgroups
  auto tile = [&](int64_t cols) {
    p.ptiles = (a->headdim + cols - 1) / cols;
    p.tiles = a->groups * ((a->heads / a->groups * p.ptiles + 3) / 4);
    const int64_t room = slots / p.tiles;
    const int64_t want = std::max<int64_t>({1, room / 2, room - a->seqs / 2});
    seg = ((a->tokens + want - 1) / want + chunk - 1) / chunk * chunk;
    seg = std::clamp(seg, (a->tokens > 5 * chunk * a->seqs ? 2 : 5) * chunk, kSegMax);
    return std::max(a->seqs, a->tokens / seg + a->seqs / 2) * p.tiles;
  };
  p.narrow = tile(32) < slots / 4 * 3 && tile(16) <= slots;
  if (!p.narrow) tile(32);
  if (a->tokens > seg) {
    // a cut prompt has more than seg tokens, so at most 2 len / seg segments, and
    // less than len / seg + 1
    p.seg_len = seg;
    p.cut_prompts = std::min(a->seqs, a->tokens / seg);
    p.cut_slots = std::min(2 * a->tokens / seg, a->tokens / seg + p.cut_prompts);
    const size_t states = static_cast<size_t>(a->heads * a->headdim * a->dstate) * 4;
    p.parts = (p.cut_slots * states + 255) / 256 * 256;
    p.workspace = p.parts + static_cast<size_t>(p.cut_slots * a->heads) * 4;
  }
  return p;
}

// The scan's sizes, and how it runs.
mss_status check_scan_shape(const mss_head_scan_args* a, HeadScanPlan* plan) {
  if (a == nullptr || a->struct_size != sizeof(mss_head_scan_args) || a->reserved0 != 0)
    return MSS_ERR_BAD_STRUCT;
  if (bad_dtype(a->io_dtype)) return MSS_ERR_UNSUPPORTED_DTYPE;
  if (a->tokens < 0 || a->tokens > kMaxTokens || a->seqs < 1 || a->seqs > kMaxSeqs ||
      a->cache_slots < 1 || a->cache_slots > kMaxInt)
    return MSS_ERR_BAD_SHAPE;
  const mss_status st = check_head_shape(a->heads, a->headdim, a->dstate, a->groups);
  if (st != MSS_OK) return st;
  *plan = head_scan_plan(a);
  if ((a->seqs + plan->cut_slots) * plan->tiles > kMaxGroups ||
      plan->cut_prompts * ((a->heads * a->headdim * a->dstate + 1023) / 1024) > kMaxGroups)
    return MSS_ERR_BAD_SHAPE;
  return MSS_OK;
}

mss_status check_step_shape(const mss_head_step_args* a) {
  if (a == nullptr || a->struct_size != sizeof(mss_head_step_args) || a->reserved0 != 0)
    return MSS_ERR_BAD_STRUCT;
  if (bad_dtype(a->io_dtype)) return MSS_ERR_UNSUPPORTED_DTYPE;
  if (a->rows < 1 || a->rows > kMaxInt || a->cache_slots < 1 || a->cache_slots > kMaxInt ||
      a->width < 1 || a->width > MSS_MAX_CONV_WIDTH)
    return MSS_ERR_BAD_SHAPE;
  const mss_status st = check_head_shape(a->heads, a->headdim, a->dstate, a->groups);
  if (st != MSS_OK) return st;
  const int64_t chans = a->heads * a->headdim + 2 * a->groups * a->dstate;
  // (a workgroup's columns are 64 or more, or at least half of the head's, once
  // there are 256 workgroups)
  if (chans > kMaxInt || a->rows > kMaxInt / chans ||
      a->rows * a->heads > kMaxGroups / (2 * ((a->headdim + 63) / 64)))
    return MSS_ERR_BAD_SHAPE;
  return MSS_OK;
}

mss::Prompts prompts(int64_t tokens, int64_t seqs, int64_t slots, const int32_t* cu,
                     const int32_t* slot, const int32_t* resume) {
  return {static_cast<int>(tokens), static_cast<int>(seqs), static_cast<int>(slots), cu, slot, resume};
}

}  // namespace

extern "C" {

mss_status mss_causal_conv1d_prompts(const mss_conv_prompts_args* a, void* stream) {
  if (a == nullptr || a->struct_size != sizeof(mss_conv_prompts_args) || a->reserved0 != 0)
    return MSS_ERR_BAD_STRUCT;
  if (bad_dtype(a->io_dtype)) return MSS_ERR_UNSUPPORTED_DTYPE;
  if (a->tokens < 0 || a->tokens > kMaxTokens || a->dim < 1 || a->dim > kMaxInt / 4 || a->width < 1 ||
      a->width > MSS_MAX_CONV_WIDTH || a->seqs < 1 || a->seqs > kMaxSeqs || a->cache_slots < 1 ||
      a->cache_slots > kMaxInt)
    return MSS_ERR_BAD_SHAPE;
  if (a->activation != MSS_ACT_NONE && a->activation != MSS_ACT_SILU) return MSS_ERR_BAD_STRUCT;
  const int64_t T = a->tokens, W = a->width, es = elem(a->io_dtype);
  const int64_t colgroups = (a->dim + 1024 / es - 1) / (1024 / es);  // a wave's 16 bytes a lane
  const int64_t run = std::clamp(T * colgroups / kConvWaves, kConvShortRun, kConvRun);
  const int64_t nruns = (T + run - 1) / run;
  if ((nruns + a->seqs) * colgroups > 4 * kMaxGroups) return MSS_ERR_BAD_SHAPE;
  if (a->weight == nullptr || a->cu_seqlens == nullptr || (W > 1 && a->window == nullptr) ||
      (T > 0 && (a->x == nullptr || a->out == nullptr)))
    return MSS_ERR_NULL_POINTER;
  if (!strides_nonneg(a->x_stride, 2) || !strides_nonneg(a->out_stride, 2) ||
      !strides_nonneg(a->weight_stride, 2))
    return MSS_ERR_BAD_STRIDE;
  const int64_t xs[2] = {T, a->dim}, ws[2] = {a->dim, W};
  if (T > 0 && !non_overlapping(xs, a->out_stride, 2)) return MSS_ERR_BAD_STRIDE;
  if (W > 1 && !cache_stride_ok(a->cache_slots, a->dim * (W - 1), a->window_stride))
    return MSS_ERR_BAD_STRIDE;
  if (!aligned(a->x, es) || !aligned(a->out, es) || !aligned(a->window, es) || !aligned(a->weight, 4) ||
      !aligned(a->bias, 4) || !aligned(a->cu_seqlens, 4) || !aligned(a->slots, 4) || !aligned(a->resume, 4))
    return MSS_ERR_MISALIGNED;
  const Extent ins[] = {T > 0 ? extent_of(a->x, xs, a->x_stride, 2, es) : Extent{},
                        extent_of(a->weight, ws, a->weight_stride, 2, 4),
                        vec(a->bias, a->dim, 4), vec(a->cu_seqlens, a->seqs + 1, 4),
                        vec(a->slots, a->seqs, 4), vec(a->resume, a->seqs, 4)};
  const Extent eo = T > 0 ? extent_of(a->out, xs, a->out_stride, 2, es) : Extent{};
  const Extent ew = W > 1 ? cache_extent(a->window, a->cache_slots, a->dim * (W - 1), a->window_stride, es)
                          : Extent{};
  if (any_overlap(eo, ins) || any_overlap(ew, ins) || overlaps(eo, ew)) return MSS_ERR_ALIASING;

  mss::ConvPromptsArgs k{};
  k.q = prompts(T, a->seqs, a->cache_slots, a->cu_seqlens, a->slots, a->resume);
  k.dim = static_cast<int>(a->dim);
  k.width = static_cast<int>(W);
  k.silu = a->activation == MSS_ACT_SILU ? 1 : 0;
  for (int i = 0; i < 2; ++i) {
    k.sx[i] = xs[i] == 1 ? 1 : a->x_stride[i];
    k.so[i] = xs[i] == 1 ? 1 : a->out_stride[i];
    k.sw[i] = a->weight_stride[i];
  }
  k.swin = a->window_stride;
  k.colgroups = static_cast<int>(colgroups);
  k.run = static_cast<int>(run);
  k.nruns = nruns;
  k.x = a->x;
  k.weight = a->weight;
  k.bias = a->bias;
  k.window = a->window;
  k.out = a->out;
  const hipError_t e = mss::launch_conv_prompts(k, a->io_dtype == MSS_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MSS_OK : MSS_ERR_HIP;
}

size_t mss_head_scan_prompts_workspace_size(const mss_head_scan_args* a, mss_status* status) {
  HeadScanPlan plan;
  const mss_status st = check_scan_shape(a, &plan);
  if (status != nullptr) *status = st;
  return st == MSS_OK ? plan.workspace : 0;
}

mss_status mss_head_scan_prompts(const mss_head_scan_args* a, void* stream) {
  HeadScanPlan plan;
  const mss_status shape = check_scan_shape(a, &plan);
  if (shape != MSS_OK) return shape;
  const int64_t T = a->tokens, H = a->heads, P = a->headdim, N = a->dstate, G = a->groups;
  const int64_t es = elem(a->io_dtype);
  if (a->A_log == nullptr || a->cu_seqlens == nullptr || a->state == nullptr ||
      (T > 0 && (a->x == nullptr || a->dt_raw == nullptr || a->B == nullptr || a->C == nullptr ||
                 a->out == nullptr)))
    return MSS_ERR_NULL_POINTER;
  if (!strides_nonneg(a->x_stride, 3) || !strides_nonneg(a->dt_stride, 2) || !strides_nonneg(a->B_stride, 3) ||
      !strides_nonneg(a->C_stride, 3) || (a->z != nullptr && !strides_nonneg(a->z_stride, 3)) ||
      !strides_nonneg(a->out_stride, 3))
    return MSS_ERR_BAD_STRIDE;
  if (T > 0 && ((P > 1 && (a->x_stride[2] != 1 || a->out_stride[2] != 1 ||
                           (a->z != nullptr && a->z_stride[2] != 1))) ||
                (N > 1 && (a->B_stride[2] != 1 || a->C_stride[2] != 1))))
    return MSS_ERR_BAD_STRIDE;
  // 64 rows of a tile are addressed with 32-bit byte offsets
  constexpr int64_t kMaxRow = (int64_t{1} << 31) / (65 * 4);
  if (T > 1 && (a->x_stride[0] > kMaxRow || a->B_stride[0] > kMaxRow || a->C_stride[0] > kMaxRow ||
                (a->z != nullptr && a->z_stride[0] > kMaxRow) || a->out_stride[0] > kMaxRow))
    return MSS_ERR_BAD_STRIDE;
  const int64_t xs[3] = {T, H, P}, ds[2] = {T, H}, bs[3] = {T, G, N};
  if (T > 0 && !non_overlapping(xs, a->out_stride, 3)) return MSS_ERR_BAD_STRIDE;
  if (H * P > kMaxInt * 64 / N || !cache_stride_ok(a->cache_slots, H * P * N, a->state_stride))
    return MSS_ERR_BAD_STRIDE;
  if (!aligned(a->x, es) || !aligned(a->dt_raw, es) || !aligned(a->B, es) || !aligned(a->C, es) ||
      !aligned(a->z, es) || !aligned(a->out, es) || !aligned(a->A_log, 4) || !aligned(a->D, 4) ||
      !aligned(a->dt_bias, 4) || !aligned(a->state, 4) || !aligned(a->cu_seqlens, 4) ||
      !aligned(a->slots, 4) || !aligned(a->resume, 4) || !aligned(a->workspace, 256))
    return MSS_ERR_MISALIGNED;
  const bool any = T > 0;
  const Extent none{};
  const Extent ins[] = {any ? extent_of(a->x, xs, a->x_stride, 3, es) : none,
                        any ? extent_of(a->dt_raw, ds, a->dt_stride, 2, es) : none,
                        any ? extent_of(a->B, bs, a->B_stride, 3, es) : none,
                        any ? extent_of(a->C, bs, a->C_stride, 3, es) : none,
                        any ? extent_of(a->z, xs, a->z_stride, 3, es) : none,
                        vec(a->A_log, H, 4), vec(a->D, H, 4), vec(a->dt_bias, H, 4),
                        vec(a->cu_seqlens, a->seqs + 1, 4), vec(a->slots, a->seqs, 4),
                        vec(a->resume, a->seqs, 4)};
  const Extent eo = any ? extent_of(a->out, xs, a->out_stride, 3, es) : none;
  const Extent es_ = cache_extent(a->state, a->cache_slots, H * P * N, a->state_stride, 4);
  if (any_overlap(eo, ins) || any_overlap(es_, ins) || overlaps(eo, es_)) return MSS_ERR_ALIASING;
  if (plan.workspace > 0) {
    if (a->workspace == nullptr || a->workspace_bytes < plan.workspace) return MSS_ERR_WORKSPACE_TOO_SMALL;
    const Extent ew = vec(a->workspace, static_cast<int64_t>(plan.workspace), 1);
    if (any_overlap(ew, ins) || overlaps(ew, eo) || overlaps(ew, es_)) return MSS_ERR_ALIASING;
  }

  mss::HeadScanArgs k{};
  // 16-byte vectors: every row start aligned, every row a whole number of them
  // and before the next one
  const int64_t V = 16 / es;
  auto vectors = [&](const void* p, const int64_t* st, int64_t outer, int64_t inner) {
    return aligned(p, 16) && st[0] % V == 0 && st[0] >= inner && st[0] <= kMaxRow &&
           (outer == 1 || st[1] % V == 0) && inner % V == 0;
  };
  // 8 columns at a time leave the kernel, whatever the type
  k.vec = any && P % 8 == 0 && vectors(a->x, a->x_stride, H, P) && vectors(a->B, a->B_stride, G, N) &&
          vectors(a->C, a->C_stride, G, N) && vectors(a->out, a->out_stride, H, P) &&
          (a->z == nullptr || vectors(a->z, a->z_stride, H, P));
  k.narrow = k.vec && plan.narrow;
  k.ptiles = static_cast<int>(plan.narrow && !k.vec ? (P + 31) / 32 : plan.ptiles);
  k.seg_len = static_cast<int>(plan.seg_len);
  k.cut_slots = static_cast<int>(plan.cut_slots);
  k.cut_prompts = static_cast<int>(plan.cut_prompts);
  k.parts = static_cast<float*>(a->workspace);
  k.decays = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + plan.parts);
  k.q = prompts(T, a->seqs, a->cache_slots, a->cu_seqlens, a->slots, a->resume);
  k.heads = static_cast<int>(H);
  k.headdim = static_cast<int>(P);
  k.dstate = static_cast<int>(N);
  k.groups = static_cast<int>(G);
  k.softplus = a->delta_softplus != 0 ? 1 : 0;
  std::memcpy(k.sx, a->x_stride, sizeof(k.sx));
  std::memcpy(k.sdt, a->dt_stride, sizeof(k.sdt));
  std::memcpy(k.sB, a->B_stride, sizeof(k.sB));
  std::memcpy(k.sC, a->C_stride, sizeof(k.sC));
  std::memcpy(k.sz, a->z_stride, sizeof(k.sz));
  std::memcpy(k.so, a->out_stride, sizeof(k.so));
  k.sstate = a->state_stride;
  k.x = a->x;
  k.dt = a->dt_raw;
  k.A_log = a->A_log;
  k.B = a->B;
  k.C = a->C;
  k.D = a->D;
  k.z = a->z;
  k.dt_bias = a->dt_bias;
  k.state = a->state;
  k.out = a->out;
  const hipError_t e = mss::launch_head_scan(k, a->io_dtype == MSS_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MSS_OK : MSS_ERR_HIP;
}

mss_status mss_head_scan_step(const mss_head_step_args* a, void* stream) {
  const mss_status shape = check_step_shape(a);
  if (shape != MSS_OK) return shape;
  const int64_t R = a->rows, H = a->heads, P = a->headdim, N = a->dstate, G = a->groups, W = a->width;
  const int64_t es = elem(a->io_dtype), chans = H * P + 2 * G * N;
  if (a->state == nullptr || (W > 1 && a->window == nullptr) || a->xbc == nullptr || a->dt_raw == nullptr ||
      a->A_log == nullptr || a->weight == nullptr || a->out == nullptr)
    return MSS_ERR_NULL_POINTER;
  if (!strides_nonneg(a->xbc_stride, 2) || !strides_nonneg(a->dt_stride, 2) ||
      !strides_nonneg(a->weight_stride, 2) || (a->z != nullptr && !strides_nonneg(a->z_stride, 3)) ||
      !strides_nonneg(a->out_stride, 3))
    return MSS_ERR_BAD_STRIDE;
  const int64_t xs[2] = {R, chans}, ds[2] = {R, H}, ws[2] = {chans, W}, os[3] = {R, H, P};
  if (!non_overlapping(os, a->out_stride, 3)) return MSS_ERR_BAD_STRIDE;
  if (!cache_stride_ok(a->cache_slots, H * P * N, a->state_stride) ||
      (W > 1 && !cache_stride_ok(a->cache_slots, chans * (W - 1), a->window_stride)))
    return MSS_ERR_BAD_STRIDE;
  if (!aligned(a->state, 4) || !aligned(a->window, es) || !aligned(a->xbc, es) || !aligned(a->dt_raw, es) ||
      !aligned(a->z, es) || !aligned(a->out, es) || !aligned(a->A_log, 4) || !aligned(a->weight, 4) ||
      !aligned(a->bias, 4) || !aligned(a->D, 4) || !aligned(a->dt_bias, 4) || !aligned(a->slots, 4))
    return MSS_ERR_MISALIGNED;
  const Extent ins[] = {extent_of(a->xbc, xs, a->xbc_stride, 2, es), extent_of(a->dt_raw, ds, a->dt_stride, 2, es),
                        extent_of(a->z, os, a->z_stride, 3, es), extent_of(a->weight, ws, a->weight_stride, 2, 4),
                        vec(a->A_log, H, 4), vec(a->bias, chans, 4), vec(a->D, H, 4), vec(a->dt_bias, H, 4),
                        vec(a->slots, R, 4)};
  const Extent outs[] = {extent_of(a->out, os, a->out_stride, 3, es),
                         cache_extent(a->state, a->cache_slots, H * P * N, a->state_stride, 4),
                         W > 1 ? cache_extent(a->window, a->cache_slots, chans * (W - 1), a->window_stride, es)
                               : Extent{}};
  for (int i = 0; i < 3; ++i) {
    if (any_overlap(outs[i], ins)) return MSS_ERR_ALIASING;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return MSS_ERR_ALIASING;
  }

  mss::HeadStepArgs k{};
  k.rows = static_cast<int>(R);
  k.heads = static_cast<int>(H);
  k.headdim = static_cast<int>(P);
  k.dstate = static_cast<int>(N);
  k.groups = static_cast<int>(G);
  k.width = static_cast<int>(W);
  k.softplus = a->delta_softplus != 0 ? 1 : 0;
  k.cache_slots = static_cast<int>(a->cache_slots);
  std::memcpy(k.sx, a->xbc_stride, sizeof(k.sx));
  std::memcpy(k.sdt, a->dt_stride, sizeof(k.sdt));
  std::memcpy(k.sw, a->weight_stride, sizeof(k.sw));
  std::memcpy(k.sz, a->z_stride, sizeof(k.sz));
  std::memcpy(k.so, a->out_stride, sizeof(k.so));
  k.sstate = a->state_stride;
  k.swin = a->window_stride;
  k.xbc = a->xbc;
  k.dt = a->dt_raw;
  k.A_log = a->A_log;
  k.weight = a->weight;
  k.bias = a->bias;
  k.D = a->D;
  k.z = a->z;
  k.dt_bias = a->dt_bias;
  k.slots = a->slots;
  k.state = a->state;
  k.window = a->window;
  k.out = a->out;
  const hipError_t e = mss::launch_head_step(k, a->io_dtype == MSS_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MSS_OK : MSS_ERR_HIP;
}

mss_status mss_rms_norm(const mss_norm_args* a, void* stream) {
  if (a == nullptr || a->struct_size != sizeof(mss_norm_args) || a->reserved0 != 0) return MSS_ERR_BAD_STRUCT;
  if (bad_dtype(a->io_dtype) || bad_dtype(a->residual_dtype)) return MSS_ERR_UNSUPPORTED_DTYPE;
  if (a->quant != MSS_QUANT_NONE && a->quant != MSS_QUANT_ROW && a->quant != MSS_QUANT_BLOCK)
    return MSS_ERR_BAD_STRUCT;
  const int64_t R = a->rows, D = a->dim;
  if (R < 1 || R > kMaxInt || D < 1 || D > kMaxNormDim ||
      (a->quant == MSS_QUANT_BLOCK && D % MSS_SCALE_BLOCK != 0) || !(a->eps >= 0.0f) ||
      R > kMaxThreads / (D <= 2048 ? 64 : D <= 8192 ? 256 : 1024) - 3)
    return MSS_ERR_BAD_SHAPE;
  if (a->x == nullptr || a->weight == nullptr || a->out == nullptr ||
      (a->quant != MSS_QUANT_NONE && a->scale == nullptr))
    return MSS_ERR_NULL_POINTER;
  const int64_t es = elem(a->io_dtype), rs = elem(a->residual_dtype);
  const int64_t eso = a->quant == MSS_QUANT_NONE ? es : 1;
  const bool in_place = a->residual_out != nullptr && a->residual_out == a->residual;
  if (a->x_stride < 0 || (a->residual != nullptr && a->residual_stride < 0) ||
      (R > 1 && (a->out_stride < D || (a->residual_out != nullptr && a->residual_out_stride < D) ||
                 (in_place && a->residual_out_stride != a->residual_stride))))
    return MSS_ERR_BAD_STRIDE;
  if (!aligned(a->x, es) || !aligned(a->residual, rs) || !aligned(a->weight, 4) || !aligned(a->out, eso) ||
      !aligned(a->scale, 4) || !aligned(a->residual_out, rs))
    return MSS_ERR_MISALIGNED;
  const int64_t sz[2] = {R, D};
  auto rows = [&](const void* p, int64_t stride, int64_t e) {
    const int64_t st[2] = {stride, 1};
    return extent_of(p, sz, st, 2, e);
  };
  const int64_t nscale = a->quant == MSS_QUANT_BLOCK ? R * (D / MSS_SCALE_BLOCK) : R;
  const Extent ex = rows(a->x, a->x_stride, es), er = rows(a->residual, a->residual_stride, rs);
  const Extent ew = vec(a->weight, D, 4);
  const Extent eo = rows(a->out, a->out_stride, eso), ero = rows(a->residual_out, a->residual_out_stride, rs);
  const Extent esc = a->quant == MSS_QUANT_NONE ? Extent{} : vec(a->scale, nscale, 4);
  const Extent ins[] = {ex, er, ew};
  if (any_overlap(eo, ins) || any_overlap(esc, ins) || overlaps(ero, ex) || overlaps(ero, ew) ||
      (!in_place && overlaps(ero, er)) || overlaps(eo, ero) || overlaps(eo, esc) || overlaps(ero, esc))
    return MSS_ERR_ALIASING;
  mss::NormArgs k{};
  k.rows = R;
  k.dim = static_cast<int>(D);
  k.sx = a->x_stride;
  k.sr = a->residual_stride;
  k.so = a->out_stride;
  k.sro = a->residual_out_stride;
  k.eps = a->eps;
  k.x = a->x;
  k.res = a->residual;
  k.weight = a->weight;
  k.out = a->out;
  k.scale = a->scale;
  k.res_out = a->residual_out;
  const hipError_t e = mss::launch_norm(k, a->io_dtype == MSS_BF16, a->residual_dtype == MSS_BF16, a->quant,
                                        static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MSS_OK : MSS_ERR_HIP;
}

}  // extern "C"

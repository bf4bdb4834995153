// vocab_loss.hip -- cross entropy and distillation over a vocabulary: which rows
// count, their targets' logits, the softmax and its gradient, gfx950.  The three
// products are in vocab_gemm.hip.
//
// Rows that count are packed one behind another (x, and everything that is
// computed of it), so that ignored rows cost no products, and whatever they hold
// reaches nothing.
#include "mss.h"
#include "mss_train.hpp"
#include "vocab_gemm.hpp"

namespace mss {
namespace {

__device__ inline float wave_sum(float v) {
  v = row_sum16(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}
// (a NaN is dropped: the sums behind it keep it)
__device__ inline float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

__device__ inline float teacher_at(const LossArgs& a, int64_t row, int k) {
  const int64_t i = row * a.steach[0] + k * a.steach[1];
  return a.teacher_bf16 ? io_traits<bf16_t>::load(static_cast<const bf16_t*>(a.teacher) + i)
                        : static_cast<const float*>(a.teacher)[i];
}
__device__ inline int id_at(const LossArgs& a, int64_t row, int k) {
  const int64_t id = a.ids[row * a.sids[0] + k * a.sids[1]];
  return id >= 0 && id < a.vocab ? static_cast<int>(id) : -1;
}

// One wave a row: whether it counts, and the shares of its entries.
__global__ __launch_bounds__(256) void rows_kernel(LossArgs a) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (row >= a.rows) return;
  bool any = false;
  float top = -INFINITY;
  for (int k = lane; k < a.entries; k += 64) {
    const bool on = id_at(a, row, k) >= 0;
    any |= on;
    if (on && a.teacher != nullptr) top = fmaxf(top, teacher_at(a, row, k));
  }
  any = __any(any);
  if (lane == 0) {
    a.counts[row] = any ? 1 : 0;
    if (!any) a.loss[row] = a.lse[row] = 0.0f;
  }
  if (!any || a.teacher == nullptr) return;
  top = wave_max(top);
  float sum = 0.0f;
  for (int k = lane; k < a.entries; k += 64)
    if (id_at(a, row, k) >= 0) sum += expf((teacher_at(a, row, k) - top) * a.inv_tau);
  sum = wave_sum(sum);
  const float log_sum = logf(sum);
  float known = 0.0f;
  for (int k = lane; k < a.entries; k += 64) {
    float t = 0.0f;
    if (id_at(a, row, k) >= 0) {
      const float u = (teacher_at(a, row, k) - top) * a.inv_tau;
      t = expf(u) / sum;
      if (t != 0.0f) known += t * (u - log_sum);
    }
    a.share[static_cast<int64_t>(row) * a.entries + k] = t;
  }
  known = wave_sum(known);
  if (lane == 0) a.known[row] = known;
}

// The rows that count, in order: one workgroup, 4 rows a thread at a time.
__global__ __launch_bounds__(1024) void place_kernel(LossArgs a) {
  __shared__ int waves[16];
  int base = 0;
  for (int first = 0; first < a.rows; first += 4096) {
    const int r0 = first + threadIdx.x * 4;
    int on[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      on[i] = r0 + i < a.rows ? a.counts[r0 + i] : 0;
      n += on[i];
    }
    int upto = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      if (static_cast<int>(threadIdx.x & 63) >= o) upto += v;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) waves[threadIdx.x >> 6] = upto;
    __syncthreads();
    int at = base + upto - n;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < static_cast<int>(threadIdx.x >> 6)) at += waves[i];
      base += waves[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i < a.rows) {
        a.place[r0 + i] = on[i] ? at : -1;
        if (on[i]) a.row_of[at++] = r0 + i;
      }
  }
  if (threadIdx.x == 0) *a.live = base;
}

// An fp32 value as the sum of three bf16 ones (exact: 3 x 8 bits), or a bf16 one.
template <typename IO>
__device__ inline void to_planes(float v, uint16_t* p, int64_t plane, int planes) {
  for (int i = 0; i < planes; ++i) {
    const uint16_t q = bf16_bits(v);
    p[i * plane] = q;
    v -= __uint_as_float(static_cast<uint32_t>(q) << 16);
  }
}

constexpr int kMaxWords = (1 << 22) / 64 / 32;  // of the largest vocabulary's tiles

// One workgroup a row that counts: its x as an operand, its ids, and the tiles of
// the vocabulary that hold one.
template <typename IO>
__global__ __launch_bounds__(256) void pack_kernel(LossArgs a, int tile_shift) {
  const int j = blockIdx.x;
  if (j >= *a.live) return;
  const int row = a.row_of[j];
  const IO* x = static_cast<const IO*>(a.x) + row * a.sx;
  uint16_t* xp = a.xp + j * a.dpad;
  const int64_t plane = static_cast<int64_t>(a.rows) * a.dpad;
  __shared__ uint32_t where[kMaxWords];
  for (int i = threadIdx.x; i < a.where_words; i += 256) where[i] = 0;
  for (int c = threadIdx.x; c < a.dpad; c += 256)
    to_planes<IO>(c < a.dim ? io_traits<IO>::load(x + c) : 0.0f, xp + c, plane, a.planes);
  __syncthreads();
  for (int k = threadIdx.x; k < a.entries; k += 256) {
    const int id = id_at(a, row, k);
    a.near[static_cast<int64_t>(j) * a.entries + k] = id;
    if (id >= 0) atomicOr(where + (id >> tile_shift >> 5), 1u << (id >> tile_shift & 31));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.where_words; i += 256) a.where[static_cast<int64_t>(j) * a.where_words + i] = where[i];
}

template <typename IO>
__global__ __launch_bounds__(256) void pack_weight_kernel(LossArgs a) {
  const int v = blockIdx.x;
  const IO* w = static_cast<const IO*>(a.weight) + v * a.sw;
  for (int c = threadIdx.x; c < a.dpad; c += 256)
    to_planes<IO>(c < a.dim ? io_traits<IO>::load(w + c) : 0.0f, a.wp + v * a.dpad + c, a.wp_plane, a.planes);
}

// A row's sum of e^z from its tiles, as sum e^from with an integer `from`, so that
// a logit's distance from it keeps its last bits.  Every thread of the workgroup
// takes part and has it.
struct RowSum {
  float from, sum;
};
__device__ inline RowSum row_sum(const LossArgs& a, int i, float* meet) {
  const float2* st = a.stats + static_cast<int64_t>(i) * a.tiles;
  float top = -INFINITY;
  for (int t = threadIdx.x; t < a.tiles; t += 256) top = fmaxf(top, st[t].x);
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) meet[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(meet[0], meet[1]), fmaxf(meet[2], meet[3]));
  const float from = top == -INFINITY ? 0.0f : top;
  float s = 0.0f;
  for (int t = threadIdx.x; t < a.tiles; t += 256) s += st[t].y * expf(st[t].x - from);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) meet[4 + (threadIdx.x >> 6)] = s;
  __syncthreads();
  s = (meet[4] + meet[5]) + (meet[6] + meet[7]);
  return {from, s};
}

// Loss and gradient of the rows of a piece: a workgroup of row i writes loss and
// lse (blockIdx.y 0) and its columns of dz.
template <typename IO>
__global__ __launch_bounds__(256) void softmax_kernel(LossArgs a, int first, bool grad, int cols, int tile_shift) {
  __shared__ float meet[8];
  __shared__ int2 lost[4];
  const int i = blockIdx.x, j = first + i, live = *a.live;
  if (j >= live) return;
  const int row = a.row_of[j];
  const RowSum all = row_sum(a, i, meet);
  const int* near = a.near + static_cast<int64_t>(j) * a.entries;
  const float* picked = a.picked + static_cast<int64_t>(j) * a.entries;
  const float* share = a.teacher != nullptr ? a.share + static_cast<int64_t>(row) * a.entries : nullptr;
  if (blockIdx.y == 0) {
    const float log_sum = logf(all.sum);
    float s = 0.0f;
    for (int k = threadIdx.x; k < a.entries; k += 256)
      if (near[k] >= 0) {
        const float t = share != nullptr ? share[k] : 1.0f;
        if (t != 0.0f) s += t * ((all.from - picked[k]) + log_sum);
      }
    s = wave_sum(s);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) meet[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = (meet[0] + meet[1]) + (meet[2] + meet[3]);
      a.loss[row] = a.tau2 * (share != nullptr ? s + a.known[row] : s);
      a.lse[row] = all.from + log_sum;
    }
  }
  if (!grad) return;
  const float c = (a.row_weight != nullptr ? a.row_weight[row] : 1.0f / static_cast<float>(live)) * a.back;
  const float by = c / all.sum;
  const int c0 = blockIdx.y * cols, c1 = min(c0 + cols, static_cast<int>(a.vpad));
  const float2* st = a.stats + static_cast<int64_t>(i) * a.tiles;
  const int64_t plane = static_cast<int64_t>(a.piece) * a.vpad;
  uint16_t* dz = a.dz + i * a.vpad;
  for (int v = c0 + threadIdx.x; v < c1; v += 256) {
    float p = 0.0f;
    if (v < a.vocab) {
      float z;
      if constexpr (sizeof(IO) == 2) {
        const int code = static_cast<const uint16_t*>(a.probs)[i * a.vpad + v];
        z = code == 65535 ? -INFINITY : st[v >> tile_shift].x - static_cast<float>(code) * (1.0f / kCodeSteps);
      } else {
        z = static_cast<const float*>(a.probs)[i * a.vpad + v];
      }
      p = expf(z - all.from) * by;
    }
    to_planes<IO>(p, dz + v, plane, a.planes);
  }
  __syncthreads();
  float most = 0.0f;
  int2 best = make_int2(-1, 0);
  for (int k = threadIdx.x; k < a.entries; k += 256) {
    const int id = near[k];
    if (id < c0 || id >= c1) continue;
    float t = 1.0f;
    if (share != nullptr) {  // all shares of this id
      t = 0.0f;
      for (int q = 0; q < a.entries; ++q)
        if (near[q] == id) t += share[q];
    }
    const float v = fmaf(-t, all.sum, expf(picked[k] - all.from)) * by;
    to_planes<IO>(v, dz + id, plane, a.planes);
    const float miss = v - __uint_as_float(static_cast<uint32_t>(bf16_bits(v)) << 16);
    if (fabsf(miss) > most) {
      most = fabsf(miss);
      best = make_int2(id, __float_as_int(miss));
    }
  }
  if constexpr (sizeof(IO) == 2) {
    // the entry that lost most, of equal ones the one with the lowest id
    auto better = [](int2 p, int2 q) __attribute__((always_inline)) {
      const float x = fabsf(__int_as_float(p.y)), y = fabsf(__int_as_float(q.y));
      return x > y || (x == y && p.x < q.x);
    };
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const int2 q = make_int2(__shfl_xor(best.x, o, 64), __shfl_xor(best.y, o, 64));
      if (better(q, best)) best = q;
    }
    if ((threadIdx.x & 63) == 0) lost[threadIdx.x >> 6] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < 4; ++w)
        if (better(lost[w], best)) best = lost[w];
      a.fix[i * a.fixes + blockIdx.y] = best;
    }
  }
}

// The sum of c loss, in 64 bits and a fixed order; rows that do not count have
// no part in it, whatever their weights.
__global__ __launch_bounds__(1024) void total_kernel(LossArgs a) {
  __shared__ double meet[16];
  const int live = *a.live;
  double s = 0.0;
  for (int j = threadIdx.x; j < live; j += 1024) {
    const int row = a.row_of[j];
    s += static_cast<double>(a.loss[row]) * (a.row_weight != nullptr ? a.row_weight[row] : 1.0f);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) meet[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = 0.0;
  for (int i = 0; i < 16; ++i) s += meet[i];
  *a.total = static_cast<float>(a.row_weight != nullptr ? s : s / max(live, 1));
}

// dx of every row: the splits' sums of a row of this piece and what its dz lost, 0
// for one that does not count.
template <typename IO>
__global__ __launch_bounds__(256) void dx_kernel(LossArgs a, int first) {
  const int row = blockIdx.x, j = a.place[row];
  if (j < 0 ? first != 0 : j < first || j >= first + a.piece) return;
  const int splits = dx_splits(a, dx_tiles(a, min(a.piece, *a.live - first)));
  for (int c = threadIdx.x; c < a.dim; c += 256) {
    float s = 0.0f;
    if (j >= 0)
      for (int q = 0; q < splits; ++q)
        s += a.part[(static_cast<int64_t>(q) * a.piece + (j - first)) * a.dpad + c];
    if (sizeof(IO) == 2 && j >= 0)
      for (int q = 0; q < a.fixes; ++q) {
        const int2 f = a.fix[(j - first) * a.fixes + q];
        if (f.x >= 0) s = fmaf(__int_as_float(f.y), io_traits<IO>::load(static_cast<const IO*>(a.weight) + f.x * a.sw + c), s);
      }
    io_traits<IO>::store(static_cast<IO*>(a.dx) + row * a.sdx + c, s);
  }
}

template <typename IO>
__global__ __launch_bounds__(256) void dw_kernel(LossArgs a) {
  const int64_t v = blockIdx.x;
  for (int c = threadIdx.x; c < a.dim; c += 256)
    io_traits<IO>::store(static_cast<IO*>(a.dweight) + v * a.sdw + c, a.dw_sum[v * a.dpad + c]);
}

template <typename IO>
__global__ __launch_bounds__(256) void scale_kernel(const IO* in, const float* factor, IO* out, int64_t n) {
  const float f = *factor;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    io_traits<IO>::store(out + i, io_traits<IO>::load(in + i) * f);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

template <typename IO>
hipError_t launch_io(const LossArgs& a, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.rows);
  const bool grad = a.dx != nullptr || a.dweight != nullptr;
  if (rows > 0) rows_kernel<<<(rows + 3) / 4, 256, 0, s>>>(a);
  place_kernel<<<1, 1024, 0, s>>>(a);
  if (rows == 0) {  // (dweight and the total are 0)
    if (a.total != nullptr) total_kernel<<<1, 1024, 0, s>>>(a);
    return a.dweight != nullptr ? launch_dw(a, 0, sizeof(IO) == 2, s) : hipGetLastError();
  }
  const int shift = loss_vocab_tile(a.small) == 64 ? 6 : 7;
  pack_kernel<IO><<<rows, 256, 0, s>>>(a, shift);
  if (a.pack_w) pack_weight_kernel<IO><<<static_cast<unsigned>(a.vocab), 256, 0, s>>>(a);
  for (int p = 0; p < a.pieces; ++p) {
    const int first = p * a.piece;
    const unsigned n = static_cast<unsigned>(std::min(a.piece, a.rows - first));
    hipError_t e = launch_logits(a, first, sizeof(IO) == 2, grad, s);
    if (e != hipSuccess) return e;
    const int64_t cols = grad ? up256((a.vpad + a.fixes - 1) / a.fixes) : a.vpad;
    softmax_kernel<IO><<<dim3(n, grad ? a.fixes : 1), 256, 0, s>>>(a, first, grad, static_cast<int>(cols), shift);
    if (a.dx != nullptr) {
      if ((e = launch_dx(a, first, s)) != hipSuccess) return e;
      dx_kernel<IO><<<rows, 256, 0, s>>>(a, first);
    }
    if (a.dweight != nullptr && (e = launch_dw(a, first, sizeof(IO) == 2, s)) != hipSuccess) return e;
  }
  if (a.total != nullptr) total_kernel<<<1, 1024, 0, s>>>(a);
  if (a.dweight != nullptr && a.pieces > 1)
    dw_kernel<IO><<<static_cast<unsigned>(a.vocab), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_loss(const LossArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_io<bf16_t>(a, stream) : launch_io<float>(a, stream);
}

hipError_t launch_scale(const void* in, const float* factor, void* out, int64_t n, bool bf16,
                        hipStream_t stream) {
  const unsigned g = static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 8192));
  if (bf16)
    scale_kernel<<<g, 256, 0, stream>>>(static_cast<const bf16_t*>(in), factor, static_cast<bf16_t*>(out), n);
  else
    scale_kernel<<<g, 256, 0, stream>>>(static_cast<const float*>(in), factor, static_cast<float*>(out), n);
  return hipGetLastError();
}

}  // namespace mss

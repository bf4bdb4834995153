// vocab_gemm.hip -- the three products of the losses over a vocabulary, gfx950:
//   logits  z[i, v]     = scale sum_d x[i, d] w[v, d], with each tile's softmax sums
//   dx      part[i, d]  = sum_v dz[i, v] w[v, d], cut over v
//   dweight dw[v, d]    = sum_i dz[i, v] x[i, d]
//
// Operands are bf16 planes: one, or three whose sum is an fp32 value.  The
// product of two values in three planes takes the six products of planes whose
// orders sum to at most two; what is left out is below 2^-24 of it.
//
// A workgroup's tile of the product stays in its waves' accumulators.  Tiles of
// both operands, 64 of the summed axis at a time, go from memory into one of two
// LDS stages past the registers while the matrix instructions work from the
// other; one barrier a step.  An operand whose summed axis is contiguous lies in
// LDS as rows of 128 bytes and is read 16 bytes a lane; one whose other axis is
// contiguous lies there as it does in memory and is read through the transposing
// LDS read.  LDS loads put a lane's 16 bytes behind those of the lane before it,
// so that the swizzles that keep the reads free of bank conflicts are applied to
// the addresses in memory.  Rows past an operand's end lie past its buffer's
// range and read 0.
#include "mss.h"
#include "vocab_gemm.hpp"

namespace mss {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
#define MSS_LDS __attribute__((address_space(3)))

constexpr int kStep = 64;  // of the summed axis

// One operand of a tile, in bytes: rows of the tile's axis from `base` on, or rows
// of the summed one with the tile's axis contiguous.  A row is `stride` behind the
// one before it, its columns 64 .. 127 are `panel` behind its columns 0 .. 63.
// `span` from base on may be read (of a plane).
struct Side {
  const char* base;
  int64_t plane, span, panel;
  int stride;
};

__device__ inline int plane_of(int pair, bool second) {
  // (0,0) (0,1) (1,0) (0,2) (1,1) (2,0), two bits each
  return (second ? 0x184 : 0x910) >> (2 * pair) & 3;
}

// How ROWS rows (KC: of the tile's axis, 64 wide; else 64 rows of the summed axis,
// ROWS wide) of one operand lie in LDS, are loaded by NT threads, and are read as
// the fragments of 32 x 32 x 16 products.
template <bool KC, int ROWS, int NT>
struct Panel {
  static constexpr int kBytes = ROWS * kStep * 2;
  static constexpr int kLoads = kBytes / 16 / NT;
  static constexpr int kVecs = KC ? 8 : ROWS / 8;  // 16-byte vectors of a row
  static_assert(kBytes % (16 * NT) == 0 && NT % kVecs == 0, "whole loads");

  // The vector in which vector c of row r lies.  KC: sixteen rows side by side are
  // read at one vector each, two rows to the width of all banks, so every two
  // spread over the eight.  Otherwise rows r ..
  // r + 3 and r + 8 .. r + 11 are read at 64 bytes each: they spread over the
  // 64-byte parts of a row as far as there are any.
  __device__ static inline int swizzle(int r, int c) {
    if constexpr (KC) return c ^ (r >> 1 & 7);
    if constexpr (kVecs >= 32) return c ^ (((r & 3) | (r >> 1 & 4)) << 2);
    if constexpr (kVecs == 16) return c ^ ((r & 3) << 2);
    return c ^ ((r >> 1 & 1) << 2);
  }
  __device__ static inline int first_row() { return static_cast<int>(threadIdx.x) / kVecs; }
  // vector in memory of this thread's loads: the same for all whose rows are a
  // whole number of swizzle periods apart, which every second or every one is
  static constexpr int kApart = NT / kVecs;
  static_assert(kApart % (KC ? 16 : 8) == 0 && (KC || kApart % 16 == 0 || kVecs == 32), "loads share one or two swizzles");
  __device__ static inline int column(int i) {
    return swizzle(first_row() + i * kApart, static_cast<int>(threadIdx.x) % kVecs);
  }

  // One step's loads, from summed index k on (none if it is past the end: they
  // read 0).  `dim`: where the summed axis ends in a row (KC), a multiple of 8.
  struct Loads {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t off, odd, next;
    char MSS_LDS* lds;
    __device__ inline Loads(const Side& s, int64_t at, int k, int dim, bool any, char MSS_LDS* stage) {
      const int64_t from = KC ? k / kStep * s.panel : static_cast<int64_t>(k) * s.stride;
      const int64_t left = any ? s.span - from : 0;
      const int range = static_cast<int>(left < 0 ? 0 : left < kRsrcRange ? left : kRsrcRange);
      rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(s.base) + at + from, 0, range, kRsrcFlags);
      const uint32_t row = static_cast<uint32_t>(first_row() * s.stride), panel = static_cast<uint32_t>(s.panel);
      off = row + column(0) / 8 * panel + column(0) % 8 * 16;
      odd = row + column(1) / 8 * panel + column(1) % 8 * 16;
      next = static_cast<uint32_t>(kApart * s.stride);
      if (KC && k + column(0) * 8 >= dim) {
        off = odd = kOffNone;
        next = 0;
      }
      lds = stage + uniform(static_cast<int>(threadIdx.x) >> 6) * 1024;
    }
    __device__ inline void issue(int i) const {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (MSS_LDS void*)(lds + i * NT * 16), 16, (i & 1 ? odd : off) + i * next, 0, 0, 0);
    }
  };

  // The fragments of N x 32 rows from `row` on, at summed indices 16 ks .. 16 ks + 15.
  static constexpr int kReads = KC ? 1 : 2;  // LDS reads of one
  template <int N>
  __device__ static inline void fragments(const char MSS_LDS* lds, int row, int ks, bf16x8 (&f)[N]) {
    const int lane = static_cast<int>(threadIdx.x) & 63;
    if constexpr (KC) {
      const char MSS_LDS* p = lds + (row + (lane & 31)) * 128 + swizzle(lane, 2 * ks + (lane >> 5)) * 16;
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = *reinterpret_cast<const bf16x8 MSS_LDS*>(p + i * 32 * 128);
    } else {
      // a group of 16 lanes reads 4 rows of 32 bytes and turns them about
      const int k = 8 * (lane >> 5) + ((lane & 15) >> 2);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = row / 8 + 4 * i + 2 * (lane >> 4 & 1) + ((lane & 3) >> 1);
        const char MSS_LDS* p = lds + k * (ROWS * 2) + swizzle(k, c) * 16 + (lane & 1) * 8 + ks * 16 * ROWS * 2;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((s16x4 MSS_LDS*)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((s16x4 MSS_LDS*)(p + 4 * ROWS * 2));
        f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  }
};

// A tile of WM x WN waves, each with IM x IN products of 32 x 32.
template <bool KCA, bool KCB, int WM, int WN, int IM, int IN>
struct Tile {
  static constexpr int kThreads = 64 * WM * WN, kM = 32 * WM * IM, kN = 32 * WN * IN;
  typedef Panel<KCA, kM, kThreads> A;
  typedef Panel<KCB, kN, kThreads> B;
  static constexpr int kStage = A::kBytes + B::kBytes;

  __device__ static inline int wave_m() { return uniform(static_cast<int>(threadIdx.x) >> 6) / WN * (32 * IM); }
  __device__ static inline int wave_n() { return uniform(static_cast<int>(threadIdx.x) >> 6) % WN * (32 * IN); }

  struct Frags {
    bf16x8 a[IM], b[IN];
    __device__ inline void read(const char MSS_LDS* stage, int ks) {
      A::fragments(stage, wave_m(), ks, a);
      B::fragments(stage + A::kBytes, wave_n(), ks, b);
    }
    __device__ inline void multiply(f32x16 (&acc)[IM][IN]) const {
#pragma unroll
      for (int i = 0; i < IM; ++i)
#pragma unroll
        for (int j = 0; j < IN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  };

  // What one stage adds.
  __device__ static inline void multiply(const char MSS_LDS* stage, f32x16 (&acc)[IM][IN]) {
#pragma unroll
    for (int ks = 0; ks < kStep / 16; ++ks) {
      Frags f;
      f.read(stage, ks);
      f.multiply(acc);
    }
  }

  // The sum over summed indices [k0, k1) (k0 a multiple of 64) of all pairs of planes.
  // While a part's products run, the next part's fragments are read.  At a step's
  // last part they come from the other stage, whose loads had a step's time to
  // land; then every wave has read this stage, and the loads of the step after the
  // next go there.
  __device__ static inline void run(const Side& a, const Side& b, int k0, int k1, int dim, int pairs, char MSS_LDS* lds,
                                    f32x16 (&acc)[IM][IN]) {
    const int total = (k1 - k0 + kStep - 1) / kStep * pairs;
    if (total <= 0) return;
    int pair = 0, k = k0, asked = 0;
    auto advance = [&]() __attribute__((always_inline)) {
      ++asked;
      k += kStep;
      if (k >= k1) {
        k = k0;
        ++pair;
      }
    };
    auto load = [&](char MSS_LDS* stage) __attribute__((always_inline)) {
      const typename A::Loads la(a, plane_of(pair, false) * a.plane, k, dim, asked < total, stage);
      const typename B::Loads lb(b, plane_of(pair, true) * b.plane, k, dim, asked < total, stage + A::kBytes);
#pragma unroll
      for (int i = 0; i < A::kLoads; ++i) la.issue(i);
#pragma unroll
      for (int i = 0; i < B::kLoads; ++i) lb.issue(i);
      advance();
    };
    constexpr int kLoads = A::kLoads + B::kLoads, kReads = IM * A::kReads + IN * B::kReads;
    load(lds);
    load(lds + kStage);
    wait_loads<kLoads>();
    __syncthreads();
    Frags now, next;
    now.read(lds, 0);
    for (int s = 0; s < total; s += 2) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half == 1 && s + 1 >= total) break;
        char MSS_LDS* here = lds + half * kStage;
        char MSS_LDS* there = lds + (1 - half) * kStage;
#pragma unroll
        for (int ks = 0; ks < kStep / 16; ++ks) {
          if (ks < kStep / 16 - 1) {
            next.read(here, ks + 1);
          } else {
            wait_loads<0>();
            __syncthreads();
            next.read(there, 0);
            load(here);
          }
          now.multiply(acc);
#pragma unroll
          for (int m = 0; m < IM * IN; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product,
            __builtin_amdgcn_sched_group_barrier(0x100, (kReads + IM * IN - 1) / (IM * IN), 0);  // LDS reads
            if (ks == kStep / 16 - 1) __builtin_amdgcn_sched_group_barrier(0x010, (kLoads + IM * IN - 1) / (IM * IN), 0);
          }
          now = next;
        }
      }
    }
    wait_loads<0>();
    __syncthreads();  // (the stages are free)
  }
  template <int N>
  __device__ static inline void wait_loads() {
    static_assert(N < 64, "a six-bit count");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4) << 14);  // vmcnt(N)
  }
};

template <int IM, int IN>
__device__ inline void clear(f32x16 (&acc)[IM][IN]) {
#pragma unroll
  for (int i = 0; i < IM; ++i)
#pragma unroll
    for (int j = 0; j < IN; ++j) acc[i][j] = f32x16{0};
}

// The row of the tile's first axis that element e of an accumulator holds.
__device__ inline int acc_row(int e) { return 8 * (e >> 2) + 4 * (static_cast<int>(threadIdx.x) >> 5 & 1) + (e & 3); }

__device__ inline int live_rows(const LossArgs& a, int first) { return max(min(a.piece, *a.live - first), 0); }

// The operands.
__device__ inline Side x_side(const LossArgs& a, int row, int d) {
  const int64_t panel = a.xrows * 128, from = d / 64 * panel + static_cast<int64_t>(row) * 128;
  return {reinterpret_cast<const char*>(a.xp) + from, a.xrows * a.dpad * 2, a.xrows * a.dpad * 2 - from, panel, 128};
}
__device__ inline Side w_side(const LossArgs& a, int v, int d) {
  if (a.pack_w) {
    const int64_t panel = static_cast<int64_t>(a.vocab) * 128, from = d / 64 * panel + static_cast<int64_t>(v) * 128;
    return {reinterpret_cast<const char*>(a.wp) + from, a.vocab * a.dpad * 2, a.vocab * a.dpad * 2 - from, panel, 128};
  }
  const int64_t from = (v * a.sw + d) * 2;
  return {reinterpret_cast<const char*>(a.wp) + from, 0, ((a.vocab - 1) * a.sw + a.dim) * 2 - from, 128,
          static_cast<int>(a.sw * 2)};
}
__device__ inline Side z_side(const LossArgs& a, int row, int v) {
  const int64_t panel = static_cast<int64_t>(a.piece) * 128, from = v / 64 * panel + static_cast<int64_t>(row) * 128;
  return {reinterpret_cast<const char*>(a.dz) + from, a.piece * a.vpad * 2, a.piece * a.vpad * 2 - from, panel, 128};
}
// Where the summed axis of logits ends in the rows of weights.
__device__ inline int w_cols(const LossArgs& a) { return a.pack_w ? static_cast<int>(a.dpad) : a.dim; }

// Which tile of mt x nt a workgroup takes: workgroups of one XCD (every eighth)
// take tiles side by side, in strips of 4 of the first axis, so that what one
// reads the others find in the XCD's cache.
struct At {
  int m, n;
};
__device__ inline At tile_of(int l, int mt, int nt) {
  const int strip = l / (4 * nt), in = l - strip * 4 * nt, wide = min(4, mt - strip * 4);
  return {strip * 4 + in % wide, in / wide};
}
__device__ inline At tile_at(int id, int mt, int nt) {
  const int total = mt * nt, per = (total + 7) / 8;
  const int l = (id & 7) * per + (id >> 3);
  return (id >> 3) >= per || l >= total ? At{-1, -1} : tile_of(l, mt, nt);
}
unsigned tile_blocks(int64_t mt, int64_t nt) { return static_cast<unsigned>((mt * nt + 7) / 8 * 8); }

// ---------------------------------------------------------------- logits

// Tiles of vocabulary x rows: a lane holds one row's values at 16 IM IN entries.
template <bool BF16, typename T, int IM, int IN>
__global__ __launch_bounds__(T::kThreads) void logits_kernel(LossArgs a, int first, bool keep) {
  __shared__ __attribute__((aligned(256))) char lds[2 * T::kStage];
  static_assert(2 * T::kStage >= T::kThreads / 64 * IM * 32 * 32 * 4, "room for the waves' logits");
  const int rows = live_rows(a, first), lane = threadIdx.x & 63;
  const At at = tile_at(blockIdx.x, (a.vocab + T::kM - 1) / T::kM, (rows + T::kN - 1) / T::kN);
  if (at.m < 0) return;
  const int v0 = at.m * T::kM, i0 = at.n * T::kN;
  f32x16 acc[IM][IN];
  clear(acc);
  char MSS_LDS* sh = (char MSS_LDS*)lds;
  T::run(w_side(a, v0, 0), x_side(a, first + i0, 0), 0, a.dim, w_cols(a), a.planes == 1 ? 1 : 6, sh, acc);

  constexpr int kWide = 32 * IM;  // entries of a wave: those that share a maximum
  const int wv = v0 + T::wave_m(), wi = i0 + T::wave_n();
  if (wv >= a.vocab) return;
  const int tile = wv / kWide;
  float MSS_LDS* mine = reinterpret_cast<float MSS_LDS*>(sh + uniform(static_cast<int>(threadIdx.x) >> 6) * (kWide * 32 * 4));
#pragma unroll
  for (int j = 0; j < IN; ++j) {
    const int i = wi + 32 * j + (lane & 31);
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int m = 0; m < IM; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float z = acc[m][j][e] * a.scale;
        if (wv + 32 * m + acc_row(e) >= a.vocab) z = -INFINITY;
        acc[m][j][e] = z;
        top = fmaxf(top, z);
      }
    top = ceilf(fmaxf(top, __shfl_xor(top, 32, 64)));
    const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int m = 0; m < IM; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) sum += fast_exp2((acc[m][j][e] - from) * kLog2e);
    sum += __shfl_xor(sum, 32, 64);
    if (i < rows && lane < 32) a.stats[static_cast<int64_t>(i) * a.tiles + tile] = make_float2(top, sum);
    // The rows' logits in LDS, [32 rows][kWide] with the 16-byte vectors of a row
    // turned by the row; this wave's own.
#pragma unroll
    for (int m = 0; m < IM; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = 8 * m + 2 * q + (lane >> 5), r = lane & 31;
        *reinterpret_cast<f32x4 MSS_LDS*>(mine + r * kWide + (c ^ (r & (kWide / 4 - 1))) * 4) =
            f32x4{acc[m][j][4 * q], acc[m][j][4 * q + 1], acc[m][j][4 * q + 2], acc[m][j][4 * q + 3]};
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // entries of these rows among this wave's
    bool hit = false;
    if (i < rows && lane < 32)
      hit = a.where[static_cast<int64_t>(first + i) * a.where_words + (tile >> 5)] >> (tile & 31) & 1;
    uint64_t hits = __ballot(hit);
    while (hits != 0) {
      const int r = __builtin_ctzll(hits);
      hits &= hits - 1;
      const int64_t k0 = static_cast<int64_t>(first + wi + 32 * j + r) * a.entries;
      for (int k = lane; k < a.entries; k += 64) {
        const int v = a.near[k0 + k] - wv;
        if (v >= 0 && v < kWide) a.picked[k0 + k] = mine[r * kWide + ((v >> 2) ^ (r & (kWide / 4 - 1))) * 4 + (v & 3)];
      }
    }
    if (keep) {
      // 8 entries a lane, 8 rows of a panel one behind another
#pragma unroll
      for (int q = 0; q < kWide / 64 * 4; ++q) {
        const int r = q % 4 * 8 + (lane >> 3), c = q / 4 * 8 + (lane & 7), turn = r & (kWide / 4 - 1);
        const f32x4 lo = *reinterpret_cast<const f32x4 MSS_LDS*>(mine + r * kWide + ((2 * c) ^ turn) * 4);
        const f32x4 hi = *reinterpret_cast<const f32x4 MSS_LDS*>(mine + r * kWide + ((2 * c + 1) ^ turn) * 4);
        const float t = __shfl(top, r, 64);
        if (wi + 32 * j + r >= rows || wv + q / 4 * 64 >= a.vocab) continue;
        const int64_t o = (static_cast<int64_t>(wv / 64 + q / 4) * a.piece + wi + 32 * j + r) * 64 + (lane & 7) * 8;
        if constexpr (BF16) {
          uint32_t code[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            code[e] = static_cast<uint32_t>(fminf(rintf((t - (e < 4 ? lo[e & 3] : hi[e & 3])) * kCodeSteps), 65535.0f));
          uint4 p;
          p.x = code[0] | code[1] << 16;
          p.y = code[2] | code[3] << 16;
          p.z = code[4] | code[5] << 16;
          p.w = code[6] | code[7] << 16;
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.probs) + o) = p;
        } else {
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.probs) + o) = lo;
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.probs) + o + 4) = hi;
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// ---------------------------------------------------------------- dx

template <typename T, int IM, int IN>
__global__ __launch_bounds__(T::kThreads) void dx_part_kernel(LossArgs a, int first) {
  __shared__ __attribute__((aligned(256))) char lds[2 * T::kStage];
  const int rows = live_rows(a, first), lane = threadIdx.x & 63;
  const int mt = (rows + T::kM - 1) / T::kM, nt = (a.dim + T::kN - 1) / T::kN;
  if (mt == 0) return;
  // tiles of one part side by side: those of an XCD read the same rows of weights
  const int splits = dx_splits(a, mt * nt), per = (a.vocab + kStep - 1) / kStep;
  const int all = mt * nt * splits, share = (all + 7) / 8, l = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= share || l >= all) return;
  const int split = l / (mt * nt);
  const At at = tile_of(l - split * (mt * nt), mt, nt);
  const int k0 = static_cast<int>(static_cast<int64_t>(per) * split / splits) * kStep;
  const int k1 = static_cast<int>(static_cast<int64_t>(per) * (split + 1) / splits) * kStep;
  const int i0 = at.m * T::kM, d0 = at.n * T::kN;
  f32x16 acc[IM][IN];
  clear(acc);
  T::run(z_side(a, i0, 0), w_side(a, 0, d0), k0, k1, k1, a.planes == 1 ? 1 : 6, (char MSS_LDS*)lds, acc);
  float* part = a.part + static_cast<int64_t>(split) * a.piece * a.dpad;
#pragma unroll
  for (int i = 0; i < IM; ++i)
#pragma unroll
    for (int j = 0; j < IN; ++j) {
      const int d = d0 + T::wave_n() + 32 * j + (lane & 31), r0 = i0 + T::wave_m() + 32 * i;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (d < a.dim && r0 + acc_row(e) < rows) part[static_cast<int64_t>(r0 + acc_row(e)) * a.dpad + d] = acc[i][j][e];
    }
}

// ---------------------------------------------------------------- dweight

// What the largest dz of each row lost when it was rounded to bf16, times the
// row's x: without it a row's error would be that of its target's rounding, as
// much again as dweight's own.  The rows whose entry lies in this tile are packed
// 64 at a time, in order, into a step of their own: a sparse panel and the rows'
// x.
template <typename T, int IM, int IN>
__device__ inline void add_lost(const LossArgs& a, int first, int rows, int v0, int d0, char* lds, f32x16 (&acc)[IM][IN]) {
  __shared__ int counts[T::kThreads / 64];
  __shared__ int2 list[T::kThreads + 64];  // i, and v - v0 with the lost bits of a bf16
  char MSS_LDS* sh = (char MSS_LDS*)lds;
  const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
  int held = 0;
  auto step = [&](int n) __attribute__((always_inline)) {
    for (int i = t; i < T::A::kBytes / 16; i += T::kThreads) reinterpret_cast<uint4*>(lds)[i] = make_uint4(0, 0, 0, 0);
    for (int q = t; q < kStep * T::B::kVecs; q += T::kThreads) {
      const int r = q / T::B::kVecs, c = q % T::B::kVecs, d = d0 + c * 8;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < n && d < a.dpad)
        x = *reinterpret_cast<const uint4*>(a.xp + (d / 64 * a.xrows + first + list[r].x) * 64 + d % 64);
      *reinterpret_cast<uint4*>(lds + T::A::kBytes + (r * T::B::kVecs + T::B::swizzle(r, c)) * 16) = x;
    }
    __syncthreads();
    if (t < n) {
      const int v = list[t].y >> 16;
      *reinterpret_cast<uint16_t*>(lds + t * (T::kM * 2) + T::A::swizzle(t, v >> 3) * 16 + (v & 7) * 2) =
          static_cast<uint16_t>(list[t].y);
    }
    __syncthreads();
    T::multiply(sh, acc);
    __syncthreads();
  };
  for (int base = 0; base < rows; base += T::kThreads) {
    int2 f = make_int2(-1, 0);
    if (base + t < rows) f = a.fix[base + t];
    const bool in = f.x >= v0 && f.x < v0 + T::kM;
    const uint64_t mask = __ballot(in);
    if (lane == 0) counts[wave] = __popcll(mask);
    __syncthreads();
    int at = held + __popcll(mask & ((1ull << lane) - 1));
    int sum = 0;
    for (int w = 0; w < T::kThreads / 64; ++w) {
      if (w < wave) at += counts[w];
      sum += counts[w];
    }
    if (in) list[at] = make_int2(base + t, (f.x - v0) << 16 | bf16_bits(__int_as_float(f.y)));
    __syncthreads();
    held += sum;
    while (held >= kStep) {
      step(kStep);
      held -= kStep;
      // (at most kThreads - 1 are left: each thread moves one)
      int2 rest = make_int2(0, 0);
      if (t < held) rest = list[t + kStep];
      __syncthreads();
      if (t < held) list[t] = rest;
      __syncthreads();
    }
  }
  if (held > 0) step(held);
}

template <typename IO, typename T, int IM, int IN>
__global__ __launch_bounds__(T::kThreads) void dw_tile_kernel(LossArgs a, int first) {
  __shared__ __attribute__((aligned(256))) char lds[2 * T::kStage];
  const int rows = live_rows(a, first), lane = threadIdx.x & 63;
  if (first > 0 && rows == 0) return;
  const At at = tile_at(blockIdx.x, (a.vocab + T::kM - 1) / T::kM, (a.dim + T::kN - 1) / T::kN);
  if (at.m < 0) return;
  const int v0 = at.m * T::kM, d0 = at.n * T::kN;
  f32x16 acc[IM][IN];
  clear(acc);
  T::run(z_side(a, 0, v0), x_side(a, first, d0), 0, rows, rows, a.planes == 1 ? 1 : 6, (char MSS_LDS*)lds, acc);
  if (a.planes == 1) add_lost<T>(a, first, rows, v0, d0, lds, acc);
  const int d1 = d0 + T::wave_n() + (lane & 31);
#pragma unroll
  for (int i = 0; i < IM; ++i)
#pragma unroll
    for (int j = 0; j < IN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int v = v0 + T::wave_m() + 32 * i + acc_row(e), d = d1 + 32 * j;
        if (v >= a.vocab || d >= a.dim) continue;
        if (a.pieces == 1) {
          io_traits<IO>::store(static_cast<IO*>(a.dweight) + v * a.sdw + d, acc[i][j][e]);
        } else {
          float* p = a.dw_sum + v * a.dpad + d;
          *p = acc[i][j][e] + (first > 0 ? *p : 0.0f);
        }
      }
}

// ---------------------------------------------------------------- launches

template <bool A, bool B>
using Big = Tile<A, B, 2, 4, 4, 2>;    // 256 x 256, 8 waves
template <bool A, bool B>
using Small = Tile<A, B, 2, 2, 2, 1>;  // 128 x 64, 4 waves (dx: 64 x 128)

int64_t tiles(int64_t n, int64_t of) { return (n + of - 1) / of; }

}  // namespace

int loss_vocab_tile(bool small) { return small ? 64 : 128; }

hipError_t launch_logits(const LossArgs& a, int first, bool io_bf16, bool keep, hipStream_t stream) {
  const int n = std::min(a.piece, a.rows - first);
  if (a.small) {
    typedef Small<true, true> T;
    const unsigned g = tile_blocks(tiles(a.vocab, T::kM), tiles(n, T::kN));
    if (io_bf16) logits_kernel<true, T, 2, 1><<<g, T::kThreads, 0, stream>>>(a, first, keep);
    else logits_kernel<false, T, 2, 1><<<g, T::kThreads, 0, stream>>>(a, first, keep);
  } else {
    typedef Big<true, true> T;
    const unsigned g = tile_blocks(tiles(a.vocab, T::kM), tiles(n, T::kN));
    if (io_bf16) logits_kernel<true, T, 4, 2><<<g, T::kThreads, 0, stream>>>(a, first, keep);
    else logits_kernel<false, T, 4, 2><<<g, T::kThreads, 0, stream>>>(a, first, keep);
  }
  return hipGetLastError();
}

hipError_t launch_dx(const LossArgs& a, int first, hipStream_t stream) {
  const int n = std::min(a.piece, a.rows - first);
  const int64_t m = a.small ? 64 : 256, w = a.small ? 128 : 256;
  int64_t g = 0;  // the most that any count of live rows asks for
  for (int64_t mt = 1; mt <= tiles(n, m); ++mt) {
    const int64_t t = mt * tiles(a.dim, w);
    g = std::max<int64_t>(g, (t * dx_splits(a, static_cast<int>(t)) + 7) / 8 * 8);
  }
  if (a.small) dx_part_kernel<Tile<true, false, 2, 2, 1, 2>, 1, 2><<<static_cast<unsigned>(g), 256, 0, stream>>>(a, first);
  else dx_part_kernel<Big<true, false>, 4, 2><<<static_cast<unsigned>(g), 512, 0, stream>>>(a, first);
  return hipGetLastError();
}

hipError_t launch_dw(const LossArgs& a, int first, bool io_bf16, hipStream_t stream) {
  if (a.small) {
    typedef Small<false, false> T;
    const unsigned g = tile_blocks(tiles(a.vocab, T::kM), tiles(a.dim, T::kN));
    if (io_bf16) dw_tile_kernel<bf16_t, T, 2, 1><<<g, T::kThreads, 0, stream>>>(a, first);
    else dw_tile_kernel<float, T, 2, 1><<<g, T::kThreads, 0, stream>>>(a, first);
  } else {
    typedef Big<false, false> T;
    const unsigned g = tile_blocks(tiles(a.vocab, T::kM), tiles(a.dim, T::kN));
    if (io_bf16) dw_tile_kernel<bf16_t, T, 4, 2><<<g, T::kThreads, 0, stream>>>(a, first);
    else dw_tile_kernel<float, T, 4, 2><<<g, T::kThreads, 0, stream>>>(a, first);
  }
  return hipGetLastError();
}

}  // namespace mss

// head_scan.hip -- head-wise selective scan over packed prompts, gfx950.
//
// With a_t = delta_t A (A = -exp(A_log[h]) < 0) and c_i the sum of a over a
// chunk's tokens up to i, the recurrence S <- e^a_t S + delta_t x_t B_t^T gives
// for a chunk of Q tokens entered with state S (P x N)
//   y_i = sum_{j<=i} (C_i . B_j) e^(c_i - c_j) delta_j x_j  +  e^c_i S C_i  +  D x_i
//   S  <- e^c_Q S + sum_j e^(c_Q - c_j) delta_j x_j B_j^T
// which are matrix products: C B^T (shared by the heads of a group), its decayed
// lower triangle with x, C with the entering state, and x with B.
//
// A wave walks one head's tile of 32 columns p chunk by chunk, with the state in
// MFMA accumulators; a workgroup's four waves are tiles of one group, which
// share the chunk's B and C in LDS and form C B^T together.  Every product is
// laid out so that one product's accumulators are the next one's operand:
//   C B^T  as [j x i]: lane (g, c) holds column i = 16 it + c, eight rows j
//   Y^T    as [p x i] = X^T M^T + S C^T: M^T is the decayed C B^T as it lies
//   S      as [n x p] = B^T V: as it lies the operand [p x n] of S C^T
// (lane = 16 g + c; an operand fragment holds one row or column c and the eight
// K-slots of g; an accumulator tile one column c and the rows 4 g .. 4 g + 3, so
// two tiles whose rows are 8 g + r and 8 g + 4 + r make the slots 8 g .. 8 g + 7
// of a fragment.)  X^T and B^T come from row-major LDS tiles by transposing
// reads; the K order of token slots, {0,1,4,5,2,3,6,7} within each 8, lets one
// transposing read meet each LDS bank twice, with rows' 16-byte chunks swizzled
// by the row number (a plain order would meet them four times).
//
// bf16 inputs enter the products as they are.  What is rounded to bf16 besides:
// the decayed C B^T and the entering state where they make y (one rounding of
// each term, the size of y's own).  The state itself stays in fp32: its addends
// delta e^(..) x are split into three bf16 parts (24 bits), so states are
// as exact as an fp32 sum.  fp32 inputs use the fp32 matrix instruction, with
// nothing rounded.  The sums c are taken in 64 bits and kept as two floats.
//
// A prompt longer than a.seg_len is cut into segments: one pass forms what each
// segment adds to a zero state, one composes the states entering the segments
// (and the state the prompt leaves), and the walk then runs all segments at once.
//
// A chunk that holds an infinity or a NaN in x or B is walked token by token
// (0 times it would reach tokens before it, and splitting loses an infinity).
#include "mss_head.hpp"

namespace mss {
namespace {

constexpr int kWaves = 4;
constexpr int kCols = 32;  // columns p of a wave's tile

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// ------------------------------------------------------- operand fragments

template <typename IO>
struct Frag;
template <>
struct Frag<bf16_t> {
  bf16x8 v;
  __device__ inline float get(int e) const { return static_cast<float>(v[e]); }
  __device__ inline void set(int e, float x) { v[e] = static_cast<__bf16>(x); }
};
template <>
struct Frag<float> {
  float v[8];
  __device__ inline float get(int e) const { return v[e]; }
  __device__ inline void set(int e, float x) { v[e] = x; }
};

__device__ inline f32x4 mma(const Frag<bf16_t>& a, const Frag<bf16_t>& b, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
}
// 16x16x4 takes one K-slot of each g: eight of them cover the same 32 slots.
__device__ inline f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 acc) {
#pragma unroll
  for (int e = 0; e < 8; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], acc, 0, 0, 0);
  return acc;
}

// e^x for a sum of many exponents (x in powers of two), never below the normal
// range: an infinite state stays infinite, as it does token by token, where 0
// would make it a NaN, and what it adds to a finite one is below any rounding.
__device__ inline float long_decay(float x) { return fmaxf(fast_exp2(x), 1.17549435e-38f); }

// Token order of a fragment's eight slots.
__device__ constexpr int tok(int e) { return (e & 1) | ((e & 2) << 1) | ((e & 4) >> 1); }

// ------------------------------------------------------- LDS tiles
// Row-major [rows][COLS], 16-byte chunks swizzled by the row.
template <typename IO, int COLS>
struct Tile {
  static constexpr int kChunks = COLS * static_cast<int>(sizeof(IO)) / 16;  // of a row: 4 or more
  static constexpr int kElems = 16 / sizeof(IO);
  __device__ static inline int offset(int row, int chunk) {
    const int s = kChunks >= 8 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
    return (row * kChunks + s) * 16;
  }
  // row r, columns col .. col+7 (col a multiple of 8)
  __device__ static inline Frag<IO> row(const char* t, int r, int col) {
    Frag<IO> f;
    if constexpr (sizeof(IO) == 2) {
      f.v = *reinterpret_cast<const bf16x8*>(t + offset(r, col / 8));
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(t + offset(r, col / 4));
      const f32x4 b = *reinterpret_cast<const f32x4*>(t + offset(r, col / 4 + 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) f.v[i] = a[i], f.v[4 + i] = b[i];
    }
    return f;
  }
  // rows r0 + tok(0..7), one column a lane: col0 + 8 (c / 4) + c % 4 + 4 half
  __device__ static inline Frag<IO> col(const char* t, int r0, int col0, int half, int c) {
    Frag<IO> f;
    if constexpr (sizeof(IO) == 2) {
      union {
        s16x4 h[2];
        bf16x8 v;
      } u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // the lane names 4 columns of one row; it receives 4 rows of its column
        const int lr = c >> 2;
        const int r = r0 + (lr & 1) + ((lr & 2) << 1) + 2 * h;
        char* p = const_cast<char*>(t) + offset(r, col0 / 8 + (c & 3)) + 8 * half;
        u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
      }
      f.v = u.v;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f.v[e] = *reinterpret_cast<const float*>(t + offset(r0 + tok(e), (col0 + 8 * (c >> 2) + 4 * half) / 4) +
                                                 4 * (c & 3));
    }
    return f;
  }
};

// 16 bytes from element-aligned memory; elements from n on read as 0.
typedef u32x4 __attribute__((aligned(2))) u32x4_loose;
template <typename IO>
__device__ inline u32x4 load16(const IO* p, int n) {
  constexpr int kE = 16 / sizeof(IO);
  if (n >= kE) return *reinterpret_cast<const u32x4_loose*>(p);
  union {
    IO e[kE];
    u32x4 v;
  } u;
  u.v = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kE; ++i)
    if (i < n) u.e[i] = p[i];
  return u.v;
}

// Whether any of the elements is an infinity or a NaN.
template <typename IO>
__device__ inline bool not_finite(u32x4 v) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(IO) == 2) {
      top |= ((v[i] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
    } else {
      top |= ((v[i] & 0x7fffffffu) + 0x00800000u) & 0x80000000u;
    }
  }
  return top != 0;
}

// ------------------------------------------------------- segments

// Segments of a prompt of `len` tokens, and the tokens of each but the last.
__device__ inline int segments(const HeadScanArgs& a, int len) {
  return a.seg_len > 0 ? max(1, (len + a.seg_len - 1) / a.seg_len) : 1;
}
template <int Q>
__device__ inline int segment_tokens(int len, int n) {
  return ((len + n - 1) / n + Q - 1) / Q * Q;
}

struct Where {
  int seq;    // -1: none
  int seg, nseg;
  int index;  // of the prompt among the cut ones, or of the segment among all their segments
};

// The prompt and segment with place `at` among the segments of the prompts
// that are cut (or, by_prompt, the prompt with place `at` among those and its
// first segment's place): every lane of the wave takes part.
__device__ inline Where find_cut(const HeadScanArgs& a, int at, bool by_prompt) {
  const int lane = threadIdx.x & 63;
  int segs_before = 0, cut_before = 0;
  for (int base = 0; base < a.q.seqs; base += 64) {
    const int i = base + lane;
    int n = 0;
    if (i < a.q.seqs) {
      const Span sp = prompt_span(a.q, i);
      n = segments(a, sp.end - sp.begin);
    }
    const int segs = n > 1 ? n : 0, one = n > 1 ? 1 : 0;
    int si = segs, ci = one;  // inclusive sums over the lanes
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int s = __shfl_up(si, o, 64), c = __shfl_up(ci, o, 64);
      if (lane >= o) si += s, ci += c;
    }
    const int count = by_prompt ? cut_before + ci : segs_before + si;
    const uint64_t hit = __ballot(one != 0 && count > at);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      const int before = segs_before + __shfl(si, l, 64) - __shfl(segs, l, 64);
      return {uniform(base + l), uniform(by_prompt ? 0 : at - before), uniform(__shfl(n, l, 64)),
              uniform(by_prompt ? before : at)};
    }
    segs_before += __shfl(si, 63, 64);
    cut_before += __shfl(ci, 63, 64);
  }
  return {-1, 0, 0, 0};
}

// ------------------------------------------------------- the walk

template <typename IO, int NP, int Q>
struct Shape {
  static constexpr int kUnits = Q == 64 ? 6 : 2;  // 32 x 16 pieces of the lower triangle
  using BC = Tile<IO, NP>;
  using X = Tile<IO, kCols>;
  struct Lds {
    char b[Q * NP * sizeof(IO)];
    char c[Q * NP * sizeof(IO)];
    char x[kWaves][Q * kCols * sizeof(IO)];
    f32x4 s[kUnits * 2][64];
    float sum[kWaves][2][Q];   // c_i as two floats, in powers of two
    float delta[kWaves][Q];
    float left[kWaves][Q];     // delta_j e^(c_Q - c_j)
    int odd[2];                // a chunk holds something not finite
  };
};

// AGG: only what a segment adds to a zero state, and its decay.
template <typename IO, int NP, int Q, bool AGG>
__global__ __launch_bounds__(256, 2) void head_scan_kernel(HeadScanArgs a) {
  using S = Shape<IO, NP, Q>;
  using BC = typename S::BC;
  using X = typename S::X;
  constexpr int kE = 16 / sizeof(IO);
  constexpr int kK = NP / 32;                          // K-steps over the states
  constexpr int kT = Q / 32;                           // K-steps over the tokens
  constexpr int kLoadBC = Q * BC::kChunks / 256;       // 16-byte loads a thread
  constexpr int kLoadX = Q * X::kChunks / 64;          // 16-byte loads a lane
  __shared__ __attribute__((aligned(16))) typename S::Lds lds;

  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, c = lane & 15;

  // which tile of which segment
  const int jobs = a.heads / a.groups * a.ptiles;      // of one group
  const int quads = (jobs + kWaves - 1) / kWaves;
  const int gq = blockIdx.x % (a.groups * quads);
  const int where = blockIdx.x / (a.groups * quads);
  const int grp = gq / quads;
  const int job = gq % quads * kWaves + wave;
  Where w;
  if (where < a.cut_slots) {
    w = find_cut(a, where, false);
    if (w.seq < 0) return;
  } else {
    w = {where - a.cut_slots, 0, 1, 0};
  }
  const Span sp = prompt_span(a.q, w.seq);
  const int len = sp.end - sp.begin;
  if (where >= a.cut_slots && segments(a, len) > 1) return;
  const int slot = slot_of(a.q.slots, a.q.cache_slots, w.seq);
  if (slot < 0) return;
  const int per = segment_tokens<Q>(len, w.nseg);
  const int begin = sp.begin + w.seg * per;
  const int end = min(sp.end, begin + per);
  const bool cut = w.nseg > 1;
  const bool from_cache = resumes(a.q, w.seq);
  if (len == 0 && from_cache) return;

  const bool on = job < jobs;
  const int h = grp * (a.heads / a.groups) + (on ? job / a.ptiles : 0);
  const int p0 = (on ? job % a.ptiles : 0) * kCols;
  const int pc = on ? a.headdim - p0 : 0;              // this tile's columns
  const int64_t hp = static_cast<int64_t>(h) * a.headdim + p0;
  float* cache = a.state + slot * a.sstate + hp * a.dstate;
  float* part = cut ? a.parts + (static_cast<int64_t>(w.index) * a.heads * a.headdim + hp) * a.dstate : nullptr;

  // the state: tile [n = 32 q + 8 g + 4 tn + r][p = 8 (c / 4) + c % 4 + 4 tp]
  f32x4 st[kK][2][2];
  const int pcol = 8 * (c >> 2) + (c & 3);
  const float* enter = AGG ? nullptr : cut ? part : from_cache ? cache : nullptr;
#pragma unroll
  for (int q = 0; q < kK; ++q)
#pragma unroll
    for (int tp = 0; tp < 2; ++tp) {
      const int p = pcol + 4 * tp, n = 32 * q + 8 * g;
      float v[8] = {};
      if (enter != nullptr) load_part<float, 8>(enter + static_cast<int64_t>(p) * a.dstate + n, p < pc ? a.dstate - n : 0, v);
#pragma unroll
      for (int tn = 0; tn < 2; ++tn)
        st[q][tn][tp] = f32x4{v[4 * tn], v[4 * tn + 1], v[4 * tn + 2], v[4 * tn + 3]};
    }

  const IO* xh = static_cast<const IO*>(a.x) + h * a.sx[1] + p0;
  const IO* Bg = static_cast<const IO*>(a.B) + grp * a.sB[1];
  const IO* Cg = static_cast<const IO*>(a.C) + grp * a.sC[1];
  const IO* dth = static_cast<const IO*>(a.dt) + h * a.sdt[1];
  const float rate = -expf(a.A_log[h]) * kLog2e;
  const float bias = a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f;
  const float skip = a.D != nullptr ? a.D[h] : 0.0f;

  u32x4 pb[kLoadBC], pcc[AGG ? 1 : kLoadBC], px[kLoadX];
  float pdt = 0.0f;
  auto fetch = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoadBC; ++i) {
      const int k = i * 256 + static_cast<int>(threadIdx.x);
      const int r = t + k / BC::kChunks, n = k % BC::kChunks * kE;
      const int valid = r < end ? a.dstate - n : 0;
      pb[i] = load16<IO>(Bg + r * a.sB[0] + n, valid);
      if constexpr (!AGG) pcc[i] = load16<IO>(Cg + r * a.sC[0] + n, valid);
    }
#pragma unroll
    for (int i = 0; i < kLoadX; ++i) {
      const int k = i * 64 + lane;
      const int r = t + k / X::kChunks, p = k % X::kChunks * kE;
      px[i] = load16<IO>(xh + r * a.sx[0] + p, r < end ? pc - p : 0);
    }
    const int r = t + lane;
    pdt = lane < Q && r < end ? io_traits<IO>::load(dth + r * a.sdt[0]) : 0.0f;
  };

  if (threadIdx.x < 2) lds.odd[threadIdx.x] = 0;
  double total = 0.0;  // the segment's decay (AGG)
  fetch(begin);
  __syncthreads();
  int par = 0;
  for (int t = begin; t < end; t += Q, par ^= 1) {
    // ---- this chunk into LDS
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kLoadBC; ++i) {
      const int k = i * 256 + static_cast<int>(threadIdx.x);
      const int o = BC::offset(k / BC::kChunks, k % BC::kChunks);
      *reinterpret_cast<u32x4*>(lds.b + o) = pb[i];
      odd |= not_finite<IO>(pb[i]);
      if constexpr (!AGG) *reinterpret_cast<u32x4*>(lds.c + o) = pcc[i];
    }
#pragma unroll
    for (int i = 0; i < kLoadX; ++i) {
      const int k = i * 64 + lane;
      *reinterpret_cast<u32x4*>(lds.x[wave] + X::offset(k / X::kChunks, k % X::kChunks)) = px[i];
      odd |= not_finite<IO>(px[i]);
    }
    if (odd) lds.odd[par] = 1;
    // ---- time steps and the sums of their exponents
    const bool live = lane < Q && t + lane < end;
    float dl = pdt + bias;
    dl = live ? (a.softplus ? softplus(dl) : dl) : 0.0f;
    double sum = static_cast<double>(dl * rate);
#pragma unroll
    for (int o = 1; o < Q; o *= 2) {
      const double up = __shfl_up(sum, o, 64);
      if (lane >= o) sum += up;
    }
    const double last = __shfl(sum, Q - 1, 64);
    const float decay = long_decay(static_cast<float>(last));
    if (AGG) total += last;
    if (lane < Q) {
      const float hi = static_cast<float>(sum);
      lds.sum[wave][0][lane] = hi;
      lds.sum[wave][1][lane] = static_cast<float>(sum - hi);
      lds.delta[wave][lane] = dl;
      lds.left[wave][lane] = dl * fast_exp2(static_cast<float>(last - sum));
    }
    __syncthreads();
    const bool walk = lds.odd[par] != 0;
    if (threadIdx.x == 0) lds.odd[par ^ 1] = 0;
    if (t + Q < end) fetch(t + Q);

    if constexpr (!AGG) {
      // ---- C B^T, two tiles [j x i] a piece, shared out over the waves
      if (!walk) {
#pragma unroll
        for (int k = 0; k < S::kUnits * 2 / kWaves; ++k) {
          const int tile = k * kWaves + wave;
          const int unit = tile >> 1, half = tile & 1;
          const int ks = unit >> 2, it = ks ? unit - 2 : unit;
          const int j = 32 * ks + 8 * (c >> 2) + ((c & 1) | ((c & 2) << 1)) + 2 * half;
          f32x4 acc = {0, 0, 0, 0};
#pragma unroll
          for (int q = 0; q < kK; ++q)
            acc = mma(BC::row(lds.b, j, 32 * q + 8 * g), BC::row(lds.c, 16 * it + c, 32 * q + 8 * g), acc);
          lds.s[tile][lane] = acc;
        }
      }
      __syncthreads();
    }

    if (on && !walk) {
      Frag<IO> xt[kT][2];
#pragma unroll
      for (int ks = 0; ks < kT; ++ks)
#pragma unroll
        for (int tp = 0; tp < 2; ++tp) xt[ks][tp] = X::col(lds.x[wave], 32 * ks + 8 * g, 0, tp, c);
      if constexpr (!AGG) {
        Frag<IO> sb[kK][2];  // the state as an operand [p x n]
#pragma unroll
        for (int q = 0; q < kK; ++q)
#pragma unroll
          for (int tp = 0; tp < 2; ++tp)
#pragma unroll
            for (int e = 0; e < 8; ++e) sb[q][tp].set(e, st[q][e >> 2][tp][e & 3]);
#pragma unroll
        for (int it = 0; it < Q / 16; ++it) {
          const int i = 16 * it + c;
          const float ch = lds.sum[wave][0][i], cl = lds.sum[wave][1][i];
          f32x4 y[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
          for (int q = 0; q < kK; ++q) {
            const Frag<IO> cf = BC::row(lds.c, i, 32 * q + 8 * g);
#pragma unroll
            for (int tp = 0; tp < 2; ++tp) y[tp] = mma(sb[q][tp], cf, y[tp]);
          }
          const float ei = long_decay(ch);
#pragma unroll
          for (int tp = 0; tp < 2; ++tp) y[tp] *= ei;
#pragma unroll
          for (int ks = 0; ks <= it / 2; ++ks) {
            const int unit = ks ? it + 2 : it;
            const f32x4 s0 = lds.s[2 * unit][lane], s1 = lds.s[2 * unit + 1][lane];
            Frag<IO> m;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int j = 32 * ks + 8 * g + tok(e);
              float d = ch - lds.sum[wave][0][j];
              if constexpr (sizeof(IO) == 4) d += cl - lds.sum[wave][1][j];
              const float v = (e < 4 ? s0[e & 3] : s1[e & 3]) * (fast_exp2(d) * lds.delta[wave][j]);
              m.set(e, j <= i ? v : 0.0f);
            }
#pragma unroll
            for (int tp = 0; tp < 2; ++tp) y[tp] = mma(xt[ks][tp], m, y[tp]);
          }
          // ---- skip, gate, out: lane holds token i, columns 8 g .. 8 g + 7
          const int r = t + i;
          const int n = r < end ? pc - 8 * g : 0;
          const Frag<IO> xi = X::row(lds.x[wave], i, 8 * g);
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(skip, xi.get(e), y[e >> 2][e & 3]);
          if (a.z != nullptr) {
            float z[8];
            load_part<IO, 8>(static_cast<const IO*>(a.z) + r * a.sz[0] + h * a.sz[1] + p0 + 8 * g, n, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= silu(z[e]);
          }
          store_part<IO, 8>(static_cast<IO*>(a.out) + r * a.so[0] + h * a.so[1] + p0 + 8 * g, n, o);
        }
      }
      // ---- the state
#pragma unroll
      for (int q = 0; q < kK; ++q)
#pragma unroll
        for (int tn = 0; tn < 2; ++tn)
#pragma unroll
          for (int tp = 0; tp < 2; ++tp) st[q][tn][tp] *= decay;
#pragma unroll
      for (int ks = 0; ks < kT; ++ks) {
        constexpr int kParts = sizeof(IO) == 2 ? 3 : 1;
        Frag<IO> v[2][kParts];
#pragma unroll
        for (int tp = 0; tp < 2; ++tp)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float r = xt[ks][tp].get(e) * lds.left[wave][32 * ks + 8 * g + tok(e)];
#pragma unroll
            for (int k = 0; k < kParts; ++k) {
              v[tp][k].set(e, r);
              r -= v[tp][k].get(e);
            }
          }
#pragma unroll
        for (int q = 0; q < kK; ++q)
#pragma unroll
          for (int tn = 0; tn < 2; ++tn) {
            const Frag<IO> bt = BC::col(lds.b, 32 * ks + 8 * g, 32 * q, tn, c);
#pragma unroll
            for (int tp = 0; tp < 2; ++tp)
#pragma unroll
              for (int k = kParts - 1; k >= 0; --k) st[q][tn][tp] = mma(bt, v[tp][k], st[q][tn][tp]);
          }
      }
    } else if (on) {
      // ---- token by token
      for (int i = 0; i < Q && t + i < end; ++i) {
        const float dti = lds.delta[wave][i], e = fast_exp2(dti * rate);
        float y[2], x[2];
#pragma unroll
        for (int tp = 0; tp < 2; ++tp) {
          const int p = pcol + 4 * tp;
          x[tp] = io_traits<IO>::load(reinterpret_cast<const IO*>(lds.x[wave] + X::offset(i, p / kE)) + p % kE);
          y[tp] = 0.0f;
        }
#pragma unroll
        for (int q = 0; q < kK; ++q) {
          const Frag<IO> b = BC::row(lds.b, i, 32 * q + 8 * g);
          const Frag<IO> cf = BC::row(lds.c, i, 32 * q + 8 * g);
#pragma unroll
          for (int tp = 0; tp < 2; ++tp)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (32 * q + 8 * g + k < a.dstate) {  // the others stay 0, whatever x is
                const float s = fmaf(e, st[q][k >> 2][tp][k & 3], dti * x[tp] * b.get(k));
                st[q][k >> 2][tp][k & 3] = s;
                if (!AGG) y[tp] = fmaf(cf.get(k), s, y[tp]);
              }
            }
        }
        if constexpr (!AGG) {
          const int64_t r = t + i;
#pragma unroll
          for (int tp = 0; tp < 2; ++tp) {
            const int p = pcol + 4 * tp;
            y[tp] += __shfl_xor(y[tp], 16, 64);
            y[tp] += __shfl_xor(y[tp], 32, 64);
            if (g == 0 && p < pc) {
              float o = fmaf(skip, x[tp], y[tp]);
              if (a.z != nullptr)
                o *= silu(io_traits<IO>::load(static_cast<const IO*>(a.z) + r * a.sz[0] + h * a.sz[1] + p0 + p));
              io_traits<IO>::store(static_cast<IO*>(a.out) + r * a.so[0] + h * a.so[1] + p0 + p, o);
            }
          }
        }
      }
    }
    __syncthreads();
  }

  // ---- the state that the segment leaves
  if (!on || (!AGG && cut)) return;
  float* leave = AGG ? part : cache;
#pragma unroll
  for (int q = 0; q < kK; ++q)
#pragma unroll
    for (int tp = 0; tp < 2; ++tp) {
      const int p = pcol + 4 * tp, n = 32 * q + 8 * g;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = st[q][e >> 2][tp][e & 3];
      store_part<float, 8>(leave + static_cast<int64_t>(p) * a.dstate + n, p < pc ? a.dstate - n : 0, v);
    }
  if (AGG && lane == 0 && p0 == 0) a.decays[static_cast<int64_t>(w.index) * a.heads + h] = long_decay(static_cast<float>(total));
}

// The states entering the segments of a cut prompt, in place of what the
// segments add, and the state the prompt leaves: four states a thread, kAhead
// segments loaded before the first is used.
__global__ __launch_bounds__(256) void head_scan_carry_kernel(HeadScanArgs a, int blocks) {
  constexpr int kAhead = 8;
  const Where w = find_cut(a, blockIdx.x / blocks, true);
  if (w.seq < 0) return;
  const int nseg = min(w.nseg, a.cut_slots - w.index);  // (less only for a cu_seqlens that runs backwards)
  const int slot = slot_of(a.q.slots, a.q.cache_slots, w.seq);
  if (slot < 0) return;
  const int64_t all = static_cast<int64_t>(a.heads) * a.headdim * a.dstate;
  const int64_t i = (static_cast<int64_t>(blockIdx.x % blocks) * 256 + threadIdx.x) * 4;
  const int n = static_cast<int>(min(all - i, static_cast<int64_t>(4)));
  if (n <= 0) return;
  int h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = static_cast<int>(min(i + k, all - 1) / (static_cast<int64_t>(a.headdim) * a.dstate));
  float* cache = a.state + slot * a.sstate + i;
  float* part = a.parts + w.index * all + i;
  const float* decay = a.decays + static_cast<int64_t>(w.index) * a.heads;
  float s[4] = {};
  if (resumes(a.q, w.seq)) load_part<float, 4>(cache, n, s);
  for (int k0 = 0; k0 < nseg; k0 += kAhead) {
    float v[kAhead][4], d[kAhead][4];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t at = min(k0 + k, nseg - 1);
      load_part<float, 4>(part + at * all, n, v[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[k][e] = decay[at * a.heads + h[e]];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k0 + k < nseg) {
        store_part<float, 4>(part + (k0 + k) * all, n, s);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = fmaf(d[k][e], s[e], v[k][e]);
      }
    }
  }
  store_part<float, 4>(cache, n, s);
}

template <typename IO, int NP, int Q>
hipError_t launch_n(const HeadScanArgs& a, hipStream_t stream) {
  const int64_t tiles = static_cast<int64_t>(a.groups) * ((a.heads / a.groups * a.ptiles + kWaves - 1) / kWaves);
  if (a.cut_slots > 0) {
    head_scan_kernel<IO, NP, Q, true><<<dim3(static_cast<unsigned>(a.cut_slots * tiles)), 256, 0, stream>>>(a);
    const int64_t blocks = (static_cast<int64_t>(a.heads) * a.headdim * a.dstate + 1023) / 1024;
    head_scan_carry_kernel<<<dim3(static_cast<unsigned>(blocks * a.cut_prompts)), 256, 0, stream>>>(
        a, static_cast<int>(blocks));
  }
  head_scan_kernel<IO, NP, Q, false>
      <<<dim3(static_cast<unsigned>((a.cut_slots + a.q.seqs) * tiles)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

// Chunks of 64 tokens in bf16 and 32 in fp32, whose tiles are twice as wide.
template <typename IO>
hipError_t launch_t(const HeadScanArgs& a, hipStream_t stream) {
  constexpr int Q = sizeof(IO) == 2 ? 64 : 32;
  if (a.dstate <= 32) return launch_n<IO, 32, Q>(a, stream);
  if (a.dstate <= 64) return launch_n<IO, 64, Q>(a, stream);
  return launch_n<IO, 128, Q>(a, stream);
}

}  // namespace

hipError_t launch_head_scan(const HeadScanArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_t<bf16_t>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace mss

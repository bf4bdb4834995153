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
// A wave walks one head's tile of 32 columns p (16 in calls with few tiles) chunk
// by chunk, with the state in
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
// bf16 inputs enter the products as they are.  The decayed C B^T and the entering
// state are split into two bf16 parts where they make y: each term is off by
// 2^-16 at most, far below y's own rounding (one part alone took 545 us where this
// takes 598, on the batch below, and left y off by 1.9e-3, where its rounding
// leaves 1.66e-3).  The state itself stays in fp32: its addends delta e^(..) x are
// split into three bf16 parts (24 bits), so states are as exact as an fp32 sum.
// fp32 inputs use the fp32 matrix instruction, with nothing rounded.  The sums c
// are taken in 64 bits and kept as two floats.
//
// A prompt longer than a.seg_len is cut into segments: one pass forms what each
// segment adds to a zero state, one composes the states entering the segments, and
// the walk then runs all segments at once: the last one's writes the cache entry.
//
// What bounds it: instructions.  A chunk of 64 tokens costs a wave 196 MFMAs of 16
// cycles and 1450 VALU instructions (states of 128; counted); with two waves a SIMD
// (two workgroups of 80 KB of LDS and 227 registers a CU) the SIMDs issue in 64% of
// their cycles, and the waits between a chunk's products take most of the rest.
// 80 heads of 64 x 128, 8 x 4096 tokens in bf16: 597 to 616 us from box to box, 140
// TFLOP/s of the 4 P N a token that the recurrence needs; 24 heads, one prompt of
// 32768: 217 to 224 us (walk 149, sums 64, states between 16 in a profile); 200
// tokens of 24 heads: 27 us, four chunks one after the other.  Measured and not
// kept, before the outputs' operands had two parts: three waves a SIMD for the
// sums (same time); two parts for the addends of states that only outputs read (one
// long prompt 4% faster, a short one 4% slower); steps left to the compiler's
// schedule, without the barriers between them (4% at most).
//
// A chunk that holds an infinity or a NaN in x, B or C is walked token by token
// (0 times one in x would reach tokens before it, splitting loses an infinity, and
// infinities of both signs would meet in a sum that the recurrence does not form),
// and so is one with values of 2^kLargeExponent or more in x or C B^T, or with time
// steps or a rate whose sums or exponentials pass fp32.
#include "mss_head.hpp"

namespace mss {
namespace {

constexpr int kWaves = 4;
constexpr int kCols = 32;  // columns of x in LDS; a wave's tile of columns p is these or the first 16

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// ------------------------------------------------------- operand fragments

template <typename IO>
struct Frag;
template <>
struct Frag<bf16_t> {
  union {
    bf16x8 v;
    uint32_t w[4];
  };
  __device__ inline float get(int e) const { return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16); }
  __device__ inline void set2(int e, float x, float y) { w[e / 2] = bf16x2_bits(x, y); }
  // what x is more than slot e (exact: one instruction, with no unpacking).  The
  // pair (-1, 0) comes from a register: as a constant the compiler encodes it as
  // (0, -1)'s inline form and the wrong half is taken.
  __device__ inline float more(int e, float x) const {
    uint32_t minus = e & 1 ? 0xbf800000u : 0x0000bf80u;
    asm("" : "+s"(minus));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w[e / 2]), __builtin_bit_cast(bf16x2, minus), x,
                                           false);
  }
};
template <>
struct Frag<float> {
  float v[8];
  __device__ inline float get(int e) const { return v[e]; }
  __device__ inline void set2(int e, float x, float y) { v[e] = x, v[e + 1] = y; }
  __device__ inline float more(int e, float x) const { return x - v[e]; }
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
// Row-major [rows][COLS], 16-byte chunks swizzled by the row.  A lane's address
// is formed once (`lane_*`); each read xors a constant into its swizzled bits
// and adds a constant, so the reads of a loop share a few addresses.
template <typename IO, int COLS>
struct Tile {
  static constexpr int kChunks = COLS * static_cast<int>(sizeof(IO)) / 16;  // of a row: 4 or more
  static constexpr int kElems = 16 / sizeof(IO);
  static constexpr int kRow = COLS * static_cast<int>(sizeof(IO));          // bytes
  static constexpr int kMask = kChunks >= 8 ? 7 : 3;
  __device__ static inline int swizzle(int row) { return kChunks >= 8 ? row & 7 : (row >> 1) & 3; }
  __device__ static inline int offset(int row, int chunk) { return row * kRow + (chunk ^ swizzle(row)) * 16; }
  // byte distance and xor that take a lane from a chunk to the one `by` (a constant) further
  __device__ static constexpr int flip(int by) { return (by & kMask) * 16; }
  __device__ static constexpr int ahead(int by) { return (by & ~kMask) * 16; }

  // Row fragments: row r, columns 32 q + 8 g .. + 7.  Rows 16 apart share an address.
  __device__ static inline int lane_row(int r, int g) { return offset(r, sizeof(IO) == 2 ? g : 2 * g); }
  __device__ static inline Frag<IO> row(const char* t, int lane, int rows, int q) {
    Frag<IO> f;
    if constexpr (sizeof(IO) == 2) {
      f.v = *reinterpret_cast<const bf16x8*>(t + (lane ^ flip(4 * q)) + ahead(4 * q) + rows * kRow);
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(t + lane + ahead(8 * q) + rows * kRow);
      const f32x4 b = *reinterpret_cast<const f32x4*>(t + (lane ^ 16) + ahead(8 * q) + rows * kRow);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.v[i] = a[i], f.v[4 + i] = b[i];
    }
    return f;
  }
  // Column fragments: rows 32 ks + 8 g + tok(0..7), one column a lane: 32 q +
  // 8 (c / 4) + c % 4 + 4 half.  bf16: the lane names 4 columns of one row and
  // receives 4 rows of its column.
  __device__ static inline int lane_col(int g, int c) {
    if constexpr (sizeof(IO) == 2) return offset(8 * g + ((c >> 2) & 1) + ((c >> 1) & 4), c & 3);
    return offset(8 * g, 2 * (c >> 2)) + 4 * (c & 3);
  }
  // (of a tile of 16 columns: the lane's column is c)
  __device__ static inline int lane_col16(int g, int c) {
    if constexpr (sizeof(IO) == 2) return offset(8 * g + ((c >> 2) & 1) + ((c >> 1) & 4), (c & 3) >> 1) + 8 * (c & 1);
    return offset(8 * g, c >> 2) + 4 * (c & 3);
  }
  __device__ static inline Frag<IO> col(const char* t, int lane, int ks, int q, int half) {
    Frag<IO> f;
    if constexpr (sizeof(IO) == 2) {
      union {
        s16x4 h[2];
        bf16x8 v;
      } u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // two rows on: bit 1 of the row, which is bit 1 of an 8-chunk swizzle
        // and bit 0 of a 4-chunk one
        const int x = flip(4 * q) ^ (h ? (kChunks >= 8 ? 32 : 16) : 0);
        char* p = const_cast<char*>(t) + (lane ^ x) + ahead(4 * q) + (32 * ks + 2 * h) * kRow + 8 * half;
        u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
      }
      f.v = u.v;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f.v[e] = *reinterpret_cast<const float*>(t + (lane ^ ((tok(e) ^ half) * 16)) + ahead(8 * q) +
                                                 (32 * ks + tok(e)) * kRow);
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

// `rows` rows `stride` bytes apart: offsets past them read as 0 and write
// nothing.  (A row's columns end before the next row starts.)
__device__ inline __amdgpu_buffer_rsrc_t rows_of(const void* p, int rows, int stride) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, rows * stride, kRsrcFlags);
}
__device__ inline u32x4 buf_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// E (4 or 8) elements as they lie in memory, as fp32, and back.
template <typename IO, int E>
struct Raw {
  static constexpr int kWords = E * static_cast<int>(sizeof(IO)) / 4, kW = kWords < 4 ? kWords : 4, kV = kWords / kW;
  typedef uint32_t vec __attribute__((ext_vector_type(kW)));
  vec v[kV];
  __device__ inline float get(int e) const {
    if constexpr (sizeof(IO) == 2)
      return __uint_as_float(e & 1 ? v[0][e / 2] & 0xffff0000u : v[0][e / 2] << 16);
    else
      return __uint_as_float(v[e / 4][e & 3]);
  }
  __device__ inline void set(const float* f) {
    if constexpr (sizeof(IO) == 2) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) v[0][i] = bf16x2_bits(f[2 * i], f[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i / 4][i & 3] = __float_as_uint(f[i]);
    }
  }
  __device__ inline void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if constexpr (kW == 4)
        v[i] = __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * i, 0, 0));
      else
        v[i] = __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    }
  }
  __device__ inline void store(__amdgpu_buffer_rsrc_t r, uint32_t off) const {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if constexpr (kW == 4)
        __builtin_amdgcn_raw_buffer_store_b128(v[i], r, off + 16 * i, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b64(v[i], r, off, 0, 0);
    }
  }
};

// Largest exponent fields seen: 0x7f80 in one of the halves (the whole, in
// fp32) tells an infinity or a NaN, 2^e is field 127 + e.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <typename IO>
__device__ inline uint32_t top_exponents(u32x4 v, uint32_t top) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(IO) == 2)
      top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, v[i] & 0x7f807f80u),
                                                                   __builtin_bit_cast(u16x2, top)));
    else
      top = max(top, v[i] & 0x7f800000u);
  }
  return top;
}
template <typename IO>
__device__ inline bool reaches(uint32_t top, int exponent) {
  const uint32_t field = static_cast<uint32_t>(127 + exponent) << 7;
  return (top >> 16) >= field || (sizeof(IO) == 2 && (top & 0xffffu) >= field);
}

// Sums over the lanes up to each one, in 64 bits: rotations within the 16-lane
// rows, then each row's last lane broadcast into the next row, and lane 31 into
// the upper half.
template <int CTRL, int ROWS>
__device__ inline double add_moved(double v) {
  const uint64_t b = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, true);
  const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, true);
  return v + __longlong_as_double((static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32) | static_cast<uint32_t>(lo));
}
__device__ inline double lane_sums(double v) {
  v = add_moved<0x111, 0xF>(v);  // row_shr:1
  v = add_moved<0x112, 0xF>(v);
  v = add_moved<0x114, 0xF>(v);
  v = add_moved<0x118, 0xF>(v);
  v = add_moved<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  return add_moved<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
}
__device__ inline double lane_value(double v, int l) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), l);
  return __longlong_as_double((static_cast<uint64_t>(hi) << 32) | lo);
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

// What a chunk's tokens contribute to its exponentials, one value a token and
// wave.  e^(c_i - c_j) is taken as a product of two factors about a reference
// between them: for the 16 x 32 piece (it, ks) of the triangle the sum at token
// 32 ks + 15 where the piece meets the diagonal (near), at token 31 for the
// pieces past the first 32 tokens (far).  The near factors may exceed 1, by as
// much as 16 tokens decay; a chunk where one passes 2^kSteep takes each
// exponential by itself.  The two factors are multiplied with each other before
// anything else (one of them alone, next to large inputs, would pass the largest
// fp32, next to small ones the smallest): what the inputs meet is the decay.  A
// time step below 2^-kSteep, whose column factor could leave the normal range,
// makes a chunk steep as well (8 x 4096 tokens of 80 heads: 593 us at decays of 2^-3 a
// token, 617 us at 2^-4.5, where every chunk is steep).
constexpr float kSteep = 60.0f;
// From here on a value of x, or of C B^T, takes the token-by-token walk, as an
// infinity does: below it, and with the time steps and growth below, no product
// that the chunked form makes of a chunk's own tokens overflows by itself.
constexpr int kLargeExponent = 60;
// A chunk is walked token by token where a time step lies past kLargeStep (or is
// not finite: the sums over the tokens would be, and differences of those NaN), a
// token grows the state by more than 2^kGrowth (2^32 over a chunk), or a decay
// rate overflows.
constexpr float kLargeStep = 0x1p20f;
constexpr float kGrowth = 0.5f;
// Values that are formed anew at each place that uses them.  The walk's loop
// needs nearly every register for its tiles: addresses kept across it would push
// them out to memory, and each of their reloads would wait for every load in
// flight.
__device__ inline int anew(int v) {
  asm volatile("" : "+s"(v));
  return v;
}
__device__ inline int thread_anew() {
  int v = threadIdx.x;
  asm volatile("" : "+v"(v));
  return v;
}
// Keeps the reads of one step from moving up into the step before, where their
// registers are still in use.
__device__ inline void step_end() { __builtin_amdgcn_sched_barrier(0); }

template <int Q>
struct Times {
  float enter[Q];       // e^c_i
  float row_near[Q];    // e^(c_i - near)
  float col_near[Q];    // delta_j e^(near - c_j)
  float row_far[Q];     // e^(c_i - far), i >= 32
  float col_far[Q];     // delta_j e^(far - c_j), j < 32
  float left[Q];        // delta_j e^(c_Q - c_j)
  float sum[2][Q];      // c_i as two floats, in powers of two
  float delta[Q];
};

template <int Q>
struct SumTimes {
  float left[Q], delta[Q];
};

template <typename IO, int NP, int Q>
struct Shape {
  static constexpr int kUnits = Q == 64 ? 6 : 2;  // 32 x 16 pieces of the lower triangle
  using BC = Tile<IO, NP>;
  using X = Tile<IO, kCols>;
  struct Walk {
    char b[Q * NP * sizeof(IO)];
    char c[Q * NP * sizeof(IO)];
    char x[kWaves][Q * kCols * sizeof(IO)];
    f32x4 s[kUnits * 2][64];
    Times<Q> time[2][kWaves];
    int odd[2];  // a chunk is walked token by token
  };
  struct Sum {
    char b[Q * NP * sizeof(IO)];
    alignas(16) char c[16];  // (no C)
    char x[kWaves][Q * kCols * sizeof(IO)];
    SumTimes<Q> time[2][kWaves];
    int odd[2];
  };
};

// AGG: only what a segment adds to a zero state, and its decay.  VEC: rows are
// whole 16-byte vectors (else element by element at their ends).
// NT: accumulator tiles over a wave's columns, 16 each.
template <typename IO, int NP, int Q, int NT, bool AGG, bool VEC>
__global__ __launch_bounds__(256, 2) void head_scan_kernel(HeadScanArgs a) {
  using S = Shape<IO, NP, Q>;
  using BC = typename S::BC;
  using X = typename S::X;
  constexpr int kE = 16 / sizeof(IO);
  constexpr int kES = sizeof(IO);
  constexpr int kK = NP / 32;                          // K-steps over the states
  constexpr int kT = Q / 32;                           // K-steps over the tokens
  constexpr int kLoadBC = Q * BC::kChunks / 256;       // 16-byte loads a thread
  constexpr int kChunksX = NT * kES;                   // 16-byte chunks of a row of x
  constexpr int kLoadX = Q * kChunksX / 64;            // 16-byte loads a lane
  constexpr int kRowsBC = 256 / BC::kChunks, kRowsX = 64 / kChunksX;  // rows between them
  constexpr int kOut = 4 * NT;                         // columns of a token that a lane writes
  constexpr int kParts = sizeof(IO) == 2 ? 2 : 1;      // of an fp32 operand of the outputs
  constexpr int kAddParts = sizeof(IO) == 2 ? 3 : 1;   // of one of the state's addends
  using Lds = std::conditional_t<AGG, typename S::Sum, typename S::Walk>;
  __shared__ __attribute__((aligned(16))) Lds lds;

  const int wave = uniform(threadIdx.x >> 6);

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
  const int begin = uniform(sp.begin + w.seg * per);
  const int end = uniform(min(sp.end, begin + per));
  const bool cut = w.nseg > 1;
  const bool from_cache = resumes(a.q, w.seq);
  if (len == 0 && from_cache) return;
  if (AGG && w.seg == w.nseg - 1) return;  // nothing enters after it

  const bool on = job < jobs;
  const int h = grp * (a.heads / a.groups) + (on ? job / a.ptiles : 0);
  const int p0 = (on ? job % a.ptiles : 0) * 16 * NT;
  const int pc = on ? a.headdim - p0 : 0;              // this tile's columns
  const int64_t hp = static_cast<int64_t>(h) * a.headdim + p0;
  float* cache = a.state + slot * a.sstate + hp * a.dstate;
  float* part = cut ? a.parts + (static_cast<int64_t>(w.index) * a.heads * a.headdim + hp) * a.dstate : nullptr;

  // the state: tile [n = 32 q + 8 g + 4 tn + r][p = 8 (c / 4) + c % 4 + 4 tp], or p = c
  f32x4 st[kK][2][NT];
  // an infinite state has no second part; one that would round to an infinite
  // first part is walked token by token
  bool split = true, huge = false;
  auto column = [](int th) { return NT == 2 ? 8 * ((th >> 2) & 3) + (th & 3) : th & 15; };
  auto lane_colx = [](int g, int c) { return NT == 2 ? X::lane_col(g, c) : X::lane_col16(g, c); };
  // where this tile's state lies in memory: what a cut prompt's segment enters
  // with or adds, or the prompt's cache entry
  float* home = cut ? part : cache;
  auto state_in = [&](bool from) __attribute__((always_inline)) {
    const int th = thread_anew(), n0 = 8 * ((th >> 4) & 3), N = anew(a.dstate);
    const float* at = home + static_cast<int64_t>(column(th)) * N + n0;
    const int ps = pc - column(th);
    bool over = false, near = false;
#pragma unroll
    for (int q = 0; q < kK; ++q)
#pragma unroll
      for (int tp = 0; tp < NT; ++tp) {
        float v[8] = {};
        if (from) load_part<float, 8>(at + 4 * tp * N + 32 * q, 4 * tp < ps ? N - n0 - 32 * q : 0, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          st[q][e >> 2][tp][e & 3] = v[e];
          over |= !(fabsf(v[e]) < INFINITY);
          near |= fabsf(v[e]) >= 0x1p127f && fabsf(v[e]) < INFINITY;
        }
        step_end();
      }
    if constexpr (kParts > 1 && !AGG) {
      split = __ballot(over) == 0;
      huge = __ballot(near) != 0;
    }
  };
  auto state_out = [&]() __attribute__((always_inline)) {
    const int th = thread_anew(), n0 = 8 * ((th >> 4) & 3), N = anew(a.dstate);
    float* at = home + static_cast<int64_t>(column(th)) * N + n0;
    const int ps = pc - column(th);
#pragma unroll
    for (int q = 0; q < kK; ++q)
#pragma unroll
      for (int tp = 0; tp < NT; ++tp) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = st[q][e >> 2][tp][e & 3];
        store_part<float, 8>(at + 4 * tp * N + 32 * q, 4 * tp < ps ? N - n0 - 32 * q : 0, v);
        step_end();
      }
  };
  state_in(!AGG && (cut || from_cache));

  const float rate = -expf(a.A_log[h]) * kLog2e;
  const float bias = a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f;
  const float skip = a.D != nullptr ? a.D[h] : 0.0f;

  // rows of the chunk to be fetched next, and of the one being walked
  const IO* xf = static_cast<const IO*>(a.x) + begin * a.sx[0] + h * a.sx[1] + p0;
  const IO* Bf = static_cast<const IO*>(a.B) + begin * a.sB[0] + grp * a.sB[1];
  const IO* Cf = static_cast<const IO*>(a.C) + begin * a.sC[0] + grp * a.sC[1];
  const IO* zw = static_cast<const IO*>(a.z) + begin * a.sz[0] + h * a.sz[1] + p0;
  IO* ow = static_cast<IO*>(a.out) + begin * a.so[0] + h * a.so[1] + p0;
  const bool gate = a.z != nullptr;

  u32x4 pb[kLoadBC], pcc[AGG ? 1 : kLoadBC], px[kLoadX];
  auto fetch = [&](int t) __attribute__((always_inline)) {
    const int th = thread_anew();
    // this thread's chunks of B and C, and this lane's of x: row and column of the first
    const int rb = th / BC::kChunks, nb = th % BC::kChunks * kE;
    const int rx = (th & 63) / kChunksX, nx = (th & 63) % kChunksX * kE;
    if constexpr (VEC) {
      // byte offsets from the chunk's first row (a tile spans less than 2 GiB)
      const int eX = static_cast<int>(a.sx[0]) * kES, eB = static_cast<int>(a.sB[0]) * kES;
      const int eC = static_cast<int>(a.sC[0]) * kES;
      const int rows = max(min(end - t, Q), 0);
      uint32_t o = nx < pc ? rx * eX + nx * kES : kOffNone;
      const auto rX = rows_of(xf, rows, eX);
#pragma unroll
      for (int i = 0; i < kLoadX; ++i, o += kRowsX * eX) px[i] = buf_load16(rX, o);
      o = nb < a.dstate ? rb * eB + nb * kES : kOffNone;
      const auto rB = rows_of(Bf, rows, eB);
#pragma unroll
      for (int i = 0; i < kLoadBC; ++i, o += kRowsBC * eB) pb[i] = buf_load16(rB, o);
      if constexpr (!AGG) {
        o = nb < a.dstate ? rb * eC + nb * kES : kOffNone;
        const auto rC = rows_of(Cf, rows, eC);
#pragma unroll
        for (int i = 0; i < kLoadBC; ++i, o += kRowsBC * eC) pcc[i] = buf_load16(rC, o);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoadBC; ++i) {
        const int r = rb + i * kRowsBC;
        const int valid = t + r < end ? a.dstate - nb : 0;
        pb[i] = load16<IO>(Bf + r * a.sB[0] + nb, valid);
        if constexpr (!AGG) pcc[i] = load16<IO>(Cf + r * a.sC[0] + nb, valid);
      }
#pragma unroll
      for (int i = 0; i < kLoadX; ++i) {
        const int r = rx + i * kRowsX;
        px[i] = load16<IO>(xf + r * a.sx[0] + nx, t + r < end ? pc - nx : 0);
      }
    }
    xf += Q * a.sx[0];
    Bf += Q * a.sB[0];
    Cf += Q * a.sC[0];
  };
  // one token a lane (past the segment's end: its last one, which is not used)
  auto fetch_dt = [&](int t) __attribute__((always_inline)) {
    const IO* dth = static_cast<const IO*>(a.dt) + h * a.sdt[1];
    return dth[min(t + (thread_anew() & 63), end - 1) * a.sdt[0]];
  };
  double total = 0.0;   // the segment's decay (AGG)
  float decay = 1.0f;   // of the chunk that times() last formed
  bool steep = false, wild = false;  // of that chunk
  auto times = [&](int t, IO raw, int par) __attribute__((always_inline)) {
    const int lane = thread_anew() & 63;
    float dl = io_traits<IO>::load(&raw) + bias;
    const float sp = softplus(dl);
    dl = a.softplus ? sp : dl;
    dl = lane < Q && t + lane < end ? dl : 0.0f;
    const float power = dl * rate;
    wild = __ballot(!(fabsf(dl) <= kLargeStep && power <= kGrowth && power > -INFINITY)) != 0;
    const double sum = lane_sums(static_cast<double>(power));
    const double last = lane_value(sum, Q - 1);
    decay = long_decay(static_cast<float>(last));
    if (AGG) total += last;
    auto& m = lds.time[par][wave];
    const float left = dl * fast_exp2(static_cast<float>(last - sum));
    if constexpr (AGG) {
      if (Q == 64 || lane < Q) {
        m.left[lane] = left;
        m.delta[lane] = dl;
      }
    } else {
      const double n0 = lane_value(sum, 15), n1 = lane_value(sum, 47), far = lane_value(sum, 31);
      const float dn = static_cast<float>(sum - (Q == 64 && lane >= 32 ? n1 : n0)), df = static_cast<float>(sum - far);
      // far factors that are used: rows from 32 on, columns before
      const float grow = lane < 32 ? -df : df;
      const bool tiny = dl != 0.0f && fabsf(dl) < fast_exp2(-kSteep);
      steep = __ballot((Q == 64 || lane < Q) && (tiny || fabsf(dn) > kSteep || (Q == 64 && grow > kSteep))) != 0;
      const float hi = static_cast<float>(sum);
      if (Q == 64 || lane < Q) {
        m.enter[lane] = long_decay(hi);
        m.row_near[lane] = fast_exp2(dn);
        m.col_near[lane] = dl * fast_exp2(-dn);
        if constexpr (Q == 64) {
          m.row_far[lane] = fast_exp2(df);
          m.col_far[lane] = dl * fast_exp2(-df);
        }
        m.left[lane] = left;
        m.sum[0][lane] = hi;
        m.sum[1][lane] = static_cast<float>(sum - hi);
        m.delta[lane] = dl;
      }
    }
  };

  if (threadIdx.x < 2) lds.odd[threadIdx.x] = 0;
  if (begin < end) {
    fetch(begin);
    times(begin, fetch_dt(begin), 0);
  }
  __syncthreads();
  int par = 0, t = begin;
  for (;;) {
  bool walk = false;
  for (; t < end; t += Q, par ^= 1) {
    // ---- this chunk into LDS
    uint32_t odd = 0;
    const int th = thread_anew();
    const int wB = BC::offset(th / BC::kChunks, th % BC::kChunks);
    const int wX = X::offset((th & 63) / kChunksX, (th & 63) % kChunksX);
#pragma unroll
    for (int i = 0; i < kLoadBC; ++i) {
      *reinterpret_cast<u32x4*>(lds.b + wB + i * kRowsBC * BC::kRow) = pb[i];
      if constexpr (AGG) odd = top_exponents<IO>(pb[i], odd);
      if constexpr (!AGG) *reinterpret_cast<u32x4*>(lds.c + wB + i * kRowsBC * BC::kRow) = pcc[i];
    }
#pragma unroll
    for (int i = 0; i < kLoadX; ++i) {
      *reinterpret_cast<u32x4*>(lds.x[wave] + wX + i * kRowsX * X::kRow) = px[i];
      odd = top_exponents<IO>(px[i], odd);
    }
    if (reaches<IO>(odd, kLargeExponent) || huge || wild) lds.odd[par] = 1;
    const IO raw = fetch_dt(t + Q);
    // the next chunk's rows: in the sums, which have registers to spare, a whole
    // chunk ahead; in the walk, once the outputs have left theirs.  (Past the end:
    // zeros; under a condition the old values would stay live until here.)
    if constexpr (AGG) {
      step_end();
      fetch(t + Q);
    }
    __syncthreads();
    if (threadIdx.x == 0) lds.odd[par ^ 1] = 0;
    if constexpr (AGG) {
      walk = uniform(lds.odd[par]) != 0;
      if (walk) break;
    }
    const auto& m = lds.time[par][wave];

    f32x4 y[AGG ? 1 : Q / 16][NT];
    if constexpr (!AGG) {
      const int th = thread_anew(), c = th & 15, g = (th & 63) >> 4, lane = th & 63;
      const int lrow = BC::lane_row(c, g);
      // ---- C B^T, three tiles [j x i] a wave (Q = 64): tokens j of its half of
      // one 32 with the tiles i that reach it, so that a fragment of B serves two
      // or three tiles, and one of C these and the state's
      constexpr int kPer = S::kUnits * 2 / kWaves;
      const int half = wave & 1;
      const bool upper = Q == 64 && wave >= 2;  // j in 32 .. 63, and one tile of the lower 32
      const int jr = 8 * (c >> 2) + ((c & 1) | ((c & 2) << 1)) + 2 * half;
      const int lj = BC::lane_row(jr, g), lju = upper ? lj + 32 * BC::kRow : lj;
      f32x4 acc[kPer];
      // ---- S C^T: the state's fragments each serve every tile of tokens
#pragma unroll
      for (int q = 0; q < kK; ++q) {
        Frag<IO> sb[NT], cf[Q / 16];
#pragma unroll
        for (int it = 0; it < Q / 16; ++it) cf[it] = BC::row(lds.c, lrow, 16 * it, q);
        const Frag<IO> b = BC::row(lds.b, lju, 0, q);
        if constexpr (Q == 64) {
          const f32x4 z = {0, 0, 0, 0};
          if (upper) {
            const Frag<IO> b0 = BC::row(lds.b, lj, 0, q);
            acc[0] = mma(b, cf[2], q == 0 ? z : acc[0]);
            acc[1] = mma(b, cf[3], q == 0 ? z : acc[1]);
            acc[2] = mma(b0, cf[3], q == 0 ? z : acc[2]);
          } else {
#pragma unroll
            for (int k = 0; k < 3; ++k) acc[k] = mma(b, cf[k], q == 0 ? z : acc[k]);
          }
        } else {
          acc[0] = mma(b, wave >= 2 ? cf[1] : cf[0], q == 0 ? f32x4{0, 0, 0, 0} : acc[0]);
        }
#pragma unroll
        for (int tp = 0; tp < NT; ++tp)
#pragma unroll
          for (int e = 0; e < 8; e += 2) sb[tp].set2(e, st[q][e >> 2][tp][e & 3], st[q][e >> 2][tp][(e & 3) + 1]);
#pragma unroll
        for (int it = 0; it < Q / 16; ++it)
#pragma unroll
          for (int tp = 0; tp < NT; ++tp) y[it][tp] = mma(sb[tp], cf[it], q == 0 ? f32x4{0, 0, 0, 0} : y[it][tp]);
        if (kParts > 1 && split) {
          Frag<IO> rest[NT];
#pragma unroll
          for (int tp = 0; tp < NT; ++tp)
#pragma unroll
            for (int e = 0; e < 8; e += 2)
              rest[tp].set2(e, sb[tp].more(e, st[q][e >> 2][tp][e & 3]), sb[tp].more(e + 1, st[q][e >> 2][tp][(e & 3) + 1]));
#pragma unroll
          for (int it = 0; it < Q / 16; ++it)
#pragma unroll
            for (int tp = 0; tp < NT; ++tp) y[it][tp] = mma(rest[tp], cf[it], y[it][tp]);
        }
      }
      // (an infinity or a NaN in B or C is one in C B^T)
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = max(top, __float_as_uint(acc[k][r]) & 0x7f800000u);
      if (reaches<float>(top, kLargeExponent)) lds.odd[par] = 1;
      // piece (ks, it) is number it (ks = 0) or it + 2
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int unit = Q == 64 ? (upper ? (k < 2 ? 4 + k : 3) : k) : wave >> 1;
        lds.s[2 * unit + half][lane] = acc[k];
      }
      step_end();
      __syncthreads();
      walk = uniform(lds.odd[par]) != 0;
      if (walk) break;
    }

    if constexpr (!AGG) {
      {
        const int th = thread_anew(), c = th & 15, g = (th & 63) >> 4, lane = th & 63;
        const int lxc = lane_colx(g, c);
        const int lx = X::offset(c, kOut * g / kE) + kOut * g % kE * kES;  // columns kOut g of token c
        // the gate, on its way while the chunk's own tokens are added
        Raw<IO, kOut> z[VEC ? Q / 16 : 1];
        if constexpr (VEC) {
          const int eZ = static_cast<int>(a.sz[0]) * kES;
          const auto rZ = rows_of(zw, gate ? min(end - t, Q) : 0, eZ);
          uint32_t o = kOut * g < pc ? c * eZ + kOut * g * kES : kOffNone;
#pragma unroll
          for (int it = 0; it < Q / 16; ++it, o += 16 * eZ) z[it].load(rZ, o);
        }
#pragma unroll
        for (int it = 0; it < Q / 16; ++it) {
          const float ei = m.enter[16 * it + c];
#pragma unroll
          for (int tp = 0; tp < NT; ++tp) y[it][tp] *= ei;
        }
        step_end();
        // the chunk's own tokens
#pragma unroll
        for (int ks = 0; ks < kT; ++ks) {
          Frag<IO> xt[NT];
#pragma unroll
          for (int tp = 0; tp < NT; ++tp) xt[tp] = X::col(lds.x[wave], lxc, ks, 0, tp);
          constexpr int kIt = Q / 16;
          Frag<IO> w[kIt][kParts];
#pragma unroll
          for (int it = 2 * ks; it < kIt; ++it) {
            const int i = 16 * it + c;
            const int unit = ks ? it + 2 : it;
            const bool far = it / 2 > ks;
            const f32x4 s0 = lds.s[2 * unit][lane], s1 = lds.s[2 * unit + 1][lane];
            const int below = 16 * (it & 1) + c - 8 * g;  // token slots up to this one are summed
            float v[8];
            if (!steep) {
              const float row = far ? m.row_far[i] : m.row_near[i];
              const float* col = (far ? m.col_far : m.col_near) + 32 * ks + 8 * g;
              const f32x4 c0 = *reinterpret_cast<const f32x4*>(col), c1 = *reinterpret_cast<const f32x4*>(col + 4);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[e] = (e < 4 ? s0[e & 3] : s1[e & 3]) * (row * (tok(e) < 4 ? c0[tok(e) & 3] : c1[tok(e) & 3]));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int j = 32 * ks + 8 * g + tok(e);
                const float d = (m.sum[0][i] - m.sum[0][j]) + (m.sum[1][i] - m.sum[1][j]);
                v[e] = (e < 4 ? s0[e & 3] : s1[e & 3]) * (fast_exp2(d) * m.delta[j]);
              }
            }
            if (!far) {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = tok(e) <= below ? v[e] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              w[it][0].set2(e, v[e], v[e + 1]);
              if constexpr (kParts > 1) w[it][1].set2(e, w[it][0].more(e, v[e]), w[it][0].more(e + 1, v[e + 1]));
            }
          }
#pragma unroll
          for (int k = 0; k < kParts; ++k)
#pragma unroll
            for (int it = 2 * ks; it < kIt; ++it)
#pragma unroll
              for (int tp = 0; tp < NT; ++tp) y[it][tp] = mma(xt[tp], w[it][k], y[it][tp]);
          step_end();
        }
        const int eO = static_cast<int>(a.so[0]) * kES;
        const auto rO = rows_of(ow, min(end - t, Q), eO);
        uint32_t to = kOut * g < pc ? c * eO + kOut * g * kES : kOffNone;
#pragma unroll
        for (int it = 0; it < Q / 16; ++it) {
          const int i = 16 * it + c;
          // ---- skip, gate, out: lane holds token i, columns kOut g .. kOut g + kOut - 1
          Raw<IO, kOut> xi;
#pragma unroll
          for (int k = 0; k < xi.kV; ++k)
            xi.v[k] = *reinterpret_cast<const typename Raw<IO, kOut>::vec*>(lds.x[wave] + (lx ^ 16 * k) + 16 * it * X::kRow);
          float o[kOut];
#pragma unroll
          for (int e = 0; e < kOut; ++e) o[e] = fmaf(skip, xi.get(e), y[it][e >> 2][e & 3]);
          if constexpr (VEC) {
            if (gate) {
#pragma unroll
              for (int e = 0; e < kOut; ++e) o[e] *= silu(z[it].get(e));
            }
            Raw<IO, kOut> u;
            u.set(o);
            u.store(rO, to);
            to += 16 * eO;
          } else {
            const int n = t + i < end ? pc - kOut * g : 0;
            if (gate) {
              float zz[kOut];
              load_part<IO, kOut>(zw + i * a.sz[0] + kOut * g, n, zz);
#pragma unroll
              for (int e = 0; e < kOut; ++e) o[e] *= silu(zz[e]);
            }
            store_part<IO, kOut>(ow + i * a.so[0] + kOut * g, n, o);
          }
          step_end();
        }
      }
    }

    // ---- the next chunk's rows and time steps
    if constexpr (!AGG) fetch(t + Q);
    step_end();
    const float dec = decay;
    if constexpr (!AGG) times(t + Q, raw, par ^ 1);
    step_end();

    // ---- the state
    {
      const int th = thread_anew(), c = th & 15, g = (th & 63) >> 4;
      const int lcol = BC::lane_col(g, c), lxc = lane_colx(g, c);
#pragma unroll
      for (int q = 0; q < kK; ++q)
#pragma unroll
        for (int tn = 0; tn < 2; ++tn)
#pragma unroll
          for (int tp = 0; tp < NT; ++tp) st[q][tn][tp] *= dec;
#pragma unroll
      for (int ks = 0; ks < kT; ++ks) {
        Frag<IO> xt[NT], v[NT][kAddParts];
#pragma unroll
        for (int tp = 0; tp < NT; ++tp) xt[tp] = X::col(lds.x[wave], lxc, ks, 0, tp);
        const float* left = m.left + 32 * ks + 8 * g;
        const f32x4 l0 = *reinterpret_cast<const f32x4*>(left), l1 = *reinterpret_cast<const f32x4*>(left + 4);
#pragma unroll
        for (int tp = 0; tp < NT; ++tp)
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            float r0 = xt[tp].get(e) * (tok(e) < 4 ? l0[tok(e) & 3] : l1[tok(e) & 3]);
            float r1 = xt[tp].get(e + 1) * (tok(e + 1) < 4 ? l0[tok(e + 1) & 3] : l1[tok(e + 1) & 3]);
#pragma unroll
            for (int k = 0; k < kAddParts; ++k) {
              v[tp][k].set2(e, r0, r1);
              r0 = v[tp][k].more(e, r0);
              r1 = v[tp][k].more(e + 1, r1);
            }
          }
#pragma unroll
        for (int q = 0; q < kK; ++q) {
          Frag<IO> bt[2];
#pragma unroll
          for (int tn = 0; tn < 2; ++tn) bt[tn] = BC::col(lds.b, lcol, ks, q, tn);
#pragma unroll
          for (int k = kAddParts - 1; k >= 0; --k)
#pragma unroll
            for (int tn = 0; tn < 2; ++tn)
#pragma unroll
              for (int tp = 0; tp < NT; ++tp) st[q][tn][tp] = mma(bt[tn], v[tp][k], st[q][tn][tp]);
        }
        step_end();
      }
    }
    if constexpr (AGG) times(t + Q, raw, par ^ 1);
    zw += Q * a.sz[0];
    ow += Q * a.so[0];
    __syncthreads();
  }
  if (!walk) break;
    const auto& m = lds.time[par][wave];
    if (on) {
      // ---- token by token, the state in memory: nothing of this may take
      // registers from the products
      state_out();
      const int th = thread_anew(), g = (th & 63) >> 4, N = anew(a.dstate);
#pragma unroll 1
      for (int i = 0; i < Q && t + i < end; ++i) {
        const float dti = m.delta[i], e = fast_exp2(dti * rate);
#pragma unroll 1
        for (int p = column(th), tp = 0; tp < NT; ++tp, p += 4) {
          const float x = io_traits<IO>::load(reinterpret_cast<const IO*>(lds.x[wave] + X::offset(i, p / kE)) + p % kE);
          float y = 0.0f;
#pragma unroll 1
          for (int n = 8 * g; n < NP; n += 32) {
            const int valid = p < pc ? N - n : 0;
            float* at = home + static_cast<int64_t>(p) * N + n;
            float s[8], b[8], cc[8];
            load_part<float, 8>(at, valid, s);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const int o = BC::offset(i, (n + r) / kE);
              b[r] = io_traits<IO>::load(reinterpret_cast<const IO*>(lds.b + o) + (n + r) % kE);
              cc[r] = AGG ? 0.0f : io_traits<IO>::load(reinterpret_cast<const IO*>(lds.c + o) + (n + r) % kE);
              s[r] = fmaf(e, s[r], dti * x * b[r]);
              if (!AGG && r < valid) y = fmaf(cc[r], s[r], y);
            }
            store_part<float, 8>(at, valid, s);
          }
          if constexpr (!AGG) {
            y += __shfl_xor(y, 16, 64);
            y += __shfl_xor(y, 32, 64);
            if (g == 0 && p < pc) {
              float o = fmaf(skip, x, y);
              if (gate) o *= silu(io_traits<IO>::load(zw + i * a.sz[0] + p));
              io_traits<IO>::store(ow + i * a.so[0] + p, o);
            }
          }
        }
      }
      state_in(true);
    }
    if constexpr (!AGG) fetch(t + Q);
    times(t + Q, fetch_dt(t + Q), par ^ 1);
    zw += Q * a.sz[0];
    ow += Q * a.so[0];
    t += Q;
    par ^= 1;
    __syncthreads();
  }

  // ---- the state that the segment leaves
  if (!on || (!AGG && w.seg < w.nseg - 1)) return;
  if (!AGG) home = cache;
  state_out();
  if (AGG && (threadIdx.x & 63) == 0 && p0 == 0) a.decays[static_cast<int64_t>(w.index) * a.heads + h] = long_decay(static_cast<float>(total));
}

// The states entering the segments of a cut prompt, in place of what the
// segments add (the last one's place holds nothing yet): four states a thread,
// kAhead segments loaded before the first is used.
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
  const float* cache = a.state + slot * a.sstate + i;
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
        for (int e = 0; e < 4; ++e) s[e] = s[e] == 0.0f ? v[k][e] : fmaf(d[k][e], s[e], v[k][e]);  // (d may be infinite)
      }
    }
  }
}

template <typename IO, int NP, int Q, int NT, bool VEC>
hipError_t launch_v(const HeadScanArgs& a, hipStream_t stream) {
  const int64_t tiles = static_cast<int64_t>(a.groups) * ((a.heads / a.groups * a.ptiles + kWaves - 1) / kWaves);
  if (a.cut_slots > 0) {
    head_scan_kernel<IO, NP, Q, NT, true, VEC><<<dim3(static_cast<unsigned>(a.cut_slots * tiles)), 256, 0, stream>>>(a);
    const int64_t blocks = (static_cast<int64_t>(a.heads) * a.headdim * a.dstate + 1023) / 1024;
    head_scan_carry_kernel<<<dim3(static_cast<unsigned>(blocks * a.cut_prompts)), 256, 0, stream>>>(
        a, static_cast<int>(blocks));
  }
  head_scan_kernel<IO, NP, Q, NT, false, VEC>
      <<<dim3(static_cast<unsigned>((a.cut_slots + a.q.seqs) * tiles)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename IO, int NP, int Q>
hipError_t launch_n(const HeadScanArgs& a, hipStream_t stream) {
  if (!a.vec) return launch_v<IO, NP, Q, 2, false>(a, stream);
  return a.narrow ? launch_v<IO, NP, Q, 1, true>(a, stream) : launch_v<IO, NP, Q, 2, true>(a, stream);
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

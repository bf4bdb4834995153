// mss_head.hpp -- shapes, pointers and device helpers of the head-wise
// operations: conv and scan over packed prompts, the one-token step, the norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mss_device.hpp"

namespace mss {

constexpr int kMaxHeadState = 128;
constexpr int kScaleBlock = 128;

// Packed prompts and their cache entries (device pointers).
struct Prompts {
  int tokens, seqs, cache_slots;
  const int32_t* cu;      // [seqs + 1]
  const int32_t* slots;   // [seqs] or null
  const int32_t* resume;  // [seqs] or null
};

struct ConvPromptsArgs {
  Prompts q;
  int dim, width, silu;
  int run;         // rows a wave walks
  int64_t nruns;   // waves along the rows
  int colgroups;   // waves along the channels
  int64_t sx[2], so[2], sw[2], swin;
  const void* x;
  const float* weight;
  const float* bias;
  void* window;
  void* out;
};

struct HeadScanArgs {
  Prompts q;
  int heads, headdim, dstate, groups, softplus;
  int64_t sx[3], sdt[2], sB[3], sC[3], sz[3], so[3], sstate;
  const void* x;
  const void* dt;
  const float* A_log;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* dt_bias;
  float* state;
  void* out;
  int vec;          // rows of x, B, C, z and out are whole aligned 16-byte vectors
  int narrow;       // tiles of 16 columns (vec only), not 32
  int ptiles;       // tiles of a head
  int seg_len;      // longer prompts are cut into segments of at most this many tokens (0: none is)
  int cut_slots;    // room for the segments of all cut prompts
  int cut_prompts;  // at most this many prompts are cut
  float* parts;     // workspace [cut_slots][H][P][N]
  float* decays;    // workspace [cut_slots][H]
};

struct HeadStepArgs {
  int rows, heads, headdim, dstate, groups, width, softplus, cache_slots;
  int64_t sx[2], sdt[2], sw[2], sz[3], so[3], sstate, swin;
  const void* xbc;
  const void* dt;
  const float* A_log;
  const float* weight;
  const float* bias;
  const float* D;
  const void* z;
  const float* dt_bias;
  const int32_t* slots;
  float* state;
  void* window;
  void* out;
};

struct NormArgs {
  int64_t rows;
  int dim;
  int64_t sx, sr, so, sro;
  float eps;
  const void* x;
  const void* res;
  const float* weight;
  void* out;
  float* scale;
  void* res_out;
};

hipError_t launch_conv_prompts(const ConvPromptsArgs& a, bool io_bf16, hipStream_t stream);
hipError_t launch_head_scan(const HeadScanArgs& a, bool io_bf16, hipStream_t stream);
hipError_t launch_head_step(const HeadStepArgs& a, bool io_bf16, hipStream_t stream);
hipError_t launch_norm(const NormArgs& a, bool io_bf16, bool res_bf16, int quant, hipStream_t stream);

// ---------------------------------------------------------------- device side

// Bounds of prompt i, forced into [0, tokens] so that no value in cu_seqlens
// can lead an access out of bounds.
struct Span {
  int begin, end;
};
__device__ inline Span prompt_span(const Prompts& q, int i) {
  const int a = min(max(q.cu[i], 0), q.tokens);
  return {a, min(max(q.cu[i + 1], a), q.tokens)};
}
// The cache entry of prompt (or row) i, or -1 for one that is to be skipped.
__device__ inline int slot_of(const int32_t* slots, int cache_slots, int i) {
  const int s = slots != nullptr ? slots[i] : i;
  return s >= 0 && s < cache_slots ? s : -1;
}
__device__ inline bool resumes(const Prompts& q, int i) {
  return q.resume != nullptr && q.resume[i] != 0;
}
// The prompt that holds row t, or seqs for a row behind the last one: the
// prompts that end at or before t, counted 64 at a time (one load for most
// batches, where a bisection would wait for one load after another).  Every
// lane of the wave takes part.
__device__ inline int prompt_of(const Prompts& q, int t) {
  int count = 0;
  for (int base = 0; base < q.seqs; base += 64) {
    const int i = base + static_cast<int>(threadIdx.x & 63);
    const int n = __popcll(__ballot(i < q.seqs && q.cu[min(i, q.seqs - 1) + 1] <= t));
    count += n;
    if (n < 64) break;
  }
  return uniform(count);
}

// Vectors of V elements as fp32.  Rows start at any element, so the accesses
// are declared element-aligned; the hardware takes unaligned 16-byte accesses.
template <typename IO, int V>
struct vecio;
template <int V>
struct vecio<float, V> {
  typedef float __attribute__((ext_vector_type(V), aligned(4))) raw;
  __device__ static inline void load(const float* p, float* v) {
    const raw q = *reinterpret_cast<const raw*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = q[i];
  }
  __device__ static inline void store(float* p, const float* v) {
    raw q;
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = v[i];
    *reinterpret_cast<raw*>(p) = q;
  }
  // past the caches
  __device__ static inline void store_past(float* p, const float* v) {
    raw q;
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = v[i];
    __builtin_nontemporal_store(q, reinterpret_cast<raw*>(p));
  }
};
template <int V>
struct vecio<bf16_t, V> {
  typedef uint32_t __attribute__((ext_vector_type(V / 2), aligned(2))) raw;
  __device__ static inline void load(const bf16_t* p, float* v) {
    const raw q = *reinterpret_cast<const raw*>(p);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
  __device__ static inline void store(bf16_t* p, const float* v) {
    raw q;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) q[i] = bf16x2_bits(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<raw*>(p) = q;
  }
};

// The first `n` of V elements (n <= 0: none); the others read as 0.
template <typename IO, int V>
__device__ inline void load_part(const IO* p, int n, float* v) {
  if (n >= V) {
    vecio<IO, V>::load(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < n ? io_traits<IO>::load(p + i) : 0.0f;
  }
}
template <typename IO, int V, bool PAST = false>
__device__ inline void store_part(IO* p, int n, const float* v) {
  if (n >= V) {
    if constexpr (PAST)
      vecio<IO, V>::store_past(p, v);
    else
      vecio<IO, V>::store(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) io_traits<IO>::store(p + i, v[i]);
  }
}

}  // namespace mss

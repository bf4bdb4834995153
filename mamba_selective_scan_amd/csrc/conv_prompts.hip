// conv_prompts.hip -- causal depthwise conv1d with optional SiLU over packed
// prompts, with a cache of windows by slot, for gfx950 (wave64).
//
//   pre[t,d] = bias[d] + sum_k w[d,k] * x~[t-(W-1)+k,d]
//   out[t,d] = silu(pre) or pre
// where x~ extends each prompt to the left with its cached window or zeros
// (the conv of conv1d.hip, prompt by prompt).
//
// A stream like conv1d.hip's: bound by HBM bandwidth.  A wave walks a run of
// packed rows with a 16-byte vector of channels per lane and the last W-1 rows
// in registers, whatever prompts the run crosses.  The rows that reach into a
// cached window are the first W-1 of a prompt: those, and the window that the
// prompt leaves, belong to a job of their own (one per prompt and channel
// vector, in the same launch), so a window has one reader, which is also its
// writer, however many waves share the prompt.  5376 channels x 32768 rows in
// bf16, 24 prompts: 155 us, 4.5 TB/s, where a copy reaches 5.1 (165 us with
// four rows ahead; runs of 16 or 64 rows: 169 and 163 us).
#include "mss_head.hpp"

namespace mss {
namespace {

constexpr int kWaves = 4;   // jobs per workgroup
constexpr int kAhead = 8;   // rows loaded before the first of them is used

// A row's vector of channels as it lies in memory (a load in flight holds no
// more registers than its bytes), and as fp32.
template <typename IO, int V>
struct Row {
  typename vecio<IO, V>::raw q;
  __device__ inline float get(int i) const {
    if constexpr (sizeof(IO) == 4)
      return q[i];
    else
      return __uint_as_float(i & 1 ? q[i / 2] & 0xffff0000u : q[i / 2] << 16);
  }
};
template <typename IO, int V, bool UNIT>
__device__ inline Row<IO, V> load_cols(const IO* row, int64_t sd, int n) {
  Row<IO, V> r;
  if (UNIT && n >= V) {
    r.q = *reinterpret_cast<const typename vecio<IO, V>::raw*>(row);
    return r;
  }
  union {
    IO e[V];
    Row<IO, V> r;
  } u;
  u.r.q = typename vecio<IO, V>::raw(0);
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) u.e[i] = row[i * sd];
  return u.r;
}
template <typename IO, int V, bool UNIT>
__device__ inline void store_cols(IO* row, int64_t sd, int n, const float* v) {
  if constexpr (UNIT) {
    store_part<IO, V>(row, n, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) io_traits<IO>::store(row + i * sd, v[i]);
  }
}

template <typename IO, int W, bool UNIT>
__global__ __launch_bounds__(64 * kWaves) void conv_prompts_kernel(ConvPromptsArgs a) {
  constexpr int V = 16 / sizeof(IO);
  constexpr int H = W - 1;  // rows of history
  const int lane = threadIdx.x & 63;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kWaves + uniform(threadIdx.x >> 6);
  const int64_t which = job / a.colgroups;
  const int c = (static_cast<int>(job % a.colgroups) * 64 + lane) * V;
  const int nc = min(V, a.dim - c);  // this lane's channels (none when <= 0)
  if (which >= a.nruns + a.q.seqs) return;

  const IO* x = static_cast<const IO*>(a.x) + static_cast<int64_t>(c) * a.sx[1];
  IO* out = static_cast<IO*>(a.out) + static_cast<int64_t>(c) * a.so[1];
  float wk[W][V], bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // (a weight whose taps lie together, as layers hold it, in one vector)
    const int d = min(c + i, a.dim - 1);
    if (W == 4 && a.sw[1] == 1) {
      float t[4];
      vecio<float, 4>::load(a.weight + d * a.sw[0], t);
#pragma unroll
      for (int k = 0; k < W; ++k) wk[k][i] = t[k];
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) wk[k][i] = a.weight[d * a.sw[0] + k * a.sw[1]];
    }
    bias[i] = 0.0f;
  }
  if (a.bias != nullptr) load_part<float, V>(a.bias + c, nc, bias);
  Row<IO, V> win[H > 0 ? H : 1];
  auto slide = [&](const Row<IO, V>& v) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k + 1 < H; ++k) win[k] = win[k + 1];
    if constexpr (H > 0) win[H - 1] = v;
  };
  auto filter = [&](const Row<IO, V>& v, float* y) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float acc = bias[i];
#pragma unroll
      for (int k = 0; k < H; ++k) acc = fmaf(wk[k][i], win[k].get(i), acc);
      acc = fmaf(wk[H][i], v.get(i), acc);
      y[i] = a.silu ? silu(acc) : acc;
    }
  };

  if (which < a.nruns) {
    // rows [t, t1) that no window reaches
    int t = static_cast<int>(which) * a.run;
    const int t1 = min(t + a.run, a.q.tokens);
    int s = prompt_of(a.q, t);
    if (s >= a.q.seqs) return;
    Span sp = prompt_span(a.q, s);
    bool keep = slot_of(a.q.slots, a.q.cache_slots, s) >= 0;
#pragma unroll
    for (int k = 0; k < H; ++k) win[k] = load_cols<IO, V, UNIT>(x + max(t - H + k, 0) * a.sx[0], a.sx[1], nc);
    for (; t < t1; t += kAhead) {
      Row<IO, V> v[kAhead];
#pragma unroll
      for (int r = 0; r < kAhead; ++r)
        v[r] = load_cols<IO, V, UNIT>(x + min(t + r, t1 - 1) * a.sx[0], a.sx[1], nc);
#pragma unroll
      for (int r = 0; r < kAhead; ++r) {
        if (t + r < t1) {
          while (t + r >= sp.end) {  // into the next prompt that has this row
            if (++s >= a.q.seqs) return;
            sp = prompt_span(a.q, s);
            keep = slot_of(a.q.slots, a.q.cache_slots, s) >= 0;
          }
          if (keep && t + r - sp.begin >= H) {
            float y[V];
            filter(v[r], y);
            store_cols<IO, V, UNIT>(out + (t + r) * a.so[0], a.so[1], nc, y);
          }
          slide(v[r]);
        }
      }
    }
    return;
  }

  if constexpr (H > 0) {
    const int s = static_cast<int>(which - a.nruns);
    const int slot = slot_of(a.q.slots, a.q.cache_slots, s);
    if (slot < 0 || nc <= 0) return;
    const Span sp = prompt_span(a.q, s);
    const int len = sp.end - sp.begin;
    const bool from_cache = resumes(a.q, s);
    if (len == 0 && from_cache) return;
    IO* cache = static_cast<IO*>(a.window) + slot * a.swin + static_cast<int64_t>(c) * H;
    union Loose {
      IO e[V];
      Row<IO, V> r;
    };
#pragma unroll
    for (int k = 0; k < H; ++k) {
      Loose u;
      u.r.q = typename vecio<IO, V>::raw(0);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (from_cache && i < nc) u.e[i] = cache[i * H + k];
      win[k] = u.r;
    }
    // the first H rows, with the window sliding over them; after them the
    // window holds the samples before row min(len, H)
#pragma unroll
    for (int r = 0; r < H; ++r) {
      if (r < len) {
        float y[V];
        const Row<IO, V> v = load_cols<IO, V, UNIT>(x + (sp.begin + r) * a.sx[0], a.sx[1], nc);
        filter(v, y);
        store_cols<IO, V, UNIT>(out + (sp.begin + r) * a.so[0], a.so[1], nc, y);
        slide(v);
      }
    }
    if (len > H) {
#pragma unroll
      for (int k = 0; k < H; ++k)
        win[k] = load_cols<IO, V, UNIT>(x + (sp.end - H + k) * a.sx[0], a.sx[1], nc);
    }
#pragma unroll
    for (int k = 0; k < H; ++k) {
      Loose u;
      u.r = win[k];
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < nc) cache[i * H + k] = u.e[i];
    }
  }
}

template <typename IO, int W>
hipError_t launch_w(const ConvPromptsArgs& a, hipStream_t stream) {
  const int64_t jobs = (a.nruns + (W > 1 ? a.q.seqs : 0)) * a.colgroups;
  if (jobs == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>((jobs + kWaves - 1) / kWaves)), block(64 * kWaves);
  if (a.sx[1] == 1 && a.so[1] == 1)
    conv_prompts_kernel<IO, W, true><<<grid, block, 0, stream>>>(a);
  else
    conv_prompts_kernel<IO, W, false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_t(const ConvPromptsArgs& a, hipStream_t stream) {
  switch (a.width) {
    case 1: return launch_w<IO, 1>(a, stream);
    case 2: return launch_w<IO, 2>(a, stream);
    case 3: return launch_w<IO, 3>(a, stream);
    default: return launch_w<IO, 4>(a, stream);
  }
}

}  // namespace

hipError_t launch_conv_prompts(const ConvPromptsArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_t<bf16_t>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace mss

// causal_conv.cu -- short depthwise causal conv1d over prompts, and for one new
// token of every sequence.
//
//   out_t[c] = act(bias[c] + sum_{k<K} w[c][k] * x_{t-(K-1)+k}[c])
//
// within each sequence; the K-1 positions before its first token come from the
// cache (carry) or are zero.  Accumulated in fp32 in ascending k, rounded once.
//
// Bound by memory: every input is read once and every output written once, with
// K FMAs (and an exp and a reciprocal) a value.  A thread owns 16 bytes of
// channels and walks kTokens rows with the last K-1 rows in registers, so x is
// read once but for the K-1 rows before each walk (from L2).
#include <cuda_runtime.h>

#include "sequence.cuh"

namespace b200conv {
namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 32;   // rows of one thread's walk
constexpr int kBatch = 8;     // rows loaded together

struct ConvArgs {
  const void *x, *w, *bias;
  const int *offsets, *slots;
  void *state, *out;
  int n, l, c, state_slots, silu, carry;
  long long x_sn, x_st, o_sn, o_st;
  int groups;       // channel vectors a row
  int tiles;        // walks a sequence (dense) or a call (packed)
};

// The taps of V channels: [V][K] in memory, [K][V] in registers.
template <typename T, int K, int V, bool VEC>
__device__ __forceinline__ void load_taps(const T* p, float (&w)[K][V]) {
  float flat[K][V];
#pragma unroll
  for (int i = 0; i < K; ++i) load_f32<T, V, VEC>(p + i * V, flat[i]);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][v] = flat[(v * K + k) / V][(v * K + k) % V];
}

template <typename T, int K, int V, bool VEC>
struct Walk {
  const ConvArgs& p;
  int ch;
  float w[K][V], b[V];

  __device__ __forceinline__ Walk(const ConvArgs& args, int channel) : p(args), ch(channel) {
    load_taps<T, K, V, VEC>(static_cast<const T*>(p.w) + (long long)ch * K, w);
    if (p.bias) {
      load_f32<T, V, VEC>(static_cast<const T*>(p.bias) + ch, b);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] = 0.0f;
    }
  }

  __device__ __forceinline__ T* state_row(int slot, int j) const {
    return static_cast<T*>(p.state) + ((long long)slot * (K - 1) + j) * p.c + ch;
  }
  // Row `pos` of a sequence whose first row is x; before the first, the cache or zero.
  __device__ __forceinline__ void row(const T* x, int pos, int slot, float (&v)[V]) const {
    if (pos >= 0) {
      load_f32<T, V, VEC>(x + pos * p.x_st, v);
    } else if (p.carry) {
      load_f32<T, V, VEC>(state_row(slot, K - 1 + pos), v);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.0f;
    }
  }

  // Positions [from, to) of the sequence whose rows start at x and out.
  __device__ __forceinline__ void run(const T* x, T* out, int from, int to, int slot) const {
    if (from >= to) return;
    float win[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) row(x, from - (K - 1) + j, slot, win[j]);
    for (int at = from; at < to; at += kBatch) {
      float in[kBatch][V];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (at + u < to) load_f32<T, V, VEC>(x + (at + u) * p.x_st, in[u]);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (at + u >= to) break;
        float acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          acc[v] = b[v];
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const int j = u + k - (K - 1);      // row at + j
            acc[v] = fmaf(w[k][v], j < 0 ? win[j + K - 1][v] : in[j < 0 ? 0 : j][v], acc[v]);
          }
          if (p.silu) acc[v] = silu(acc[v]);
        }
        store_f32<T, V, VEC>(out + (at + u) * p.o_st, acc);
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = in[kBatch - (K - 1) + j][v];
    }
  }

  // The new window: the last K-1 rows, older ones from the old window where the
  // sequence is shorter.  The thread that reads a sequence's old window is the
  // one that calls this, after its reads.
  __device__ __forceinline__ void keep(const T* x, int len, int slot) const {
    float v[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) row(x, len - (K - 1) + j, slot, v[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_f32<T, V, VEC>(state_row(slot, j), v[j]);
  }
};

template <typename T, int K, int V, bool VEC>
__global__ void __launch_bounds__(kThreads) causal_conv_kernel(const ConvArgs p) {
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long walk_id = id / p.groups;
  const int ch = (int)(id - walk_id * p.groups) * V;
  const T* x = static_cast<const T*>(p.x) + ch;
  T* out = static_cast<T*>(p.out) + ch;
  if (!p.offsets) {
    if (walk_id >= (long long)p.n * p.tiles) return;
    const int seq = (int)(walk_id / p.tiles);
    const int from = (int)(walk_id - (long long)seq * p.tiles) * kTokens;
    const int slot = slot_of(p.slots, seq, p.state_slots);
    if (slot < 0) return;
    const Walk<T, K, V, VEC> walk(p, ch);
    x += seq * p.x_sn;
    walk.run(x, out + seq * p.o_sn, from, min(from + kTokens, p.l), slot);
    if (p.state && from == 0) walk.keep(x, p.l, slot);
    return;
  }
  if (walk_id >= p.tiles) return;
  const int first = (int)walk_id * kTokens;
  const bool last_walk = walk_id == p.tiles - 1;
  const int end = last_walk ? p.l : first + kTokens;
  // The sequence that row `first` lies in, or the first one that starts there or
  // later: the first with an end above `first`, or that starts at or after it.
  int lo_seq = 0, hi_seq = p.n;
  while (lo_seq < hi_seq) {
    const int mid = (lo_seq + hi_seq) >> 1;
    if (__ldg(p.offsets + mid + 1) > first || __ldg(p.offsets + mid) >= first) hi_seq = mid;
    else lo_seq = mid + 1;
  }
  if (lo_seq >= p.n) return;
  const Walk<T, K, V, VEC> walk(p, ch);
  for (int seq = lo_seq; seq < p.n; ++seq) {
    int lo, hi;
    packed_range(p.offsets, seq, p.l, &lo, &hi);
    if (lo >= end && !last_walk) break;
    const int slot = slot_of(p.slots, seq, p.state_slots);
    if (slot < 0) continue;
    const T* xs = x + lo * p.x_st;
    T* os = out + lo * p.o_st;
    // The first K-1 tokens read the old window, which the walk that holds the
    // sequence's first row replaces: that walk computes them all, even past its
    // end, and the next one begins after them.
    if (lo >= first) {
      walk.run(xs, os, 0, min(hi, max(end, lo + K - 1)) - lo, slot);
      if (p.state) walk.keep(xs, hi - lo, slot);
    } else {
      walk.run(xs, os, max(first, lo + K - 1) - lo, min(hi, end) - lo, slot);
    }
  }
}

struct StepArgs {
  const void *x, *w, *bias;
  const int* slots;
  void *state, *out;
  int n, c, state_slots, silu;
  long long x_sn, o_sn;
  int groups;
};

template <typename T, int K, int V, bool VEC>
__global__ void __launch_bounds__(kThreads) causal_conv_step_kernel(const StepArgs p) {
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long seq = id / p.groups;
  if (seq >= p.n) return;
  const int ch = (int)(id - seq * p.groups) * V;
  const int slot = slot_of(p.slots, (int)seq, p.state_slots);
  if (slot < 0) return;
  T* state = static_cast<T*>(p.state) + (long long)slot * (K - 1) * p.c + ch;
  float win[K][V], acc[V];
#pragma unroll
  for (int k = 0; k < K - 1; ++k) load_f32<T, V, VEC>(state + (long long)k * p.c, win[k]);
  load_f32<T, V, VEC>(static_cast<const T*>(p.x) + seq * p.x_sn + ch, win[K - 1]);
  float w[K][V];
  load_taps<T, K, V, VEC>(static_cast<const T*>(p.w) + (long long)ch * K, w);
  if (p.bias) {
    load_f32<T, V, VEC>(static_cast<const T*>(p.bias) + ch, acc);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < K; ++k) acc[v] = fmaf(w[k][v], win[k][v], acc[v]);
    if (p.silu) acc[v] = silu(acc[v]);
  }
  store_f32<T, V, VEC>(static_cast<T*>(p.out) + seq * p.o_sn + ch, acc);
#pragma unroll
  for (int k = 0; k < K - 1; ++k) store_f32<T, V, VEC>(state + (long long)k * p.c, win[k + 1]);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, int K>
cudaError_t conv_typed(ConvArgs p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  p.tiles = p.l > 0 ? (p.l - 1) / kTokens + 1 : 1;   // without rows there are still windows to write
  const bool vec = on16(p.x) && on16(p.w) && on16(p.out) && on16(p.state) && on16(p.bias) && p.c % V == 0 && p.x_sn % V == 0 &&
                   p.x_st % V == 0 && p.o_sn % V == 0 && p.o_st % V == 0;
  p.groups = vec ? p.c / V : p.c;
  const long long walks = p.offsets ? p.tiles : (long long)p.n * p.tiles;
  const long long blocks = (walks * p.groups + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (vec) causal_conv_kernel<T, K, V, true><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  else causal_conv_kernel<T, K, 1, false><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int K>
cudaError_t step_typed(StepArgs p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = on16(p.x) && on16(p.w) && on16(p.out) && on16(p.state) && on16(p.bias) && p.c % V == 0 && p.x_sn % V == 0 &&
                   p.o_sn % V == 0;
  p.groups = vec ? p.c / V : p.c;
  const long long blocks = ((long long)p.n * p.groups + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (vec) causal_conv_step_kernel<T, K, V, true><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  else causal_conv_step_kernel<T, K, 1, false><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// f(K) for the tap counts of the two operators, 2 .. 8.
template <typename F>
cudaError_t with_taps(int k, F f) {
  switch (k) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5: return f(std::integral_constant<int, 5>{});
    case 6: return f(std::integral_constant<int, 6>{});
    case 7: return f(std::integral_constant<int, 7>{});
    case 8: return f(std::integral_constant<int, 8>{});
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_causal_conv(const conv1d_causal_desc_t& d, conv_dtype_t dt, const void* x, const void* w,
                               const void* bias, const int* offsets, void* state, const int* slots, void* out,
                               cudaStream_t s) {
  ConvArgs p{};
  p.x = x; p.w = w; p.bias = bias; p.offsets = offsets; p.slots = slots; p.state = state; p.out = out;
  p.n = d.n; p.l = d.l; p.c = d.c; p.state_slots = d.state_slots;
  p.silu = d.activation == CONV_ACT_SILU;
  p.carry = d.carry && state;
  p.x_sn = d.x_stride[0]; p.x_st = d.x_stride[1]; p.o_sn = d.out_stride[0]; p.o_st = d.out_stride[1];
  return with_taps(d.k, [&](auto k) {
    switch (dt) {
      case CONV_F16: return conv_typed<__half, k()>(p, s);
      case CONV_BF16: return conv_typed<__nv_bfloat16, k()>(p, s);
      default: return conv_typed<float, k()>(p, s);
    }
  });
}

cudaError_t launch_causal_conv_step(const conv1d_causal_desc_t& d, conv_dtype_t dt, const void* x, const void* w,
                                    const void* bias, void* state, const int* slots, void* out, cudaStream_t s) {
  StepArgs p{};
  p.x = x; p.w = w; p.bias = bias; p.slots = slots; p.state = state; p.out = out;
  p.n = d.n; p.c = d.c; p.state_slots = d.state_slots;
  p.silu = d.activation == CONV_ACT_SILU;
  p.x_sn = d.x_stride[0]; p.o_sn = d.out_stride[0];
  return with_taps(d.k, [&](auto k) {
    switch (dt) {
      case CONV_F16: return step_typed<__half, k()>(p, s);
      case CONV_BF16: return step_typed<__nv_bfloat16, k()>(p, s);
      default: return step_typed<float, k()>(p, s);
    }
  });
}

}  // namespace b200conv

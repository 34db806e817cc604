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
// channels and walks up to 64 rows with the last K-1 rows in registers, so x is
// read once but for the K-1 rows before each walk (from L2).  Rows come through a
// ring of eight in shared memory that each thread fills for itself with cp.async:
// the bytes in flight then cost no registers, of which the taps and the window
// (2K - 1 values a channel) already take most.  4 x 4096 rows of 4096 bf16 channels,
// K = 4, silu: 50 us = 5.4 TB/s, 82 % of the copy rate; with the rows in flight held
// in registers (8 at a time, twice) 64 us, without any in flight while the others
// are worked on 91 us.  Two or four rows worked on together, eight channel bytes a
// thread, or registers capped for more blocks an SM: 52 to 120 us.
// Where 16-byte accesses are not possible a thread owns one channel: 4096 rows of 4092
// bf16 channels 26 us, 2.6 TB/s.
#include <cuda_runtime.h>

#include "sequence.cuh"

namespace b200conv {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;      // rows on their way
constexpr int kLoose = 4;      // rows loaded together where 16-byte accesses are not possible: their
                               // sums are kept for put_far, 64 registers in all (8 rows: 122, 32 us for 26)
constexpr int kBytes = 16;     // of channels a thread

struct ConvArgs {
  const void *x, *w, *bias;
  const int *offsets, *slots;
  void *state, *out;
  int n, l, c, state_slots, silu, carry;
  long long x_sn, x_st, o_sn, o_st;
  int groups;       // channel vectors a row
  int tokens;       // rows of one thread's walk
  int tiles;        // walks a sequence (dense) or a call (packed)
};

// Threads are laid out over channel vectors (x) and walks or sequences (y), so that
// none has to divide: a row of blocks along x covers the channels.
__device__ __forceinline__ bool my_place(int groups, int* group, long long* item) {
  *group = blockIdx.x * blockDim.x + threadIdx.x;
  *item = ((long long)blockIdx.z * gridDim.y + blockIdx.y) * blockDim.y + threadIdx.y;
  return *group < groups;
}

// silu of the sums above kFar, and the outputs of the others.  fp16 has none that differ:
// it holds nothing below 2^-24, and silu_near gives -0 there.
template <typename T>
constexpr bool kHasFar = !std::is_same_v<T, __half>;
template <int V>
__device__ __forceinline__ void activate(float (&v)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 y = silu_near(make_float2(v[i], v[i + 1]));
      v[i] = y.x;
      v[i + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = silu_near(v[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void put_far(const float (&sums)[V], T* out) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (sums[i] < kFar) st_f32(out + i, silu_far(sums[i]));
}

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

// acc += w * x, two channels to a packed instruction.
template <int V>
__device__ __forceinline__ void multiply_add(const float (&w)[V], const float (&x)[V], float (&acc)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const float2 r = __ffma2_rn(make_float2(w[v], w[v + 1]), make_float2(x[v], x[v + 1]), make_float2(acc[v], acc[v + 1]));
      acc[v] = r.x;
      acc[v + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(w[v], x[v], acc[v]);
  }
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

  // The next sums from the window and the row after it, which the window takes up.
  __device__ __forceinline__ void step(float (&win)[K - 1][V], const float (&now)[V], float (&acc)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = b[v];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) multiply_add<V>(w[k], win[k], acc);
    multiply_add<V>(w[K - 1], now, acc);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) win[k][v] = k < K - 2 ? win[k < K - 2 ? k + 1 : k][v] : now[v];
  }

  // Positions [from, to) of the sequence whose rows start at x and out.
  __device__ __forceinline__ void run(const T* x, T* out, int from, int to, int slot) const {
    if (from >= to) return;
    float win[K - 1][V];
    const T* ahead = x + from * p.x_st;
    T* here = out + from * p.o_st;
    if constexpr (VEC) {
      float low = 0.0f;      // of the sums
      // kAhead rows of this thread's own 16 bytes are on their way into shared memory
      // while one is worked on.  Only the thread itself reads them, so its own copies
      // are all it waits for.
      extern __shared__ uint4 ring[];
      uint4* mine = ring + threadIdx.y * blockDim.x + threadIdx.x;
      const int step_of = blockDim.x * blockDim.y;
      auto fetch = [&](int row_in_ring, int count) {
        if (count > 0) copy_async<16>(mine + row_in_ring * step_of, ahead);
        ahead += p.x_st;
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int f = 0; f < kAhead; ++f) fetch(f, to - from - f);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) row(x, from - (K - 1) + j, slot, win[j]);
      for (int at = from, row_in_ring = 0; at < to; ++at) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        float now[V], acc[V];
        load_f32<T, V, true>(reinterpret_cast<const T*>(mine + row_in_ring * step_of), now);
        asm volatile("" ::: "memory");       // read before the next copy into the same place is issued
        fetch(row_in_ring, to - at - kAhead);
        row_in_ring = row_in_ring + 1 == kAhead ? 0 : row_in_ring + 1;
        step(win, now, acc);
        if (p.silu) {
          low = lowest<V>(acc, low);
          activate<V>(acc);
        }
        store_f32<T, V, true>(here, acc);
        here += p.o_st;
      }
      // a later walk of this thread reuses the ring: nothing may be on its way into it
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (kHasFar<T> && low < kFar) far(x, out, from, to, slot);
    } else {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) row(x, from - (K - 1) + j, slot, win[j]);
      T in[kLoose][V], next[kLoose][V];
      auto fetch = [&](T(&to_regs)[kLoose][V], int count) {
#pragma unroll
        for (int u = 0; u < kLoose; ++u) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (u < count) to_regs[u][v] = ahead[v];
          ahead += p.x_st;
        }
      };
      fetch(in, to - from);
      for (int at = from; at < to; at += kLoose) {
        fetch(next, to - at - kLoose);
        float sums[kLoose][V], low = 0.0f;
#pragma unroll
        for (int u = 0; u < kLoose; ++u) {
          float acc[V], now[V];
#pragma unroll
          for (int v = 0; v < V; ++v) now[v] = Store<T>::to_f32(in[u][v]);
          step(win, now, sums[u]);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] = sums[u][v];
          if (p.silu) {
            low = lowest<V>(acc, low);
            activate<V>(acc);
          }
          if (at + u < to) store_f32<T, V, false>(here, acc);
          here += p.o_st;
        }
        if (kHasFar<T> && low < kFar) {
#pragma unroll
          for (int u = 0; u < kLoose; ++u)
            if (at + u < to) put_far<T, V>(sums[u], here - (kLoose - u) * p.o_st);
        }
#pragma unroll
        for (int u = 0; u < kLoose; ++u)
#pragma unroll
          for (int v = 0; v < V; ++v) in[u][v] = next[u][v];
      }
    }
  }

  // Once more over the rows of a walk of which some have sums far out.  What they read
  // is as it was: the old window is replaced after the walk that reads it.  As little
  // code as it can be, for the sake of the walks that have none (5120 packed rows: 13.8 us
  // a call, 14.2 with the taps' loop unrolled).
  __device__ __forceinline__ void far(const T* x, T* out, int from, int to, int slot) const {
    const T* taps = static_cast<const T*>(p.w) + (long long)ch * K;
#pragma unroll 1
    for (int t = from; t < to; ++t) {
      float sums[V], v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sums[i] = b[i];
#pragma unroll 1
      for (int k = 0; k < K; ++k) {
        row(x, t - (K - 1) + k, slot, v);
#pragma unroll
        for (int i = 0; i < V; ++i) sums[i] = fmaf(ld_f32(taps + i * K + k), v[i], sums[i]);
      }
      put_far<T, V>(sums, out + t * p.o_st);
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
  int place;
  long long walk_id;
  if (!my_place(p.groups, &place, &walk_id)) return;
  const int ch = place * V;
  const T* x = static_cast<const T*>(p.x) + ch;
  T* out = static_cast<T*>(p.out) + ch;
  if (!p.offsets) {
    if (walk_id >= (long long)p.n * p.tiles) return;
    const int seq = (int)(walk_id < 0x7fffffff ? (unsigned)walk_id / (unsigned)p.tiles : walk_id / p.tiles);
    const int from = (int)(walk_id - (long long)seq * p.tiles) * p.tokens;
    const int slot = slot_of(p.slots, seq, p.state_slots);
    if (slot < 0) return;
    const Walk<T, K, V, VEC> walk(p, ch);
    x += seq * p.x_sn;
    walk.run(x, out + seq * p.o_sn, from, min(from + p.tokens, p.l), slot);
    if (p.state && from == 0) walk.keep(x, p.l, slot);
    return;
  }
  if (walk_id >= p.tiles) return;
  const int first = (int)walk_id * p.tokens;
  const bool last_walk = walk_id == p.tiles - 1;
  const int end = last_walk ? p.l : first + p.tokens;
  // The sequence that row `first` lies in, or the first one that starts there or
  // later: the first with an end above `first`, or that starts at or after it.
  // Halved down to 16 candidates; those are compared at once instead of one load
  // after another.
  auto reaches = [&](int seq) { return __ldg(p.offsets + seq + 1) > first || __ldg(p.offsets + seq) >= first; };
  int lo_seq = 0, hi_seq = p.n;
  while (hi_seq - lo_seq > 16) {
    const int mid = (lo_seq + hi_seq) >> 1;
    if (reaches(mid)) hi_seq = mid;
    else lo_seq = mid + 1;
  }
  int before = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) before += lo_seq + i < hi_seq && !reaches(lo_seq + i);
  lo_seq += before;
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
  int place;
  long long seq;
  if (!my_place(p.groups, &place, &seq) || seq >= p.n) return;
  const int ch = place * V;
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
  }
  T* out = static_cast<T*>(p.out) + seq * p.o_sn + ch;
  float sums[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sums[v] = acc[v];
  if (p.silu) activate<V>(acc);
  store_f32<T, V, VEC>(out, acc);
  if (kHasFar<T> && p.silu && lowest<V>(sums, 0.0f) < kFar) put_far<T, V>(sums, out);
#pragma unroll
  for (int k = 0; k < K - 1; ++k) store_f32<T, V, VEC>(state + (long long)k * p.c, win[k + 1]);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Launch over `groups` channel vectors x `items`, kept to whole rows of blocks with
// few idle threads; `bytes` of shared memory a thread.
template <typename Args>
cudaError_t launch(void (*kernel)(const Args), const Args& p, int groups, long long items, int bytes, cudaStream_t s) {
  const int gx = (groups + kThreads - 1) / kThreads, bx = (groups + gx - 1) / gx, by = kThreads / bx;
  const long long gy = (items + by - 1) / by, y = gy < 32768 ? gy : 32768, z = (gy + y - 1) / y;
  if (z > 65535) return cudaErrorInvalidConfiguration;
  kernel<<<dim3((unsigned)gx, (unsigned)y, (unsigned)z), dim3(bx, by), bx * by * bytes, s>>>(p);
  return cudaGetLastError();
}

// Threads below which walks are made shorter: a little under the 51200 of 5120 rows of
// 1280 fp16 channels in walks of 16, the fastest there.  No other sizes were swept.
constexpr long long kFullThreads = 148 * 324;

template <typename T, int K>
cudaError_t conv_typed(ConvArgs p, cudaStream_t s) {
  constexpr int V = kBytes / sizeof(T);
  const bool vec = on16(p.x) && on16(p.w) && on16(p.out) && on16(p.state) && on16(p.bias) && p.c % V == 0 && p.x_sn % V == 0 &&
                   p.x_st % V == 0 && p.o_sn % V == 0 && p.o_st % V == 0;
  p.groups = vec ? p.c / V : p.c;
  // Long walks read the taps and the rows before them less often (64 rows: 51 us for
  // 4 x 4096 rows of 4096 bf16 channels, 16 rows: 60 us); short ones give a small
  // call's threads to more SMs (5120 rows of 1280: 12.0 us with 16 rows, 19.9 with 64).
  long long walks = 0;
  for (p.tokens = 64;; p.tokens /= 2) {
    p.tiles = p.l > 0 ? (p.l - 1) / p.tokens + 1 : 1;   // without rows there are still windows to write
    walks = p.offsets ? p.tiles : (long long)p.n * p.tiles;
    if (p.tokens == 8 || walks * p.groups >= kFullThreads) break;
  }
  return vec ? launch(causal_conv_kernel<T, K, V, true>, p, p.groups, walks, kAhead * kBytes, s)
             : launch(causal_conv_kernel<T, K, 1, false>, p, p.groups, walks, 0, s);
}

template <typename T, int K>
cudaError_t step_typed(StepArgs p, cudaStream_t s) {
  constexpr int V = kBytes / sizeof(T);
  const bool vec = on16(p.x) && on16(p.w) && on16(p.out) && on16(p.state) && on16(p.bias) && p.c % V == 0 && p.x_sn % V == 0 &&
                   p.o_sn % V == 0;
  p.groups = vec ? p.c / V : p.c;
  return vec ? launch(causal_conv_step_kernel<T, K, V, true>, p, p.groups, p.n, 0, s)
             : launch(causal_conv_step_kernel<T, K, 1, false>, p, p.groups, p.n, 0, s);
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

// selective_scan.cu -- the selective state space recurrence over prompts, and
// for one new token of every sequence.
//
// For channel d of a sequence, S states s, group g = d / (D / G):
//
//   delta_t = dt_t[d] + dt_bias[d], then log(1 + exp(delta)) with softplus
//   h_t[s]  = exp(delta_t a[d][s]) h_{t-1}[s] + delta_t b_t[g][s] x_t[d]
//   out_t   = (sum_s c_t[g][s] h_t[s] + D[d] x_t[d]) silu(z_t[d])
//
// all in fp32 whatever the io type, out rounded once.
//
// Prompts are bound by the exponentials: one a (token, channel, state), 16 a
// clock and SM in the special-function units, where reading and writing a
// token's four io values costs a quarter of that.  kLanes lanes share a channel
// with kStates states each in registers; a block of 128 threads holds 128 / kLanes
// channels and walks the sequence in tiles of 64 tokens staged in shared
// memory, the next tile in flight by cp.async.  Per tile the delta and
// delta * x of each (token, channel) are computed once, spread over the channel's
// lanes, and the sums over states of kLanes (at least 8) tokens are reduced
// together, so that each lane ends with the sums of its own tokens.
//
// A call with too few channels to fill the device cuts the sequences into
// chunks: scan_chunk_kernel leaves each chunk's final state from zero and its
// sum of delta in the workspace, and every chunk of scan_kernel folds those
// before it into its first state (the decay over a chunk is exp(a sum delta)).
// That doubles the exponentials, so it needs more than two chunks to pay.
#include <cuda_runtime.h>

#include "sequence.cuh"

namespace b200conv {
namespace {

constexpr int kThreads = 128;

struct ScanArgs {
  const void *x, *dt, *b, *c, *z;
  const float *a, *d, *dt_bias;
  const int *offsets, *slots;
  float* state;
  void* out;
  float *ws_state, *ws_sum;    // chunked: [n][chunks][D][S] states (0: the first, j + 1: after chunk j from zero), [n][chunks][D] sums
  int n, l, channels, states, groups, state_slots, softplus, carry;
  long long x_s[2], dt_s[2], z_s[2], b_s[2], c_s[2], out_s[2];
  int chunk, chunks;           // tokens a chunk (a multiple of 64), chunks a sequence
  int tiles;                   // channel tiles a group
  int x_v, dt_v, z_v, b_v, c_v, out_v;   // bytes an access: 16, 8, 4, or 0 for single elements
};

// Copies tiles of kRows x cols elements (cols <= kCols) of a tensor's consecutive
// rows into shared rows kPitch elements apart, by all threads.  `bytes`: an access
// (16, 8, 4, or 0 for single elements), cols and every address multiples of it.
// The 16-byte form keeps each thread's address from tile to tile: worked out anew,
// the five tensors' addresses took as long as a third of the recursion itself.
template <typename T, int kRows, int kCols, int kPitch>
struct Stager {
  static constexpr int E = 16 / sizeof(T), kPer = kCols / E > 0 ? kCols / E : 1;
  static constexpr int kStep = kThreads / kPer > 0 ? kThreads / kPer : 1;     // rows between a thread's accesses
  static constexpr bool kFits = kCols % E == 0 && kPer <= kThreads && kRows % kStep == 0;
  const T* src;
  long long stride;
  int cols, bytes, r0, to;
  __device__ __forceinline__ void init(const T* base, long long row_stride, int width, int access) {
    src = base;
    stride = row_stride;
    cols = width;
    bytes = access;
    r0 = threadIdx.x / kPer;
    const int q = (threadIdx.x % kPer) * E;
    to = r0 * kPitch + q;
    if (kFits && bytes == 16) {
      src += r0 * stride + q;
      if (q >= cols) r0 = kRows;        // past the edge: never a row
    }
  }
  template <int N>
  __device__ __forceinline__ void by(T* dst, int rows) {
    constexpr int kE = N / sizeof(T) > 0 ? N / sizeof(T) : 1, kAcross = kCols / kE > 0 ? kCols / kE : 1;
    for (int i = threadIdx.x; i < rows * kAcross; i += kThreads) {
      const int r = i / kAcross, q = (i % kAcross) * kE;
      if (q < cols) copy_async<N>(dst + r * kPitch + q, src + r * stride + q);
    }
  }
  // The next `rows` rows.
  __device__ __forceinline__ void next(T* dst, int rows) {
    if (kFits && bytes == 16) {
#pragma unroll
      for (int r = 0; r < kRows; r += kStep)
        if (r0 + r < rows) copy_async<16>(dst + to + r * kPitch, src + r * stride);
    } else if (bytes == 16) {
      by<16>(dst, rows);
    } else if (bytes == 8) {
      by<8>(dst, rows);
    } else if (bytes == 4) {
      by<4>(dst, rows);
    } else {
#pragma unroll 8
      for (int i = threadIdx.x; i < rows * kCols; i += kThreads) {
        const int r = i / kCols, q = i % kCols;
        if (q < cols) dst[r * kPitch + q] = src[r * stride + q];
      }
    }
    src += kRows * stride;
  }
};

template <typename T, int kStates, int kLanes>
struct Shape {
  static constexpr int kChannels = kThreads / kLanes;
  static constexpr int kWide = kStates * kLanes;             // states, padded
  static constexpr int kTile = kWide <= 32 ? 64 : 32;        // tokens staged together
  static constexpr int kTogether = kLanes > 8 ? kLanes : 8;  // tokens reduced together
  static constexpr int kOwn = kTogether / kLanes;            // of which each lane ends with
  static constexpr int kSub = kStates > 4 ? 4 : 8;           // tokens whose exponentials are in flight
  static constexpr int kMany = 32 / kTogether;               // groups in a row
  static constexpr int kRow = kTile + 8;                     // floats a channel of delta
  static constexpr int kPitch = kChannels + 16 / sizeof(T);  // elements a row of x: 16 bytes more, against bank conflicts
  // shared memory, in bytes
  static constexpr int kRawX = kTile * kPitch * sizeof(T);
  static constexpr int kRawB = kTile * kWide * sizeof(T);
  static constexpr int kStage = 3 * kRawX + 2 * kRawB;
  static constexpr int kOut = 2 * kStage;
  static constexpr int kDelta = kOut + kRawX;
  static constexpr int kB = kDelta + 2 * kChannels * kRow * 4;
  static constexpr int kBytes = kB + 2 * kTile * kWide * 4;
  static_assert(kTile % kTogether == 0 && (kStates == 1 || kStates % 2 == 0), "");
};

// Sequence, channel tile and tokens of a block.
struct Where {
  int seq, group, ch, count;   // first channel, channels
  int lo, len;                 // packed: first row; tokens of the sequence
  int slot;
};
template <int kChannels>
__device__ __forceinline__ bool locate(const ScanArgs& p, Where* w) {
  const int per_seq = p.tiles * p.groups;
  w->seq = blockIdx.x / per_seq;
  const int t = blockIdx.x - w->seq * per_seq;
  w->group = t / p.tiles;
  const int per_group = p.channels / p.groups, at = (t - w->group * p.tiles) * kChannels;
  w->ch = w->group * per_group + at;
  w->count = min(kChannels, per_group - at);
  w->slot = slot_of(p.slots, w->seq, p.state_slots);
  w->lo = 0;
  w->len = p.l;
  if (p.offsets) {
    int hi;
    packed_range(p.offsets, w->seq, p.l, &w->lo, &hi);
    w->len = hi - w->lo;
  }
  return w->slot >= 0;
}

template <typename T>
__device__ __forceinline__ const T* rows_of(const ScanArgs& p, const void* base, const long long (&s)[2], const Where& w,
                                            int col) {
  return static_cast<const T*>(base) + (p.offsets ? 0 : w.seq * s[0]) + w.lo * s[1] + col;
}

// The values of two tokens for each of kStates neighbouring states.
template <int kStates>
__device__ __forceinline__ void load_pairs(const float* p, float2 (&v)[kStates]) {
  if constexpr (kStates == 1) {
    v[0] = *reinterpret_cast<const float2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < kStates; i += 2) {
      const float4 two = *reinterpret_cast<const float4*>(p + 2 * i);
      v[i] = make_float2(two.x, two.y);
      v[i + 1] = make_float2(two.z, two.w);
    }
  }
}

// The sums over a channel's lanes of kCount tokens' y: at each step a lane passes on
// one half of its tokens and adds its partner's share of the other, so that lane l
// ends with tokens l * kOwn .. of the group in y[0 .. kOwn - 1].
// With fewer tokens than lanes the last steps add the same token's shares.
template <int kOff, int kCount, int kAll>
__device__ __forceinline__ void reduce_lanes(float (&y)[kAll], int lane) {
  if constexpr (kOff > 0 && kCount == 1) {
    y[0] += __shfl_xor_sync(0xffffffffu, y[0], kOff);
    reduce_lanes<kOff / 2, 1>(y, lane);
  } else if constexpr (kOff > 0) {
    const bool upper = lane & kOff;
#pragma unroll
    for (int i = 0; i < kCount / 2; ++i) {
      const float give = upper ? y[i] : y[i + kCount / 2];
      const float take = upper ? y[i + kCount / 2] : y[i];
      y[i] = take + __shfl_xor_sync(0xffffffffu, give, kOff);
    }
    reduce_lanes<kOff / 2, kCount / 2>(y, lane);
  }
}

// kFull: states == kStates * kLanes.  kEnds: the chunk's final state from zero and its sum of delta, no output.
template <typename T, int kStates, int kLanes, bool kFull, bool kEnds>
__global__ void __launch_bounds__(kThreads) scan_kernel(const ScanArgs p) {
  using L = Shape<T, kStates, kLanes>;
  extern __shared__ __align__(16) unsigned char smem[];
  Where w;
  if (!locate<L::kChannels>(p, &w)) return;
  const int chunk = blockIdx.y, begin = chunk * p.chunk;
  const bool last = begin + p.chunk >= w.len;
  // a chunk without tokens has nothing to do, but for the first one's state of an empty sequence
  if (begin >= w.len && chunk > 0) return;
  const int end = last ? w.len : begin + p.chunk;
  const int lane = threadIdx.x % kLanes, cl = threadIdx.x / kLanes;
  const bool live = cl < w.count;
  const int ch = w.ch + (live ? cl : 0);
  const int s0 = lane * kStates, have = kFull ? kStates : min(max(p.states - s0, 0), kStates);

  float2 a2[kStates];          // a log2(e), twice
  float h[kStates];
  const float* a = p.a + (long long)ch * p.states + s0;
  float* cache = p.state ? p.state + ((long long)w.slot * p.channels + ch) * p.states + s0 : nullptr;
  const long long ws_row = ((long long)w.seq * p.chunks * p.channels + ch) * p.states + s0;
  const long long ws_step = (long long)p.channels * p.states;
#pragma unroll
  for (int i = 0; i < kStates; ++i) {
    const float v = i < have ? __ldg(a + i) * kLog2e : 0.0f;
    a2[i] = make_float2(v, v);
    h[i] = 0.0f;
  }
  if constexpr (kEnds) {
    if (last) return;            // nothing follows it
    if (chunk == 0 && live) {
#pragma unroll
      for (int i = 0; i < kStates; ++i)
        if (i < have) p.ws_state[ws_row + i] = p.carry ? cache[i] : 0.0f;
    }
  } else if (p.chunks > 1 && !(chunk == 0 && last)) {
#pragma unroll
    for (int i = 0; i < kStates; ++i)
      if (i < have) h[i] = p.ws_state[ws_row + i];
    for (int j = 0; j < chunk; ++j) {
      const float sum = p.ws_sum[((long long)w.seq * p.chunks + j) * p.channels + ch];
#pragma unroll
      for (int i = 0; i < kStates; ++i)
        if (i < have) h[i] = fmaf(decay(a2[i].x, sum), h[i], p.ws_state[ws_row + (j + 1) * ws_step + i]);
    }
  } else if (p.carry) {
#pragma unroll
    for (int i = 0; i < kStates; ++i)
      if (i < have) h[i] = cache[i];
  }

  const T* x = rows_of<T>(p, p.x, p.x_s, w, w.ch);
  const T* dt = rows_of<T>(p, p.dt, p.dt_s, w, w.ch);
  const T* z = p.z && !kEnds ? rows_of<T>(p, p.z, p.z_s, w, w.ch) : nullptr;
  const T* b = rows_of<T>(p, p.b, p.b_s, w, w.group * p.states);
  const T* c = rows_of<T>(p, p.c, p.c_s, w, w.group * p.states);
  T* out = kEnds ? nullptr : const_cast<T*>(rows_of<T>(p, p.out, p.out_s, w, w.ch));
  const float bias = p.dt_bias ? __ldg(p.dt_bias + ch) : 0.0f;
  const float skip = !kEnds && p.d ? __ldg(p.d + ch) : 0.0f;

  auto raw = [&](int stage, int which) {
    return reinterpret_cast<T*>(smem + stage * L::kStage + (which < 3 ? which * L::kRawX : 3 * L::kRawX + (which - 3) * L::kRawB));
  };
  T* out_tile = reinterpret_cast<T*>(smem + L::kOut);
  float* delta_of = reinterpret_cast<float*>(smem + L::kDelta) + cl * L::kRow;
  float* dx_of = delta_of + L::kChannels * L::kRow;
  // b and c in fp32, the two tokens of a pair side by side: [token / 2][state][token % 2]
  float* bf = reinterpret_cast<float*>(smem + L::kB);
  float* cf = bf + L::kTile * L::kWide;

  Stager<T, L::kTile, L::kChannels, L::kPitch> sx, sdt, sz;
  Stager<T, L::kTile, L::kWide, L::kWide> sb, sc;
  sx.init(x + begin * p.x_s[1], p.x_s[1], w.count, p.x_v);
  sdt.init(dt + begin * p.dt_s[1], p.dt_s[1], w.count, p.dt_v);
  sb.init(b + begin * p.b_s[1], p.b_s[1], p.states, p.b_v);
  if (z) sz.init(z + begin * p.z_s[1], p.z_s[1], w.count, p.z_v);
  if (!kEnds) sc.init(c + begin * p.c_s[1], p.c_s[1], p.states, p.c_v);
  auto fetch = [&](int at, int to) {
    const int rows = min(L::kTile, end - at);
    sx.next(raw(to, 0), rows);
    sdt.next(raw(to, 1), rows);
    if (z) sz.next(raw(to, 2), rows);
    sb.next(raw(to, 3), rows);
    if (!kEnds) sc.next(raw(to, 4), rows);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto put = [&](int at) {           // out_tile's rows, from token `at`
    const int rows = min(L::kTile, end - at);
    T* to = out + at * p.out_s[1];
    constexpr int E = 16 / sizeof(T), kPer = L::kChannels / E;
    if (kPer > 0 && p.out_v == 16) {
      for (int i = threadIdx.x; i < rows * kPer; i += kThreads) {
        const int r = i / (kPer > 0 ? kPer : 1), q = (i % (kPer > 0 ? kPer : 1)) * E;
        if (q < w.count)
          *reinterpret_cast<uint4*>(to + r * p.out_s[1] + q) = *reinterpret_cast<const uint4*>(out_tile + r * L::kPitch + q);
      }
    } else {
      for (int i = threadIdx.x; i < rows * L::kChannels; i += kThreads) {
        const int r = i / L::kChannels, q = i % L::kChannels;
        if (q < w.count) to[r * p.out_s[1] + q] = out_tile[r * L::kPitch + q];
      }
    }
  };

  float sum = 0.0f;            // of delta, over this lane's tokens
  if (begin < end) fetch(begin, 0);
  for (int at = begin, turn = 0; at < end; at += L::kTile, turn ^= 1) {
    const int rows = min(L::kTile, end - at);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (!kEnds && at > begin) put(at - L::kTile);
    if (at + L::kTile < end) fetch(at + L::kTile, turn ^ 1);

    const T *xr = raw(turn, 0), *dr = raw(turn, 1), *zr = raw(turn, 2), *br = raw(turn, 3), *cr = raw(turn, 4);
    // Each pass loads all its values before it stores any: a store in between would
    // hold back the loads after it, which the compiler cannot tell apart from it.
    constexpr int kTurns = L::kTile / kLanes, kBatch = kTurns > 8 ? 8 : kTurns;
#pragma unroll 1
    for (int t0 = lane; t0 < rows; t0 += kBatch * kLanes) {
      float de[kBatch], xv[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        de[i] = ld_f32(dr + (t0 + i * kLanes) * L::kPitch + cl) + bias;
        xv[i] = ld_f32(xr + (t0 + i * kLanes) * L::kPitch + cl);
      }
      if (p.softplus) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) de[i] = softplus(de[i]);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        delta_of[t0 + i * kLanes] = de[i];
        dx_of[t0 + i * kLanes] = de[i] * xv[i];
        if (kEnds && t0 + i * kLanes < rows) sum += de[i];
      }
    }
    constexpr int kPairs = L::kTile / 2 * L::kWide, kPairTurns = (kPairs + kThreads - 1) / kThreads,
                  kPairBatch = kPairTurns > 4 ? 4 : kPairTurns;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < kPairs && i0 / L::kWide * 2 < rows; i0 += kPairBatch * kThreads) {
      float2 b2[kPairBatch], c2[kPairBatch];
#pragma unroll
      for (int k = 0; k < kPairBatch; ++k) {
        const int i = i0 + k * kThreads, s = i % L::kWide, t = i / L::kWide * 2;
        b2[k] = c2[k] = make_float2(0.0f, 0.0f);
        if ((kPairs % (kPairBatch * kThreads) == 0 || i < kPairs) && (kFull || s < p.states)) {
          const T *b0 = br + t * L::kWide + s, *c0 = cr + t * L::kWide + s;
          b2[k] = make_float2(ld_f32(b0), ld_f32(b0 + L::kWide));
          if (!kEnds) c2[k] = make_float2(ld_f32(c0), ld_f32(c0 + L::kWide));
        }
      }
#pragma unroll
      for (int k = 0; k < kPairBatch; ++k) {
        const int i = i0 + k * kThreads;
        if (kPairs % (kPairBatch * kThreads) == 0 || i < kPairs) {
          reinterpret_cast<float2*>(bf)[i] = b2[k];
          if (!kEnds) reinterpret_cast<float2*>(cf)[i] = c2[k];
        }
      }
    }
    __syncthreads();

    // kSub tokens from t: the states advance, and y gets this lane's share of the sums
    // over them.  The exponentials and additions of all tokens come first, two tokens
    // to a packed instruction; only the h chain itself is sequential.  kTail: tokens
    // from `rows` on leave the states alone.
    auto sub = [&](auto tail, int t, float* y) {
      constexpr bool kTail = decltype(tail)::value;
      constexpr int kSub = L::kSub;
      float2 e[kSub / 2][kStates], add[kSub / 2][kStates];
#pragma unroll
      for (int q = 0; q < kSub; q += 4) {
        const float4 de = *reinterpret_cast<const float4*>(delta_of + t + q);
        const float4 dx = *reinterpret_cast<const float4*>(dx_of + t + q);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 d2 = k ? make_float2(de.z, de.w) : make_float2(de.x, de.y);
          const float2 x2 = k ? make_float2(dx.z, dx.w) : make_float2(dx.x, dx.y);
#pragma unroll
          for (int i = 0; i < kStates; ++i) {
            const float2 arg = __ffma2_rn(d2, a2[i], make_float2(kEx2Bias, kEx2Bias));
            e[q / 2 + k][i] = make_float2(ex2(arg.x), ex2(arg.y));
          }
          load_pairs<kStates>(bf + (t + q + 2 * k) * L::kWide + s0 * 2, add[q / 2 + k]);
#pragma unroll
          for (int i = 0; i < kStates; ++i) add[q / 2 + k][i] = __fmul2_rn(x2, add[q / 2 + k][i]);
        }
      }
#pragma unroll
      for (int q = 0; q < kSub / 2; ++q) {
        float2 sum2 = make_float2(0.0f, 0.0f);
        float2 ct[kStates];
        if (!kEnds) load_pairs<kStates>(cf + (t + 2 * q) * L::kWide + s0 * 2, ct);
#pragma unroll
        for (int i = 0; i < kStates; ++i) {
          float h0 = fmaf(e[q][i].x, h[i], add[q][i].x);
          if (!kFull && i >= have) h0 = 0.0f;
          if (kTail && t + 2 * q >= rows) h0 = h[i];
          float h1 = fmaf(e[q][i].y, h0, add[q][i].y);
          if (!kFull && i >= have) h1 = 0.0f;
          if (kTail && t + 2 * q + 1 >= rows) h1 = h0;
          h[i] = h1;
          if (!kEnds) sum2 = __ffma2_rn(ct[i], make_float2(h0, h1), sum2);
        }
        y[2 * q] = sum2.x;
        y[2 * q + 1] = sum2.y;
      }
    };
    auto group = [&](auto tail, int t, float* own) {
      float y[L::kTogether];
#pragma unroll
      for (int q = 0; q < L::kTogether; q += L::kSub) sub(tail, t + q, y + q);
      if constexpr (!kEnds) {
        reduce_lanes<kLanes / 2, L::kTogether>(y, lane);
#pragma unroll
        for (int i = 0; i < L::kOwn; ++i) own[i] = y[i];
      }
    };
    // kMany groups before the outputs of any
    auto groups = [&](auto tail, auto many, int t) {
      constexpr int kMany = decltype(many)::value, kAll = kMany * L::kOwn;
      float own[kAll], xv[kAll], zv[kAll];
#pragma unroll
      for (int g = 0; g < kMany; ++g) group(tail, t + g * L::kTogether, own + g * L::kOwn);
      if constexpr (!kEnds) {
#pragma unroll
        for (int g = 0; g < kAll; ++g) {
          const int at_t = t + g / L::kOwn * L::kTogether + lane * L::kOwn + g % L::kOwn;
          xv[g] = ld_f32(xr + at_t * L::kPitch + cl);
          zv[g] = z ? ld_f32(zr + at_t * L::kPitch + cl) : 0.0f;
        }
        if (p.d) {
#pragma unroll
          for (int g = 0; g < kAll; ++g) own[g] = fmaf(skip, xv[g], own[g]);
        }
        if (z) {
#pragma unroll
          for (int g = 0; g < kAll; ++g) own[g] *= silu(zv[g]);
        }
#pragma unroll
        for (int g = 0; g < kAll; ++g)
          st_f32(out_tile + (t + g / L::kOwn * L::kTogether + lane * L::kOwn + g % L::kOwn) * L::kPitch + cl, own[g]);
      }
    };
    int t = 0;
    for (; t + L::kMany * L::kTogether <= rows; t += L::kMany * L::kTogether)
      groups(std::false_type{}, std::integral_constant<int, L::kMany>{}, t);
    for (; t < rows; t += L::kTogether) groups(std::true_type{}, std::integral_constant<int, 1>{}, t);
  }
  if (!kEnds && begin < end) {
    __syncthreads();
    put(begin + (end - 1 - begin) / L::kTile * L::kTile);
  }

  if constexpr (kEnds) {
#pragma unroll
    for (int off = 1; off < kLanes; off *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < kStates; ++i)
      if (i < have) p.ws_state[ws_row + (chunk + 1) * ws_step + i] = h[i];
    if (lane == 0) p.ws_sum[((long long)w.seq * p.chunks + chunk) * p.channels + ch] = sum;
  } else if (last && live && cache) {
#pragma unroll
    for (int i = 0; i < kStates; ++i)
      if (i < have) cache[i] = h[i];
  }
}

// ------------------------------ single tokens ----------------------------------

struct StepArgs {
  const void *x, *dt, *b, *c, *z;
  const float *a, *d, *dt_bias;
  const int* slots;
  float* state;
  void* out;
  int n, channels, states, groups, state_slots, softplus;
  long long x_s, dt_s, z_s, b_s, c_s, out_s;
  int bc_vec;                  // b and c in accesses of four states
};

// Bound by the states, 8 bytes a state moved.  A block works on one sequence.  kLanes
// lanes share a channel, four neighbouring states a lane and turn (one 16-byte
// access with VEC), and go through kMine channels together: b and c are loaded and
// converted once for them, each lane prepares and finishes one channel's token
// (delta and the gate), and that many loads are in flight.  One channel at a time
// took 260 instructions for four states, mostly addresses and the softplus.
template <typename T, int kLanes, int kMine, bool VEC>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const StepArgs p) {
  constexpr int kAcross = 32 / kLanes, kSub = kLanes / kMine;   // channels side by side; lanes that hold one channel's token
  const int seq = blockIdx.z * gridDim.y + blockIdx.y;
  if (seq >= p.n) return;
  const int slot = slot_of(p.slots, seq, p.state_slots);
  if (slot < 0) return;
  const int lane = threadIdx.x % kLanes;
  const int first = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kAcross * kMine + threadIdx.x % 32 / kLanes;
  const int mine = first + lane / kSub * kAcross;
  float xv = 0.0f, delta = 0.0f, skip = 0.0f, gate = 1.0f;
  if (mine < p.channels) {
    xv = ld_f32(static_cast<const T*>(p.x) + seq * p.x_s + mine);
    delta = ld_f32(static_cast<const T*>(p.dt) + seq * p.dt_s + mine);
    if (p.z) gate = ld_f32(static_cast<const T*>(p.z) + seq * p.z_s + mine);
    if (p.dt_bias) delta += __ldg(p.dt_bias + mine);
    if (p.d) skip = __ldg(p.d + mine);
  }
  // with several channels a turn they are all of one group
  const int group = p.groups > 1 ? min(first, p.channels - 1) / (p.channels / p.groups) : 0;
  const T* b = static_cast<const T*>(p.b) + seq * p.b_s + group * p.states;
  const T* c = static_cast<const T*>(p.c) + seq * p.c_s + group * p.states;
  float* state = p.state + (long long)slot * p.channels * p.states;
  float de2[kMine], dx[kMine], y[kMine];
#pragma unroll
  for (int q = 0; q < kMine; ++q) y[q] = 0.0f;
  bool ready = false;
  for (int s = lane * 4; s < (p.states + 3) / 4 * 4 || !ready; s += kLanes * 4) {
    const int have = min(max(p.states - s, 0), 4);
    float av[kMine][4], h[kMine][4], bv[4], cv[4];
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int ch = min(first + q * kAcross, p.channels - 1);
      const float *hp = state + (long long)ch * p.states + s, *ap = p.a + (long long)ch * p.states + s;
      if (VEC && have == 4) {
        load_f32<float, 4, true>(hp, h[q]);
        load_f32<float, 4, true>(ap, av[q]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[q][i] = i < have ? hp[i] : 0.0f;
          av[q][i] = i < have ? __ldg(ap + i) : 0.0f;
        }
      }
    }
    if (p.bc_vec && have == 4) {
      load_f32<T, 4, true>(b + s, bv);
      load_f32<T, 4, true>(c + s, cv);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bv[i] = i < have ? ld_f32(b + s + i) : 0.0f;
        cv[i] = i < have ? ld_f32(c + s + i) : 0.0f;
      }
    }
    if (!ready) {                 // behind the loads' issue: they do not wait for it
      ready = true;
      if (p.softplus) delta = softplus(delta);
      const float mine_de2 = delta * kLog2e, mine_dx = delta * xv;
#pragma unroll
      for (int q = 0; q < kMine; ++q) {
        de2[q] = __shfl_sync(0xffffffffu, mine_de2, q * kSub, kLanes);
        dx[q] = __shfl_sync(0xffffffffu, mine_dx, q * kSub, kLanes);
      }
    }
    if (have == 0) continue;      // nothing of a lane past the states enters the sums, not even 0 * inf
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!VEC && i >= have) break;
        h[q][i] = fmaf(decay(av[q][i], de2[q]), h[q][i], dx[q] * bv[i]);
        y[q] = fmaf(cv[i], h[q][i], y[q]);
      }
      if (first + q * kAcross < p.channels) {
        float* hp = state + (long long)(first + q * kAcross) * p.states + s;
        if (VEC && have == 4) {
          store_f32<float, 4, true>(hp, h[q]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < have) hp[i] = h[q][i];
        }
      }
    }
  }
  reduce_lanes<kLanes / 2, kMine>(y, lane);
  if (lane % kSub == 0 && mine < p.channels) {
    float v = y[0];
    if (p.d) v = fmaf(skip, xv, v);
    if (p.z) v *= silu(gate);
    st_f32(static_cast<T*>(p.out) + seq * p.out_s + mine, v);
  }
}

// -------------------------------- launches -------------------------------------

// The widest access that a tensor's rows allow: base, row stride, tile width and
// row width all multiples of it.  Copies into shared memory go down to 4 bytes.
int access_bytes(const void* p, const long long* stride, long long cols_a, long long cols_b, int esz) {
  for (int v = 16; v >= 4; v /= 2) {
    if (reinterpret_cast<uintptr_t>(p) % v == 0 && stride[0] * esz % v == 0 && stride[1] * esz % v == 0 &&
        cols_a * esz % v == 0 && cols_b * esz % v == 0)
      return v;
  }
  return 0;
}

template <typename T, int kStates, int kLanes, bool kFull>
cudaError_t scan_shaped(ScanArgs p, cudaStream_t s) {
  using L = Shape<T, kStates, kLanes>;
  const int per_group = p.channels / p.groups, esz = sizeof(T);
  p.tiles = (per_group + L::kChannels - 1) / L::kChannels;
  const long long part = L::kChannels;
  p.x_v = access_bytes(p.x, p.x_s, per_group, part, esz);
  p.dt_v = access_bytes(p.dt, p.dt_s, per_group, part, esz);
  p.z_v = access_bytes(p.z, p.z_s, per_group, part, esz);
  p.b_v = access_bytes(p.b, p.b_s, p.states, p.states, esz);
  p.c_v = access_bytes(p.c, p.c_s, p.states, p.states, esz);
  p.out_v = access_bytes(p.out, p.out_s, per_group, part, esz);
  const long long blocks = (long long)p.n * p.groups * p.tiles;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)p.chunks);
  auto run = [&](auto kernel) {
    if (L::kBytes > 48 * 1024) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
      if (e != cudaSuccess) return e;
    }
    kernel<<<grid, kThreads, L::kBytes, s>>>(p);
    return cudaGetLastError();
  };
  if (p.chunks > 1) {
    cudaError_t e = run(scan_kernel<T, kStates, kLanes, kFull, true>);
    if (e != cudaSuccess) return e;
  }
  return run(scan_kernel<T, kStates, kLanes, kFull, false>);
}

template <typename T>
cudaError_t scan_typed(const ScanArgs& p, const ScanPlan& plan, cudaStream_t s) {
#define B200CONV_SCAN(S, L, F) \
  if (plan.states_per_lane == S && plan.lanes == L && (!F || p.states == S * L)) return scan_shaped<T, S, L, F>(p, s)
  B200CONV_SCAN(2, 8, true);
  B200CONV_SCAN(4, 2, false);
  B200CONV_SCAN(4, 4, false);
  B200CONV_SCAN(4, 8, false);
  B200CONV_SCAN(4, 16, false);
  B200CONV_SCAN(4, 32, false);
  B200CONV_SCAN(8, 32, false);
#undef B200CONV_SCAN
  return cudaErrorInvalidValue;
}

constexpr int kStepMine = 4;
constexpr long long kManySteps = 148 * 2 * kThreads;   // threads

template <typename T>
cudaError_t step_typed(StepArgs p, cudaStream_t s) {
  const bool vec = ((reinterpret_cast<uintptr_t>(p.state) | reinterpret_cast<uintptr_t>(p.a)) & 15) == 0 && p.states % 4 == 0;
  p.bc_vec = ((reinterpret_cast<uintptr_t>(p.b) | reinterpret_cast<uintptr_t>(p.c)) & (4 * sizeof(T) - 1)) == 0 &&
             p.b_s % 4 == 0 && p.c_s % 4 == 0 && p.states % 4 == 0;
  int lanes = 1;
  while (lanes * 4 < p.states && lanes < 32) lanes *= 2;
  // Several channels a turn where that still leaves every SM a few blocks, and where a
  // warp's channels share b and c.
  int mine = lanes < kStepMine ? lanes : kStepMine;
  const int together = 32 / lanes * mine;
  if ((long long)p.n * p.channels * lanes / mine < kManySteps || (p.groups > 1 && p.channels / p.groups % together != 0)) mine = 1;
  const int across = kThreads / lanes * mine, y = p.n < 32768 ? p.n : 32768;
  const dim3 grid((p.channels + across - 1) / across, y, (unsigned)((p.n + y - 1LL) / y));
  if (grid.z > 65535) return cudaErrorInvalidConfiguration;
  auto with = [&](auto l) {
    auto run = [&](auto kernel) {
      kernel<<<grid, kThreads, 0, s>>>(p);
      return cudaGetLastError();
    };
    constexpr int kMine = l() < kStepMine ? l() : kStepMine;
    if (mine > 1) return vec ? run(scan_step_kernel<T, l(), kMine, true>) : run(scan_step_kernel<T, l(), kMine, false>);
    return vec ? run(scan_step_kernel<T, l(), 1, true>) : run(scan_step_kernel<T, l(), 1, false>);
  };
  switch (lanes) {
    case 1: return with(std::integral_constant<int, 1>{});
    case 2: return with(std::integral_constant<int, 2>{});
    case 4: return with(std::integral_constant<int, 4>{});
    case 8: return with(std::integral_constant<int, 8>{});
    case 16: return with(std::integral_constant<int, 16>{});
    default: return with(std::integral_constant<int, 32>{});
  }
}

}  // namespace

constexpr int kChunkStep = 64;   // chunks are whole tiles

// Pure in the descriptor and the device's SM count.
ScanPlan plan_scan(const selective_scan_desc_t& d, int sm_count) {
  ScanPlan plan{};
  plan.states_per_lane = 4;
  plan.lanes = 2;
  while (plan.lanes * plan.states_per_lane < d.s) {
    if (plan.lanes < 32) plan.lanes *= 2;
    else plan.states_per_lane *= 2;
  }
  if (d.s == 16) {
    plan.states_per_lane = 2;
    plan.lanes = 8;
  }
  const int channels = kThreads / plan.lanes;
  const long long per_group = d.d / d.groups;
  const long long blocks = (long long)d.n * d.groups * ((per_group + channels - 1) / channels);
  plan.chunk = d.l > 0 ? (d.l + kChunkStep - 1) / kChunkStep * kChunkStep : kChunkStep;
  plan.chunks = 1;
  // With chunks every token is gone over twice, so three are the fewest that can pay.
  const long long want = blocks > 0 ? 4LL * sm_count / blocks : 0, most = (d.l + 2LL * kChunkStep - 1) / (2 * kChunkStep);
  const long long chunks = want < most ? want : most;
  if (chunks >= 4) {
    plan.chunk = (int)(((d.l + chunks - 1) / chunks + kChunkStep - 1) / kChunkStep * kChunkStep);
    plan.chunks = (d.l + plan.chunk - 1) / plan.chunk;
  }
  if (plan.chunks > 1) {
    const size_t rows = (size_t)d.n * plan.chunks * d.d;
    plan.sum_offset = (rows * d.s * sizeof(float) + 255) & ~size_t(255);
    plan.workspace_bytes = plan.sum_offset + ((rows * sizeof(float) + 255) & ~size_t(255));
  }
  return plan;
}

cudaError_t launch_selective_scan(const selective_scan_desc_t& d, conv_dtype_t dt, const selective_scan_tensors_t& t,
                                  const ScanPlan& plan, void* workspace, cudaStream_t s) {
  ScanArgs p{};
  p.x = t.x; p.dt = t.dt; p.b = t.b; p.c = t.c; p.z = t.z; p.a = t.a; p.d = t.d; p.dt_bias = t.dt_bias;
  p.offsets = t.offsets; p.slots = t.slots; p.state = t.state; p.out = t.out;
  p.n = d.n; p.l = d.l; p.channels = d.d; p.states = d.s; p.groups = d.groups; p.state_slots = d.state_slots;
  p.softplus = d.softplus; p.carry = d.carry && t.state;
  for (int i = 0; i < 2; ++i) {
    p.x_s[i] = d.x_stride[i]; p.dt_s[i] = d.dt_stride[i]; p.z_s[i] = d.z_stride[i];
    p.b_s[i] = d.b_stride[i]; p.c_s[i] = d.c_stride[i]; p.out_s[i] = d.out_stride[i];
  }
  p.chunk = plan.chunk; p.chunks = plan.chunks;
  p.ws_state = static_cast<float*>(workspace);
  p.ws_sum = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + plan.sum_offset);
  switch (dt) {
    case CONV_F16: return scan_typed<__half>(p, plan, s);
    case CONV_BF16: return scan_typed<__nv_bfloat16>(p, plan, s);
    default: return scan_typed<float>(p, plan, s);
  }
}

cudaError_t launch_selective_scan_step(const selective_scan_desc_t& d, conv_dtype_t dt, const selective_scan_tensors_t& t,
                                       cudaStream_t s) {
  StepArgs p{};
  p.x = t.x; p.dt = t.dt; p.b = t.b; p.c = t.c; p.z = t.z; p.a = t.a; p.d = t.d; p.dt_bias = t.dt_bias;
  p.slots = t.slots; p.state = t.state; p.out = t.out;
  p.n = d.n; p.channels = d.d; p.states = d.s; p.groups = d.groups; p.state_slots = d.state_slots; p.softplus = d.softplus;
  p.x_s = d.x_stride[0]; p.dt_s = d.dt_stride[0]; p.z_s = d.z_stride[0];
  p.b_s = d.b_stride[0]; p.c_s = d.c_stride[0]; p.out_s = d.out_stride[0];
  switch (dt) {
    case CONV_F16: return step_typed<__half>(p, s);
    case CONV_BF16: return step_typed<__nv_bfloat16>(p, s);
    default: return step_typed<float>(p, s);
  }
}

}  // namespace b200conv

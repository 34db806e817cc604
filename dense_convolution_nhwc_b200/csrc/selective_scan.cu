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
// Prompts.  The floor is the exponentials: one a (token, channel, state) and four
// more a (token, channel) for softplus and gate, 16 a clock and SM in the
// special-function units.  8192 tokens of 4096 channels and 16 states are 671 million,
// 144 us; their 270 MB of io would take 41 us.  What the kernel spends its time on
// besides is issue slots and shared-memory reads, so both are kept down:
//  * kLanes lanes share a channel, kStates states each in registers; four states a
//    lane (of 16) read b, c and delta a quarter as often as one would.
//  * Two tokens' arguments, additions and sums are one packed instruction each; only
//    the h chain itself is sequential.  A tile of 32 tokens is one straight piece of
//    code (in pieces of 16: 334 us, of 8: 366 us, when this took 309).
//  * The sums over a channel's lanes are taken for 8 tokens together, so that each lane
//    ends with its own tokens' sums (24 instructions for 8 tokens, not 6 for each).
//  * The rest is done by other warps beside the scanning ones: a helping thread owns one
//    token of a tile and eight channels, loads x, dt and z straight into registers a
//    tile ahead, works out delta and delta x, and finishes the tile before while the
//    scanners are at this one.  Done by the scanning warps themselves between their
//    tiles, the call took 393 us.  b becomes fp32 pairs on the way, c stays as it comes:
//    both in fp32 the shared-memory reads bound the kernel, neither the conversions do.
// 8192 tokens of 4096 bf16 channels: 311 us (46 % of the special functions' rate; 128 blocks
// on 148 SMs, bound by the latency of one scanning warp a scheduler: 75 clocks a token).
// 16 sequences of 512 tokens: 240 us (60 %).
//
// A call with too few channels to fill the device cuts the sequences into chunks: a
// first launch leaves each chunk's final state from zero and its sum of delta in the
// workspace, and every chunk of the second folds those before it into its first state
// (the decay over a chunk is exp(a sum delta), see fold).  That doubles the exponentials.  16384
// tokens of 96 fp32 channels: 36 us.
#include <cuda_runtime.h>

#include "sequence.cuh"

namespace b200conv {
namespace {

constexpr int kThreads = 128;     // of a step's block
constexpr int kScanners = 128;    // threads of a prompt's block that hold states

struct ScanArgs {
  const void *x, *dt, *b, *c, *z;
  const float *a, *d, *dt_bias;
  const int *offsets, *slots;
  float* state;
  void* out;
  float *ws_state, *ws_sum;    // chunked: [n][chunks][D][S] states (0: the first, j + 1: after chunk j from zero), [n][chunks][D] thirds of sums
  int n, l, channels, states, groups, state_slots, softplus, carry;
  long long x_s[2], dt_s[2], z_s[2], b_s[2], c_s[2], out_s[2];
  int chunk, chunks;           // tokens a chunk (a multiple of kTile), chunks a sequence
  int tiles;                   // channel tiles a group
  int x_v, dt_v, z_v, b_v, c_v, out_v;   // bytes an access: 16, 8, 4, or 0 for single elements
};

// Copies tiles of kRows x cols elements (cols <= kCols) of a tensor's consecutive
// rows into shared rows kCols elements apart, by kN threads of which this is `me`.
// `bytes`: an access (16, 8, 4, or 0 for single elements), cols and every address
// multiples of it.  In the 16-byte form each thread keeps its address from tile to tile
// where a tile's rows are a multiple of those that the threads cover together (kFits:
// fp32 with 16 states, say; with 16-bit types they cover 64 rows and the addresses are
// worked out anew).
template <typename T, int kRows, int kCols, int kN>
struct Stager {
  static constexpr int E = 16 / sizeof(T), kPer = kCols / E > 0 ? kCols / E : 1;
  static constexpr int kStep = kN / kPer > 0 ? kN / kPer : 1;     // rows between a thread's accesses
  static constexpr bool kFits = kCols % E == 0 && kPer <= kN && kRows % kStep == 0;
  const T* src;
  long long stride;
  int cols, bytes, me, r0, to;
  __device__ __forceinline__ void init(const T* base, long long row_stride, int width, int access, int thread) {
    src = base;
    stride = row_stride;
    cols = width;
    bytes = access;
    me = thread;
    r0 = me / kPer;
    const int q = (me % kPer) * E;
    to = r0 * kCols + q;
    if (kFits && bytes == 16) {
      src += r0 * stride + q;
      if (q >= cols) r0 = kRows;        // past the edge: never a row
    }
  }
  template <int N>
  __device__ __forceinline__ void by(T* dst, int rows) {
    constexpr int kE = N / sizeof(T) > 0 ? N / sizeof(T) : 1, kAcross = kCols / kE > 0 ? kCols / kE : 1;
    for (int i = me; i < rows * kAcross; i += kN) {
      const int r = i / kAcross, q = (i % kAcross) * kE;
      if (q < cols) copy_async<N>(dst + r * kCols + q, src + r * stride + q);
    }
  }
  // Not inlined: its registers are not the kernel's.
  static __device__ __noinline__ void by_element(T* dst, const T* src, long long stride, int rows, int cols, int me) {
    // several loads, then their stores: one after the other each would wait for the last
    constexpr int kAll = (kRows * kCols + kN - 1) / kN, kBatch = kAll < 8 ? kAll : 8;
    for (int i0 = me; i0 < rows * kCols; i0 += kBatch * kN) {
      T v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kN, r = i / kCols, q = i % kCols;
        if (r < rows && q < cols) v[k] = src[r * stride + q];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kN, r = i / kCols, q = i % kCols;
        if (r < rows && q < cols) dst[i] = v[k];
      }
    }
  }
  // The next `rows` rows.
  __device__ __forceinline__ void next(T* dst, int rows) {
    if (kFits && bytes == 16) {
#pragma unroll
      for (int r = 0; r < kRows; r += kStep)
        if (r0 + r < rows) copy_async<16>(dst + to + r * kCols, src + r * stride);
    } else if (bytes == 16) {
      by<16>(dst, rows);
    } else if (bytes == 8) {
      by<8>(dst, rows);
    } else if (bytes == 4) {
      by<4>(dst, rows);
    } else {
      by_element(dst, src, stride, rows, cols, me);
    }
    src += kRows * stride;
  }
};

// One token's values of kHold neighbouring channels.
template <typename T, int kHold>
struct Held {
  static constexpr int kAccess = kHold * sizeof(T) < 16 ? kHold * sizeof(T) : 16;
  alignas(16) T v[kHold];
  // `count` of them are there; vec: all, and kAccess bytes at a time.
  __device__ __forceinline__ void load(const T* p, bool vec, int count) {
    if (vec) {
      using Word = std::conditional_t<kAccess == 16, uint4, std::conditional_t<kAccess == 8, uint2, uint32_t>>;
#pragma unroll
      for (int i = 0; i < (int)(kHold * sizeof(T) / kAccess); ++i)
        reinterpret_cast<Word*>(v)[i] = __ldg(reinterpret_cast<const Word*>(p) + i);
    } else {
#pragma unroll
      for (int i = 0; i < kHold; ++i) v[i] = i < count ? p[i] : Store<T>::from_f32(0.0f);
    }
  }
  __device__ __forceinline__ float at(int i) const { return Store<T>::to_f32(v[i]); }
};

// Barrier kId, or kId + 1 for the second stage, of kN threads.  An arrival orders the
// thread's accesses before it ahead of those after the wait that it completes; no
// fence is needed.  (Ids as immediates, with a branch on the stage, measured 7 % slower.)
template <int kId, int kN>
__device__ __forceinline__ void bar_sync(int stage = 0) {
  asm volatile("bar.sync %0, %1;" ::"r"(kId + stage), "n"(kN) : "memory");
}
template <int kId, int kN>
__device__ __forceinline__ void bar_arrive(int stage) {
  asm volatile("bar.arrive %0, %1;" ::"r"(kId + stage), "n"(kN) : "memory");
}

constexpr int kSms = 148;
constexpr int kTile = 32;   // tokens a tile, one to a lane of the helping warps

template <typename T, int kStates, int kLanes>
struct Shape {
  static constexpr int kChannels = kScanners / kLanes;
  static constexpr int kHold = kChannels < 8 ? kChannels : 8;      // channels a helping thread
  static constexpr int kParts = kChannels / kHold;                 // helping threads a token
  static constexpr int kHelpers = kParts * kTile;
  static constexpr int kBlock = kScanners + kHelpers;
  static constexpr int kWide = kStates * kLanes;             // states, padded
  static constexpr int kTogether = kLanes > 8 ? kLanes : 8;  // tokens reduced together
  static constexpr int kOwn = kTogether / kLanes;            // of which each lane ends with
  static constexpr int kSub = kStates > 4 ? 4 : 8;           // tokens whose exponentials are in flight
  static constexpr int kRow = kTile + 4;                     // floats a channel of delta
  static constexpr int kRing = kWide <= 64 ? 3 : 2;          // tiles of b and c
  // shared memory, in bytes
  static constexpr int kDelta = kChannels * kRow * 4;        // delta, later y; and delta x: a stage of each
  static constexpr int kPairs = kTile * kWide * 4;           // b in fp32: a stage
  static constexpr int kRaw = kTile * kWide * (int)sizeof(T);
  static constexpr int kAtB = 4 * kDelta, kAtRaw = kAtB + 2 * kPairs, kBytes = kAtRaw + 2 * kRing * kRaw;
  static_assert(kTile % kTogether == 0 && kStates % 2 == 0 && kPairs / 8 % kHelpers == 0, "");
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
    float other[kCount / 2];
#pragma unroll
    for (int i = 0; i < kCount / 2; ++i) {
      const float give = upper ? y[i] : y[i + kCount / 2];
      y[i] = upper ? y[i + kCount / 2] : y[i];
      other[i] = __shfl_xor_sync(0xffffffffu, give, kOff);
    }
    if constexpr (kCount >= 4) {
#pragma unroll
      for (int i = 0; i < kCount / 2; i += 2) {
        const float2 sum = __fadd2_rn(make_float2(y[i], y[i + 1]), make_float2(other[i], other[i + 1]));
        y[i] = sum.x;
        y[i + 1] = sum.y;
      }
    } else {
      y[0] += other[0];
    }
    reduce_lanes<kOff / 2, kCount / 2>(y, lane);
  }
}

// Where a token's delta lies in the row of a channel of part `part` of kParts: a whole
// number of eights further on for each part, so that the neighbouring threads of a
// helping warp, which are the parts of the same tokens, write to different banks.
template <int kParts>
__device__ __forceinline__ int turned(int token, int part) {
  return kParts > 1 ? (token + part * (kTile / kParts)) % kTile : token;
}

// kStates neighbouring values.
template <typename T, int kStates>
__device__ __forceinline__ void load_states(const T* p, float (&v)[kStates]) {
  constexpr int kBytes = kStates * sizeof(T), kAccess = kBytes < 16 ? kBytes : 16;
  using Word = std::conditional_t<kAccess == 16, uint4, std::conditional_t<kAccess == 8, uint2, uint32_t>>;
  Word raw[kBytes / kAccess];
#pragma unroll
  for (int i = 0; i < kBytes / kAccess; ++i) raw[i] = reinterpret_cast<const Word*>(p)[i];
  const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
  for (int i = 0; i < kStates; ++i) v[i] = Store<T>::to_f32(e[i]);
}

// The state after a chunk that was entered with h and that ends with `from` when it is
// entered with zero: exp(a sum delta) h + from.  Over a chunk the exponent leaves fp32's
// range where no token's does, so the decay comes as three factors of a third of it,
// each kept within 2^-120 .. 2^120.  Past that the product of a nonzero h (2^-149 at
// least) overflows and that of a finite one vanishes as it should; a state of zero stays
// zero and an infinite one infinite, as they do token by token.
__device__ __forceinline__ float fold(float a, float third_of_sum, float h, float from) {
  const float e = ex2(fminf(fmaxf(fmaf(a, third_of_sum, kEx2Bias), -120.0f), 120.0f));
  return fmaf(e, e * (e * h), from);
}

// kFull: states == kStates * kLanes.  kEnds: the chunk's final state from zero and its sum of delta, no output.
template <typename T, int kStates, int kLanes, bool kFull, bool kEnds, int kBlocks>
__global__ void __launch_bounds__(Shape<T, kStates, kLanes>::kBlock, kBlocks) scan_kernel(const ScanArgs p) {
  using L = Shape<T, kStates, kLanes>;
  constexpr int kReady = 1, kDone = 3, kHelp = 5;      // barriers; the first two have one for each stage
  extern __shared__ __align__(16) unsigned char smem[];
  Where w;
  if (!locate<L::kChannels>(p, &w)) return;
  const int chunk = blockIdx.y, begin = chunk * p.chunk;
  const bool last = begin + p.chunk >= w.len;
  // a chunk without tokens has nothing to do, but for the first one's state of an empty sequence
  if (begin >= w.len && chunk > 0) return;
  if (kEnds && last) return;      // nothing follows it
  const int end = last ? w.len : begin + p.chunk, tiles = (end - begin + kTile - 1) / kTile;

  auto delta_at = [&](int stage) { return reinterpret_cast<float*>(smem + stage * L::kDelta); };        // [channel][kRow]
  auto dx_at = [&](int stage) { return reinterpret_cast<float*>(smem + (2 + stage) * L::kDelta); };
  // b in fp32, the two tokens of a pair side by side: [token / 2][state][token % 2]
  auto pairs_at = [&](int stage) { return reinterpret_cast<float*>(smem + L::kAtB + stage * L::kPairs); };
  auto b_at = [&](int turn) { return reinterpret_cast<T*>(smem + L::kAtRaw + 2 * turn * L::kRaw); };    // [token][kWide]
  auto c_at = [&](int turn) { return reinterpret_cast<T*>(smem + L::kAtRaw + (2 * turn + 1) * L::kRaw); };

  if (threadIdx.x >= kScanners) {
    // ---- helping warps: everything but the recursion, token `row` of each tile and channels c0 .. of the block
    const int me = threadIdx.x - kScanners, row = me / L::kParts, part = me % L::kParts, c0 = part * L::kHold;
    const int row_at = turned<L::kParts>(row, part);       // of the token in delta and delta x
    const int count = min(max(w.count - c0, 0), L::kHold);
    const int ch = w.ch + (count > 0 ? c0 : 0);
    float bias[L::kHold], skip[L::kHold], sum[L::kHold];
#pragma unroll
    for (int k = 0; k < L::kHold; ++k) {
      bias[k] = p.dt_bias && k < count ? __ldg(p.dt_bias + ch + k) : 0.0f;
      skip[k] = !kEnds && p.d && k < count ? __ldg(p.d + ch + k) : 0.0f;
      sum[k] = 0.0f;
    }
    const T* x = rows_of<T>(p, p.x, p.x_s, w, ch) + (begin + row) * p.x_s[1];
    const T* dt = rows_of<T>(p, p.dt, p.dt_s, w, ch) + (begin + row) * p.dt_s[1];
    const T* z = p.z && !kEnds ? rows_of<T>(p, p.z, p.z_s, w, ch) + (begin + row) * p.z_s[1] : nullptr;
    T* out = kEnds ? nullptr : const_cast<T*>(rows_of<T>(p, p.out, p.out_s, w, ch)) + (begin + row) * p.out_s[1];
    using H = Held<T, L::kHold>;
    const bool x_vec = count == L::kHold && p.x_v >= H::kAccess, dt_vec = count == L::kHold && p.dt_v >= H::kAccess;
    const bool z_vec = count == L::kHold && p.z_v >= H::kAccess, out_vec = count == L::kHold && p.out_v >= H::kAccess;
    H next_x, next_dt, next_z, now_x, now_dt, now_z, past_x, past_z;
    auto load = [&](int tile) {
      if (begin + tile * kTile + row < end && count > 0) {
        next_x.load(x, x_vec, count);
        next_dt.load(dt, dt_vec, count);
        if (z) next_z.load(z, z_vec, count);
      }
      x += kTile * p.x_s[1];
      dt += kTile * p.dt_s[1];
      if (z) z += kTile * p.z_s[1];
    };
    auto finish = [&](int tile) {
      if constexpr (!kEnds) {
        if (begin + tile * kTile + row < end && count > 0) {
          const float* y = delta_at(tile & 1) + c0 * L::kRow + row_at;
          H to;
          float v[L::kHold];
#pragma unroll
          for (int k = 0; k < L::kHold; ++k) v[k] = y[k * L::kRow];
          if (p.d) {
#pragma unroll
            for (int k = 0; k < L::kHold; ++k) v[k] = fmaf(skip[k], past_x.at(k), v[k]);
          }
          if (z) {
#pragma unroll
            for (int k = 0; k < L::kHold; k += 2) {
              const float2 gate = silu(make_float2(past_z.at(k), past_z.at(k + 1)));
              const float2 two = __fmul2_rn(make_float2(v[k], v[k + 1]), gate);
              v[k] = two.x;
              v[k + 1] = two.y;
            }
          }
#pragma unroll
          for (int k = 0; k < L::kHold; ++k) to.v[k] = Store<T>::from_f32(v[k]);
          if (out_vec) {
            using Word = std::conditional_t<H::kAccess == 16, uint4, std::conditional_t<H::kAccess == 8, uint2, uint32_t>>;
#pragma unroll
            for (int i = 0; i < (int)(L::kHold * sizeof(T) / H::kAccess); ++i)
              reinterpret_cast<Word*>(out)[i] = reinterpret_cast<const Word*>(to.v)[i];
          } else {
#pragma unroll
            for (int k = 0; k < L::kHold; ++k)
              if (k < count) out[k] = to.v[k];
          }
        }
        out += kTile * p.out_s[1];
      }
    };
    Stager<T, kTile, L::kWide, L::kHelpers> sb, sc;
    sb.init(rows_of<T>(p, p.b, p.b_s, w, w.group * p.states) + begin * p.b_s[1], p.b_s[1], p.states, p.b_v, me);
    if (!kEnds) sc.init(rows_of<T>(p, p.c, p.c_s, w, w.group * p.states) + begin * p.c_s[1], p.c_s[1], p.states, p.c_v, me);
    auto fetch = [&](int tile) {
      const int rows = min(kTile, end - begin - tile * kTile);
      if (rows > 0) {
        sb.next(b_at(tile % L::kRing), rows);
        if (!kEnds) sc.next(c_at(tile % L::kRing), rows);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (!kFull) {       // the states that are not there: zeros, which no tile overwrites
      const int pad = L::kWide - p.states;
      for (int i = me; i < 2 * L::kRing * kTile * pad; i += L::kHelpers)
        b_at(0)[i / pad * L::kWide + p.states + i % pad] = Store<T>::from_f32(0.0f);
    }
    load(0);                // first: where b and c are copied element by element, the fetches wait for them
#pragma unroll
    for (int i = 0; i < L::kRing - 1; ++i) fetch(i);
    for (int tile = 0; tile < tiles; ++tile) {
      const int stage = tile & 1;
      now_x = next_x;
      now_dt = next_dt;
      now_z = next_z;
      if (tile + 1 < tiles) load(tile + 1);
      float de[L::kHold];
#pragma unroll
      for (int k = 0; k < L::kHold; ++k) de[k] = now_dt.at(k) + bias[k];
      if (p.softplus) {
#pragma unroll
        for (int k = 0; k < L::kHold; k += 2) {
          const float2 two = softplus(make_float2(de[k], de[k + 1]));
          de[k] = two.x;
          de[k + 1] = two.y;
        }
      }
#pragma unroll
      for (int k = 0; k < L::kHold; ++k) {
        delta_at(stage)[(c0 + k) * L::kRow + row_at] = de[k];
        dx_at(stage)[(c0 + k) * L::kRow + row_at] = de[k] * now_x.at(k);
        if (kEnds && begin + tile * kTile + row < end) sum[k] += de[k];
      }
      // this tile's b and c are here, and for every helper
      asm volatile("cp.async.wait_group %0;" ::"n"(L::kRing - 2) : "memory");
      bar_sync<kHelp, L::kHelpers>();
      const T* raw = b_at(tile % L::kRing);
      float2* pairs = reinterpret_cast<float2*>(pairs_at(stage));
      constexpr int kTurns = L::kPairs / 8 / L::kHelpers, kBatch = kTurns > 8 ? 8 : kTurns;
#pragma unroll 1
      for (int i0 = me; i0 < L::kPairs / 8; i0 += kBatch * L::kHelpers) {
        float2 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = i0 + k * L::kHelpers;
          const T* from = raw + i / L::kWide * 2 * L::kWide + i % L::kWide;
          v[k] = make_float2(ld_f32(from), ld_f32(from + L::kWide));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) pairs[i0 + k * L::kHelpers] = v[k];
      }
      bar_arrive<kReady, L::kBlock>(stage);
      if (tile > 0) bar_sync<kDone, L::kBlock>(stage ^ 1);
      fetch(tile + L::kRing - 1);
      if (tile > 0) finish(tile - 1);
      past_x = now_x;
      past_z = now_z;
    }
    if (tiles > 0) {
      bar_sync<kDone, L::kBlock>((tiles - 1) & 1);
      finish(tiles - 1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (kEnds) {
      // over the rows: a warp's by shuffles, the warps' through the stage that no scanner reads any more
      float* sums = dx_at(0);
      bar_sync<kHelp, L::kHelpers>();
#pragma unroll
      for (int k = 0; k < L::kHold; ++k) {
#pragma unroll
        for (int off = L::kParts; off < 32; off *= 2) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], off);
        if (me % 32 < L::kParts) sums[me / 32 * L::kChannels + c0 + k] = sum[k];
      }
      bar_sync<kHelp, L::kHelpers>();
      for (int c = me; c < w.count; c += L::kHelpers) {
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < L::kHelpers / 32; ++i) all += sums[i * L::kChannels + c];
        p.ws_sum[((long long)w.seq * p.chunks + chunk) * p.channels + w.ch + c] = all * (1.0f / 3.0f);
      }
    }
    return;
  }

  // ---- scanning warps: kLanes lanes a channel, kStates states a lane
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
    if (chunk == 0 && live) {
#pragma unroll
      for (int i = 0; i < kStates; ++i)
        if (i < have) p.ws_state[ws_row + i] = p.carry ? cache[i] : 0.0f;
    }
  } else if (p.chunks > 1 && !(chunk == 0 && last)) {
#pragma unroll
    for (int i = 0; i < kStates; ++i)
      if (i < have) h[i] = p.ws_state[ws_row + i];
    const float *sums = p.ws_sum + (long long)w.seq * p.chunks * p.channels + ch, *ends = p.ws_state + ws_row + ws_step;
    constexpr int kAhead = 8;      // chunks whose loads are in flight together
    for (int j = 0; j < chunk; j += kAhead) {
      float sum[kAhead], from[kAhead][kStates];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool there = j + u < chunk;
        sum[u] = there ? sums[(j + u) * (long long)p.channels] : 0.0f;
#pragma unroll
        for (int i = 0; i < kStates; ++i) from[u][i] = there && i < have ? ends[(j + u) * ws_step + i] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < kStates; ++i)
          if (j + u < chunk && i < have) h[i] = fold(a2[i].x, sum[u], h[i], from[u][i]);
    }
  } else if (p.carry) {
#pragma unroll
    for (int i = 0; i < kStates; ++i)
      if (i < have) h[i] = cache[i];
  }

  for (int tile = 0; tile < tiles; ++tile) {
    const int stage = tile & 1, rows = min(kTile, end - begin - tile * kTile);
    float* delta_of = delta_at(stage) + cl * L::kRow;
    const int part = cl / L::kHold;
    const float *dx_of = dx_at(stage) + cl * L::kRow, *bf = pairs_at(stage);
    const T* cr = c_at(tile % L::kRing);
    bar_sync<kReady, L::kBlock>(stage);

    // kSub tokens from t: the states advance, and y gets this lane's share of the sums
    // over them.  The exponentials and additions of all tokens come first, two tokens
    // to a packed instruction; only the h chain itself is sequential.  kTail: tokens
    // from `rows` on leave the states alone.
    auto sub = [&](auto tail, int t, float* y) {
      constexpr bool kTail = decltype(tail)::value;
      constexpr int kSub = L::kSub;
      const int t_at = turned<L::kParts>(t, part);
      float2 e[kSub / 2][kStates], add[kSub / 2][kStates];
#pragma unroll
      for (int q = 0; q < kSub; q += 4) {
        const float4 de = *reinterpret_cast<const float4*>(delta_of + t_at + q);
        const float4 dx = *reinterpret_cast<const float4*>(dx_of + t_at + q);
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
        float ct[2][kStates];
        if (!kEnds) {
          load_states<T, kStates>(cr + (t + 2 * q) * L::kWide + s0, ct[0]);
          load_states<T, kStates>(cr + (t + 2 * q + 1) * L::kWide + s0, ct[1]);
        }
#pragma unroll
        for (int i = 0; i < kStates; ++i) {
          float h0 = fmaf(e[q][i].x, h[i], add[q][i].x);
          if (!kFull && i >= have) h0 = 0.0f;
          if (kTail && t + 2 * q >= rows) h0 = h[i];
          float h1 = fmaf(e[q][i].y, h0, add[q][i].y);
          if (!kFull && i >= have) h1 = 0.0f;
          if (kTail && t + 2 * q + 1 >= rows) h1 = h0;
          h[i] = h1;
          if (!kEnds) sum2 = __ffma2_rn(make_float2(ct[0][i], ct[1][i]), make_float2(h0, h1), sum2);
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
    // kMany groups, then their sums in the place of their deltas: a store in between
    // would hold back the next group's loads
    auto groups = [&](auto tail, auto many, int t) {
      constexpr int kMany = decltype(many)::value;
      float own[kMany * L::kOwn];
#pragma unroll
      for (int g = 0; g < kMany; ++g) group(tail, t + g * L::kTogether, own + g * L::kOwn);
      if constexpr (!kEnds) {
        __syncwarp();
#pragma unroll
        for (int g = 0; g < kMany; ++g)
#pragma unroll
          for (int i = 0; i < L::kOwn; ++i)
            delta_of[turned<L::kParts>(t + g * L::kTogether, part) + lane * L::kOwn + i] = own[g * L::kOwn + i];
      }
    };
    if (rows == kTile) {
      groups(std::false_type{}, std::integral_constant<int, kTile / L::kTogether>{}, 0);
    } else {
      for (int t = 0; t < rows; t += L::kTogether) groups(std::true_type{}, std::integral_constant<int, 1>{}, t);
    }
    bar_arrive<kDone, L::kBlock>(stage);
  }

  if (!live) return;
  if constexpr (kEnds) {
#pragma unroll
    for (int i = 0; i < kStates; ++i)
      if (i < have) p.ws_state[ws_row + (chunk + 1) * ws_step + i] = h[i];
  } else if (last && cache) {
#pragma unroll
    for (int i = 0; i < kStates; ++i)
      if (i < have) cache[i] = h[i];
  }
}

// ------------------------------ single tokens ----------------------------------

constexpr int kWalkBlocks = 5;      // of a walking step, an SM

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
// took 260 instructions for four states, mostly addresses and the softplus (192
// sequences of 4096 channels, 16 states: 38 us, with four channels 26 us = 4.1 TB/s).
template <typename T, int kLanes, int kMine, bool VEC>
__global__ void __launch_bounds__(kThreads, 6) scan_step_kernel(const StepArgs p) {
  constexpr int kAcross = 32 / kLanes, kSub = kLanes / kMine;   // channels side by side; lanes that hold one channel's token
  const int seq = blockIdx.z * gridDim.y + blockIdx.y;
  if (seq >= p.n) return;
  const int lane = threadIdx.x % kLanes;
  const int first = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kAcross * kMine + threadIdx.x % 32 / kLanes;
  const int mine = first + lane / kSub * kAcross;
  // Only the state hangs on the slot: everything else is asked for before the slot is looked at.
  const int slot = slot_of(p.slots, seq, p.state_slots);
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
  float* state = p.state + (long long)max(slot, 0) * p.channels * p.states;
  float de2[kMine], dx[kMine], y[kMine];
#pragma unroll
  for (int q = 0; q < kMine; ++q) y[q] = 0.0f;
  // the lanes past the states take part in the first turn's shuffles
  for (int s = lane * 4, turn = 0; turn == 0 || s < p.states; s += kLanes * 4, ++turn) {
    const int have = min(max(p.states - s, 0), 4);
    float av[kMine][4], h[kMine][4], bv[4], cv[4];
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
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const float* ap = p.a + (long long)min(first + q * kAcross, p.channels - 1) * p.states + s;
      if (VEC && have == 4) {
        load_f32<float, 4, true>(ap, av[q]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) av[q][i] = i < have ? __ldg(ap + i) : 0.0f;
      }
    }
    if (slot < 0) return;         // the whole block's
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const float* hp = state + (long long)min(first + q * kAcross, p.channels - 1) * p.states + s;
      if (VEC && have == 4) {
        load_f32<float, 4, true>(hp, h[q]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[q][i] = i < have ? hp[i] : 0.0f;
      }
    }
    if (turn == 0) {
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

// The same where a block goes through several sequences (all accesses of four states,
// at most 4 kLanes of them): a is read once, and the next sequence's state, token, b
// and c are on their way while the present one's are worked on, its slot two ahead.
// 192 sequences of 4096 channels, 16 states, their slots scattered: 20.2 us = 5.3 TB/s, 81 %
// of the copy rate.
template <typename T, int kLanes, int kMine>
__global__ void __launch_bounds__(kThreads, kWalkBlocks) scan_step_walk_kernel(const StepArgs p) {
  constexpr int kAcross = 32 / kLanes, kSub = kLanes / kMine;
  const int lane = threadIdx.x % kLanes, s = lane * 4;
  const bool have = s < p.states;
  const int first = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kAcross * kMine + threadIdx.x % 32 / kLanes;
  const int mine = first + lane / kSub * kAcross, mine_in = min(mine, p.channels - 1);
  const int group = p.groups > 1 ? min(first, p.channels - 1) / (p.channels / p.groups) : 0;
  const float bias = p.dt_bias ? __ldg(p.dt_bias + mine_in) : 0.0f, skip = p.d ? __ldg(p.d + mine_in) : 0.0f;
  float av[kMine][4];
  int at[kMine];               // of the lane's states in a slot
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    at[q] = min(first + q * kAcross, p.channels - 1) * p.states + s;
    if (have) load_f32<float, 4, true>(p.a + at[q], av[q]);
  }
  struct Next {
    T x, dt, z;
    Held<T, 4> b, c;
    float h[kMine][4];
  } next;
  auto load = [&](int seq, int slot) {
    if (slot < 0) return;
    next.x = static_cast<const T*>(p.x)[seq * p.x_s + mine_in];
    next.dt = static_cast<const T*>(p.dt)[seq * p.dt_s + mine_in];
    if (p.z) next.z = static_cast<const T*>(p.z)[seq * p.z_s + mine_in];
    if (have) {
      next.b.load(static_cast<const T*>(p.b) + seq * p.b_s + group * p.states + s, true, 4);
      next.c.load(static_cast<const T*>(p.c) + seq * p.c_s + group * p.states + s, true, 4);
      const float* state = p.state + (long long)slot * p.channels * p.states;
#pragma unroll
      for (int q = 0; q < kMine; ++q) load_f32<float, 4, true>(state + at[q], next.h[q]);
    }
  };
  auto slot_at = [&](long long seq) { return seq < p.n ? slot_of(p.slots, (int)seq, p.state_slots) : -1; };
  const int step = gridDim.y;
  int slot = slot_at(blockIdx.y), slot_next = slot_at((long long)blockIdx.y + step);
  load(blockIdx.y, slot);
  for (long long seq = blockIdx.y; seq < p.n; seq += step) {
    Next now = next;
    const int slot_now = slot;
    slot = slot_next;
    slot_next = slot_at(seq + 2LL * step);
    if (seq + step < p.n) load((int)(seq + step), slot);
    if (slot_now < 0) continue;
    const float xv = Store<T>::to_f32(now.x);
    float delta = Store<T>::to_f32(now.dt) + bias;
    if (p.softplus) delta = softplus(delta);
    const float mine_de2 = delta * kLog2e, mine_dx = delta * xv;
    float y[kMine];
    float* state = p.state + (long long)slot_now * p.channels * p.states;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const float de2 = __shfl_sync(0xffffffffu, mine_de2, q * kSub, kLanes);
      const float dx = __shfl_sync(0xffffffffu, mine_dx, q * kSub, kLanes);
      y[q] = 0.0f;
      if (have) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          now.h[q][i] = fmaf(decay(av[q][i], de2), now.h[q][i], dx * now.b.at(i));
          y[q] = fmaf(now.c.at(i), now.h[q][i], y[q]);
        }
        if (first + q * kAcross < p.channels) store_f32<float, 4, true>(state + at[q], now.h[q]);
      }
    }
    reduce_lanes<kLanes / 2, kMine>(y, lane);
    if (lane % kSub == 0 && mine < p.channels) {
      float v = y[0];
      if (p.d) v = fmaf(skip, xv, v);
      if (p.z) v *= silu(Store<T>::to_f32(now.z));
      st_f32(static_cast<T*>(p.out) + seq * p.out_s + mine, v);
    }
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
    kernel<<<grid, L::kBlock, L::kBytes, s>>>(p);
    return cudaGetLastError();
  };
  if (p.chunks > 1) {
    cudaError_t e = run(scan_kernel<T, kStates, kLanes, kFull, true, 2>);
    if (e != cudaSuccess) return e;
  }
  // With a block an SM at most, the registers of two make a better schedule (8192 tokens
  // of 4096 channels: 311 us with 147 registers, 334 with the 128 of two blocks an SM).
  // Built for the states that fill their lanes alone.
  if constexpr (kFull) {
    if (blocks * p.chunks <= kSms) return run(scan_kernel<T, kStates, kLanes, kFull, false, 1>);
  }
  return run(scan_kernel<T, kStates, kLanes, kFull, false, (L::kBytes > 110 * 1024 ? 1 : 2)>);
}

template <typename T>
cudaError_t scan_typed(const ScanArgs& p, const ScanPlan& plan, cudaStream_t s) {
#define B200CONV_SCAN(S, L, F) \
  if (plan.states_per_lane == S && plan.lanes == L && (!F || p.states == S * L)) return scan_shaped<T, S, L, F>(p, s)
  B200CONV_SCAN(4, 4, true);
  B200CONV_SCAN(2, 4, false);
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
    if constexpr (kMine > 1) {
      // Five blocks an SM, each through two sequences or more (192 sequences of 4096
      // channels, 16 states: 20.2 us against 26.4 with a block a sequence; 64: 6.5 and 7.9;
      // four and six blocks an SM 20.9 and 27.8).
      const long long walk = (long long)kSms * kWalkBlocks / grid.x;
      if (mine > 1 && vec && p.bc_vec && p.states <= 4 * lanes && walk > 0 && 2 * walk <= p.n) {
        scan_step_walk_kernel<T, l(), kMine><<<dim3(grid.x, (unsigned)walk), kThreads, 0, s>>>(p);
        return cudaGetLastError();
      }
    }
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

constexpr int kLeastChunk = 64, kMostChunks = 128;

// Pure in the descriptor and the device's SM count.
ScanPlan plan_scan(const selective_scan_desc_t& d, int sm_count) {
  ScanPlan plan{};
  // Four states a lane: with two the shared-memory reads of b, c and delta bound the
  // kernel (8192 tokens of 4096 channels, 16 states: 359 us on 8 lanes where 4 took 322;
  // 16 sequences of 512 tokens 338 and 251).
  plan.states_per_lane = d.s <= 8 ? 2 : 4;
  plan.lanes = 4;
  while (plan.lanes * plan.states_per_lane < d.s) {
    if (plan.lanes < 32) plan.lanes *= 2;
    else plan.states_per_lane *= 2;
  }
  const int channels = kScanners / plan.lanes;
  const long long per_group = d.d / d.groups;
  const long long blocks = (long long)d.n * d.groups * ((per_group + channels - 1) / channels);
  plan.chunk = d.l > 0 ? (d.l + kTile - 1) / kTile * kTile : kTile;
  plan.chunks = 1;
  // Cut, every token is gone over twice: it pays from four chunks on (8192 tokens of
  // 2048 channels, 4 chunks: 236 us against 322; 2048 of 3000, 3 chunks: 89 against 84).
  // Two blocks an SM are enough, and a chunk's start is worked out from all chunks
  // before it, so not too many (16384 tokens of 32 channels: 27.5 us in 148 chunks,
  // 38.6 in 256) nor too short ones.
  // Packed sequences share their rows, and the longest decides: chunks of the size
  // that cuts all of them together into as many (a shorter sequence is one chunk, gone
  // over once), from half the device idle on.  Chunks past a sequence's end still cost
  // a block each, so sixteen times as many at most.  11 sequences in 10813 rows: of 48
  // channels 65 us cut as if each had all the rows, 19.7 so; of 300 uncut 135, so 81.
  long long want = blocks > 0 ? 2LL * sm_count / blocks : 0;
  if (d.packed && want >= 2) want *= d.n < 16 ? d.n : 16;
  const long long most = (d.l + kLeastChunk - 1LL) / kLeastChunk;
  long long chunks = want < most ? want : most;
  if (chunks > kMostChunks) chunks = kMostChunks;
  if (chunks >= 4) {
    plan.chunk = (int)(((d.l + chunks - 1) / chunks + kTile - 1) / kTile * kTile);
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

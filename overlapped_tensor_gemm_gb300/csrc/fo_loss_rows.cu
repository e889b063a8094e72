// Row kernels of the losses (formulas in fo_loss.cuh).
//
// Bound by HBM.  A row's columns are shared by a team of 1 to 8 CTAs.  One warp of a CTA orders the
// copies of its columns (cp.async.bulk, 32 KB each, into a ring of slots in shared memory, rows
// ahead); the others compute on them.
//   Statistics: every warp sums what it sees of a row and tells its part to every CTA of the team;
// one warp of each CTA, another one for each row, adds the parts.  Nobody waits for it but the
// gradient.
//   Policy loss with gradient: the row waits in shared memory for its sum, so that the logits are
// read once, is turned into its gradient in place and copied from there (where both have one type).
// Two sets of eight warps take the rows in turn, so that one's waits are covered by the other.
//   Backward: the gradient alone, from statistics given.
// Statistics alone and gradients alone run two CTAs on an SM, for the same reason; the policy loss
// has one, for room.
//
// Measured, 4096 rows of 8 x 16384 bf16: statistics with entropy 157 us (6.8 TB/s), policy loss with a
// quarter of the rows masked 305 (6.1 TB/s; clusters of 4 use 144 of 152 SMs); gradients alone, 1024 rows,
// 79 us (6.7 TB/s).
//
// A thread sums relative to a column of its own that is near its maximum (at most 16 octaves below),
// so that a new maximum does not cost a pass; log2 domain, two columns per instruction.
#include <atomic>
#include <cfloat>
#include <cstring>

#include "fo_loss.cuh"
#include "fo_wide.cuh"

namespace fo {
namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr double kLog2e = 1.4426950408889634;
constexpr float kOctaves = 16.f;  // a sum's reference may lie so far below its maximum
// 2^d is 0 in fp32 from here on down: where d multiplies it, d ends here (0 times -infinity)
constexpr float kFarBelow = -160.f;
constexpr int kChunkGroups = kLossChunk / 16;

// How a kernel's CTA is made up
template <int kMode>
struct Shape {
  static constexpr bool kOne = kMode == kLossPolicy;
  static constexpr int kPerSm = kOne ? 1 : 2;
  static constexpr int kSets = kOne ? 2 : 1;            // sets of warps that take the rows in turn
  static constexpr int kWarps = 8;                      // warps of a set
  static constexpr int kMore = kOne ? 2 : 1;            // warps that order the copies in, and the copies out
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kAll = kSets * kThreads;
  static constexpr int kSlots = kOne ? 6 : 3;
  static constexpr int kZeros = kOne ? 8192 : 0;        // bytes of zeros behind the ring
  static constexpr int kBatch = kChunkGroups / kThreads;  // groups of a chunk per thread
};
constexpr int kLossFit = 2;   // a row's chunks in one CTA, where more CTAs can share it: both sets' rows and the
                              // next one's copies have room
constexpr uint64_t kLossDrainNs = 2000000000ull;

typedef uint64_t Pair;
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair both(float f) { return pack2(f, f); }
__device__ __forceinline__ float sum2(Pair a) {
  float x, y;
  unpack2(a, x, y);
  return x + y;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A group: the 16 bytes of a vector, 8 or 4 columns
template <typename T>
struct Group;
template <>
struct Group<uint16_t> {
  static constexpr int kCols = 8;
  // the largest of n groups
  template <int n>
  static __device__ __forceinline__ float top(const uint4 (&q)[n]) {
    uint32_t m = max_bf16x2(max_bf16x2(q[0].x, q[0].y), max_bf16x2(q[0].z, q[0].w));
#pragma unroll
    for (int k = 1; k < n; ++k)
      m = max_bf16x2(m, max_bf16x2(max_bf16x2(q[k].x, q[k].y), max_bf16x2(q[k].z, q[k].w)));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  // the columns less base
  static __device__ __forceinline__ void above(const uint4& q, float nbase, Pair (&v)[4]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo, hi;
      asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; add.f32.bf16 %0, l, %3; add.f32.bf16 %1, h, %3;}"
          : "=f"(lo), "=f"(hi)
          : "r"(w[k]), "f"(nbase));
      v[k] = pack2(lo, hi);
    }
  }
};
template <>
struct Group<float> {
  static constexpr int kCols = 4;
  template <int n>
  static __device__ __forceinline__ float top(const uint4 (&q)[n]) {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < n; ++k)
      m = fmax3(fmax3(m, __uint_as_float(q[k].x), __uint_as_float(q[k].y)), __uint_as_float(q[k].z),
                __uint_as_float(q[k].w));
    return m;
  }
  static __device__ __forceinline__ void above(const uint4& q, float nbase, Pair (&v)[2]) {
    v[0] = fadd2(pack2(__uint_as_float(q.x), __uint_as_float(q.y)), both(nbase));
    v[1] = fadd2(pack2(__uint_as_float(q.z), __uint_as_float(q.w)), both(nbase));
  }
};
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
template <int kPairs>
__device__ __forceinline__ void store_group(uint16_t* p, const Pair (&v)[kPairs]) {
  uint32_t q[kPairs];
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    float x, y;
    unpack2(v[k], x, y);
    q[k] = pack_bf16x2(x, y);
  }
  if constexpr (kPairs == 4) {
    *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
  }
}
template <int kPairs>
__device__ __forceinline__ void store_group(float* p, const Pair (&v)[kPairs]) {
#pragma unroll
  for (int k = 0; k < kPairs; k += 2) {
    float f[4];
    unpack2(v[k], f[0], f[1]);
    unpack2(v[k + 1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 2 * k) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// The sum over each eight lanes, in all of them
__device__ __forceinline__ double eighth_sum(double v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What is subtracted for a reference m: finite also where every column is -infinity
__device__ __forceinline__ float base_of(float m) { return fmaxf(m, -FLT_MAX); }

// A part of a row's statistics: reference m, s = sum 2^d, t = sum 2^d d with d = (z - m) c
struct __align__(16) Part {  // (moved by 16-byte stores: st.async faults on a place that is not aligned)
  float m, s, t, reserved;
};

// ln s in twice fp32: the exponent's share in two products of which one is exact, and the logarithm of a
// number near 1
__device__ __forceinline__ Wide wide_log(float s) {
  const int bits = __float_as_int(s);
  if (static_cast<uint32_t>(bits) - 0x00800000u >= 0x7f000000u) return wide(logf(s));  // 0, subnormal, infinite, NaN
  const int e = (bits - 0x3f400000) >> 23;  // s = 2^e m, m from 3/4 to 3/2
  const float m = __int_as_float(bits - (e << 23)), n = static_cast<float>(e);
  // ln 2 = 0.693145751953125 (16 bits) + 1.42860677e-6
  return plus(wide(n * 0.693145751953125f), wide(fmaf(n, 1.42860677e-6f, logf(m))));
}

// ex2.approx cuts its results off: they are 5.0e-8 too small in the mean (3e-8 the spread about that; measured
// on a GB300 over 6 million arguments from -12 to 0), which would show in every row's logarithm with the same
// sign.  The largest column's own term, the 1 of a sum s, is exact: a part (s - 1) / s of the mean is added
// back in logp and lse.  The entropy goes without it: it is less than a rounding of an entropy above 1/2, and
// smaller ones have a small s - 1.
constexpr float kExpMean = 5.0e-8f;

// The parts of all lanes as one, in every lane
template <bool kEnt>
__device__ __forceinline__ Part join(Part v, float c) {
  const float m = warp_max(v.m), d = (base_of(v.m) - base_of(m)) * c;
  // (parts without a finite column have s = 0, whatever their factor)
  const float f = fast_exp2(d);
  Part r;
  r.m = m;
  r.t = kEnt ? warp_sum(f * fmaf(v.s, fmaxf(d, kFarBelow), v.t)) : 0.f;
  r.s = warp_sum(f * v.s);
  r.reserved = 0.f;
  return r;
}
template <bool kEnt>
__device__ __forceinline__ Part merge(const Part& v, const Part& w, float c) {
  Part r;
  r.m = fmaxf(v.m, w.m);
  const float dv = (base_of(v.m) - base_of(r.m)) * c, dw = (base_of(w.m) - base_of(r.m)) * c;
  const float fv = fast_exp2(dv), fw = fast_exp2(dw);
  r.t = kEnt ? fv * fmaf(v.s, fmaxf(dv, kFarBelow), v.t) + fw * fmaf(w.s, fmaxf(dw, kFarBelow), w.t) : 0.f;
  r.s = fv * v.s + fw * w.s;
  r.reserved = 0.f;
  return r;
}

// A thread's sums over a row: s and t relative to m, two columns side by side
struct Sums {
  float m;
  Pair s, t;
};
// n groups in shared memory, `pitch` apart, into the sums
template <typename TZ, bool kEnt, int n, int pitch>
__device__ __forceinline__ void add_groups(const uint4* src, float c, float slack, Sums& v) {
  constexpr int kPairs = Group<TZ>::kCols / 2;
  uint4 q[n];
#pragma unroll
  for (int k = 0; k < n; ++k) q[k] = src[k * pitch];
  const float top = Group<TZ>::top(q);
  if (top > v.m + slack) {
    const float d = (base_of(v.m) - base_of(top)) * c;
    const Pair f = both(fast_exp2(d));
    if (kEnt) v.t = mul2(f, ffma2(v.s, both(fmaxf(d, kFarBelow)), v.t));
    v.s = mul2(f, v.s);
    v.m = top;
  }
  const float nbase = -base_of(v.m);
  const Pair c2 = both(c), before = v.t;
#pragma unroll
  for (int k = 0; k < n; ++k) {
    Pair x[kPairs];
    Group<TZ>::above(q[k], nbase, x);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      const Pair d = mul2(x[e], c2);
      float lo, hi;
      unpack2(d, lo, hi);
      const Pair w = pack2(fast_exp2(lo), fast_exp2(hi));
      v.s = fadd2(v.s, w);
      if (kEnt) v.t = ffma2(w, d, v.t);
    }
  }
  if (kEnt && !(sum2(v.t) < INFINITY)) {  // 0 times -infinity: again, with d at least kFarBelow
    v.t = before;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      Pair x[kPairs];
      Group<TZ>::above(src[k * pitch], nbase, x);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        float lo, hi;
        unpack2(mul2(x[e], c2), lo, hi);
        v.t = ffma2(pack2(fast_exp2(lo), fast_exp2(hi)), pack2(fmaxf(lo, kFarBelow), fmaxf(hi, kFarBelow)), v.t);
      }
    }
  }
}

// How a row's gradient is made: 2^d (k0 + k1 d) with d = (z - base) c
struct Slope {
  float base, c, k0, k1;
};
template <bool kEnt>
__device__ __forceinline__ float slope_at(const Slope& g, float z) {
  const float d = (z - g.base) * g.c;
  return fast_exp2(d) * (kEnt ? fmaf(fmaxf(d, kFarBelow), g.k1, g.k0) : g.k0);
}
template <typename TZ, typename TD, bool kEnt>
__device__ __forceinline__ void put_group(const uint4& q, const Slope& g, TD* to) {
  constexpr int kPairs = Group<TZ>::kCols / 2;
  const Pair c2 = both(g.c), k0 = both(g.k0), k1 = both(g.k1);
  Pair x[kPairs];
  Group<TZ>::above(q, -g.base, x);
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    float lo, hi;
    unpack2(mul2(x[e], c2), lo, hi);
    const Pair w = pack2(fast_exp2(lo), fast_exp2(hi));
    x[e] = kEnt ? mul2(w, ffma2(pack2(fmaxf(lo, kFarBelow), fmaxf(hi, kFarBelow)), k1, k0)) : mul2(w, k0);
  }
  store_group<kPairs>(to, x);
}

// A place in the ring that advances chunk by chunk
template <int kSlots>
struct Place {
  uint32_t slot = 0, turn = 0;  // turn: parity of the slot's use
  __device__ __forceinline__ void next() {
    if (++slot == kSlots) {
      slot = 0;
      turn ^= 1;
    }
  }
  __device__ __forceinline__ void skip(int n) {
    for (; n > 0; --n) next();
  }
};

__device__ __forceinline__ bool offsets_fine(const int32_t* off, int n, int64_t rows, uint32_t* ctrl) {
  int bad = -1;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int32_t v = off[i];
    if (v < 0 || v > rows || (i > 0 && off[i - 1] > v)) bad = i;
  }
  if (!__syncthreads_or(bad >= 0)) return true;
  if (bad >= 0 && blockIdx.x == 0) note_error(ctrl, FO_ERR_RANGE, kSiteOffsets, bad);
  return false;
}

// Sum of the counted rows' weights over the computing warps, in the same order in every CTA
// (compensated: any number of rows)
template <int kWarps>
__device__ __forceinline__ float total_weight(const LossArgs& a, float* buf) {
  float sum = 0.f, low = 0.f;
  constexpr int kTogether = 4;  // (loads under way at once)
  for (int64_t i = threadIdx.x; i < a.rows; i += kTogether * 32 * kWarps) {
    int32_t y[kTogether];
    float w[kTogether];
#pragma unroll
    for (int k = 0; k < kTogether; ++k) {
      const int64_t at = i + k * 32 * kWarps;
      y[k] = at < a.rows ? a.targets[at] : -1;
      w[k] = at < a.rows && a.weights ? a.weights[at] : 1.f;
    }
#pragma unroll
    for (int k = 0; k < kTogether; ++k) {
      const float x = (y[k] >= 0 && y[k] < a.first[a.P] ? w[k] : 0.f) - low, next = sum + x;
      low = (next - sum) - x;
      sum = next;
    }
  }
  sum = warp_sum(sum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[warp] = sum;
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
  return warp_sum(lane < kWarps ? buf[lane] : 0.f);
}

constexpr int kBoxes = 4;

template <typename S>
struct Smem {
  uint64_t full[S::kSlots], empty[S::kSlots], made[S::kSlots], told[kBoxes], ready[S::kSets];
  Part part[kBoxes][kLossMaxCtas * S::kWarps];
  float4 slope[S::kSets];          // base, k0, k1, own of a set's row (Slope)
  double sums[S::kSets * S::kWarps][4];
  float buf[S::kSets * S::kWarps];
};

// A lane's row of a batch of 32
struct RowIn {
  int32_t y;
  bool on;
};

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// A wait that depends on copies, or on this row's other warps: an abort that an earlier call left
// behind does not end it
__device__ __forceinline__ bool wait_full(uint64_t* bar, uint32_t parity, const LossArgs& a) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || mbar_wait_drain(bar, parity, a.timeout_ns));
}
static __device__ __noinline__ bool wait_told_slow(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_cluster(bar, parity))
    if (global_timer_ns() - t0 > limit_ns) return false;
  return true;
}
__device__ __forceinline__ bool wait_told(uint64_t* bar, uint32_t parity, const LossArgs& a) {
  return __all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity) || wait_told_slow(bar, parity, a.timeout_ns));
}

// kEnt: forward: the entropy is wanted; policy and backward: it has a gradient.  (The policy loss's
// statistics have the entropy anyway.)
template <typename TZ, typename TD, int kMode, bool kEnt>
__global__ void __launch_bounds__(Shape<kMode>::kAll + 32 * Shape<kMode>::kMore, Shape<kMode>::kPerSm)
    loss_rows_kernel(const __grid_constant__ LossArgs a) {
  typedef Shape<kMode> S;
  typedef Place<S::kSlots> P;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ Smem<S> sm;
  constexpr bool kStat = kMode != kLossBackward;
  constexpr bool kStatEnt = kMode == kLossPolicy || (kMode == kLossForward && kEnt);
  constexpr int kCols = Group<TZ>::kCols, kPairs = kCols / 2;
  constexpr int kSlots = S::kSlots, kSets = S::kSets, kWarps = S::kWarps, kThreads = S::kThreads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x % a.ctas);
  const int64_t team = blockIdx.x / a.ctas, teams = gridDim.x / a.ctas;
  const bool together = kStat && a.ctas > 1;  // launched as clusters
  const bool grad = kMode != kLossForward && a.gradient;
  const bool twice = kStat && grad && a.twice;
  // gradients are made in the slots, in the logits' place, and copied from there
  const bool out = kMode == kLossPolicy && sizeof(TZ) == sizeof(TD) && grad && !twice;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], out ? 1 : kWarps);
      mbar_init(&sm.made[i], kWarps);
    }
    for (int i = 0; i < kBoxes; ++i) mbar_init(&sm.told[i], together ? 1 : kWarps);
    for (int i = 0; i < kSets; ++i) mbar_init(&sm.ready[i], 1);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  for (int k = threadIdx.x * 16; k < S::kZeros; k += blockDim.x * 16)
    *reinterpret_cast<uint4*>(ring + kSlots * kLossChunk + k) = make_uint4(0, 0, 0, 0);
  if (S::kZeros) fence_proxy_async_shared();
  int64_t row0 = 0, rows = a.rows;
  if (kMode == kLossForward && a.offsets) let_next_start();  // (the pairs' kernel, which waits for this one)
  if (kMode == kLossBackward && a.offsets) wait_for_previous();
  if (a.offsets) {
    // (every CTA sees the same offsets: all of them leave)
    const bool fine = kStat ? offsets_fine(a.offsets, 2 * a.pairs + 1, a.rows, a.ctrl) : *a.fine != 0;
    if (kStat && blockIdx.x == 0 && threadIdx.x == 0) *a.fine = fine;
    if (!fine) return;
    row0 = a.offsets[0];
    rows = a.offsets[2 * a.pairs] - row0;
  }
  // this CTA's groups, and how many chunks they are
  const int g_lo = static_cast<int>(static_cast<int64_t>(a.groups[a.P]) * rank / a.ctas);
  const int g_hi = static_cast<int>(static_cast<int64_t>(a.groups[a.P]) * (rank + 1) / a.ctas);
  const int chunks = (g_hi - g_lo + kChunkGroups - 1) / kChunkGroups;
  // the team's rows: team, team + teams, .. from the first row on, or from the last one back
  const int mine = rows > team ? static_cast<int>((rows - team + teams - 1) / teams) : 0;
  const int64_t stride = a.backwards ? -teams : teams;
  int64_t i = row0 + (a.backwards ? rows - 1 - team : team);
  auto fetch = [&](int n) {  // this lane's row of the batch that starts at the team's row n
    RowIn r = {-1, false};
    if (n + lane < mine) {
      const int64_t k = i + lane * stride;
      r.y = a.targets[k];
      r.on = r.y >= 0 && r.y < a.first[a.P] && (!a.weights || a.weights[k] != 0.f);
    }
    return r;
  };
  const RowIn first = fetch(0);  // (asked for in front of the barrier)
  if (together) cluster_sync_all(); else __syncthreads();

  if (warp == kSets * kWarps) {
    // the copies, in the order in which the chunks are used: of each row for its statistics, and (twice)
    // again for its gradient
    RowIn r = {-1, false};
    uint32_t count = 0;
    bool fine = true;
    auto copy_row = [&](int64_t row) {
      int rk = 0;
      for (int c = 0; c < chunks && fine; ++c, ++count) {
        const uint32_t slot = count % kSlots, turn = count / kSlots;
        if (turn > 0 && !wait_full(&sm.empty[slot], (turn - 1) & 1, a)) {
          fine = false;
          break;
        }
        if (lane == 0) {
          int g = g_lo + c * kChunkGroups;
          const int end = g + kChunkGroups < g_hi ? g + kChunkGroups : g_hi;
          uint8_t* dst = ring + slot * kLossChunk;
          mbar_arrive_expect_tx(&sm.full[slot], static_cast<uint32_t>(end - g) * 16u);
          while (g < end) {
            while (g >= a.groups[rk + 1]) ++rk;
            const int stop = end < a.groups[rk + 1] ? end : a.groups[rk + 1];
            const uint8_t* src = static_cast<const uint8_t*>(a.z[rk]) + row * a.ldz[rk] * sizeof(TZ) +
                                 static_cast<int64_t>(g - a.groups[rk]) * 16;
            bulk_load(dst, src, static_cast<uint32_t>(stop - g) * 16u, &sm.full[slot]);
            dst += (stop - g) * 16;
            g = stop;
          }
        }
        __syncwarp();
      }
    };
    for (int n = 0; n < mine && fine; ++n, i += stride) {
      if ((n & 31) == 0) r = n ? fetch(n) : first;
      if (!__shfl_sync(0xffffffffu, r.on, n & 31)) continue;
      copy_row(i);
      if (twice) copy_row(i);
    }
    if (!fine && lane == 0) raise_error(a.ctrl, FO_ERR_TIMEOUT, kSiteEmpty, blockIdx.x);
    // no copy may be in flight behind a CTA whose computing warps gave up
    for (uint32_t k = count > kSlots ? count - kSlots : 0; k < count; ++k)
      mbar_wait_drain(&sm.full[k % kSlots], (k / kSlots) & 1, kLossDrainNs);
  } else if (warp > kSets * kWarps) {
    // the copies of the gradients, in the order in which they are made; rows that do not count are
    // copies of zeros
    RowIn r = {-1, false};
    P place;
    bool fine = true;
    for (int n = 0; n < mine && out && fine; ++n, i += stride) {
      if ((n & 31) == 0) r = n ? fetch(n) : first;
      const bool on = __shfl_sync(0xffffffffu, r.on, n & 31);
      int rk = 0;
      for (int g = g_lo; g < g_hi && fine;) {
        const int left = g_hi - g, end = g + (left < kChunkGroups ? left : kChunkGroups);
        if (on && !wait_full(&sm.made[place.slot], place.turn, a)) {
          fine = false;
          break;
        }
        if (lane == 0) {
          const uint8_t* src = ring + (on ? place.slot * kLossChunk : kSlots * kLossChunk);
          while (g < end) {
            while (g >= a.groups[rk + 1]) ++rk;
            int stop = end < a.groups[rk + 1] ? end : a.groups[rk + 1];
            if (!on && stop > g + S::kZeros / 16) stop = g + S::kZeros / 16;
            bulk_store(static_cast<uint8_t*>(a.d[rk]) +
                           (i * a.ldd[rk] * sizeof(TD) + static_cast<int64_t>(g - a.groups[rk]) * 16),
                       src, static_cast<uint32_t>(stop - g) * 16u);
            if (on) src += (stop - g) * 16;
            g = stop;
          }
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          if (on) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            mbar_arrive(&sm.empty[place.slot]);
          }
        }
        __syncwarp();
        g = end;
        if (on) place.next();
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!fine && lane == 0) raise_error(a.ctrl, FO_ERR_TIMEOUT, kSiteDrain, blockIdx.x);
  } else {
    const float c = static_cast<float>(a.scale * kLog2e);
    const float slack = kOctaves / c;
    float per_weight = 1.f;
    if (kMode == kLossPolicy && a.mean) {
      const float total = total_weight<kSets * kWarps>(a, sm.buf);
      per_weight = total == 0.f ? 0.f : 1.f / total;
    }
    const int set = kSets > 1 ? warp / kWarps : 0, tid = kSets > 1 ? threadIdx.x % kThreads : threadIdx.x;
    // columns behind a rank's last whole group: one each for the first threads of a row's first CTA
    const int t_rk = tid >> 3;
    int t_col = -1;
    if (rank == 0 && t_rk < a.P) {
      const int ragged = a.cols[t_rk] % kCols;
      if ((tid & 7) < ragged) t_col = a.cols[t_rk] - ragged + (tid & 7);
    }
    double sums[4] = {0.0, 0.0, 0.0, 0.0};  // stats of the rows that this warp finished (lane 0)
    RowIn r = {-1, false};
    int y_rk = 0, y_col = 0, y_group = -1;               // this lane's row: where the target is
    float z_y = 0.f;
    float in0 = 0.f, in1 = 0.f, in2 = 0.f, in3 = 0.f;    // what else goes with it (backward: its Slope)
    uint32_t count = 0;                                  // rows that counted so far
    P place;
    bool fine = true;
    for (int n = 0; n < mine; ++n, i += stride) {
      const int at = n & 31;
      if (at == 0) {
        r = n ? fetch(n) : first;
        const int64_t k = i + lane * stride;
        if (warp == 0 && rank == 0 && n + lane < mine && !r.on) {
          if (r.y >= a.first[a.P]) note_error(a.ctrl, FO_ERR_RANGE, kSiteTargets, static_cast<uint32_t>(k));
          if (a.logp) a.logp[k] = 0.f;
          if (a.lse) a.lse[k] = 0.f;
          if (a.entropy) a.entropy[k] = 0.f;
          if (kStat && a.stat) a.stat[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (r.on) {
          y_rk = 0;
          while (r.y >= a.first[y_rk + 1]) ++y_rk;
          y_col = r.y - a.first[y_rk];
          // (read now: no CTA writes a gradient over a row before every warp has told its part of it)
          z_y = load1(static_cast<const TZ*>(a.z[y_rk]) + k * a.ldz[y_rk] + y_col);
          const int whole = a.groups[y_rk + 1] - a.groups[y_rk];
          y_group = y_col / kCols < whole ? a.groups[y_rk] + y_col / kCols : -1;
        }
        if (kMode == kLossPolicy && r.on) {
          in0 = a.weights ? a.weights[k] : 1.f;
          in1 = a.advantages[k];
          if (a.old_logp) in2 = a.old_logp[k];
          if (a.ref_logp) in3 = a.ref_logp[k];
        }
        if (kMode == kLossBackward && r.on) {
          float da, dh = 0.f, log_s = 0.f, entropy = 0.f;
          if (a.coef) {
            int lo = 0, hi = 2 * a.pairs - 1;  // the sequence: the last one that starts at or in front of row k
            while (lo < hi) {
              const int mid = (lo + hi + 1) >> 1;
              if (a.offsets[mid] <= k) lo = mid; else hi = mid - 1;
            }
            da = a.coef[lo];
            const float4 st = a.stat[k];
            in0 = st.x;
            log_s = st.y;
          } else {
            da = a.dlogp[k];
            if (kEnt) {
              dh = a.dentropy[k];
              entropy = a.in_entropy[k];
            }
            in0 = a.in_lse[k] / a.scale;
          }
          in1 = -a.scale * exp2f(-log_s) * (kEnt ? fmaf(dh, entropy, da) : da);
          in2 = -a.scale * dh * kLn2;
          in3 = a.scale * da;
        }
      }
      if (!__shfl_sync(0xffffffffu, r.on, at)) {
        if (grad && n % kSets == set) {
          const Pair zero[kPairs] = {};
          int rk = 0;
          for (int g = g_lo + tid; g < g_hi && !out; g += kThreads) {
            while (g >= a.groups[rk + 1]) ++rk;
            store_group<kPairs>(
                static_cast<TD*>(a.d[rk]) + i * a.ldd[rk] + static_cast<int64_t>(g - a.groups[rk]) * kCols, zero);
          }
          if (t_col >= 0) store1(static_cast<TD*>(a.d[t_rk]) + i * a.ldd[t_rk] + t_col, 0.f);
        }
        continue;
      }
      const uint32_t q = count++;
      if (kSets > 1 && q % kSets != static_cast<uint32_t>(set)) {
        place.skip(twice ? 2 * chunks : chunks);
        continue;
      }
      const int col_y = __shfl_sync(0xffffffffu, y_col, at), rk_y = __shfl_sync(0xffffffffu, y_rk, at);
      const int group_y = __shfl_sync(0xffffffffu, y_group, at) - g_lo;
      const float zy = __shfl_sync(0xffffffffu, z_y, at);
      const float z_t = t_col >= 0 ? load1(static_cast<const TZ*>(a.z[t_rk]) + i * a.ldz[t_rk] + t_col) : -INFINITY;
      const P start = place;
      float4 w;  // the row's Slope, and what its target's column has more

      if (kStat) {
        Sums some = {-INFINITY, 0, 0};
        for (int k = 0; k < chunks; ++k, place.next()) {
          if (!wait_full(&sm.full[place.slot], place.turn, a)) {
            fine = false;
            break;
          }
          const int left = g_hi - g_lo - k * kChunkGroups;
          const uint4* src = reinterpret_cast<const uint4*>(ring + place.slot * kLossChunk) + tid;
          if (left >= kChunkGroups) {
            add_groups<TZ, kStatEnt, S::kBatch, kThreads>(src, c, slack, some);
          } else {
            for (int g = tid; g < left; g += kThreads)
              add_groups<TZ, kStatEnt, 1, 1>(src + (g - tid), c, slack, some);
          }
          if (!grad || twice) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[place.slot]);
          }
        }
        if (!fine) break;
        Part v = {some.m, sum2(some.s), sum2(some.t), 0.f};
        if (t_col >= 0) v = merge<kStatEnt>(v, Part{z_t, fast_exp2((z_t - base_of(z_t)) * c), 0.f, 0.f}, c);
        v = join<kStatEnt>(v, c);
        // the warp's part to every CTA of the row.  A box is free again when the row kBoxes - kSets back
        // has been told by all: the warps that added the row kBoxes back told that one afterwards
        const uint32_t box = q % kBoxes, back = q - (kBoxes - kSets);
        if (q >= kBoxes - kSets && !wait_told(&sm.told[back % kBoxes], (back / kBoxes) & 1, a)) {
          fine = false;
          break;
        }
        if (!together) {
          if (lane == 0) {
            sm.part[box][warp % kWarps] = v;
            mbar_arrive(&sm.told[box]);
          }
        } else if (lane < a.ctas) {
          if (warp % kWarps == 0 && lane == 0)
            mbar_arrive_expect_tx(&sm.told[box], static_cast<uint32_t>(a.ctas * kWarps * sizeof(Part)));
          const uint32_t to = map_to_cta(smem_u32(&sm.part[box][rank * kWarps + warp % kWarps]), lane);
          // (a store that counts at the barrier by itself: an arrival with release would wait for the
          // gradients under way to memory)
          asm volatile(
              "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
              "r"(__float_as_uint(v.m)), "r"(__float_as_uint(v.s)), "r"(__float_as_uint(v.t)), "r"(0),
              "r"(map_to_cta(smem_u32(&sm.told[box]), lane))
              : "memory");
        }
        __syncwarp();
        // one warp of each CTA adds the row's parts
        if (static_cast<int>(q / kSets % kWarps) == warp % kWarps) {
          if (!wait_told(&sm.told[box], (q / kBoxes) & 1, a)) {
            fine = false;
            break;
          }
          v = Part{-INFINITY, 0.f, 0.f, 0.f};
          for (int k = lane; k < a.ctas * kWarps; k += 32) v = merge<kStatEnt>(v, sm.part[box][k], c);
          v = join<kStatEnt>(v, c);
          // p_j = 2^((z_j - base) c - log_s)
          const float base = base_of(v.m), log_s = log2f(v.s), dz = zy - base, dy = a.scale * dz;
          const Wide total = plus(wide_log(v.s), wide(kExpMean - __fdividef(kExpMean, v.s)));
          const Wide wide_lp = plus(Wide{dy, fmaf(a.scale, dz, -dy)}, Wide{-total.hi, -total.lo});
          const float lp = wide_lp.hi;
          const float entropy = kStatEnt ? kLn2 * (log_s - v.t / v.s) : 0.f;
          if (rank == 0 && lane == 0) {
            if (a.logp) a.logp[i] = lp;
            if (a.lse) a.lse[i] = fmaf(base, a.scale, total.hi) + total.lo;
            if (kMode == kLossForward && a.entropy) a.entropy[i] = entropy;
            if (a.stat) a.stat[i] = make_float4(base, log_s, wide_lp.hi, wide_lp.lo);
          }
          if (kMode == kLossPolicy) {
            // the loss through this row: da = dL/dlogp, dh = dL/dH
            const float weight = __shfl_sync(0xffffffffu, in0, at) * per_weight;
            const float adv = __shfl_sync(0xffffffffu, in1, at);
            const float old = __shfl_sync(0xffffffffu, in2, at), ref = __shfl_sync(0xffffffffu, in3, at);
            const float ratio = expf(a.old_logp ? lp - old : 0.f);
            const float held = fminf(fmaxf(ratio, a.ratio_lo), a.ratio_hi) * adv;
            // (a ratio may leave fp32: without an advantage it counts nothing all the same)
            const float free = adv == 0.f && ratio == INFINITY ? 0.f : ratio * adv;
            const bool clipped = held < free;
            float kl = 0.f, dkl = 0.f;
            if (a.ref_logp) {
              const float x = ref - lp;
              dkl = expm1f(x);
              kl = dkl - x;
              if (rank == 0) sums[1] += static_cast<double>(weight) * kl;
              if (a.kl_coef == 0.f) kl = dkl = 0.f;  // (a statistic alone: it may be infinite)
            }
            const float da = weight * ((clipped ? 0.f : -free) - a.kl_coef * dkl), dh = -a.entropy_coef * weight;
            if (rank == 0) {
              const float loss = -(clipped ? held : free) + a.kl_coef * kl - a.entropy_coef * entropy;
              sums[0] += static_cast<double>(weight) * loss;
              if (clipped) sums[2] += weight;
              sums[3] += static_cast<double>(weight) * entropy;
            }
            if (grad && lane == 0) {
              const float inv = -a.scale * exp2f(-log_s);
              const float k0 = inv * (kEnt ? da + dh * (entropy - kLn2 * log_s) : da);
              sm.slope[set] = make_float4(base, k0, inv * dh * kLn2, a.scale * da);
              mbar_arrive(&sm.ready[set]);
            }
          }
        }
        if (kMode == kLossForward || !grad) continue;
        if (!wait_full(&sm.ready[set], (q / kSets) & 1, a)) {
          fine = false;
          break;
        }
        w = sm.slope[set];
      } else {
        w.x = __shfl_sync(0xffffffffu, in0, at);
        w.y = __shfl_sync(0xffffffffu, in1, at);
        w.z = kEnt ? __shfl_sync(0xffffffffu, in2, at) : 0.f;
        w.w = __shfl_sync(0xffffffffu, in3, at);
      }

      // the gradient: dz_j = own 1[j = y] + 2^d (k0 + k1 d) with d = (z_j - base) c
      const Slope slope = {w.x, c, w.y, w.z};
      const bool kept = kStat && !twice;  // the chunks have waited in their slots
      if (kept) place = start;
      int rk = 0;
      for (int k = 0; k < chunks; ++k, place.next()) {
        if (!kept && !wait_full(&sm.full[place.slot], place.turn, a)) {
          fine = false;
          break;
        }
        const int g0 = g_lo + k * kChunkGroups, left = g_hi - g0;
        uint4* src = reinterpret_cast<uint4*>(ring + place.slot * kLossChunk) + tid;
        if (kMode == kLossPolicy && sizeof(TZ) == sizeof(TD) && out) {
          if (left >= kChunkGroups) {
            uint4 x[S::kBatch];
#pragma unroll
            for (int j = 0; j < S::kBatch; ++j) x[j] = src[j * kThreads];
#pragma unroll
            for (int j = 0; j < S::kBatch; ++j)
              put_group<TZ, TD, kEnt>(x[j], slope, reinterpret_cast<TD*>(src + j * kThreads));
          } else {
            for (int g = tid; g < left; g += kThreads)
              put_group<TZ, TD, kEnt>(src[g - tid], slope, reinterpret_cast<TD*>(src + (g - tid)));
          }
          const int at_y = group_y - k * kChunkGroups;
          if (at_y >= 0 && at_y < left && at_y < kChunkGroups && at_y % kThreads == tid)
            store1(reinterpret_cast<TD*>(src + (at_y - tid)) + col_y % kCols, slope_at<kEnt>(slope, zy) + w.w);
          fence_proxy_async_shared();
        } else {
          while (g0 >= a.groups[rk + 1]) ++rk;
          if (left >= kChunkGroups && g0 + kChunkGroups <= a.groups[rk + 1]) {
            TD* to = static_cast<TD*>(a.d[rk]) + i * a.ldd[rk] +
                     static_cast<int64_t>(g0 + tid - a.groups[rk]) * kCols;
            uint4 x[S::kBatch];  // (all read first: a store might be to what is read next)
#pragma unroll
            for (int j = 0; j < S::kBatch; ++j) x[j] = src[j * kThreads];
#pragma unroll
            for (int j = 0; j < S::kBatch; ++j) put_group<TZ, TD, kEnt>(x[j], slope, to + j * kThreads * kCols);
          } else {
            int r2 = rk;
            for (int g = tid; g < left && g < kChunkGroups; g += kThreads) {
              while (g0 + g >= a.groups[r2 + 1]) ++r2;
              put_group<TZ, TD, kEnt>(src[g - tid], slope,
                                      static_cast<TD*>(a.d[r2]) + i * a.ldd[r2] +
                                          static_cast<int64_t>(g0 + g - a.groups[r2]) * kCols);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(out ? &sm.made[place.slot] : &sm.empty[place.slot]);
      }
      if (!fine) break;
      // the columns behind the groups, and the target's column again by the thread that has just written it
      if (t_col >= 0)
        store1(static_cast<TD*>(a.d[t_rk]) + i * a.ldd[t_rk] + t_col,
               slope_at<kEnt>(slope, z_t) + (t_rk == rk_y && t_col == col_y ? w.w : 0.f));
      if (!out && group_y >= 0 && group_y < g_hi - g_lo && group_y % kChunkGroups % kThreads == tid)
        store1(static_cast<TD*>(a.d[rk_y]) + i * a.ldd[rk_y] + col_y, slope_at<kEnt>(slope, zy) + w.w);
    }
    if (!fine && lane == 0) {
      raise_error(a.ctrl, FO_ERR_TIMEOUT, kSiteFull, blockIdx.x);
      sums[0] = static_cast<double>(NAN);
    }
    if (kMode == kLossPolicy && rank == 0) {
      if (lane == 0)
        for (int k = 0; k < 4; ++k) sm.sums[warp][k] = sums[k];
      asm volatile("bar.sync 1, %0;" ::"n"(S::kAll) : "memory");
      if (warp == 0) {
        // eight lanes for each of the four values; the team that comes last adds everyone's sums, in
        // the order of the teams.  A team whose waits ran out counts as well (or the next launch that counts on
        // this context would take another CTA for its last); its loss is NaN
        const int k = lane >> 3;
        double s = 0.0;
        for (int q = lane & 7; q < kSets * kWarps; q += 8) s += sm.sums[q][k];
        s = eighth_sum(s);
        int last = 0;
        if ((lane & 7) == 0) {
          a.part[team * 4 + k] = s;
          __threadfence();
        }
        __syncwarp();
        if (lane == 0)
          last = atomicInc(a.ctrl + kCtrlDone, static_cast<unsigned>(teams - 1)) == static_cast<unsigned>(teams - 1);
        if (__shfl_sync(0xffffffffu, last, 0)) {
          __threadfence();
          s = 0.0;
          for (int64_t b = lane & 7; b < teams; b += 8) s += __ldcg(a.part + b * 4 + k);
          s = eighth_sum(s);
          if ((lane & 7) == 0) a.stats[k] = static_cast<float>(s);
        }
      }
    }
  }
  __syncwarp();
  if (together) cluster_sync_all();  // no CTA leaves while another may still store into it
}

template <typename TZ, typename TD>
void (*kernel_of(const LossKind& k))(LossArgs) {
  if (k.mode == kLossPolicy)
    return k.entropy ? loss_rows_kernel<TZ, TD, kLossPolicy, true> : loss_rows_kernel<TZ, TD, kLossPolicy, false>;
  if (k.mode == kLossBackward)
    return k.entropy ? loss_rows_kernel<TZ, TD, kLossBackward, true> : loss_rows_kernel<TZ, TD, kLossBackward, false>;
  // writes no gradient: one type of it is enough
  return k.entropy ? loss_rows_kernel<TZ, uint16_t, kLossForward, true>
                   : loss_rows_kernel<TZ, uint16_t, kLossForward, false>;
}

// Teams of `ctas` CTAs of one cluster that the current device holds at once: which SMs may share a cluster differs
// from chip to chip.  0: none.  (All kernels of a mode have one shape.)
template <int kMode>
int clusters(int ctas) {
  typedef Shape<kMode> S;
  const auto kernel = loss_rows_kernel<uint16_t, uint16_t, kMode, true>;
  constexpr int smem = S::kSlots * kLossChunk + S::kZeros;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -1;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(S::kAll + 32 * S::kMore);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : -1;
}
// The same, asked once per device and mode (what host threads share is atomic)
int clusters_of(int device, bool one, int size) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][2][kLossSizes];  // the answer and 1
  const bool keep = device >= 0 && device < kDevices;
  if (keep)
    if (const int n = known[device][one][size].load(std::memory_order_relaxed)) return n - 1;
  const int n = one ? clusters<kLossPolicy>(1 << size) : clusters<kLossForward>(1 << size);
  if (n < 0) {
    cudaGetLastError();
    return 0;
  }
  if (keep) known[device][one][size].store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace

int loss_rows_parts(int num_sms) { return num_sms; }

cudaError_t loss_rows_launch(LossArgs a, const LossKind& k, int device, int num_sms, cudaStream_t s) {
  const bool one = k.mode == kLossPolicy;
  const int threads = one ? Shape<kLossPolicy>::kAll : Shape<kLossForward>::kAll;
  const int smem = one ? Shape<kLossPolicy>::kSlots * kLossChunk + Shape<kLossPolicy>::kZeros
                       : Shape<kLossForward>::kSlots * kLossChunk;
  const int cols = k.z32 ? Group<float>::kCols : Group<uint16_t>::kCols;
  for (int r = 0; r < a.P; ++r) a.groups[r + 1] = a.groups[r] + a.cols[r] / cols;
  LossShape shape;
  shape.rows = a.rows;
  shape.groups = a.groups[a.P];
  shape.chunk_groups = kChunkGroups;
  shape.threads = threads;
  shape.waits = one;
  shape.slots = Shape<kLossPolicy>::kSlots;
  shape.fit = kLossFit;
  shape.reads_alone = k.mode == kLossForward;
  shape.exchange = k.mode != kLossBackward;
  shape.places = num_sms * (one ? Shape<kLossPolicy>::kPerSm : Shape<kLossForward>::kPerSm);
  for (int i = 0; i < kLossSizes; ++i) {
    const int most = shape.places >> i;
    const int n = i > 0 && shape.exchange ? clusters_of(device, one, i) : most;
    shape.teams[i] = n < most ? n : most;
  }
  const LossCut cut = loss_cut(shape);
  a.ctas = cut.ctas;
  a.twice = cut.twice && a.gradient;
  void (*kernel)(LossArgs) = k.z32 ? (k.d32 ? kernel_of<float, float>(k) : kernel_of<float, uint16_t>(k))
                                   : (k.d32 ? kernel_of<uint16_t, float>(k) : kernel_of<uint16_t, uint16_t>(k));
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(cut.teams * a.ctas));
  cfg.blockDim = dim3(threads + 32 * (one ? Shape<kLossPolicy>::kMore : Shape<kLossForward>::kMore));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (k.mode != kLossBackward && a.ctas > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = a.ctas;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (k.early) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fo

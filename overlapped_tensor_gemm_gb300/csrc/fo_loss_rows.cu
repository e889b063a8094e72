// Row kernels of the losses (formulas in fo_loss.cuh).
//
// Bound by HBM: the logits are read once (the gradient of a policy loss waits for its row's sum, and
// the row waits in shared memory), the gradients written once.  A row belongs to a cluster of 1 to 8
// CTAs, each with a range of its columns that fits shared memory beside the copies under way for the
// next rows.  One warp orders the copies (cp.async.bulk, 32 KB each, into a ring of slots); sixteen
// warps walk a row's slots twice: for the row's statistics, then for its gradient, after which a slot
// takes a chunk of a later row.  Between the walks every warp tells every CTA of the row its part of
// the statistics (stores into their shared memory and an arrival at their barrier): one exchange a
// row, over which the copies go on.
//
// A thread sums relative to a column of its own that is near its maximum (at most 16 octaves below),
// so that a new maximum does not cost a pass; log2 domain, two columns per instruction.
#include <cfloat>
#include <cstring>

#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr double kLog2e = 1.4426950408889634;
constexpr float kOctaves = 16.f;  // a sum's reference may lie so far below its maximum
// 2^d is 0 in fp32 from here on down: where d multiplies it, d ends here (0 times -infinity)
constexpr float kFarBelow = -160.f;
constexpr int kChunkGroups = kLossChunk / 16;
constexpr int kLossFit = 4;  // a row's chunks in one CTA, where more CTAs can share it
constexpr int kBatch = kChunkGroups / (32 * kLossWarps);  // groups of a chunk per thread
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
  static __device__ __forceinline__ void pairs(const uint4& q, Pair (&v)[4]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
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
  static __device__ __forceinline__ void pairs(const uint4& q, Pair (&v)[2]) {
    v[0] = pack2(__uint_as_float(q.x), __uint_as_float(q.y));
    v[1] = pack2(__uint_as_float(q.z), __uint_as_float(q.w));
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

// What is subtracted for a reference m: finite also where every column is -infinity
__device__ __forceinline__ float base_of(float m) { return fmaxf(m, -FLT_MAX); }

// A part of a row's statistics: reference m, s = sum 2^d, t = sum 2^d d with d = (z - m) c
struct Part {
  float m, s, t, z_y;  // z_y: the target's logit (0 in the parts that do not have it)
};

// The parts of all lanes as one, in every lane
template <bool kEnt>
__device__ __forceinline__ Part join(Part v, float c) {
  const float m = warp_max(v.m), d = (base_of(v.m) - base_of(m)) * c;
  // (parts without a finite column have s = 0, whatever their factor)
  const float f = fast_exp2(d);
  Part r;
  r.m = m;
  if (kEnt) r.t = warp_sum(f * fmaf(v.s, fmaxf(d, kFarBelow), v.t));
  r.s = warp_sum(f * v.s);
  r.z_y = warp_sum(v.z_y);
  return r;
}
template <bool kEnt>
__device__ __forceinline__ Part merge(const Part& v, const Part& w, float c) {
  Part r;
  r.m = fmaxf(v.m, w.m);
  const float dv = (base_of(v.m) - base_of(r.m)) * c, dw = (base_of(w.m) - base_of(r.m)) * c;
  const float fv = fast_exp2(dv), fw = fast_exp2(dw);
  if (kEnt) r.t = fv * fmaf(v.s, fmaxf(dv, kFarBelow), v.t) + fw * fmaf(w.s, fmaxf(dw, kFarBelow), w.t);
  r.s = fv * v.s + fw * w.s;
  r.z_y = v.z_y + w.z_y;
  return r;
}

// A thread's sums over a row: s and t relative to m, two columns side by side
struct Sums {
  float m;
  Pair s, t;
};
// n groups into the sums
template <typename TZ, bool kEnt, int n>
__device__ __forceinline__ void add_groups(const uint4 (&q)[n], float c, float slack, Sums& v) {
  constexpr int kPairs = Group<TZ>::kCols / 2;
  const float top = Group<TZ>::top(q);
  if (top > v.m + slack) {
    const float d = (base_of(v.m) - base_of(top)) * c;
    const Pair f = both(fast_exp2(d));
    if (kEnt) v.t = mul2(f, ffma2(v.s, both(fmaxf(d, kFarBelow)), v.t));
    v.s = mul2(f, v.s);
    v.m = top;
  }
  const Pair base = both(-base_of(v.m)), c2 = both(c);
#pragma unroll
  for (int k = 0; k < n; ++k) {
    Pair x[kPairs];
    Group<TZ>::pairs(q[k], x);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      float lo, hi;
      unpack2(mul2(fadd2(x[e], base), c2), lo, hi);
      const Pair w = pack2(fast_exp2(lo), fast_exp2(hi));
      v.s = fadd2(v.s, w);
      if (kEnt) v.t = ffma2(w, pack2(fmaxf(lo, kFarBelow), fmaxf(hi, kFarBelow)), v.t);
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
  const Pair nbase = both(-g.base), c2 = both(g.c), k0 = both(g.k0), k1 = both(g.k1);
  Pair x[kPairs];
  Group<TZ>::pairs(q, x);
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    float lo, hi;
    unpack2(mul2(fadd2(x[e], nbase), c2), lo, hi);
    const Pair w = pack2(fast_exp2(lo), fast_exp2(hi));
    x[e] = kEnt ? mul2(w, ffma2(pack2(fmaxf(lo, kFarBelow), fmaxf(hi, kFarBelow)), k1, k0)) : mul2(w, k0);
  }
  store_group<kPairs>(to, x);
}

// A place in the ring that advances chunk by chunk
struct Place {
  uint32_t slot = 0, turn = 0;  // turn: parity of the slot's use
  __device__ __forceinline__ void next() {
    if (++slot == kLossSlots) {
      slot = 0;
      turn ^= 1;
    }
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
__device__ __forceinline__ float total_weight(const LossArgs& a, float* buf) {
  float sum = 0.f, low = 0.f;
  for (int64_t i = threadIdx.x; i < a.rows; i += 32 * kLossWarps) {
    const int32_t y = a.targets[i];
    if (y < 0 || y >= a.first[a.P]) continue;
    const float x = (a.weights ? a.weights[i] : 1.f) - low, next = sum + x;
    low = (next - sum) - x;
    sum = next;
  }
  sum = warp_sum(sum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[warp] = sum;
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kLossWarps) : "memory");
  return warp_sum(lane < kLossWarps ? buf[lane] : 0.f);
}

struct Smem {
  uint64_t full[kLossSlots], empty[kLossSlots], told[2];
  Part part[2][kLossMaxCtas * kLossWarps];
  float buf[kLossWarps];
};

// A lane's row of a batch of 32
struct RowIn {
  int32_t y;
  bool on;
};

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
__global__ void __launch_bounds__(kLossThreads, 1) loss_rows_kernel(const __grid_constant__ LossArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ Smem sm;
  constexpr bool kStat = kMode != kLossBackward;
  constexpr bool kStatEnt = kMode == kLossPolicy || (kMode == kLossForward && kEnt);
  constexpr int kCols = Group<TZ>::kCols, kPairs = kCols / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int rank = static_cast<int>(blockIdx.x % a.ctas);
  const int64_t team = blockIdx.x / a.ctas, teams = gridDim.x / a.ctas;
  const bool together = kStat && a.ctas > 1;  // launched as clusters
  if (tid == 0) {
    for (int i = 0; i < kLossSlots; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kLossWarps);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&sm.told[i], a.ctas * kLossWarps);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  int64_t row0 = 0, rows = a.rows;
  if (a.offsets) {
    // (every CTA sees the same offsets: all of them leave)
    if (!offsets_fine(a.offsets, 2 * a.pairs + 1, a.rows, a.ctrl)) return;
    row0 = a.offsets[0];
    rows = a.offsets[2 * a.pairs] - row0;
  }
  if (together) cluster_sync_all(); else __syncthreads();

  // this CTA's groups, and how many chunks they are
  const int g_lo = static_cast<int>(static_cast<int64_t>(a.groups[a.P]) * rank / a.ctas);
  const int g_hi = static_cast<int>(static_cast<int64_t>(a.groups[a.P]) * (rank + 1) / a.ctas);
  const int chunks = (g_hi - g_lo + kChunkGroups - 1) / kChunkGroups;
  const bool grad = kMode != kLossForward && a.d[0];
  const bool twice = kStat && grad && a.twice;
  const int64_t mine = rows > team ? (rows - team + teams - 1) / teams : 0;  // the team's rows: team, team + teams, ..
  auto row_at = [&](int64_t n) {
    const int64_t k = team + n * teams;
    return row0 + (a.backwards ? rows - 1 - k : k);
  };
  auto fetch = [&](int64_t n) {  // this lane's row of the batch that starts at n
    RowIn r = {-1, false};
    if (n + lane < mine) {
      const int64_t i = row_at(n + lane);
      r.y = a.targets[i];
      r.on = r.y >= 0 && r.y < a.first[a.P] && (!a.weights || a.weights[i] != 0.f);
    }
    return r;
  };

  if (warp == kLossWarps) {
    // the copies, in the order in which the chunks are used
    RowIn r = {-1, false};
    uint32_t count = 0;
    bool fine = true;
    for (int64_t n = 0; n < mine && fine; ++n) {
      if ((n & 31) == 0) r = fetch(n);
      if (!__shfl_sync(0xffffffffu, r.on, n & 31)) continue;
      const int64_t i = row_at(n);
      for (int pass = 0; pass < (twice ? 2 : 1) && fine; ++pass) {
        int rk = 0;
        for (int c = 0; c < chunks; ++c, ++count) {
          const uint32_t slot = count % kLossSlots, turn = count / kLossSlots;
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
              const uint8_t* src = static_cast<const uint8_t*>(a.z[rk]) + i * a.ldz[rk] * sizeof(TZ) +
                                   static_cast<int64_t>(g - a.groups[rk]) * 16;
              bulk_load(dst, src, static_cast<uint32_t>(stop - g) * 16u, &sm.full[slot]);
              dst += (stop - g) * 16;
              g = stop;
            }
          }
          __syncwarp();
        }
      }
    }
    if (!fine && lane == 0) raise_error(a.ctrl, FO_ERR_TIMEOUT, kSiteEmpty, blockIdx.x);
    // no copy may be in flight behind a CTA whose computing warps gave up
    for (uint32_t k = count > kLossSlots ? count - kLossSlots : 0; k < count; ++k)
      mbar_wait_drain(&sm.full[k % kLossSlots], (k / kLossSlots) & 1, kLossDrainNs);
  } else {
    const float c = static_cast<float>(a.scale * kLog2e);
    const float slack = kOctaves / c;
    float per_weight = 1.f;
    if (kMode == kLossPolicy && a.mean) {
      const float total = total_weight(a, sm.buf);
      per_weight = total == 0.f ? 0.f : 1.f / total;
    }
    // columns behind a rank's last whole group: one each for the first threads of a row's first CTA
    const int t_rk = tid >> 3;
    int t_col = -1;
    if (rank == 0 && t_rk < a.P) {
      const int ragged = a.cols[t_rk] % kCols;
      if ((tid & 7) < ragged) t_col = a.cols[t_rk] - ragged + (tid & 7);
    }
    double sums[4] = {0.0, 0.0, 0.0, 0.0};  // thread 0 of a row's first CTA: stats
    RowIn r = {-1, false};
    float in0 = 0.f, in1 = 0.f, in2 = 0.f, in3 = 0.f;
    uint32_t told = 0;
    Place place;
    bool fine = true;
    for (int64_t n = 0; n < mine; ++n) {
      const int64_t i = row_at(n);
      const int at = static_cast<int>(n & 31);
      if (at == 0) {
        r = fetch(n);
        const int64_t k = n + lane < mine ? row_at(n + lane) : 0;
        if (kStat && warp == 0 && rank == 0 && n + lane < mine && !r.on) {
          if (r.y >= a.first[a.P]) note_error(a.ctrl, FO_ERR_RANGE, kSiteTargets, static_cast<uint32_t>(k));
          if (a.logp) a.logp[k] = 0.f;
          if (a.lse) a.lse[k] = 0.f;
          if (a.entropy) a.entropy[k] = 0.f;
          if (a.stat) a.stat[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (kMode == kLossPolicy && r.on) {
          in0 = a.weights ? a.weights[k] : 1.f;
          in1 = a.advantages[k];
          if (a.old_logp) in2 = a.old_logp[k];
          if (a.ref_logp) in3 = a.ref_logp[k];
        }
        if (kMode == kLossBackward && r.on) {
          if (a.coef) {
            int lo = 0, hi = 2 * a.pairs - 1;  // the sequence: the last one that starts at or in front of row k
            while (lo < hi) {
              const int mid = (lo + hi + 1) >> 1;
              if (a.offsets[mid] <= k) lo = mid; else hi = mid - 1;
            }
            in0 = a.coef[lo];
            const float4 st = a.stat[k];
            in2 = st.x;
            in3 = st.y;
          } else {
            in0 = a.dlogp[k];
            if (kEnt) in1 = a.dentropy[k];
            in2 = a.in_lse[k] / a.scale;
            in3 = kEnt ? a.in_entropy[k] : 0.f;
          }
        }
      }
      const int32_t y = __shfl_sync(0xffffffffu, r.y, at);
      if (!__shfl_sync(0xffffffffu, r.on, at)) {
        if (grad) {
          const Pair zero[kPairs] = {};
          int rk = 0;
          for (int g = g_lo + tid; g < g_hi; g += 32 * kLossWarps) {
            while (g >= a.groups[rk + 1]) ++rk;
            store_group<kPairs>(static_cast<TD*>(a.d[rk]) + i * a.ldd[rk] + static_cast<int64_t>(g - a.groups[rk]) * kCols, zero);
          }
          if (t_col >= 0) store1(static_cast<TD*>(a.d[t_rk]) + i * a.ldd[t_rk] + t_col, 0.f);
        }
        continue;
      }
      // the target's place: a group of this CTA, or a column behind the groups
      int y_rk = 0;
      while (y >= a.first[y_rk + 1]) ++y_rk;
      const int y_col = y - a.first[y_rk];
      const int whole = a.groups[y_rk + 1] - a.groups[y_rk];
      const int y_group = y_col < whole * kCols ? a.groups[y_rk] + y_col / kCols : -1;
      const bool y_here = t_col >= 0 && t_rk == y_rk && t_col == y_col;
      const float z_t = t_col >= 0 ? load1(static_cast<const TZ*>(a.z[t_rk]) + i * a.ldz[t_rk] + t_col) : -INFINITY;

      // first walk: the row's statistics
      Part v;
      const Place start = place;
      if (kStat) {
        v = Part{z_t, t_col >= 0 ? fast_exp2((z_t - base_of(z_t)) * c) : 0.f, 0.f, y_here ? z_t : 0.f};
        Sums sums2 = {-INFINITY, 0, 0};
        for (int k = 0; k < chunks; ++k, place.next()) {
          if (!wait_full(&sm.full[place.slot], place.turn, a)) {
            fine = false;
            break;
          }
          const int g0 = g_lo + k * kChunkGroups, left = g_hi - g0;
          const uint4* src = reinterpret_cast<const uint4*>(ring + place.slot * kLossChunk) + tid;
          if (left >= kChunkGroups) {
            uint4 q[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) q[j] = src[j * 32 * kLossWarps];
            add_groups<TZ, kStatEnt>(q, c, slack, sums2);
          } else {
            for (int g = tid; g < left; g += 32 * kLossWarps) {
              const uint4 q[1] = {src[g - tid]};
              add_groups<TZ, kStatEnt>(q, c, slack, sums2);
            }
          }
          const int at_y = y_group - g0;
          if (at_y >= 0 && at_y < left && at_y < kChunkGroups && at_y % (32 * kLossWarps) == tid)
            v.z_y = load1(reinterpret_cast<const TZ*>(src - tid + at_y) + y_col % kCols);
          if (!grad || twice) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[place.slot]);
          }
        }
        v = merge<kStatEnt>(v, Part{sums2.m, sum2(sums2.s), sum2(sums2.t), 0.f}, c);
        if (!fine) break;
        // every warp's part to every CTA of the row
        v = join<kStatEnt>(v, c);
        Part* const box = sm.part[told & 1];
        uint64_t* const bar = &sm.told[told & 1];
        if (!together) {
          if (lane == 0) {
            box[warp] = v;
            mbar_arrive(bar);
          }
        } else if (lane < a.ctas) {
          const uint32_t to = map_to_cta(smem_u32(box + rank * kLossWarps + warp), lane);
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v.m), "f"(v.s), "f"(v.t),
                       "f"(v.z_y)
                       : "memory");
          mbar_arrive_cluster(map_to_cta(smem_u32(bar), lane));
        }
        if (!wait_told(bar, (told >> 1) & 1, a)) {
          fine = false;
          break;
        }
        ++told;
        v = Part{-INFINITY, 0.f, 0.f, 0.f};
        for (int k = lane; k < (together ? a.ctas : 1) * kLossWarps; k += 32) v = merge<kStatEnt>(v, box[k], c);
        v = join<kStatEnt>(v, c);
      }

      // the row: p_j = 2^((z_j - base) c - log_s)
      float base, log_s, entropy = 0.f, dy = 0.f;
      if (kStat) {
        base = base_of(v.m);
        log_s = log2f(v.s);
        dy = (v.z_y - base) * c;
        if (kStatEnt) entropy = kLn2 * (log_s - v.t / v.s);
        if (rank == 0 && tid == 0) {
          if (a.logp) a.logp[i] = kLn2 * (dy - log_s);
          if (a.lse) a.lse[i] = fmaf(base, a.scale, kLn2 * log_s);
          if (kMode == kLossForward && a.entropy) a.entropy[i] = entropy;
          if (a.stat) a.stat[i] = make_float4(base, log_s, dy, 0.f);
        }
      }
      if (kMode == kLossForward) continue;
      // the loss through this row: da = dL/dlogp, dh = dL/dH
      const float v0 = __shfl_sync(0xffffffffu, in0, at), v1 = __shfl_sync(0xffffffffu, in1, at);
      const float v2 = __shfl_sync(0xffffffffu, in2, at), v3 = __shfl_sync(0xffffffffu, in3, at);
      float da = v0, dh = v1;
      if (kMode == kLossBackward) {
        base = v2;
        log_s = a.coef ? v3 : 0.f;
        if (kEnt) entropy = v3;
      } else {
        const float lp = kLn2 * (dy - log_s), w = v0 * per_weight, adv = v1;
        const float ratio = expf(a.old_logp ? lp - v2 : 0.f);
        const float held = fminf(fmaxf(ratio, a.ratio_lo), a.ratio_hi) * adv, free = ratio * adv;
        const bool clipped = held < free;
        float kl = 0.f, dkl = 0.f;
        if (a.ref_logp) {
          const float x = v3 - lp;
          dkl = expm1f(x);
          kl = dkl - x;
        }
        da = w * ((clipped ? 0.f : -free) - a.kl_coef * dkl);
        dh = -a.entropy_coef * w;
        if (rank == 0 && tid == 0) {
          const float loss = -(clipped ? held : free) + a.kl_coef * kl - a.entropy_coef * entropy;
          sums[0] += static_cast<double>(w) * loss;
          sums[1] += static_cast<double>(w) * kl;
          if (clipped) sums[2] += w;
          sums[3] += static_cast<double>(w) * entropy;
        }
      }
      if (!grad) continue;

      // second walk: dz_j = own 1[j = y] + 2^d (k0 + k1 d) with d = (z_j - base) c
      const float own = a.scale * da;
      const float inv = exp2f(-log_s);
      const float k0 = -a.scale * inv * (kEnt ? da + dh * (entropy - kLn2 * log_s) : da);
      const float k1 = -a.scale * inv * dh * kLn2;
      const Slope slope = {base, c, k0, k1};
      if (t_col >= 0)
        store1(static_cast<TD*>(a.d[t_rk]) + i * a.ldd[t_rk] + t_col, slope_at<kEnt>(slope, z_t) + (y_here ? own : 0.f));
      if (kStat && !twice) place = start;
      int rk = 0;
      for (int k = 0; k < chunks; ++k, place.next()) {
        if ((!kStat || twice) && !wait_full(&sm.full[place.slot], place.turn, a)) {
          fine = false;
          break;
        }
        const int g0 = g_lo + k * kChunkGroups, left = g_hi - g0;
        while (g0 >= a.groups[rk + 1]) ++rk;
        const uint4* src = reinterpret_cast<const uint4*>(ring + place.slot * kLossChunk) + tid;
        if (left >= kChunkGroups && g0 + kChunkGroups <= a.groups[rk + 1]) {
          TD* to = static_cast<TD*>(a.d[rk]) + i * a.ldd[rk] + static_cast<int64_t>(g0 + tid - a.groups[rk]) * kCols;
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            put_group<TZ, TD, kEnt>(src[j * 32 * kLossWarps], slope, to + j * 32 * kLossWarps * kCols);
        } else {
          int r2 = rk;
          for (int g = tid; g < left && g < kChunkGroups; g += 32 * kLossWarps) {
            while (g0 + g >= a.groups[r2 + 1]) ++r2;
            put_group<TZ, TD, kEnt>(src[g - tid], slope,
                                    static_cast<TD*>(a.d[r2]) + i * a.ldd[r2] +
                                        static_cast<int64_t>(g0 + g - a.groups[r2]) * kCols);
          }
        }
        const int at_y = y_group - g0;  // the thread that wrote the target's group writes its column again
        if (at_y >= 0 && at_y < left && at_y < kChunkGroups && at_y % (32 * kLossWarps) == tid)
          store1(static_cast<TD*>(a.d[y_rk]) + i * a.ldd[y_rk] + y_col,
                 slope_at<kEnt>(slope, load1(reinterpret_cast<const TZ*>(src - tid + at_y) + y_col % kCols)) + own);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[place.slot]);
      }
      if (!fine) break;
    }
    if (!fine && lane == 0) raise_error(a.ctrl, FO_ERR_TIMEOUT, kSiteFull, blockIdx.x);
    if (kMode == kLossPolicy && rank == 0 && warp == 0 && fine) {
      // the row's team that comes last adds everyone's sums, in the order of the teams
      int last = 0;
      if (lane == 0) {
        for (int k = 0; k < 4; ++k) a.part[team * 4 + k] = sums[k];
        __threadfence();
        last = atomicInc(a.ctrl + kCtrlDone, static_cast<unsigned>(teams - 1)) == static_cast<unsigned>(teams - 1);
      }
      if (__shfl_sync(0xffffffffu, last, 0)) {
        __threadfence();
        for (int k = 0; k < 4; ++k) {
          double s = 0.0;
          for (int64_t b = lane; b < teams; b += 32) s += __ldcg(a.part + b * 4 + k);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == 0) a.stats[k] = static_cast<float>(s);
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

}  // namespace

int loss_rows_parts(int num_sms) { return num_sms; }

cudaError_t loss_rows_launch(LossArgs a, const LossKind& k, int num_sms, cudaStream_t s) {
  const int cols = k.z32 ? Group<float>::kCols : Group<uint16_t>::kCols;
  for (int r = 0; r < a.P; ++r) a.groups[r + 1] = a.groups[r] + a.cols[r] / cols;
  const int64_t chunks = (a.groups[a.P] + kChunkGroups - 1) / kChunkGroups;
  const bool resident = k.mode == kLossPolicy && a.d[0];  // a row waits in shared memory for its sum
  // CTAs of a row: more where a row would leave little room for the next ones' copies, and where
  // there are fewer rows than SMs
  a.ctas = 1;
  while (resident && a.ctas < kLossMaxCtas && chunks > a.ctas * kLossFit) a.ctas *= 2;
  if (resident && chunks > static_cast<int64_t>(a.ctas) * (kLossSlots - 1)) {
    a.twice = 1;
    a.ctas = 1;
  }
  while (a.ctas < kLossMaxCtas && a.rows * a.ctas * 2 <= num_sms && a.groups[a.P] >= a.ctas * 2 * 32 * kLossWarps)
    a.ctas *= 2;
  void (*kernel)(LossArgs) = k.z32 ? (k.d32 ? kernel_of<float, float>(k) : kernel_of<float, uint16_t>(k))
                                   : (k.d32 ? kernel_of<uint16_t, float>(k) : kernel_of<uint16_t, uint16_t>(k));
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLossSmem);
  if (e != cudaSuccess) return e;
  // teams of CTAs that fit the GPU at once (clusters of 2 all SMs, of 4 144, of 8 120 of 152)
  const int fit = num_sms * (a.ctas <= 2 ? 152 : a.ctas == 4 ? 144 : 120) / 152 / a.ctas;
  const int64_t teams = a.rows < 1 ? 1 : a.rows < fit ? a.rows : fit;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(teams * a.ctas));
  cfg.blockDim = dim3(kLossThreads);
  cfg.dynamicSmemBytes = kLossSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = k.mode != kLossBackward && a.ctas > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fo

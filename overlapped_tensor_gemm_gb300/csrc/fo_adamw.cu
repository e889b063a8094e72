// AdamW over many tensors in few launches, the gradients' norm, and 8-bit states as values.
//
//   g = c gradient,  c = grad_scale, times max_norm / (|grad_scale| norm) where that is below 1
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   w = w - lr (weight_decay w + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// Bound by HBM: every value is read once and written once (fp32 master, bf16 copy and gradient, fp32
// states: 28 bytes an element).  The tensors' addresses are kernel parameters (no table in memory
// that a captured launch would have to keep).  A warp takes a block of 256 elements, two groups of
// four per lane, so that every access of the warp is whole lines in all types.
//
// Measured, 176M parameters: 757-762 us (6.5 TB/s), 8-bit states 461-469 us (6.1 TB/s: 77 instructions an element),
// norm of bf16 gradients 57 us, unpacking to bf16 166-175.
//
// 8-bit states.  A block has its own ranges: m is e4m3 times max|m| / 448; v is one of 255 values
// evenly spaced in log2 between the block's smallest and largest v (few percent apart: rows of a
// weight differ by powers of two, elements of one by less).  Both are rounded up or down at random:
// m moves by 1 - b1 of its distance to g in a step, v by 1 - b2, which is mostly less than half the
// distance of two values, so that rounded to the nearest they would stay where they are.  In the mean
// v's rounding adds nothing to it, to first order in the distance (levels_of).
#include <cfloat>
#include <cmath>
#include <cstring>

#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include <cuda_fp8.h>

#include "fo_attn_common.cuh"
#include "fo_host.h"
#include "fo_ptx.cuh"
#include "fo_wide.cuh"

namespace fo {
namespace {

constexpr int kBlock = 256;           // elements of a block: 8 per lane of a warp
constexpr int kAdamThreads = 256;     // norm, unpacking
constexpr int kCtasPerSm = 4;
constexpr int kStepThreads = 256;
// CTAs of a step per SM.  8-bit states: as many as have the registers for a block under way beside the one
// that is computed (4 without it: 742 us for 176M parameters with norm and unpacking, 706 with it).  32 bits
// need less arithmetic than that, and fewer places in memory at once (3: 839 us with the norm, 2: 823, 1: 925;
// 2 with the registers of 2: 833; all of it with masters.  Without them, in bf16, the registers of 3 spill 8 bytes,
// 36 with fp32 gradients: not timed).
constexpr int kStepCtas8 = 3, kStepCtas32 = 2;
constexpr int kListTensors = 400;     // tensors of one launch
constexpr int kAhead = 4;             // see run_of
constexpr float kMaxE4m3 = 448.f;
constexpr float kOctaves = 24.f;      // v's values span at most 2^24

struct TensorRef {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_range;
  int64_t n;
  uint32_t index;       // place in the caller's list
  uint32_t reserved;
};
struct TensorList {
  int64_t blocks;
  int32_t count;
  int32_t kind;                   // KindBit
  int64_t first[kListTensors];    // blocks of the tensors in front of each (side by side: a search meets few lines)
  TensorRef t[kListTensors];
};
enum KindBit : int { kParam32 = 1, kGrad32 = 2, kMaster = 4, kStates8 = 8 };

struct StepArgs {
  float lr, eps, weight_decay, grad_scale, max_norm;
  float beta1, beta2, rest1, rest2;   // rest = 1 - beta, before either is rounded
  float one;                          // 1, which the compiler does not know
  float fix1, fix2;                   // 1 / (1 - b1^t), 1 / (1 - b2^t)
  double exact1, exact2;              // the betas
  int64_t step;
  uint32_t seed_low, seed_high;
  const float* lr_dev;
  const int32_t* step_dev;
  const float* norm;
  uint32_t* ctrl;
};
static_assert(sizeof(TensorList) + sizeof(StepArgs) <= 32764, "kernel parameters");

// Blocks that a warp of the norm or of the unpacking takes in a row: several, loaded at once, where there
// are enough for every warp
__host__ __device__ inline int run_of(int64_t blocks, int64_t warps) {
  return blocks >= 4 * kAhead * warps ? kAhead : 1;
}
// The tensor of block b: the last one that starts at or in front of it
template <typename List>
__device__ __forceinline__ int tensor_of(const List& l, int64_t b) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= b) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// 32 bits scattered: two rounds of xor-shift and multiply (constants of C. Wellons' search for
// functions of this form whose output bits depend evenly on all input bits)
__host__ __device__ __forceinline__ uint32_t scatter(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7feb352du;
  x = (x ^ (x >> 15)) * 0x846ca68bu;
  return x ^ (x >> 16);
}

typedef uint64_t Pair;  // two fp32 values
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair sub2(Pair a, Pair b) {
  Pair r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair both(float f) { return pack2(f, f); }
// (numbers below 2^-126 count as 0)
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_sqrt(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 4 elements from p on as they lie there, the first n of them inside the tensor.  (What is read is
// converted later: a wait inside a condition would keep the next load back.)
template <bool kFull>
__device__ __forceinline__ float4 load4(const float* p, int n) {
  if (kFull || n >= 4) return *reinterpret_cast<const float4*>(p);
  return make_float4(0 < n ? p[0] : 0.f, 1 < n ? p[1] : 0.f, 2 < n ? p[2] : 0.f, 0.f);
}
template <bool kFull>
__device__ __forceinline__ uint2 load4(const uint16_t* p, int n) {
  if (kFull || n >= 4) return *reinterpret_cast<const uint2*>(p);
  return make_uint2((0 < n ? p[0] : 0u) | (1 < n ? static_cast<uint32_t>(p[1]) << 16 : 0u), 2 < n ? p[2] : 0u);
}
template <bool kFull>
__device__ __forceinline__ uint32_t load4(const uint8_t* p, int n) {
  if (kFull || n >= 4) return *reinterpret_cast<const uint32_t*>(p);
  return (0 < n ? p[0] : 0u) | (1 < n ? static_cast<uint32_t>(p[1]) << 8 : 0u) |
         (2 < n ? static_cast<uint32_t>(p[2]) << 16 : 0u);
}
__device__ __forceinline__ void values(const float4& q, Pair (&v)[2]) {
  v[0] = pack2(q.x, q.y);
  v[1] = pack2(q.z, q.w);
}
__device__ __forceinline__ void values(const uint2& q, Pair (&v)[2]) {
  v[0] = pack2(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u));
  v[1] = pack2(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xFFFF0000u));
}
template <bool kFull>
__device__ __forceinline__ void store4(float* p, int n, const Pair (&v)[2]) {
  float f[4];
  unpack2(v[0], f[0], f[1]);
  unpack2(v[1], f[2], f[3]);
  if (kFull || n >= 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) p[k] = f[k];
  }
}
template <bool kFull>
__device__ __forceinline__ void store4(uint16_t* p, int n, const Pair (&v)[2]) {
  uint32_t q[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float x, y;
    unpack2(v[k], x, y);
    q[k] = pack_bf16x2(x, y);
  }
  if (kFull || n >= 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) p[k] = static_cast<uint16_t>(q[k >> 1] >> (16 * (k & 1)));
  }
}
template <bool kFull>
__device__ __forceinline__ void store4(uint8_t* p, int n, uint32_t q) {
  if (kFull || n >= 4) {
    *reinterpret_cast<uint32_t*>(p) = q;
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) p[k] = static_cast<uint8_t>(q >> (8 * k));
  }
}

// A half of `pair` in fp32 (an addition that takes one f16 operand: no conversion)
__device__ __forceinline__ float low_half(uint32_t pair, float plus) {
  float r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; add.f32.f16 %0, l, %2;}" : "=f"(r) : "r"(pair), "f"(plus));
  return r;
}
__device__ __forceinline__ float high_half(uint32_t pair, float plus) {
  float r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; add.f32.f16 %0, h, %2;}" : "=f"(r) : "r"(pair), "f"(plus));
  return r;
}
// 4 e4m3 values
__device__ __forceinline__ void from_e4m3(uint32_t q, Pair (&v)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q >> (16 * k)), __NV_E4M3);
    const uint32_t pair = h.x | static_cast<uint32_t>(h.y) << 16;
    v[k] = pack2(low_half(pair, 0.f), high_half(pair, 0.f));
  }
}
// 4 codes of v as values: a code is the low byte of an f16 from 1024 on, where steps are 1.  (Zeros are
// rare: without them no code is looked at by itself.)
__device__ __forceinline__ void from_levels(uint32_t q, float low, float gap, Pair (&v)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t pair = __byte_perm(q, 0x64646464u, k ? 0x4342 : 0x4140);
    float x, y;
    unpack2(ffma2(pack2(low_half(pair, -1025.f), high_half(pair, -1025.f)), both(gap), both(low)), x, y);
    v[k] = pack2(fast_exp2(x), fast_exp2(y));
  }
  if ((q - 0x01010101u) & ~q & 0x80808080u) {  // a byte is 0
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x, y;
      unpack2(v[k], x, y);
      v[k] = pack2(q >> (16 * k) & 0xFFu ? x : 0.f, q >> (16 * k + 8) & 0xFFu ? y : 0.f);
    }
  }
}
// 4 values of m, in units of the scale (at most 448 and a few units in the last place), up or down to e4m3:
// a random part of a step is added and what a step holds below is cut off.  Times 2^-120 the ranges of
// e4m3, its subnormal one too, are those of fp32: an e4m3 number is the bits from the 20th on, and the sign.
// The quotient is m over the scale rounded once (a product with an approximate inverse, corrected by what it
// leaves: P. Markstein, IBM J. Res. Dev. 34, 1990): a last bit of it can decide a code.
__device__ __forceinline__ uint32_t to_e4m3(const Pair (&m)[2], float scale, float inv_scale, const uint32_t* word) {
  uint32_t sum[4], sign[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float x, y;
    const Pair q = mul2(m[k], both(inv_scale)), rest = ffma2(q, both(-scale), m[k]);
    unpack2(mul2(ffma2(rest, both(inv_scale), q), both(0x1p-120f)), x, y);
    sign[2 * k] = __float_as_uint(x);
    sign[2 * k + 1] = __float_as_uint(y);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sum[k] = (sign[k] << 4) + __byte_perm(word[k], 0, 0x4104);  // (low half, 8 up)
  const uint32_t code = __byte_perm(__byte_perm(sum[0], sum[1], 0x0073), __byte_perm(sum[2], sum[3], 0x0073), 0x5410);
  const uint32_t high = __byte_perm(__byte_perm(sign[0], sign[1], 0x0073), __byte_perm(sign[2], sign[3], 0x0073), 0x5410);
  return code | (high & 0x80808080u);
}
// The codes of two v (low bytes).  y = (log2 v - low) / gap counts codes from 1; with s = y - 1/2 less
// its nearest whole number w, y is w and a part s + 1/2; up with probability part - bend part (1 - part)
// (the mean of the two values, not of their logarithms, is v: to first order in gap).  Up or not is the
// sum of w and part less a random number rounded up.  Zeros are not looked at.
struct Levels {
  float per_gap, offset, bend;  // 1 / gap, -low / gap - 1/2, gap ln 2 / 2
};
__device__ __forceinline__ Pair add2_up(Pair a, Pair b) {
  Pair r;
  asm("add.rp.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void levels_of(Pair v, const Levels& l, uint32_t word0, uint32_t word1,
                                          uint32_t (&code)[2]) {
  const Pair magic = both(12582913.f);  // 1.5 2^23 + 1: a sum's last bits are the nearest whole number and 1
  float a, b, x, y;
  unpack2(v, a, b);
  unpack2(ffma2(pack2(fast_log2(a), fast_log2(b)), both(l.per_gap), both(l.offset)), x, y);
  const Pair at = pack2(fminf(fmaxf(x, -0.5f), 253.5f), fminf(fmaxf(y, -0.5f), 253.5f));
  const Pair sum = fadd2(at, magic), s = sub2(at, sub2(sum, magic));
  const Pair part = ffma2(s, ffma2(s, both(l.bend), both(1.f)), both(fmaf(l.bend, -0.25f, 0.5f)));
  // 2^23 and the random number's upper half
  const Pair r = fadd2(pack2(__uint_as_float(__byte_perm(word0, 0x4B000000u, 0x7432)),
                             __uint_as_float(__byte_perm(word1, 0x4B000000u, 0x7432))),
                       both(-8388608.f));
  unpack2(add2_up(sum, ffma2(r, both(-0x1p-16f), part)), x, y);
  code[0] = __float_as_uint(x);
  code[1] = __float_as_uint(y);
}
// A bf16 value next to w, by the upper half of `word`; infinities and NaN stay
__device__ __forceinline__ float cut_bf16(float w, uint32_t word) {
  const float q = __uint_as_float((__float_as_uint(w) + (word >> 16)) & 0xFFFF0000u);
  return fabsf(w) <= FLT_MAX ? q : w;
}

// Corrections of a step that is read from memory: 1 / (1 - b^t) by repeated squaring in fp64
__device__ __forceinline__ float correction(double beta, int64_t t) {
  double p = 1.0, b = beta;
  for (; t > 0; t >>= 1) {
    if (t & 1) p *= b;
    b *= b;
  }
  return static_cast<float>(1.0 / (1.0 - p));
}

// What a step's blocks share
struct Step {
  float beta1, beta2, rest1, rest2, one, eps, decay, rate, fix2, c;
  uint32_t key;
  bool cut;
};
// A block as it lies in memory
template <bool kP32, bool kG32, bool kHasMaster, bool k8>
struct Raw {
  typedef typename std::conditional<kP32, float, uint16_t>::type TP;
  typedef typename std::conditional<kG32, float, uint16_t>::type TG;
  typedef typename std::conditional<kHasMaster, float, TP>::type TW;
  typedef typename std::conditional<k8, uint8_t, float>::type TS;
  decltype(load4<true>(static_cast<const TG*>(nullptr), 0)) g[2];
  decltype(load4<true>(static_cast<const TW*>(nullptr), 0)) w[2];
  decltype(load4<true>(static_cast<const TS*>(nullptr), 0)) m[2], v[2];
  float scale;
  float2 range;
  template <bool kFull>
  __device__ __forceinline__ void load(const TensorRef& t, int64_t blk, int n) {
    const int lane = threadIdx.x & 31;
    const int64_t at = blk * kBlock + lane * 4;
    n -= lane * 4;
    const TW* const tw = (kHasMaster ? reinterpret_cast<const TW*>(t.master) : static_cast<const TW*>(t.param)) + at;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      g[q] = load4<kFull>(static_cast<const TG*>(t.grad) + at + q * 128, n - q * 128);
      w[q] = load4<kFull>(tw + q * 128, n - q * 128);
      m[q] = load4<kFull>(static_cast<const TS*>(t.m) + at + q * 128, n - q * 128);
      v[q] = load4<kFull>(static_cast<const TS*>(t.v) + at + q * 128, n - q * 128);
    }
    if constexpr (k8) {
      scale = t.m_scale[blk];
      range = reinterpret_cast<const float2*>(t.v_range)[blk];
    }
  }
};
// One block, the first n of its elements inside the tensor.  Squares, roots and quotients keep to
// numbers from 2^-126 on: a smaller v counts as that in the root (its update is smaller for it).
template <bool kP32, bool kG32, bool kHasMaster, bool k8, bool kFull>
__device__ __forceinline__ void step_block(const TensorRef& t, int64_t blk, int n, const Step& a,
                                           const Raw<kP32, kG32, kHasMaster, k8>& raw) {
  typedef typename std::conditional<kP32, float, uint16_t>::type TP;
  const int lane = threadIdx.x & 31;
  const int64_t at = blk * kBlock + lane * 4;
  n -= lane * 4;
  Pair g[4], w[4], m[4], v[4];
  if constexpr (k8) {
    from_e4m3(raw.m[0], reinterpret_cast<Pair(&)[2]>(m[0]));
    from_e4m3(raw.m[1], reinterpret_cast<Pair(&)[2]>(m[2]));
    from_levels(raw.v[0], raw.range.x, raw.range.y, reinterpret_cast<Pair(&)[2]>(v[0]));
    from_levels(raw.v[1], raw.range.x, raw.range.y, reinterpret_cast<Pair(&)[2]>(v[2]));
  } else {
    values(raw.m[0], reinterpret_cast<Pair(&)[2]>(m[0]));
    values(raw.m[1], reinterpret_cast<Pair(&)[2]>(m[2]));
    values(raw.v[0], reinterpret_cast<Pair(&)[2]>(v[0]));
    values(raw.v[1], reinterpret_cast<Pair(&)[2]>(v[2]));
  }
  values(raw.g[0], reinterpret_cast<Pair(&)[2]>(g[0]));
  values(raw.g[1], reinterpret_cast<Pair(&)[2]>(g[2]));
  values(raw.w[0], reinterpret_cast<Pair(&)[2]>(w[0]));
  values(raw.w[1], reinterpret_cast<Pair(&)[2]>(w[2]));

  // (the bits of values that are not negative are ordered as the values are)
  float top_m = 0.f;
  uint32_t top_v = 0, min_v = 0xFFFFFFFFu;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const Pair x = mul2(g[q], both(a.c));
    if (k8) {
      // each product and the sum rounded once (see to_e4m3).  An addition of the packed products becomes one
      // operation with one of them, with .rn too: one block in six had another scale then
      m[q] = ffma2(both(a.one), mul2(both(a.beta1), mul2(m[q], both(raw.scale))), mul2(both(a.rest1), x));
    } else {
      m[q] = ffma2(both(a.beta1), m[q], mul2(both(a.rest1), x));
    }
    v[q] = ffma2(both(a.beta2), v[q], mul2(mul2(both(a.rest2), x), x));
    float x0, x1, y0, y1;
    unpack2(v[q], x0, x1);
    unpack2(mul2(pack2(fmaxf(x0, FLT_MIN), fmaxf(x1, FLT_MIN)), both(a.fix2)), y0, y1);
    unpack2(fadd2(pack2(fast_sqrt(y0), fast_sqrt(y1)), both(a.eps)), y0, y1);
    const Pair change = mul2(mul2(both(a.rate), m[q]), pack2(fast_inverse(y0), fast_inverse(y1)));
    w[q] = sub2(w[q], ffma2(both(a.decay), w[q], change));
    if (k8) {
      top_v = max(top_v, max(__float_as_uint(x0), __float_as_uint(x1)));
      min_v = min(min_v, min(__float_as_uint(x0), __float_as_uint(x1)));
      unpack2(m[q], y0, y1);
      top_m = fmax3(top_m, fabsf(y0), fabsf(y1));
    }
  }
  uint32_t word[8];
  if (k8 || a.cut) {
    const uint32_t base =
        scatter(scatter(a.key + t.index) + static_cast<uint32_t>(blk)) + static_cast<uint32_t>(lane * 4) * 0x9E3779B9u;
#pragma unroll
    for (int k = 0; k < 8; ++k) word[k] = scatter(base + static_cast<uint32_t>((k & 4) * 32 + (k & 3)) * 0x9E3779B9u);
  }
  if constexpr (k8) {
    top_m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_m)));
    top_v = __reduce_max_sync(0xffffffffu, top_v);
    min_v = __reduce_min_sync(0xffffffffu, min_v);
    const bool zeros = min_v == 0;
    if (zeros) {  // the smallest of the others: the bits of 0, less one, come last
      min_v = 0xFFFFFFFFu;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x, y;
        unpack2(v[q], x, y);
        min_v = min(min_v, min(__float_as_uint(x) - 1u, __float_as_uint(y) - 1u));
      }
      min_v = __reduce_min_sync(0xffffffffu, min_v) + 1u;
    }
    float scale = 0.f, inv_scale = 0.f, low = 0.f, gap = 0.f;
    Levels l = {0.f, -0.5f, 0.f};
    if (top_m > 1e-30f) {  // smaller ones are kept as zeros
      scale = top_m * (1.f / kMaxE4m3);
      inv_scale = fast_inverse(scale);
    }
    if (top_v != 0) {
      const float top = fast_log2(fmaxf(__uint_as_float(top_v), FLT_MIN));
      low = fmaxf(fast_log2(fmaxf(__uint_as_float(min_v), FLT_MIN)), top - kOctaves);
      gap = (top - low) * (1.f / 254.f);
      if (gap > 0.f) {
        l.per_gap = __fdividef(1.f, gap);
        l.offset = -low * l.per_gap - 0.5f;
        l.bend = 0.34657359f * gap;
      }
    }
    uint8_t* const tm = static_cast<uint8_t*>(t.m) + at;
    uint8_t* const tv = static_cast<uint8_t*>(t.v) + at;
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      uint32_t c0[2], c1[2];
      levels_of(v[q], l, word[2 * q], word[2 * q + 1], c0);
      levels_of(v[q + 1], l, word[2 * q + 2], word[2 * q + 3], c1);
      uint32_t code = __byte_perm(__byte_perm(c0[0], c0[1], 0x0040), __byte_perm(c1[0], c1[1], 0x0040), 0x5410);
      if (zeros) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x, y;
          unpack2(v[q + k], x, y);
          if (!(x > 0.f)) code &= ~(0xFFu << (16 * k));
          if (!(y > 0.f)) code &= ~(0xFF00u << (16 * k));
        }
      }
      store4<kFull>(tm + q * 64, n - q * 64, to_e4m3(reinterpret_cast<Pair(&)[2]>(m[q]), scale, inv_scale, word + 2 * q));
      store4<kFull>(tv + q * 64, n - q * 64, code);
    }
    if (lane == 0) {
      t.m_scale[blk] = scale;
      reinterpret_cast<float2*>(t.v_range)[blk] = make_float2(low, gap);
    }
  } else {
    float* const tm = static_cast<float*>(t.m) + at;
    float* const tv = static_cast<float*>(t.v) + at;
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      store4<kFull>(tm + q * 64, n - q * 64, reinterpret_cast<Pair(&)[2]>(m[q]));
      store4<kFull>(tv + q * 64, n - q * 64, reinterpret_cast<Pair(&)[2]>(v[q]));
    }
  }
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    if (kHasMaster) store4<kFull>(t.master + at + q * 64, n - q * 64, reinterpret_cast<Pair(&)[2]>(w[q]));
    if (!kP32 && !kHasMaster && a.cut) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x, y;
        unpack2(w[q + k], x, y);
        w[q + k] = pack2(cut_bf16(x, word[2 * q + 2 * k] * 0x9E3779B9u),
                         cut_bf16(y, word[2 * q + 2 * k + 1] * 0x9E3779B9u));
      }
    }
    store4<kFull>(static_cast<TP*>(t.param) + at + q * 64, n - q * 64, reinterpret_cast<Pair(&)[2]>(w[q]));
  }
}

template <bool kP32, bool kG32, bool kHasMaster, bool k8>
__global__ void __launch_bounds__(kStepThreads, kStepCtas8)
    adamw_kernel(const __grid_constant__ TensorList l, const __grid_constant__ StepArgs a, bool cut) {
  __shared__ float fixes[2];
  Step s;
  s.c = a.grad_scale;
  if (a.norm) {
    const float norm = *a.norm;
    if (!(norm <= FLT_MAX)) return;  // infinite or NaN: nothing is written
    const float whole = norm * fabsf(a.grad_scale);
    if (a.max_norm > 0.f && whole > a.max_norm) s.c *= a.max_norm / whole;
  }
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const int64_t step = a.step_dev ? *a.step_dev : a.step;
  float fix1 = a.fix1;
  s.fix2 = a.fix2;
  if (a.step_dev) {
    if (step < 1) {
      if (blockIdx.x == 0 && threadIdx.x == 0)
        note_error(a.ctrl, FO_ERR_RANGE, kSiteStep, static_cast<uint32_t>(step));
      return;
    }
    if (threadIdx.x < 2) fixes[threadIdx.x] = correction(threadIdx.x ? a.exact2 : a.exact1, step);
    __syncthreads();
    fix1 = fixes[0];
    s.fix2 = fixes[1];
  }
  s.beta1 = a.beta1;
  s.beta2 = a.beta2;
  s.rest1 = a.rest1;
  s.rest2 = a.rest2;
  s.one = a.one;
  s.eps = a.eps;
  s.decay = lr * a.weight_decay;
  s.rate = lr * fix1;
  s.key = scatter(scatter(a.seed_low ^ scatter(static_cast<uint32_t>(step))) ^ a.seed_high);
  s.cut = cut;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kStepThreads / 32);
  int64_t b = static_cast<int64_t>(blockIdx.x) * (kStepThreads / 32) + (threadIdx.x >> 5);
  if (b >= l.blocks) return;
  int i = tensor_of(l, b);
  // while a block is computed the warp's next one comes, where the same tensor has it whole
  Raw<kP32, kG32, kHasMaster, k8> next;
  bool have = false;
  for (; b < l.blocks; b += warps) {
    while (i + 1 < l.count && l.first[i + 1] <= b) ++i;
    const TensorRef& t = l.t[i];
    const int64_t blk = b - l.first[i], left = t.n - blk * kBlock;
    if (left >= kBlock) {
      if (!have) next.template load<true>(t, blk, kBlock);
      const Raw<kP32, kG32, kHasMaster, k8> now = next;
      have = left >= (warps + 1) * kBlock;
      if (have) next.template load<true>(t, blk + warps, kBlock);
      step_block<kP32, kG32, kHasMaster, k8, true>(t, blk, kBlock, s, now);
    } else {
      Raw<kP32, kG32, kHasMaster, k8> now;
      now.template load<false>(t, blk, static_cast<int>(left));
      step_block<kP32, kG32, kHasMaster, k8, false>(t, blk, static_cast<int>(left), s, now);
      have = false;
    }
  }
}

// Fixed-order sum over the CTA, in thread 0
__device__ __forceinline__ Wide block_sum(Wide v, Wide* buf) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < kAdamThreads / 32; ++w) v = plus(v, buf[w]);
  return v;
}

// Squares of one list's gradients; the CTA that comes last adds the CTAs' sums in order to what the
// lists in front left, and behind the last list takes the root
struct NormArgs {
  Wide* part;      // [0]: sum of the lists so far; then one per CTA
  float* norm;
  int32_t first, last;
  uint32_t* ctrl;
};
template <bool kG32>
__global__ void __launch_bounds__(kAdamThreads) grad_norm_kernel(const __grid_constant__ TensorList l,
                                                                 const __grid_constant__ NormArgs a) {
  typedef typename std::conditional<kG32, float, uint16_t>::type TG;
  __shared__ Wide buf[kAdamThreads / 32];
  __shared__ bool last;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAdamThreads / 32);
  const int run = run_of(l.blocks, warps);
  int64_t b = (static_cast<int64_t>(blockIdx.x) * (kAdamThreads / 32) + (threadIdx.x >> 5)) * run;
  Wide total = {0.f, 0.f};
  if (b < l.blocks) {
    int i = tensor_of(l, b);
    while (b < l.blocks) {
      float sum = 0.f;  // at most 512 squares in fp32
#pragma unroll 1
      for (int turn = 0; turn < 64 / kAhead && b < l.blocks; ++turn, b += warps * run) {
        while (i + 1 < l.count && l.first[i + 1] <= b) ++i;
        Pair s = 0;
        const int64_t blk = b - l.first[i];
        if (run == kAhead && l.t[i].n - blk * kBlock >= kAhead * kBlock) {  // whole blocks of this tensor
          // (16 bytes a lane: a block is one load in bf16, two in fp32)
          constexpr int kLoads = kAhead * (kG32 ? 2 : 1);
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const TG*>(l.t[i].grad) + blk * kBlock) + lane;
          uint4 g[kLoads];
#pragma unroll
          for (int q = 0; q < kLoads; ++q) g[q] = p[q * 32];
#pragma unroll
          for (int q = 0; q < kLoads; ++q) {
            Pair x[2], y[2];
            if constexpr (kG32) {
              x[0] = pack2(__uint_as_float(g[q].x), __uint_as_float(g[q].y));
              x[1] = pack2(__uint_as_float(g[q].z), __uint_as_float(g[q].w));
            } else {
              values(make_uint2(g[q].x, g[q].y), x);
              values(make_uint2(g[q].z, g[q].w), y);
              s = ffma2(y[0], y[0], ffma2(y[1], y[1], s));
            }
            s = ffma2(x[0], x[0], ffma2(x[1], x[1], s));
          }
        } else {
          int j = i;
          for (int64_t k = b; k < b + run && k < l.blocks; ++k) {
            while (j + 1 < l.count && l.first[j + 1] <= k) ++j;
            const TensorRef& t = l.t[j];
            const int64_t at = (k - l.first[j]) * kBlock + lane * 4, left = t.n - at;
            const int n = left < kBlock ? static_cast<int>(left < 0 ? 0 : left) : kBlock;
            const TG* const tg = static_cast<const TG*>(t.grad) + at;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              Pair v[2];
              values(load4<false>(tg + q * 128, n - q * 128), v);
              s = ffma2(v[0], v[0], ffma2(v[1], v[1], s));
            }
          }
        }
        float x, y;
        unpack2(s, x, y);
        sum += x + y;
      }
      total = plus(total, wide(sum));
    }
  }
  total = block_sum(total, buf);
  if (threadIdx.x == 0) {
    a.part[1 + blockIdx.x] = total;
    __threadfence();
    last = atomicInc(a.ctrl + kCtrlDone, gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  total = Wide{0.f, 0.f};
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kAdamThreads) {
    const float2 p = __ldcg(reinterpret_cast<const float2*>(a.part + 1 + i));
    total = plus(total, Wide{p.x, p.y});
  }
  __syncthreads();
  total = block_sum(total, buf);
  if (threadIdx.x == 0) {
    if (!a.first) {
      const float2 p = __ldcg(reinterpret_cast<const float2*>(a.part));
      total = plus(total, Wide{p.x, p.y});
    }
    a.part[0] = total;
    if (a.last) a.norm[0] = sqrtf(total.hi + total.lo);
  }
}

struct UnpackList {
  int64_t blocks;
  int32_t count;
  int32_t reserved;
  int64_t first[kListTensors];
  struct Ref {
    const uint8_t* m;
    const uint8_t* v;
    const float* m_scale;
    const float* v_range;
    void* m_out;
    void* v_out;
    int64_t n;
  } t[kListTensors];
};
static_assert(sizeof(UnpackList) <= 32764, "kernel parameters");

// count blocks; the first n elements of each are inside the tensor
template <typename T, int count, bool kFull>
__device__ __forceinline__ void unpack_blocks(const UnpackList::Ref& t, int64_t blk, int n) {
  const int lane = threadIdx.x & 31;
  const int64_t at = blk * kBlock + lane * 4;
  n -= lane * 4;
  uint32_t mq[count][2], vq[count][2];
  float scale[count];
  float2 range[count];
#pragma unroll
  for (int u = 0; u < count; ++u) {
    scale[u] = t.m_scale[blk + u];
    range[u] = reinterpret_cast<const float2*>(t.v_range)[blk + u];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      mq[u][q] = load4<kFull>(t.m + at + u * kBlock + q * 128, n - q * 128);
      vq[u][q] = load4<kFull>(t.v + at + u * kBlock + q * 128, n - q * 128);
    }
  }
#pragma unroll
  for (int u = 0; u < count; ++u)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      Pair m[2], v[2];
      from_e4m3(mq[u][q], m);
      from_levels(vq[u][q], range[u].x, range[u].y, v);
      m[0] = mul2(m[0], both(scale[u]));
      m[1] = mul2(m[1], both(scale[u]));
      store4<kFull>(static_cast<T*>(t.m_out) + at + u * kBlock + q * 128, n - q * 128, m);
      store4<kFull>(static_cast<T*>(t.v_out) + at + u * kBlock + q * 128, n - q * 128, v);
    }
}

template <typename T>
__global__ void __launch_bounds__(kAdamThreads) unpack_kernel(const __grid_constant__ UnpackList l) {
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAdamThreads / 32);
  const int run = run_of(l.blocks, warps);
  int64_t b = (static_cast<int64_t>(blockIdx.x) * (kAdamThreads / 32) + (threadIdx.x >> 5)) * run;
  if (b >= l.blocks) return;
  int i = tensor_of(l, b);
  for (; b < l.blocks; b += warps * run) {
    while (i + 1 < l.count && l.first[i + 1] <= b) ++i;
    const int64_t blk = b - l.first[i];
    if (run == kAhead && l.t[i].n - blk * kBlock >= kAhead * kBlock) {  // whole blocks of this tensor
      unpack_blocks<T, kAhead, true>(l.t[i], blk, kBlock);
    } else {
      int j = i;
      for (int64_t k = b; k < b + run && k < l.blocks; ++k) {
        while (j + 1 < l.count && l.first[j + 1] <= k) ++j;
        const int64_t one = k - l.first[j], left = l.t[j].n - one * kBlock;
        unpack_blocks<T, 1, false>(l.t[j], one, static_cast<int>(left < kBlock ? left : kBlock));
      }
    }
  }
}

typedef void (*StepKernel)(TensorList, StepArgs, bool);
template <bool kP32, bool kMast>
StepKernel step_kernel_of(int kind) {
  if (kind & kGrad32)
    return kind & kStates8 ? adamw_kernel<kP32, true, kMast, true> : adamw_kernel<kP32, true, kMast, false>;
  return kind & kStates8 ? adamw_kernel<kP32, false, kMast, true> : adamw_kernel<kP32, false, kMast, false>;
}
StepKernel step_kernel(int kind) {
  if (kind & kParam32) return step_kernel_of<true, false>(kind);
  return kind & kMaster ? step_kernel_of<false, true>(kind) : step_kernel_of<false, false>(kind);
}

int grid_for(fo_ctx* ctx, int64_t blocks, int threads = kAdamThreads, int per_sm = kCtasPerSm) {
  const int64_t ctas = (blocks + threads / 32 - 1) / (threads / 32);
  const int64_t most = static_cast<int64_t>(host_num_sms(ctx)) * per_sm;
  return static_cast<int>(ctas < most ? ctas : most);
}

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

fo_status check_ptr(const void* p, const char* what, int i, int align = 16) {
  if (!p) return host_failf(FO_ERR_INVALID_ARG, "%s[%d]: null pointer", what, i);
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return host_failf(FO_ERR_UNSUPPORTED, "%s[%d]: pointer not %d-byte aligned", what, i, align);
  return FO_OK;
}

struct Span {
  uintptr_t lo, hi;
  int tensor;
  const char* what;
  bool written;
};
// Spans by address, each with the one in front of it or itself that reaches furthest
struct Spans {
  std::vector<Span> at, reach;
  void seal() {
    std::sort(at.begin(), at.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
    reach = at;
    for (size_t i = 1; i < reach.size(); ++i)
      if (reach[i - 1].hi > reach[i].hi) reach[i] = reach[i - 1];
  }
  // one that meets lo .. hi, or null
  const Span* meets(uintptr_t lo, uintptr_t hi) const {
    const auto next = std::lower_bound(at.begin(), at.end(), hi, [](const Span& a, uintptr_t v) { return a.lo < v; });
    const size_t n = next - at.begin();
    return n > 0 && reach[n - 1].hi > lo ? &reach[n - 1] : nullptr;
  }
};
Span span_of(const void* p, int64_t bytes, int tensor, const char* what, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + static_cast<uintptr_t>(bytes), tensor, what, written};
}

}  // namespace
}  // namespace fo

using namespace fo;

struct fo_adamw_group {
  std::vector<TensorList> lists;       // by kind
  std::vector<fo_adamw_tensor> tensors;
  Spans written, used;                 // what a step writes; that and the gradients
};

// One value beside the group's tensors (null: none)
static fo_status check_beside(const Spans& spans, const void* p, const char* what) {
  if (!p) return FO_OK;
  const Span x = span_of(p, 4, 0, what, false);
  if (const Span* hit = spans.meets(x.lo, x.hi))
    return host_failf(FO_ERR_INVALID_ARG, "%s overlaps %s[%d]", what, hit->what, hit->tensor);
  return FO_OK;
}

extern "C" {

fo_status fo_adamw_group_create(const fo_adamw_tensor* tensors, int count, fo_adamw_group** out) try {
  if (!out) return host_fail(FO_ERR_INVALID_ARG, "null out pointer");
  *out = nullptr;
  if (count < 0 || (count > 0 && !tensors)) return host_fail(FO_ERR_INVALID_ARG, "null tensor array");
  Spans used, written;
  for (int i = 0; i < count; ++i) {
    const fo_adamw_tensor& t = tensors[i];
    if (t.n < 0) return host_failf(FO_ERR_SHAPE, "tensor %d: negative size", i);
    if (t.n > (1ll << 39)) return host_failf(FO_ERR_UNSUPPORTED, "tensor %d: more than 2^39 elements", i);
    if (t.param_dtype != FO_BF16 && t.param_dtype != FO_F32)
      return host_failf(FO_ERR_INVALID_ARG, "param[%d]: unknown dtype", i);
    if (t.grad_dtype != FO_BF16 && t.grad_dtype != FO_F32)
      return host_failf(FO_ERR_INVALID_ARG, "grad[%d]: unknown dtype", i);
    if (t.master && t.param_dtype == FO_F32)
      return host_failf(FO_ERR_INVALID_ARG, "master[%d]: an fp32 parameter has none", i);
    if ((t.m_scale != nullptr) != (t.v_range != nullptr))
      return host_failf(FO_ERR_INVALID_ARG, "tensor %d: m_scale and v_range go together", i);
    if (t.n == 0) continue;
    const bool eight = t.m_scale != nullptr;
    FO_TRY_HOST(check_ptr(t.param, "param", i));
    FO_TRY_HOST(check_ptr(t.grad, "grad", i));
    if (t.master) FO_TRY_HOST(check_ptr(t.master, "master", i));
    FO_TRY_HOST(check_ptr(t.m, "m", i));
    FO_TRY_HOST(check_ptr(t.v, "v", i));
    if (eight) {
      FO_TRY_HOST(check_ptr(t.m_scale, "m_scale", i, 4));
      FO_TRY_HOST(check_ptr(t.v_range, "v_range", i, 8));
    }
    auto add = [&](const void* p, int64_t bytes, const char* what, bool writes) {
      if (!p) return;
      used.at.push_back(span_of(p, bytes, i, what, writes));
      if (writes) written.at.push_back(used.at.back());
    };
    const int64_t state = eight ? t.n : 4 * t.n;
    add(t.param, t.n * (t.param_dtype == FO_F32 ? 4 : 2), "param", true);
    add(t.grad, t.n * (t.grad_dtype == FO_F32 ? 4 : 2), "grad", false);
    add(t.master, 4 * t.n, "master", true);
    add(t.m, state, "m", true);
    add(t.v, state, "v", true);
    add(t.m_scale, 4 * blocks_of(t.n), "m_scale", true);
    add(t.v_range, 8 * blocks_of(t.n), "v_range", true);
  }
  used.seal();
  written.seal();
  // each against what starts in front of it: a written one against all, a gradient against the written ones
  const Span* all = nullptr;
  const Span* writes = nullptr;
  for (const Span& x : used.at) {
    const Span* hit = x.written ? all : writes;
    if (hit && hit->hi > x.lo)
      return host_failf(FO_ERR_INVALID_ARG, "%s[%d] overlaps %s[%d]", x.what, x.tensor, hit->what, hit->tensor);
    if (!all || x.hi > all->hi) all = &x;
    if (x.written && (!writes || x.hi > writes->hi)) writes = &x;
  }
  fo_adamw_group* g = new fo_adamw_group();
  try {
    g->tensors.assign(tensors, tensors + count);
    g->used = std::move(used);
    g->written = std::move(written);
    for (int kind = 0; kind < 16; ++kind) {
      int open = -1;  // list that takes the kind's next tensor
      for (int i = 0; i < count; ++i) {
        const fo_adamw_tensor& t = tensors[i];
        const int k = (t.param_dtype == FO_F32 ? kParam32 : 0) | (t.grad_dtype == FO_F32 ? kGrad32 : 0) |
                      (t.master ? kMaster : 0) | (t.m_scale ? kStates8 : 0);
        if (k != kind || t.n == 0) continue;
        if (open < 0 || g->lists[open].count == kListTensors) {
          g->lists.emplace_back();
          open = static_cast<int>(g->lists.size()) - 1;
          std::memset(&g->lists[open], 0, sizeof(TensorList));
          g->lists[open].kind = kind;
        }
        TensorList& l = g->lists[open];
        l.first[l.count] = l.blocks;
        l.t[l.count++] =
            TensorRef{t.param, t.grad, t.master, t.m, t.v, t.m_scale, t.v_range, t.n, static_cast<uint32_t>(i), 0};
        l.blocks += blocks_of(t.n);
      }
    }
  } catch (...) {
    delete g;
    throw;
  }
  *out = g;
  return FO_OK;
} catch (...) {
  return host_fail(FO_ERR_OOM, "out of host memory");
}

fo_status fo_adamw_group_destroy(fo_adamw_group* group) {
  delete group;
  return FO_OK;
}

fo_status fo_grad_norm(fo_ctx* ctx, const fo_adamw_group* group, float* norm, void* stream) {
  if (!group) return host_fail(FO_ERR_INVALID_ARG, "null group");
  FO_TRY_HOST(check_ptr(norm, "norm", 0, 4));
  FO_TRY_HOST(check_beside(group->used, norm, "norm"));
  FO_TRY_HOST(host_check_ctx(ctx, 1));
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (group->lists.empty()) {
    const cudaError_t e = cudaMemsetAsync(norm, 0, sizeof(float), s);
    return e == cudaSuccess ? FO_OK : host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  }
  void* part = nullptr;
  FO_TRY_HOST(host_buffer_kept(ctx, kSlotGradNorm, (1 + static_cast<size_t>(host_num_sms(ctx)) * kCtasPerSm) * 8, s,
                               &part));
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.part = static_cast<Wide*>(part);
  a.norm = norm;
  a.ctrl = host_ctrl(ctx);
  for (size_t i = 0; i < group->lists.size(); ++i) {
    const TensorList& l = group->lists[i];
    a.first = i == 0;
    a.last = i + 1 == group->lists.size();
    const int grid = grid_for(ctx, l.blocks);
    if (l.kind & kGrad32) {
      grad_norm_kernel<true><<<grid, kAdamThreads, 0, s>>>(l, a);
    } else {
      grad_norm_kernel<false><<<grid, kAdamThreads, 0, s>>>(l, a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  }
  return FO_OK;
}

fo_status fo_adamw_step(fo_ctx* ctx, const fo_adamw_group* group, const fo_adamw_params* prm, void* stream) {
  if (!group) return host_fail(FO_ERR_INVALID_ARG, "null group");
  if (!prm) return host_fail(FO_ERR_INVALID_ARG, "null parameters");
  if (!(prm->beta1 >= 0.0 && prm->beta1 < 1.0 && prm->beta2 >= 0.0 && prm->beta2 < 1.0))
    return host_fail(FO_ERR_INVALID_ARG, "beta1 and beta2 must be from 0 to below 1");
  if (!(prm->eps >= 0.f) || !std::isfinite(prm->eps))
    return host_fail(FO_ERR_INVALID_ARG, "eps must be finite and not negative");
  if ((!prm->lr_dev && !std::isfinite(prm->lr)) || !std::isfinite(prm->weight_decay) ||
      !std::isfinite(prm->grad_scale) || !std::isfinite(prm->max_norm))
    return host_fail(FO_ERR_INVALID_ARG, "lr, weight_decay, grad_scale and max_norm must be finite");
  if (!prm->step_dev && prm->step < 1)
    return host_failf(FO_ERR_INVALID_ARG, "step=%lld: the first is 1", (long long)prm->step);
  if (prm->max_norm > 0.f && !prm->norm) return host_fail(FO_ERR_INVALID_ARG, "max_norm needs norm");
  if (prm->stochastic != 0 && prm->stochastic != 1) return host_fail(FO_ERR_INVALID_ARG, "stochastic must be 0 or 1");
  if (prm->lr_dev) FO_TRY_HOST(check_ptr(prm->lr_dev, "lr_dev", 0, 4));
  if (prm->step_dev) FO_TRY_HOST(check_ptr(prm->step_dev, "step_dev", 0, 4));
  if (prm->norm) FO_TRY_HOST(check_ptr(prm->norm, "norm", 0, 4));
  FO_TRY_HOST(check_beside(group->written, prm->lr_dev, "lr_dev"));
  FO_TRY_HOST(check_beside(group->written, prm->step_dev, "step_dev"));
  FO_TRY_HOST(check_beside(group->written, prm->norm, "norm"));
  FO_TRY_HOST(host_check_ctx(ctx, 1));
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  StepArgs a;
  std::memset(&a, 0, sizeof(a));
  a.lr = prm->lr;
  a.exact1 = prm->beta1;
  a.exact2 = prm->beta2;
  a.beta1 = static_cast<float>(prm->beta1);
  a.beta2 = static_cast<float>(prm->beta2);
  a.rest1 = static_cast<float>(1.0 - prm->beta1);
  a.rest2 = static_cast<float>(1.0 - prm->beta2);
  a.one = 1.f;
  a.eps = prm->eps;
  a.weight_decay = prm->weight_decay;
  a.grad_scale = prm->grad_scale;
  a.max_norm = prm->max_norm;
  a.step = prm->step;
  if (!prm->step_dev) {
    const double t = static_cast<double>(prm->step);
    a.fix1 = static_cast<float>(1.0 / (1.0 - std::pow(prm->beta1, t)));
    a.fix2 = static_cast<float>(1.0 / (1.0 - std::pow(prm->beta2, t)));
  }
  a.seed_low = static_cast<uint32_t>(prm->seed);
  a.seed_high = static_cast<uint32_t>(prm->seed >> 32);
  a.lr_dev = prm->lr_dev;
  a.step_dev = prm->step_dev;
  a.norm = prm->norm;
  a.ctrl = host_ctrl(ctx);
  for (const TensorList& l : group->lists) {
    const int grid = grid_for(ctx, l.blocks, kStepThreads, l.kind & kStates8 ? kStepCtas8 : kStepCtas32);
    step_kernel(l.kind)<<<grid, kStepThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        l, a, prm->stochastic && !(l.kind & (kParam32 | kMaster)));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  }
  return FO_OK;
}

fo_status fo_adamw_unpack(fo_ctx* ctx, const fo_adamw_group* group, void* const* m, void* const* v, int dtype,
                          void* stream) try {
  if (!group) return host_fail(FO_ERR_INVALID_ARG, "null group");
  if (dtype != FO_BF16 && dtype != FO_F32) return host_failf(FO_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  const int count = static_cast<int>(group->tensors.size());
  if (count > 0 && (!m || !v)) return host_fail(FO_ERR_INVALID_ARG, "null tensor array");
  std::vector<Span> outs;
  outs.reserve(2 * group->tensors.size());
  for (int i = 0; i < count; ++i) {
    const int64_t n = group->tensors[i].n;
    if (!group->tensors[i].m_scale || n == 0) continue;
    FO_TRY_HOST(check_ptr(m[i], "m", i));
    FO_TRY_HOST(check_ptr(v[i], "v", i));
    outs.push_back(span_of(m[i], n * (dtype == FO_F32 ? 4 : 2), i, "m", true));
    outs.push_back(span_of(v[i], n * (dtype == FO_F32 ? 4 : 2), i, "v", true));
  }
  std::sort(outs.begin(), outs.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  for (size_t i = 0; i < outs.size(); ++i) {
    if (i > 0 && outs[i - 1].hi > outs[i].lo)
      return host_failf(FO_ERR_INVALID_ARG, "%s[%d] overlaps %s[%d]", outs[i].what, outs[i].tensor, outs[i - 1].what,
                        outs[i - 1].tensor);
    if (const Span* hit = group->used.meets(outs[i].lo, outs[i].hi))
      return host_failf(FO_ERR_INVALID_ARG, "%s[%d] overlaps the group's %s[%d]", outs[i].what, outs[i].tensor,
                        hit->what, hit->tensor);
  }
  FO_TRY_HOST(host_check_ctx(ctx, 1));
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  UnpackList l;
  for (int i = 0; i < count;) {
    std::memset(&l, 0, sizeof(l));
    for (; i < count && l.count < kListTensors; ++i) {
      const fo_adamw_tensor& t = group->tensors[i];
      if (!t.m_scale || t.n == 0) continue;
      l.first[l.count] = l.blocks;
      l.t[l.count++] = UnpackList::Ref{static_cast<const uint8_t*>(t.m), static_cast<const uint8_t*>(t.v), t.m_scale,
                                       t.v_range, m[i], v[i], t.n};
      l.blocks += blocks_of(t.n);
    }
    if (l.count == 0) break;
    const int grid = grid_for(ctx, l.blocks);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FO_F32) {
      unpack_kernel<float><<<grid, kAdamThreads, 0, s>>>(l);
    } else {
      unpack_kernel<uint16_t><<<grid, kAdamThreads, 0, s>>>(l);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  }
  return FO_OK;
} catch (...) {
  return host_fail(FO_ERR_OOM, "out of host memory");
}

}  // extern "C"

// Rotary positions: each pair (x1, x2) of a head's first rot_dim dimensions turns by the angle
// position * frequency,
//   y1 = A (x1 cos - x2 sin),  y2 = A (x2 cos + x1 sin),
// and the backward pass turns by the opposite angle (the rotation's transpose).
//
// Bound by HBM: the matrix is read and written once.  A CTA takes a few token rows, computes
// their cos / sin once into shared memory (they serve every head), then walks the heads with
// 16-byte accesses.  Angles: a frequency is a fraction of a turn per position, held as a 64-bit
// fixed-point number; position * fraction wraps modulo one turn by integer overflow.  The fraction
// is rounded to 2^-64, so the angle is off by position * 2^-65 of a turn (2^-34 at position 2^31)
// and by its rounding to fp32 for the sine and cosine, at most 2^-26 of a turn at any position (a
// product in fp32 would be off by 0.1 rad at position 2^20).  Measured: 16384 tokens of 40 heads of
// 128, bf16: 57 us (5.85 TB/s, 86% of a copy).
#include <cuda_bf16.h>

#include <cmath>
#include <cstring>

#include "fo_host.h"
#include "fo_internal.h"
#include "fo_ptx.cuh"

namespace fo {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = FO_ROPE_MAX_PAIRS;
constexpr int kRopeMaxRows = 8;  // token rows per CTA

struct RopeArgs {
  const void* x[kMaxP];
  void* y[kMaxP];
  int64_t ld_x[kMaxP], ld_y[kMaxP];
  const int32_t* positions[kMaxP];  // null: start + r * rank_stride + row
  int64_t start, rank_stride, m, total_rows;
  int32_t heads, dim, pairs, rows_per_cta;
  int32_t copy_rest;  // 1: dimensions behind rot_dim are copied (0: in place)
  float amp, sign;
  uint64_t turns[kRopeMaxPairs];
};

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int n = 8;
  __device__ static void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(q[k] << 16);
      v[2 * k + 1] = __uint_as_float(q[k] & 0xFFFF0000u);
    }
  }
  __device__ static void store(uint16_t* p, const float (&v)[8]) {
    st_v4_u32(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
  __device__ static float get(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
  __device__ static void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xFFFFu); }
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
  __device__ static void unpack(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
  __device__ static void store(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
  __device__ static float get(const float* p) { return *p; }
  __device__ static void put(float* p, float v) { *p = v; }
};

// A row of all ranks' rows: its rank and its place there
struct RowOf {
  int rk = 0;
  int64_t row;
  __device__ __forceinline__ RowOf(const RopeArgs& a, int64_t all) : row(all) {
    while (row >= a.m) {
      row -= a.m;
      ++rk;
    }
  }
};

// kVec: whole 16-byte vectors (half layout: rot_dim / 2 and head_dim multiples of the vector;
// interleaved: rot_dim and head_dim); otherwise pair by pair.
template <typename T, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 cs[];  // [rows_per_cta][pairs]: A cos, A sin
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows_per_cta;
  const int rows = static_cast<int>(a.total_rows - row0 < a.rows_per_cta ? a.total_rows - row0 : a.rows_per_cta);
  for (int i = threadIdx.x; i < rows * a.pairs; i += kRopeThreads) {
    const int q = i / a.pairs, f = i - q * a.pairs;
    const int rk = static_cast<int>((row0 + q) / a.m);
    const int64_t row = row0 + q - rk * a.m;
    const int32_t* given = a.positions[rk];
    const int64_t pos = given ? static_cast<int64_t>(given[row]) : a.start + rk * a.rank_stride + row;
    const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * a.turns[f]);  // in [-1/2, 1/2) of a turn
    float s, c;
    sincospif(__ll2float_rn(turn) * 0x1p-63f, &s, &c);
    cs[i] = make_float2(a.amp * c, a.amp * a.sign * s);
  }
  __syncthreads();
  constexpr int V = kVec ? Vec<T>::n : 1;
  // items of a head: turning vectors (half layout: one item turns a vector of each half), then
  // vectors behind rot_dim
  const int turning = kInterleaved ? (kVec ? 2 * a.pairs / V : a.pairs) : a.pairs / V;
  const int rest = a.copy_rest ? (a.dim - 2 * a.pairs) / V : 0;
  const int per_head = turning + rest, per_row = per_head * a.heads, total = rows * per_row;
  // Two items at a time, their loads first (in place no load may pass an earlier store by itself):
  // interleaved pairs 74 -> 66 us, fp32 72 -> 69 us at 16K and 8K tokens of 40 heads; the bf16 half
  // layout, which loads two vectors per item anyway, is faster with more threads resident (58 us).
  constexpr int kBatch = kVec && (kInterleaved || sizeof(T) == 4) ? 2 : 1;
  for (int i0 = threadIdx.x; i0 < total; i0 += kBatch * kRopeThreads) {
    const T* x[kBatch];
    T* y[kBatch];
    const float2* t[kBatch];
    int u[kBatch];
    uint4 raw[kBatch][2];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * kRopeThreads < total ? i0 + b * kRopeThreads : i0;
      const int q = i / per_row, j = i - q * per_row, h = j / per_head;
      u[b] = j - h * per_head;
      RowOf r(a, row0 + q);
      x[b] = static_cast<const T*>(a.x[r.rk]) + r.row * a.ld_x[r.rk] + static_cast<int64_t>(h) * a.dim;
      y[b] = static_cast<T*>(a.y[r.rk]) + r.row * a.ld_y[r.rk] + static_cast<int64_t>(h) * a.dim;
      t[b] = cs + q * a.pairs;
      if constexpr (kVec) {
        const int c = u[b] < turning ? u[b] * V : 2 * a.pairs + (u[b] - turning) * V;
        raw[b][0] = *reinterpret_cast<const uint4*>(x[b] + c);
        if (!kInterleaved && u[b] < turning) raw[b][1] = *reinterpret_cast<const uint4*>(x[b] + a.pairs + c);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (i0 + b * kRopeThreads >= total) break;
      if (u[b] >= turning) {
        const int c = 2 * a.pairs + (u[b] - turning) * V;
        if constexpr (kVec) {
          *reinterpret_cast<uint4*>(y[b] + c) = raw[b][0];
        } else {
          y[b][c] = x[b][c];
        }
      } else if constexpr (!kVec) {
        const int c1 = kInterleaved ? 2 * u[b] : u[b], c2 = kInterleaved ? 2 * u[b] + 1 : u[b] + a.pairs;
        const float2 w = t[b][u[b]];
        const float x1 = Vec<T>::get(x[b] + c1), x2 = Vec<T>::get(x[b] + c2);
        Vec<T>::put(y[b] + c1, x1 * w.x - x2 * w.y);
        Vec<T>::put(y[b] + c2, x2 * w.x + x1 * w.y);
      } else if constexpr (kInterleaved) {
        float v[V], o[V];
        Vec<T>::unpack(raw[b][0], v);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          const float2 w = t[b][u[b] * (V / 2) + k];
          o[2 * k] = v[2 * k] * w.x - v[2 * k + 1] * w.y;
          o[2 * k + 1] = v[2 * k + 1] * w.x + v[2 * k] * w.y;
        }
        Vec<T>::store(y[b] + u[b] * V, o);
      } else {
        float v1[V], v2[V];
        Vec<T>::unpack(raw[b][0], v1);
        Vec<T>::unpack(raw[b][1], v2);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float2 w = t[b][u[b] * V + k];
          const float o1 = v1[k] * w.x - v2[k] * w.y;
          v2[k] = v2[k] * w.x + v1[k] * w.y;
          v1[k] = o1;
        }
        Vec<T>::store(y[b] + u[b] * V, v1);
        Vec<T>::store(y[b] + a.pairs + u[b] * V, v2);
      }
    }
  }
}

template <typename T>
void launch(const RopeArgs& a, bool interleaved, bool vec, unsigned grid, int smem, cudaStream_t s) {
  if (interleaved) {
    vec ? rope_kernel<T, true, true><<<grid, kRopeThreads, smem, s>>>(a)
        : rope_kernel<T, true, false><<<grid, kRopeThreads, smem, s>>>(a);
  } else {
    vec ? rope_kernel<T, false, true><<<grid, kRopeThreads, smem, s>>>(a)
        : rope_kernel<T, false, false><<<grid, kRopeThreads, smem, s>>>(a);
  }
}

fo_status rope_run(fo_ctx* ctx, const fo_mat* X, int P, const fo_rope_table* table, int head_dim, int layout,
                   const int32_t* const* positions, int64_t start, int64_t rank_stride, const fo_mat* Y, float sign,
                   void* stream) {
  if (!X || !Y || !table) return host_fail(FO_ERR_INVALID_ARG, "null matrix array or table");
  if (P < 1 || P > kMaxP) return host_failf(FO_ERR_INVALID_ARG, "P=%d outside [1, %d]", P, kMaxP);
  if (layout != FO_ROPE_HALF && layout != FO_ROPE_INTERLEAVED)
    return host_failf(FO_ERR_INVALID_ARG, "unknown layout %d", layout);
  if (table->rot_dim < 2 || table->rot_dim % 2 != 0 || table->rot_dim > 2 * kRopeMaxPairs)
    return host_fail(FO_ERR_INVALID_ARG, "table not initialised (fo_rope_table_init)");
  if (head_dim < table->rot_dim)
    return host_failf(FO_ERR_SHAPE, "head_dim %d below the table's rot_dim %d", head_dim, table->rot_dim);
  const int64_t m = X[0].rows, cols = X[0].cols;
  const int32_t dtype = X[0].dtype;
  if (dtype != FO_BF16 && dtype != FO_F32) return host_fail(FO_ERR_INVALID_ARG, "X: unknown dtype");
  if (cols < 1 || cols % head_dim != 0)
    return host_failf(FO_ERR_SHAPE, "%lld columns are no whole number of heads of %d", (long long)cols, head_dim);
  if (cols > (1 << 26)) return host_fail(FO_ERR_UNSUPPORTED, "more than 2^26 columns");
  bool in_place = true;
  for (int r = 0; r < P; ++r) {
    FO_TRY_HOST(host_check_mat(X[r], dtype, "X", r));
    FO_TRY_HOST(host_check_mat(Y[r], dtype, "Y", r));
    if (X[r].rows != m || X[r].cols != cols || Y[r].rows != m || Y[r].cols != cols)
      return host_fail(FO_ERR_SHAPE, "X and Y must all have one shape");
    if (positions && !positions[r] && m > 0) return host_failf(FO_ERR_INVALID_ARG, "positions[%d]: null pointer", r);
    if (positions && reinterpret_cast<uintptr_t>(positions[r]) % 4 != 0)
      return host_failf(FO_ERR_UNSUPPORTED, "positions[%d]: not 4-byte aligned", r);
    in_place = in_place && host_same_view(X[r], Y[r]);
  }
  const HostList views[] = {{X, P, false, "X"}, {Y, P, true, "Y"}};
  const int over[][2] = {{1, 0}};
  FO_TRY_HOST(host_check_apart(views, 2, over, 1));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  if (m == 0) return FO_OK;
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  for (int r = 0; r < P; ++r) {
    a.x[r] = X[r].ptr;
    a.y[r] = Y[r].ptr;
    a.ld_x[r] = X[r].ld;
    a.ld_y[r] = Y[r].ld;
    a.positions[r] = positions ? positions[r] : nullptr;
  }
  a.start = start;
  a.rank_stride = rank_stride;
  a.m = m;
  a.total_rows = m * P;
  a.heads = static_cast<int32_t>(cols / head_dim);
  a.dim = head_dim;
  a.pairs = table->rot_dim / 2;
  a.copy_rest = in_place ? 0 : 1;
  a.amp = table->amplitude;
  a.sign = sign;
  std::memcpy(a.turns, table->turns, sizeof(a.turns[0]) * a.pairs);
  // a CTA's rows: enough pairs for its threads to compute, one row each while rows are few
  int rows = kRopeThreads / a.pairs;
  rows = rows < 1 ? 1 : rows > kRopeMaxRows ? kRopeMaxRows : rows;
  while (rows > 1 && (a.total_rows + rows - 1) / rows < 4 * host_num_sms(ctx)) rows /= 2;
  a.rows_per_cta = rows;
  const int64_t grid = (a.total_rows + rows - 1) / rows;
  if (grid > 0x7fffffffll) return host_fail(FO_ERR_UNSUPPORTED, "too many rows");
  const int v = dtype == FO_F32 ? 4 : 8;
  const bool vec = head_dim % v == 0 && (layout == FO_ROPE_INTERLEAVED ? 2 * a.pairs : a.pairs) % v == 0;
  const int smem = rows * a.pairs * static_cast<int>(sizeof(float2));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == FO_F32) {
    launch<float>(a, layout == FO_ROPE_INTERLEAVED, vec, static_cast<unsigned>(grid), smem, s);
  } else {
    launch<uint16_t>(a, layout == FO_ROPE_INTERLEAVED, vec, static_cast<unsigned>(grid), smem, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FO_OK : host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
}

// Numbers of about 100 bits as the sum of two doubles, |lo| at most half a step of hi: a frequency
// in double alone would be off by 2^-55 of a turn per position.  Sums and products are those of
// error-free transformations (Dekker, Knuth); every function below is host code.
struct Wide {
  double hi, lo;
};
Wide sum_of(double a, double b) {  // exact
  const double s = a + b, t = s - a;
  return Wide{s, (a - (s - t)) + (b - t)};
}
Wide product_of(double a, double b) {  // exact
  const double p = a * b;
  return Wide{p, std::fma(a, b, -p)};
}
Wide operator+(const Wide& a, const Wide& b) {
  const Wide s = sum_of(a.hi, b.hi), t = sum_of(a.lo, b.lo), u = sum_of(s.hi, s.lo + t.hi);
  return sum_of(u.hi, u.lo + t.lo);
}
Wide operator-(const Wide& a, const Wide& b) { return a + Wide{-b.hi, -b.lo}; }
Wide operator*(const Wide& a, const Wide& b) {
  const Wide p = product_of(a.hi, b.hi);
  return sum_of(p.hi, p.lo + (a.hi * b.lo + a.lo * b.hi));
}
Wide operator/(const Wide& a, const Wide& b) {
  const double q = a.hi / b.hi;
  const Wide r = a - b * Wide{q, 0.0};
  const double q2 = r.hi / b.hi;
  const Wide r2 = r - b * Wide{q2, 0.0};
  return sum_of(q, q2) + Wide{r2.hi / b.hi, 0.0};
}
// exp(x) = exp(x / 4096)^4096, |x| < 1000: 18 terms of the series leave less than 2^-90
Wide exp_of(const Wide& x) {
  const Wide r = {std::ldexp(x.hi, -12), std::ldexp(x.lo, -12)};
  Wide e = {1.0, 0.0};
  for (int k = 18; k > 0; --k) e = Wide{1.0, 0.0} + r * e / Wide{static_cast<double>(k), 0.0};
  for (int k = 0; k < 12; ++k) e = e * e;
  return e;
}
// ln(x), x from 1/2 to 2: one Newton step on exp(y) = x from the double
Wide near_log(double x) {
  const Wide y = {std::log(x), 0.0};
  return y + (Wide{x, 0.0} * exp_of(Wide{0.0, 0.0} - y) - Wide{1.0, 0.0});
}
Wide log_of(double x) {
  int e = 0;
  const double m = std::frexp(x, &e);
  return near_log(m) + Wide{static_cast<double>(e), 0.0} * near_log(2.0);
}
constexpr Wide kTwoPi = {6.283185307179586, 2.4492935982947064e-16};

// x modulo 1, times 2^64, rounded
uint64_t fixed_of(Wide x) {
  x = sum_of(x.hi - std::floor(x.hi), x.lo);
  const double scaled = std::ldexp(x.hi, 64), whole = std::floor(scaled);
  const int64_t rest = std::llrint((scaled - whole) + std::ldexp(x.lo, 64));
  // (just below a whole turn hi may be 1, just above one the sum may be negative: both wrap)
  const uint64_t w = whole >= 18446744073709551616.0 ? 0u
                     : whole < 0.0                   ? 0u - static_cast<uint64_t>(-whole)
                                                     : static_cast<uint64_t>(whole);
  return w + static_cast<uint64_t>(rest);
}

}  // namespace
}  // namespace fo

using namespace fo;

extern "C" {

fo_status fo_rope_table_init(fo_rope_table* table, int rot_dim, double base, const fo_rope_scaling* scaling) {
  if (!table) return host_fail(FO_ERR_INVALID_ARG, "null table");
  std::memset(table, 0, sizeof(*table));
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 2 * kRopeMaxPairs)
    return host_failf(FO_ERR_UNSUPPORTED, "rot_dim %d: an even number from 2 to %d", rot_dim, 2 * kRopeMaxPairs);
  if (!(base > 1.0) || !std::isfinite(base)) return host_fail(FO_ERR_INVALID_ARG, "base must be above 1");
  const int kind = scaling ? scaling->kind : FO_ROPE_UNSCALED;
  if (kind < FO_ROPE_UNSCALED || kind > FO_ROPE_RAMPED)
    return host_failf(FO_ERR_INVALID_ARG, "unknown scaling %d", kind);
  double factor = 1.0, length = 0.0, lo = 0.0, hi = 0.0;
  if (kind != FO_ROPE_UNSCALED) {
    factor = scaling->factor;
    if (!(factor > 0.0) || !std::isfinite(factor)) return host_fail(FO_ERR_INVALID_ARG, "factor must be positive");
  }
  double amplitude = 1.0;
  if (kind == FO_ROPE_BANDED || kind == FO_ROPE_RAMPED) {
    length = static_cast<double>(scaling->original_length);
    lo = scaling->low;
    hi = scaling->high;
    if (!(length > 0.0) || !(lo > 0.0) || !(hi > lo) || !std::isfinite(hi))
      return host_fail(FO_ERR_INVALID_ARG, "original_length must be positive and 0 < low < high");
  }
  double ramp0 = 0.0, ramp1 = 0.0;
  if (kind == FO_ROPE_RAMPED) {
    amplitude = factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0;
    // index of the pair that makes `turns` turns over original_length positions
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(length / (kTwoPi.hi * turns)) / (2.0 * std::log(base));
    };
    ramp0 = std::floor(pair_of(hi));
    ramp1 = std::ceil(pair_of(lo));
    if (ramp0 < 0.0) ramp0 = 0.0;
    if (ramp1 > rot_dim - 1.0) ramp1 = rot_dim - 1.0;
  }
  const Wide zero = {0.0, 0.0}, one = {1.0, 0.0}, per_turn = one / kTwoPi, per_factor = one / Wide{factor, 0.0};
  const Wide ratio = exp_of(Wide{-2.0, 0.0} / Wide{static_cast<double>(rot_dim), 0.0} * log_of(base));
  Wide f = one;
  for (int i = 0; i < rot_dim / 2; ++i, f = f * ratio) {
    Wide keep = zero;  // share of the unscaled frequency
    if (kind == FO_ROPE_UNSCALED) {
      keep = one;
    } else if (kind == FO_ROPE_BANDED) {
      keep = (Wide{length, 0.0} * f * per_turn - Wide{lo, 0.0}) / sum_of(hi, -lo);
    } else if (kind == FO_ROPE_RAMPED) {
      const double width = ramp1 - ramp0;
      keep = one - Wide{i - ramp0, 0.0} / Wide{width > 0.001 ? width : 0.001, 0.0};
    }
    if (keep.hi < 0.0) keep = zero;
    if (keep.hi > 1.0 || (keep.hi == 1.0 && keep.lo > 0.0)) keep = one;
    table->turns[i] = fixed_of(((one - keep) * f * per_factor + keep * f) * per_turn);
  }
  table->rot_dim = rot_dim;
  table->amplitude = static_cast<float>(amplitude);
  return FO_OK;
}

fo_status fo_rope(fo_ctx* ctx, const fo_mat* X, int P, const fo_rope_table* table, int head_dim, int layout,
                  const int32_t* const* positions, int64_t start, int64_t rank_stride, const fo_mat* Y,
                  void* stream) {
  return rope_run(ctx, X, P, table, head_dim, layout, positions, start, rank_stride, Y, 1.f, stream);
}

fo_status fo_rope_backward(fo_ctx* ctx, const fo_mat* dY, int P, const fo_rope_table* table, int head_dim,
                           int layout, const int32_t* const* positions, int64_t start, int64_t rank_stride,
                           const fo_mat* dX, void* stream) {
  return rope_run(ctx, dY, P, table, head_dim, layout, positions, start, rank_stride, dX, -1.f, stream);
}

}  // extern "C"

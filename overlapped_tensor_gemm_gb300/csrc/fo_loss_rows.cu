// Row kernels of the losses (formulas in fo_loss.cuh).
#include <cfloat>

#include "fo_loss.cuh"

namespace fo {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// exp(d) is 0 in fp32 from here on down: where d multiplies it, d ends here (0 times -infinity)
constexpr float kFarBelow = -128.f;

// 8 columns from p on
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(q[k] << 16);
    v[2 * k + 1] = __uint_as_float(q[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// Running statistics of some columns: m = max z (-infinity: none), s and t relative to it
struct Stat {
  float m, s, t;
};
// What is subtracted for a maximum m: finite also where every column is -infinity
__device__ __forceinline__ float base_of(float m) { return fmaxf(m, -FLT_MAX); }

template <bool kEnt>
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  const float base = base_of(r.m);
  // columns without a finite one have s = 0, whatever their factor
  const float da = base_of(a.m) - base, db = base_of(b.m) - base;
  const float ea = fast_exp2(da * kLog2e), eb = fast_exp2(db * kLog2e);
  r.s = a.s * ea + b.s * eb;
  r.t = kEnt ? ea * (a.t + a.s * da) + eb * (b.t + b.s * db) : 0.f;
  return r;
}

// The statistics of a whole row, in every thread
template <bool kEnt>
__device__ __forceinline__ Stat join_block(Stat v, Stat* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat w;
    w.m = __shfl_xor_sync(0xffffffffu, v.m, o);
    w.s = __shfl_xor_sync(0xffffffffu, v.s, o);
    w.t = kEnt ? __shfl_xor_sync(0xffffffffu, v.t, o) : 0.f;
    v = join<kEnt>(v, w);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __syncthreads();  // the last row's readers have left the buffer
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = buf[lane & (warps - 1)];
  for (int o = warps >> 1; o > 0; o >>= 1) {
    Stat w;
    w.m = __shfl_xor_sync(0xffffffffu, v.m, o);
    w.s = __shfl_xor_sync(0xffffffffu, v.s, o);
    w.t = kEnt ? __shfl_xor_sync(0xffffffffu, v.t, o) : 0.f;
    v = join<kEnt>(v, w);
  }
  return v;
}

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

// Whether row i counts; an id behind the vocabulary is reported (by one thread)
__device__ __forceinline__ bool counts(const LossArgs& a, int64_t i, int32_t y, bool report) {
  if (y >= a.first[a.P]) {
    if (report) note_error(a.ctrl, FO_ERR_RANGE, kSiteTargets, static_cast<uint32_t>(i));
    return false;
  }
  return y >= 0 && (!a.weights || a.weights[i] != 0.f);
}

// Sum of the counted rows' weights in the same order in every CTA (compensated: any number of rows)
__device__ __forceinline__ float total_weight(const LossArgs& a, float* buf) {
  float sum = 0.f, low = 0.f;
  for (int64_t i = threadIdx.x; i < a.rows; i += blockDim.x) {
    if (!counts(a, i, a.targets[i], false)) continue;
    const float x = (a.weights ? a.weights[i] : 1.f) - low, next = sum + x;
    low = (next - sum) - x;
    sum = next;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) buf[warp] = sum;
  __syncthreads();
  sum = buf[lane & (warps - 1)];
  for (int o = warps >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();
  return sum;
}

template <typename TZ, typename TD, int kMode, bool kEnt>
__global__ void __launch_bounds__(kLossThreads, 2) loss_rows_kernel(const __grid_constant__ LossArgs a) {
  __shared__ Stat buf[kLossThreads / 32];
  __shared__ float fbuf[kLossThreads / 32];
  __shared__ bool last;
  int64_t row0 = 0, rows = a.rows;
  if (a.offsets) {
    if (!offsets_fine(a.offsets, 2 * a.pairs + 1, a.rows, a.ctrl)) return;
    row0 = a.offsets[0];
    rows = a.offsets[2 * a.pairs];
  }
  float per_weight = 1.f;
  if (kMode == kLossPolicy && a.mean) {
    const float total = total_weight(a, fbuf);
    per_weight = total == 0.f ? 0.f : 1.f / total;
  }
  const bool grad = kMode != kLossForward && a.d[0];
  double sums[4] = {0.0, 0.0, 0.0, 0.0};  // thread 0: stats
  for (int64_t i = row0 + blockIdx.x; i < rows; i += gridDim.x) {
    const int32_t y = a.targets[i];
    const bool on = counts(a, i, y, kMode != kLossBackward && threadIdx.x == 0);
    if (!on) {
      if (kMode != kLossBackward && threadIdx.x == 0) {
        if (a.logp) a.logp[i] = 0.f;
        if (a.lse) a.lse[i] = 0.f;
        if (a.entropy) a.entropy[i] = 0.f;
        if (a.stat) a.stat[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (grad) {
        const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < a.P; ++r) {
          TD* d = static_cast<TD*>(a.d[r]) + i * a.ldd[r];
          for (int c = threadIdx.x * 8; c < a.cols[r]; c += kLossThreads * 8) {
            if (c + 8 <= a.cols[r]) {
              store8(d + c, zero);
            } else {
              for (int k = c; k < a.cols[r]; ++k) store1(d + k, 0.f);
            }
          }
        }
      }
      continue;
    }
    int ry = 0;
    while (y >= a.first[ry + 1]) ++ry;
    const int cy = y - a.first[ry];
    // the row's statistics: p_j = exp(z_j - base) * inv
    float base, inv, log_s, d_y, entropy = 0.f;
    if (kMode != kLossBackward) {
      // (read before join_block's barriers: a gradient over the logits may be written behind them)
      const float z_y = load1(static_cast<const TZ*>(a.z[ry]) + i * a.ldz[ry] + cy);
      Stat v = {-INFINITY, 0.f, 0.f};
      for (int r = 0; r < a.P; ++r) {
        const TZ* z = static_cast<const TZ*>(a.z[r]) + i * a.ldz[r];
        for (int c = threadIdx.x * 8; c < a.cols[r]; c += kLossThreads * 8) {
          float x[8];
          if (c + 8 <= a.cols[r]) {
            load8(z + c, x);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = c + k < a.cols[r] ? load1(z + c + k) : -INFINITY;
          }
          float top = x[0];
#pragma unroll
          for (int k = 1; k < 8; ++k) top = fmaxf(top, x[k]);
          top *= a.scale;
          if (top > v.m) {
            const float step = base_of(v.m) - base_of(top), e = fast_exp2(step * kLog2e);
            if (kEnt) v.t = e * (v.t + v.s * step);
            v.s *= e;
            v.m = top;
          }
          const float b = base_of(v.m);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float d = fmaf(x[k], a.scale, -b), e = fast_exp2(d * kLog2e);
            v.s += e;
            if (kEnt) v.t = fmaf(e, fmaxf(d, kFarBelow), v.t);
          }
        }
      }
      v = join_block<kEnt>(v, buf);
      base = base_of(v.m);
      inv = 1.f / v.s;
      log_s = logf(v.s);
      if (kEnt) entropy = log_s - v.t * inv;
      d_y = fmaf(z_y, a.scale, -base);
      if (threadIdx.x == 0) {
        if (a.logp) a.logp[i] = d_y - log_s;
        if (a.lse) a.lse[i] = base + log_s;
        if (a.entropy) a.entropy[i] = entropy;
        if (a.stat) a.stat[i] = make_float4(base, log_s, d_y, 0.f);
      }
    } else {
      const float4 st = a.stat ? a.stat[i] : make_float4(a.in_lse[i], 0.f, 0.f, 0.f);
      base = st.x;
      log_s = st.y;
      inv = a.stat ? expf(-log_s) : 1.f;
      if (kEnt) entropy = a.in_entropy[i];
    }
    // the loss through this row: a = dL/dlogp, h = dL/dH
    float da = 0.f, dh = 0.f;
    if (kMode == kLossPolicy) {
      const float lp = d_y - log_s, w = (a.weights ? a.weights[i] : 1.f) * per_weight, adv = a.advantages[i];
      const float ratio = expf(a.old_logp ? lp - a.old_logp[i] : 0.f);
      const float held = fminf(fmaxf(ratio, a.ratio_lo), a.ratio_hi) * adv, free = ratio * adv;
      const bool clipped = held < free;
      float kl = 0.f, dkl = 0.f;
      if (a.ref_logp) {
        const float x = a.ref_logp[i] - lp;
        dkl = expm1f(x);
        kl = dkl - x;
      }
      da = w * ((clipped ? 0.f : -free) - a.kl_coef * dkl);
      dh = -a.entropy_coef * w;
      if (threadIdx.x == 0) {
        const float loss = -(clipped ? held : free) + a.kl_coef * kl - a.entropy_coef * entropy;
        sums[0] += static_cast<double>(w) * loss;
        sums[1] += static_cast<double>(w) * kl;
        if (clipped) sums[2] += w;
        sums[3] += static_cast<double>(w) * entropy;
      }
    }
    if (kMode == kLossBackward) {
      if (a.coef) {
        int lo = 0, hi = 2 * a.pairs - 1;  // the sequence: the last one that starts at or in front of row i
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (a.offsets[mid] <= i) lo = mid; else hi = mid - 1;
        }
        da = a.coef[lo];
      } else {
        da = a.dlogp[i];
        if (kEnt) dh = a.dentropy[i];
      }
    }
    if (!grad) continue;
    const float own = a.scale * da;
    const float c0 = -a.scale * inv * (kEnt ? da + dh * (entropy - log_s) : da), c1 = -a.scale * inv * dh;
    for (int r = 0; r < a.P; ++r) {
      const TZ* z = static_cast<const TZ*>(a.z[r]) + i * a.ldz[r];
      TD* d = static_cast<TD*>(a.d[r]) + i * a.ldd[r];
      for (int c = threadIdx.x * 8; c < a.cols[r]; c += kLossThreads * 8) {
        const bool whole = c + 8 <= a.cols[r];
        float x[8];
        if (whole) {
          load8(z + c, x);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = c + k < a.cols[r] ? load1(z + c + k) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float dk = fmaf(x[k], a.scale, -base), e = fast_exp2(dk * kLog2e);
          x[k] = e * (kEnt ? fmaf(fmaxf(dk, kFarBelow), c1, c0) : c0);
        }
        if (r == ry && static_cast<uint32_t>(cy - c) < 8u) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k == cy) x[k] += own;
        }
        if (whole) {
          store8(d + c, x);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < a.cols[r]) store1(d + c + k, x[k]);
        }
      }
    }
  }
  if (kMode != kLossPolicy) return;
  // the CTA that comes last adds everyone's sums, in the order of the CTAs
  if (threadIdx.x == 0) {
    for (int k = 0; k < 4; ++k) a.part[blockIdx.x * 4 + k] = sums[k];
    __threadfence();
    last = atomicInc(a.ctrl + kCtrlDone, gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (last && threadIdx.x < 4) {
    __threadfence();
    double s = 0.0;
    for (unsigned b = 0; b < gridDim.x; ++b) s += __ldcg(a.part + b * 4 + threadIdx.x);
    a.stats[threadIdx.x] = static_cast<float>(s);
  }
}

template <typename TZ, typename TD>
cudaError_t launch(const LossArgs& a, const LossKind& k, int grid, cudaStream_t s) {
  void (*kernel)(LossArgs) = nullptr;
  if (k.mode == kLossPolicy) {
    kernel = k.entropy ? loss_rows_kernel<TZ, TD, kLossPolicy, true> : loss_rows_kernel<TZ, TD, kLossPolicy, false>;
  } else if (k.mode == kLossBackward) {
    kernel = k.entropy ? loss_rows_kernel<TZ, TD, kLossBackward, true> : loss_rows_kernel<TZ, TD, kLossBackward, false>;
  } else {  // writes no gradient: one type of it is enough
    kernel = k.entropy ? loss_rows_kernel<TZ, uint16_t, kLossForward, true>
                       : loss_rows_kernel<TZ, uint16_t, kLossForward, false>;
  }
  kernel<<<grid, kLossThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

int loss_rows_parts(int num_sms) { return 2 * num_sms; }

cudaError_t loss_rows_launch(const LossArgs& a, const LossKind& k, int num_sms, cudaStream_t s) {
  const int64_t most = loss_rows_parts(num_sms);
  const int grid = static_cast<int>(a.rows < 1 ? 1 : a.rows < most ? a.rows : most);
  if (k.z32) return k.d32 ? launch<float, float>(a, k, grid, s) : launch<float, uint16_t>(a, k, grid, s);
  return k.d32 ? launch<uint16_t, float>(a, k, grid, s) : launch<uint16_t, uint16_t>(a, k, grid, s);
}

}  // namespace fo

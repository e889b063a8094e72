// Norms before and after a block with gate and residual: forward (formulas in fo_norm.cuh).
#include "fo_norm.cuh"

namespace fo {
namespace {

// T: most threads of a CTA; 64 registers a thread, so 1024 threads share an SM.  kFull, kPlaced:
// what norm_fwd_kernel_of says, known while compiling.
template <typename TR, typename TA, typename TP, bool kVec, bool kFull, bool kPlaced, int T>
__global__ void __launch_bounds__(T, 1024 / T) norm_fwd_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float buf[2 * kSumBuf];
  __shared__ uint64_t bars[kNormMaxStages];
  int turn = 0;
  const int rpc = blockDim.x / a.tpr, t = threadIdx.x % a.tpr, sub = threadIdx.x / a.tpr;
  const bool has_y = kFull || a.has_y, post = kFull || a.w_post != nullptr, pre = kFull || a.pre;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  if (kPlaced) place_pars<TP>(a, smem, 0, a.w_post, a.gate);
  const float* const par = reinterpret_cast<const float*>(smem + a.par_off);
  Walk walk;
  walk.start(a, smem, bars, rpc);
  RowAt at{0, static_cast<int64_t>(blockIdx.x) * rpc + sub};
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rpc; row0 < a.total_rows; row0 += walk.step) {
    const uint8_t* st = walk.next(a, row0);
    if (!st) return;
    const bool live = kFull || row0 + sub < a.total_rows;
    if (live) at.wrap(a.m);
    Pair r[kC][4];
    float ss[1];
    float inv = 1.f;
    if (post) {
      Pair sq = 0;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int c = (i * a.tpr + t) * 8, n = kFull ? 8 : live ? a.cols - c : 0;
        if (n <= 0) continue;
        Pair y[4];
        get8<TA, kVec, kInY>(a, st, at, sub, c, n, y);
#pragma unroll
        for (int k = 0; k < 4; ++k) sq = ffma2(y[k], y[k], sq);
      }
      ss[0] = sum2(sq);
      row_sum<1>(ss, a.tpr, buf, turn);
      inv = rsqrtf(ss[0] * inv_cols + a.eps);
    }
    Pair sq = 0;
    const Pair inv2 = both(inv), alpha2 = both(a.alpha);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = (i * a.tpr + t) * 8, n = kFull ? 8 : live ? a.cols - c : 0;
      if (n <= 0) continue;
      get8<TR, kVec, kInR>(a, st, at, sub, c, n, r[i]);
      if (has_y) {
        Pair y[4], w[4];
        get8<TA, kVec, kInY>(a, st, at, sub, c, n, y);
        if (kFull) {
          if (kPlaced) {
            load8(par + c, 8, w);
          } else {
            pars8<TP, true>(a.w_post, a.gate, c, n, w);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = mul2(mul2(y[k], inv2), w[k]);
        } else {
          if (post) {
            par8<TP, kVec>(a.w_post, c, n, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = mul2(mul2(y[k], inv2), w[k]);
          }
          if (a.gate_mode != kGateNone) {
            if (a.gate_mode == kGateToken) {
              get8<TP, kVec, kInGate>(a, st, at, sub, c, n, w);
            } else {
              par8<TP, kVec>(a.gate, c, n, w);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = mul2(y[k], w[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) r[i][k] = ffma2(alpha2, r[i][k], y[k]);
        put8<TR, kVec>(a.r_out, a.ld_r_out, at, c, n, r[i]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) sq = ffma2(r[i][k], r[i][k], sq);
    }
    if (pre) {
      ss[0] = sum2(sq);
      row_sum<1>(ss, a.tpr, buf, turn);
      const Pair scale = both(rsqrtf(ss[0] * inv_cols + a.eps));
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int c = (i * a.tpr + t) * 8, n = kFull ? 8 : live ? a.cols - c : 0;
        if (n <= 0) continue;
        Pair w[4];
        par8<TP, kVec>(a.w_pre, c, n, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = mul2(mul2(r[i][k], scale), w[k]);
        put8<TA, kVec>(a.x, a.ld_x, at, c, n, w);
      }
    }
    at.row += walk.step;
  }
}

template <bool kVec, bool kFull, bool kPlaced, int T>
NormKernel of(bool r32, bool a32, bool p32) {
  typedef uint16_t H;
  constexpr bool kNarrow = kPlaced || kFull;  // 16-bit matrices always leave room for the parameters
  const int i = (r32 ? 4 : 0) + (a32 ? 2 : 0) + (p32 ? 1 : 0);
  const NormKernel k[8] = {norm_fwd_kernel<H, H, H, kVec, kFull, kNarrow, T>,
                           norm_fwd_kernel<H, H, float, kVec, kFull, kNarrow, T>,
                           norm_fwd_kernel<H, float, H, kVec, kFull, kPlaced, T>,
                           norm_fwd_kernel<H, float, float, kVec, kFull, kPlaced, T>,
                           norm_fwd_kernel<float, H, H, kVec, kFull, kPlaced, T>,
                           norm_fwd_kernel<float, H, float, kVec, kFull, kPlaced, T>,
                           norm_fwd_kernel<float, float, H, kVec, kFull, kPlaced, T>,
                           norm_fwd_kernel<float, float, float, kVec, kFull, kPlaced, T>};
  return k[i];
}

}  // namespace

NormKernel norm_fwd_kernel_of(bool r32, bool a32, bool p32, bool vec, bool full, bool placed, int threads) {
  if (full && threads <= 256)
    return placed ? of<true, true, true, 256>(r32, a32, p32) : of<true, true, false, 256>(r32, a32, p32);
  if (full) return placed ? of<true, true, true, 512>(r32, a32, p32) : of<true, true, false, 512>(r32, a32, p32);
  if (!vec)
    return threads <= 512 ? of<false, false, false, 512>(r32, a32, p32) : of<false, false, false, 1024>(r32, a32, p32);
  if (threads <= 256) return of<true, false, false, 256>(r32, a32, p32);
  return threads <= 512 ? of<true, false, false, 512>(r32, a32, p32) : of<true, false, false, 1024>(r32, a32, p32);
}

}  // namespace fo

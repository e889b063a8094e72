// Norms before and after a block with gate and residual: backward (formulas in fo_norm.cuh).
#include "fo_norm.cuh"

namespace fo {
namespace {

// Full forms have a post norm or not
enum Form { kAnyForm, kPlainForm, kPostForm };

// T: most threads of a CTA; up to 512 threads share an SM (128 registers each: 32 of them hold
// the sums over tokens).  One sum s = sum_tokens t u (u = Y / rms(Y), or Y) serves both the gate,
// dg = w_post s, and the post norm, dw_post = g s; a gate per token enters s itself.
// kForm, kPlaced: what norm_bwd_kernel_of says, known while compiling (tested for every row they
// cost 15%).
template <typename TR, typename TA, typename TP, bool kVec, Form kForm, bool kPlaced, int T>
__global__ void __launch_bounds__(T, T <= 512 ? 512 / T : 1) norm_bwd_kernel(const __grid_constant__ NormArgs a) {
  constexpr bool kFull = kForm != kAnyForm;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float buf[2 * kSumBuf];
  __shared__ uint64_t bars[kNormMaxStages];
  int turn = 0;
  const int rpc = blockDim.x / a.tpr, t = threadIdx.x % a.tpr, sub = threadIdx.x / a.tpr;
  const bool has_y = kFull || a.has_y, post = kFull ? kForm == kPostForm : a.w_post != nullptr, pre = kFull || a.pre;
  const bool has_dr = kFull || a.has_dr, token = !kFull && a.gate_mode == kGateToken;
  const bool placed = kPlaced || (kVec && !kFull && a.par_pitch != 0);
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  Pair acc[2][kC][4];  // sums over this thread's tokens: dw_pre, s
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[v][i][k] = 0;
  if (placed) {
    place_pars<TP>(a, smem, 0, a.w_pre, nullptr);
    place_pars<TP>(a, smem, 1, a.w_post, a.gate);
  }
  const float* const par = reinterpret_cast<const float*>(smem + a.par_off);
  auto w_pre8 = [&](int c, int n, Pair (&v)[4]) {
    if (placed) {
      load8(par + c, 8, v);
    } else {
      par8<TP, kVec>(a.w_pre, c, n, v);
    }
  };
  auto gw_post8 = [&](int c, int n, Pair (&v)[4]) {  // (the row gate's product with w_post)
    if (placed) {
      load8(par + a.par_pitch / 4 + c, 8, v);
    } else {
      pars8<TP, kVec>(a.w_post, a.gate, c, n, v);
    }
  };
  Walk walk;
  walk.start(a, smem, bars, rpc);
  RowAt at{0, static_cast<int64_t>(blockIdx.x) * rpc + sub};
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rpc; row0 < a.total_rows; row0 += walk.step) {
    const uint8_t* st = walk.next(a, row0);
    if (!st) return;
    const bool live = kFull || row0 + sub < a.total_rows;
    if (live) at.wrap(a.m);
    // sums of R'^2, dX w_pre R' and Y^2: everything the two norms need before t is known
    Pair q3[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = (i * a.tpr + t) * 8, n = kFull ? 8 : live ? a.cols - c : 0;
      if (n <= 0) continue;
      if (pre) {
        Pair r[4], dx[4], w[4];
        w_pre8(c, n, w);
        get8<TR, kVec, kInR>(a, st, at, sub, c, n, r);
        get8<TA, kVec, kInDx>(a, st, at, sub, c, n, dx);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          q3[0] = ffma2(r[k], r[k], q3[0]);
          q3[1] = ffma2(mul2(dx[k], w[k]), r[k], q3[1]);
        }
      }
      if (post) {
        Pair y[4];
        get8<TA, kVec, kInY>(a, st, at, sub, c, n, y);
#pragma unroll
        for (int k = 0; k < 4; ++k) q3[2] = ffma2(y[k], y[k], q3[2]);
      }
    }
    float s3[3] = {sum2(q3[0]), sum2(q3[1]), sum2(q3[2])};
    if (pre || post) row_sum<3>(s3, a.tpr, buf, turn);
    const float inv_r = pre ? rsqrtf(s3[0] * inv_cols + a.eps) : 0.f;
    const float mean_r = s3[1] * inv_r * inv_cols;  // mean(dX w_pre n)
    const float inv_y = post ? rsqrtf(s3[2] * inv_cols + a.eps) : 1.f;
    const Pair inv_r2 = both(inv_r), mean_r2 = both(-mean_r), inv_y2 = both(inv_y), alpha2 = both(a.alpha);
    Pair q1 = 0;
    Pair dr[kC][4];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = (i * a.tpr + t) * 8, n = kFull ? 8 : live ? a.cols - c : 0;
      if (n <= 0) continue;
      if (has_dr) {
        get8<TR, kVec, kInDr>(a, st, at, sub, c, n, dr[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) dr[i][k] = 0;
      }
      if (pre) {
        Pair r[4], dx[4], w[4];
        w_pre8(c, n, w);
        get8<TR, kVec, kInR>(a, st, at, sub, c, n, r);
        get8<TA, kVec, kInDx>(a, st, at, sub, c, n, dx);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const Pair nk = mul2(r[k], inv_r2);
          acc[0][i][k] = ffma2(dx[k], nk, acc[0][i][k]);
          dr[i][k] = ffma2(inv_r2, ffma2(nk, mean_r2, mul2(dx[k], w[k])), dr[i][k]);
        }
      }
      Pair o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = mul2(alpha2, dr[i][k]);
      put8<TR, kVec>(a.r_out, a.ld_r_out, at, c, n, o);
      if (!has_y) continue;
      // dr = t becomes dz w_post
      Pair y[4], w[4];
      get8<TA, kVec, kInY>(a, st, at, sub, c, n, y);
      if (post) {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = mul2(y[k], inv_y2);
      }
      if (token) {
        Pair g[4];
        if (post) {
          par8<TP, kVec>(a.w_post, c, n, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = mul2(dr[i][k], mul2(y[k], w[k]));  // t z
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = mul2(dr[i][k], y[k]);
        }
        put8<TP, kVec>(a.dgate, a.ld_dgate, at, c, n, o);
        get8<TP, kVec, kInGate>(a, st, at, sub, c, n, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) dr[i][k] = mul2(dr[i][k], g[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[1][i][k] = ffma2(dr[i][k], y[k], acc[1][i][k]);
      gw_post8(c, n, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dr[i][k] = mul2(dr[i][k], w[k]);
        q1 = ffma2(dr[i][k], y[k], q1);
      }
    }
    if (has_y) {
      Pair mean_y2 = 0;
      if (post) {
        float s1[1] = {sum2(q1)};
        row_sum<1>(s1, a.tpr, buf, turn);
        mean_y2 = both(-s1[0] * inv_cols * inv_y);
      }
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int c = (i * a.tpr + t) * 8, n = kFull ? 8 : live ? a.cols - c : 0;
        if (n <= 0) continue;
        if (post) {
          Pair y[4];
          get8<TA, kVec, kInY>(a, st, at, sub, c, n, y);
#pragma unroll
          for (int k = 0; k < 4; ++k) dr[i][k] = mul2(inv_y2, ffma2(y[k], mean_y2, dr[i][k]));
        }
        put8<TA, kVec>(a.x, a.ld_x, at, c, n, dr[i]);
      }
    }
    at.row += walk.step;
  }
  // column sums: the CTA's row groups in order, then one partial row per CTA and vector (a
  // fixed order: the same inputs give the same bits)
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 3 * a.cols;
  float* sums = reinterpret_cast<float*>(smem);  // [row groups][cols]: the stages are done with
#pragma unroll
  for (int v = 0; v < 3; ++v) {  // dw_pre, dgate = w_post s, dw_post = g s
    if (v == 0 ? !pre : v == 1 ? !(has_y && a.gate_mode == kGateRow) : !post) continue;
    float* out = rpc > 1 ? sums + sub * a.cols : part + v * a.cols;
    const TP* by = static_cast<const TP*>(v == 1 ? a.w_post : v == 2 ? a.gate : nullptr);
    if (rpc > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = (i * a.tpr + t) * 8, n = a.cols - c;
      if (n <= 0) continue;
      Pair w[4];
      pars8<TP, false>(by, nullptr, c, n, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = mul2(w[k], acc[v == 0 ? 0 : 1][i][k]);
      if constexpr (kVec) {
        store8(out + c, 8, w);
      } else {  // a row of sums starts at any multiple of 4 bytes
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x, y;
          unpack2(w[k], x, y);
          if (2 * k < n) out[c + 2 * k] = x;
          if (2 * k + 1 < n) out[c + 2 * k + 1] = y;
        }
      }
    }
    if (rpc > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float s = 0.f;
        for (int q = 0; q < rpc; ++q) s += sums[q * a.cols + c];
        part[v * a.cols + c] = s;
      }
    }
  }
}

template <bool kVec, Form kForm, bool kPlaced, int T>
NormKernel of(bool r32, bool a32, bool p32) {
  typedef uint16_t H;
  constexpr bool kNarrow = kPlaced || kForm != kAnyForm;  // 16-bit matrices always leave room for the parameters
  const int i = (r32 ? 4 : 0) + (a32 ? 2 : 0) + (p32 ? 1 : 0);
  const NormKernel k[8] = {norm_bwd_kernel<H, H, H, kVec, kForm, kNarrow, T>,
                           norm_bwd_kernel<H, H, float, kVec, kForm, kNarrow, T>,
                           norm_bwd_kernel<H, float, H, kVec, kForm, kPlaced, T>,
                           norm_bwd_kernel<H, float, float, kVec, kForm, kPlaced, T>,
                           norm_bwd_kernel<float, H, H, kVec, kForm, kPlaced, T>,
                           norm_bwd_kernel<float, H, float, kVec, kForm, kPlaced, T>,
                           norm_bwd_kernel<float, float, H, kVec, kForm, kPlaced, T>,
                           norm_bwd_kernel<float, float, float, kVec, kForm, kPlaced, T>};
  return k[i];
}

template <Form kForm>
NormKernel full_of(bool r32, bool a32, bool p32, bool placed, int threads) {
  if (threads <= 256) return of<true, kForm, true, 256>(r32, a32, p32);
  return placed ? of<true, kForm, true, 512>(r32, a32, p32) : of<true, kForm, false, 512>(r32, a32, p32);
}

}  // namespace

NormKernel norm_bwd_kernel_of(bool r32, bool a32, bool p32, bool vec, bool full, bool post, bool placed, int threads) {
  if (full)
    return post ? full_of<kPostForm>(r32, a32, p32, placed, threads)
                : full_of<kPlainForm>(r32, a32, p32, placed, threads);
  constexpr Form any = kAnyForm;
  if (!vec) return threads <= 512 ? of<false, any, false, 512>(r32, a32, p32) : of<false, any, false, 1024>(r32, a32, p32);
  if (threads <= 256) return of<true, any, false, 256>(r32, a32, p32);
  return threads <= 512 ? of<true, any, false, 512>(r32, a32, p32) : of<true, any, false, 1024>(r32, a32, p32);
}

}  // namespace fo

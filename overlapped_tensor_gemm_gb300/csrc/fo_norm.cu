// Norms before and after a block, fused with its gate and residual scale, and their backward.
//
//   z  = Y w_post / rms(Y)            (z = Y without a post norm),  rms(v) = sqrt(mean(v^2) + eps)
//   R' = a R + g z                    (the residual stream after the block)
//   X  = R' w_pre / rms(R')           (the next block's input)
//
// backward, from X's gradient dX and the gradient dR' that reaches R' by its other uses, with
// n = R' / rms(R'), u = Y / rms(Y):
//   t  = dR' + (dX w_pre - n mean(dX w_pre n)) / rms(R'),   dw_pre = sum_tokens dX n
//   dR = a t,   dg = t z (summed over tokens where g is one row),   dz = g t
//   dw_post = sum_tokens dz u,   dY = (dz w_post - u mean(dz w_post u)) / rms(Y)
//
// Both directions are bound by HBM: every matrix is read once and written once, a row stays in
// its threads' registers between the reductions and the stores.  `tpr` threads share a row,
// each with C groups of 8 columns (8-column group i*tpr + t); all arithmetic is fp32, each
// output is rounded once to its type (X from the unrounded R').
#include <cuda_bf16.h>

#include <cmath>
#include <cstring>

#include "fo_host.h"
#include "fo_internal.h"
#include "fo_ptx.cuh"

namespace fo {
namespace {

constexpr int kNormMaxCols = 16384;
constexpr int kNormThreads = 256;  // threads of a CTA where a row needs fewer

enum GateMode : int32_t { kGateNone = 0, kGateRow = 1, kGateToken = 2 };

struct NormArgs {
  const void* r[kMaxP];       // residual stream in (backward: R', after the block)
  const void* y[kMaxP];       // block output
  const void* gate[kMaxP];    // kGateToken: [m, H]; kGateRow: gate[0], one row
  void* r_out[kMaxP];         // forward: R'; backward: dR
  void* x[kMaxP];             // forward: X; backward: dY
  const void* dx[kMaxP];
  const void* dr_out[kMaxP];
  void* dgate[kMaxP];         // kGateToken
  int64_t ld_r[kMaxP], ld_y[kMaxP], ld_gate[kMaxP], ld_r_out[kMaxP], ld_x[kMaxP], ld_dx[kMaxP], ld_dr_out[kMaxP],
      ld_dgate[kMaxP];
  const void* w_post;
  const void* w_pre;
  int64_t m, total_rows;      // rows per rank, rows of all ranks
  int32_t cols, tpr, gate_mode;
  int32_t gate_f32, post_f32, pre_f32;  // types of the parameters (1: fp32, 0: bf16)
  float alpha, eps;
  float* part;                // backward: [grid][3][cols] column sums (pre, gate, post)
};

// 8 columns of a row from column c on, the first n of them inside the row (n >= 1)
__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(q[k] << 16);
      v[2 * k + 1] = __uint_as_float(q[k] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? __uint_as_float(static_cast<uint32_t>(p[k]) << 16) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? p[k] : 0.f;
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    st_v4_u32(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = static_cast<uint16_t>(pack_bf16x2(v[k], 0.f) & 0xFFFFu);
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = v[k];
  }
}
template <typename T>
__device__ __forceinline__ void load8_of(const void* base, int64_t off, int n, float (&v)[8]) {
  load8(static_cast<const T*>(base) + off, n, v);
}
// a parameter of either type (uniform branch; parameters other than per-token gates come from L1/L2)
__device__ __forceinline__ void load8_par(const void* base, int64_t off, int f32, int n, float (&v)[8]) {
  if (f32) {
    load8(static_cast<const float*>(base) + off, n, v);
  } else {
    load8(static_cast<const uint16_t*>(base) + off, n, v);
  }
}
__device__ __forceinline__ void store8_par(void* base, int64_t off, int f32, int n, const float (&v)[8]) {
  if (f32) {
    store8(static_cast<float*>(base) + off, n, v);
  } else {
    store8(static_cast<uint16_t*>(base) + off, n, v);
  }
}

constexpr int kSumBuf = 32 * 3;  // one half of row_sum's buffer: 32 warps, at most 3 values

// Sums of N values over the tpr threads of a row; every thread of the CTA takes part.  tpr is
// 32 or a multiple of it; with more than one warp per row the warps' sums meet in `buf`, of
// which successive calls use alternate halves (so one barrier per call is enough).
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float* buf, int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (tpr == 32) return;
  float* b = buf + turn * kSumBuf;
  turn ^= 1;
  const int warp = threadIdx.x >> 5, wpr = tpr >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) b[warp * N + k] = v[k];
  __syncthreads();
  const int w0 = warp / wpr * wpr;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  for (int w = 0; w < wpr; ++w)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += b[(w0 + w) * N + k];
}

template <typename TR, typename TA, int C>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float buf[2 * kSumBuf];
  int turn = 0;
  const int rpc = blockDim.x / a.tpr, t = threadIdx.x % a.tpr, sub = threadIdx.x / a.tpr;
  const bool has_y = a.y[0] != nullptr, post = a.w_post != nullptr, pre = a.x[0] != nullptr;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rpc; row0 < a.total_rows;
       row0 += static_cast<int64_t>(gridDim.x) * rpc) {
    const int64_t grow = row0 + sub;
    const bool live = grow < a.total_rows;
    const int rk = live ? static_cast<int>(grow / a.m) : 0;
    const int64_t row = live ? grow - rk * a.m : 0;
    float r[C][8], y[C][8];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = (i * a.tpr + t) * 8, n = live ? a.cols - c : 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i][k] = y[i][k] = 0.f;
      if (n > 0) {
        load8_of<TR>(a.r[rk], row * a.ld_r[rk] + c, n, r[i]);
        if (has_y) load8_of<TA>(a.y[rk], row * a.ld_y[rk] + c, n, y[i]);
      }
    }
    if (has_y) {
      float inv = 1.f;
      if (post) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) ss[0] = fmaf(y[i][k], y[i][k], ss[0]);
        row_sum<1>(ss, a.tpr, buf, turn);
        inv = 1.f / sqrtf(ss[0] * inv_cols + a.eps);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = (i * a.tpr + t) * 8, n = live ? a.cols - c : 0;
        if (n <= 0) continue;
        if (post) {
          float w[8];
          load8_par(a.w_post, c, a.post_f32, n, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[i][k] = y[i][k] * inv * w[k];
        }
        if (a.gate_mode != kGateNone) {
          float g[8];
          load8_par(a.gate[a.gate_mode == kGateToken ? rk : 0],
                    (a.gate_mode == kGateToken ? row * a.ld_gate[rk] : 0) + c, a.gate_f32, n, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[i][k] *= g[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) r[i][k] = fmaf(a.alpha, r[i][k], y[i][k]);
        store8(static_cast<TR*>(a.r_out[rk]) + row * a.ld_r_out[rk] + c, n, r[i]);
      }
    }
    if (pre) {
      ss[0] = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) ss[0] = fmaf(r[i][k], r[i][k], ss[0]);
      row_sum<1>(ss, a.tpr, buf, turn);
      const float inv = 1.f / sqrtf(ss[0] * inv_cols + a.eps);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = (i * a.tpr + t) * 8, n = live ? a.cols - c : 0;
        if (n <= 0) continue;
        float w[8];
        load8_par(a.w_pre, c, a.pre_f32, n, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = r[i][k] * inv * w[k];
        store8(static_cast<TA*>(a.x[rk]) + row * a.ld_x[rk] + c, n, w);
      }
    }
  }
}

template <typename TR, typename TA, int C>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float buf[2 * kSumBuf];
  extern __shared__ float sums[];  // [rows per CTA][cols]: column sums of the CTA's row groups
  int turn = 0;
  const int rpc = blockDim.x / a.tpr, t = threadIdx.x % a.tpr, sub = threadIdx.x / a.tpr;
  const bool has_y = a.y[0] != nullptr, post = a.w_post != nullptr, pre = a.dx[0] != nullptr;
  const bool has_dr = a.dr_out[0] != nullptr;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  float acc_pre[C][8], acc_gate[C][8], acc_post[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc_pre[i][k] = acc_gate[i][k] = acc_post[i][k] = 0.f;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rpc; row0 < a.total_rows;
       row0 += static_cast<int64_t>(gridDim.x) * rpc) {
    const int64_t grow = row0 + sub;
    const bool live = grow < a.total_rows;
    const int rk = live ? static_cast<int>(grow / a.m) : 0;
    const int64_t row = live ? grow - rk * a.m : 0;
    float r[C][8], y[C][8], dx[C][8], dr[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = (i * a.tpr + t) * 8, n = live ? a.cols - c : 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i][k] = y[i][k] = dx[i][k] = dr[i][k] = 0.f;
      if (n > 0) {
        if (pre) {
          load8_of<TR>(a.r[rk], row * a.ld_r[rk] + c, n, r[i]);
          load8_of<TA>(a.dx[rk], row * a.ld_dx[rk] + c, n, dx[i]);
        }
        if (has_y) load8_of<TA>(a.y[rk], row * a.ld_y[rk] + c, n, y[i]);
        if (has_dr) load8_of<TR>(a.dr_out[rk], row * a.ld_dr_out[rk] + c, n, dr[i]);
      }
    }
    // sums of R'^2, dX w_pre R' and Y^2: everything the two norms need before t is known
    float s3[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = (i * a.tpr + t) * 8, n = live ? a.cols - c : 0;
      if (n <= 0) continue;
      if (pre) {
        float w[8];
        load8_par(a.w_pre, c, a.pre_f32, n, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s3[0] = fmaf(r[i][k], r[i][k], s3[0]);
          s3[1] = fmaf(dx[i][k] * w[k], r[i][k], s3[1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s3[2] = fmaf(y[i][k], y[i][k], s3[2]);
    }
    row_sum<3>(s3, a.tpr, buf, turn);
    const float inv_r = pre ? 1.f / sqrtf(s3[0] * inv_cols + a.eps) : 0.f;
    const float mean_r = s3[1] * inv_r * inv_cols;  // mean(dX w_pre n)
    const float inv_y = post ? 1.f / sqrtf(s3[2] * inv_cols + a.eps) : 1.f;
    float s1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = (i * a.tpr + t) * 8, n = live ? a.cols - c : 0;
      if (n <= 0) continue;
      if (pre) {
        float w[8];
        load8_par(a.w_pre, c, a.pre_f32, n, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float nk = r[i][k] * inv_r;
          acc_pre[i][k] = fmaf(dx[i][k], nk, acc_pre[i][k]);
          dr[i][k] = fmaf(inv_r, dx[i][k] * w[k] - nk * mean_r, dr[i][k]);
        }
      }
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = a.alpha * dr[i][k];
      store8(static_cast<TR*>(a.r_out[rk]) + row * a.ld_r_out[rk] + c, n, o);
      if (!has_y) continue;
      // dr = t; y becomes u, dr becomes dz w_post
      float w[8], g[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = g[k] = 1.f;
      if (post) load8_par(a.w_post, c, a.post_f32, n, w);
      if (a.gate_mode != kGateNone)
        load8_par(a.gate[a.gate_mode == kGateToken ? rk : 0],
                  (a.gate_mode == kGateToken ? row * a.ld_gate[rk] : 0) + c, a.gate_f32, n, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        y[i][k] *= inv_y;
        o[k] = dr[i][k] * (y[i][k] * w[k]);  // t z
        acc_gate[i][k] += o[k];
        const float dz = dr[i][k] * g[k];
        acc_post[i][k] = fmaf(dz, y[i][k], acc_post[i][k]);
        dr[i][k] = dz * w[k];
        s1[0] = fmaf(dr[i][k], y[i][k], s1[0]);
      }
      if (a.gate_mode == kGateToken)
        store8_par(a.dgate[rk], row * a.ld_dgate[rk] + c, a.gate_f32, n, o);
    }
    if (has_y) {
      float mean_y = 0.f;
      if (post) {
        row_sum<1>(s1, a.tpr, buf, turn);
        mean_y = s1[0] * inv_cols;
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = (i * a.tpr + t) * 8, n = live ? a.cols - c : 0;
        if (n <= 0) continue;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = post ? inv_y * (dr[i][k] - y[i][k] * mean_y) : dr[i][k];
        store8(static_cast<TA*>(a.x[rk]) + row * a.ld_x[rk] + c, n, o);
      }
    }
  }
  // column sums: the CTA's row groups in order, then one partial row per CTA and vector (a
  // fixed order: the same inputs give the same bits)
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 3 * a.cols;
#pragma unroll
  for (int v = 0; v < 3; ++v) {
    float(&acc)[C][8] = v == 0 ? acc_pre : v == 1 ? acc_gate : acc_post;
    if (v == 0 ? !pre : v == 1 ? !(has_y && a.gate_mode == kGateRow) : !post) continue;
    if (rpc > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = (i * a.tpr + t) * 8 + k;
          if (c < a.cols) sums[sub * a.cols + c] = acc[i][k];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float s = 0.f;
        for (int q = 0; q < rpc; ++q) s += sums[q * a.cols + c];
        part[v * a.cols + c] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = (i * a.tpr + t) * 8 + k;
          if (c < a.cols) part[v * a.cols + c] = acc[i][k];
        }
    }
  }
}

// out_v[c] = sum over the partial rows, 32 columns per block (32 x 32 threads: coalesced reads,
// then a fixed-order sum through shared memory)
struct ColSumArgs {
  const float* part;
  void* out[3];
  int32_t f32[3];
  int32_t cols, rows;
};
__global__ void col_sum_kernel(const __grid_constant__ ColSumArgs a) {
  __shared__ float tile[32][33];
  const int v = blockIdx.y;
  if (!a.out[v]) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < a.cols)
    for (int r = threadIdx.y; r < a.rows; r += 32) s += a.part[(static_cast<int64_t>(r) * 3 + v) * a.cols + c];
  tile[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.cols) {
    s = 0.f;
    for (int r = 0; r < 32; ++r) s += tile[r][threadIdx.x];
    if (a.f32[v]) {
      static_cast<float*>(a.out[v])[c] = s;
    } else {
      static_cast<uint16_t*>(a.out[v])[c] = static_cast<uint16_t>(pack_bf16x2(s, 0.f) & 0xFFFFu);
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// threads per row: a multiple of 32 that covers the row with 8 C columns each
int threads_per_row(int64_t cols, int c) {
  int t = 32;
  while (static_cast<int64_t>(t) * 8 * c < cols) t *= 2;
  return t;
}

typedef void (*NormKernel)(const NormArgs);

template <int C>
NormKernel fwd_kernel(bool r32, bool a32) {
  return r32 ? (a32 ? norm_fwd_kernel<float, float, C> : norm_fwd_kernel<float, uint16_t, C>)
             : (a32 ? norm_fwd_kernel<uint16_t, float, C> : norm_fwd_kernel<uint16_t, uint16_t, C>);
}
template <int C>
NormKernel bwd_kernel(bool r32, bool a32) {
  return r32 ? (a32 ? norm_bwd_kernel<float, float, C> : norm_bwd_kernel<float, uint16_t, C>)
             : (a32 ? norm_bwd_kernel<uint16_t, float, C> : norm_bwd_kernel<uint16_t, uint16_t, C>);
}

// `list` (null: absent) as P matrices of one shape and type
fo_status check_list(const fo_mat* list, const char* what, int P, int64_t rows, int64_t cols, int32_t dtype) {
  if (!list) return FO_OK;
  for (int r = 0; r < P; ++r) {
    FO_TRY_HOST(host_check_mat(list[r], dtype, what, r));
    if (list[r].rows != rows || list[r].cols != cols)
      return host_failf(FO_ERR_SHAPE, "%s[%d] must be [%lld, %lld]", what, r, (long long)rows, (long long)cols);
  }
  return FO_OK;
}
fo_status check_vector(const fo_mat* v, const char* what, int64_t cols) {
  if (!v) return FO_OK;
  if (v->dtype != FO_BF16 && v->dtype != FO_F32) return host_failf(FO_ERR_INVALID_ARG, "%s: unknown dtype", what);
  FO_TRY_HOST(host_check_mat(*v, v->dtype, what, 0));
  if (v->rows != 1 || v->cols != cols) return host_failf(FO_ERR_SHAPE, "%s must be [1, %lld]", what, (long long)cols);
  return FO_OK;
}
fo_status check_dtype(const fo_mat& a, const char* what) {
  return a.dtype == FO_BF16 || a.dtype == FO_F32 ? FO_OK : host_failf(FO_ERR_INVALID_ARG, "%s: unknown dtype", what);
}

// No written matrix may meet another matrix of the call, but for one pair that a row's threads
// read before they write it (`in_place`, per rank).
struct View {
  const fo_mat* m;
  int n;
  bool written;
  const char* name;
};
fo_status check_apart(const View* v, int n, const int (*in_place)[2], int n_in_place) {
  for (int i = 0; i < n; ++i) {
    if (!v[i].m || !v[i].written) continue;
    for (int j = 0; j < n; ++j) {
      if (!v[j].m || (j == i && v[i].n == 1)) continue;
      for (int p = 0; p < v[i].n; ++p)
        for (int q = 0; q < v[j].n; ++q) {
          if (i == j && p == q) continue;
          if (!host_mats_overlap(v[i].m[p], v[j].m[q])) continue;
          bool fine = false;
          for (int k = 0; k < n_in_place; ++k)
            if (in_place[k][0] == i && in_place[k][1] == j && p == q && host_same_view(v[i].m[p], v[j].m[q]))
              fine = true;
          if (!fine)
            return host_failf(FO_ERR_INVALID_ARG, "%s[%d] overlaps %s[%d]", v[i].name, p, v[j].name, q);
        }
    }
  }
  return FO_OK;
}

struct NormCall {
  int64_t m = 0, cols = 0;
  int32_t tr = FO_BF16, ta = FO_BF16;
  int32_t gate_mode = kGateNone;
};

// What both directions share: the residual stream's and the activations' shapes and types, the
// parameters
fo_status check_norm(const fo_mat* R, const fo_mat* Y, const fo_mat* act2, int P, const fo_norm_params* prm,
                     NormCall* c) {
  if (P < 1 || P > kMaxP) return host_failf(FO_ERR_INVALID_ARG, "P=%d outside [1, %d]", P, kMaxP);
  if (!prm) return host_fail(FO_ERR_INVALID_ARG, "null parameters");
  if (!Y && !act2) return host_fail(FO_ERR_INVALID_ARG, "neither a block output nor a normed output");
  c->m = R[0].rows;
  c->cols = R[0].cols;
  c->tr = R[0].dtype;
  c->ta = Y ? Y[0].dtype : act2[0].dtype;
  FO_TRY_HOST(check_dtype(R[0], "residual"));
  FO_TRY_HOST(check_dtype(Y ? Y[0] : act2[0], "activations"));
  if (c->cols < 1) return host_fail(FO_ERR_SHAPE, "rows must have at least one column");
  if (c->cols > kNormMaxCols)
    return host_failf(FO_ERR_UNSUPPORTED, "%lld columns: at most %d", (long long)c->cols, kNormMaxCols);
  if (!(prm->eps >= 0.f) || !std::isfinite(prm->eps) || !std::isfinite(prm->residual_scale))
    return host_fail(FO_ERR_INVALID_ARG, "eps must be finite and not negative, residual_scale finite");
  FO_TRY_HOST(check_list(Y, "Y", P, c->m, c->cols, c->ta));
  FO_TRY_HOST(check_vector(prm->w_post, "w_post", c->cols));
  FO_TRY_HOST(check_vector(prm->w_pre, "w_pre", c->cols));
  if ((prm->w_pre != nullptr) != (act2 != nullptr))
    return host_fail(FO_ERR_INVALID_ARG, "w_pre goes with a normed output: both or neither");
  if (!Y && (prm->w_post || prm->gate || prm->residual_scale != 1.f))
    return host_fail(FO_ERR_INVALID_ARG, "w_post, gate and residual_scale need a block output");
  if (prm->gate) {
    if (prm->gate_per_token != 0 && prm->gate_per_token != 1)
      return host_fail(FO_ERR_INVALID_ARG, "gate_per_token must be 0 or 1");
    FO_TRY_HOST(check_dtype(prm->gate[0], "gate"));
    c->gate_mode = prm->gate_per_token ? kGateToken : kGateRow;
    if (prm->gate_per_token) {
      FO_TRY_HOST(check_list(prm->gate, "gate", P, c->m, c->cols, prm->gate[0].dtype));
    } else {
      FO_TRY_HOST(check_vector(prm->gate, "gate", c->cols));
    }
  }
  return FO_OK;
}

void fill(const fo_mat* list, int P, const void** ptr, int64_t* ld) {
  for (int r = 0; r < P && list; ++r) {
    ptr[r] = list[r].ptr;
    ld[r] = list[r].ld;
  }
}
void fill(const fo_mat* list, int P, void** ptr, int64_t* ld) {
  for (int r = 0; r < P && list; ++r) {
    ptr[r] = list[r].ptr;
    ld[r] = list[r].ld;
  }
}
void fill_common(NormArgs* a, const NormCall& c, int P, const fo_norm_params* prm) {
  std::memset(a, 0, sizeof(*a));
  a->m = c.m;
  a->total_rows = c.m * P;
  a->cols = static_cast<int32_t>(c.cols);
  a->gate_mode = c.gate_mode;
  if (prm->gate) {
    fill(prm->gate, prm->gate_per_token ? P : 1, a->gate, a->ld_gate);
    a->gate_f32 = prm->gate[0].dtype == FO_F32;
  }
  if (prm->w_post) {
    a->w_post = prm->w_post->ptr;
    a->post_f32 = prm->w_post->dtype == FO_F32;
  }
  if (prm->w_pre) {
    a->w_pre = prm->w_pre->ptr;
    a->pre_f32 = prm->w_pre->dtype == FO_F32;
  }
  a->alpha = prm->residual_scale;
  a->eps = prm->eps;
}

}  // namespace
}  // namespace fo

using namespace fo;

extern "C" {

fo_status fo_norm_residual(fo_ctx* ctx, const fo_mat* R, const fo_mat* Y, int P, const fo_norm_params* prm,
                           const fo_mat* R_out, const fo_mat* X, void* stream) {
  if (!R) return host_fail(FO_ERR_INVALID_ARG, "null matrix array");
  NormCall c;
  FO_TRY_HOST(check_norm(R, Y, X, P, prm, &c));
  if ((Y != nullptr) != (R_out != nullptr))
    return host_fail(FO_ERR_INVALID_ARG, "R_out goes with a block output: both or neither");
  FO_TRY_HOST(check_list(R, "R", P, c.m, c.cols, c.tr));
  FO_TRY_HOST(check_list(R_out, "R_out", P, c.m, c.cols, c.tr));
  FO_TRY_HOST(check_list(X, "X", P, c.m, c.cols, c.ta));
  const View views[] = {{R, P, false, "R"},         {Y, P, false, "Y"},
                        {R_out, P, true, "R_out"},  {X, P, true, "X"},
                        {prm->gate, prm->gate_per_token ? P : 1, false, "gate"},
                        {prm->w_post, 1, false, "w_post"}, {prm->w_pre, 1, false, "w_pre"}};
  const int in_place[][2] = {{2, 0}, {3, 1}};  // R_out over R, X over Y
  FO_TRY_HOST(check_apart(views, 7, in_place, 2));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  if (c.m == 0) return FO_OK;
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  NormArgs a;
  fill_common(&a, c, P, prm);
  fill(R, P, a.r, a.ld_r);
  fill(Y, P, a.y, a.ld_y);
  fill(R_out, P, a.r_out, a.ld_r_out);
  fill(X, P, a.x, a.ld_x);
  const bool r32 = c.tr == FO_F32, a32 = c.ta == FO_F32;
  const int cc = c.cols <= 256 ? 1 : 2;
  a.tpr = threads_per_row(c.cols, cc);
  const int threads = a.tpr > kNormThreads ? a.tpr : kNormThreads, rpc = threads / a.tpr;
  const int64_t blocks = (a.total_rows + rpc - 1) / rpc, cap = static_cast<int64_t>(host_num_sms(ctx)) * 16;
  const NormKernel k = cc == 1 ? fwd_kernel<1>(r32, a32) : fwd_kernel<2>(r32, a32);
  k<<<static_cast<unsigned>(blocks < cap ? blocks : cap), threads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FO_OK : host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
}

fo_status fo_norm_residual_backward(fo_ctx* ctx, const fo_mat* R_out, const fo_mat* Y, const fo_mat* dX,
                                    const fo_mat* dR_out, int P, const fo_norm_params* prm, const fo_mat* dR,
                                    const fo_mat* dY, const fo_norm_grads* grads, void* stream) {
  if (!R_out || !dR || !grads) return host_fail(FO_ERR_INVALID_ARG, "null matrix array");
  if (!dX && !dR_out) return host_fail(FO_ERR_INVALID_ARG, "neither dX nor dR_out");
  NormCall c;
  FO_TRY_HOST(check_norm(R_out, Y, dX, P, prm, &c));
  if ((Y != nullptr) != (dY != nullptr))
    return host_fail(FO_ERR_INVALID_ARG, "dY goes with a block output: both or neither");
  FO_TRY_HOST(check_list(R_out, "R_out", P, c.m, c.cols, c.tr));
  FO_TRY_HOST(check_list(dX, "dX", P, c.m, c.cols, c.ta));
  FO_TRY_HOST(check_list(dR_out, "dR_out", P, c.m, c.cols, c.tr));
  FO_TRY_HOST(check_list(dR, "dR", P, c.m, c.cols, c.tr));
  FO_TRY_HOST(check_list(dY, "dY", P, c.m, c.cols, c.ta));
  if ((grads->w_post != nullptr) != (prm->w_post != nullptr) || (grads->w_pre != nullptr) != (prm->w_pre != nullptr) ||
      (grads->gate != nullptr) != (prm->gate != nullptr))
    return host_fail(FO_ERR_INVALID_ARG, "every parameter of the call needs its gradient, and no other");
  FO_TRY_HOST(check_vector(grads->w_post, "dw_post", c.cols));
  FO_TRY_HOST(check_vector(grads->w_pre, "dw_pre", c.cols));
  const bool token = c.gate_mode == kGateToken;
  if (token) {
    FO_TRY_HOST(check_list(grads->gate, "dgate", P, c.m, c.cols, prm->gate[0].dtype));
  } else {
    FO_TRY_HOST(check_vector(grads->gate, "dgate", c.cols));
  }
  const View views[] = {{R_out, P, false, "R_out"}, {Y, P, false, "Y"},   {dX, P, false, "dX"},
                        {dR_out, P, false, "dR_out"}, {dR, P, true, "dR"}, {dY, P, true, "dY"},
                        {prm->gate, token ? P : 1, false, "gate"},
                        {prm->w_post, 1, false, "w_post"}, {prm->w_pre, 1, false, "w_pre"},
                        {grads->gate, token ? P : 1, true, "dgate"},
                        {grads->w_post, 1, true, "dw_post"}, {grads->w_pre, 1, true, "dw_pre"}};
  const int in_place[][2] = {{4, 3}, {5, 2}};  // dR over dR_out, dY over dX
  FO_TRY_HOST(check_apart(views, 12, in_place, 2));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NormArgs a;
  fill_common(&a, c, P, prm);
  fill(R_out, P, a.r, a.ld_r);
  fill(Y, P, a.y, a.ld_y);
  fill(dX, P, a.dx, a.ld_dx);
  fill(dR_out, P, a.dr_out, a.ld_dr_out);
  fill(dR, P, a.r_out, a.ld_r_out);
  fill(dY, P, a.x, a.ld_x);
  if (token) fill(grads->gate, P, a.dgate, a.ld_dgate);
  const bool r32 = c.tr == FO_F32, a32 = c.ta == FO_F32;
  const int cc = c.cols <= 256 ? 1 : 2;
  a.tpr = threads_per_row(c.cols, cc);
  const int threads = a.tpr > kNormThreads ? a.tpr : kNormThreads, rpc = threads / a.tpr;
  const int64_t blocks = (a.total_rows + rpc - 1) / rpc;
  const int64_t per_sm = threads >= 1024 ? 1 : threads >= 512 ? 1 : 2;
  const int64_t cap = static_cast<int64_t>(host_num_sms(ctx)) * per_sm;
  const int grid = static_cast<int>(blocks < cap ? blocks : cap);
  void* part = nullptr;
  FO_TRY_HOST(host_buffer_kept(ctx, kSlotNormPart, static_cast<size_t>(cap) * 3 * c.cols * 4, s, &part));
  a.part = static_cast<float*>(part);
  if (grid > 0) {
    const NormKernel k = cc == 1 ? bwd_kernel<1>(r32, a32) : bwd_kernel<2>(r32, a32);
    const int smem = rpc > 1 ? static_cast<int>(rpc * c.cols * 4) : 0;
    k<<<grid, threads, smem, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  }
  ColSumArgs cs;
  std::memset(&cs, 0, sizeof(cs));
  cs.part = a.part;
  cs.cols = a.cols;
  cs.rows = grid;
  const fo_mat* outs[3] = {grads->w_pre, token ? nullptr : grads->gate, grads->w_post};
  bool any = false;
  for (int v = 0; v < 3; ++v)
    if (outs[v]) {
      cs.out[v] = outs[v]->ptr;
      cs.f32[v] = outs[v]->dtype == FO_F32;
      any = true;
    }
  if (any) {
    col_sum_kernel<<<dim3((a.cols + 31) / 32, 3), dim3(32, 32), 0, s>>>(cs);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  }
  return FO_OK;
}

}  // extern "C"

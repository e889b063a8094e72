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
// Both directions are bound by HBM: every matrix is read once and written once.  A persistent CTA
// walks its rows; while it computes one, the next ones' matrices arrive in shared memory by bulk
// copies (cp.async.bulk, one mbarrier per stage), because a row is a chain of two reductions with
// little to overlap inside.  `tpr` threads share a row, 16 columns each (8-column groups t and
// tpr + t), and read it from shared memory again after each reduction: the sums over tokens take
// the registers.  All arithmetic is fp32, in packed pairs (two columns per instruction: with one,
// instruction issue took longer than the copies); each output is rounded once to its type (X
// from the unrounded R').  Measured, 16384 rows of 8192, all bf16: forward 171 us (6.3 TB/s),
// backward 287 us (5.6 TB/s).
#pragma once

#include <cuda_bf16.h>

#include "fo_attn_common.cuh"
#include "fo_internal.h"
#include "fo_ptx.cuh"

namespace fo {

constexpr int kNormMaxCols = 16384;
constexpr int kNormThreads = 256;             // threads of a CTA where a row needs fewer
constexpr int kNormSmem = 224 * 1024;         // shared memory of an SM that its CTAs may take
constexpr int kNormStatic = 2 * 1024;         // of it, per CTA: static and the system's
constexpr int kNormMaxStages = 4;

enum GateMode : int32_t { kGateNone = 0, kGateRow = 1, kGateToken = 2 };

// A matrix that the kernel reads.  Staged: the whole 16-byte vectors of its rows arrive in shared
// memory; a row's ragged end, and rows that are not staged, are read from global memory.
struct NormIn {
  const void* ptr[kMaxP];
  int64_t ld[kMaxP];          // elements
  uint32_t off, pitch;        // in a stage: first row, distance of rows (bytes)
  uint32_t bytes;             // copied per row (a multiple of 16; 0: not staged)
  int32_t esz;
};
enum InId : int { kInR = 0, kInY = 1, kInGate = 2, kInDx = 3, kInDr = 4, kIns = 5 };

struct NormArgs {
  NormIn in[kIns];            // backward: R = the residual stream after the block
  void* r_out[kMaxP];         // forward: R'; backward: dR
  void* x[kMaxP];             // forward: X; backward: dY
  void* dgate[kMaxP];         // kGateToken
  int64_t ld_r_out[kMaxP], ld_x[kMaxP], ld_dgate[kMaxP];
  const void* w_post;
  const void* w_pre;
  const void* gate;           // kGateRow
  int64_t m, total_rows;      // rows per rank, rows of all ranks
  int32_t cols, tpr, gate_mode, stages;
  uint32_t stage_bytes;
  uint32_t par_off, par_pitch;  // gate w_post (backward: w_pre, then it) in shared memory, fp32 (pitch 0: not)
  int32_t has_y, pre, has_dr;
  float alpha, eps;
  float* part;                // backward: [grid][3][cols] column sums (pre, gate, post)
  uint64_t timeout_ns;
  uint32_t* ctrl;
};

typedef void (*NormKernel)(const NormArgs);
// the kernel for rows of `threads` threads; vec: every matrix is staged and rows are whole groups
// of 8 columns
// full: a block's output and a norm behind it (backward: and a gradient of the residual stream)
// are given, the gate not per token, and rows fill their threads (at most 512); forward: with post
// norm and gate.  placed: the parameters lie in shared memory (backward, 256 threads: always)
NormKernel norm_fwd_kernel_of(bool r32, bool a32, bool p32, bool vec, bool full, bool placed, int threads);
NormKernel norm_bwd_kernel_of(bool r32, bool a32, bool p32, bool vec, bool full, bool post, bool placed, int threads);

namespace {

constexpr int kC = 2;  // 8-column groups per thread
typedef uint64_t Pair;  // two fp32 columns

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

// 8 columns of a row from column c on, the first n of them inside the row (n >= 1)
__device__ __forceinline__ void load8(const uint16_t* p, int n, Pair (&v)[4]) {
  uint32_t q[4];
  if (n >= 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    q[0] = w.x; q[1] = w.y; q[2] = w.z; q[3] = w.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      q[k] = (2 * k < n ? p[2 * k] : 0u) | (2 * k + 1 < n ? static_cast<uint32_t>(p[2 * k + 1]) << 16 : 0u);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = pack2(__uint_as_float(q[k] << 16), __uint_as_float(q[k] & 0xFFFF0000u));
}
__device__ __forceinline__ void load8(const float* p, int n, Pair (&v)[4]) {
  if (n >= 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = pack2(a.x, a.y); v[1] = pack2(a.z, a.w);
    v[2] = pack2(b.x, b.y); v[3] = pack2(b.z, b.w);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = pack2(2 * k < n ? p[2 * k] : 0.f, 2 * k + 1 < n ? p[2 * k + 1] : 0.f);
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int n, const Pair (&v)[4]) {
  uint32_t q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float x, y;
    unpack2(v[k], x, y);
    q[k] = pack_bf16x2(x, y);
  }
  if (n >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = static_cast<uint16_t>(q[k >> 1] >> (16 * (k & 1)));
  }
}
__device__ __forceinline__ void store8(float* p, int n, const Pair (&v)[4]) {
  float f[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) unpack2(v[k], f[2 * k], f[2 * k + 1]);
  if (n >= 8) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = f[k];
  }
}

// Where a row is: rank and row inside it; advances by a fixed number of rows
struct RowAt {
  int rk;
  int64_t row;
  __device__ __forceinline__ void wrap(int64_t m) {
    while (row >= m) {
      row -= m;
      ++rk;
    }
  }
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Warp 0: the copies of the row group that starts at row0, into the stage at `dst`
__device__ __forceinline__ void fill_stage(const NormArgs& a, uint8_t* dst, uint64_t* bar, int64_t row0, int rpc,
                                           int lane) {
  const int rows = static_cast<int>(a.total_rows - row0 < rpc ? a.total_rows - row0 : rpc);
  if (lane == 0) {
    uint32_t tx = 0;
#pragma unroll
    for (int i = 0; i < kIns; ++i) tx += a.in[i].bytes * rows;
    mbar_arrive_expect_tx(bar, tx);
  }
  __syncwarp();
  for (int k = lane; k < rows * kIns; k += 32) {
    const int i = k % kIns, q = k / kIns;
    const NormIn& in = a.in[i];
    if (in.bytes == 0) continue;
    RowAt r{0, row0 + q};
    r.wrap(a.m);
    bulk_load(dst + in.off + q * in.pitch, static_cast<const uint8_t*>(in.ptr[r.rk]) + r.row * in.ld[r.rk] * in.esz,
              in.bytes, bar);
  }
}

// 8 columns of matrix I in the thread's row; `here`: the row in the stage
template <typename T, bool kVec, int I>
__device__ __forceinline__ void get8(const NormArgs& a, const uint8_t* stage, const RowAt& r, int q, int c, int n,
                                     Pair (&v)[4]) {
  const NormIn& in = a.in[I];
  if (kVec || (in.bytes && n >= 8)) {
    load8(reinterpret_cast<const T*>(stage + in.off + q * in.pitch) + c, 8, v);
  } else {
    load8(static_cast<const T*>(in.ptr[r.rk]) + r.row * in.ld[r.rk] + c, n, v);
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ void par8(const void* base, int c, int n, Pair (&v)[4]) {
  load8(static_cast<const T*>(base) + c, kVec ? 8 : n, v);
}
// Parameters: 8 columns of f and, where it is there, times g (null f: ones).  Where there is room
// (par_pitch) the products lie in shared memory in fp32: read from L2 and unpacked anew for every
// row, the vectors of a wide row are as many bytes as the row itself.
template <typename T, bool kVec>
__device__ __forceinline__ void pars8(const void* f, const void* g, int c, int n, Pair (&v)[4]) {
  if (f) {
    par8<T, kVec>(f, c, n, v);
    if (!g) return;
    Pair w[4];
    par8<T, kVec>(g, c, n, w);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], w[k]);
  } else if (g) {
    par8<T, kVec>(g, c, n, v);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = both(1.f);
  }
}
// Called by every thread; Walk::start has the barrier behind it.
template <typename T>
__device__ __forceinline__ void place_pars(const NormArgs& a, uint8_t* smem, int k, const void* f, const void* g) {
  float* to = reinterpret_cast<float*>(smem + a.par_off + k * a.par_pitch);
  for (int c = threadIdx.x * 8; c < a.cols; c += blockDim.x * 8) {  // kVec: whole groups of 8
    Pair v[4];
    pars8<T, true>(f, g, c, 8, v);
    store8(to + c, 8, v);
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ void put8(void* const* base, const int64_t* ld, const RowAt& r, int c, int n,
                                     const Pair (&v)[4]) {
  store8(static_cast<T*>(base[r.rk]) + r.row * ld[r.rk] + c, kVec ? 8 : n, v);
}

// Waits, with a limit each, for the stages that are armed while the group at row0 is due in stage s
static __device__ __noinline__ void drain_stages(const NormArgs& a, uint64_t* bars, int s, uint32_t phase,
                                                 int64_t row0, int64_t step) {
  for (int k = 0; k < a.stages && row0 < a.total_rows; ++k, row0 += step) {
    mbar_wait_drain(&bars[s], phase, kAttnDrainNs);
    if (++s == a.stages) {
      s = 0;
      phase ^= 1u;
    }
  }
}

// The CTA's walk over its row groups: start() arms the first stages; next() waits for the group's
// stage and refills the one before it, which every thread has left.
struct Walk {
  uint8_t* base;
  uint64_t* bars;
  int64_t step;
  int rpc, s, phase;
  __device__ void start(const NormArgs& a, uint8_t* smem, uint64_t* b, int rows_per_cta) {
    base = smem;
    bars = b;
    rpc = rows_per_cta;
    step = static_cast<int64_t>(gridDim.x) * rpc;
    s = phase = 0;
    if (threadIdx.x == 0) {
      for (int k = 0; k < a.stages; ++k) mbar_init(&bars[k], 1);
      fence_barrier_init();
      fence_proxy_async_shared();
    }
    __syncthreads();
    if (threadIdx.x < 32)
      for (int k = 0; k < a.stages - 1; ++k) {
        const int64_t row = (static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(k) * gridDim.x) * rpc;
        if (row < a.total_rows) fill_stage(a, base + k * a.stage_bytes, &bars[k], row, rpc, threadIdx.x);
      }
  }
  __device__ const uint8_t* next(const NormArgs& a, int64_t row0) {
    __syncthreads();
    const int64_t row = row0 + step * (a.stages - 1);
    if (threadIdx.x < 32 && row < a.total_rows) {
      const int ahead = s == 0 ? a.stages - 1 : s - 1;
      fill_stage(a, base + ahead * a.stage_bytes, &bars[ahead], row, rpc, threadIdx.x);
    }
    // the copies depend on nothing but memory: an abort that an earlier call left behind does not
    // end this wait.  A warp gives up as a whole, and then waits for every copy in flight.
    const bool ok = __all_sync(0xffffffffu, mbar_try_wait(&bars[s], phase) ||
                                                mbar_wait_drain(&bars[s], phase, a.timeout_ns));
    if (!ok) {
      raise_error(a.ctrl, FO_ERR_TIMEOUT, kSiteFull, blockIdx.x);
      drain_stages(a, bars, s, phase, row0, step);
    }
    const uint8_t* here = base + s * a.stage_bytes;
    if (++s == a.stages) {
      s = 0;
      phase ^= 1;
    }
    return ok ? here : nullptr;
  }
};

constexpr int kSumBuf = 32 * 3;  // one half of row_sum's buffer: 32 warps, at most 3 values

// Sums of N values over the tpr threads of a row; every thread of the CTA takes part.  tpr is
// 32 times a power of two, or a multiple of 32 and the CTA's only row; with more than one warp per
// row the warps' sums meet in `buf`, of which successive calls use alternate halves (so one barrier
// per call is enough).
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float* buf, int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (tpr == 32) return;
  float* b = buf + turn * kSumBuf;
  turn ^= 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wpr = tpr >> 5;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) b[k * 32 + warp] = v[k];
  __syncthreads();
  const int w0 = (wpr & (wpr - 1)) == 0 ? warp & ~(wpr - 1) : 0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = lane < wpr ? b[k * 32 + w0 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
}

}  // namespace
}  // namespace fo

// What the attention kernels share: the tensor-memory form of the MMA, packed fp32 arithmetic,
// and (training kernels) the blocks of packed sequences.
#pragma once

#include <stdint.h>

#include "fo_internal.h"
#include "fo_ptx.cuh"

namespace fo {

// D (TMEM) += A (TMEM) * B (shared memory descriptor), A = [128 rows in lanes, 16
// 16-bit elements per 8 columns]: the form whose A operand never passes through
// shared memory.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Packed fp32 pairs (sm_100-family f32x2 instructions): two scores per instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Division by a number that the host knows, for 0 <= n < 2^31: with 2^(s-1) < d <= 2^s and
// mul = floor(2^(31+s) / d) + 1, mul d exceeds 2^(31+s) by at most d <= 2^s, so n mul / 2^(31+s)
// exceeds n / d by less than 1/d.  (A CTA's place from six divisions took 1000 cycles before its
// first load.)
struct FastDiv {
  uint32_t mul, shift;
  static FastDiv by(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return FastDiv{static_cast<uint32_t>((1ull << (31 + s)) / d + 1), 31 + s};
  }
  __host__ __device__ __forceinline__ int of(int n) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul >> shift);
  }
};

constexpr int kBlockInts = 8;        // a table entry: q0, q_len, k0, k_len, block, 3 unused

// One block of a sequence: its query rows q0 .. q0 + q_len and key rows k0 .. k0 + k_len, and
// the index of this block of `unit` rows inside it.
struct Block {
  int q0, q_len, k0, k_len, blk;
};

struct Blocks {           // how a kernel finds its blocks
  const int32_t* table;   // null: one sequence of mq queries and mk keys
  int32_t mq, mk, causal;
  int32_t count;          // entries without a table; upper bound with one
  int32_t unit, by_keys;  // rows per block; 1: blocks of key rows
};

// The e-th block; false past the last one.  Blocks with the most work come first: a causal
// sequence's last queries see the most keys, its first keys are seen by the most queries.
__device__ __forceinline__ bool block_at(const Blocks& b, int e, Block* out) {
  if (b.table) {  // e is inside the table's memory: entry and count are read at once
    const int32_t* t = b.table + kBlockInts * (1 + static_cast<int64_t>(e));
    const int4 w = *reinterpret_cast<const int4*>(t);
    const int blk = t[4], n = b.table[0];
    *out = Block{w.x, w.y, w.z, w.w, blk};
    return e < n;
  }
  if (e >= b.count) return false;
  *out = Block{0, b.mq, 0, b.mk, b.by_keys ? e : b.count - 1 - e};
  return true;
}

// Keys that queries [q, q + n) of a sequence see: [0, key_end)
__host__ __device__ __forceinline__ int key_end(int causal, int q_end, int q_len, int k_len) {
  if (!causal) return k_len;
  const int e = q_end + (k_len - q_len);
  return e < 0 ? 0 : e > k_len ? k_len : e;
}
// Queries that see a key of [k, ...): [query_begin, q_len)
__host__ __device__ __forceinline__ int query_begin(int causal, int k, int q_len, int k_len) {
  if (!causal) return 0;
  const int q = k - (k_len - q_len);
  return q < 0 ? 0 : q > q_len ? q_len : q;
}

// Arguments of the training kernels: P independent ranks of one shape.
struct TrainArgs {
  // per rank r: Q = r, K = P + r, V = 2P + r, dO = 3P + r (boxes of 64 columns x 128 rows)
  CUtensorMap maps[4 * kMaxP];
  const uint16_t *o[kMaxP], *d_o[kMaxP];
  uint16_t *out_o[kMaxP], *dq[kMaxP], *dk[kMaxP], *dv[kMaxP];
  float* lse[kMaxP];
  int64_t ld_o[kMaxP], ld_do[kMaxP], ld_lse[kMaxP], ld_dq[kMaxP], ld_dk[kMaxP], ld_dv[kMaxP];
  float* delta;                 // backward: [P][heads][mq]
  // Backward, a block's walk cut into `splits` parts (1: not cut): part s of rank r writes its
  // fp32 sums to part[((s * P + r) * rows + row) * cols + col] (dV: part_v), which are added after
  int32_t splits;
  float *part, *part_v;
  int32_t short_walks;          // some walks may be short (kFineWalk)
  int32_t delta_mode;           // dQ: a DeltaMode
  float* eps;                   // kDeltaMeasure: [splits][P][heads][mq]
  Blocks blocks;
  int32_t P, heads, kv_heads;
  FastDiv by_q[2], by_k[2], by_group, by_splits;  // heads * P and heads; kv_heads * P and kv_heads
  int32_t mq;
  float scale, scale_log2;      // of the scores; times log2(e)
  uint64_t timeout_ns;
  uint32_t* ctrl;
};

constexpr uint64_t kAttnDrainNs = 200ull * 1000 * 1000;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBlk = 128;                     // queries or keys per block
constexpr uint32_t kHalf = kBlk * 128;        // 64 columns of a block: 128 rows of one 128-byte swizzle atom

// A whole warp waits: every lane tests the phase (one broadcast access, no exchange between
// lanes), only a phase that is not complete yet takes lane 0 into the bounded loop.
__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, const TrainArgs& p, uint32_t site, int lane) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  uint32_t ok = 0;
  if (lane == 0) ok = mbar_wait(bar, parity, p.ctrl, p.timeout_ns, site, blockIdx.x) ? 1u : 0u;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// One block of a [rows, heads * D] matrix: D / 64 boxes of 64 columns, one after the other
template <int D>
__device__ __forceinline__ void load_block(const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int col, int row) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_2d(map, dst + c * kHalf, bar, col + c * 64, row);
}

// Loads a block whose rows are terms of a sum; called by a whole warp.  The block's `full`
// barrier completes once it is in place; with rows behind the sequence (valid < 128) the load
// completes on `fix` first and the rows are cleared.  False when that wait gave up.
template <int D>
__device__ bool load_summed(const TrainArgs& p, const CUtensorMap* map, uint8_t* dst, uint64_t* full, uint64_t* fix,
                            uint32_t& fix_uses, int col, int row, int valid, int lane) {
  uint64_t* bar = valid < kBlk ? fix : full;
  if (lane == 0) {
    mbar_arrive_expect_tx(bar, D / 64 * kHalf);
    load_block<D>(map, dst, bar, col, row);
  }
  if (valid >= kBlk) return true;
  const uint32_t parity = fix_uses & 1u;
  ++fix_uses;
  if (!attn_wait(fix, parity, p, kSiteFull, lane)) {
    if (lane == 0) mbar_wait_drain(fix, parity, kAttnDrainNs);
    return false;
  }
  for (int c = 0; c < D / 64; ++c)
    for (int i = valid * 8 + lane; i < kBlk * 8; i += 32)
      *reinterpret_cast<uint4*>(dst + c * kHalf + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) mbar_arrive(full);
  return true;
}

// True for one lane of a converged warp, the same one every time.  The compiler knows that code
// under it runs in one thread, and issuing an MMA takes less of it: 40 cycles per small MMA in a
// loop of its own, 46 under `lane == 0`, 68 predicated; on a warp that competes with the softmax
// warps for issue slots it made the kernels 10-20% faster.
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r != 0;
}

// One MMA with the accumulation known at compile time.
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "n"(kAdd ? 1 : 0)
      : "memory");
}

// D[128 x 128] = A B^T over the D head dimensions, both operands K-major tiles (shared memory
// offsets enter a descriptor in units of 16 bytes)
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint32_t a, uint32_t b) {
  constexpr uint32_t idesc = umma_idesc_bf16(128, 128);
  const uint64_t ad = umma_sdesc_sw128(a), bd = umma_sdesc_sw128(b);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
    if (k == 0) {
      mma_ss<false>(d_tmem, ad, bd, idesc);
    } else {
      mma_ss<true>(d_tmem, ad + off, bd + off, idesc);
    }
  }
}

// D[128 x D] += A B over 128 summed rows: A bf16 in TMEM (rows kPart h + 2c, kPart h + 2c + 1 of the
// sum in column kPart h + c: each group of kPart score columns, overwritten in its first half), B the
// tile's rows as they lie (MN-major)
template <int D, int kPart>
__device__ __forceinline__ void issue_grad(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, bool first) {
  constexpr uint32_t idesc = umma_idesc_bf16_bmn(128, D);
  const uint64_t bd = umma_sdesc_sw128_mn(b, kHalf);
#pragma unroll
  for (int k = 0; k < kBlk / 16; ++k)
    umma_ts(d_tmem, a_tmem + k * 16 / kPart * kPart + k * 16 % kPart / 2, bd + k * (2048 >> 4), idesc,
            first && k == 0 ? 0u : 1u);
}

// Weights and dS enter their products as bf16.  Over many keys the roundings average out; in a
// short sequence (a walk of at most kFineWalk blocks) a single weight's rounding reaches a whole
// row of the result.  There they are split into two bf16 parts, both multiplied: the products are
// then as exact as the fp32 sums, and so short a walk is bound by latency, not by the tensor pipe.
// Instantiations with kShort look at each walk; long single sequences run those without (the test
// and its code cost their loops 4%).
constexpr int kFineWalk = 2;
// what bf16 leaves of a pair whose rounding is `hi`
__device__ __forceinline__ uint32_t rest_bf16x2(float a, float b, uint32_t hi) {
  return pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}

__device__ __forceinline__ void attn_publish(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// 16 columns of this warp's lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// A warp's 32 accumulator rows, N columns from col0 on, times `scale`, to the first `rows` rows of a
// matrix at `out` (16-byte aligned rows); zero: nothing was accumulated.  `stage`: 32 * N * sizeof(T)
// bytes of shared memory that nothing reads any more.  A thread's row is turned there, so that a
// store covers whole lines: with each lane storing its own row (32 lines per instruction) a tile's
// rows took 2300 cycles.  16-byte pieces change places inside a row by the row's index (no bank
// conflicts in either direction).
template <int N, typename T>
__device__ __forceinline__ void attn_store_rows(uint32_t taddr, int col0, float scale, uint8_t* stage, T* out,
                                                int64_t ld, int rows, bool zero) {
  constexpr int kPieces = N * static_cast<int>(sizeof(T)) / 16, kPer = 16 / static_cast<int>(sizeof(T));
  static_assert(kPieces == 4 || kPieces == 8 || kPieces == 16, "pieces of a row");
  auto at = [&](int row, int piece) {
    return reinterpret_cast<uint4*>(stage + (row * kPieces + (piece ^ (kPieces == 4 ? row >> 1 & 3 : row & 7))) * 16);
  };
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = 0; c < N; c += 32) {
    uint32_t v[32];
    if (zero) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = 0u;
    } else {
      tmem_ld32(taddr + col0 + c, v);
      tmem_wait_ld();
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * scale);
#pragma unroll
    for (int k = 0; k < 32 / kPer; ++k) {
      uint4 w;
      if constexpr (sizeof(T) == 4) {
        w = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      } else {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[i] = pack_bf16x2(__uint_as_float(v[8 * k + 2 * i]), __uint_as_float(v[8 * k + 2 * i + 1]));
        w = make_uint4(q[0], q[1], q[2], q[3]);
      }
      *at(lane, c / kPer + k) = w;
    }
  }
  __syncwarp();
#pragma unroll 4
  for (int i = 0; i < kPieces; ++i) {
    const int row = (i * 32 + lane) / kPieces, piece = lane % kPieces;
    if (row < rows) *reinterpret_cast<uint4*>(out + row * ld + piece * kPer) = *at(row, piece);
  }
  __syncwarp();  // the stage may be written again
}

// What the dQ pass does about delta's error (see there)
enum DeltaMode : int32_t { kDeltaCorrect = 0, kDeltaMeasure = 1, kDeltaGiven = 2 };

// fo_attn_fwd.cu
cudaError_t attn_fwd_configure();
cudaError_t attn_fwd_launch(const TrainArgs& a, int dim, cudaStream_t s);
// fo_attn_bwd.cu
cudaError_t attn_bwd_configure();
cudaError_t attn_delta_launch(const TrainArgs& a, int dim, cudaStream_t s);
cudaError_t attn_delta_add_launch(const TrainArgs& a, cudaStream_t s);  // delta += sum over the parts of eps
cudaError_t attn_dkv_launch(const TrainArgs& a, int dim, cudaStream_t s);
cudaError_t attn_dq_launch(const TrainArgs& a, int dim, cudaStream_t s);
// out[r][row, col] = sum over the parts, rounded to bf16, for the rows of the sequences
struct PartSumArgs {
  const float* part[2];
  uint16_t* out[2][kMaxP];
  int64_t ld_out[2][kMaxP];
  int64_t rows;
  int32_t cols, splits, P, outputs;
  const int32_t* off;           // packed sequences: their first and last boundary
  const int32_t* table;         // and their block table (empty: nothing was computed)
  int32_t n;
};
cudaError_t attn_part_sum_launch(const PartSumArgs& a, cudaStream_t s);

}  // namespace fo

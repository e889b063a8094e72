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
  if (b.table) {
    if (e >= b.table[0]) return false;
    const int32_t* t = b.table + kBlockInts * (1 + e);
    *out = Block{t[0], t[1], t[2], t[3], t[4]};
    return true;
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
  const uint16_t *q[kMaxP], *k[kMaxP], *v[kMaxP];
  int64_t ld_q[kMaxP], ld_k[kMaxP], ld_v[kMaxP];
  const uint16_t *o[kMaxP], *d_o[kMaxP];
  uint16_t *out_o[kMaxP], *dq[kMaxP], *dk[kMaxP], *dv[kMaxP];
  float* lse[kMaxP];
  int64_t ld_o[kMaxP], ld_do[kMaxP], ld_lse[kMaxP], ld_dq[kMaxP], ld_dk[kMaxP], ld_dv[kMaxP];
  float* delta;                 // backward: [P][heads][mq]
  Blocks blocks;
  int32_t P, heads, kv_heads;
  int32_t mq;
  float scale, scale_log2;      // of the scores; times log2(e)
  uint64_t timeout_ns;
  uint32_t* ctrl;
};

// fo_attn_bwd.cu
cudaError_t attn_bwd_configure();
cudaError_t attn_delta_launch(const TrainArgs& a, int dim, cudaStream_t s);
cudaError_t attn_dkv_launch(const TrainArgs& a, int dim, cudaStream_t s);
cudaError_t attn_dq_launch(const TrainArgs& a, int dim, cudaStream_t s);

}  // namespace fo

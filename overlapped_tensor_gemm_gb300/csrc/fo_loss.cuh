// Losses from the logits of a column-parallel output projection, and their gradients.
//
// A row of logits lies in P matrices, each rank's columns of the vocabulary.  With z = scale times
// the logits and m = max z, all in fp32:
//   d_j = z_j - m,  s = sum exp d,  logp = d_y - log s,  lse = m + log s,
//   H = log s - (sum exp(d) d) / s,   p_j = exp(d_j) / s,
//   d logp / dz_j = 1[j = y] - p_j,   d H / dz_j = -p_j (d_j - log s + H).
// A loss enters a row's gradient through two numbers, a = dL/dlogp and h = dL/dH:
//   dz_j = a 1[j = y] - p_j (a + h (d_j - log s + H)).
#pragma once

#include <cuda_bf16.h>

#include "fo_attn_common.cuh"
#include "fo_internal.h"
#include "fo_loss_cut.h"
#include "fo_ptx.cuh"

namespace fo {

constexpr int kLossChunk = 32768;   // bytes of a copy

enum LossMode : int {
  kLossForward = 0,   // statistics alone
  kLossPolicy = 1,    // statistics, the policy loss, and (LossArgs::gradient) the gradient
  kLossBackward = 2   // the gradient, from statistics given
};

struct LossArgs {
  const void* z[kMaxP];
  void* d[kMaxP];             // null where a rank has no columns, or no gradient is wanted
  int64_t ldz[kMaxP], ldd[kMaxP];
  int32_t cols[kMaxP];
  int32_t first[kMaxP + 1];   // vocabulary ids: rank r has first[r] .. first[r + 1]
  int32_t groups[kMaxP + 1];  // the whole 16-byte groups of columns: rank r has groups[r] .. groups[r + 1]
  int32_t ctas;               // CTAs of one row: each takes a range of the groups
  int32_t twice;              // a CTA's range does not fit: it is copied again for the gradient
  int32_t backwards;          // rows from the last one on
  int32_t gradient;           // whether a gradient is wanted
  int32_t P;
  int64_t rows;
  float scale;
  const int32_t* targets;
  float* logp;                // outputs, each may be null
  float* lse;
  float* entropy;
  float4* stat;               // (m, log2 s, logp in twice fp32) of every row: what the preference loss keeps
  const float* in_lse;        // backward: statistics given (or stat)
  const float* in_entropy;
  const float* dlogp;         // a of every row (or coef, by sequence)
  const float* dentropy;      // h
  const float* old_logp;      // policy
  const float* advantages;
  const float* ref_logp;
  const float* weights;
  float ratio_lo, ratio_hi, kl_coef, entropy_coef;
  int32_t mean;
  float* stats;
  double* part;               // [grid][4] sums of stats
  const int32_t* offsets;     // packed sequences: rows offsets[0] .. offsets[2 pairs] take part
  int32_t pairs;
  const float* coef;          // a of every sequence's counted rows
  int32_t* fine;              // whether the offsets are (the statistics' launch writes it, the next two read it)
  uint64_t timeout_ns;
  uint32_t* ctrl;
};

// The pairs' scores, losses and coefficients from the rows' log-probabilities
struct PairArgs {
  const int32_t* offsets;
  const int32_t* targets;
  int64_t rows;
  int32_t pairs, vocab, kind, average;
  const float4* stat;
  const float* ref_logp;
  float beta, smoothing, margin;
  const int32_t* fine;
  int32_t more;               // a gradient's launch follows
  float* coef;                // [2 pairs]
  float* pair_loss;           // [pairs]
  float* margins;
  float* loss;
  uint32_t* ctrl;
};

struct LossKind {
  bool z32, d32;   // types of logits and gradients
  int mode;
  bool entropy;    // the entropy is wanted or has a gradient
  bool early;      // may start while the launch in front of it ends (it waits for that one's results itself)
};

// Between the launches of one call: what follows may start; wait for what is in front
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// fo_loss_rows.cu
cudaError_t loss_rows_launch(LossArgs a, const LossKind& k, int device, int num_sms, cudaStream_t s);
int loss_rows_parts(int num_sms);   // rows of LossArgs::part that any launch may use

}  // namespace fo

// Losses from sharded logits: argument checks, the pairs of the preference loss, launches (formulas
// in fo_loss.cuh).
#include <cmath>
#include <cstring>

#include "fo_host.h"
#include "fo_loss.cuh"
#include "fo_wide.cuh"

namespace fo {
namespace {

constexpr int kPairThreads = 256;

// Loss of a gap and its derivative
__device__ __forceinline__ float pair_loss(int kind, float beta, float gap, float* slope) {
  const float x = beta * gap;
  if (kind == FO_PREF_SQUARED) {
    const float d = gap - 0.5f / beta;
    *slope = 2.f * d;
    return d * d;
  }
  if (kind == FO_PREF_HINGE) {
    *slope = x < 1.f ? -beta : 0.f;
    return fmaxf(1.f - x, 0.f);
  }
  const float e = expf(-fabsf(x));  // log(1 + exp(-x)), of a number at most 1
  *slope = -beta * (x >= 0.f ? e / (1.f + e) : 1.f / (1.f + e));
  return fmaxf(-x, 0.f) + log1pf(e);
}

// One CTA per pair, half of it per sequence: scores, loss and coefficient; the last CTA averages the
// losses in order.  A pair's gap is a small difference of long sums: the log-probabilities come,
// and are summed, in twice fp32.
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const __grid_constant__ PairArgs a) {
  constexpr int kHalf = kPairThreads / 2, kWarps = kHalf / 32;
  __shared__ Wide sums[2][kWarps];
  __shared__ int counted[2][kWarps];
  if (a.more) let_next_start();
  wait_for_previous();
  if (!*a.fine) return;
  const int half = threadIdx.x / kHalf, at = threadIdx.x % kHalf, lane = threadIdx.x & 31;
  const int seq = blockIdx.x + half * a.pairs, end = a.offsets[seq + 1];
  Wide sum = {0.f, 0.f};
  int n = 0;
#pragma unroll 4
  for (int i = a.offsets[seq] + at; i < end; i += kHalf) {
    const int32_t y = a.targets[i];
    const float4 st = a.stat[i];  // (rows that do not count: 0)
    const float r = a.ref_logp ? a.ref_logp[i] : 0.f;
    const bool on = y >= 0 && y < a.vocab;
    sum = plus(sum, plus(Wide{on ? st.z : 0.f, on ? st.w : 0.f}, wide(on ? -r : 0.f)));
    n += on;
  }
  sum = warp_sum(sum);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    sums[half][at >> 5] = sum;
    counted[half][at >> 5] = n;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  int last = 0;
  if (threadIdx.x == 0) {
    Wide score[2];
    float share[2];
    for (int h = 0; h < 2; ++h) {
      score[h] = sums[h][0];
      n = counted[h][0];
      for (int w = 1; w < kWarps; ++w) {
        score[h] = plus(score[h], sums[h][w]);
        n += counted[h][w];
      }
      share[h] = 1.f;
      if (a.average) {  // (a quotient and what it leaves)
        const float count = static_cast<float>(n > 1 ? n : 1), q = score[h].hi / count;
        score[h] = plus(wide(q), wide((fmaf(-q, count, score[h].hi) + score[h].lo) / count));
        share[h] = 1.f / count;
      }
    }
    const Wide wide_gap = plus(plus(score[0], Wide{-score[1].hi, -score[1].lo}), wide(-a.margin));
    const float gap = wide_gap.hi + wide_gap.lo;
    float slope, back;
    float loss = pair_loss(a.kind, a.beta, gap, &slope);
    if (a.smoothing != 0.f) {
      loss = (1.f - a.smoothing) * loss + a.smoothing * pair_loss(a.kind, a.beta, -gap, &back);
      slope = (1.f - a.smoothing) * slope - a.smoothing * back;
    }
    const float each = slope / static_cast<float>(a.pairs);
    a.coef[blockIdx.x] = each * share[0];
    a.coef[blockIdx.x + a.pairs] = -each * share[1];
    if (a.margins) a.margins[blockIdx.x] = a.beta * gap;
    a.pair_loss[blockIdx.x] = loss;
    __threadfence();
    last = atomicInc(a.ctrl + kCtrlDone, gridDim.x - 1) == gridDim.x - 1;
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  sum = Wide{0.f, 0.f};
  for (int i = lane; i < a.pairs; i += 32) sum = plus(sum, wide(__ldcg(a.pair_loss + i)));
  sum = warp_sum(sum);
  if (lane == 0) a.loss[0] = (sum.hi + sum.lo) / static_cast<float>(a.pairs);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// A vector of 4-byte entries as a matrix view, for the overlap check
fo_mat vec(const void* p, int64_t n) {
  fo_mat m;
  std::memset(&m, 0, sizeof(m));
  m.ptr = const_cast<void*>(p);
  m.dtype = FO_F32;
  m.rows = p ? 1 : 0;
  m.cols = m.ld = n;
  return m;
}
fo_status check_vec(const void* p, int64_t n, bool wanted, const char* what) {
  if (!p && wanted && n > 0) return host_failf(FO_ERR_INVALID_ARG, "%s: null pointer", what);
  if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
    return host_failf(FO_ERR_UNSUPPORTED, "%s: pointer not 4-byte aligned", what);
  return FO_OK;
}
bool positive(float v) { return v > 0.f && std::isfinite(v); }

// Shapes and types of the logits and of their gradient (null: none); fills the matrices of *a
fo_status check_logits(const fo_mat* logits, int P, const fo_mat* d, const int32_t* targets, float scale, LossArgs* a,
                       LossKind* k) {
  std::memset(a, 0, sizeof(*a));
  std::memset(k, 0, sizeof(*k));
  if (!logits) return host_fail(FO_ERR_INVALID_ARG, "null matrix array");
  if (P < 1 || P > kMaxP) return host_failf(FO_ERR_INVALID_ARG, "P=%d outside [1, %d]", P, kMaxP);
  if (!positive(scale)) return host_fail(FO_ERR_INVALID_ARG, "scale must be positive and finite");
  int64_t vocab = 0;
  for (int r = 0; r < P; ++r) {
    if (logits[r].dtype != FO_BF16 && logits[r].dtype != FO_F32)
      return host_failf(FO_ERR_INVALID_ARG, "logits[%d]: unknown dtype", r);
    FO_TRY_HOST(host_check_mat(logits[r], logits[0].dtype, "logits", r));
    if (logits[r].rows != logits[0].rows)
      return host_failf(FO_ERR_SHAPE, "logits[%d]: %lld rows, logits[0] %lld", r, (long long)logits[r].rows,
                        (long long)logits[0].rows);
    if (d) {
      if (d[r].dtype != FO_BF16 && d[r].dtype != FO_F32)
        return host_failf(FO_ERR_INVALID_ARG, "dlogits[%d]: unknown dtype", r);
      FO_TRY_HOST(host_check_mat(d[r], d[0].dtype, "dlogits", r));
      if (d[r].rows != logits[r].rows || d[r].cols != logits[r].cols)
        return host_failf(FO_ERR_SHAPE, "dlogits[%d] must have the shape of logits[%d]", r, r);
      a->d[r] = d[r].ptr;
      a->ldd[r] = d[r].ld;
    }
    a->z[r] = logits[r].ptr;
    a->ldz[r] = logits[r].ld;
    a->cols[r] = static_cast<int32_t>(logits[r].cols);
    a->first[r] = static_cast<int32_t>(vocab);
    vocab += logits[r].cols;
    if (vocab > (1ll << 30)) return host_fail(FO_ERR_UNSUPPORTED, "a vocabulary above 2^30");
  }
  if (vocab < 1) return host_fail(FO_ERR_SHAPE, "the vocabulary must have at least one entry");
  a->first[P] = static_cast<int32_t>(vocab);
  a->gradient = d != nullptr;
  a->P = P;
  a->rows = logits[0].rows;
  a->scale = scale;
  a->targets = targets;
  fo_opts o;
  std::memset(&o, 0, sizeof(o));
  a->timeout_ns = host_timeout_ns(o);
  k->z32 = logits[0].dtype == FO_F32;
  k->d32 = d && d[0].dtype == FO_F32;
  return check_vec(targets, a->rows, true, "targets");
}
const int kInPlace[][2] = {{1, 0}};  // dlogits over logits: lists 1 and 0 of every call

fo_status run_rows(fo_ctx* ctx, const LossArgs& a, const LossKind& k, cudaStream_t s) {
  const cudaError_t e = loss_rows_launch(a, k, host_device(ctx), host_num_sms(ctx), s);
  return e == cudaSuccess ? FO_OK : host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace
}  // namespace fo

using namespace fo;

extern "C" {

fo_status fo_token_logprobs(fo_ctx* ctx, const fo_mat* logits, int P, const int32_t* targets, float scale,
                            float* logp, float* lse, float* entropy, void* stream) {
  LossArgs a;
  LossKind k;
  FO_TRY_HOST(check_logits(logits, P, nullptr, targets, scale, &a, &k));
  if (!logp && !lse && !entropy && a.rows > 0) return host_fail(FO_ERR_INVALID_ARG, "no output");
  FO_TRY_HOST(check_vec(logp, a.rows, false, "logp"));
  FO_TRY_HOST(check_vec(lse, a.rows, false, "lse"));
  FO_TRY_HOST(check_vec(entropy, a.rows, false, "entropy"));
  const fo_mat v[] = {vec(targets, a.rows), vec(logp, a.rows), vec(lse, a.rows), vec(entropy, a.rows)};
  const HostList views[] = {{logits, P, false, "logits"}, {&v[0], 1, false, "targets"}, {&v[1], 1, true, "logp"},
                            {&v[2], 1, true, "lse"},      {&v[3], 1, true, "entropy"}};
  FO_TRY_HOST(host_check_apart(views, 5));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  if (a.rows == 0) return FO_OK;
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  a.logp = logp;
  a.lse = lse;
  a.entropy = entropy;
  a.ctrl = host_ctrl(ctx);
  k.mode = kLossForward;
  k.entropy = entropy != nullptr;
  return run_rows(ctx, a, k, static_cast<cudaStream_t>(stream));
}

fo_status fo_token_logprobs_backward(fo_ctx* ctx, const fo_mat* logits, int P, const int32_t* targets, float scale,
                                     const float* lse, const float* entropy, const float* dlogp,
                                     const float* dentropy, const fo_mat* dlogits, void* stream) {
  if (!dlogits) return host_fail(FO_ERR_INVALID_ARG, "null matrix array");
  LossArgs a;
  LossKind k;
  FO_TRY_HOST(check_logits(logits, P, dlogits, targets, scale, &a, &k));
  FO_TRY_HOST(check_vec(lse, a.rows, true, "lse"));
  FO_TRY_HOST(check_vec(dlogp, a.rows, true, "dlogp"));
  FO_TRY_HOST(check_vec(dentropy, a.rows, false, "dentropy"));
  FO_TRY_HOST(check_vec(entropy, a.rows, dentropy != nullptr, "entropy"));
  const fo_mat v[] = {vec(targets, a.rows), vec(lse, a.rows), vec(dentropy ? entropy : nullptr, a.rows),
                      vec(dlogp, a.rows), vec(dentropy, a.rows)};
  const HostList views[] = {{logits, P, false, "logits"},   {dlogits, P, true, "dlogits"},
                            {&v[0], 1, false, "targets"},   {&v[1], 1, false, "lse"},
                            {&v[2], 1, false, "entropy"},   {&v[3], 1, false, "dlogp"},
                            {&v[4], 1, false, "dentropy"}};
  FO_TRY_HOST(host_check_apart(views, 7, kInPlace, 1));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  if (a.rows == 0) return FO_OK;
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  a.backwards = 1;  // the rows whose statistics were taken last may still be in L2
  a.in_lse = lse;
  a.in_entropy = entropy;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.ctrl = host_ctrl(ctx);
  k.mode = kLossBackward;
  k.entropy = dentropy != nullptr;
  return run_rows(ctx, a, k, static_cast<cudaStream_t>(stream));
}

fo_status fo_policy_loss(fo_ctx* ctx, const fo_mat* logits, int P, const int32_t* targets, const float* old_logp,
                         const float* advantages, const float* ref_logp, const float* weights,
                         const fo_policy_params* prm, float* logp, float* stats, const fo_mat* dlogits,
                         void* stream) {
  if (!prm) return host_fail(FO_ERR_INVALID_ARG, "null parameters");
  LossArgs a;
  LossKind k;
  FO_TRY_HOST(check_logits(logits, P, dlogits, targets, prm->scale, &a, &k));
  if (!(prm->clip_low >= 0.f) || !(prm->clip_low <= 1.f) || !(prm->clip_high >= 0.f) || !std::isfinite(prm->clip_high))
    return host_fail(FO_ERR_INVALID_ARG, "clip_low must be from 0 to 1, clip_high finite and not negative");
  if (!std::isfinite(prm->kl_coef) || !std::isfinite(prm->entropy_coef))
    return host_fail(FO_ERR_INVALID_ARG, "kl_coef and entropy_coef must be finite");
  if (!ref_logp && prm->kl_coef != 0.f) return host_fail(FO_ERR_INVALID_ARG, "kl_coef needs ref_logp");
  if (prm->mean != 0 && prm->mean != 1) return host_fail(FO_ERR_INVALID_ARG, "mean must be 0 or 1");
  FO_TRY_HOST(check_vec(stats, 4, true, "stats"));
  FO_TRY_HOST(check_vec(advantages, a.rows, true, "advantages"));
  FO_TRY_HOST(check_vec(old_logp, a.rows, false, "old_logp"));
  FO_TRY_HOST(check_vec(ref_logp, a.rows, false, "ref_logp"));
  FO_TRY_HOST(check_vec(weights, a.rows, false, "weights"));
  FO_TRY_HOST(check_vec(logp, a.rows, false, "logp"));
  const fo_mat v[] = {vec(targets, a.rows),  vec(old_logp, a.rows), vec(advantages, a.rows), vec(ref_logp, a.rows),
                      vec(weights, a.rows), vec(logp, a.rows),     vec(stats, 4)};
  const HostList views[] = {{logits, P, false, "logits"},     {dlogits, P, true, "dlogits"},
                            {&v[0], 1, false, "targets"},     {&v[1], 1, false, "old_logp"},
                            {&v[2], 1, false, "advantages"},  {&v[3], 1, false, "ref_logp"},
                            {&v[4], 1, false, "weights"},     {&v[5], 1, true, "logp"},
                            {&v[6], 1, true, "stats"}};
  FO_TRY_HOST(host_check_apart(views, 9, kInPlace, 1));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* part = nullptr;
  FO_TRY_HOST(host_buffer_kept(ctx, kSlotLoss, loss_rows_parts(host_num_sms(ctx)) * 4 * sizeof(double), s, &part));
  a.logp = logp;
  a.old_logp = old_logp;
  a.advantages = advantages;
  a.ref_logp = ref_logp;
  a.weights = weights;
  a.ratio_lo = 1.f - prm->clip_low;
  a.ratio_hi = 1.f + prm->clip_high;
  a.kl_coef = prm->kl_coef;
  a.entropy_coef = prm->entropy_coef;
  a.mean = prm->mean;
  a.stats = stats;
  a.part = static_cast<double*>(part);
  a.ctrl = host_ctrl(ctx);
  k.mode = kLossPolicy;
  k.entropy = prm->entropy_coef != 0.f;
  return run_rows(ctx, a, k, s);
}

fo_status fo_preference_loss(fo_ctx* ctx, const fo_mat* logits, int P, const int32_t* targets, const int32_t* offsets,
                             int num_pairs, const float* ref_logp, const fo_preference_params* prm, float* logp,
                             float* margins, float* loss, const fo_mat* dlogits, void* stream) {
  if (!prm) return host_fail(FO_ERR_INVALID_ARG, "null parameters");
  LossArgs a;
  LossKind k;
  FO_TRY_HOST(check_logits(logits, P, dlogits, targets, prm->scale, &a, &k));
  if (prm->kind < FO_PREF_SIGMOID || prm->kind > FO_PREF_HINGE)
    return host_failf(FO_ERR_INVALID_ARG, "unknown kind %d", prm->kind);
  if (prm->average != 0 && prm->average != 1) return host_fail(FO_ERR_INVALID_ARG, "average must be 0 or 1");
  if (!positive(prm->beta)) return host_fail(FO_ERR_INVALID_ARG, "beta must be positive and finite");
  if (!(prm->label_smoothing >= 0.f) || !(prm->label_smoothing <= 1.f))
    return host_fail(FO_ERR_INVALID_ARG, "label_smoothing must be from 0 to 1");
  if (!std::isfinite(prm->margin)) return host_fail(FO_ERR_INVALID_ARG, "margin must be finite");
  if (num_pairs < 1 || num_pairs > (1 << 20))
    return host_failf(FO_ERR_INVALID_ARG, "num_pairs=%d outside [1, 2^20]", num_pairs);
  if (a.rows > (1ll << 30)) return host_fail(FO_ERR_UNSUPPORTED, "more than 2^30 rows");
  const int64_t seqs = 2 * static_cast<int64_t>(num_pairs);
  FO_TRY_HOST(check_vec(offsets, seqs + 1, true, "offsets"));
  FO_TRY_HOST(check_vec(loss, 1, true, "loss"));
  FO_TRY_HOST(check_vec(ref_logp, a.rows, false, "ref_logp"));
  FO_TRY_HOST(check_vec(logp, a.rows, false, "logp"));
  FO_TRY_HOST(check_vec(margins, num_pairs, false, "margins"));
  const fo_mat v[] = {vec(targets, a.rows), vec(offsets, seqs + 1), vec(ref_logp, a.rows), vec(logp, a.rows),
                      vec(margins, num_pairs), vec(loss, 1)};
  const HostList views[] = {{logits, P, false, "logits"},    {dlogits, P, true, "dlogits"},
                            {&v[0], 1, false, "targets"},    {&v[1], 1, false, "offsets"},
                            {&v[2], 1, false, "ref_logp"},   {&v[3], 1, true, "logp"},
                            {&v[4], 1, true, "margins"},     {&v[5], 1, true, "loss"}};
  FO_TRY_HOST(host_check_apart(views, 8, kInPlace, 1));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // statistics of every row; coefficients and losses of the pairs
  void* work = nullptr;
  const size_t bytes = static_cast<size_t>(a.rows * 16 + seqs * 4 + num_pairs * 4 + 4);
  FO_TRY_HOST(host_buffer_kept(ctx, kSlotLoss, bytes, s, &work));
  float4* stat = static_cast<float4*>(work);
  PairArgs p;
  std::memset(&p, 0, sizeof(p));
  p.offsets = offsets;
  p.targets = targets;
  p.rows = a.rows;
  p.pairs = num_pairs;
  p.vocab = a.first[P];
  p.kind = prm->kind;
  p.average = prm->average;
  p.stat = stat;
  p.ref_logp = ref_logp;
  p.beta = prm->beta;
  p.smoothing = prm->label_smoothing;
  p.margin = prm->margin;
  p.coef = reinterpret_cast<float*>(stat + a.rows);
  p.pair_loss = p.coef + seqs;
  p.margins = margins;
  p.loss = loss;
  a.fine = reinterpret_cast<int32_t*>(p.pair_loss + num_pairs);
  p.fine = a.fine;
  p.more = dlogits != nullptr;
  p.ctrl = a.ctrl = host_ctrl(ctx);
  a.offsets = offsets;
  a.pairs = num_pairs;
  a.stat = stat;
  LossArgs back = a;
  a.gradient = 0;
  a.logp = logp;
  k.mode = kLossForward;
  FO_TRY_HOST(run_rows(ctx, a, k, s));
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(num_pairs);
  cfg.blockDim = dim3(kPairThreads);
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, pair_kernel, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  if (!dlogits) return FO_OK;
  back.coef = p.coef;
  back.backwards = 1;
  k.mode = kLossBackward;
  k.early = true;
  return run_rows(ctx, back, k, s);
}

}  // extern "C"

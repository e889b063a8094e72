// Attention with row statistics and its backward pass, for training: P independent ranks (each
// holds all tokens of its own heads), shared key/value heads, packed sequences of any length,
// query and key lengths that differ.
//
//   S = scale Q K^T (over the mask's pairs), LSE_i = log sum_j exp S_ij, O = exp(S - LSE) V
//   P = exp(S - LSE), delta_i = sum_d dO_id O_id, dS = P (dO V^T - delta)
//   dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO
//
// Work is cut into blocks of a sequence's query rows (forward, dQ) or key rows (dK / dV).  One
// sequence: the block of an index follows from the lengths.  Packed sequences: a small kernel
// reads the offsets on the device, checks them and writes a table of blocks, longest first.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "fo_attn_common.cuh"
#include "fo_host.h"
#include "fo_internal.h"
#include "fo_ptx.cuh"

namespace fo {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 1024;

struct PlanArgs {
  const int32_t *q_off, *k_off;
  int32_t n, mq, mk, causal;
  int32_t unit[2], by_keys[2], cap[2];
  int32_t* table[2];
  uint32_t* ctrl;
};

// Blocks of packed sequences in order of decreasing work (a counting sort over 1024 classes;
// the order inside a class does not matter to any result).  One CTA per table, one warp per
// sequence.  Bad offsets: FO_ERR_RANGE is recorded and the table stays empty.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ int start[kPlanBuckets];
  __shared__ int bad;
  const int tb = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* table = a.table[tb];
  for (int i = threadIdx.x; i < kPlanBuckets; i += kPlanThreads) start[i] = 0;
  if (threadIdx.x == 0) bad = -1;
  __syncthreads();
  for (int s = threadIdx.x; s <= a.n; s += kPlanThreads) {
    const int q = a.q_off[s], k = a.k_off[s];
    const int qp = s ? a.q_off[s - 1] : 0, kp = s ? a.k_off[s - 1] : 0;
    if (q < qp || k < kp || q < 0 || k < 0 || q > a.mq || k > a.mk) bad = s;
  }
  __syncthreads();
  if (bad >= 0) {
    if (threadIdx.x == 0) {
      table[0] = 0;
      note_error(a.ctrl, FO_ERR_RANGE, kSiteOffsets, static_cast<uint32_t>(bad));
    }
    return;
  }
  const int unit = a.unit[tb], by_keys = a.by_keys[tb];
  auto each = [&](auto&& f) {
    for (int s = warp; s < a.n; s += kPlanThreads / 32) {
      const int q0 = a.q_off[s], ql = a.q_off[s + 1] - q0, k0 = a.k_off[s], kl = a.k_off[s + 1] - k0;
      const int rows = by_keys ? kl : ql, nb = (rows + unit - 1) / unit;
      for (int b = lane; b < nb; b += 32) {
        const int end = (b + 1) * unit < rows ? (b + 1) * unit : rows;
        const int work = by_keys ? ql - query_begin(a.causal, b * unit, ql, kl) : key_end(a.causal, end, ql, kl);
        const int w = (work + 127) / 128;
        f(w < kPlanBuckets ? w : kPlanBuckets - 1, Block{q0, ql, k0, kl, b});
      }
    }
  };
  each([&](int w, const Block&) { atomicAdd(&start[w], 1); });
  __syncthreads();
  // start[w] = entries of a class above w: an inclusive scan from the top, less the class itself
  const int w = kPlanBuckets - 1 - threadIdx.x;
  const int own = start[w];
  int sum = own;
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  __shared__ int warp_sum[32];
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < warp; ++i) before += warp_sum[i];
  start[w] = before + sum - own;
  if (threadIdx.x == kPlanThreads - 1) table[0] = before + sum < a.cap[tb] ? before + sum : a.cap[tb];
  __syncthreads();
  each([&](int c, const Block& b) {
    const int at = atomicAdd(&start[c], 1);
    if (at >= a.cap[tb]) return;
    int32_t* t = table + kBlockInts * (1 + at);
    t[0] = b.q0;
    t[1] = b.q_len;
    t[2] = b.k0;
    t[3] = b.k_len;
    t[4] = b.blk;
  });
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct Call {
  int P, heads, kv_heads, dim;
  int64_t mq, mk;
  const int32_t *q_off, *k_off;
  int n;  // packed sequences, 0: one sequence
  int causal;
  float scale;
};

fo_status check_shape(const fo_mat* list, const char* what, int P, int64_t rows, int64_t cols, int32_t dtype) {
  if (!list) return host_failf(FO_ERR_INVALID_ARG, "%s: null matrix array", what);
  for (int r = 0; r < P; ++r) {
    FO_TRY_HOST(host_check_mat(list[r], dtype, what, r));
    if (list[r].rows != rows || list[r].cols != cols)
      return host_failf(FO_ERR_SHAPE, "%s[%d] must be [%lld, %lld]", what, r, (long long)rows, (long long)cols);
  }
  return FO_OK;
}

fo_status check_call(const fo_mat* Q, const fo_mat* K, const fo_mat* V, int P, int heads, int kv_heads, int head_dim,
                     const fo_attn_mask* mask, const fo_opts* opts, Call* c) {
  if (P < 1 || P > kMaxP) return host_failf(FO_ERR_INVALID_ARG, "P=%d outside [1, %d]", P, kMaxP);
  if (!Q || !K || !V || !mask) return host_fail(FO_ERR_INVALID_ARG, "null matrix array or mask");
  if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0)
    return host_failf(FO_ERR_INVALID_ARG, "heads=%d must be a positive multiple of kv_heads=%d", heads, kv_heads);
  if (head_dim != 64 && head_dim != 128) return host_fail(FO_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (mask->causal != 0 && mask->causal != 1) return host_fail(FO_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!(mask->scale >= 0.f) || !std::isfinite(mask->scale))
    return host_fail(FO_ERR_INVALID_ARG, "scale must be positive, or 0 for 1/sqrt(head_dim)");
  if (mask->num_seqs < 0) return host_fail(FO_ERR_INVALID_ARG, "num_seqs < 0");
  if ((mask->num_seqs > 0) != (mask->q_offsets != nullptr) || (mask->k_offsets && !mask->q_offsets))
    return host_fail(FO_ERR_INVALID_ARG, "num_seqs > 0 goes with q_offsets");
  if (reinterpret_cast<uintptr_t>(mask->q_offsets) % 4 != 0 || reinterpret_cast<uintptr_t>(mask->k_offsets) % 4 != 0)
    return host_fail(FO_ERR_UNSUPPORTED, "offsets not 4-byte aligned");
  FO_TRY_HOST(host_check_opts(opts));
  c->P = P;
  c->heads = heads;
  c->kv_heads = kv_heads;
  c->dim = head_dim;
  c->mq = Q[0].rows;
  c->mk = K[0].rows;
  c->n = mask->num_seqs;
  c->q_off = mask->q_offsets;
  c->k_off = mask->k_offsets ? mask->k_offsets : mask->q_offsets;
  c->causal = mask->causal;
  c->scale = mask->scale > 0.f ? mask->scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(head_dim)));
  FO_TRY_HOST(check_shape(Q, "Q", P, c->mq, static_cast<int64_t>(heads) * head_dim, FO_BF16));
  FO_TRY_HOST(check_shape(K, "K", P, c->mk, static_cast<int64_t>(kv_heads) * head_dim, FO_BF16));
  FO_TRY_HOST(check_shape(V, "V", P, c->mk, static_cast<int64_t>(kv_heads) * head_dim, FO_BF16));
  if (c->n > 0 && !mask->k_offsets && c->mk != c->mq)
    return host_fail(FO_ERR_SHAPE, "without k_offsets K must have as many rows as Q");
  if (c->n > (1 << 24)) return host_fail(FO_ERR_UNSUPPORTED, "more than 2^24 sequences");
  return FO_OK;
}

// Upper bound of the blocks of `unit` rows: exact for one sequence, one more per packed sequence
int64_t block_bound(const Call& c, int64_t rows, int unit) {
  return c.n > 0 ? rows / unit + c.n : (rows + unit - 1) / unit;
}

struct Cut {
  int unit;
  bool by_keys;
};

// Blocks for up to two cuts of the call's rows; packed sequences: their workspace, then the table kernel
fo_status make_blocks(fo_ctx* ctx, const Call& c, const Cut* cuts, int n, cudaStream_t s, Blocks* out) {
  PlanArgs p;
  std::memset(&p, 0, sizeof(p));
  int64_t at = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t bound = block_bound(c, cuts[i].by_keys ? c.mk : c.mq, cuts[i].unit);
    if (bound * c.heads * c.P > 0x7fffffffll) return host_fail(FO_ERR_UNSUPPORTED, "too many blocks");
    out[i] = Blocks{nullptr, static_cast<int32_t>(c.mq), static_cast<int32_t>(c.mk), c.causal,
                    static_cast<int32_t>(bound), cuts[i].unit, cuts[i].by_keys ? 1 : 0};
    p.unit[i] = cuts[i].unit;
    p.by_keys[i] = out[i].by_keys;
    p.cap[i] = out[i].count;
    at += (bound + 1) * kBlockInts;
  }
  if (c.n == 0) return FO_OK;
  void* buf = nullptr;
  FO_TRY_HOST(host_buffer_kept(ctx, kSlotAttnTable, static_cast<size_t>(at) * 4, s, &buf));
  int32_t* t = static_cast<int32_t*>(buf);
  for (int i = 0; i < n; ++i) {
    p.table[i] = t;
    out[i].table = t;
    t += (static_cast<int64_t>(out[i].count) + 1) * kBlockInts;
  }
  p.q_off = c.q_off;
  p.k_off = c.k_off;
  p.n = c.n;
  p.mq = static_cast<int32_t>(c.mq);
  p.mk = static_cast<int32_t>(c.mk);
  p.causal = c.causal;
  p.ctrl = host_ctrl(ctx);
  plan_kernel<<<n, kPlanThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FO_OK : host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
}

constexpr int64_t kPartBytes = 256ll << 20;  // most workspace for partial sums
constexpr int kPartWalk = 8;                 // fewest blocks of a part

// Parts that a pass's walks are cut into: two CTAs per SM are wanted (the last, longest-first
// wave then fills), each part of at least kPartWalk blocks of the longest possible walk, their
// partial sums (`bytes` each) within kPartBytes.
int split_of(int sms, int64_t items, int64_t walk, size_t bytes) {
  int64_t s = (2 * sms + items - 1) / items;
  if (s > walk / kPartWalk) s = walk / kPartWalk;
  if (bytes > 0 && s > kPartBytes / static_cast<int64_t>(bytes)) s = kPartBytes / static_cast<int64_t>(bytes);
  return s < 1 ? 1 : static_cast<int>(s);
}

// pointers and row pitches of P matrices
template <typename T>
void fill(const fo_mat* list, int P, T** ptr, int64_t* ld) {
  for (int r = 0; r < P; ++r) {
    ptr[r] = static_cast<T*>(list[r].ptr);
    ld[r] = list[r].ld;
  }
}

constexpr int kFwdUnit = 256;  // query rows of a forward block: two tiles

// Operand map of a [rows, cols] matrix, read in blocks of 128 rows; an empty matrix has none
// (its call has no block that reads it)
fo_status add_maps(CUtensorMap* maps, const fo_mat* list, int P) {
  for (int r = 0; r < P; ++r)
    if (list[r].rows > 0)
      FO_TRY_HOST(host_encode_map(&maps[r], list[r].ptr, list[r].rows, list[r].cols, list[r].ld, kBlk));
  return FO_OK;
}

fo_status fill_args(fo_ctx* ctx, const Call& c, const fo_mat* Q, const fo_mat* K, const fo_mat* V,
                    const fo_opts* opts, TrainArgs* a) {
  std::memset(a, 0, sizeof(*a));
  FO_TRY_HOST(add_maps(a->maps, Q, c.P));
  FO_TRY_HOST(add_maps(a->maps + c.P, K, c.P));
  FO_TRY_HOST(add_maps(a->maps + 2 * c.P, V, c.P));
  a->P = c.P;
  a->heads = c.heads;
  a->kv_heads = c.kv_heads;
  a->by_q[0] = FastDiv::by(static_cast<uint32_t>(c.heads) * c.P);
  a->by_q[1] = FastDiv::by(c.heads);
  a->by_k[0] = FastDiv::by(static_cast<uint32_t>(c.kv_heads) * c.P);
  a->by_k[1] = FastDiv::by(c.kv_heads);
  a->by_group = FastDiv::by(c.heads / c.kv_heads);
  a->mq = static_cast<int32_t>(c.mq);
  a->short_walks = c.n > 0 || c.mk <= kFineWalk * kBlk || c.mq <= kFineWalk * kBlk;
  a->scale = c.scale;
  a->scale_log2 = static_cast<float>(static_cast<double>(c.scale) * 1.4426950408889634);
  fo_opts o;
  std::memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  a->timeout_ns = host_timeout_ns(o);
  a->ctrl = host_ctrl(ctx);
  constexpr int kDevices = 64;  // kernel attributes are a device's own; host threads may come here at once
  static std::atomic<bool> done[kDevices];
  const int device = host_device(ctx);
  if (device >= kDevices || !done[device]) {
    cudaError_t e = attn_fwd_configure();
    if (e == cudaSuccess) e = attn_bwd_configure();
    if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, "attention kernel configuration failed");
    if (device < kDevices) done[device] = true;
  }
  return FO_OK;
}

}  // namespace
}  // namespace fo

using namespace fo;

extern "C" {

fo_status fo_attn_forward(fo_ctx* ctx, const fo_mat* Q, const fo_mat* K, const fo_mat* V, int P, int heads,
                          int kv_heads, int head_dim, const fo_attn_mask* mask, const fo_mat* O, const fo_mat* LSE,
                          const fo_opts* opts, void* stream) {
  Call c;
  FO_TRY_HOST(check_call(Q, K, V, P, heads, kv_heads, head_dim, mask, opts, &c));
  FO_TRY_HOST(check_shape(O, "O", P, c.mq, static_cast<int64_t>(heads) * head_dim, FO_BF16));
  FO_TRY_HOST(check_shape(LSE, "LSE", P, heads, c.mq, FO_F32));
  const HostList views[] = {{Q, P, false, "Q"},
                            {K, P, false, "K"},
                            {V, P, false, "V"},
                            {O, P, true, "O"},
                            {LSE, P, true, "LSE"}};
  FO_TRY_HOST(host_check_apart(views, 5));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  if (c.mq == 0) return FO_OK;
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TrainArgs a;
  FO_TRY_HOST(fill_args(ctx, c, Q, K, V, opts, &a));
  fill(O, P, a.out_o, a.ld_o);
  fill(LSE, P, a.lse, a.ld_lse);
  const Cut cut = {kFwdUnit, false};
  FO_TRY_HOST(make_blocks(ctx, c, &cut, 1, s, &a.blocks));
  const cudaError_t e = attn_fwd_launch(a, head_dim, s);
  return e == cudaSuccess ? FO_OK : host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
}

fo_status fo_attn_backward(fo_ctx* ctx, const fo_mat* Q, const fo_mat* K, const fo_mat* V, const fo_mat* O,
                           const fo_mat* LSE, const fo_mat* dO, int P, int heads, int kv_heads, int head_dim,
                           const fo_attn_mask* mask, const fo_mat* dQ, const fo_mat* dK, const fo_mat* dV,
                           const fo_opts* opts, void* stream) {
  Call c;
  FO_TRY_HOST(check_call(Q, K, V, P, heads, kv_heads, head_dim, mask, opts, &c));
  const int64_t qc = static_cast<int64_t>(heads) * head_dim, kc = static_cast<int64_t>(kv_heads) * head_dim;
  FO_TRY_HOST(check_shape(O, "O", P, c.mq, qc, FO_BF16));
  FO_TRY_HOST(check_shape(LSE, "LSE", P, heads, c.mq, FO_F32));
  FO_TRY_HOST(check_shape(dO, "dO", P, c.mq, qc, FO_BF16));
  FO_TRY_HOST(check_shape(dQ, "dQ", P, c.mq, qc, FO_BF16));
  FO_TRY_HOST(check_shape(dK, "dK", P, c.mk, kc, FO_BF16));
  FO_TRY_HOST(check_shape(dV, "dV", P, c.mk, kc, FO_BF16));
  const HostList views[] = {{Q, P, false, "Q"},     {K, P, false, "K"},   {V, P, false, "V"},
                            {O, P, false, "O"},     {LSE, P, false, "LSE"}, {dO, P, false, "dO"},
                            {dQ, P, true, "dQ"},    {dK, P, true, "dK"},  {dV, P, true, "dV"}};
  FO_TRY_HOST(host_check_apart(views, 9));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  if (c.mq == 0 && c.mk == 0) return FO_OK;
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TrainArgs a;
  FO_TRY_HOST(fill_args(ctx, c, Q, K, V, opts, &a));
  FO_TRY_HOST(add_maps(a.maps + 3 * P, dO, P));
  for (int r = 0; r < P; ++r) {
    a.o[r] = static_cast<const uint16_t*>(O[r].ptr);
    a.ld_o[r] = O[r].ld;
    a.d_o[r] = static_cast<const uint16_t*>(dO[r].ptr);
    a.ld_do[r] = dO[r].ld;
  }
  fill(LSE, P, a.lse, a.ld_lse);
  fill(dQ, P, a.dq, a.ld_dq);
  fill(dK, P, a.dk, a.ld_dk);
  fill(dV, P, a.dv, a.ld_dv);
  // dQ (which corrects delta), then dK / dV: a walk that would leave SMs idle is cut into parts
  const int group = heads / kv_heads;
  int splits[2];
  size_t part_bytes = 0;
  for (int pass = 0; pass < 2; ++pass) {
    const bool keys = pass == 1;
    const int64_t rows = keys ? c.mk : c.mq, items = block_bound(c, rows, kBlk) * (keys ? kv_heads : heads) * P;
    const int64_t walk = keys ? (c.mq + kBlk - 1) / kBlk * group : (c.mk + kBlk - 1) / kBlk;
    const size_t bytes = static_cast<size_t>(P) * rows * (keys ? 2 * kc : qc) * 4;  // of one part's sums
    splits[pass] = items > 0 ? split_of(host_num_sms(ctx), items, walk, bytes) : 1;
    if (splits[pass] > 1 && splits[pass] * bytes > part_bytes) part_bytes = splits[pass] * bytes;
  }
  // Every workspace before the first launch: a call that cannot have them enqueues nothing.
  void *delta = nullptr, *part = nullptr;
  FO_TRY_HOST(host_buffer_kept(ctx, kSlotAttnStats, static_cast<size_t>(P) * heads * c.mq * 4, s, &delta));
  if (part_bytes > 0) FO_TRY_HOST(host_buffer_kept(ctx, kSlotAttnPart, part_bytes, s, &part));
  a.delta = static_cast<float*>(delta);
  const Cut cuts[2] = {{kBlk, true}, {kBlk, false}};
  Blocks b[2];
  FO_TRY_HOST(make_blocks(ctx, c, cuts, 2, s, b));
  cudaError_t e = attn_delta_launch(a, head_dim, s);
  for (int pass = 0; pass < 2 && e == cudaSuccess; ++pass) {
    const bool keys = pass == 1;
    const int64_t rows = keys ? c.mk : c.mq, cols = keys ? kc : qc;
    a.blocks = b[keys ? 0 : 1];
    if (a.blocks.count == 0) continue;
    a.splits = splits[pass];
    a.by_splits = FastDiv::by(a.splits);
    a.delta_mode = kDeltaCorrect;
    if (a.splits > 1) {
      a.part = static_cast<float*>(part);
      a.part_v = a.part + static_cast<int64_t>(a.splits) * P * rows * cols;
      if (!keys) {  // no CTA sees a whole row: measure delta's error, then compute with the corrected one
        a.eps = a.part;  // (smaller than the partial sums, which come after it)
        a.delta_mode = kDeltaMeasure;
        e = cudaMemsetAsync(a.eps, 0, static_cast<size_t>(a.splits) * P * heads * c.mq * 4, s);
        if (e == cudaSuccess) e = attn_dq_launch(a, head_dim, s);
        if (e == cudaSuccess) e = attn_delta_add_launch(a, s);
        if (e != cudaSuccess) break;
        a.delta_mode = kDeltaGiven;
      }
    }
    e = keys ? attn_dkv_launch(a, head_dim, s) : attn_dq_launch(a, head_dim, s);
    if (a.splits > 1 && e == cudaSuccess) {
      PartSumArgs ps;
      std::memset(&ps, 0, sizeof(ps));
      ps.part[0] = a.part;
      ps.part[1] = a.part_v;
      for (int r = 0; r < P; ++r) {
        ps.out[0][r] = keys ? a.dk[r] : a.dq[r];
        ps.ld_out[0][r] = keys ? a.ld_dk[r] : a.ld_dq[r];
        ps.out[1][r] = a.dv[r];
        ps.ld_out[1][r] = a.ld_dv[r];
      }
      ps.rows = rows;
      ps.cols = static_cast<int32_t>(cols);
      ps.splits = a.splits;
      ps.P = P;
      ps.outputs = keys ? 2 : 1;
      ps.table = a.blocks.table;
      ps.off = c.n > 0 ? (keys ? c.k_off : c.q_off) : nullptr;
      ps.n = c.n;
      e = attn_part_sum_launch(ps, s);
    }
  }
  return e == cudaSuccess ? FO_OK : host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"

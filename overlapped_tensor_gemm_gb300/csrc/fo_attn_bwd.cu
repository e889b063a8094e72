// Backward of attention on the tensor cores (tcgen05, accumulators in TMEM), the probabilities
// recomputed from the row statistics:
//
//   P = exp(S - LSE), S = scale Q K^T;  delta_i = sum_d dO_id O_id;  dS = P (dO V^T - delta)
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// Two passes over the (query, key) pairs: one holds a block of 128 keys and walks the queries
// (dK, dV: four products), one holds a block of 128 queries and walks the keys (dQ: three).
// Seven products instead of the five of a single pass, but each gradient is summed in TMEM by
// the one CTA that owns it: no atomics, no fp32 gradient in memory, the same bits every time.
// A single pass would add dQ's 128 x 128 fp32 block to memory once per pair of blocks: 64 KiB
// through shared memory twice, by estimate about as long as the two products it saves (not built).
//
// The pass over the queries computes S and dP transposed (keys on the TMEM lanes), so that P^T
// and dS^T, written as bf16 over the scores they came from, are the A operands of the products
// that follow straight from TMEM; the pass over the keys computes them upright for the same
// reason.  Q and dO (K in the other pass) are read from one shared-memory tile in both
// orientations: K-major for the scores, MN-major for the gradients.
//
// CTA layout (384 threads, one CTA per SM): warp 0 loads (TMA), warp 1 issues the MMAs, warp 2
// loads the row statistics (dK / dV), warps 4-11 compute P and dS: two warps per 32 TMEM lanes,
// one per 64 columns.
//
// Rows behind a sequence belong to another one or to nobody and may hold anything.  As rows of
// a product's A operand, or as its columns, they only reach results that are not stored or that
// a select sets to zero; as terms of a sum (Q and dO in dK / dV, K in dQ) they would turn the
// sum into NaN even with weight 0, so the loader clears them in shared memory.
//
// Measured: 16384 tokens, 8 heads on 2, causal 1195-1210 us for both passes (1145 TFLOP/s counting
// five products, 1600 counting the seven executed); 8192 tokens, 32 heads on 8: 1202 us; head_dim
// 64, 8192 tokens, 16 heads: 484-488 us.  A step of dK / dV takes 2200 cycles, of which its four
// products are 2048; a CTA spends 4000 cycles before its first step and 4000 after its last.  Bound
// by a CTA's chain of score product, softmax and gradient product; without its softmax arithmetic a
// pass is 5% faster, with half its loads not at all.
#include <cuda_bf16.h>

#include "fo_attn_common.cuh"
#include "fo_internal.h"
#include "fo_ptx.cuh"

namespace fo {
namespace {

constexpr int kThreads = 384;
constexpr int kWorkWarps = 8;                 // warps 4-11
constexpr uint32_t kTmem = 512;

// 64 columns of this warp's lanes
__device__ __forceinline__ void load64(uint32_t taddr, float (&v)[64]) {
  uint32_t w[2][32];
  tmem_ld32(taddr, w[0]);
  tmem_ld32(taddr + 32, w[1]);
  tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < 64; ++k) v[k] = __uint_as_float(w[k >> 5][k & 31]);
}
// their bf16 values, two per column, over the first 32 of them; fine: what bf16 leaves of them over
// the other 32
__device__ __forceinline__ void store64_bf16(uint32_t taddr, const float (&v)[64], bool fine) {
  uint32_t w[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
  tmem_st32(taddr, w);
  if (fine) {
#pragma unroll
    for (int k = 0; k < 32; ++k) w[k] = rest_bf16x2(v[2 * k], v[2 * k + 1], w[k]);
    tmem_st32(taddr + 32, w);
  }
  tmem_wait_st();
}
// D += A B with A from such columns
template <int D>
__device__ __forceinline__ void issue_grad64(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, bool first, bool fine) {
  issue_grad<D, 64>(d_tmem, a_tmem, b, first);
  if (fine) issue_grad<D, 64>(d_tmem, a_tmem + 32, b, false);
}

// Part `split` of a walk: n iterations from i0 on
__device__ __forceinline__ void part_of(int walk, int split, int splits, int* i0, int* n) {
  *i0 = 0;
  *n = walk;
  if (splits == 1) return;
  *i0 = static_cast<int>(static_cast<int64_t>(walk) * split / splits);
  *n = static_cast<int>(static_cast<int64_t>(walk) * (split + 1) / splits) - *i0;
}

// ---------------------------------------------------------------------------
// dK / dV: a block of 128 keys of one key/value head; walks the query heads of its group and
// their blocks of 128 queries.
//
// TMEM: S^T (then P^T) [0, 128), dP^T (then dS^T) [128, 256), dV [256, 256 + D), dK behind it.
// One buffer each (head_dim 128): the tensor pipe runs dV_i and S_{i+1} while the working warps
// turn dP_i into dS_i, and dK_i and dP_{i+1} while they turn S_{i+1} into P_{i+1}.  The MMAs of
// a CTA execute in the order in which its one issuing thread issues them: S_{i+1} overwrites P_i
// after dV_i has read it, dP_{i+1} overwrites dS_i after dK_i has.
// ---------------------------------------------------------------------------
constexpr uint32_t kColP = 128, kColV = 256;
// head_dim 64 leaves room for a second S^T: scores then never wait for the weights they would
// overwrite.  The weights may then be written for block i + 1 before the issuing warp has looked
// at those of block i: a parity tells a phase from the next one, not from the one after, so each
// buffer's weights have a barrier of their own.
template <int D>
struct DkvCols {
  static constexpr int bufs = D == 64 ? 2 : 1;
  static constexpr uint32_t k = 256 + D;
  __device__ static uint32_t s(int i) { return bufs == 2 && (i & 1) ? 384 : 0; }
  __device__ static int buf(int i) { return i % bufs; }
  __device__ static uint32_t parity(int i) { return (i / bufs) & 1; }
};

template <int D>
struct DkvSmem {
  static constexpr uint32_t tile = D / 64 * kHalf;
  static constexpr uint32_t k = 0, v = tile, q = 2 * tile, d_o = 4 * tile, stats = 6 * tile;  // q, d_o: 2 stages
  static constexpr uint32_t ctl = stats + 2 * 2 * kBlk * 4;
};
struct alignas(8) DkvCtl {
  uint64_t kv_full, q_full[2], do_full[2], empty[2], st_full[2], st_empty[2];
  uint64_t s_full[2], p_full[2], dp_full, ds_full, acc_full, fix, drain;
  uint32_t tmem_base, pad;
};
template <int D>
constexpr int dkv_smem() {
  return static_cast<int>(DkvSmem<D>::ctl + sizeof(DkvCtl) + 1024);
}

// The walk over the query heads and their blocks
struct QueryWalk {
  int h0, first, per_head, i0, n;  // first query head, first block, blocks per head, iterations [i0, i0 + n)
};
// Where it stands: query head and block of an iteration
struct QueryAt {
  int h, qb, end;
  __device__ __forceinline__ explicit QueryAt(const QueryWalk& w) : h(w.h0), qb(w.first), end(w.first + w.per_head) {
    if (w.i0 > 0 && w.per_head > 0) {
      h += w.i0 / w.per_head;
      qb += w.i0 % w.per_head;
    }
  }
  __device__ __forceinline__ void next(const QueryWalk& w) {
    if (++qb == end) {
      qb = w.first;
      ++h;
    }
  }
};

template <int D, bool kShort>
__global__ void __launch_bounds__(kThreads, 1) attn_dkv_kernel(const __grid_constant__ TrainArgs p) {
  using L = DkvSmem<D>;
  using Cols = DkvCols<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  DkvCtl* ctl = reinterpret_cast<DkvCtl*>(smem + L::ctl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = p.by_splits.of(blockIdx.x), split = blockIdx.x - item * p.splits;
  const int e = p.by_k[0].of(item), ph = item - e * p.kv_heads * p.P;
  const int rk = p.by_k[1].of(ph), kvh = ph - rk * p.kv_heads;
  Block b;
  if (!block_at(p.blocks, e, &b)) return;
  const int group = p.by_k[1].of(p.heads), key0 = b.blk * kBlk;
  QueryWalk w;
  w.h0 = kvh * group;
  w.first = query_begin(p.blocks.causal, key0, b.q_len, b.k_len) / kBlk;
  w.per_head = (b.q_len + kBlk - 1) / kBlk - w.first;
  if (w.per_head < 0) w.per_head = 0;
  const int walk = group * w.per_head;
  const bool fine = kShort && w.per_head <= kFineWalk;
  part_of(walk, split, p.splits, &w.i0, &w.n);

  if (threadIdx.x == 0) {
    // the first loads go out before anything else
    mbar_init(&ctl->kv_full, 1);
    fence_barrier_init();
    fence_proxy_async_shared();
    if (w.n > 0) {
      mbar_arrive_expect_tx(&ctl->kv_full, 2 * L::tile);
      load_block<D>(&p.maps[p.P + rk], smem + L::k, &ctl->kv_full, kvh * D, b.k0 + key0);
      load_block<D>(&p.maps[2 * p.P + rk], smem + L::v, &ctl->kv_full, kvh * D, b.k0 + key0);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->q_full[s], 1);
      mbar_init(&ctl->do_full[s], 1);
      mbar_init(&ctl->empty[s], 1);
      mbar_init(&ctl->st_full[s], 1);
      mbar_init(&ctl->st_empty[s], kWorkWarps);
    }
    mbar_init(&ctl->s_full[0], 1);
    mbar_init(&ctl->s_full[1], 1);
    mbar_init(&ctl->p_full[0], kWorkWarps);
    mbar_init(&ctl->p_full[1], kWorkWarps);
    mbar_init(&ctl->dp_full, 1);
    mbar_init(&ctl->ds_full, kWorkWarps);
    mbar_init(&ctl->acc_full, 1);
    mbar_init(&ctl->fix, 1);
    mbar_init(&ctl->drain, 1);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const uint32_t sbase = smem_u32(smem);
  float* stats = reinterpret_cast<float*>(smem + L::stats);  // [stage][lse, delta][128]

  if (warp < 4) {
    if (warp == 0) {  // ---- loads
      uint32_t fix_uses = 0;
      int armed = 0;  // iterations whose loads have been issued
      bool ok = true, q_armed = false;
      QueryAt at(w);
      for (int i = 0; ok && i < w.n; ++i, at.next(w)) {
        const int st = i & 1;
        const uint32_t free_parity = ((i >> 1) & 1) ^ 1;
        const int h = at.h, qb = at.qb;
        const int valid = b.q_len - qb * kBlk;
        q_armed = false;
        ok = attn_wait(&ctl->empty[st], free_parity, p, kSiteEmpty, lane);
        if (!ok) break;
        ok = load_summed<D>(p, &p.maps[rk], smem + L::q + st * L::tile, &ctl->q_full[st], &ctl->fix, fix_uses, h * D,
                            b.q0 + qb * kBlk, valid, lane);
        if (!ok) break;
        q_armed = true;
        ok = load_summed<D>(p, &p.maps[3 * p.P + rk], smem + L::d_o + st * L::tile, &ctl->do_full[st], &ctl->fix,
                            fix_uses, h * D, b.q0 + qb * kBlk, valid, lane);
        if (!ok) break;
        armed = i + 1;
        q_armed = false;
      }
      if (lane == 0 && w.n > 0) {  // no copy in flight when the CTA leaves, whichever warp gave up
        mbar_wait_drain(&ctl->kv_full, 0, kAttnDrainNs);
        for (int i = armed - 2 < 0 ? 0 : armed - 2; i < armed + (q_armed ? 1 : 0); ++i) {
          mbar_wait_drain(&ctl->q_full[i & 1], (i >> 1) & 1, kAttnDrainNs);
          if (i < armed) mbar_wait_drain(&ctl->do_full[i & 1], (i >> 1) & 1, kAttnDrainNs);
        }
      }
    } else if (warp == 1 && w.n > 0) {  // ---- MMAs
      const uint32_t ka = sbase + L::k, va = sbase + L::v;
      bool ok = attn_wait(&ctl->kv_full, 0, p, kSiteFull, lane) &&
                attn_wait(&ctl->q_full[0], 0, p, kSiteFull, lane);
      bool issued = false;
      if (ok) {
        tc_fence_after();
        if (elect_lane()) {
          issue_scores<D>(tmem + Cols::s(0), ka, sbase + L::q);
          umma_commit(&ctl->s_full[0]);
        }
        __syncwarp();
        issued = true;
        ok = attn_wait(&ctl->do_full[0], 0, p, kSiteFull, lane);
        if (ok && elect_lane()) {
          issue_scores<D>(tmem + kColP, va, sbase + L::d_o);
          umma_commit(&ctl->dp_full);
        }
        __syncwarp();
      }
      for (int i = 0; ok && i < w.n; ++i) {
        const int st = i & 1, nx = st ^ 1;
        const uint32_t ph = i & 1, nph = ((i + 1) >> 1) & 1;
        const bool more = i + 1 < w.n;
        // The waits for the next block's operands stand between two groups of MMAs, where they pass
        // while the first group runs.
        if (Cols::bufs == 2 && more) {
          ok = attn_wait(&ctl->q_full[nx], nph, p, kSiteFull, lane);
          if (!ok) break;
          if (elect_lane()) {
            issue_scores<D>(tmem + Cols::s(i + 1), ka, sbase + L::q + nx * L::tile);
            umma_commit(&ctl->s_full[Cols::buf(i + 1)]);
          }
          __syncwarp();
        }
        ok = attn_wait(&ctl->p_full[Cols::buf(i)], Cols::parity(i), p, kSiteTmemFull, lane);
        if (!ok) break;
        tc_fence_after();
        if (elect_lane())
          issue_grad64<D>(tmem + kColV, tmem + Cols::s(i), sbase + L::d_o + st * L::tile, i == 0, fine);
        __syncwarp();
        if (Cols::bufs == 1 && more) {
          ok = attn_wait(&ctl->q_full[nx], nph, p, kSiteFull, lane);
          if (!ok) break;
          if (elect_lane()) {
            issue_scores<D>(tmem + Cols::s(i + 1), ka, sbase + L::q + nx * L::tile);
            umma_commit(&ctl->s_full[0]);
          }
          __syncwarp();
        }
        ok = attn_wait(&ctl->ds_full, ph, p, kSiteTmemFull, lane);
        if (!ok) break;
        tc_fence_after();
        if (elect_lane()) {
          issue_grad64<D>(tmem + Cols::k, tmem + kColP, sbase + L::q + st * L::tile, i == 0, fine);
          umma_commit(&ctl->empty[st]);  // dV_i and dK_i have read the stage
        }
        __syncwarp();
        if (more) {
          ok = attn_wait(&ctl->do_full[nx], nph, p, kSiteFull, lane);
          if (!ok) break;
          if (elect_lane()) {
            issue_scores<D>(tmem + kColP, va, sbase + L::d_o + nx * L::tile);
            umma_commit(&ctl->dp_full);
          }
          __syncwarp();
        }
      }
      if (ok && elect_lane()) umma_commit(&ctl->acc_full);
      if (issued && elect_lane()) {  // and no MMA
        umma_commit(&ctl->drain);
        mbar_wait_drain(&ctl->drain, 0, kAttnDrainNs);
      }
    } else if (warp == 2) {  // ---- row statistics of the queries
      QueryAt at(w);
      for (int i = 0; i < w.n; ++i, at.next(w)) {
        const int st = i & 1;
        const int h = at.h, qb = at.qb;
        if (!attn_wait(&ctl->st_empty[st], ((i >> 1) & 1) ^ 1, p, kSiteEmpty, lane)) break;
        const float* lse = p.lse[rk] + h * p.ld_lse[rk] + b.q0;
        const float* del = p.delta + (static_cast<int64_t>(rk) * p.heads + h) * p.mq + b.q0;
        float* out = stats + st * 2 * kBlk;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = k * 32 + lane, q = qb * kBlk + c;
          const float l = q < b.q_len ? lse[q] : -INFINITY;
          // a query without keys, or behind the sequence: weight exp(s - infinity) = 0
          out[c] = l == -INFINITY ? INFINITY : l * kLog2e;
          out[kBlk + c] = q < b.q_len ? del[q] : 0.f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->st_full[st]);
      }
    }
  } else {  // ---- P and dS
    const int quad = warp & 3, hf = (warp - 4) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int key = key0 + quad * 32 + lane;  // this thread's row of S^T
    const int off = b.k_len - b.q_len;
    const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
    bool ok = true;
    QueryAt at(w);
    for (int i = 0; i < w.n; ++i, at.next(w)) {
      const int st = i & 1;
      const uint32_t ph = i & 1;
      const int qb = at.qb;
      const float* lse = stats + st * 2 * kBlk + hf * 64;
      const float* del = lse + kBlk;
      ok = attn_wait(&ctl->st_full[st], (i >> 1) & 1, p, kSiteFull, lane) &&
           attn_wait(&ctl->s_full[Cols::buf(i)], Cols::parity(i), p, kSiteTmemFull, lane);
      if (!ok) break;
      tc_fence_after();
      float s[64];
      load64(lanes + Cols::s(i) + hf * 64, s);
#pragma unroll
      for (int k = 0; k < 64; k += 4) {
        const float4 l = *reinterpret_cast<const float4*>(lse + k);
        float x0, x1, x2, x3;
        unpack2(ffma2(pack2(s[k], s[k + 1]), c2, pack2(-l.x, -l.y)), x0, x1);
        unpack2(ffma2(pack2(s[k + 2], s[k + 3]), c2, pack2(-l.z, -l.w)), x2, x3);
        s[k] = fast_exp2(x0);
        s[k + 1] = fast_exp2(x1);
        s[k + 2] = fast_exp2(x2);
        s[k + 3] = fast_exp2(x3);
      }
      // a query sees this key from query key - off on
      if (p.blocks.causal && key0 + kBlk - 1 > qb * kBlk + off) {
        const int from = key - off - qb * kBlk - hf * 64;
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (k < from) s[k] = 0.f;
      }
      store64_bf16(lanes + Cols::s(i) + hf * 64, s, fine);
      attn_publish(&ctl->p_full[Cols::buf(i)], lane);
      ok = attn_wait(&ctl->dp_full, ph, p, kSiteTmemFull, lane);
      if (!ok) break;
      tc_fence_after();
      float dp[64];
      load64(lanes + kColP + hf * 64, dp);
#pragma unroll
      for (int k = 0; k < 64; k += 4) {
        const float4 d = *reinterpret_cast<const float4*>(del + k);
        dp[k] = s[k] * (dp[k] - d.x);
        dp[k + 1] = s[k + 1] * (dp[k + 1] - d.y);
        dp[k + 2] = s[k + 2] * (dp[k + 2] - d.z);
        dp[k + 3] = s[k + 3] * (dp[k + 3] - d.w);
      }
      store64_bf16(lanes + kColP + hf * 64, dp, fine);
      attn_publish(&ctl->ds_full, lane);
      if (lane == 0) mbar_arrive(&ctl->st_empty[st]);
    }
    if (ok && w.n > 0) ok = attn_wait(&ctl->acc_full, 0, p, kSiteDrain, lane);
    if (ok) {
      tc_fence_after();
      // the tiles of K and V have been read: their memory turns the rows
      const int first = key0 + quad * 32, rows = b.k_len - first;
      const int64_t row = b.k0 + first;
      if (p.splits > 1) {
        const int64_t ld = static_cast<int64_t>(p.kv_heads) * D;
        const int64_t at = ((static_cast<int64_t>(split) * p.P + rk) * p.blocks.mk + row) * ld + kvh * D + hf * (D / 2);
        uint8_t* stage = smem + L::k + (warp - 4) * (32 * D / 2 * 4);
        attn_store_rows<D / 2>(lanes + kColV, hf * (D / 2), 1.f, stage, p.part_v + at, ld, rows, w.n == 0);
        attn_store_rows<D / 2>(lanes + Cols::k, hf * (D / 2), p.scale, stage, p.part + at, ld, rows, w.n == 0);
      } else {
        uint8_t* stage = smem + L::k + (warp - 4) * (32 * D / 2 * 2);
        const int col = kvh * D + hf * (D / 2);
        attn_store_rows<D / 2>(lanes + kColV, hf * (D / 2), 1.f, stage, p.dv[rk] + row * p.ld_dv[rk] + col, p.ld_dv[rk],
                               rows, w.n == 0);
        attn_store_rows<D / 2>(lanes + Cols::k, hf * (D / 2), p.scale, stage, p.dk[rk] + row * p.ld_dk[rk] + col,
                               p.ld_dk[rk], rows, w.n == 0);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// ---------------------------------------------------------------------------
// dQ: a block of 128 queries of one query head; walks the blocks of 128 keys it sees.
//
// TMEM: S (then dS) [0, 128) and [128, 256) in turn, dP [256, 384), dQ [384, 384 + D).  While the
// working warps turn S_i and dP_i into dS_i the tensor pipe runs S_{i+1}; dP_{i+1} follows as
// soon as they have read dP_i, dQ_i once dS_i is written.
//
// delta.  dS = P (dP - delta) with delta = sum_j P_j dP_j = sum_d dO_d O_d; the kernel is given O
// rounded to bf16, and where a row attends to few keys the two terms cancel and that rounding is
// most of dS's error (rows of 1-8 keys: dQ's and dK's error 2.3 times the output's rounding).
// But sum_j dS_j of a row is exactly what delta is off by, and costs one sum.  So this pass runs
// before dK / dV, which then have the corrected delta; and a block whose dS is off by more than
// 2^-11 (2-norm over its rows of the error's sum against that of |dS|) walks its keys a second
// time.  For spread attention these are the first one or two blocks of a sequence; where a few keys
// hold most of a row's weight, |dS| is small beside delta's error and most blocks do (8192 tokens,
// 32 heads, scores of standard deviation 4 and 8: 1730-1810 us backward instead of 1200).
// Instantiations with kShort sum |dS| over every key.  The others take a quarter of them for all
// (every key: 3% more time at 8192 tokens): keys 4 and 5 of each 8, so that where the first keys
// hold much of dS it is estimated low and the block walks again; two keys of opposite dS that hold
// all of it, both among the sampled, would let through four times as much.
//
// Two warps issue, one the scores and one the gradient: what an issuing warp spends on barriers
// passes while the pipe runs the other's.  dS_{i+1} waits for the scores alone and may be written
// before the gradient's warp has looked at dS_i, so each score buffer's dS has its own barrier.
// ---------------------------------------------------------------------------
constexpr uint32_t kColDp = 256, kColDq = 384;
constexpr int kKStages = 3, kVStages = 2;

template <int D>
struct DqSmem {
  static constexpr uint32_t tile = D / 64 * kHalf;
  static constexpr uint32_t q = 0, d_o = tile, k = 2 * tile, v = k + kKStages * tile, ctl = v + kVStages * tile;
};
struct alignas(8) DqCtl {
  uint64_t q_full, k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2], s_free[2], dp_full, dp_free, ds_full[2], acc_full, fix, drain[2];
  uint32_t tmem_base, pad;
};
template <int D>
constexpr int dq_smem() {
  return static_cast<int>(DqSmem<D>::ctl + sizeof(DqCtl) + 1024);
}

template <int D, bool kShort>
__global__ void __launch_bounds__(kThreads, 1) attn_dq_kernel(const __grid_constant__ TrainArgs p) {
  using L = DqSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  DqCtl* ctl = reinterpret_cast<DqCtl*>(smem + L::ctl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = p.by_splits.of(blockIdx.x), split = blockIdx.x - item * p.splits;
  const int e = p.by_q[0].of(item), ph = item - e * p.heads * p.P;
  const int rk = p.by_q[1].of(ph), h = ph - rk * p.heads;
  Block b;
  if (!block_at(p.blocks, e, &b)) return;
  const int kvh = p.by_group.of(h), query0 = b.blk * kBlk;
  const int q_end = query0 + kBlk < b.q_len ? query0 + kBlk : b.q_len;
  // key blocks [i0, i0 + n) of the walk
  const int walk = (key_end(p.blocks.causal, q_end, b.q_len, b.k_len) + kBlk - 1) / kBlk;
  const bool fine = kShort && walk <= kFineWalk;
  int i0, n;
  part_of(walk, split, p.splits, &i0, &n);

  if (threadIdx.x == 0) {
    // the first loads go out before anything else
    mbar_init(&ctl->q_full, 1);
    for (int s = 0; s < kVStages; ++s) mbar_init(&ctl->v_full[s], 1);
    fence_barrier_init();
    fence_proxy_async_shared();
    if (n > 0) {
      mbar_arrive_expect_tx(&ctl->q_full, 2 * L::tile);
      load_block<D>(&p.maps[rk], smem + L::q, &ctl->q_full, h * D, b.q0 + query0);
      load_block<D>(&p.maps[3 * p.P + rk], smem + L::d_o, &ctl->q_full, h * D, b.q0 + query0);
      mbar_arrive_expect_tx(&ctl->v_full[0], L::tile);
      load_block<D>(&p.maps[2 * p.P + rk], smem + L::v, &ctl->v_full[0], kvh * D, b.k0 + i0 * kBlk);
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&ctl->k_full[s], 1);
      mbar_init(&ctl->k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) mbar_init(&ctl->v_empty[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->s_full[s], 1);
      mbar_init(&ctl->s_free[s], 1);
      mbar_init(&ctl->ds_full[s], kWorkWarps);
      mbar_init(&ctl->drain[s], 1);
    }
    mbar_init(&ctl->dp_full, 1);
    mbar_init(&ctl->dp_free, kWorkWarps);
    mbar_init(&ctl->acc_full, 1);
    mbar_init(&ctl->fix, 1);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const uint32_t sbase = smem_u32(smem);

  // what each role carries from one round over the keys to the next
  bool ok = true, issued = false;
  uint32_t fix_uses = 0, kph = 0, vph = 0;
  int ks = 0, vs = 0;
  const int quad = warp & 3, hf = (warp - 4) >> 2;
  const int query = query0 + quad * 32 + lane;  // a working thread's row of S
  const bool live = query < b.q_len;
  float lse2 = INFINITY, delta = 0.f;
  const int64_t stat = (static_cast<int64_t>(rk) * p.heads + h) * p.mq + b.q0 + query;
  if (warp >= 4 && live) {
    const float l = p.lse[rk][h * p.ld_lse[rk] + b.q0 + query];
    lse2 = l == -INFINITY ? INFINITY : l * kLog2e;
    delta = p.delta[stat];
  }
  float* const sums = reinterpret_cast<float*>(smem + L::v);  // between rounds: [error, size][half][128 rows]

  for (int round = 0;; ++round) {
    const int g0 = round * n;  // blocks before this round: the barriers' phases count on
    float err = 0.f, size = 0.f;
    if (warp < 4) {
      if (warp == 0) {  // ---- loads
        int k_armed = g0, v_armed = g0 > 0 ? g0 : n > 0 ? 1 : 0;  // blocks whose loads have been issued
        for (int i = 0; ok && i < n; ++i) {
          const int g = g0 + i;
          ks = g % kKStages;
          vs = g % kVStages;
          ok = attn_wait(&ctl->k_empty[ks], ((g / kKStages) & 1) ^ 1, p, kSiteEmpty, lane) &&
               load_summed<D>(p, &p.maps[p.P + rk], smem + L::k + ks * L::tile, &ctl->k_full[ks], &ctl->fix, fix_uses,
                              kvh * D, b.k0 + (i0 + i) * kBlk, b.k_len - (i0 + i) * kBlk, lane);
          if (!ok) break;
          k_armed = g + 1;
          ok = attn_wait(&ctl->v_empty[vs], ((g / kVStages) & 1) ^ 1, p, kSiteEmpty, lane);
          if (!ok) break;
          if (lane == 0 && g > 0) {
            mbar_arrive_expect_tx(&ctl->v_full[vs], L::tile);
            load_block<D>(&p.maps[2 * p.P + rk], smem + L::v + vs * L::tile, &ctl->v_full[vs], kvh * D,
                          b.k0 + (i0 + i) * kBlk);
          }
          v_armed = g + 1;
        }
        if (lane == 0 && n > 0) {  // no copy in flight after the round, whichever warp gave up
          mbar_wait_drain(&ctl->q_full, 0, kAttnDrainNs);
          for (int i = k_armed - kKStages < 0 ? 0 : k_armed - kKStages; i < k_armed; ++i)
            mbar_wait_drain(&ctl->k_full[i % kKStages], (i / kKStages) & 1, kAttnDrainNs);
          for (int i = v_armed - kVStages < 0 ? 0 : v_armed - kVStages; i < v_armed; ++i)
            mbar_wait_drain(&ctl->v_full[i % kVStages], (i / kVStages) & 1, kAttnDrainNs);
        }
      } else if (warp == 1 && n > 0) {  // ---- MMAs of S and dP
        const uint32_t qa = sbase + L::q, da = sbase + L::d_o;
        ok = ok && attn_wait(&ctl->q_full, 0, p, kSiteFull, lane);
        for (int i = g0; ok && i < g0 + n; ++i) {
          // S_i overwrites dS_{i-2}, which dQ_{i-2} has read; dP_i overwrites dP_{i-1}, which has been read
          ok = attn_wait(&ctl->k_full[ks], kph, p, kSiteFull, lane) &&
               (i < 2 || attn_wait(&ctl->s_free[i & 1], ((i >> 1) & 1) ^ 1, p, kSiteTmemEmpty, lane));
          if (!ok) break;
          tc_fence_after();
          if (elect_lane()) {
            issue_scores<D>(tmem + (i & 1) * 128, qa, sbase + L::k + ks * L::tile);
            umma_commit(&ctl->s_full[i & 1]);
          }
          __syncwarp();
          issued = true;
          ok = attn_wait(&ctl->v_full[vs], vph, p, kSiteFull, lane) &&
               (i < 1 || attn_wait(&ctl->dp_free, (i - 1) & 1, p, kSiteTmemEmpty, lane));
          if (!ok) break;
          tc_fence_after();
          if (elect_lane()) {
            issue_scores<D>(tmem + kColDp, da, sbase + L::v + vs * L::tile);
            umma_commit(&ctl->dp_full);
            umma_commit(&ctl->v_empty[vs]);
          }
          __syncwarp();
          if (++ks == kKStages) {
            ks = 0;
            kph ^= 1;
          }
          if (++vs == kVStages) {
            vs = 0;
            vph ^= 1;
          }
        }
      } else if (warp == 2 && n > 0) {  // ---- MMAs of dQ
        for (int i = g0; ok && i < g0 + n; ++i) {
          ok = attn_wait(&ctl->ds_full[i & 1], (i >> 1) & 1, p, kSiteTmemFull, lane);
          if (!ok) break;
          tc_fence_after();
          if (elect_lane()) {
            issue_grad64<D>(tmem + kColDq, tmem + (i & 1) * 128, sbase + L::k + ks * L::tile, i == g0, fine);
            umma_commit(&ctl->s_free[i & 1]);
            umma_commit(&ctl->k_empty[ks]);
          }
          __syncwarp();
          issued = true;
          if (++ks == kKStages) ks = 0;
        }
      }
    } else {  // ---- P and dS
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      const int see = key_end(p.blocks.causal, query + 1, b.q_len, b.k_len);          // keys of this row
      const int all = key_end(p.blocks.causal, query0 + 1, b.q_len, b.k_len);         // keys of the block's first row
      const uint64_t c2 = pack2(p.scale_log2, p.scale_log2), l2 = pack2(-lse2, -lse2);
      uint64_t err2 = 0;
      for (int i = 0; ok && i < n; ++i) {
        const int g = g0 + i;
        const uint32_t buf = lanes + (g & 1) * 128 + hf * 64;
        ok = attn_wait(&ctl->s_full[g & 1], (g >> 1) & 1, p, kSiteTmemFull, lane);
        if (!ok) break;
        tc_fence_after();
        float s[64];
        load64(buf, s);
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          float x0, x1;
          unpack2(ffma2(pack2(s[k], s[k + 1]), c2, l2), x0, x1);
          s[k] = fast_exp2(x0);
          s[k + 1] = fast_exp2(x1);
        }
        ok = attn_wait(&ctl->dp_full, g & 1, p, kSiteTmemFull, lane);
        if (!ok) break;
        tc_fence_after();
        float dp[64];
        load64(lanes + kColDp + hf * 64, dp);
        attn_publish(&ctl->dp_free, lane);
#pragma unroll
        for (int k = 0; k < 64; ++k) s[k] = s[k] * (dp[k] - delta);
        if ((i0 + i + 1) * kBlk > all) {  // keys that this row does not see: whatever they hold
          const int upto = see - (i0 + i) * kBlk - hf * 64;
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (k >= upto) s[k] = 0.f;
        }
        // (of use in the first round alone; a branch here measured 10% slower at head_dim 64)
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          err2 = fadd2(err2, pack2(s[k], s[k + 1]));
          if (kShort || k % 8 == 4) size += fabsf(s[k]) + fabsf(s[k + 1]);
        }
        store64_bf16(buf, s, fine);
        attn_publish(&ctl->ds_full[g & 1], lane);
      }
      float x, y;
      unpack2(err2, x, y);
      err = x + y;
      if (!kShort) size *= 4.f;
    }
    if (round > 0 || n == 0 || p.delta_mode == kDeltaGiven) break;
    // delta's error, row by row, and whether the block is worth a second round
    __syncwarp();
    if (warp >= 4) {
      const int row = quad * 32 + lane;
      sums[hf * kBlk + row] = live ? err : 0.f;
      sums[(2 + hf) * kBlk + row] = live ? size : 0.f;
    }
    __syncthreads();
    if (warp >= 4) {
      const int row = quad * 32 + lane;
      const float e = sums[row] + sums[kBlk + row];
      delta += e;
      if (live && hf == 0 && ok) {
        if (p.delta_mode == kDeltaMeasure) {
          p.eps[static_cast<int64_t>(split) * p.P * p.heads * p.mq + stat] = e;
        } else {
          p.delta[stat] = delta;
        }
      }
    }
    if (p.delta_mode == kDeltaMeasure) break;
    float e2 = 0.f, a2 = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float e = sums[k * 32 + lane] + sums[kBlk + k * 32 + lane];
      const float a = sums[2 * kBlk + k * 32 + lane] + sums[3 * kBlk + k * 32 + lane];
      e2 = fmaf(e, e, e2);
      a2 = fmaf(a, a, a2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      e2 += __shfl_xor_sync(0xffffffffu, e2, o);
      a2 += __shfl_xor_sync(0xffffffffu, a2, o);
    }
    if (!(e2 > 0x1p-22f * a2)) break;
    __syncthreads();  // every warp has read the sums: the stage may be loaded again
    fence_proxy_async_shared();
  }
  if (n > 0 && warp == 2 && ok && elect_lane()) umma_commit(&ctl->acc_full);
  if ((warp == 1 || warp == 2) && issued && elect_lane()) {  // no MMA in flight when the CTA leaves
    umma_commit(&ctl->drain[warp - 1]);
    mbar_wait_drain(&ctl->drain[warp - 1], 0, kAttnDrainNs);
  }
  if (warp >= 4) {
    if (ok && n > 0) ok = attn_wait(&ctl->acc_full, 0, p, kSiteDrain, lane);
    if (ok && p.delta_mode != kDeltaMeasure) {
      tc_fence_after();
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      // the tiles of K have been read: their memory turns the rows
      const int first = query0 + quad * 32, rows = b.q_len - first;
      const int64_t row = b.q0 + first;
      if (p.splits > 1) {
        const int64_t ld = static_cast<int64_t>(p.heads) * D;
        const int64_t at = ((static_cast<int64_t>(split) * p.P + rk) * p.mq + row) * ld + h * D + hf * (D / 2);
        attn_store_rows<D / 2>(lanes + kColDq, hf * (D / 2), p.scale, smem + L::k + (warp - 4) * (32 * D / 2 * 4),
                               p.part + at, ld, rows, n == 0);
      } else {
        attn_store_rows<D / 2>(lanes + kColDq, hf * (D / 2), p.scale, smem + L::k + (warp - 4) * (32 * D / 2 * 2),
                               p.dq[rk] + row * p.ld_dq[rk] + h * D + hf * (D / 2), p.ld_dq[rk], rows, n == 0);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// delta[rank][head][row] = sum_d dO O, D / 8 lanes per (row, head) with 16-byte loads
template <int D>
__global__ void __launch_bounds__(256) delta_kernel(const __grid_constant__ TrainArgs p) {
  constexpr int kLanes = D / 8;
  const int64_t total = static_cast<int64_t>(p.P) * p.mq * p.heads;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int sub = threadIdx.x % kLanes;
  float s = 0.f;
  int rk = 0, h = 0;
  int64_t row = 0;
  if (i < total) {
    h = static_cast<int>(i % p.heads);
    const int64_t r = i / p.heads;
    rk = static_cast<int>(r / p.mq);
    row = r - static_cast<int64_t>(rk) * p.mq;
    const uint4 x = *reinterpret_cast<const uint4*>(p.o[rk] + row * p.ld_o[rk] + h * D + sub * 8);
    const uint4 y = *reinterpret_cast<const uint4*>(p.d_o[rk] + row * p.ld_do[rk] + h * D + sub * 8);
    const uint32_t a[4] = {x.x, x.y, x.z, x.w}, c[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s = fmaf(__uint_as_float(a[k] << 16), __uint_as_float(c[k] << 16), s);
      s = fmaf(__uint_as_float(a[k] & 0xFFFF0000u), __uint_as_float(c[k] & 0xFFFF0000u), s);
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (i < total && sub == 0) p.delta[(static_cast<int64_t>(rk) * p.heads + h) * p.mq + row] = s;
}

// delta += its error, summed over the parts of the walk in order
__global__ void __launch_bounds__(256) delta_add_kernel(const __grid_constant__ TrainArgs p) {
  const int64_t total = static_cast<int64_t>(p.P) * p.heads * p.mq;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  float e = 0.f;
  for (int s = 0; s < p.splits; ++s) e += p.eps[s * total + i];
  p.delta[i] += e;
}

// Sums of the parts in order (the same inputs give the same bits), 4 columns per thread
__global__ void __launch_bounds__(256) part_sum_kernel(const __grid_constant__ PartSumArgs a) {
  if (a.table && a.table[0] == 0) return;
  const int v = blockIdx.y, per_row = a.cols / 4;
  const int64_t total = a.P * a.rows * per_row, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t grow = i / per_row, row = grow % a.rows;
  const int c = static_cast<int>(i - grow * per_row) * 4, rk = static_cast<int>(grow / a.rows);
  if (a.off && (row < a.off[0] || row >= a.off[a.n])) return;
  const float* part = a.part[v] + grow * a.cols + c;
  const int64_t stride = a.P * a.rows * a.cols;
  float4 s = *reinterpret_cast<const float4*>(part);
  for (int k = 1; k < a.splits; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(part + k * stride);
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  *reinterpret_cast<uint2*>(a.out[v][rk] + row * a.ld_out[v][rk] + c) =
      make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

}  // namespace

template <typename K>
static cudaError_t configure(K* kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

cudaError_t attn_bwd_configure() {
  cudaError_t e = configure(attn_dkv_kernel<64, false>, dkv_smem<64>());
  if (e == cudaSuccess) e = configure(attn_dkv_kernel<64, true>, dkv_smem<64>());
  if (e == cudaSuccess) e = configure(attn_dkv_kernel<128, false>, dkv_smem<128>());
  if (e == cudaSuccess) e = configure(attn_dkv_kernel<128, true>, dkv_smem<128>());
  if (e == cudaSuccess) e = configure(attn_dq_kernel<64, false>, dq_smem<64>());
  if (e == cudaSuccess) e = configure(attn_dq_kernel<64, true>, dq_smem<64>());
  if (e == cudaSuccess) e = configure(attn_dq_kernel<128, false>, dq_smem<128>());
  if (e == cudaSuccess) e = configure(attn_dq_kernel<128, true>, dq_smem<128>());
  return e;
}
static_assert(dkv_smem<128>() <= 232448 && dq_smem<128>() <= 232448, "shared memory of one CTA");

cudaError_t attn_delta_launch(const TrainArgs& a, int dim, cudaStream_t s) {
  const int64_t threads = static_cast<int64_t>(a.P) * a.mq * a.heads * (dim / 8);
  if (threads == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>((threads + 255) / 256);
  if (dim == 64) {
    delta_kernel<64><<<grid, 256, 0, s>>>(a);
  } else {
    delta_kernel<128><<<grid, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t attn_part_sum_launch(const PartSumArgs& a, cudaStream_t s) {
  const int64_t work = a.P * a.rows * (a.cols / 4);
  if (work == 0) return cudaSuccess;
  part_sum_kernel<<<dim3(static_cast<unsigned>((work + 255) / 256), a.outputs), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t attn_delta_add_launch(const TrainArgs& a, cudaStream_t s) {
  const int64_t total = static_cast<int64_t>(a.P) * a.heads * a.mq;
  if (total == 0) return cudaSuccess;
  delta_add_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t attn_dkv_launch(const TrainArgs& a, int dim, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.blocks.count) * a.kv_heads * a.P * a.splits;
  if (grid == 0) return cudaSuccess;
  const auto kernel = dim == 64 ? (a.short_walks ? attn_dkv_kernel<64, true> : attn_dkv_kernel<64, false>)
                                : (a.short_walks ? attn_dkv_kernel<128, true> : attn_dkv_kernel<128, false>);
  kernel<<<grid, kThreads, dim == 64 ? dkv_smem<64>() : dkv_smem<128>(), s>>>(a);
  return cudaGetLastError();
}

cudaError_t attn_dq_launch(const TrainArgs& a, int dim, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.blocks.count) * a.heads * a.P * a.splits;
  if (grid == 0) return cudaSuccess;
  const auto kernel = dim == 64 ? (a.short_walks ? attn_dq_kernel<64, true> : attn_dq_kernel<64, false>)
                                : (a.short_walks ? attn_dq_kernel<128, true> : attn_dq_kernel<128, false>);
  kernel<<<grid, kThreads, dim == 64 ? dq_smem<64>() : dq_smem<128>(), s>>>(a);
  return cudaGetLastError();
}

}  // namespace fo

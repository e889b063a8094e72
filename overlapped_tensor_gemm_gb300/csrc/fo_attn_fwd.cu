// Attention forward with row statistics on the tensor cores (tcgen05, accumulators in TMEM):
// one pass over the keys with the running maximum and sum of the softmax.
//
// A CTA takes 256 queries of one head as two tiles of 128 that share every K and V block, so a
// block is loaded once per 256 queries and one tile's softmax runs while the tensor pipe works
// for the other.  384 threads, one CTA per SM: warp 0 loads (TMA), warp 1 issues the MMAs, warps
// 4-7 and 8-11 are the softmax of tile 0 and tile 1 (a thread holds a whole query row: no
// exchange between threads; two threads per row measured 3% slower).
//
// TMEM: per tile the scores (128 columns), the output (head_dim) and the bf16 weights, which the
// product with V reads as its A operand.  A thread's MMAs execute in issue order, which is what
// keeps scores from overwriting weights that are still to be read.  (One issuing warp per tile
// measured 20% slower: the two tiles' products interleave and both finish late.)
//
// The output is rescaled only where a row's maximum grew by more than 2^8 since the last time
// (the sum and the final division use the same reference, so this is exact); the weights, at
// most 2^8, enter the product with V as bf16: half a step, 2^-9 of a weight's binade, as for any
// bf16 operand, averaged over the keys.
// Measured: 8192 tokens, 32 heads on 8, causal 391 us (1407 TFLOP/s of the pairs that attend); 16384
// tokens, 8 heads on 2: 384 us (1431); head_dim 64, 8192 tokens, 16 heads: 178 us (770).  Bound by
// a tile's chain of scores, softmax and P V; the tensor pipe is active about three quarters of the
// time at full size.  These are scores of standard deviation 1; with 4 and 8, where maxima rise by
// more than 2^8 late in a row and their blocks are computed again, 8192 tokens take 570 and 618 us.
#include <cuda_bf16.h>

#include "fo_attn_common.cuh"
#include "fo_internal.h"
#include "fo_ptx.cuh"

namespace fo {
namespace {

constexpr int kThreads = 384;
constexpr int kTileWarps = 4;
constexpr uint32_t kTmem = 512;
constexpr float kRescale = 8.0f;  // log2 units
constexpr float kLn2 = 0.6931471805599453f;

// TMEM columns of tile t.  head_dim 128 fills TMEM: the weights lie over the scores they came from
// and P V has to be issued before the next scores.  head_dim 64 has room for weights of their own:
// the next scores go first and P V leaves the softmax's way.
template <int D>
struct Cols {
  static constexpr bool apart = D == 64;
  __device__ static uint32_t s(int t) { return t * 128; }
  __device__ static uint32_t o(int t) { return 256 + t * D; }
  __device__ static uint32_t p(int t) { return apart ? 384 + t * 64 : t * 128; }
};

template <int D>
struct Smem {
  static constexpr int ks = D == 64 ? 4 : 2, vs = D == 64 ? 4 : 3;  // stages of keys and of values
  static constexpr uint32_t tile = D / 64 * kHalf;
  static constexpr uint32_t q = 0, k = 2 * tile, v = k + ks * tile, ctl = v + vs * tile;
};
constexpr int kMaxStages = 4;
struct alignas(8) Ctl {
  uint64_t q_full[2], k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[2], p_full[2], o_done[2], fix, drain;
  uint32_t tmem_base, pad;
};
template <int D>
constexpr int smem_bytes() {
  return static_cast<int>(Smem<D>::ctl + sizeof(Ctl) + 1024);
}
static_assert(smem_bytes<128>() <= 232448, "shared memory of one CTA");

// A warp's 32 output rows times `scale` as bf16 to `row` (null: not stored), each lane its own; zero:
// nothing was accumulated.  (Turned in shared memory into whole lines first, as the backward does it,
// the kernel took 403 instead of 395 us at 8192 tokens: the walk over the keys spilled more.)
__device__ __forceinline__ void store_rows(uint32_t taddr, int n, float scale, uint16_t* row, bool zero) {
  for (int c = 0; c < n; c += 32) {
    uint32_t v[32];
    if (zero) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = 0u;
    } else {
      tmem_ld32(taddr + c, v);
      tmem_wait_ld();
    }
    if (row) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        st_v4_u32(row + c + 8 * k,
                  pack_bf16x2(__uint_as_float(v[8 * k + 0]) * scale, __uint_as_float(v[8 * k + 1]) * scale),
                  pack_bf16x2(__uint_as_float(v[8 * k + 2]) * scale, __uint_as_float(v[8 * k + 3]) * scale),
                  pack_bf16x2(__uint_as_float(v[8 * k + 4]) * scale, __uint_as_float(v[8 * k + 5]) * scale),
                  pack_bf16x2(__uint_as_float(v[8 * k + 6]) * scale, __uint_as_float(v[8 * k + 7]) * scale));
    }
    __syncwarp();
  }
}

template <int D, bool kShort>
__global__ void __launch_bounds__(kThreads, 1) attn_fwd_kernel(const __grid_constant__ TrainArgs p) {
  using L = Smem<D>;
  constexpr int kKStages = L::ks, kVStages = L::vs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + L::ctl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = p.by_q[0].of(blockIdx.x), ph = blockIdx.x - e * p.heads * p.P;
  const int rk = p.by_q[1].of(ph), h = ph - rk * p.heads;
  Block b;
  if (!block_at(p.blocks, e, &b)) return;
  const int kvh = p.by_group.of(h);
  // first query of each tile and the key blocks it walks
  int q0[2], n[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    q0[t] = b.blk * 2 * kBlk + t * kBlk;
    const int end = q0[t] + kBlk < b.q_len ? q0[t] + kBlk : b.q_len;
    n[t] = q0[t] < b.q_len ? (key_end(p.blocks.causal, end, b.q_len, b.k_len) + kBlk - 1) / kBlk : 0;
  }
  const int nmax = n[0] > n[1] ? n[0] : n[1];
  const bool fine = kShort && nmax <= kFineWalk;  // the rest of the weights over the scores
  const bool apart = Cols<D>::apart && !fine;

  if (threadIdx.x == 0) {
    // the first loads go out before anything else
    mbar_init(&ctl->q_full[0], 1);
    mbar_init(&ctl->q_full[1], 1);
    for (int s = 0; s < kKStages; ++s) mbar_init(&ctl->k_full[s], 1);
    fence_barrier_init();
    fence_proxy_async_shared();
    if (nmax > 0) {
      mbar_arrive_expect_tx(&ctl->k_full[0], L::tile);
      load_block<D>(&p.maps[p.P + rk], smem + L::k, &ctl->k_full[0], kvh * D, b.k0);
    }
    for (int t = 0; t < 2; ++t)
      if (n[t] > 0) {
        mbar_arrive_expect_tx(&ctl->q_full[t], L::tile);
        load_block<D>(&p.maps[rk], smem + L::q + t * L::tile, &ctl->q_full[t], h * D, b.q0 + q0[t]);
      }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&ctl->s_full[t], 1);
      mbar_init(&ctl->p_full[t], kTileWarps);
      mbar_init(&ctl->o_done[t], 1);
    }
    for (int s = 0; s < kKStages; ++s) mbar_init(&ctl->k_empty[s], 1);
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&ctl->v_full[s], 1);
      mbar_init(&ctl->v_empty[s], 1);
    }
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

  if (warp == 0) {  // ---- loads
    uint32_t fix_uses = 0;
    int k_armed = nmax > 0 ? 1 : 0, v_armed = 0;  // blocks whose loads have been issued
    bool ok = true;
    for (int j = 0; ok && j < nmax; ++j) {
      const int ks = j % kKStages, vs = j % kVStages;
      ok = attn_wait(&ctl->k_empty[ks], ((j / kKStages) & 1) ^ 1, p, kSiteEmpty, lane);
      if (!ok) break;
      if (lane == 0 && j > 0) {
        mbar_arrive_expect_tx(&ctl->k_full[ks], L::tile);
        load_block<D>(&p.maps[p.P + rk], smem + L::k + ks * L::tile, &ctl->k_full[ks], kvh * D, b.k0 + j * kBlk);
      }
      k_armed = j + 1;
      ok = attn_wait(&ctl->v_empty[vs], ((j / kVStages) & 1) ^ 1, p, kSiteEmpty, lane) &&
           load_summed<D>(p, &p.maps[2 * p.P + rk], smem + L::v + vs * L::tile, &ctl->v_full[vs], &ctl->fix, fix_uses,
                          kvh * D, b.k0 + j * kBlk, b.k_len - j * kBlk, lane);
      if (ok) v_armed = j + 1;
    }
    if (lane == 0) {  // no copy in flight when the CTA leaves, whichever warp gave up
      for (int t = 0; t < 2; ++t)
        if (n[t] > 0) mbar_wait_drain(&ctl->q_full[t], 0, kAttnDrainNs);
      for (int j = k_armed - kKStages < 0 ? 0 : k_armed - kKStages; j < k_armed; ++j)
        mbar_wait_drain(&ctl->k_full[j % kKStages], (j / kKStages) & 1, kAttnDrainNs);
      for (int j = v_armed - kVStages < 0 ? 0 : v_armed - kVStages; j < v_armed; ++j)
        mbar_wait_drain(&ctl->v_full[j % kVStages], (j / kVStages) & 1, kAttnDrainNs);
    }
  } else if (warp == 1 && nmax > 0) {  // ---- MMAs
    bool ok = attn_wait(&ctl->k_full[0], 0, p, kSiteFull, lane), issued = false;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (!ok || n[t] == 0) continue;
      ok = attn_wait(&ctl->q_full[t], 0, p, kSiteFull, lane);
      if (!ok) continue;
      tc_fence_after();
      if (elect_lane()) {
        issue_scores<D>(tmem + Cols<D>::s(t), sbase + L::q + t * L::tile, sbase + L::k);
        umma_commit(&ctl->s_full[t]);
      }
      __syncwarp();
      issued = true;
    }
    // Waits that do not depend on the softmax stand between two groups of MMAs, where they pass
    // while the first group runs, and the stages that the last block has left are released there.
    int ks = 1, vs = 0;  // stages of block j + 1's keys and of block j's values
    uint32_t kph = 0, vph = 0;
    ok = ok && attn_wait(&ctl->v_full[0], 0, p, kSiteFull, lane);
    for (int j = 0; ok && j < nmax; ++j) {
      const bool more = j + 1 < nmax;
      const int vn = vs + 1 == kVStages ? 0 : vs + 1;
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const bool here = j < (t ? n[1] : n[0]), scores = j + 1 < (t ? n[1] : n[0]);
        auto operands = [&]() -> bool {
          return !more || (t == 0 ? attn_wait(&ctl->k_full[ks], kph, p, kSiteFull, lane)
                                  : attn_wait(&ctl->v_full[vn], vn == 0 ? vph ^ 1 : vph, p, kSiteFull, lane));
        };
        if (apart) ok = operands();
        if (ok && here) {
          ok = attn_wait(&ctl->p_full[t], j & 1, p, kSiteTmemFull, lane);
          if (!ok) break;
          tc_fence_after();
          if (!apart) {
            if (elect_lane()) {
              issue_grad<D, 128>(tmem + Cols<D>::o(t), tmem + Cols<D>::p(t), sbase + L::v + vs * L::tile, j == 0);
              if (fine)
                issue_grad<D, 128>(tmem + Cols<D>::o(t), tmem + Cols<D>::s(t) + 64, sbase + L::v + vs * L::tile, false);
              umma_commit(&ctl->o_done[t]);
            }
            __syncwarp();
          }
        }
        if (!apart) ok = operands();
        if (!ok) break;
        if (elect_lane()) {
          if (scores) {
            issue_scores<D>(tmem + Cols<D>::s(t), sbase + L::q + t * L::tile, sbase + L::k + ks * L::tile);
            umma_commit(&ctl->s_full[t]);
          }
          if (apart && here) {
            issue_grad<D, 128>(tmem + Cols<D>::o(t), tmem + Cols<D>::p(t), sbase + L::v + vs * L::tile, j == 0);
            umma_commit(&ctl->o_done[t]);
          }
          if (t == 0) {  // block j's scores and block j - 1's products with V were the last issued of both tiles
            umma_commit(&ctl->k_empty[ks == 0 ? kKStages - 1 : ks - 1]);
            if (j > 0) umma_commit(&ctl->v_empty[vs == 0 ? kVStages - 1 : vs - 1]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      if (++ks == kKStages) {
        ks = 0;
        kph ^= 1;
      }
      vs = vn;
      if (vs == 0) vph ^= 1;
    }
    if (issued && elect_lane()) {  // and no MMA
      umma_commit(&ctl->drain);
      mbar_wait_drain(&ctl->drain, 0, kAttnDrainNs);
    }
  } else if (warp >= 4) {  // ---- softmax
    const int t = (warp - 4) >> 2, quad = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t sc = lanes + Cols<D>::s(t), oc = lanes + Cols<D>::o(t), pc = lanes + Cols<D>::p(t);
    const int query = q0[t] + quad * 32 + lane;
    const int see = query < b.q_len ? key_end(p.blocks.causal, query + 1, b.q_len, b.k_len) : 0;  // keys of this row
    const int all = key_end(p.blocks.causal, q0[t] + 1, b.q_len, b.k_len);                        // of the tile's first row
    const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
    float m_ref = -INFINITY;
    uint64_t sum = pack2(0.f, 0.f);
    bool ok = true;
    for (int j = 0; j < n[t]; ++j) {
      ok = attn_wait(&ctl->s_full[t], j & 1, p, kSiteTmemFull, lane);
      if (!ok) break;
      tc_fence_after();
      const bool edge = (j + 1) * kBlk > all;  // a block with keys that some row does not see
      const int upto = see - j * kBlk;
      // the row's maximum in this block, four independent chains
      float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto maxima = [&](uint32_t (&w)[32], int c) {
        if (edge) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (c * 32 + k >= upto) w[k] = 0xff800000u;  // -infinity, whatever the key holds
        }
#pragma unroll
        for (int k = 0; k < 16; ++k)
          mq[k & 3] = fmax3(mq[k & 3], __uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
      };
      uint64_t bsum[2];
      uint32_t packed[64];
      auto weights = [&](const uint32_t (&w)[32], int c, uint64_t nm) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float x0, x1;
          unpack2(ffma2(pack2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1])), c2, nm), x0, x1);
          const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
          packed[c * 16 + k] = pack_bf16x2(e0, e1);
          bsum[k & 1] = fadd2(bsum[k & 1], pack2(e0, e1));
        }
      };
      // every chunk of 32 scores: `f`, while the next chunk is on its way from TMEM
      auto chunks = [&](auto&& f) {
        uint32_t wa[32], wb[32];
        tmem_ld32(sc, wa);
        tmem_wait_ld();
        tmem_ld32(sc + 32, wb);
        f(wa, 0);
        tmem_wait_ld();
        tmem_ld32(sc + 64, wa);
        f(wb, 1);
        tmem_wait_ld();
        tmem_ld32(sc + 96, wb);
        f(wa, 2);
        tmem_wait_ld();
        f(wb, 3);
      };
      auto block_max = [&]() { return fmax3(fmaxf(mq[0], mq[1]), mq[2], mq[3]) * p.scale_log2; };
      // The weights against the reference so far, so that they do not wait for this block's
      // maximum; a block that exceeds the reference by more than 2^8 (rare) computes them again.
      float alpha = 1.f;
      bool again = j == 0;
      if (j == 0) {
        chunks([&](uint32_t (&w)[32], int c) { maxima(w, c); });
        m_ref = block_max();
      } else {
        const uint64_t nm = m_ref == -INFINITY ? 0 : pack2(-m_ref, -m_ref);
        bsum[0] = bsum[1] = 0;
        chunks([&](uint32_t (&w)[32], int c) {
          maxima(w, c);
          weights(w, c, nm);
        });
        const float mx = block_max();
        if (mx > m_ref + kRescale) {
          alpha = fast_exp2(m_ref - mx);
          m_ref = mx;
          again = true;
        }
      }
      if (__any_sync(0xffffffffu, again)) {
        const uint64_t nm = m_ref == -INFINITY ? 0 : pack2(-m_ref, -m_ref);  // no key: every weight 0
        bsum[0] = bsum[1] = 0;
        chunks([&](uint32_t (&w)[32], int c) {
          maxima(w, c);
          weights(w, c, nm);
        });
        if (j > 0) {
          // the output must hold every earlier block before it is rescaled
          ok = attn_wait(&ctl->o_done[t], (j - 1) & 1, p, kSiteDrain, lane);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            tmem_ld32(oc + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
            tmem_st32(oc + c, v);
          }
        }
      }
      sum = ffma2(sum, pack2(alpha, alpha), fadd2(bsum[0], bsum[1]));
      if (fine) {
        // chunks from the last: each one's rests go over scores that have been read
        const uint64_t nm = m_ref == -INFINITY ? 0 : pack2(-m_ref, -m_ref);
#pragma unroll
        for (int c = 3; c >= 0; --c) {
          uint32_t w[32], rest[16];
          tmem_ld32(sc + c * 32, w);
          tmem_wait_ld();
          maxima(w, c);  // (the keys that this row does not see)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x0, x1;
            unpack2(ffma2(pack2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1])), c2, nm), x0, x1);
            rest[k] = rest_bf16x2(fast_exp2(x0), fast_exp2(x1), packed[c * 16 + k]);
          }
          tmem_st16(sc + 64 + c * 16, rest);
        }
      }
      if (apart && j > 0) {  // the last block's weights have been read
        ok = attn_wait(&ctl->o_done[t], (j - 1) & 1, p, kSiteDrain, lane);
        if (!ok) break;
        tc_fence_after();
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = packed[c * 32 + k];
        tmem_st32(pc + c * 32, w);
      }
      tmem_wait_st();
      attn_publish(&ctl->p_full[t], lane);
    }
    if (ok && n[t] > 0) ok = attn_wait(&ctl->o_done[t], (n[t] - 1) & 1, p, kSiteDrain, lane);
    if (ok && q0[t] < b.q_len) {
      tc_fence_after();
      float lo, hi;
      unpack2(sum, lo, hi);
      const float l = lo + hi;
      const bool live = query < b.q_len;
      const int64_t row = b.q0 + query;
      const bool none = l == 0.f;  // no key; a NaN among the row's scores stays one in both outputs
      if (live) p.lse[rk][h * p.ld_lse[rk] + row] = none ? -INFINITY : fmaf(m_ref, kLn2, logf(l));
      store_rows(oc, D, none ? 0.f : 1.f / l, live ? p.out_o[rk] + row * p.ld_o[rk] + h * D : nullptr, n[t] == 0);
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

}  // namespace

template <typename K>
static cudaError_t configure(K* kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

cudaError_t attn_fwd_configure() {
  cudaError_t e = configure(attn_fwd_kernel<64, false>, smem_bytes<64>());
  if (e == cudaSuccess) e = configure(attn_fwd_kernel<64, true>, smem_bytes<64>());
  if (e == cudaSuccess) e = configure(attn_fwd_kernel<128, false>, smem_bytes<128>());
  if (e == cudaSuccess) e = configure(attn_fwd_kernel<128, true>, smem_bytes<128>());
  return e;
}

cudaError_t attn_fwd_launch(const TrainArgs& a, int dim, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.blocks.count) * a.heads * a.P;
  if (grid == 0) return cudaSuccess;
  const auto kernel = dim == 64 ? (a.short_walks ? attn_fwd_kernel<64, true> : attn_fwd_kernel<64, false>)
                                : (a.short_walks ? attn_fwd_kernel<128, true> : attn_fwd_kernel<128, false>);
  kernel<<<grid, kThreads, dim == 64 ? smem_bytes<64>() : smem_bytes<128>(), s>>>(a);
  return cudaGetLastError();
}

}  // namespace fo

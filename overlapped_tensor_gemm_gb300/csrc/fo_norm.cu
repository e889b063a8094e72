// Norms before and after a block with gate and residual: argument checks, launch plans and the
// sums over tokens (formulas in fo_norm.cuh).
#include <cmath>
#include <cstring>

#include "fo_host.h"
#include "fo_norm.cuh"

namespace fo {
namespace {

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

// How a call runs: a row's threads (16 columns each), the stages of its matrices, the CTAs
struct Launch {
  NormKernel kernel;
  int threads, grid, smem;
};

fo_status plan_launch(fo_ctx* ctx, NormArgs* a, bool backward, bool r32, bool a32, bool p32, Launch* l) {
  a->tpr = 32;
  while (a->tpr < kNormThreads && a->tpr * 8 * kC < a->cols) a->tpr *= 2;
  if (a->tpr * 8 * kC < a->cols) a->tpr = (a->cols + 32 * 8 * kC - 1) / (32 * 8 * kC) * 32;  // one row per CTA
  l->threads = a->tpr > kNormThreads ? a->tpr : kNormThreads;
  const int rpc = l->threads / a->tpr;
  // matrices that fit two stages are staged, the others are read directly
  uint32_t stage = 0;
  bool vec = a->cols % 8 == 0;
  for (int i = 0; i < kIns; ++i) {
    NormIn& in = a->in[i];
    if (!in.ptr[0]) continue;
    const uint32_t bytes = static_cast<uint32_t>(a->cols) * in.esz / 16 * 16;
    const uint32_t size = (bytes * rpc + 127) / 128 * 128;
    if (bytes == 0 || 2 * (stage + size) > kNormSmem - kNormStatic) {
      vec = false;
      continue;
    }
    in.off = stage;
    in.pitch = in.bytes = bytes;
    stage += size;
  }
  a->stage_bytes = stage;
  // CTAs per SM by registers; two stages and, where they fit as well, the parameters
  int ctas = backward ? (l->threads < 512 ? 512 / l->threads : 1) : 1024 / l->threads;
  while (ctas > 1 && 2 * static_cast<int>(stage) > kNormSmem / ctas - kNormStatic) --ctas;
  const int room = kNormSmem / ctas - kNormStatic;
  // the common form of a whole block has kernels without the tests that the other forms need
  bool full = vec && l->threads <= 512 && a->has_y && a->pre && a->cols == a->tpr * 8 * kC && a->total_rows % rpc == 0;
  full = full && (backward ? a->has_dr && a->gate_mode != kGateToken : a->w_post && a->gate_mode == kGateRow);
  const int slots = backward ? 2 : 1;
  int pitch = (a->cols * 4 + 127) / 128 * 128;
  if (!vec || !(full || (backward && (a->w_post || a->w_pre || a->gate))) ||
      2 * static_cast<int>(stage) + slots * pitch > room)
    pitch = 0;
  // its backward kernels for 256 threads, and all of them for 16-bit matrices, have the parameters
  // placed (a backward with an fp32 stream and 2048 or 4096 columns, where two stages leave no room
  // for them beside a second CTA, runs the general kernel)
  if (pitch == 0 && ((backward && l->threads <= 256) || (!r32 && !a32))) full = false;
  a->par_pitch = pitch;
  a->stages = stage ? (room - slots * pitch) / static_cast<int>(stage) : 2;
  if (a->stages > kNormMaxStages) a->stages = kNormMaxStages;
  a->par_off = a->stages * stage;
  l->smem = static_cast<int>(a->par_off) + slots * pitch;
  if (backward && rpc > 1 && l->smem < rpc * a->cols * 4) l->smem = rpc * a->cols * 4;
  l->kernel = backward ? norm_bwd_kernel_of(r32, a32, p32, vec, full, a->w_post, pitch > 0, l->threads)
                       : norm_fwd_kernel_of(r32, a32, p32, vec, full, pitch > 0, l->threads);
  const int64_t row_groups = (a->total_rows + rpc - 1) / rpc, cap = static_cast<int64_t>(host_num_sms(ctx)) * ctas;
  l->grid = static_cast<int>(row_groups < cap ? row_groups : cap);
  if (l->smem > 44 * 1024 &&
      cudaFuncSetAttribute(l->kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem) != cudaSuccess)
    return host_fail(FO_ERR_CUDA, "norm kernel configuration failed");
  return FO_OK;
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

struct NormCall {
  int64_t m = 0, cols = 0;
  int32_t tr = FO_BF16, ta = FO_BF16, tp = -1;  // residual stream, activations, parameters
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
  const fo_mat* all[3] = {prm->w_post, prm->w_pre, prm->gate};
  for (const fo_mat* v : all) {
    if (!v) continue;
    if (c->tp >= 0 && v->dtype != c->tp)
      return host_fail(FO_ERR_UNSUPPORTED, "w_post, w_pre and gate must have one type");
    c->tp = v->dtype;
  }
  return FO_OK;
}

void fill(const fo_mat* list, int P, void** ptr, int64_t* ld) {
  for (int r = 0; r < P && list; ++r) {
    ptr[r] = list[r].ptr;
    ld[r] = list[r].ld;
  }
}
void fill_in(const fo_mat* list, int P, NormIn* in) {
  for (int r = 0; r < P && list; ++r) {
    in->ptr[r] = list[r].ptr;
    in->ld[r] = list[r].ld;
    in->esz = list[r].dtype == FO_F32 ? 4 : 2;
  }
}
void fill_common(NormArgs* a, fo_ctx* ctx, const NormCall& c, int P, const fo_norm_params* prm) {
  std::memset(a, 0, sizeof(*a));
  a->m = c.m;
  a->total_rows = c.m * P;
  a->cols = static_cast<int32_t>(c.cols);
  a->gate_mode = c.gate_mode;
  if (c.gate_mode == kGateToken) fill_in(prm->gate, P, &a->in[kInGate]);
  if (c.gate_mode == kGateRow) a->gate = prm->gate[0].ptr;
  a->w_post = prm->w_post ? prm->w_post->ptr : nullptr;
  a->w_pre = prm->w_pre ? prm->w_pre->ptr : nullptr;
  a->alpha = prm->residual_scale;
  a->eps = prm->eps;
  fo_opts o;
  std::memset(&o, 0, sizeof(o));
  a->timeout_ns = host_timeout_ns(o);
  a->ctrl = host_ctrl(ctx);
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
  const HostList views[] = {{R, P, false, "R"},         {Y, P, false, "Y"},
                        {R_out, P, true, "R_out"},  {X, P, true, "X"},
                        {prm->gate, prm->gate_per_token ? P : 1, false, "gate"},
                        {prm->w_post, 1, false, "w_post"}, {prm->w_pre, 1, false, "w_pre"}};
  const int in_place[][2] = {{2, 0}, {3, 1}};  // R_out over R, X over Y
  FO_TRY_HOST(host_check_apart(views, 7, in_place, 2));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  if (c.m == 0) return FO_OK;
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  NormArgs a;
  fill_common(&a, ctx, c, P, prm);
  fill_in(R, P, &a.in[kInR]);
  fill_in(Y, P, &a.in[kInY]);
  fill(R_out, P, a.r_out, a.ld_r_out);
  fill(X, P, a.x, a.ld_x);
  a.has_y = Y != nullptr;
  a.pre = X != nullptr;
  Launch l;
  FO_TRY_HOST(plan_launch(ctx, &a, false, c.tr == FO_F32, c.ta == FO_F32, c.tp == FO_F32, &l));
  l.kernel<<<l.grid, l.threads, l.smem, static_cast<cudaStream_t>(stream)>>>(a);
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
  const HostList views[] = {{R_out, P, false, "R_out"}, {Y, P, false, "Y"},   {dX, P, false, "dX"},
                        {dR_out, P, false, "dR_out"}, {dR, P, true, "dR"}, {dY, P, true, "dY"},
                        {prm->gate, token ? P : 1, false, "gate"},
                        {prm->w_post, 1, false, "w_post"}, {prm->w_pre, 1, false, "w_pre"},
                        {grads->gate, token ? P : 1, true, "dgate"},
                        {grads->w_post, 1, true, "dw_post"}, {grads->w_pre, 1, true, "dw_pre"}};
  const int in_place[][2] = {{4, 3}, {5, 2}};  // dR over dR_out, dY over dX
  FO_TRY_HOST(host_check_apart(views, 12, in_place, 2));
  FO_TRY_HOST(host_check_ctx(ctx, P));
  DeviceGuard dev(host_device(ctx));
  if (!dev.ok) return host_fail(FO_ERR_CUDA, "cudaSetDevice failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NormArgs a;
  fill_common(&a, ctx, c, P, prm);
  if (dX) fill_in(R_out, P, &a.in[kInR]);  // without a norm behind, R_out itself is not read
  fill_in(Y, P, &a.in[kInY]);
  fill_in(dX, P, &a.in[kInDx]);
  fill_in(dR_out, P, &a.in[kInDr]);
  fill(dR, P, a.r_out, a.ld_r_out);
  fill(dY, P, a.x, a.ld_x);
  if (token) fill(grads->gate, P, a.dgate, a.ld_dgate);
  a.has_y = Y != nullptr;
  a.pre = dX != nullptr;
  a.has_dr = dR_out != nullptr;
  Launch l;
  FO_TRY_HOST(plan_launch(ctx, &a, true, c.tr == FO_F32, c.ta == FO_F32, c.tp == FO_F32, &l));
  const int grid = l.grid;
  const fo_mat* outs[3] = {grads->w_pre, token ? nullptr : grads->gate, grads->w_post};
  const bool any = outs[0] || outs[1] || outs[2];  // sums over tokens
  if (any) {
    void* part = nullptr;
    const size_t part_bytes = static_cast<size_t>(host_num_sms(ctx)) * 2 * 3 * c.cols * 4;  // two CTAs per SM at most
    FO_TRY_HOST(host_buffer_kept(ctx, kSlotNormPart, part_bytes, s, &part));
    a.part = static_cast<float*>(part);
  }
  if (grid > 0) {
    l.kernel<<<grid, l.threads, l.smem, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  }
  ColSumArgs cs;
  std::memset(&cs, 0, sizeof(cs));
  cs.part = a.part;
  cs.cols = a.cols;
  cs.rows = grid;
  for (int v = 0; v < 3; ++v)
    if (outs[v]) {
      cs.out[v] = outs[v]->ptr;
      cs.f32[v] = outs[v]->dtype == FO_F32;
    }
  if (any) {
    col_sum_kernel<<<dim3((a.cols + 31) / 32, 3), dim3(32, 32), 0, s>>>(cs);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(FO_ERR_CUDA, cudaGetErrorString(e));
  }
  return FO_OK;
}

}  // extern "C"

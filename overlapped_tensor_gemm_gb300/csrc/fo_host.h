// Host services of fo_api.cu used by the other host modules (not public ABI).
#pragma once

#include "fo_internal.h"

#define FO_TRY_HOST(expr)           \
  do {                              \
    fo_status st_ = (expr);         \
    if (st_ != FO_OK) return st_;   \
  } while (0)

namespace fo {
// Workspace slots of host_buffer / host_buffer_kept.
enum HostSlot : int {
  kSlotAttnK = 0,       // query-split attention: K received
  kSlotAttnV = 1,       // query-split attention: V^T slots
  kSlotNormPart = 2,    // norm backward: partial column sums
  kSlotAttnTable = 3,   // attention forward / backward: block tables of packed sequences
  kSlotAttnStats = 4,   // attention backward: per-row statistics
  kSlotAttnPart = 5,    // attention backward: partial sums (dK and dV; dQ and delta's error)
  kSlotLoss = 6,        // policy loss: partial sums; preference loss: row statistics, pairs
  kSlotGradNorm = 7,    // gradient norm: partial sums
};
fo_status host_buffer(fo_ctx* ctx, int slot, size_t bytes, void** out);  // attention workspace slots 0..7
fo_status host_flags(fo_ctx* ctx, uint32_t** out);                       // arrival flags [rank*P + slice]
uint32_t host_next_epoch(fo_ctx* ctx);
uint32_t* host_ctrl(fo_ctx* ctx);
int host_num_sms(fo_ctx* ctx);
cudaStream_t host_link(fo_ctx* ctx, int r);
cudaEvent_t host_ev_hop(fo_ctx* ctx, int r, int t);
fo_status host_fork(fo_ctx* ctx, int P, cudaStream_t s);
fo_status host_join(fo_ctx* ctx, int P, cudaStream_t s);
fo_status host_copy_rows(void* dst, int64_t dld, const void* src, int64_t sld, int64_t rows, int64_t cols,
                         size_t esz, cudaStream_t s);
fo_status host_write_flag(cudaStream_t s, uint32_t* flag, uint32_t value);
fo_status host_encode_map(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                          CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
fo_status host_check_mat(const fo_mat& a, int32_t dtype, const char* what, int r);
fo_status host_fail(fo_status st, const char* msg);
fo_status host_failf(fo_status st, const char* fmt, ...);
fo_status host_check_ctx(const fo_ctx* ctx, int P);  // null context, P out of range
fo_status host_check_opts(const fo_opts* opts);      // null: fine
int host_device(const fo_ctx* ctx);
// As host_buffer, for calls that a stream capture may hold: a buffer that has to grow stays
// allocated until the context is destroyed (a captured launch may still use it), and growth
// while `s` is being captured is refused (FO_ERR_UNSUPPORTED: make the call once before).
fo_status host_buffer_kept(fo_ctx* ctx, int slot, size_t bytes, cudaStream_t s, void** out);
// True when an element of `a` may be an element of `b`: their address ranges meet and, where
// both have one row pitch, so do their column ranges (views of one wider matrix may not).
bool host_mats_overlap(const fo_mat& a, const fo_mat& b);
bool host_same_view(const fo_mat& a, const fo_mat& b);
// The matrices of a call: no written one may meet another, but for pairs of lists that a kernel
// reads before it writes (in_place: written list, read list), rank by rank and as one view.
struct HostList {
  const fo_mat* m;   // null: absent
  int n;
  bool written;
  const char* name;
};
fo_status host_check_apart(const HostList* lists, int n, const int (*in_place)[2] = nullptr, int n_in_place = 0);
bool host_copies_first();  // host order of a ring's copies and the kernel that waits on them
uint64_t host_timeout_ns(const fo_opts& o);
int host_grid(fo_ctx* ctx, const fo_opts& o, int work);
void host_phase_record(fo_ctx* ctx, int i, cudaStream_t s);     // serial baselines' phase events
void host_phase_done(fo_ctx* ctx, bool gemm_first);

// Makes the context's device current for a call and the caller's device again after it.
struct DeviceGuard {
  int before = -1;
  bool ok = false;
  explicit DeviceGuard(int device) {
    if (cudaGetDevice(&before) != cudaSuccess) before = -1;
    ok = cudaSetDevice(device) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (before >= 0) cudaSetDevice(before);
  }
};
}  // namespace fo

// The handle behind the C ABI and the few host-side pieces its entry points share
// (muon_api.cu: the dense step and the orthogonaliser; muon_views.cu: views and 8-bit state).
#pragma once

#include <exception>
#include <utility>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "muon.h"
#include "muon_internal.h"

namespace muon {

constexpr unsigned long long kTimeoutNs = 4000000000ull;  // bounded waits give up after 4 s

// An NVTX range around the host-side enqueue of a call or a stage: it names the stages on a
// profiler's timeline and costs nothing when no profiler is attached.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

struct GroupPlan {
  int m, n, mp, np, cnt;
  bool skinny = false;        // MUON_MODE_HALF: every iteration on chip, no buffers in the workspace
  std::vector<int> mats;      // caller indices, in caller order
  size_t off_x[2], off_a, off_b;
  int scal_base;
  CUtensorMap tm_x[2], tm_a, tm_b;   // row views (K-major operand tiles)
  CUtensorMap tt_x[2], tt_a, tt_b;   // chunked views (MN-major operand tiles)
  CUtensorMap ts_x[2], ts_a, ts_b;   // store views (32 x 32 epilogue tiles)
};

struct Plan {
  std::vector<GroupPlan> groups;
  std::vector<int> mat_group, mat_slot, scal_idx;
  std::vector<int> ew_ntiles;
  std::vector<size_t> off_u;  // MUON_MODE_HALF: a step's normalised direction of each matrix, in the caller's layout
  size_t off_status, off_arrivals, off_rounds, off_deps, off_scal, off_norms, off_partials;
  size_t total;
};

// No exception leaves a C entry point: host tables that cannot be allocated are an error code.
template <typename F>
muon_status_t no_throw(F f) noexcept {
  try {
    return f();
  } catch (const std::exception&) {
    return MUON_ERR_INVALID_ARG;
  }
}

class DeviceGuard {
 public:
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev_) == cudaSuccess && prev_ != dev) {
      if (cudaSetDevice(dev) == cudaSuccess) switched_ = true;
    }
  }
  ~DeviceGuard() {
    if (switched_) cudaSetDevice(prev_);
  }

 private:
  int prev_ = -1;
  bool switched_ = false;
};

}  // namespace muon

struct muon_ctx {
  int device = 0;
  int num_sms = 0;
  muon_dtype_t dtype = MUON_BF16;
  muon_mode_t mode = MUON_MODE_FAST;
  int n = 0;
  std::vector<muon_shape_t> shapes;
  muon::Plan plan;
  char* ws = nullptr;
  size_t ws_bytes = 0;
  unsigned int* d_status = nullptr;
  float* d_scal = nullptr;
  float* d_partials = nullptr;
  float* d_norms = nullptr;   // ||U_i||_F in caller order
  bool fuse_shapes_ok = false;  // every group's real dimensions are multiples of 32, n <= kTcMaxFused
  int schedule = MUON_SCHEDULE_AUTO;
  // launch parameter blocks (tens of KB), reused by every call on this handle
  muon::EwParams ew;
  muon::WrParams wr;
  muon::TcParams tc;
  muon::SmallParams sm;
  muon::NsParams ns;
  muon::ViewParams vw;
  muon::SkinnyParams sk;
  muon::StateParams st;
  std::vector<float> coef;    // MUON_MODE_HALF: (a, b, c) of each iteration; empty: the hyper-parameters'
  // tracing (muon_profile_begin / muon_profile_end)
  int prof_steps_left = 0;
  std::vector<std::pair<int, cudaEvent_t>> prof_events;  // kind (-1: start of a call), event
};

namespace muon {

// muon_api.cu
bool hp_ok(const muon_hparams_t* hp, bool need_momentum);
void trace(muon_ctx* h, int kind, cudaStream_t st);
void trace_call_end(muon_ctx* h);
// Zero the counters that a call uses, in stream order before its kernels: the arrivals, the rounds, and the
// completion counters of a single launch of k iterations (0: none).  What an earlier call left behind, one that overlapped another
// on the handle for instance, does not reach this one.
cudaError_t clear_counters(const muon_ctx* h, int k, cudaStream_t st);
// One group's part of a staged Newton-Schulz launch (operands, output, tile counts; tile_begin is
// the caller's), from X buffer `cur` to `nxt`, Update tiles `tw` wide.
void stage_group(const muon_ctx* h, const GroupPlan& gp, int kind, int cur, int nxt, int tw, TcGroup* G);

// The single-launch schedule over these groups: tile tables (`wide`: with 256 x 512 Update tiles where
// every padded width allows them), and tensor maps.
void fused_tables(const std::vector<const GroupPlan*>& groups, int nslots, int k, bool fuse_write, bool wide, int pairs,
                  NsParams* q);
void fused_maps(const std::vector<const GroupPlan*>& groups, NsParams* q);
// The small-matrix kernel's groups, X_k into buffer `fin`.
void small_groups(const muon_ctx* h, const std::vector<const GroupPlan*>& groups, int fin, SmallParams* p);

// muon_views.cu: the calls of muon_api.cu on a MUON_MODE_HALF handle
muon_status_t half_step(muon_ctx* h, void* const* W, const void* const* G, void* const* M, const muon_hparams_t* hp,
                        cudaStream_t stream);
muon_status_t half_orthogonalize(muon_ctx* h, const void* const* X, void* const* O, const muon_hparams_t* hp,
                                 cudaStream_t stream);
int half_launches(const muon_ctx* h, int k);
bool half_fused_possible(const muon_ctx* h);

}  // namespace muon

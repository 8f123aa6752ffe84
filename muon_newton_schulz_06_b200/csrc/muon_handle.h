// The handle behind the C ABI, shared by the host drivers (muon_api.cu: the optimizer
// step, muon_fp8.cu: the 8-bit operators), and the helpers both use.
#pragma once

#include <string>
#include <utility>
#include <vector>

#include "muon.h"
#include "muon_internal.h"

namespace muon {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct GroupPlan {
  int s = 0, L = 0, n = 0;
  int ld_x = 0, ld_s = 0;
  int gid_base = 0;
  size_t off_x[2] = {0, 0};
  size_t off_gram = 0, off_poly = 0;
  // 3xTF32 mode: the lo parts (the arrays above hold the hi parts)
  size_t off_xlo[2] = {0, 0};
  size_t off_gram_lo = 0, off_poly_lo = 0;
};

struct MatPlan {
  int group = 0, idx = 0, gid = 0;
  int row_base = 0;  // first entry in the NorMuon row arrays (prefix of min(rows, cols))
  int64_t rows = 0, cols = 0;
  bool transposed = false;
  int n_units = 0, part_base = 0, tiles_c = 0;
};

struct ChunkPlan {
  int g_begin = 0, g_end = 0;
  size_t off_tiles[3] = {0, 0, 0};
  // the persistent launch's lists (symmetric products, update): every phase in one
  // matrix priority, larger L first, so a matrix's next phase follows its previous one
  size_t off_ptiles[2] = {0, 0};
  int n_tiles[3] = {0, 0, 0};
};

struct Plan {
  bool valid = false;
  muon_mode mode = MUON_MODE_BF16;
  std::vector<int64_t> sig;  // rows, cols pairs
  std::vector<GroupPlan> groups;
  std::vector<MatPlan> mats;
  std::vector<int> mat_of_gid;  // caller index of each global (group-major) index
  std::vector<ChunkPlan> chunks;
  std::vector<TcTile> tiles;  // host copy of every chunk's tile lists
  size_t off_partials = 0, off_scale = 0, off_tiles = 0, off_rowsq = 0, off_rowf = 0, off_sched = 0, bytes = 0;
  int total_rows = 0;
  int total_units = 0;
  // TMA maps per group (bf16 mode): X K-major (ping/pong), X MN-major (ping/pong), Gram, Poly
  std::vector<CUtensorMap> map_xk[2], map_xmn[2], map_gram, map_poly;
  // output maps (32 x 32 boxes, 64-byte swizzle) for the epilogue's TMA stores
  std::vector<CUtensorMap> map_xout[2], map_gram_out, map_poly_out;
  // 3xTF32 mode (fp32): X K-major and MN-major, Gram, Poly; hi and lo parts
  std::vector<CUtensorMap> t_xk[2][2], t_xmn[2][2], t_gram[2], t_poly[2];
  // debug mode: guard bands after every workspace region (offset, region name), their
  // offsets on the device, and the check's result words
  std::vector<std::pair<size_t, const char*>> guards;
  size_t off_guard_table = 0, off_guard_result = 0;
};

// Kernel kinds of the 8-bit operators follow muon_kernel_kind in the pending timings.
constexpr int kFp8KindBase = MUON_KIND_COUNT;

}  // namespace muon

struct muon_handle {
  int device = 0;
  int sm_count = 148;
  std::string err;
  int last_launches = 0;
  muon::EncodeTiledFn encode = nullptr;
  char* ws = nullptr;
  size_t ws_bytes = 0;
  int* dev_status = nullptr;
  int* host_status = nullptr;
  cudaEvent_t status_event = nullptr;
  bool status_pending = false;
  muon::Plan plan;
  muon::TcApplyTable* apply_table = nullptr;  // host staging of the fused weight-update table
  // TMA momentum pass of tall matrices: the tensor maps of each caller matrix and the
  // pointers they were encoded for (grad, momentum, workspace); cleared with the plan
  std::vector<CUtensorMap> ewmap;
  std::vector<const void*> ewmap_key;
  // the same for the weight-update pass (weights, final workspace X)
  std::vector<CUtensorMap> ewmap_apply;
  std::vector<const void*> ewmap_apply_key;
  // per-launch timing (muon_profile_enable)
  bool profiling = false;
  std::vector<cudaEvent_t> ev_free;
  struct Pending {
    int kind;
    cudaEvent_t a, b;
  };
  std::vector<Pending> ev_pending;
  cudaEvent_t ev_open = nullptr;
  double prof_ms[MUON_KIND_COUNT] = {};
  int64_t prof_launches[MUON_KIND_COUNT] = {};
  // muon_selftest_fail_next_alloc: the next workspace allocation reports failure
  bool fail_next_alloc = false;
  // muon_set_launch_mode
  int launch_mode = MUON_LAUNCH_AUTO;
  unsigned long long stall_ns = 0;  // muon_selftest_stall_persistent (next persistent launch)
  muon::TcPersistParams* persist = nullptr;  // host staging of the persistent launch's parameters
  // MUON_LOG set (and not "0") at muon_init: plan summaries and errors go to stderr
  bool log = false;
  // MUON_DEBUG set (and not "0") at muon_init: guard bands around workspace regions,
  // checked after every call
  bool debug = false;
  // MUON_NVTX set (and not "0") at muon_init: an NVTX range around every call and every
  // kernel launch, for timeline profilers
  bool nvtx = false;
  // the pointer lists of the last two calls that were found to be device memory of
  // `device` (a call with one of them is not checked again; loops often alternate
  // between two sets of buffers)
  std::vector<const void*> checked_ptrs[2];
  int checked_next = 0;
  // 8-bit operators: their kernels record a time-out straight in this page-locked word
  // (the device address is fp8_status_dev), so a call needs no copy to report one
  int* fp8_status = nullptr;
  int* fp8_status_dev = nullptr;
  // the end of the last call on each stream, for muon_sync and muon_destroy: these calls may
  // overlap on several streams (known by their ids, which no later stream gets again)
  struct Fp8Mark {
    unsigned long long stream;
    cudaEvent_t event;
    bool pending;
  };
  std::vector<Fp8Mark> fp8_marks;
  double prof8_ms[MUON_FP8_KIND_COUNT] = {};
  int64_t prof8_launches[MUON_FP8_KIND_COUNT] = {};
};

namespace muon {

// Restores the caller's current device on scope exit.
struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    ok = cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

// Records the detail of an error (and logs it with MUON_LOG); returns st.
muon_status fail(muon_handle* h, muon_status st, const char* fmt, ...) __attribute__((format(printf, 3, 4)));
muon_status cuda_fail(muon_handle* h, cudaError_t e, const char* what);

// Brackets one launch with events on its stream while profiling is on, and with an NVTX
// range when the handle asks for them.  kind: a muon_kernel_kind, or kFp8KindBase + a
// muon_fp8_kernel_kind.
void prof_begin(muon_handle* h, cudaStream_t st, int kind);
void prof_end(muon_handle* h, int kind, cudaStream_t st);

// Reports a device-side time-out of earlier work that has become visible; with `wait`,
// after that work has finished.  st: the stream of the call that asks.
muon_status poll_status(muon_handle* h, bool wait, cudaStream_t st);

}  // namespace muon

// Shared by the host side of the sequence operators (cc3d_seq_plan.cpp:
// plans, argument checks, C entry points) and their kernel files: the plans
// and the launch functions.
#pragma once
#include "cc3d_internal.h"
#include "cc3d_seq.h"

struct cc3d_conv1d_plan {
  cc3d_conv1d_desc_t d{};
  cc3d_seq_info_t info{};
  int32_t seg = 0;        // forward: tokens per thread
  int32_t bwd_seg = 0;    // backward: tokens per step of a thread
  int64_t bwd_rows = 0;   // backward: partial sums of dw and db
};

struct cc3d_scan_plan {
  cc3d_scan_desc_t d{};
  cc3d_seq_info_t info{};
  int32_t chunk = 0;      // forward: tokens per chunk (a multiple of 4; T rounded up when not split)
  int32_t bwd_workers = 0;  // backward: workgroups per channel tile (each takes every bwd_workers-th chunk)
  bool bwd_fits = false;  // backward: no launch has too many threads
};

struct cc3d_join_plan {
  cc3d_join_desc_t d{};
  cc3d_seq_info_t info{};
  int64_t bwd_parts = 0;    // backward: workgroups, each with a row of partial sums
  int64_t gate_parts = 0;   // backward: workgroups per gate row (0: whole gate rows per workgroup)
};

namespace cc3d {

// The runtime takes launches of fewer than 2^32 threads.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
inline bool fits(int64_t workgroups, int threads) { return workgroups <= kMaxThreads / threads; }

// Lanes that hold one row of the block join (8 channels each), a power of two.
inline int join_lanes(int c) {
  int l = 8;
  while (l * 8 < c) l *= 2;
  return l;
}
// Threads of a workgroup: rows of up to a wave share one of four waves, wider
// rows have their own.
constexpr int join_threads(int lanes) { return lanes <= 64 ? 256 : lanes; }

// Threads side by side along the channels (eight each) in a workgroup of the
// convolution's backward pass.
inline int conv1d_lanes(int c) {
  int l = 1;
  while (l < 64 && l * 8 < c) l *= 2;
  return l;
}

// Channels per wave of the scan, and the most states per wave of its forward pass.
constexpr int kScanLanes = 64;
constexpr int kScanFwdStates = 16;
constexpr int kScanMaxStates = 64;

inline int scan_tiles_per_group(const cc3d_scan_desc_t& d) {
  return (d.d / d.groups - 1) / kScanLanes + 1;
}
// States a wave holds, and waves that share one tile of channels.
inline int scan_fwd_ns(const cc3d_scan_desc_t& d) { return d.states <= 4 ? 4 : d.states <= 8 ? 8 : kScanFwdStates; }
inline int scan_fwd_waves(const cc3d_scan_desc_t& d) { return (d.states + scan_fwd_ns(d) - 1) / scan_fwd_ns(d); }
// Lanes that hold a channel's states in a call of one token, four each.
inline int scan_step_lanes(int states) {
  int l = 1;
  while (l * 4 < states) l *= 2;
  return l;
}

// The backward pass' layout.  A lane holds two neighbouring channels with
// four states each; `sg` groups of lanes of a wave hold different states, so a
// wave covers 4 * sg states of 128 / sg channels.  A workgroup is `waves`
// waves of further states by `wc` waves of further channels.
struct ScanBwdShape {
  int sg;       // 1, 2 or 4
  int sub;      // tokens walked back at a time
  int waves, wc;
  int tiles_per_group;
  int chunk;
};
inline ScanBwdShape scan_bwd_shape(const cc3d_scan_desc_t& d) {
  ScanBwdShape v;
  v.sg = d.states <= 4 ? 1 : d.states <= 8 ? 2 : 4;
  v.sub = v.sg == 1 ? 4 : 8;
  v.waves = (d.states + 4 * v.sg - 1) / (4 * v.sg);
  const int wide = d.d / d.groups, each = 128 / v.sg;
  v.wc = 1;
  while (v.wc * 2 * v.waves <= 4 && v.wc * each < wide) v.wc *= 2;
  v.tiles_per_group = (wide - 1) / (each * v.wc) + 1;
  // 64 tokens keep seven states a lane's element between them, 32 those of four-token walks
  const int most = v.sg == 1 ? 32 : 64;
  v.chunk = d.t >= most ? most : (d.t + v.sub - 1) / v.sub * v.sub;
  return v;
}

// Each returns 0, or the runtime's error code when it rejected a launch.
// Arguments have been checked.
int launch_conv1d_forward(const cc3d_conv1d_plan& p, const cc3d_conv1d_args_t& a, void* stream);
int launch_conv1d_backward(const cc3d_conv1d_plan& p, const cc3d_conv1d_args_t& a, void* stream);
int launch_scan_forward(const cc3d_scan_plan& p, const cc3d_scan_args_t& a, void* stream);
int launch_scan_backward(const cc3d_scan_plan& p, const cc3d_scan_args_t& a, void* stream);
int launch_join_forward(const cc3d_join_plan& p, const cc3d_join_args_t& a, void* stream);
int launch_join_backward(const cc3d_join_plan& p, const cc3d_join_args_t& a, void* stream);

// Sums over rows of partial sums, up to kSumJobs of them in one launch:
// dst[m] = sum over r of src[r * stride + m], the rows in a fixed order.  Jobs
// without a dst are left out (cc3d_seq_sum.hip).
struct SumJob {
  const float* src;
  float* dst;
  int64_t rows, cols, stride;
};
constexpr int kSumJobs = 5, kSumThreads = 1024;
inline int64_t sum_workgroups(int64_t cols) { return (cols + 63) / 64; }
int launch_sums(const SumJob* jobs, int n, void* stream);

}  // namespace cc3d

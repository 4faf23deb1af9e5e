// Shared by the host side of the operators on heads and groups
// (cc3d_heads_plan.cpp: plans, argument checks, C entry points) and their
// kernel files: the plans and the launch functions.
#pragma once
#include "cc3d_heads.h"
#include "cc3d_seq_internal.h"

struct cc3d_linear_plan {
  cc3d_linear_desc_t d{};
  bool steps = false;     // forward: the tokens one after another
  cc3d_seq_info_t info{};
  int32_t seg = 0, segs = 1;          // forward: tokens of a segment of the time axis (a multiple of 64), segments
  int32_t bwd_seg = 0, bwd_segs = 1;  // the same of the backward call
  bool bwd_fits = false;              // backward: no launch has too many threads
};

struct cc3d_rotary_plan {
  cc3d_rotary_desc_t d{};
  cc3d_seq_info_t info{};
  double turns[128] = {};  // of each pair, per position: its angle over 2 pi
  int32_t tokens = 1;      // of a workgroup
};

struct cc3d_group_plan {
  cc3d_group_desc_t d{};
  cc3d_seq_info_t info{};
  int32_t splits = 0;      // workgroups per sample; 0: whole samples in a workgroup's registers
  int32_t rows = 0;        // positions of a split
  int32_t bwd_splits = 0, bwd_rows = 0;  // the same of the backward call
  int64_t bwd_stats = 0;   // split: where the statistics are in the backward call's workspace, in floats
  int64_t workers = 0;     // whole samples: workgroups
};

namespace cc3d {

// --- linear attention

constexpr int kLinTokens = 64;   // segments are multiples of so many tokens
constexpr int kLinFew = 32;      // tokens of a block in calls of no more
constexpr int kLinUnits = 256;   // compute units of a card
constexpr int kLinThreads = 512; // at most, of any launch

// Widths as the kernels pad them; tokens of a block (fp32 rows of 256 columns fill
// 160 KB of LDS with fewer); columns of a state that a workgroup holds, 32 a wave,
// where the widest recurrence of a launch has `width`.
inline int linear_pad(int width) { return width <= 64 ? 64 : width <= 128 ? 128 : 256; }
constexpr int linear_tokens(int elem, int pad) { return elem == 4 && pad == 256 ? 32 : 64; }
constexpr int linear_cols(int width) { return width <= 64 ? 64 : 128; }
inline int64_t linear_blocks(int width, int cols) { return (width + cols - 1) / cols; }

// Parts of the backward call's workspace, in floats, in this order.
struct LinearSpace {
  int64_t state;    // one set of segments' states (there are two)
  int64_t blocks;   // each block's state before it, as registers hold it: for the decay's gradient
  int64_t dq, dk, dv;  // sums of shared heads, before they are joined; 0 where no head is shared
  int64_t decay;    // partial sums of dlog_decay
  int64_t total;
};
inline LinearSpace linear_bwd_space(const cc3d_linear_plan& p) {
  const auto& d = p.d;
  LinearSpace s;
  auto up = [](int64_t v) { return (v + 3) / 4 * 4; };
  const int64_t nh = int64_t(d.n) * d.heads, el = nh * d.t;
  s.state = up(nh * (p.bwd_segs - 1) * d.dk * d.dv);
  s.dq = d.q_heads == d.heads ? 0 : up(el * d.dk);
  s.dk = d.k_heads == d.heads ? 0 : up(el * d.dk);
  s.dv = d.v_heads == d.heads ? 0 : up(el * d.dv);
  const int pad = linear_pad(d.dk > d.dv ? d.dk : d.dv), cols = linear_cols(d.dk);
  const int64_t tokens = linear_tokens(d.dtype == CC3D_BF16 ? 2 : 4, pad);
  s.blocks = nh * ((d.t + tokens - 1) / tokens) * linear_blocks(d.dk, cols) * pad * cols;
  s.decay = up(2 * 2 * nh * p.bwd_segs * linear_blocks(d.dk, cols));  // (two recurrences, 64 bits each)
  s.total = 2 * s.state + s.blocks + s.dq + s.dk + s.dv + s.decay;
  return s;
}

int launch_linear_forward(const cc3d_linear_plan& p, const cc3d_linear_args_t& a, void* stream);
int launch_linear_backward(const cc3d_linear_plan& p, const cc3d_linear_args_t& a, void* stream);

// --- rotary

constexpr int kRotaryThreads = 256;
constexpr int kRotaryRow = 4096;  // channels that pass through LDS at a time
int launch_rotary(const cc3d_rotary_plan& p, const cc3d_rotary_args_t& a, bool backward, void* stream);

// --- group norm

// Lanes side by side along the channels (eight each), a power of two, and a
// workgroup's threads.
inline int group_lanes(int c) {
  int l = 1;
  while (l * 8 < c) l *= 2;
  return l;
}
inline int group_threads(int c) { return group_lanes(c) <= 256 ? 256 : group_lanes(c); }
constexpr int kGroupRows = 4;  // rows that a thread keeps in registers

int launch_group_forward(const cc3d_group_plan& p, const cc3d_group_args_t& a, void* stream);
int launch_group_backward(const cc3d_group_plan& p, const cc3d_group_args_t& a, void* stream);

}  // namespace cc3d

// Sizes at the limits of a launch (2^32 threads) and of 32-bit counts, through
// the sequence operators' plans and argument checks under the sanitizers, with
// the launches replaced by ones that only count.
#include <cstdio>
#include <initializer_list>

#include "cc3d_seq_internal.h"

static long launches = 0, checks = 0, failed = 0;

namespace cc3d {
std::atomic<uint64_t> g_fast_path{0}, g_unsupported{0}, g_invalid{0}, g_device_error{0};
int launch_conv1d_forward(const cc3d_conv1d_plan&, const cc3d_conv1d_args_t&, void*) { return ++launches, 0; }
int launch_conv1d_backward(const cc3d_conv1d_plan&, const cc3d_conv1d_args_t&, void*) { return ++launches, 0; }
int launch_scan_forward(const cc3d_scan_plan&, const cc3d_scan_args_t&, void*) { return ++launches, 0; }
int launch_scan_backward(const cc3d_scan_plan&, const cc3d_scan_args_t&, void*) { return ++launches, 0; }
int launch_join_forward(const cc3d_join_plan&, const cc3d_join_args_t&, void*) { return ++launches, 0; }
int launch_join_backward(const cc3d_join_plan&, const cc3d_join_args_t&, void*) { return ++launches, 0; }
}  // namespace cc3d

static void expect(bool ok, const char* what) {
  ++checks;
  if (!ok) {
    ++failed;
    std::printf("failed: %s\n", what);
  }
}

// A buffer of its own, 2^46 bytes from the next.
static void* at(int slot) { return reinterpret_cast<void*>(uintptr_t(slot + 1) << 46); }
static float* f32(int slot) { return static_cast<float*>(at(slot)); }

// The status of a plan; of a forward call on it; of a backward call with the
// gradients of the parameters (asked) or without.
static cc3d_status_t conv(int n, int t, int c, int k, cc3d_status_t* fwd = nullptr, cc3d_status_t* bwd = nullptr, bool asked = false) {
  cc3d_conv1d_desc_t d{n, t, c, k, CC3D_ACT_NONE, CC3D_BF16};
  cc3d_conv1d_plan_t p = nullptr;
  const cc3d_status_t st = causal_conv1d_plan(&d, &p);
  if (st != CC3D_OK) return st;
  cc3d_conv1d_args_t a{};
  a.x = {at(0), int64_t(t) * c, c};
  a.y = {at(1), int64_t(t) * c, c};
  a.w = at(2);
  if (fwd) *fwd = causal_conv1d_forward(p, &a, nullptr);
  a.y = {};
  a.dy = {at(1), int64_t(t) * c, c};
  a.dx = {at(3), int64_t(t) * c, c};
  if (asked) {
    a.dw = f32(4);
    a.db = f32(5);
  }
  a.workspace = at(6);
  a.workspace_bytes = p->info.backward_workspace_bytes;
  if (bwd) *bwd = causal_conv1d_backward(p, &a, nullptr);
  causal_conv1d_plan_destroy(p);
  return st;
}

static cc3d_status_t scan(int n, int t, int c, int s, int g, cc3d_status_t* fwd = nullptr, cc3d_status_t* bwd = nullptr, bool asked = false) {
  cc3d_scan_desc_t d{n, t, c, s, g, 1, CC3D_BF16};
  cc3d_scan_plan_t p = nullptr;
  const cc3d_status_t st = selective_scan_plan(&d, &p);
  if (st != CC3D_OK) return st;
  const int64_t gs = int64_t(g) * s;
  cc3d_scan_args_t a{};
  a.u = a.dt = {at(0), int64_t(t) * c, c};
  a.b = a.c = {at(1), t * gs, gs};
  a.y = {at(2), int64_t(t) * c, c};
  a.a = f32(3);
  a.workspace = at(4);
  a.workspace_bytes = p->info.workspace_bytes;
  if (fwd) *fwd = selective_scan_forward(p, &a, nullptr);
  a.y = {};
  a.dy = a.u;
  a.du = {at(2), int64_t(t) * c, c};
  a.db = {at(5), t * gs, gs};
  if (asked) a.da = f32(6);
  a.workspace_bytes = p->info.backward_workspace_bytes;
  if (bwd) *bwd = selective_scan_backward(p, &a, nullptr);
  selective_scan_plan_destroy(p);
  return st;
}

int main() {
  cc3d_status_t f = CC3D_OK, b = CC3D_OK;
  // the convolution: eight channels and a run of tokens a thread
  expect(conv(1 << 20, 1, 1 << 15, 4) == CC3D_ERR_UNSUPPORTED, "2^32 threads of single tokens");
  expect(conv(1 << 20, 1, (1 << 15) - 8, 4, &f) == CC3D_OK && f == CC3D_OK, "just below");
  expect(conv(1 << 20, 64, 1 << 15, 4, &f) == CC3D_ERR_UNSUPPORTED, "2^32 threads of runs of 64 tokens");
  expect(conv(1, 1, 1 << 26, 3, &f, &b, true) == CC3D_OK && f == CC3D_OK && b == CC3D_ERR_UNSUPPORTED,
         "parameter gradients of 4 * 2^26 columns");
  expect(conv(1, 1, 1 << 26, 3, nullptr, &b, false) == CC3D_OK && b == CC3D_OK, "the same call without them");
  expect(conv(1, 1, 1 << 25, 3, nullptr, &b, true) == CC3D_OK && b == CC3D_OK, "half as many");
  // the scan, one token: four states a lane
  expect(scan(1 << 19, 1, 2048, 16, 1) == CC3D_ERR_UNSUPPORTED, "2^32 lanes of single tokens");
  expect(scan((1 << 19) - 1, 1, 2048, 16, 1, &f, &b) == CC3D_OK && f == CC3D_OK && b == CC3D_OK, "one sequence fewer");
  // many tokens: 64 channels by up to 16 states a wave
  expect(scan(1 << 20, 2, 2048, 64, 1) == CC3D_ERR_UNSUPPORTED, "2^33 threads");
  expect(scan(1 << 20, 64, 1 << 11, 16, 1, &f, &b) == CC3D_OK && f == CC3D_OK && b == CC3D_OK, "2^31 threads, one chunk");
  // the backward call's chunks are more launches' threads than the forward call's one
  expect(scan(1 << 20, 129, 1 << 11, 16, 1, &f, &b) == CC3D_OK && f == CC3D_OK && b == CC3D_ERR_UNSUPPORTED,
         "2^31 threads forward, three times as many backward");
  // dB and dC of 2^33 values, joins of 2^26 workgroups: their grids go on in turns
  expect(scan(1024, 8192, 128, 64, 4, &f, &b, true) == CC3D_OK && f == CC3D_OK && b == CC3D_OK, "values in turns");
  expect(scan(32768, 65, 1024, 64, 1, &f, &b, true) == CC3D_OK && f == CC3D_OK && b == CC3D_OK, "joins in turns");
  // dA of 2^28 columns and more
  expect(scan(1, 1, 1 << 22, 64, 1, &f, &b, true) == CC3D_OK && f == CC3D_OK && b == CC3D_ERR_UNSUPPORTED, "dA");
  expect(scan(1, 1, 1 << 22, 64, 1, &f, &b, false) == CC3D_OK && b == CC3D_OK, "without dA");
  // more elements than addresses
  expect(scan(1 << 20, 1 << 20, 1 << 20, 1, 1) == CC3D_ERR_UNSUPPORTED, "2^60 elements");
  expect(scan(INT32_MAX, 1 << 30, INT32_MAX, 64, 1) == CC3D_ERR_UNSUPPORTED, "2^92 elements");
  expect(scan(INT32_MAX, 1, INT32_MAX, 64, INT32_MAX) == CC3D_ERR_UNSUPPORTED, "2^62 elements");
  expect(conv(INT32_MAX, 1 << 30, INT32_MAX, 8) == CC3D_ERR_UNSUPPORTED, "2^92 elements");
  // counts next to 2^31
  for (int c : {INT32_MAX, INT32_MAX - 6, INT32_MAX - 7})
    expect(conv(1, 1, c, 1, &f, &b) == CC3D_OK && f == CC3D_OK && b == CC3D_OK, "convolution of 2^31 - 1 channels");
  for (int c : {INT32_MAX, INT32_MAX - 63, INT32_MAX - 510})
    expect(scan(1, 1, c, 1, 1) == CC3D_ERR_UNSUPPORTED, "scan of 2^31 - 1 channels");
  expect(scan(1, 1, INT32_MAX - 511, 1, 1, &f) == CC3D_OK && f == CC3D_OK, "scan of 2^31 - 512 channels");
  expect(scan(1, 1, 1 << 26, 64, 1 << 26, &f, &b) == CC3D_OK && f == CC3D_OK && b == CC3D_ERR_UNSUPPORTED, "2^32 elements of B");
  expect(scan(1, 2, 1 << 26, 64, 1 << 26) == CC3D_ERR_UNSUPPORTED, "the same of two tokens");
  std::printf("%ld checks, %ld failed checks, %ld launches\n", checks, failed, launches);
  return failed != 0;
}

// Drives the host side of the sequence operators (plans and argument checks)
// over a grid of shapes under the sanitizers.  The launch functions are
// replaced by ones that only count: no device is involved.
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

static void* at(int slot) { return reinterpret_cast<void*>(uintptr_t(slot + 1) << 36); }

int main() {
  for (int n : {1, 2, 1560, 1 << 20})
    for (int t : {1, 2, 3, 17, 64, 65, 8193, 1 << 22, 1 << 30})
      for (int c : {1, 7, 8, 96, 500, 2048, 1 << 20}) {
        for (int k : {1, 4, 8, 9}) {
          cc3d_conv1d_desc_t d{n, t, c, k, CC3D_ACT_SILU, CC3D_BF16};
          cc3d_conv1d_plan_t p = nullptr;
          if (causal_conv1d_plan(&d, &p) != CC3D_OK) {
            expect(!p, "no plan after a refusal");
            continue;
          }
          cc3d_seq_info_t info;
          expect(causal_conv1d_plan_info(p, &info) == CC3D_OK && info.backward_workspace_bytes > 0, "conv1d info");
          expect(p->seg >= 1 && p->seg <= t && p->bwd_rows >= 1, "conv1d plan");
          cc3d_conv1d_args_t a{};
          a.x = {at(0), int64_t(t) * c, c};
          a.y = {at(4096), int64_t(t) * c, c};
          a.w = at(20000);
          const bool fits = int64_t(n) * t <= (int64_t(1) << 40) / c;
          if (fits) expect(causal_conv1d_forward(p, &a, nullptr) == CC3D_OK, "conv1d forward");
          a.y.p = a.x.p;
          expect(causal_conv1d_forward(p, &a, nullptr) == CC3D_ERR_INVALID_ARG, "conv1d in place");
          causal_conv1d_plan_destroy(p);
        }
        for (int s : {1, 5, 16, 64, 65}) {
          cc3d_scan_desc_t d{n, t, c, s, c % 4 == 0 ? 4 : 1, 1, CC3D_F32};
          cc3d_scan_plan_t p = nullptr;
          if (selective_scan_plan(&d, &p) != CC3D_OK) {
            expect(!p, "no plan after a refusal");
            continue;
          }
          expect(int64_t(p->chunk) * p->info.chunks >= t && int64_t(cc3d::scan_bwd_shape(d).chunk) * p->info.backward_chunks >= t,
                 "chunks cover the tokens");
          expect(p->bwd_workers >= 1 && p->info.workspace_bytes >= 0 && p->info.backward_workspace_bytes > 0, "scan plan");
          // two halves of one projection are read and written in place of each other's columns
          cc3d_scan_args_t a{};
          a.u = {at(0), int64_t(2) * t * c, 2 * c};
          a.y = {static_cast<float*>(at(0)) + c, int64_t(2) * t * c, 2 * c};
          a.dt = {at(8192), int64_t(t) * c, c};
          a.b = a.c = {at(40000), int64_t(t) * d.groups * s, int64_t(d.groups) * s};
          a.a = static_cast<const float*>(at(60000));
          a.h_in = static_cast<const float*>(at(80000));
          a.h_out = const_cast<float*>(a.h_in);
          a.workspace = at(100000);
          a.workspace_bytes = p->info.workspace_bytes;
          const bool fits = int64_t(n) * t <= (int64_t(1) << 40) / c / 64;
          if (fits) expect(selective_scan_forward(p, &a, nullptr) == CC3D_OK, "scan forward on halves");
          a.y.p = static_cast<float*>(at(0)) + c - 1;
          expect(selective_scan_forward(p, &a, nullptr) == CC3D_ERR_INVALID_ARG, "halves that overlap");
          selective_scan_plan_destroy(p);
        }
        for (int64_t g : {int64_t(1), int64_t(3), INT64_MAX}) {
          cc3d_join_desc_t d{int64_t(n) * t, g, c, CC3D_NORM_RMS, CC3D_NORM_LAYER, CC3D_ACT_NONE, CC3D_ACT_SILU, 1e-6f, CC3D_BF16};
          cc3d_join_plan_t p = nullptr;
          if (norm_join_plan(&d, &p) != CC3D_OK) {
            expect(!p, "no plan after a refusal");
            continue;
          }
          expect(p->bwd_parts >= 1 && p->bwd_parts <= 4096, "join workgroups");
          norm_join_plan_destroy(p);
        }
      }
  expect(launches > 0, "accepted calls reach the launch");
  std::printf("%ld checks, %ld failed checks\n", checks, failed);
  return failed != 0;
}

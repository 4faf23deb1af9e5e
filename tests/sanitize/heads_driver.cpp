// Drives the host side of the operators on heads and groups (plans and argument
// checks) over a grid of shapes, sizes next to the limits among them, under the
// sanitizers.  The launch functions are replaced by ones that only count: no
// device is involved.
#include <cstdio>
#include <initializer_list>

#include "cc3d_heads_internal.h"

static long launches = 0, checks = 0, failed = 0;

namespace cc3d {
std::atomic<uint64_t> g_fast_path{0}, g_unsupported{0}, g_invalid{0}, g_device_error{0};
int launch_linear_forward(const cc3d_linear_plan&, const cc3d_linear_args_t&, void*) { return ++launches, 0; }
int launch_linear_backward(const cc3d_linear_plan&, const cc3d_linear_args_t&, void*) { return ++launches, 0; }
int launch_rotary(const cc3d_rotary_plan&, const cc3d_rotary_args_t&, bool, void*) { return ++launches, 0; }
int launch_group_forward(const cc3d_group_plan&, const cc3d_group_args_t&, void*) { return ++launches, 0; }
int launch_group_backward(const cc3d_group_plan&, const cc3d_group_args_t&, void*) { return ++launches, 0; }
}  // namespace cc3d

static void expect(bool ok, const char* what) {
  ++checks;
  if (!ok) {
    ++failed;
    std::printf("failed: %s\n", what);
  }
}

static void* at(int slot) { return reinterpret_cast<void*>(uintptr_t(slot + 1) << 48); }

int main() {
  for (int n : {1, 3, 1560, 1 << 20, 1 << 30})
    for (int t : {1, 2, 32, 33, 64, 65, 2049, 8192, 1 << 22, 1 << 30})
      for (int h : {1, 5, 16, 1 << 16})
        for (int dk : {1, 8, 50, 64, 128, 256, 257})
          for (int dv : {1, 64, 100, 256}) {
            cc3d_linear_desc_t d{n, t, h, h, 1, h, dk, dv, 0.5f, t % 2 ? CC3D_BF16 : CC3D_F32};
            cc3d_linear_plan_t p = nullptr;
            if (linear_attention_plan(&d, &p) != CC3D_OK) {
              expect(!p, "no plan after a refusal");
              continue;
            }
            cc3d_seq_info_t info;
            expect(linear_attention_plan_info(p, &info) == CC3D_OK, "linear info");
            expect(info.workspace_bytes >= 0 && info.backward_workspace_bytes > 0, "linear sizes");
            expect(p->steps ? p->segs == 1 : p->seg % cc3d::kLinTokens == 0 && int64_t(p->seg) * p->segs >= t &&
                                                             int64_t(p->seg) * (p->segs - 1) < t, "linear segments");
            expect(p->bwd_seg % cc3d::kLinTokens == 0 && int64_t(p->bwd_seg) * p->bwd_segs >= t &&
                       int64_t(p->bwd_seg) * (p->bwd_segs - 1) < t, "linear backward segments");
            const int64_t wide = int64_t(h) * (dk > dv ? dk : dv);
            cc3d_linear_args_t a{};
            a.q = {at(0), int64_t(t) * wide, wide};
            a.k = {at(1), int64_t(t) * wide, wide};
            a.v = {at(2), int64_t(t) * wide, wide};
            a.o = {at(3), int64_t(t) * wide, wide};
            a.grad_o = {at(4), int64_t(t) * wide, wide};
            a.workspace = at(5);
            a.workspace_bytes = info.workspace_bytes;
            const bool near = int64_t(n) * t <= (int64_t(1) << 40) / wide && (t == 1 || wide < (1 << 24));
            if (near) expect(linear_attention_forward(p, &a, nullptr) == CC3D_OK, "linear forward");
            a.workspace_bytes = info.backward_workspace_bytes;
            if (near) expect(linear_attention_backward(p, &a, nullptr) == (p->bwd_fits ? CC3D_OK : CC3D_ERR_UNSUPPORTED),
                             "linear backward");
            linear_attention_plan_destroy(p);
          }
  for (int n : {1, 64, 1 << 22, 1 << 30})
    for (int t : {1, 7, 8192, 1 << 30})
      for (int hq : {1, 16, 1 << 24})
        for (int hk : {0, 4})
          for (int d : {2, 64, 100, 1024})
            for (int scaling : {0, 1, 2, 3}) {
              cc3d_rotary_desc_t r{n, t, hq, hk, d, d < 256 ? d : 256, 0, 0, scaling, CC3D_BF16, 1e4, 4.0, 4096.0, 32.0, 1.0, 1.0};
              cc3d_rotary_plan_t p = nullptr;
              if (rotary_plan(&r, &p) != CC3D_OK) {
                expect(!p, "no plan after a refusal");
                continue;
              }
              expect(p->tokens >= 1 && p->tokens <= 16, "rotary tokens");
              for (int j = 0; j < r.rot / 2; ++j) expect(p->turns[j] > 0 && p->turns[j] < 0.16, "rotary turns");
              const int64_t wide = int64_t(hq + hk) * d;
              cc3d_rotary_args_t a{};
              a.q = {at(0), t * wide, wide};
              a.q_out = {at(1), t * wide, wide};
              if (hk) {
                a.k = {at(2), t * wide, wide};
                a.k_out = {at(3), t * wide, wide};
              }
              if (int64_t(n) * t <= (int64_t(1) << 40) / wide) {
                expect(rotary_forward(p, &a, nullptr) == CC3D_OK, "rotary forward");
                a.q_out = a.q;
                a.k_out = a.k;
                expect(rotary_backward(p, &a, nullptr) == CC3D_OK, "rotary in place");
              }
              rotary_plan_destroy(p);
            }
  for (int n : {1, 3, 8192, 1 << 24})
    for (int p0 : {1, 4, 5, 33, 1560, 230400, 1 << 30})
      for (int c : {1, 7, 8, 37, 192, 515, 2048, 8192})
        for (int g : {1, c}) {
          cc3d_group_desc_t d{n, p0, c, g, CC3D_ACT_SILU, 1e-5f, CC3D_BF16};
          cc3d_group_plan_t p = nullptr;
          if (group_norm_plan(&d, &p) != CC3D_OK) {
            expect(!p, "no plan after a refusal");
            continue;
          }
          cc3d_seq_info_t info;
          expect(group_norm_plan_info(p, &info) == CC3D_OK && info.backward_workspace_bytes > 0, "group info");
          expect(p->splits ? int64_t(p->rows) * p->splits >= p0 && int64_t(p->rows) * (p->splits - 1) < p0 : p->workers >= 1,
                 "group runs");
          expect(!p->bwd_splits == !p->splits && (!p->splits || (int64_t(p->bwd_rows) * p->bwd_splits >= p0 &&
                 int64_t(p->bwd_rows) * (p->bwd_splits - 1) < p0 && p->bwd_stats >= int64_t(p->splits) * n * g * 2)),
                 "group runs backward");
          cc3d_group_args_t a{};
          a.x = {at(0), int64_t(p0) * c, c};
          a.y = {at(1), int64_t(p0) * c, c};
          a.dy = {at(2), int64_t(p0) * c, c};
          a.workspace = at(5);
          a.workspace_bytes = info.workspace_bytes;
          if (int64_t(n) * p0 <= (int64_t(1) << 40) / c) {
            expect(group_norm_forward(p, &a, nullptr) == CC3D_OK, "group forward");
            a.workspace_bytes = info.backward_workspace_bytes;
            expect(group_norm_backward(p, &a, nullptr) == CC3D_OK, "group backward");
          }
          group_norm_plan_destroy(p);
        }
  std::printf("%ld checks, %ld launches, %ld failed checks\n", checks, launches, failed);
  return failed != 0;
}

// Argument checks shared by the host sides of the sequence operators
// (cc3d_seq_plan.cpp) and of the operators on heads and groups
// (cc3d_heads_plan.cpp).
#pragma once
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>
#include <numeric>

#include "cc3d_seq_internal.h"

namespace {

inline cc3d_status_t refuse(cc3d_status_t s) {
  if (s == CC3D_ERR_UNSUPPORTED) cc3d::g_unsupported.fetch_add(1, std::memory_order_relaxed);
  if (s == CC3D_ERR_INVALID_ARG) cc3d::g_invalid.fetch_add(1, std::memory_order_relaxed);
  return s;
}

inline cc3d_status_t launched(int err) {
  if (err == 0) {
    cc3d::g_fast_path.fetch_add(1, std::memory_order_relaxed);
    return CC3D_OK;
  }
  cc3d::g_device_error.fetch_add(1, std::memory_order_relaxed);
  return CC3D_ERR_DEVICE;
}

inline int64_t ceildiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool known_dtype(int32_t v) { return v == CC3D_F32 || v == CC3D_BF16; }
inline bool known_act(int32_t v) { return v == CC3D_ACT_NONE || v == CC3D_ACT_SILU; }
inline bool known_norm(int32_t v) { return v == CC3D_NORM_NONE || v == CC3D_NORM_RMS || v == CC3D_NORM_LAYER; }
inline int64_t elem_of(int32_t dtype) { return dtype == CC3D_BF16 ? 2 : 4; }

// Work in flight the kernels are sized for: compute units of the target
// (MI355X) and its SIMDs; the kernels run on any count.
constexpr int64_t kUnits = 256;
constexpr int64_t kSimds = 1024;
// The addresses a view may span.
constexpr int64_t kMaxSpan = int64_t(1) << 46;
// Tokens of one call: token counters are 32 bits and run a chunk past the end.
constexpr int32_t kMaxTokens = 1 << 30;

// The memory a tensor covers: rows of `width` bytes at base + n*batch + t*row.
struct Region {
  uintptr_t base = 0;
  int64_t batch = 0, row = 0, n = 1, t = 1, width = 0;
  bool out = false;
  int64_t span() const { return (n - 1) * batch + (t - 1) * row + width; }
};

inline bool intersect(const Region& a, const Region& b) {
  if (a.width == 0 || b.width == 0) return false;
  if (a.base + uintptr_t(a.span()) <= b.base || b.base + uintptr_t(b.span()) <= a.base) return false;
  // Both lie on a lattice of period g: disjoint if their rows are disjoint modulo g
  // (two parts of one wider projection).
  int64_t g = 0;
  for (const Region* r : {&a, &b}) {
    if (r->n > 1) g = std::gcd(g, r->batch);
    if (r->t > 1) g = std::gcd(g, r->row);
  }
  if (g == 0) return true;
  const int64_t at = int64_t(b.base >= a.base ? (b.base - a.base) % uintptr_t(g)
                                              : (g - int64_t((a.base - b.base) % uintptr_t(g))) % g);
  return !(at >= a.width && at + b.width <= g);
}

// Rows of an output must not overlap each other.
inline bool self_overlaps(const Region& r) {
  if (r.n > 1 && r.t > 1) {
    const bool rows_inside = r.row >= r.width && r.batch >= (r.t - 1) * r.row + r.width;
    const bool batches_inside = r.batch >= r.width && r.row >= (r.n - 1) * r.batch + r.width;
    return !(rows_inside || batches_inside);
  }
  if (r.n > 1) return r.batch < r.width;
  if (r.t > 1) return r.row < r.width;
  return false;
}

// Collects the buffers of a call and checks them; the first fault sticks.
class Check {
 public:
  explicit Check(int64_t elem) : elem_(elem) {}

  void view(const cc3d_rows_t& v, int64_t n, int64_t t, int64_t c, bool out, bool required) {
    if (!v.p) {
      if (required) bad_ = true;
      return;
    }
    if (v.batch < 0 || v.row < 0 || (n > 1 && v.batch > kMaxSpan / (n - 1)) || (t > 1 && v.row > kMaxSpan / (t - 1))) {
      bad_ = true;
      return;
    }
    Region r;
    r.base = reinterpret_cast<uintptr_t>(v.p);
    r.batch = n > 1 ? v.batch * elem_ : 0;  // (strides between no two rows say nothing: views that differ there are the same)
    r.row = t > 1 ? v.row * elem_ : 0;
    r.n = n;
    r.t = t;
    r.width = c * elem_;
    r.out = out;
    if (r.base % uintptr_t(elem_) || (out && self_overlaps(r))) bad_ = true;
    add(r);
  }

  void dense(const void* p, int64_t bytes, int64_t align, bool out, bool required) {
    if (!p || bytes == 0) {
      if (!p && required) bad_ = true;
      return;
    }
    Region r;
    r.base = reinterpret_cast<uintptr_t>(p);
    r.width = bytes;
    r.out = out;
    if (r.base % uintptr_t(align)) bad_ = true;
    add(r);
  }

  // p and q may be the very same buffer (a view with the same strides too).
  void same_allowed(const void* p, const void* q) {
    if (p && p == q && same_n_ < kMaxSame) same_[same_n_++] = reinterpret_cast<uintptr_t>(p);
  }

  void workspace(void* p, int64_t have, int64_t need) {
    if (have < 0 || (have > 0 && !p) || have < need) {
      bad_ = true;
      return;
    }
    if (need > 0) dense(p, need, 16, true, true);
  }

  void require(bool ok) { bad_ |= !ok; }

  bool ok() const {
    if (bad_) return false;
    for (int i = 0; i < n_; ++i)
      for (int j = i + 1; j < n_; ++j) {
        if (!(r_[i].out || r_[j].out)) continue;
        bool same = false;
        for (int k = 0; k < same_n_; ++k) same |= r_[i].base == same_[k] && identical(r_[i], r_[j]);
        if (same && alike(r_[i]) > 2) return false;  // a third use of it: another input that is read, or written twice
        if (!same && intersect(r_[i], r_[j])) return false;
      }
    return true;
  }

 private:
  static constexpr int kMax = 32, kMaxSame = 2;
  static bool identical(const Region& a, const Region& b) {
    return a.base == b.base && a.batch == b.batch && a.row == b.row && a.n == b.n && a.t == b.t && a.width == b.width;
  }
  int alike(const Region& r) const {
    int count = 0;
    for (int i = 0; i < n_; ++i) count += identical(r_[i], r);
    return count;
  }
  void add(const Region& r) {
    if (n_ < kMax) r_[n_++] = r;
    else bad_ = true;
  }
  int64_t elem_;
  bool bad_ = false;
  int n_ = 0;
  Region r_[kMax];
  int same_n_ = 0;
  uintptr_t same_[kMaxSame] = {};
};

// Whether the sums of a backward call's parameter gradients fit one launch.
struct Summed {
  const float* dst;
  int64_t cols;
};
inline bool sums_fit(std::initializer_list<Summed> jobs) {
  int64_t workgroups = 0;
  for (const Summed& j : jobs)
    if (j.dst) workgroups += cc3d::sum_workgroups(j.cols);
  return cc3d::fits(workgroups, cc3d::kSumThreads);
}

template <class Plan, class Desc>
Plan* make_plan(const Desc* d) {
  Plan* p = new (std::nothrow) Plan;
  if (p) p->d = *d;
  return p;
}

}  // namespace


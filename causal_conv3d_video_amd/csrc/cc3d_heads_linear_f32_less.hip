// The recurrences of linear attention: fp32 tensors, widths some less than eight.
#include "cc3d_heads_linear.h"

int cc3d::linear_f32_less(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  return start_runs<float, kLess>(a, pad, out, dec, s);
}

// The recurrences of linear attention: fp32 tensors, widths eight or more.
#include "cc3d_heads_linear.h"

int cc3d::linear_f32_rest(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  return start_runs<float, kRest>(a, pad, out, dec, s);
}

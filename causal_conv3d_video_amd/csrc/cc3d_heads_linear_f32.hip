// The recurrences of linear attention on fp32 tensors.
#include "cc3d_heads_linear.h"

int cc3d::linear_runs_f32(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  return start_runs<float>(a, pad, out, dec, s);
}

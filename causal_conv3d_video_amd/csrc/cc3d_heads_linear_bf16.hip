// The recurrences of linear attention on bf16 tensors.
#include "cc3d_heads_linear.h"

int cc3d::linear_runs_bf16(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  return start_runs<bf16_s>(a, pad, out, dec, s);
}

// The recurrences of linear attention: bf16 tensors, widths eight or more.
#include "cc3d_heads_linear.h"

int cc3d::linear_bf16_rest(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  return start_runs<bf16_s, kRest>(a, pad, out, dec, s);
}

// The recurrences of linear attention: bf16 tensors, widths some less than eight.
#include "cc3d_heads_linear.h"

int cc3d::linear_bf16_less(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  return start_runs<bf16_s, kLess>(a, pad, out, dec, s);
}

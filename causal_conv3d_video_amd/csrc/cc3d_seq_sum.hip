// Fixed-order sums over rows of partial sums, several in one launch: the
// parameters' gradients of the sequence operators.
#include "cc3d_seq_device.h"

namespace {

struct SumArgs {
  cc3d::SumJob job[cc3d::kSumJobs];
  unsigned first[cc3d::kSumJobs];  // a job's first workgroup
  int n;
};

// 64 columns a workgroup; each of its 16 waves adds every 16th row, 16 loads
// at a time (a row after another would be a chain of memory latencies), and
// the waves' sums are added in their order.  1020 rows of 2575 columns: 6.6 us.
__global__ __launch_bounds__(cc3d::kSumThreads) void sum_rows(SumArgs a) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x % 64, line = threadIdx.x / 64;
  int k = 0;
  while (k + 1 < a.n && blockIdx.x >= a.first[k + 1]) ++k;
  const cc3d::SumJob job = a.job[k];
  const int64_t m = int64_t(blockIdx.x - a.first[k]) * 64 + lane;
  const float* src = job.src + (m < job.cols ? m : 0);
  float s = 0.f;
  for (int64_t r0 = line; r0 < job.rows; r0 += 256) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t r = r0 + 16 * i;
      v[i] = r < job.rows ? src[r * job.stride] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) s += v[i];
  }
  red[line][lane] = s;
  __syncthreads();
  if (line == 0 && m < job.cols) {
#pragma unroll
    for (int l = 1; l < 16; ++l) s += red[l][lane];
    job.dst[m] = s;
  }
}

}  // namespace

namespace cc3d {

int launch_sums(const SumJob* jobs, int n, void* stream) {
  SumArgs a{};
  unsigned blocks = 0;
  for (int i = 0; i < n; ++i) {
    if (!jobs[i].dst) continue;
    a.job[a.n] = jobs[i];
    a.first[a.n++] = blocks;
    blocks += unsigned(sum_workgroups(jobs[i].cols));
  }
  if (!blocks) return 0;
  return launch(sum_rows, blocks, kSumThreads, 0, static_cast<hipStream_t>(stream), a);
}

}  // namespace cc3d

// accumulate.cu -- each cached token's attention weight added to its record.
//
// The scored attention left every row's scores y (log2 units, -inf where the row does
// not see the key) and the merge every row's natural log-sum-exp.  Token j of a KV head
// gains the softmax weights of the query rows that read it,
//   sum_r 2^(y_r,j - lse_r log2 e),
// R = q_len * G rows at most 16, in one fixed order, so that the record is the same in
// every run.
#include "device.cuh"
#include "launch.h"
#include "score.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 16;

__global__ void __launch_bounds__(kThreads)
    accumulate_kernel(const DecodeArgs a, const WeightRows in, const WeightRows out) {
  __shared__ float lse[kMaxRows];
  grid_dependency_wait();
  const int h = blockIdx.y, s = blockIdx.z;
  const int n = scored_len(a, s);
  if (blockIdx.x * kThreads >= n) return;
  const int from = first_read(a, s, n);
  if (threadIdx.x < a.R) {
    const int i = threadIdx.x / a.G, g = threadIdx.x - i * a.G;
    lse[threadIdx.x] = a.out_lse[((size_t)s * a.q_len + i) * a.Hq + (size_t)h * a.G + g] * kLog2e;
  }
  __syncthreads();
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= n) return;
  float w = in.data ? in.data[s * in.seq_stride + h * in.head_stride + j] : 0.f;
  if (j >= from) {
    const float* row = a.scores + (((int64_t)s * a.Hkv + h) * a.max_len + j) * a.score_row;
    float sum = 0.f;
    for (int r = 0; r < a.R; ++r)
      if (lse[r] != -INFINITY) sum += exp2f(row[r] - lse[r]);
    w += sum;
  }
  out.data[s * out.seq_stride + h * out.head_stride + j] = w;
}

}  // namespace

cudaError_t launch_accumulate(const DecodeArgs& a, const WeightRows& in, const WeightRows& out,
                              cudaStream_t stream) {
  if (a.R > kMaxRows || a.Hkv > 65535 || a.B > 65535) return cudaErrorInvalidValue;
  if (a.max_len == 0) return cudaSuccess;
  const dim3 grid((unsigned)(((int64_t)a.max_len + kThreads - 1) / kThreads), a.Hkv, a.B);
  const cudaError_t e =
      launch_chained(accumulate_kernel, grid, dim3(kThreads), 1, stream, a, in, out);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pkv

// The second pass of the weights' gradients of the row norms (launch_column_sums,
// launch_zero_f32 of row_launch.h), in a unit of its own: one copy of its kernels.
#include "row_launch.h"

namespace tss {

namespace {

// out[col] = sum of n partials (blockIdx.y 1: out1, of the n after them): a workgroup takes 4 L columns; its groups of L
// lanes add every (1024 / L)th partial, a wave's groups are joined by shuffles
// and the 16 waves' sums in order.  L = 8 reads whole lines; narrow rows take
// L = 2, which gives them four times the workgroups.
constexpr int kReduceBlock = 1024;
template <int L>
__global__ __launch_bounds__(kReduceBlock) void column_sums_kernel(int n, int d, const float *partial, float *out0,
                                                                   float *out1) {
  __shared__ f32x4 s[kReduceBlock / 64][L];
  const int g = threadIdx.x / L, l = threadIdx.x % L;
  const int col = (blockIdx.x * L + l) * 4;
  float *out = blockIdx.y ? out1 : out0;
  if (blockIdx.y) partial += int64_t(n) * d;
  float acc[4] = {0, 0, 0, 0};
  if (col < d) {
#pragma unroll 4
    for (int p = g; p < n; p += kReduceBlock / L) {
      const f32x4 v = *reinterpret_cast<const f32x4 *>(partial + int64_t(p) * d + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = L; m < 64; m *= 2) acc[i] += __shfl_xor(acc[i], m);
  if (threadIdx.x % 64 < L) s[threadIdx.x / 64][l] = f32x4{acc[0], acc[1], acc[2], acc[3]};
  __syncthreads();
  const int c = threadIdx.x;
  if (c < 4 * L && blockIdx.x * 4 * L + c < d) {
    float sum = 0;
    for (int i = 0; i < kReduceBlock / 64; ++i) sum += s[i][c / 4][c % 4];
    out[blockIdx.x * 4 * L + c] = sum;
  }
}

__global__ void zero_f32_kernel(int n, float *p) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0;
}

}  // namespace

void launch_column_sums(int64_t n, int64_t d, const float *partial, float *out0, float *out1, hipStream_t s) {
  auto go = [&](auto kernel, int64_t cols) {
    hipLaunchKernelGGL(kernel, dim3(uint32_t((d + cols - 1) / cols), out1 ? 2 : 1), dim3(kReduceBlock), 0, s, int(n),
                       int(d), partial, out0, out1);
  };
  if (d > 2048) go(column_sums_kernel<8>, 32);
  else go(column_sums_kernel<2>, 8);
}

void launch_zero_f32(int64_t n, float *out, hipStream_t s) {
  hipLaunchKernelGGL(zero_f32_kernel, dim3(uint32_t((n + 255) / 256)), dim3(256), 0, s, int(n), out);
}

}  // namespace tss

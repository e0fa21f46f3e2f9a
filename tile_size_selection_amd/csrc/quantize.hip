// Quantisation to 8-bit floating point with a scale for each block of
// 1 x 128 or 128 x 128 elements:
//
//   v = x,  or  v = silu(gate) up  with gate | up the two halves of a row of x
//   scale = max(largest |v| of the block, 1e-30) / largest value of the type
//   q = v / scale, rounded to nearest even
//
// scale is K-block-major, scale[column block][row or row block]: the matrix
// products read the scales of one step of K for consecutive rows.
// Memory-bound: an element is read once, kept in registers while its block's
// maximum is found, and written in 8 bits.
#include "rows.h"

using namespace tss;

namespace {

constexpr int kThreads = 256;

// g / (1 + exp(-g)), to about an ulp: exp(-g) = 2^t with t = -g log2(e) in two
// parts (the rounding of the product alone would cost |g| ulps), and the
// quotient's reciprocal corrected once.  Where exp is 0 or has overflowed to
// infinity the corrections are left out: the reciprocal is 1 or 0.
__device__ __forceinline__ float silu(float g) {
  constexpr float c = -1.44269502162933349609f, c_low = -1.92596299112661746887e-8f;  // -log2(e) in two parts
  const float t = g * c;
  const float low = __builtin_fmaf(g, c_low, __builtin_fmaf(g, c, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  const bool inside = e > 0.0f && e < __builtin_inff();
  const float d = 1.0f + (inside ? __builtin_fmaf(e * 0.693147180559945309f, low, e) : e);
  const float r = __builtin_amdgcn_rcpf(d);
  return g * (inside ? __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r) : r);
}

// v of 8 columns; the gated form reads the second half of the row too.
template <typename T, bool GATED>
struct Source {
  Raw8<T> a, b;
  __device__ __forceinline__ void load(const T *row, int d, int col) {
    a = load8(row + col);
    if constexpr (GATED) b = load8(row + d + col);
  }
  __device__ __forceinline__ void clear() {
    a = zero8<T>();
    if constexpr (GATED) b = zero8<T>();
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    widen8(a, v);
    if constexpr (GATED) {
      float u[8];
      widen8(b, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = silu(v[i]) * u[i];
      }
    }
  }
};

// 1 x 128 blocks.  16 lanes hold a block; a workgroup takes 16 rows (so that
// it writes 16 neighbouring scales) and kBlocks blocks of each, whose loads
// are all in flight before the first is used.
constexpr int kBlocks = 4;

template <typename T, typename Q, bool GATED>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(int rows, int d, const T *x, uint8_t *q, float *scale,
                                                                 int col_groups) {
  const int id = xcd_run(blockIdx.x, gridDim.x);
  const int rg = id / col_groups, cg = id - rg * col_groups;
  const int row = rg * 16 + threadIdx.x / 16;
  const int col0 = cg * (kBlocks * kScaleBlock) + (threadIdx.x % 16) * 8;
  const T *xrow = x + int64_t(row) * d * (GATED ? 2 : 1);
  Source<T, GATED> src[kBlocks];
#pragma unroll
  for (int c = 0; c < kBlocks; ++c) {
    const int col = col0 + c * kScaleBlock;
    if (row < rows && col < d) src[c].load(xrow, d, col);
    else src[c].clear();
  }
#pragma unroll
  for (int c = 0; c < kBlocks; ++c) {
    const int col = col0 + c * kScaleBlock;
    float v[8], amax = 0;
    src[c].values(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_abs(amax, v[i]);
    const BlockScale<Q> s(max16(amax));
    if (row < rows && col < d) {
      *reinterpret_cast<u32x2 *>(q + int64_t(row) * d + col) = pack8(v, s);
      if (threadIdx.x % 16 == 0) scale[int64_t(col / kScaleBlock) * rows + row] = s.scale;
    }
  }
}

// 128 x 128 blocks: a workgroup holds one block, 32 elements a thread.  They
// stay as they were loaded and are widened again for the output: that is
// cheaper than the registers of the fp32 values (the gated values are kept).
constexpr int kBlockThreads = 512;

template <typename T, typename Q, bool GATED>
__global__ __launch_bounds__(kBlockThreads) void quantize_blocks_kernel(int rows, int d, const T *x, uint8_t *q,
                                                                        float *scale, int col_blocks) {
  __shared__ float red[kBlockThreads / 16];
  constexpr int R = kBlockThreads / 16, P = kScaleBlock / R;  // P passes of R rows
  const int id = xcd_run(blockIdx.x, gridDim.x);
  const int rb = id / col_blocks, cb = id - rb * col_blocks;
  const int col = cb * kScaleBlock + (threadIdx.x % 16) * 8;
  const int row0 = rb * kScaleBlock + threadIdx.x / 16;
  Source<T, GATED> src[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int row = row0 + p * R;
    if (row < rows && col < d) src[p].load(x + int64_t(row) * d * (GATED ? 2 : 1), d, col);
    else src[p].clear();
  }
  float v[P][8], amax = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    src[p].values(v[p]);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_abs(amax, v[p][i]);
  }
  amax = max16(amax);
  if (threadIdx.x % 16 == 0) red[threadIdx.x / 16] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) amax = __builtin_elementwise_maximum(amax, red[i]);
  const BlockScale<Q> s(amax);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int row = row0 + p * R;
    if constexpr (!GATED) src[p].values(v[p]);
    if (row < rows && col < d) *reinterpret_cast<u32x2 *>(q + int64_t(row) * d + col) = pack8(v[p], s);
  }
  if (threadIdx.x == 0) scale[int64_t(cb) * ((rows + kScaleBlock - 1) / kScaleBlock) + rb] = s.scale;
}

template <typename T, typename Q, bool GATED>
void launch(int64_t rows, int64_t d, const void *x, int32_t block_rows, void *q, float *scale, hipStream_t s) {
  if (block_rows == 1) {
    const int64_t cg = (d + kBlocks * kScaleBlock - 1) / (kBlocks * kScaleBlock);
    hipLaunchKernelGGL((quantize_rows_kernel<T, Q, GATED>), dim3(uint32_t((rows + 15) / 16 * cg)), dim3(kThreads), 0, s,
                       int(rows), int(d), static_cast<const T *>(x), static_cast<uint8_t *>(q), scale, int(cg));
  } else {
    const int64_t cb = (d + kScaleBlock - 1) / kScaleBlock, rb = (rows + kScaleBlock - 1) / kScaleBlock;
    hipLaunchKernelGGL((quantize_blocks_kernel<T, Q, GATED>), dim3(uint32_t(rb * cb)), dim3(kBlockThreads), 0, s,
                       int(rows), int(d), static_cast<const T *>(x), static_cast<uint8_t *>(q), scale, int(cb));
  }
}

}  // namespace

extern "C" int32_t tss_quantize_fp8(int64_t rows, int64_t d, int32_t dtype, const void *x, int32_t gated,
                                    int32_t fp8, int32_t block_rows, void *q, float *scale, void *stream) {
  if (rows < 0 || d < 1 || rows > INT32_MAX || d > INT32_MAX / 4 || (block_rows != 1 && block_rows != kScaleBlock))
    return TSS_E_ARG;
  if ((dtype != TSS_F16 && dtype != TSS_BF16 && dtype != TSS_F32) || (fp8 != TSS_E4M3 && fp8 != TSS_E5M2))
    return TSS_E_DTYPE;
  if (d % 8) return TSS_E_ALIGN;
  if (rows == 0) return TSS_OK;
  // the launch's thread count is 32 bits (either form has at most this many workgroups)
  if ((rows + 15) / 16 * ((d + 127) / 128) * kThreads > int64_t(UINT32_MAX)) return TSS_E_ARG;
  if (!x || !q || !scale) return TSS_E_ARG;
  if ((reinterpret_cast<uintptr_t>(x) & 15u) || (reinterpret_cast<uintptr_t>(q) & 15u)) return TSS_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto with_q = [&](auto t, auto qt) {
    using T = decltype(t);
    using Q = decltype(qt);
    if (gated) launch<T, Q, true>(rows, d, x, block_rows, q, scale, s);
    else launch<T, Q, false>(rows, d, x, block_rows, q, scale, s);
  };
  auto with_t = [&](auto t) {
    if (fp8 == TSS_E4M3) with_q(t, E4M3{});
    else with_q(t, E5M2{});
  };
  if (dtype == TSS_F16) with_t(_Float16{});
  else if (dtype == TSS_BF16) with_t(__bf16{});
  else with_t(float{});
  return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
}

// Quantisation to 8-bit floating point with a scale for each block of
// 1 x 128 or 128 x 128 elements:
//
//   v = x,  or  v = silu(gate) up  with gate | up the two halves of a row of x
//   scale = max(largest |v| of the block, 1e-30) / largest value of the type
//   q = v / scale, rounded to nearest even (gated, 1 x 128: as in 64 bits, for gates above -87)
//
// scale is K-block-major, scale[column block][row or row block]: the matrix
// products read the scales of one step of K for consecutive rows.
// Memory-bound: an element is read once, kept in registers while its block's
// maximum is found, and written in 8 bits.  bf16 to e4m3 with inputs that are in
// no cache, 16400 x 2048: 22.7 us (4.5 TB/s), gated 38.3 (4.4 TB/s: exp and
// reciprocal take 20 of it behind the loads), gated with 128 x 128 blocks 36.1;
// 128 x 128 blocks, 5000 x 8200: 26.5 us (4.65 TB/s; a large copy: 5.0).
#include "rows.h"

using namespace tss;

namespace {

constexpr int kThreads = 256;

// g / (1 + exp(-g)).  The argument of 2^t is off by half its ulp and by the
// constant's, so a negative g's result is off by 1.22 |g| + 8 halves of a unit
// of fp32 (2^-24 of itself), a positive one's by 8; below about -87 the
// reciprocal is less than the smallest normal number, and the result 0.  Two
// corrections (t in two parts, the reciprocal's remainder) would make it one
// unit for 40 of the 124 vector cycles that an element then takes: 41 us
// against 38 at 16400 x 2048, bf16.  Where the error could matter it is
// computed away (quantize_rows_kernel).
__device__ __forceinline__ float silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896340736f));
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
  // the least of the lane's gates, or 0
  __device__ __forceinline__ float least_gate() const {
    float g[8], least = 0;
    widen8(a, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) least = fminf(least, g[i]);
    return least;
  }
};

// The 8-bit values that 8 gated quotients can have, v * inv being off by at
// most the errors of the value and of the block's largest one (silu's, for
// gates from `gate` up) and a few roundings: the lower and the upper one in
// magnitude.  They differ where a rounding border lies between.
template <typename Q>
struct Rounded {
  u32x2 low, high;
  __device__ __forceinline__ Rounded(const float (&v)[8], float inv, float gate) {
    constexpr float half_unit = 0x1p-24f;
    const float e = __builtin_fmaf(fmaxf(gate, -88.0f), -2.44f * half_unit, 21 * half_unit);
    const float below = __builtin_fmaf(-e, inv, inv), above = __builtin_fmaf(e, inv, inv);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[i] * below;
    low = round8<Q>(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[i] * above;
    high = round8<Q>(f);
  }
  __device__ __forceinline__ bool open() const { return ((low[0] ^ high[0]) | (low[1] ^ high[1])) != 0; }
  // bit i: value i is open
  __device__ __forceinline__ uint32_t which() const {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) r |= uint32_t(((low[i / 4] ^ high[i / 4]) >> (i % 4 * 8) & 0xff) != 0) << i;
    return r;
  }
};

template <typename T>
__device__ __forceinline__ float pick(const Raw8<T> &r, int i) {
  float f[8], x;
  widen8(r, f);
  x = f[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) x = i == j ? f[j] : x;
  return x;
}

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
  uint32_t again = 0;
#pragma unroll
  for (int c = 0; c < kBlocks; ++c) {
    const int col = col0 + c * kScaleBlock;
    float v[8], amax = 0;
    src[c].values(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_abs(amax, v[i]);
    const BlockScale<Q> s(max16(amax));
    u32x2 w;
    if constexpr (GATED) {
      const Rounded<Q> r(v, s.inv, min16(src[c].least_gate()));
      again |= uint32_t(r.open()) << c;
      w = r.low;
    } else {
      w = pack8(v, s);
    }
    if (row < rows && col < d) {
      *reinterpret_cast<u32x2 *>(q + int64_t(row) * d + col) = w;
      if (threadIdx.x % 16 == 0) scale[int64_t(col / kScaleBlock) * rows + row] = s.scale;
    }
  }
  if constexpr (GATED) {
    // The values are computed, and some units of fp32 off.  Where that could
    // round one the other way (one value in 20000) it is computed again in 64
    // bits, as is the value that sets the scale, from memory, once the
    // registers of the others are free.  A block with an infinity or a NaN
    // keeps its fp32 results.
#pragma unroll 1
    for (int c = 0; c < kBlocks; ++c) {
      if (!__any(again >> c & 1)) continue;
      const int col = col0 + c * kScaleBlock;
      Source<T, true> x;
      if (row < rows && col < d) x.load(xrow, d, col);
      else x.clear();
      auto exact = [&](int i) __attribute__((always_inline)) {
        const double g = pick(x.a, i);
        return g / (1.0 + exp(-g)) * double(pick(x.b, i));
      };
      float v[8], amax = 0;
      x.values(v);
      int most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        most = __builtin_fabsf(v[i]) > amax ? i : most;
        amax = max_abs(amax, v[i]);
      }
      const BlockScale<Q> s(max16(amax));
      const Rounded<Q> r(v, s.inv, min16(x.least_gate()));
      const uint32_t open = r.which();
      u32x2 w = r.low;
      double top = fmax(fabs(exact(most)), double(kSmallestAmax));
#pragma unroll
      for (int m = 1; m < 16; m *= 2) top = fmax(top, __shfl_xor(top, m));
      const double inv = double(kLargest<Q>) / top;
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        if (!__any(open >> i & 1)) continue;
        const float t = float(exact(i) * inv);
        const float one[8] = {t, t, t, t, t, t, t, t};
        const uint32_t at = open >> i & 1 ? 0xffu << (i % 4 * 8) : 0u, b = round8<Q>(one)[0] & at;
        w[0] = i < 4 ? (w[0] & ~at) | b : w[0];
        w[1] = i < 4 ? w[1] : (w[1] & ~at) | b;
      }
      if (row < rows && col < d && s.scale < __builtin_inff())
        *reinterpret_cast<u32x2 *>(q + int64_t(row) * d + col) = w;
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
  // the launch's thread count is 32 bits
  const int64_t threads = block_rows == 1 ? (rows + 15) / 16 * ((d + kBlocks * kScaleBlock - 1) / (kBlocks * kScaleBlock)) * kThreads
                                          : (rows + 127) / 128 * ((d + 127) / 128) * kBlockThreads;
  if (threads > int64_t(UINT32_MAX)) return TSS_E_ARG;
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

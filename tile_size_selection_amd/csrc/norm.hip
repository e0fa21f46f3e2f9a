// Root-mean-square norm of x + residual and its gradients.
//
//   h = x + residual                     (fp32; written rounded to x's type)
//   r = 1 / sqrt(mean(h^2) + eps)
//   y = h r w                            (from the fp32 h; x's type, or e4m3 with a scale per 128 columns)
//
// With xhat = h r and g = dy w:
//   dx = dh + r (g - xhat mean(g xhat))  (= the residual's gradient)
//   dw = sum over rows of dy xhat
//
// Both are bound by memory: every element is read and written once and stays
// in registers between the row's reduction and its output.  5000 x 8192, fp16
// with residual: 64 us, 5.1 TB/s (a large copy: 5.0); backward, 16384 x 4096,
// bf16: 102 us, 5.3 TB/s, of which 4.7 us add up dw; 16384 x 4096 bf16 with
// residual: 106 us, to e4m3 96, with rstd 107.  One row of 4096: 2.6 us.  Rows
// narrower than a wave's 512 columns leave its lanes idle: 2^20 x 128, bf16, 338
// us (1.6 TB/s), backward 356 (3.0 TB/s).
#include "row_launch.h"

using namespace tss;

namespace {

// Sum over the wpr waves that share a row; red has one slot per wave.
__device__ __forceinline__ float row_sum(float v, float *red, int wave, int wpr) {
  v = sum64(v);
  if (wpr == 1) return v;
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  float s = 0;
  for (int i = 0; i < wpr; ++i) s += red[i];
  return s;
}

// A row is held by wpr waves (wpr > 1: one row per workgroup; wpr == 1: one
// row per wave), thread t of it holding columns (c*64*wpr + t)*8 .. +7 for
// c < CH.
template <typename T, bool FP8, int CH>
__global__ __launch_bounds__(kMaxThreads) void rms_norm_kernel(int rows, int d, const T *x, const T *residual,
                                                               const T *weight, float eps, void *y, float *scale,
                                                               T *h_out, float *rstd, int wpr) {
  __shared__ float red[kMaxThreads / 64];
  const int wave = threadIdx.x >> 6;
  const int rpb = (blockDim.x >> 6) / wpr;
  const int t = wpr == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int row = xcd_run(blockIdx.x, gridDim.x) * rpb + (wpr == 1 ? wave : 0);
  if (row >= rows) return;  // wpr > 1: rpb == 1, the whole workgroup
  const int64_t base = int64_t(row) * d;
  const int step = wpr * 64 * 8;

  Raw8<T> xr[CH], rr[CH], wr[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = t * 8 + c * step;
    const bool in = col < d;
    xr[c] = in ? load8(x + base + col) : zero8<T>();
    rr[c] = in && residual ? load8(residual + base + col) : zero8<T>();
    wr[c] = in ? load8(weight + col) : zero8<T>();
  }
  float h[CH][8], sq = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    widen8(xr[c], h[c]);
    if (residual) {
      float r[8];
      widen8(rr[c], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] += r[i];
    }
    const int col = t * 8 + c * step;
    if (h_out && col < d) store8(h_out + base + col, h[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sq += h[c][i] * h[c][i];
  }
  const float mean = row_sum(sq, red, wave, wpr) / float(d);
  const float r = 1.0f / __builtin_sqrtf(mean + eps);
  if (rstd && t == 0) rstd[row] = r;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = t * 8 + c * step;
    float w[8], v[8];
    widen8(wr[c], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = h[c][i] * r * w[i];
    if constexpr (FP8) {
      // a block of 128 columns is the chunk of 16 neighbouring lanes; columns
      // past the row hold zeros
      float amax = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = max_abs(amax, v[i]);
      const BlockScale<E4M3> s(max16(amax));
      if (col < d) {
        *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(y) + base + col) = pack8(v, s);
        if (col % kScaleBlock == 0) scale[int64_t(col / kScaleBlock) * rows + row] = s.scale;
      }
    } else {
      if (col < d) store8(static_cast<T *>(y) + base + col, v);
    }
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; a thread keeps its columns'
// share of dw in registers over the rows, and the workgroup writes it to its
// own slice of the workspace (added up in a fixed order afterwards: no
// atomics, the same bits on every run).
template <typename T, int CH, int D>
__global__ __launch_bounds__(kMaxThreads) void rms_norm_backward_kernel(int rows, int d, const T *dy, const T *hh,
                                                                        const T *weight, const float *rstd, const T *dh,
                                                                        T *dx, float *partial) {
  __shared__ float red[2][kMaxThreads / 64];
  const int wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  const int step = blockDim.x * 8;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = threadIdx.x * 8 + c * step;
    widen8(col < d ? load8(weight + col) : zero8<T>(), w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0;
  }
  // the next D rows' loads are in flight while a row is reduced and written
  Raw8<T> a[D][CH], b[D][CH], e[D][CH];
  auto load_row = [&](int s, int row) __attribute__((always_inline)) {
    const int64_t base = int64_t(row) * d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = threadIdx.x * 8 + c * step;
      const bool in = col < d && row < rows;
      a[s][c] = in ? load8(dy + base + col) : zero8<T>();
      b[s][c] = in ? load8(hh + base + col) : zero8<T>();
      e[s][c] = in && dh ? load8(dh + base + col) : zero8<T>();
    }
  };
#pragma unroll
  for (int s = 0; s < D; ++s) load_row(s, blockIdx.x + s * gridDim.x);
  int slot = 0;
  for (int row0 = blockIdx.x; row0 < rows; row0 += D * gridDim.x) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      const int row = row0 + s * gridDim.x;
      if (row >= rows) break;
      const float r = rstd[row];
      Raw8<T> ca[CH], cb[CH], ce[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        ca[c] = a[s][c];
        cb[c] = b[s][c];
        ce[c] = e[s][c];
      }
      load_row(s, row + D * gridDim.x);
      float dot = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float g[8], h[8];
        widen8(ca[c], g);
        widen8(cb[c], h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xg = h[i] * r * g[i];
          dw[c][i] += xg;
          dot += xg * w[c][i];
        }
      }
      dot = sum64(dot);
      if (nw > 1) {
        // two sets of slots: a wave writes the next row's while others may still read this row's
        if ((threadIdx.x & 63) == 0) red[slot][wave] = dot;
        __syncthreads();
        dot = 0;
        for (int i = 0; i < nw; ++i) dot += red[slot][i];
        slot ^= 1;
      }
      const float m = dot / float(d);
      const int64_t base = int64_t(row) * d;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = threadIdx.x * 8 + c * step;
        if (col >= d) continue;
        float g[8], h[8], o[8];
        widen8(ca[c], g);
        widen8(cb[c], h);
        widen8(ce[c], o);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += r * (g[i] * w[c][i] - h[i] * r * m);
        store8(dx + base + col, o);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = threadIdx.x * 8 + c * step;
    if (col < d) store8(partial + int64_t(blockIdx.x) * d + col, dw[c]);
  }
}

template <typename T, bool FP8>
int32_t launch_norm(int64_t rows, int64_t d, const void *x, const void *residual, const void *weight, float eps, void *y,
                 float *scale, void *h, float *rstd, hipStream_t s) {
  // Few rows: a row's latency is all that counts, so it is spread over as
  // many threads as it has chunks.  Many rows: four chunks a thread keep
  // more loads in flight per wave, and narrow rows need no barrier.
  const RowShape f = row_shape(d, rows < 1024 ? 1 : 4);
  const int block = f.waves == 1 ? 256 : f.waves * 64;
  const int rpb = f.waves == 1 ? 4 : 1;
  const int64_t blocks = (rows + rpb - 1) / rpb;
  if (blocks * block > int64_t(UINT32_MAX)) return TSS_E_ARG;  // the launch's thread count is 32 bits
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(uint32_t(blocks)), dim3(block), 0, s, int(rows), int(d), static_cast<const T *>(x),
                       static_cast<const T *>(residual), static_cast<const T *>(weight), eps, y, scale,
                       static_cast<T *>(h), rstd, f.waves);
  };
  if (f.chunks == 1) go(rms_norm_kernel<T, FP8, 1>);
  else if (f.chunks == 2) go(rms_norm_kernel<T, FP8, 2>);
  else go(rms_norm_kernel<T, FP8, 4>);
  return TSS_OK;
}

// Workgroups of the backward pass: 12 waves a CU and two workgroups at least,
// but each adds 8 bytes a column (its share of dw, written and read) to the 8
// a column that a row of 16-bit elements moves, so no more than one for every
// 4 rows where that still gives every CU one.
int64_t backward_blocks(int64_t rows, int64_t d) {
  constexpr int64_t cus = 256;
  const int64_t per_cu = 12 / row_shape(d, 1).waves, fill = cus * (per_cu > 2 ? per_cu : 2);
  const int64_t n = rows / 4 < cus ? cus : rows / 4 > fill ? fill : rows / 4;
  return rows < n ? rows : n;
}

template <typename T>
void launch_backward(int64_t rows, int64_t d, const void *dy, const void *h, const void *weight, const float *rstd,
                     const void *dh, void *dx, float *partial, hipStream_t s) {
  const RowShape f = row_shape(d, 1);
  const dim3 grid(uint32_t(backward_blocks(rows, d)));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(f.waves * 64), 0, s, int(rows), int(d), static_cast<const T *>(dy),
                       static_cast<const T *>(h), static_cast<const T *>(weight), rstd, static_cast<const T *>(dh),
                       static_cast<T *>(dx), partial);
  };
  if (f.chunks == 1) go(rms_norm_backward_kernel<T, 1, 2>);
  else if (f.chunks == 2) go(rms_norm_backward_kernel<T, 2, 1>);
  else go(rms_norm_backward_kernel<T, 4, 1>);
}

}  // namespace

extern "C" {

int32_t tss_rms_norm(int64_t rows, int64_t d, int32_t dtype, const void *x, const void *residual, const void *weight,
                     float eps, int32_t out_dtype, void *y, float *scale, void *residual_out, float *rstd,
                     void *stream) {
  int32_t st = check_rows(rows, d, dtype);
  if (st != TSS_OK) return st;
  if (out_dtype != dtype && out_dtype != TSS_E4M3) return TSS_E_DTYPE;
  if (!(eps >= 0)) return TSS_E_ARG;
  if (rows == 0) return TSS_OK;
  if (!x || !weight || !y || (out_dtype == TSS_E4M3 && !scale)) return TSS_E_ARG;
  if (misaligned(x) || misaligned(residual) || misaligned(weight) || misaligned(y) || misaligned(residual_out))
    return TSS_E_ALIGN;
  const bool fp8 = out_dtype == TSS_E4M3;
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto t) {
    using T = decltype(t);
    st = fp8 ? launch_norm<T, true>(rows, d, x, residual, weight, eps, y, scale, residual_out, rstd, s)
             : launch_norm<T, false>(rows, d, x, residual, weight, eps, y, scale, residual_out, rstd, s);
  };
  if (dtype == TSS_F16) go(_Float16{});
  else if (dtype == TSS_BF16) go(__bf16{});
  else go(float{});
  if (st != TSS_OK) return st;
  return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
}

int64_t tss_rms_norm_backward_workspace_size(int64_t rows, int64_t d) {
  if (rows < 0 || d < 1 || rows > kMaxRows) return TSS_E_ARG;
  if (d % 8) return TSS_E_ALIGN;
  if (d > kMaxD) return TSS_E_UNSUPPORTED;
  return backward_blocks(rows, d) * d * 4;
}

int32_t tss_rms_norm_backward(int64_t rows, int64_t d, int32_t dtype, const void *dy, const void *h,
                              const void *weight, const float *rstd, const void *dh, void *dx, float *dweight,
                              void *workspace, int64_t workspace_bytes, void *stream) {
  int32_t st = check_rows(rows, d, dtype);
  if (st != TSS_OK) return st;
  if (!dweight) return TSS_E_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) {
    launch_zero_f32(d, dweight, s);
    return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
  }
  if (!dy || !h || !weight || !rstd || !dx) return TSS_E_ARG;
  if (!workspace || workspace_bytes < tss_rms_norm_backward_workspace_size(rows, d)) return TSS_E_ARG;
  if (misaligned(dy) || misaligned(h) || misaligned(weight) || misaligned(dh) || misaligned(dx) ||
      misaligned(workspace))
    return TSS_E_ALIGN;
  float *partial = static_cast<float *>(workspace);
  if (dtype == TSS_F16) launch_backward<_Float16>(rows, d, dy, h, weight, rstd, dh, dx, partial, s);
  else if (dtype == TSS_BF16) launch_backward<__bf16>(rows, d, dy, h, weight, rstd, dh, dx, partial, s);
  else launch_backward<float>(rows, d, dy, h, weight, rstd, dh, dx, partial, s);
  launch_column_sums(backward_blocks(rows, d), d, partial, dweight, nullptr, s);
  return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
}

}  // extern "C"

// 8-bit integers with a scale for each row: tss_quantize_int8 and the host
// side of tss_gemm_int8.
//
//   v = x,  or  v = silu(gate) up  with gate | up the two halves of a row of x
//   scale[row] = max(largest |v| of the row, 1e-30) / 127,  q = v / scale, rounded to nearest even
//
// Quantising is bound by memory: a row is read once and stays in registers
// while its largest magnitude is found: 16384 x 4096, bf16: 39 us (5.2 TB/s),
// 4 x 8192: 2.4.  Gated, which takes exp and a division for each value: 85 (3.9
// TB/s) and 4.4.
#include <atomic>

#include "gemm_int8_kernel.h"
#include "plans.h"
#include "ranges.h"
#include "row_launch.h"

using namespace tss;

namespace {

// ---- quantisation ----

// A row is held by L neighbouring lanes, or (L == 64) by wpr waves, one row
// per workgroup where wpr > 1 (as in the layer norm).
template <typename T, bool GATED, int CH, int L>
__global__ __launch_bounds__(kMaxThreads) void quantize_int8_kernel(int rows, int d, int wpr, const T *x, uint8_t *q,
                                                                    float *scale) {
  __shared__ float red[kMaxThreads / 64];
  if (L < 64) wpr = 1;
  const int lanes = L * wpr, t = threadIdx.x % lanes;
  const int row = xcd_run(blockIdx.x, gridDim.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
  if (row >= rows) return;  // wpr > 1: one row, the whole workgroup
  const T *from = x + int64_t(row) * d * (GATED ? 2 : 1);
  auto col_of = [&](int c) __attribute__((always_inline)) { return (c * lanes + t) * 8; };
  Raw8<T> a[CH], b[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = col_of(c);
    a[c] = col < d ? load8(from + col) : zero8<T>();
    if constexpr (GATED) b[c] = col < d ? load8(from + d + col) : zero8<T>();
  }
  float v[CH][8], amax = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    widen8(a[c], v[c]);
    if constexpr (GATED) {
      float u[8];
      widen8(b[c], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] / (1.0f + expf(-v[c][i])) * u[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_abs(amax, v[c][i]);
  }
  amax = max_lanes<L>(amax);
  if (L == 64 && wpr > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    for (int i = 0; i < wpr; ++i) amax = __builtin_elementwise_maximum(amax, red[i]);
  }
  const BlockScale<I8> s(amax);
  if (t == 0) scale[row] = s.scale;
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (col_of(c) < d) *reinterpret_cast<u32x2 *>(q + int64_t(row) * d + col_of(c)) = pack8(v[c], s);
}

template <typename T, bool GATED>
int32_t launch_quantize(int64_t rows, int64_t d, const void *x, void *q, float *scale, hipStream_t s) {
  // One chunk a thread for few rows, whose latency counts; else two (7000 x 5120, fp16: 21.4 us, with one 32.3).
  const Team f = team_of(d, rows < 1024 || d <= 512 ? 1 : 2);
  const int block = f.waves == 1 ? 256 : f.waves * 64, rpb = f.waves == 1 ? 256 / f.lanes : 1;
  const int64_t blocks = (rows + rpb - 1) / rpb;
  if (blocks * block > int64_t(UINT32_MAX)) return TSS_E_ARG;  // the launch's thread count is 32 bits
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(uint32_t(blocks)), dim3(block), 0, s, int(rows), int(d), f.waves,
                       static_cast<const T *>(x), static_cast<uint8_t *>(q), scale);
  };
  if (f.lanes == 8) go(quantize_int8_kernel<T, GATED, 1, 8>);
  else if (f.lanes == 16) go(quantize_int8_kernel<T, GATED, 1, 16>);
  else if (f.lanes == 32) go(quantize_int8_kernel<T, GATED, 1, 32>);
  else if (f.chunks == 1) go(quantize_int8_kernel<T, GATED, 1, 64>);
  else if (f.chunks == 2) go(quantize_int8_kernel<T, GATED, 2, 64>);
  else go(quantize_int8_kernel<T, GATED, 4, 64>);
  return TSS_OK;
}

// ---- products ----

constexpr int64_t kTwoGiB = int64_t(1) << 31;
constexpr int64_t kMostK = (int64_t(1) << 17) - 1;  // 2^14 of a product, 2^31 of a sum

bool off_by(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

using Tile256 = Int8Geometry<256, 256, 2, 8, 2>;  // with its pieces: large products
using Piece256 = Int8Geometry<128, 256, 3, 8, 2>;
using Tile128 = Int8Geometry<128, 128, 3, 8, 2>;  // also one round of its own
using Tile64 = Int8Geometry<64, 128, 3, 4, 1>;  // two workgroups a CU

constexpr int kRoundsLds = Tile256::LDS_BYTES > Piece256::LDS_BYTES ? Tile256::LDS_BYTES : Piece256::LDS_BYTES;

// Dynamic LDS above 64 KiB needs an attribute per kernel and device: set on the first launch there.
template <typename Kernel>
hipError_t launch_lds(Kernel kernel, std::atomic<uint64_t> &attr_set, const Int8Args &a, int64_t blocks, int threads,
                      int lds, hipStream_t s) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(attr_set.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 163840);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit, std::memory_order_acq_rel);
  }
  hipLaunchKernelGGL(kernel, dim3(uint32_t(blocks)), dim3(threads), lds, s, a);
  return hipGetLastError();
}

template <typename G>
hipError_t launch_tile(const Int8Args &a, int64_t blocks, hipStream_t s) {
  static std::atomic<uint64_t> attr_set{0};
  return launch_lds(gemm_int8_tile_kernel<G>, attr_set, a, blocks, G::THREADS, G::LDS_BYTES, s);
}

hipError_t launch_rounds(const Int8Args &a, int64_t tiles, hipStream_t s) {
  static std::atomic<uint64_t> attr_set{0};
  const int64_t whole = tiles / kCUs * kCUs, rest = tiles - whole;
  if (rest == 0 || tile_pieces(int(rest), false) == 1) return launch_tile<Tile256>(a, tiles, s);
  return launch_lds(gemm_int8_rounds_kernel<Tile256, Piece256, Tile128>, attr_set, a,
                    whole + rest * tile_pieces(int(rest), false), Tile256::THREADS, kRoundsLds, s);
}

hipError_t launch_rows(const Int8Args &a, const Int8RowsLaunch &f, hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(uint32_t(f.workgroups)), dim3(f.waves * 64), f.waves * f.groups * 1024, s, a);
  };
  if (f.groups == 2) go(gemm_int8_rows_kernel<2, 1>);
  else go(gemm_int8_rows_kernel<1, 4>);
  return hipGetLastError();
}

hipError_t launch_join(const Int8Args &a, void *C, int32_t out_dtype, hipStream_t s) {
  const int64_t mn = int64_t(a.M) * a.N;
  const bool vec = a.N % 4 == 0;
  const int64_t want = ((vec ? mn / 4 : mn) + 255) / 256;
  const dim3 grid(uint32_t(want < 8192 ? want : 8192));
  auto go = [&](auto o) {
    using O = decltype(o);
    const int32_t *P = static_cast<const int32_t *>(a.C);
    const int64_t slice = slice_elements(a.M, a.N);
    if (vec) hipLaunchKernelGGL((int8_join_kernel<O, 4>), grid, dim3(256), 0, s, P, static_cast<O *>(C), a.sa, a.sb, mn, a.N, slice, a.splits);
    else hipLaunchKernelGGL((int8_join_kernel<O, 1>), grid, dim3(256), 0, s, P, static_cast<O *>(C), a.sa, a.sb, mn, a.N, slice, a.splits);
  };
  if (out_dtype == TSS_F32) go(float{});
  else if (out_dtype == TSS_F16) go(_Float16{});
  else go(__bf16{});
  return hipGetLastError();
}

int32_t check_product(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX) return TSS_E_ARG;
  if (K % 16) return TSS_E_ALIGN;
  // sums are 32 bits, as are the kernels' byte offsets into A and B
  if (K > kMostK || M * K >= kTwoGiB || N * K >= kTwoGiB) return TSS_E_ARG;
  return TSS_OK;
}

__global__ void zero_words_kernel(int64_t n, uint32_t *p, int tail, uint8_t *rest) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) p[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x < uint32_t(tail)) rest[threadIdx.x] = 0;
}

}  // namespace

extern "C" {

int32_t tss_quantize_int8(int64_t rows, int64_t d, int32_t dtype, const void *x, int32_t gated, void *q, float *scale,
                          void *stream) {
  int32_t st = check_rows(rows, d, dtype, INT32_MAX);
  if (st != TSS_OK) return st;
  if (rows == 0) return TSS_OK;
  if (!x || !q || !scale) return TSS_E_ARG;
  if (misaligned(x) || misaligned(q) || off_by(scale, 4)) return TSS_E_ALIGN;
  Ranges at;
  at.reads(x, rows * d * (dtype == TSS_F32 ? 4 : 2) * (gated ? 2 : 1));
  at.writes(q, rows * d);
  at.writes(scale, rows * 4);
  if (at.clash()) return TSS_E_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto t) {
    using T = decltype(t);
    st = gated ? launch_quantize<T, true>(rows, d, x, q, scale, s) : launch_quantize<T, false>(rows, d, x, q, scale, s);
  };
  if (dtype == TSS_F16) go(_Float16{});
  else if (dtype == TSS_BF16) go(__bf16{});
  else go(float{});
  if (st != TSS_OK) return st;
  return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
}

int64_t tss_gemm_int8_workspace_size(int64_t M, int64_t N, int64_t K) {
  const int32_t st = check_product(M, N, K);
  if (st != TSS_OK) return st;
  if (M == 0 || N == 0 || K == 0) return 0;
  int32_t n, ks;
  split_ranges(K, plan_int8(M, N, K).splits, &n, &ks);
  return n > 1 ? n * slice_elements(M, N) * 4 : 0;
}

int32_t tss_gemm_int8(int64_t M, int64_t N, int64_t K, const void *A, const void *B, const float *sa, const float *sb,
                      void *C, int32_t out_dtype, void *workspace, int64_t workspace_bytes, void *stream) {
  const int32_t st = check_product(M, N, K);
  if (st != TSS_OK) return st;
  if (out_dtype != TSS_F16 && out_dtype != TSS_BF16 && out_dtype != TSS_F32) return TSS_E_DTYPE;
  if (M == 0 || N == 0) return TSS_OK;
  if (!C || (K > 0 && (!A || !B || !sa || !sb))) return TSS_E_ARG;
  if (off_by(A, 16) || off_by(B, 16) || off_by(C, 16) || off_by(sa, 4) || off_by(sb, 4)) return TSS_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (K == 0) {
    const int64_t bytes = M * N * (out_dtype == TSS_F32 ? 4 : 2), words = bytes / 4, want = (words + 255) / 256 + 1;
    hipLaunchKernelGGL(zero_words_kernel, dim3(uint32_t(want < 8192 ? want : 8192)), dim3(256), 0, s, words,
                       static_cast<uint32_t *>(C), int(bytes % 4), static_cast<uint8_t *>(C) + words * 4);
    return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
  }
  const ProductPlan pl = plan_int8(M, N, K);
  Int8Args a{};
  a.A = static_cast<const int8_t *>(A);
  a.B = static_cast<const int8_t *>(B);
  a.sa = sa;
  a.sb = sb;
  a.M = int32_t(M);
  a.N = int32_t(N);
  a.K = int32_t(K);
  split_ranges(K, pl.splits, &a.splits, &a.k_split);
  const bool split = a.splits > 1;
  if (split) {
    if (!workspace || workspace_bytes < a.splits * slice_elements(M, N) * 4) return TSS_E_ARG;
    if (off_by(workspace, 16)) return TSS_E_ALIGN;
  }
  a.C = split ? workspace : C;
  a.out_dtype = split ? kInt8Sums : out_dtype;
  const int64_t tiles_m = (M + pl.bm - 1) / pl.bm, tiles_n = (N + pl.bn - 1) / pl.bn, blocks = tiles_m * tiles_n * a.splits;
  const Int8RowsLaunch rows = int8_rows_launch(M, N, K);
  // the launch's thread count is 32 bits (tiles: 512 threads at most, and a round's pieces)
  const int64_t threads = pl.bn == 16 ? rows.workgroups * rows.waves * 64 : (blocks + 2 * kCUs) * 512;
  if (threads > int64_t(UINT32_MAX)) return TSS_E_ARG;
  Ranges at;
  at.reads(A, M * K);
  at.reads(B, N * K);
  at.reads(sa, M * 4);
  at.reads(sb, N * 4);
  at.writes(C, M * N * (out_dtype == TSS_F32 ? 4 : 2));
  if (split) at.writes(workspace, a.splits * slice_elements(M, N) * 4);
  if (at.clash()) return TSS_E_ARG;
  a.tiles_m = int32_t(tiles_m);
  a.tiles_n = int32_t(tiles_n);
  hipError_t err;
  if (pl.bn == 16) {
    err = launch_rows(a, rows, s);
  } else if (pl.bm == 256) {
    err = launch_rounds(a, blocks, s);
  } else if (pl.bm == 128) {
    err = launch_tile<Tile128>(a, blocks, s);
  } else {
    err = launch_tile<Tile64>(a, blocks, s);
  }
  if (err == hipSuccess && split) err = launch_join(a, C, out_dtype, s);
  return err == hipSuccess ? TSS_OK : TSS_E_HIP;
}

}  // extern "C"

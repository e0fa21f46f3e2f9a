// Products grouped by expert in fp16 / bf16: tss_gemm_grouped and its
// gradients, on the GEMM kernel's group modes (gemm_kernel.h).
#include <atomic>

#include "gemm_kernel.h"

using namespace tss;

namespace {

constexpr int64_t kTwoGiB = int64_t(1) << 31;

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

using Tile256 = Geometry<256, 256, 64, 2, 8, 16>;
using Tile128 = Geometry<128, 128, 64, 2, 4, 16>;
using Tile64 = Geometry<64, 64, 64, 4, 4, 16>;

template <typename G, typename T, int GRP>
hipError_t launch(KernelArgs &a, int64_t z, hipStream_t s, int32_t *status) {
  a.tiles_n = int32_t((int64_t(a.N) + G::BN - 1) / G::BN);
  const int64_t tiles_m = GRP == kGroupGradB ? (int64_t(a.M) + G::BM - 1) / G::BM : max_group_tiles(a.M, a.groups, G::BM);
  a.tiles_m = int32_t(tiles_m);
  a.group_m = a.tiles_m < 4 ? a.tiles_m : 4;
  const int64_t blocks = z * tiles_m * a.tiles_n;
  if (blocks * G::THREADS > int64_t(UINT32_MAX)) {  // the launch's thread count is 32 bits
    *status = TSS_E_ARG;
    return hipSuccess;
  }
  // dynamic LDS above 64 KiB needs an attribute per kernel and device, set on the first launch there
  static std::atomic<uint64_t> attr_set{0};
  auto kernel = tiled_gemm_kernel<G, T, false, GRP>;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(attr_set.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 163840);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit, std::memory_order_acq_rel);
  }
  hipLaunchKernelGGL(kernel, dim3(uint32_t(blocks)), dim3(G::THREADS), G::lds_bytes(false), s, a);
  return hipGetLastError();
}

template <typename T, int GRP>
hipError_t launch_rows(KernelArgs &a, hipStream_t s, int32_t *status) {
  const int64_t rows = a.M / a.groups;  // of an average group
  if (rows <= 64) return launch<Tile64, T, GRP>(a, 1, s, status);
  if (rows <= 256) return launch<Tile128, T, GRP>(a, 1, s, status);
  return launch<Tile256, T, GRP>(a, 1, s, status);
}

template <typename T>
hipError_t launch_grad_b(KernelArgs &a, hipStream_t s, int32_t *status) {
  const int64_t t256 = ((int64_t(a.M) + 255) / 256) * ((int64_t(a.N) + 255) / 256) * a.groups;
  if (t256 >= 512) return launch<Tile256, T, kGroupGradB>(a, a.groups, s, status);
  return launch<Tile128, T, kGroupGradB>(a, a.groups, s, status);
}

int32_t check(int64_t T, int64_t E, int64_t K, int64_t N, int32_t dtype, int32_t out_dtype) {
  if (T < 0 || K < 0 || N < 0 || E < 1 || E > kMaxGroups) return TSS_E_ARG;
  if (T > INT32_MAX || K > INT32_MAX || N > INT32_MAX) return TSS_E_ARG;
  if (dtype != TSS_F16 && dtype != TSS_BF16) return TSS_E_DTYPE;
  if (out_dtype != TSS_F32 && out_dtype != dtype) return TSS_E_DTYPE;
  if (K % 8 || N % 8) return TSS_E_ALIGN;
  if (T * K * 2 >= kTwoGiB || T * N * 2 >= kTwoGiB || K * N * 2 >= kTwoGiB) return TSS_E_ARG;
  return TSS_OK;
}

}  // namespace

extern "C" {

int32_t tss_gemm_grouped(int64_t T, int64_t E, int64_t K, int64_t N, int32_t dtype, const void *A, const void *B,
                         const int32_t *sizes, void *C, int32_t out_dtype, void *stream) {
  int32_t st = check(T, E, K, N, dtype, out_dtype);
  if (st != TSS_OK) return st;
  if (T == 0 || N == 0) return TSS_OK;
  if (!C || !sizes || (K > 0 && (!A || !B))) return TSS_E_ARG;
  if (misaligned(A, 16) || misaligned(B, 16) || misaligned(C, 16) || misaligned(sizes, 4)) return TSS_E_ALIGN;
  KernelArgs a{};
  a.A = A;
  a.B = B;
  a.C = C;
  a.M = int32_t(T);
  a.N = int32_t(N);
  a.K = a.lda = a.k_split = int32_t(K);
  a.splits = 1;
  a.out_dtype = out_dtype;
  a.batch_stride_b = K * N;
  a.sizes = sizes;
  a.groups = int32_t(E);
  a.rows_total = int32_t(T);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t err = dtype == TSS_F16 ? launch_rows<_Float16, kGroupForward>(a, s, &st)
                                          : launch_rows<__bf16, kGroupForward>(a, s, &st);
  if (st != TSS_OK) return st;
  return err == hipSuccess ? TSS_OK : TSS_E_HIP;
}

int32_t tss_gemm_grouped_backward(int64_t T, int64_t E, int64_t K, int64_t N, int32_t dtype, const void *dC,
                                  const void *A, const void *B, const int32_t *sizes, void *dA, void *dB,
                                  int32_t db_dtype, void *stream) {
  int32_t st = check(T, E, K, N, dtype, db_dtype);
  if (st != TSS_OK) return st;
  const bool want_a = dA && T > 0 && K > 0, want_b = dB && K > 0 && N > 0;
  if (!want_a && !want_b) return TSS_OK;
  if (!sizes || (T > 0 && N > 0 && (!dC || (want_a && !B) || (want_b && K > 0 && !A)))) return TSS_E_ARG;
  if (misaligned(dC, 16) || misaligned(A, 16) || misaligned(B, 16) || misaligned(dA, 16) || misaligned(dB, 16) ||
      misaligned(sizes, 4))
    return TSS_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t err = hipSuccess;
  KernelArgs a{};
  a.splits = 1;
  a.sizes = sizes;
  a.groups = int32_t(E);
  a.rows_total = int32_t(T);
  if (want_a) {
    a.A = dC;
    a.B = B;
    a.C = dA;
    a.M = int32_t(T);
    a.N = int32_t(K);
    a.K = a.lda = a.ldb = a.k_split = int32_t(N);
    a.out_dtype = dtype;
    a.batch_stride_b = K * N;
    err = dtype == TSS_F16 ? launch_rows<_Float16, kGroupGradA>(a, s, &st) : launch_rows<__bf16, kGroupGradA>(a, s, &st);
  }
  if (want_b && err == hipSuccess && st == TSS_OK) {
    a.A = A;
    a.B = dC;
    a.C = dB;
    a.M = a.lda = int32_t(K);
    a.N = int32_t(N);
    a.K = a.k_split = int32_t(T);
    a.out_dtype = db_dtype;
    a.batch_stride_c = K * N;
    err = dtype == TSS_F16 ? launch_grad_b<_Float16>(a, s, &st) : launch_grad_b<__bf16>(a, s, &st);
  }
  if (st != TSS_OK) return st;
  return err == hipSuccess ? TSS_OK : TSS_E_HIP;
}

}  // extern "C"

// Products grouped by expert in fp16 / bf16: tss_gemm_grouped and its
// gradients, on the GEMM kernel's group modes (gemm_kernel.h).
#include <atomic>

#include "gemm_kernel.h"

using namespace tss;

namespace {

constexpr int64_t kTwoGiB = int64_t(1) << 31;

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

using Tile256 = Geometry<256, 256, 64, 2, 8, 16>;
using Piece256 = Geometry<128, 256, 64, 3, 8, 16>;
using Piece128 = Geometry<128, 128, 64, 4, 8, 16>;
using Tile128 = Geometry<128, 128, 64, 2, 4, 16>;
using Tile64 = Geometry<64, 64, 64, 4, 4, 16>;

constexpr int most(int a, int b) { return a > b ? a : b; }

template <typename G, typename Half, typename Quarter, typename T, int GRP>
hipError_t launch(KernelArgs &a, hipStream_t s, int32_t *status) {
  constexpr bool ragged = GRP != kGroupGradB, pieces = !__is_same(G, Half);
  a.tiles_n = int32_t((int64_t(a.N) + G::BN - 1) / G::BN);
  const int64_t tiles_m = ragged ? max_group_tiles(a.M, a.groups, G::BM) : (int64_t(a.M) + G::BM - 1) / G::BM;
  a.tiles_m = int32_t(tiles_m);
  a.group_m = a.tiles_m < 4 ? a.tiles_m : 4;
  const int64_t tiles = tiles_m * a.tiles_n * (ragged ? 1 : a.groups);
  // (ragged: the most there can be)
  const int64_t whole = pieces ? tiles / kCUs * kCUs : tiles, rest = tiles - whole;
  const int64_t blocks = !pieces ? tiles : whole + (ragged ? kCUs * 4 / 3 : rest * tile_pieces(int(rest), false));
  if (blocks * G::THREADS > int64_t(UINT32_MAX)) {  // the launch's thread count is 32 bits
    *status = TSS_E_ARG;
    return hipSuccess;
  }
  // dynamic LDS above 64 KiB needs an attribute per kernel and device, set on the first launch there
  static std::atomic<uint64_t> attr_set{0};
  auto kernel = grouped_gemm_kernel<G, Half, Quarter, T, GRP>;
  constexpr int lds = most(G::lds_bytes(false), most(Half::lds_bytes(false), Quarter::lds_bytes(false)));
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(attr_set.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 163840);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit, std::memory_order_acq_rel);
  }
  hipLaunchKernelGGL(kernel, dim3(uint32_t(blocks)), dim3(G::THREADS), lds, s, a);
  return hipGetLastError();
}

// Few rows in an average group: the groups' weights are the cost, and small
// tiles put more of their loads in flight.  Forward, E = 32, K = N = 2048,
// 64 x 64 against 256 x 256 tiles: 16 rows a group 57 and 61 us, 64 rows 73
// and 63, 256 rows 181 and 99.
template <typename T, int GRP>
hipError_t launch_rows(KernelArgs &a, hipStream_t s, int32_t *status) {
  if (a.M / a.groups <= 32) return launch<Tile64, Tile64, Tile64, T, GRP>(a, s, status);
  return launch<Tile256, Piece256, Piece128, T, GRP>(a, s, status);
}

// With few rows to reduce over the writes are the cost.  E = 32, K = 4096,
// N = 2048, 2 rows a group: 128 x 128 tiles 165 us, 256 x 256 178; K = N =
// 2048, 64 rows a group 99 and 100, 256 rows 143 and 136.
template <typename T>
hipError_t launch_grad_b(KernelArgs &a, hipStream_t s, int32_t *status) {
  if (a.rows_total / a.groups <= 64) return launch<Tile128, Tile128, Tile128, T, kGroupGradB>(a, s, status);
  return launch<Tile256, Piece256, Piece128, T, kGroupGradB>(a, s, status);
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

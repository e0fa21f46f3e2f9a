// Host side of the 8-bit products: tss_gemm_fp8, tss_gemm_grouped_fp8.
#include <atomic>

#include "gemm_fp8_kernel.h"
#include "plans.h"
#include "splitk_reduce.h"

using namespace tss;

namespace {

constexpr int64_t kTwoGiB = int64_t(1) << 31;

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

using Tile256 = Fp8Geometry<256, 256, 2, 8, 2>;   // with its pieces: large products
using Piece256 = Fp8Geometry<128, 256, 3, 8, 2>;
using Piece128 = Fp8Geometry<128, 128, 3, 8, 2>;  // also groups of middling size
using Tile128 = Fp8Geometry<128, 128, 2, 4, 2>;   // fp32 sums; two workgroups a CU
using Tile64 = Fp8Geometry<64, 128, 3, 4, 1>;     // two workgroups a CU
constexpr int kRoundsLds = Tile256::LDS_BYTES > Piece256::LDS_BYTES ? Tile256::LDS_BYTES : Piece256::LDS_BYTES;

// Dynamic LDS above 64 KiB needs an attribute per kernel and device: set on the first launch there.
template <typename Kernel>
hipError_t launch_lds(Kernel kernel, std::atomic<uint64_t> &attr_set, const Fp8Args &a, int64_t blocks, int threads,
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

template <typename G, int KG, bool A_E5M2, bool B_ROWS, bool GROUPED, bool EXACT>
hipError_t launch_tile(const Fp8Args &a, int64_t blocks, hipStream_t s) {
  static std::atomic<uint64_t> attr_set{0};
  return launch_lds(gemm_fp8_tile_kernel<G, KG, A_E5M2, B_ROWS, GROUPED, EXACT>, attr_set, a, blocks, KG * G::THREADS,
                    KG * G::LDS_BYTES, s);
}

// tiles: the most there can be (grouped), or all there are.
template <bool A_E5M2, bool B_ROWS, bool GROUPED>
hipError_t launch_rounds(const Fp8Args &a, int64_t tiles, hipStream_t s) {
  static std::atomic<uint64_t> attr_set{0};
  const int64_t whole = tiles / kCUs * kCUs, rest = tiles - whole;
  // no pieces: the kernel without them is 2% faster (8192^3: 458 us against 467)
  if constexpr (!GROUPED)
    if (rest == 0 || tile_pieces(int(rest), false) == 1)
      return launch_tile<Tile256, 1, A_E5M2, B_ROWS, false, false>(a, tiles, s);
  const int64_t blocks = whole + (GROUPED ? kCUs * 4 / 3 : rest * tile_pieces(int(rest), false));
  return launch_lds(gemm_fp8_rounds_kernel<Tile256, Piece256, Piece128, A_E5M2, B_ROWS, GROUPED>, attr_set, a, blocks,
                    Tile256::THREADS, kRoundsLds, s);
}

// Waves of a workgroup of the kernel for few rows.
int rows_waves(int64_t K) {
  const int64_t nk = (K + 127) / 128, nw = (nk + kRowsUnroll - 1) / kRowsUnroll;
  return int(nw > 16 ? 16 : nw);
}

template <bool A_E5M2, bool B_ROWS, bool GROUPED, bool EXACT>
hipError_t launch_rows(const Fp8Args &a, int64_t blocks, hipStream_t s) {
  const int nw = rows_waves(a.K);
  hipLaunchKernelGGL((gemm_fp8_rows_kernel<A_E5M2, B_ROWS, GROUPED, EXACT>), dim3(uint32_t(blocks)), dim3(nw * 64), nw * 1024, s,
                     a);
  return hipGetLastError();
}

template <bool A_E5M2, bool B_ROWS, bool GROUPED>
hipError_t launch(Fp8Args &a, const ProductPlan &pl, bool exact, hipStream_t s, int32_t *status) {
  a.tiles_n = int32_t((a.N + pl.bn - 1) / pl.bn);
  const int64_t tiles_m = GROUPED ? max_group_tiles(a.M, a.groups, pl.bm) : (int64_t(a.M) + pl.bm - 1) / pl.bm;
  a.tiles_m = int32_t(tiles_m);
  const int64_t blocks = tiles_m * a.tiles_n * a.splits;
  // the launch's thread count is 32 bits (tiles: 512 threads at most, and a round's pieces)
  if ((pl.bn == 16 ? blocks * rows_waves(a.K) * 64 : (blocks + 2 * kCUs) * 512) > int64_t(UINT32_MAX)) {
    *status = TSS_E_ARG;
    return hipSuccess;
  }
  auto go = [&](auto exact) {
    constexpr bool X = decltype(exact)::value;
    if (pl.bn == 16) return launch_rows<A_E5M2, B_ROWS, GROUPED, X>(a, blocks, s);
    if constexpr (!X)
      if (pl.bm == 256) return launch_rounds<A_E5M2, B_ROWS, GROUPED>(a, blocks, s);
    if (pl.bm == 128) {
      if constexpr (X) return launch_tile<Tile128, 1, A_E5M2, B_ROWS, GROUPED, true>(a, blocks, s);
      else return launch_tile<Piece128, 1, A_E5M2, B_ROWS, GROUPED, false>(a, blocks, s);
    }
    return pl.sets == 2 ? launch_tile<Tile64, 2, A_E5M2, B_ROWS, GROUPED, X>(a, blocks, s)
                        : launch_tile<Tile64, 1, A_E5M2, B_ROWS, GROUPED, X>(a, blocks, s);
  };
  return exact ? go(std::true_type{}) : go(std::false_type{});
}

// The output's type without the flag, and whether the sums are fp32.
bool take_sums(int32_t &out_dtype) {
  const bool asked = out_dtype & TSS_F32_SUMS;
  out_dtype &= ~TSS_F32_SUMS;
  return asked || out_dtype == TSS_F32;
}

int32_t check_types(int32_t a_dtype, int32_t out_dtype) {
  if (a_dtype != TSS_E4M3 && a_dtype != TSS_E5M2) return TSS_E_DTYPE;
  if (out_dtype != TSS_F16 && out_dtype != TSS_BF16 && out_dtype != TSS_F32) return TSS_E_DTYPE;
  return TSS_OK;
}

int32_t check_sizes(int64_t M, int64_t N, int64_t K, int64_t n_multiple) {
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return TSS_E_ARG;
  if (K % 16 || N % n_multiple) return TSS_E_ALIGN;
  // the kernels' byte offsets into A, B and the scales are 32 bits (the scales of 2 GiB of values take 640 MiB at most:
  // K is at least 16), as are those of 256 rows of K
  if (M * K >= kTwoGiB || N * K >= kTwoGiB || K >= int64_t(1) << 22) return TSS_E_ARG;
  return TSS_OK;
}

}  // namespace

extern "C" {

int64_t tss_gemm_fp8_workspace_size(int64_t M, int64_t N, int64_t K) {
  const int32_t st = check_sizes(M, N, K, 1);
  if (st != TSS_OK) return st;
  if (M == 0 || N == 0 || K == 0) return 0;
  // the larger of what the two ways of summing take
  int32_t n, ks, most = 1;
  for (bool exact : {false, true}) {
    split_ranges(K, plan_product(M, N, K, exact).splits, &n, &ks);
    most = n > most ? n : most;
  }
  return most > 1 ? most * slice_elements(M, N) * 4 : 0;
}

int32_t tss_gemm_fp8(int64_t M, int64_t N, int64_t K, int32_t a_dtype, const void *A, const void *B, const float *sa,
                     const float *sb, int32_t b_block_rows, void *C, int32_t out_dtype, void *workspace,
                     int64_t workspace_bytes, void *stream) {
  const bool exact = take_sums(out_dtype);
  int32_t st = check_types(a_dtype, out_dtype);
  if (st == TSS_OK) st = check_sizes(M, N, K, 1);
  if (st != TSS_OK) return st;
  if (b_block_rows != 1 && b_block_rows != 128) return TSS_E_ARG;
  if (M == 0 || N == 0) return TSS_OK;
  if (!C || (K > 0 && (!A || !B || !sa || !sb))) return TSS_E_ARG;
  if (misaligned(A, 16) || misaligned(B, 16) || misaligned(C, 16) || misaligned(sa, 4) || misaligned(sb, 4))
    return TSS_E_ALIGN;
  const ProductPlan pl = K ? plan_product(M, N, K, exact) : ProductPlan{64, 128, 1};
  Fp8Args a{};
  a.A = static_cast<const uint8_t *>(A);
  a.B = static_cast<const uint8_t *>(B);
  a.sa = sa;
  a.sb = sb;
  a.M = int32_t(M);
  a.N = int32_t(N);
  a.K = int32_t(K);
  a.groups = 1;
  a.sb_cols = int32_t(b_block_rows == 1 ? N : (N + 127) / 128);
  a.splits = 1;
  a.k_split = a.K;
  if (K) split_ranges(K, pl.splits, &a.splits, &a.k_split);
  const bool split = a.splits > 1;
  if (split) {
    if (!workspace || workspace_bytes < a.splits * slice_elements(M, N) * 4) return TSS_E_ARG;
    if (misaligned(workspace, 16)) return TSS_E_ALIGN;
  }
  a.C = split ? workspace : C;
  a.out_dtype = split ? TSS_F32 : out_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t err;
  if (a_dtype == TSS_E5M2)
    err = b_block_rows == 1 ? launch<true, true, false>(a, pl, exact, s, &st) : launch<true, false, false>(a, pl, exact, s, &st);
  else
    err = b_block_rows == 1 ? launch<false, true, false>(a, pl, exact, s, &st) : launch<false, false, false>(a, pl, exact, s, &st);
  if (st != TSS_OK) return st;
  if (err == hipSuccess && split)
    err = launch_splitk_reduce(static_cast<const float *>(workspace), C, out_dtype, 1, M * N, a.splits, s,
                               slice_elements(M, N));
  return err == hipSuccess ? TSS_OK : TSS_E_HIP;
}

int32_t tss_gemm_grouped_fp8(int64_t T, int64_t E, int64_t K, int64_t N, int32_t a_dtype, const void *A,
                             const void *B, const float *sa, const float *sb, const int32_t *sizes, void *C,
                             int32_t out_dtype, void *stream) {
  const bool exact = take_sums(out_dtype);
  int32_t st = check_types(a_dtype, out_dtype);
  if (st == TSS_OK) st = check_sizes(T, N, K, 8);
  if (st != TSS_OK) return st;
  if (E < 1 || E > kMaxGroups) return TSS_E_ARG;
  if (T == 0 || N == 0) return TSS_OK;
  if (!C || !sizes || (K > 0 && (!A || !B || !sa || !sb))) return TSS_E_ARG;
  if (misaligned(A, 16) || misaligned(B, 16) || misaligned(C, 16) || misaligned(sa, 4) || misaligned(sb, 4) ||
      misaligned(sizes, 4))
    return TSS_E_ALIGN;
  Fp8Args a{};
  a.A = static_cast<const uint8_t *>(A);
  a.B = static_cast<const uint8_t *>(B);
  a.sa = sa;
  a.sb = sb;
  a.C = C;
  a.sizes = sizes;
  a.M = int32_t(T);
  a.N = int32_t(N);
  a.K = int32_t(K);
  a.groups = int32_t(E);
  a.sb_cols = int32_t((N + 127) / 128);
  a.splits = 1;
  a.k_split = a.K;
  a.out_dtype = out_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const ProductPlan pl = plan_grouped_fp8(T, N, K, E, exact);
  const hipError_t err = a_dtype == TSS_E5M2 ? launch<true, false, true>(a, pl, exact, s, &st)
                                             : launch<false, false, true>(a, pl, exact, s, &st);
  if (st != TSS_OK) return st;
  return err == hipSuccess ? TSS_OK : TSS_E_HIP;
}

}  // extern "C"

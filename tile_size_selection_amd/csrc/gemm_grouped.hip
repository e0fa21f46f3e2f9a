// Products grouped by expert in fp16 / bf16: tss_gemm_grouped and its
// gradients (grouped_kernel.h).
#include <atomic>

#include "grouped_kernel.h"
#include "plans.h"

using namespace tss;

namespace {

constexpr int64_t kTwoGiB = int64_t(1) << 31;

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

using Tile256 = Geometry<256, 256, 64, 2, 8, 16>;
using Piece256 = Geometry<128, 256, 64, 3, 8, 16>;
using Piece128 = Geometry<128, 128, 64, 4, 8, 16>;
using Tile128 = Geometry<128, 128, 64, 2, 4, 16>;
using Tile64 = Geometry<64, 64, 64, 4, 4, 16>;

// Few rows: the weights' bytes and the length of a workgroup's walk over K are
// the cost.  A workgroup takes 16 rows and 32 columns; its waves share K in
// chunks of 32, every chunk of the weights going from memory straight into
// MFMA fragments, and their sums are joined through LDS in the order of the
// waves.  A lane of a v_mfma_f32_16x16x32 fragment holds 8 of K.
//   Forward: B's rows run along N.  A lane loads two neighbouring columns of
//   each of its 8 k, the even one for the first MFMA tile and the odd one for
//   the second: a byte permutation of the lane's own words gives both their
//   fragments.  (Eight columns a lane and 128 a workgroup need a fourth of the
//   loads but leave too few workgroups: 1 row, 6 groups, K = 2048, N = 800:
//   8.7 us against 6.0.)
//   GradA: B's rows run along the reduction, and are loaded as fragments.
// 3 rows in 8 groups, K = N = 2048: 9.5 us (64 x 64 tiles: 11.4); 62 rows in 6,
// K = 5152, N = 328: 15.9 us (21.1).
constexpr int kFewTiles = 2, kFewCols = 16 * kFewTiles;
constexpr int kFewUnroll = 4;  // chunks whose loads a wave has in flight

template <typename T, int GRP>
__global__ __launch_bounds__(1024) void grouped_rows_kernel(GroupedArgs p) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = int(count_group_tiles<16>(p.sizes, p.groups, p.M, lane)) * p.tiles_n;
  if (int(blockIdx.x) >= n) return;
  const int id = xcd_run(blockIdx.x, n), tm = id / p.tiles_n, n0 = (id - tm * p.tiles_n) * kFewCols;
  const GroupTile t = find_group_tile<16>(p.sizes, p.groups, p.M, tm, lane);
  const bool none = t.group == p.groups;  // rows of no group: zeros
  const int rows = t.row_end - t.row0, K = none ? 0 : p.K, N = p.N;
  auto rsrc = [](const void *base, uint32_t range) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, int(range), 0x00020000);
  };
  const auto rsA = rsrc(static_cast<const T *>(p.A) + int64_t(t.row0) * p.lda, uint32_t(rows) * uint32_t(p.lda) * 2u);
  const T *B = static_cast<const T *>(p.B) + (none ? 0 : int64_t(t.group) * p.b_stride);
  const auto rsB = rsrc(B, uint32_t(p.b_stride) * 2u);  // one group's: below 2 GiB
  const int fr = lane % 16, kl = lane / 16 * 8;
  const uint32_t a_off = fr < rows ? (uint32_t(fr) * uint32_t(p.lda) + uint32_t(kl)) * 2u : kOOB;

  f32x4 acc[kFewTiles];
#pragma unroll
  for (int j = 0; j < kFewTiles; ++j) acc[j] = f32x4{0, 0, 0, 0};
  for (int k0 = wave * 32; k0 < K; k0 += nw * 32 * kFewUnroll) {
    i32x4 a[kFewUnroll];
    uint32_t b[kFewUnroll][8];  // forward: a word for each k; GradA: four for each tile
#pragma unroll
    for (int u = 0; u < kFewUnroll; ++u) {
      const int k = k0 + u * nw * 32 + kl;  // K is a multiple of 8: a lane's 8 are all in or all out
      a[u] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                           rsA, k < K && a_off != kOOB ? a_off + uint32_t(k - kl) * 2u : kOOB, 0, 0));
      if constexpr (GRP == kGroupForward) {
        const int col = n0 + fr * 2;  // N is even: both columns are in or out
        const uint32_t off = k < K && col < N ? (uint32_t(k) * uint32_t(N) + uint32_t(col)) * 2u : kOOB;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          b[u][j] = uint32_t(__builtin_amdgcn_raw_buffer_load_b32(
              rsB, off == kOOB ? kOOB : off + uint32_t(j) * uint32_t(N) * 2u, 0, 0));
      } else {
#pragma unroll
        for (int j = 0; j < kFewTiles; ++j) {
          const int row = n0 + j * 16 + fr;
          const i32x4 v = __builtin_bit_cast(
              i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         rsB, k < K && row < N ? (uint32_t(row) * uint32_t(p.ldb) + uint32_t(k)) * 2u : kOOB, 0, 0));
#pragma unroll
          for (int i = 0; i < 4; ++i) b[u][j * 4 + i] = uint32_t(v[i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kFewUnroll; ++u)
#pragma unroll
      for (int j = 0; j < kFewTiles; ++j) {
        i32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[i] = GRP == kGroupForward
                     ? int(__builtin_amdgcn_perm(b[u][2 * i + 1], b[u][2 * i], j ? 0x07060302u : 0x05040100u))
                     : int(b[u][j * 4 + i]);
        acc[j] = Mfma<T>::m16(__builtin_bit_cast(i16x8, f), __builtin_bit_cast(i16x8, a[u]), acc[j]);
      }
  }
  f32x4 *red = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
  for (int j = 0; j < kFewTiles; ++j) red[(wave * kFewTiles + j) * 64 + lane] = acc[j];
  __syncthreads();
  // wave w adds up tiles w, w + nw, ...
  for (int j = wave; j < kFewTiles; j += nw) {
    f32x4 s = red[j * 64 + lane];
    for (int w = 1; w < nw; ++w) {
      const f32x4 v = red[(w * kFewTiles + j) * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
    red[j * 64 + lane] = s;  // read by this wave only so far
  }
  __syncthreads();
  // 16 rows of 32 columns, 4 neighbours a lane
  auto put = [&](auto o) __attribute__((always_inline)) {
    using O = decltype(o);
    for (int x = threadIdx.x; x < 16 * kFewCols / 4; x += blockDim.x) {
      const int r = x / (kFewCols / 4), c = x % (kFewCols / 4) * 4;
      if (r >= rows || n0 + c >= N) continue;
      typename Vec4<O>::type v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // column c + i: its tile, and its place 0 .. 15 in the tile (lane group and register)
        const int j = GRP == kGroupForward ? (c + i) % kFewTiles : (c + i) / 16;
        const int at = GRP == kGroupForward ? (c + i) / kFewTiles : (c + i) % 16;
        v[i] = convert_out<O>(red[j * 64 + at / 4 * 16 + r][at % 4]);
      }
      *reinterpret_cast<typename Vec4<O>::type *>(static_cast<O *>(p.C) + int64_t(t.row0 + r) * N + n0 + c) = v;
    }
  };
  if (p.out_dtype == TSS_F32) put(float{});
  else if (p.out_dtype == TSS_F16) put(_Float16{});
  else put(__bf16{});
}

template <typename T, int GRP>
hipError_t launch_few(GroupedArgs &a, hipStream_t s, int32_t *status) {
  a.tiles_n = int32_t((int64_t(a.N) + kFewCols - 1) / kFewCols);
  const int64_t blocks = max_group_tiles(a.M, a.groups, 16) * a.tiles_n;
  int nw = (a.K + 32 * kFewUnroll - 1) / (32 * kFewUnroll);
  nw = nw > 8 ? 8 : nw < 1 ? 1 : nw;  // (16: 6.8 us where 8 take 6.0)
  if (blocks * nw * 64 > int64_t(UINT32_MAX)) {
    *status = TSS_E_ARG;
    return hipSuccess;
  }
  hipLaunchKernelGGL((grouped_rows_kernel<T, GRP>), dim3(uint32_t(blocks)), dim3(nw * 64), nw * kFewTiles * 1024, s, a);
  return hipGetLastError();
}

constexpr int most(int a, int b) { return a > b ? a : b; }

template <typename G, typename Half, typename Quarter, typename T, int GRP>
hipError_t launch(GroupedArgs &a, hipStream_t s, int32_t *status) {
  constexpr bool ragged = GRP != kGroupGradB, pieces = !__is_same(G, Half);
  a.tiles_n = int32_t((int64_t(a.N) + G::BN - 1) / G::BN);
  const int64_t tiles_m = ragged ? max_group_tiles(a.M, a.groups, G::BM) : (int64_t(a.M) + G::BM - 1) / G::BM;
  a.tiles_m = int32_t(tiles_m);
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

template <typename T, int GRP>
hipError_t launch_rows(GroupedArgs &a, hipStream_t s, int32_t *status) {
  switch (plan_grouped_rows(a.M, a.N, a.groups)) {
    case 16: return launch_few<T, GRP>(a, s, status);
    case 64: return launch<Tile64, Tile64, Tile64, T, GRP>(a, s, status);
    default: return launch<Tile256, Piece256, Piece128, T, GRP>(a, s, status);
  }
}

template <typename T>
hipError_t launch_grad_b(GroupedArgs &a, hipStream_t s, int32_t *status) {
  if (plan_grad_b(a.rows_total, a.groups) == 128) return launch<Tile128, Tile128, Tile128, T, kGroupGradB>(a, s, status);
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
  GroupedArgs a{};
  a.A = A;
  a.B = B;
  a.C = C;
  a.M = int32_t(T);
  a.N = int32_t(N);
  a.K = a.lda = int32_t(K);
  a.out_dtype = out_dtype;
  a.b_stride = K * N;
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
  GroupedArgs a{};
  a.sizes = sizes;
  a.groups = int32_t(E);
  a.rows_total = int32_t(T);
  if (want_a) {
    a.A = dC;
    a.B = B;
    a.C = dA;
    a.M = int32_t(T);
    a.N = int32_t(K);
    a.K = a.lda = a.ldb = int32_t(N);
    a.out_dtype = dtype;
    a.b_stride = K * N;
    err = dtype == TSS_F16 ? launch_rows<_Float16, kGroupGradA>(a, s, &st) : launch_rows<__bf16, kGroupGradA>(a, s, &st);
  }
  if (want_b && err == hipSuccess && st == TSS_OK) {
    a.A = A;
    a.B = dC;
    a.C = dB;
    a.M = a.lda = int32_t(K);
    a.N = int32_t(N);
    a.K = int32_t(T);
    a.out_dtype = db_dtype;
    a.c_stride = K * N;
    err = dtype == TSS_F16 ? launch_grad_b<_Float16>(a, s, &st) : launch_grad_b<__bf16>(a, s, &st);
  }
  if (st != TSS_OK) return st;
  return err == hipSuccess ? TSS_OK : TSS_E_HIP;
}

}  // extern "C"

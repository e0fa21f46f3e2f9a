// C = (A sa) (B sb)^T on 8-bit integers, A M x K and B N x K, both
// K-contiguous, with an fp32 scale for each row of A and each row of B:
//
//   C[m][n] = sa[m] sb[n] sum_k A[m][k] B[n][k]
//
// The sum is exact: v_mfma_i32_16x16x64_i8 adds into 32-bit integers, which
// hold 2^17 products of -128 .. 127.  The scales leave the loop over K, so a
// step of it is MFMAs, fragment reads and copies only, and ranges of K are
// joined without a rounding.  As in the 16-bit kernel the B fragment is the
// MFMA's row operand: a lane holds 4 consecutive columns of one row of C.
//
// 8192^3 to bf16: 415 to 458 us by box (2.4 to 2.65 POP/s; the library's product
// 526 to 556).  Power bounds it: the clock falls to 1.6 GHz, the MFMAs are busy
// 65% of the cycles, and operands of zeros take 346 us.  Rings of half steps (3
// to 5 deep) took 441 us where this took 415, 32 x 32 x 32 MFMAs 468, four waves
// of 128 x 128 441 (400), copies right behind the barrier 435 (420).
//
// Three kernels: gemm_int8_tile_kernel stages BM x 128 and BN x 128 tiles of the
// operands through LDS; gemm_int8_rounds_kernel does so with the last round's
// tiles in pieces; gemm_int8_rows_kernel, for few rows, streams B from memory
// straight into registers.
#pragma once
#include "gemm_fp8_kernel.h"

namespace tss {

struct Int8Args {
  const int8_t *A;    // [M][K]
  const int8_t *B;    // [N][K]
  const float *sa;    // [M]
  const float *sb;    // [N]
  void *C;            // [M][N]; split K: int32 [splits][M][N], the slices slice_elements(M, N) apart
  int32_t M, N, K;
  int32_t tiles_m, tiles_n, splits;
  int32_t k_split;    // K of a range, a multiple of 128
  int32_t out_dtype;  // or kInt8Sums
};

constexpr int kInt8Sums = 0x1000;  // an out_dtype: the sums as they are (split K)

template <int BM_, int BN_, int ST_, int NW_, int WM_>
struct Int8Geometry {
  static constexpr int BM = BM_, BN = BN_, ST = ST_, NW = NW_, MF = 16, BK = 128;
  static constexpr int THREADS = NW * 64, WM = WM_, WN = NW / WM;
  static constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 16, TN = WTN / 16;
  static constexpr int CA = BK / 16;  // 16-byte chunks of a row
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int A_LOADS = A_BYTES / 1024 / NW, B_LOADS = B_BYTES / 1024 / NW, LPW = A_LOADS + B_LOADS;
  static constexpr int LDS_BYTES = ST * STAGE_BYTES;
  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "whole wave loads");
  static_assert(TM % 2 == 0 && TN >= 1, "a step runs in two halves of the rows");
  static_assert(8 * NW % 16 == 0, "the swizzle is the same for every load of a lane");
  static_assert(LDS_BYTES <= 163840 && (ST - 1) * LPW < 64, "LDS, vmcnt");
  // chunk c of row r lives at c ^ swz(r): 16 consecutive rows read at one
  // logical chunk land in 16 distinct 16-byte bank groups
  static __device__ __forceinline__ int swz(int r) { return (r / 2) % CA; }
};

struct Int8Fragment {
  i32x4 lo, hi;  // 16 bytes of each half of a block of 128 of K
};

__device__ __forceinline__ i32x4 mfma_int8(const Int8Fragment &b, const Int8Fragment &a, i32x4 c) {
  c = __builtin_amdgcn_mfma_i32_16x16x64_i8(b.lo, a.lo, c, 0, 0, 0);
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(b.hi, a.hi, c, 0, 0, 0);
}

// A sum with its scales: one rounding of the sum to fp32 and one for each
// scale, whatever follows (the empty statement keeps the compiler from making
// the last product and a conversion to fp16 one instruction, which rounds
// once: the same product would then depend on the way it ran).
__device__ __forceinline__ float scaled_sum(int sum, float sa, float sb) {
  float v = float(sum) * sa * sb;
  asm("" : "+v"(v));
  return v;
}

struct Int8Tile {
  int row0, n0, split;
};

// Tile `id` of the product, bm x bn.
template <int BM, int BN>
__device__ __forceinline__ Int8Tile int8_tile_at(const Int8Args &p, int id) {
  const int mn = p.tiles_m * p.tiles_n, split = id / mn, in = id - split * mn;
  constexpr int GM = 4;  // tile rows that share an XCD's run of tiles
  const int span = GM * p.tiles_n, first = in / span * GM, gm = min(p.tiles_m - first, GM), r = in % span;
  return {(first + r % gm) * BM, r / gm * BN, split};
}

// One tile's product.  A step of K (128) runs in two halves around its
// barrier, as in the 8-bit floating-point kernel:
//   1. rows 0 .. TM/2-1; as a row ends, its A fragment is replaced by that of
//      the row TM/2 below;
//   -- the next step's tile has landed, and this one's slot is read --
//   2. rows TM/2 .., column by column; as a column ends, its B fragment is
//      replaced by the next step's, and after the last column the A fragments
//      are; the slot is refilled meanwhile.
template <typename G>
__device__ __forceinline__ void int8_tile_product(const Int8Args &p, const Int8Tile &t, char *smem) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / G::WN, wc = wave % G::WN;
  const int row0 = t.row0, n0 = t.n0, rows = min(G::BM, p.M - row0), cols = min(G::BN, p.N - n0);
  const int kbeg = t.split * p.k_split, K = max(0, min(p.k_split, p.K - kbeg)), steps = (K + 127) / 128;

  const i32x4 rsA = buffer_rsrc(p.A + int64_t(row0) * p.K + kbeg, K ? uint32_t(rows - 1) * uint32_t(p.K) + uint32_t(K) : 0u);
  const i32x4 rsB = buffer_rsrc(p.B + int64_t(n0) * p.K + kbeg, K ? uint32_t(cols - 1) * uint32_t(p.K) + uint32_t(K) : 0u);

  // Copy plan: wave load j of an operand covers LDS chunks (j*NW + wave)*64 +
  // lane, so a lane's loads are 8*NW rows apart and at one place in their
  // rows.  Rows past the operand's last lie past its range, and read as zero;
  // so does K past its end (kOOB).
  const int cr = (wave * 64 + lane) / G::CA, cc = ((lane % G::CA) ^ G::swz(cr)) * 16;
  const uint32_t off0 = uint32_t(cr) * uint32_t(p.K) + uint32_t(cc);
  const uint32_t jstep = uint32_t(8 * G::NW) * uint32_t(p.K);
  auto issue = [&](int kt, int slot, int j) __attribute__((always_inline)) {
    char *st = smem + slot * G::STAGE_BYTES;
    const bool a = j < G::A_LOADS;
    const int jj = a ? j : j - G::A_LOADS, k0 = kt * 128;
    const lds_void *dst = (lds_void *)(st + (a ? 0 : G::A_BYTES) + (jj * G::NW + wave) * 1024);
    copy_to_lds16(a ? rsA : rsB, (k0 + cc < K ? off0 : kOOB) + uint32_t(jj) * jstep, uint32_t(k0), dst);
  };

  const int fr = lane % 16;
  const uint32_t f0 = uint32_t(fr * 128 + ((lane / 16) ^ G::swz(fr)) * 16);
  const uint32_t f1 = uint32_t(fr * 128 + ((4 + lane / 16) ^ G::swz(fr)) * 16);
  auto frag = [&](const char *base) __attribute__((always_inline)) -> Int8Fragment {
    return {*(const __attribute__((address_space(3))) i32x4 *)(base + f0),
            *(const __attribute__((address_space(3))) i32x4 *)(base + f1)};
  };

  constexpr int TM = G::TM, TN = G::TN, R = TM / 2, ST = G::ST;
  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  asm volatile("s_nop 4" ::: "memory");  // descriptors written by v_readfirstlane, before the first copy
#pragma unroll
  for (int s = 0; s < ST; ++s)
#pragma unroll
    for (int j = 0; j < G::LPW; ++j) issue(s, s, j);
  wait_vmcnt_lgkm0<(ST - 1) * G::LPW>();
  block_barrier();
  Int8Fragment fa[R], fb[TN];
  {
    const char *sta = smem + wr * G::WTM * 128, *stb = smem + G::A_BYTES + wc * G::WTN * 128;
#pragma unroll
    for (int i = 0; i < R; ++i) fa[i] = frag(sta + i * 16 * 128);
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[j] = frag(stb + j * 16 * 128);
  }
  int slot = 0;
  for (int kt = 0; kt < steps; ++kt) {
    const int next = slot + 1 == ST ? 0 : slot + 1;
    const char *sta = smem + slot * G::STAGE_BYTES + wr * G::WTM * 128;
    const char *stn = smem + next * G::STAGE_BYTES;
    const char *stna = stn + wr * G::WTM * 128, *stnb = stn + G::A_BYTES + wc * G::WTN * 128;
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma_int8(fb[j], fa[i], acc[i][j]);
      fa[i] = frag(sta + (R + i) * 16 * 128);
      __builtin_amdgcn_sched_barrier(0);
    }
    // tile kt + 1 has landed, and tile kt's slot is read
    wait_vmcnt_lgkm0<(ST - 2) * G::LPW>();
    block_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
      for (int i = 0; i < R; ++i) acc[R + i][j] = mfma_int8(fb[j], fa[i], acc[R + i][j]);
      fb[j] = frag(stnb + j * 16 * 128);
      if (j == TN - 1) {
#pragma unroll
        for (int i = 0; i < R; ++i) fa[i] = frag(stna + i * 16 * 128);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = j * G::LPW / TN; c < (j + 1) * G::LPW / TN; ++c) issue(kt + ST, slot, c);
      __builtin_amdgcn_sched_barrier(0);
    }
    slot = next;
  }
  wait_vmcnt_lgkm0<0>();  // copies past the end still land in the LDS that the epilogue reuses
  f32x4 out[TM][TN];
  const bool sums = p.out_dtype == kInt8Sums;
  float sb[TN][4];
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = n0 + wc * G::WTN + j * 16 + lane / 16 * 4 + e;
      sb[j][e] = !sums && c < p.N ? p.sb[c] : 0.0f;
    }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = row0 + wr * G::WTM + i * 16 + fr;
    const float sa = !sums && row < p.M ? p.sa[row] : 0.0f;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int s = acc[i][j][e];
        out[i][j][e] = sums ? __builtin_bit_cast(float, s) : scaled_sum(s, sa, sb[j][e]);
      }
  }
  auto store = [&](auto o) __attribute__((always_inline)) {
    using O = decltype(o);
    O *C = static_cast<O *>(p.C) + t.split * slice_elements(p.M, p.N);
    if (p.N % 8 == 0) store_tile<G, O>(out, C, smem, row0, n0, wave, wr, wc, lane, p.M, p.N);
    else store_tile_unaligned<G, O>(out, C, smem, row0, n0, wave, wr, wc, lane, p.M, p.N);
  };
  if (p.out_dtype == TSS_F16) store(_Float16{});
  else if (p.out_dtype == TSS_BF16) store(__bf16{});
  else store(float{});  // fp32, and 32-bit sums as they are
}

template <typename G>
__global__ __launch_bounds__(G::THREADS) void gemm_int8_tile_kernel(Int8Args p) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int8_tile_product<G>(p, int8_tile_at<G::BM, G::BN>(p, xcd_run(blockIdx.x, gridDim.x)), smem);
}

// Large products: one workgroup fills a CU, and the last round's tiles are cut
// into pieces (tile_pieces).
template <typename G, typename Half, typename Quarter>
__global__ __launch_bounds__(G::THREADS) void gemm_int8_rounds_kernel(Int8Args p) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  static_assert(G::THREADS == Half::THREADS && G::THREADS == Quarter::THREADS && Half::BM * 2 == G::BM &&
                    Quarter::BM * 2 == G::BM && Half::BN == G::BN && Quarter::BN * 2 == G::BN, "pieces of a tile");
  const int bid = blockIdx.x, n = p.tiles_m * p.tiles_n;
  const int whole = n / kCUs * kCUs, rest = n - whole, pieces = tile_pieces(rest, false);
  if (bid < whole) {
    int8_tile_product<G>(p, int8_tile_at<G::BM, G::BN>(p, xcd_run(bid, whole)), smem);
    return;
  }
  const int piece = xcd_run(bid - whole, rest * pieces), part = piece % pieces;
  Int8Tile t = int8_tile_at<G::BM, G::BN>(p, whole + piece / pieces);
  t.row0 += (pieces == 2 ? part : part / 2) * Half::BM;
  if (pieces == 4) t.n0 += part % 2 * Quarter::BN;
  if (t.row0 >= p.M || t.n0 >= p.N) return;
  if (pieces == 2) int8_tile_product<Half>(p, t, smem);
  else int8_tile_product<Quarter>(p, t, smem);
}

// Few rows: B's bytes are the cost, and each is used by one wave only, so it
// goes from memory straight into MFMA fragments.  A workgroup takes 16 rows
// and NC groups of 16 columns; its waves share K, block by block of 128, and
// their sums are joined through LDS (whole numbers: any order).  A (read by
// every workgroup) comes from L2; two column groups halve that.  U: blocks of K
// whose loads a wave has in flight.  4 x 8192 x 8192, weights in no cache: 16.5
// us, 4.1 TB/s of B (one group, U = 4: 18.6), 16 rows 19.2 (23.8); where one
// group gives no CU a second workgroup, 16 x 4096 x 4096, 7.8 and with two 9.4.
template <typename O>
__device__ __forceinline__ void put_int8_row(const Int8Args &p, int row, int col, const float (&v)[4]) {
  O *to = static_cast<O *>(p.C) + int64_t(row) * p.N + col;
  if (p.N % 4 == 0) {
    typename Vec4<O>::type w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = convert_out<O>(v[e]);
    *reinterpret_cast<typename Vec4<O>::type *>(to) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < p.N) to[e] = convert_out<O>(v[e]);
  }
}

template <int NC, int U>
__global__ __launch_bounds__(1024) void gemm_int8_rows_kernel(Int8Args p) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int id = xcd_run(blockIdx.x, gridDim.x);
  const int tm = id % p.tiles_m, row0 = tm * 16, n0 = id / p.tiles_m * 16 * NC;  // the rows of a column share its B
  const int rows = min(16, p.M - row0), cols = min(16 * NC, p.N - n0), K = p.K, nk = (K + 127) / 128;
  auto rsrc = [](const void *base, uint32_t range) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, int(range), 0x00020000);
  };
  const auto rsA = rsrc(p.A + int64_t(row0) * K, uint32_t(rows) * uint32_t(K));
  const auto rsB = rsrc(p.B + int64_t(n0) * K, uint32_t(cols) * uint32_t(K));
  const int fr = lane % 16, ch = lane / 16 * 16;
  const uint32_t a_off = fr < rows ? uint32_t(fr) * uint32_t(K) + uint32_t(ch) : kOOB;
  uint32_t b_off[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) b_off[c] = c * 16 + fr < cols ? uint32_t(c * 16 + fr) * uint32_t(K) + uint32_t(ch) : kOOB;
  // a lane's 16 bytes at k (zeros from K on); `ch` is its place within 64
  auto load = [&](auto rs, uint32_t off, int k) __attribute__((always_inline)) -> i32x4 {
    const uint32_t o = k + ch < K && off != kOOB ? off + uint32_t(k) : kOOB;
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0));
  };
  i32x4 acc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = i32x4{0, 0, 0, 0};
  for (int kb = wave; kb < nk; kb += nw * U) {
    Int8Fragment b[U][NC], a[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (kb + u * nw) * 128;
#pragma unroll
      for (int c = 0; c < NC; ++c) b[u][c] = {load(rsB, b_off[c], k), load(rsB, b_off[c], k + 64)};
      a[u] = {load(rsA, a_off, k), load(rsA, a_off, k + 64)};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] = mfma_int8(b[u][c], a[u], acc[c]);
  }
  i32x4 *red = reinterpret_cast<i32x4 *>(smem);  // [wave][column group][lane]
#pragma unroll
  for (int c = 0; c < NC; ++c) red[(wave * NC + c) * 64 + lane] = acc[c];
  __syncthreads();
  if (wave >= NC) return;  // one wave joins one column group
  i32x4 s = red[wave * 64 + lane];
  for (int w = 1; w < nw; ++w) {
    const i32x4 v = red[(w * NC + wave) * 64 + lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += v[e];
  }
  const int row = row0 + fr, col = n0 + wave * 16 + lane / 16 * 4;
  if (row >= p.M || col >= p.N) return;
  const float sa = p.sa[row];
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int x = s[e];
    v[e] = col + e < p.N ? scaled_sum(x, sa, p.sb[col + e]) : 0.0f;
  }
  if (p.out_dtype == TSS_F32) put_int8_row<float>(p, row, col, v);
  else if (p.out_dtype == TSS_F16) put_int8_row<_Float16>(p, row, col, v);
  else put_int8_row<__bf16>(p, row, col, v);
}

// C = scaled sum of the ranges' partial sums.  V: 4 consecutive columns (N % 4 == 0), or 1.
template <typename O, int V>
__global__ __launch_bounds__(256) void int8_join_kernel(const int32_t *P, O *C, const float *sa, const float *sb, int64_t mn,
                                                        int32_t N, int64_t slice, int32_t splits) {
  typedef int VI __attribute__((ext_vector_type(V)));
  typedef O VO __attribute__((ext_vector_type(V)));
  for (int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x; u * V < mn; u += int64_t(gridDim.x) * 256) {
    const int64_t i = u * V, row = i / N;
    const int col = int(i - row * N);
    VI sum = *reinterpret_cast<const VI *>(P + i);
    for (int s = 1; s < splits; ++s) sum += *reinterpret_cast<const VI *>(P + s * slice + i);
    VO o;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int x = sum[e];
      o[e] = convert_out<O>(scaled_sum(x, sa[row], sb[col + e]));
    }
    *reinterpret_cast<VO *>(C + i) = o;
  }
}

}  // namespace tss

// C = (A sa) (B sb)^T on 8-bit operands, A M x K and B N x K, both
// K-contiguous, with fp32 scales for each 128 of K (of a row of A; of a row
// or of 128 rows of B):
//
//   C[m][n] = sum over blocks j of 128:  sa[j][m] sb[j][n] sum_{k in j} A[m][k] B[n][k]
//
// One v_mfma_f32_16x16x128_f8f6f4 sums exactly one block of 128 of a 16 x 16
// tile, so a block's sum leaves the matrix core in 4 registers, and 4 fp32
// FMAs scale it into the accumulators: 16 vector cycles beside the MFMA's 32.
// (The MFMA's own block scales are powers of two over 32 elements; these are
// any fp32 over 128, hence the unscaled form.)  As in the fp16 kernel the B
// fragment is the MFMA's row operand: a lane holds 4 consecutive columns of
// one row of C.
//
// The 8-bit MFMA adds its products in groups with fewer bits than fp32: a
// product 2^-14 of the largest beside it is lost (measured), which leaves the
// result 1.7e-5 of its norm off, far below the rounding of a 16-bit output
// (2^-9) but not of an fp32 one (plain fp32 sums: 8e-7), nor where large
// products cancel.  With EXACT, taken for fp32 outputs and where the caller
// asks for fp32 sums, the fragments are widened to fp16 (exactly: e4m3 and e5m2
// are subsets of it) and multiplied by v_mfma_f32_16x16x32_f16, which adds in
// fp32, at half the rate.
//
// Three kernels: gemm_fp8_tile_kernel stages BM x 128 and BN x 128 tiles of the
// operands through LDS; gemm_fp8_rounds_kernel does so with the last round's
// tiles in pieces; gemm_fp8_rows_kernel, for few rows, streams B from memory
// straight into registers.
#pragma once
#include "grouped_kernel.h"

namespace tss {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Args {
  const uint8_t *A;   // [M][K]
  const uint8_t *B;   // [groups][N][K]
  const float *sa;    // [ceil(K / 128)][M]
  const float *sb;    // [groups][ceil(K / 128)][sb_cols]
  void *C;            // [M][N]; split K: fp32 [splits][M][N], the slices slice_elements(M, N) apart
  const int32_t *sizes;  // grouped: rows of each group
  int32_t M, N, K, groups;
  int32_t sb_cols;    // N, or ceil(N / 128)
  int32_t tiles_m, tiles_n, splits;
  int32_t k_split;    // K of a range, a multiple of 128
  int32_t out_dtype;
};

// A fragment: the 32 bytes that a lane holds of a block of 128 of K, as they
// are or widened to fp16.
template <bool EXACT>
struct Fragment;

template <>
struct Fragment<false> {
  i32x8 v;
  template <bool E5M2>
  __device__ __forceinline__ void set(i32x8 x) { v = x; }
};

template <>
struct Fragment<true> {
  f16x8 v[4];
  template <bool E5M2>
  __device__ __forceinline__ void set(i32x8 x) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      i32x4 w;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int s = x[q * 2 + h / 2];
        if constexpr (E5M2)  // e5m2 is the upper byte of an fp16
          w[h] = int(__builtin_amdgcn_perm(0, uint32_t(s), h % 2 ? 0x030c020cu : 0x010c000cu));
        else if (h % 2)
          w[h] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s, 1.0f, true));
        else
          w[h] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s, 1.0f, false));
      }
      v[q] = __builtin_bit_cast(f16x8, w);
    }
  }
};

// A block's sum of a 16 x 16 tile; A_E5M2 is the type of `a` (b: e4m3).
template <bool A_E5M2>
__device__ __forceinline__ f32x4 mfma_block(const Fragment<false> &b, const Fragment<false> &a) {
  // formats: 0 = e4m3, 1 = e5m2; zero scale operands select the unscaled instruction
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, f32x4{0, 0, 0, 0}, 0, A_E5M2 ? 1 : 0, 0, 0, 0, 0);
}
template <bool A_E5M2>
__device__ __forceinline__ f32x4 mfma_block(const Fragment<true> &b, const Fragment<true> &a) {
  f32x4 c = {0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[q], a.v[q], c, 0, 0, 0);
  return c;
}

// 4 bytes per lane from memory to LDS: lane i's word lands at dst + 4 i (as copy_to_lds16).
__device__ __forceinline__ void copy_to_lds4(i32x4 rs, uint32_t voff, uint32_t soff, const lds_void *dst) {
  const uint32_t m0 = uint32_t(reinterpret_cast<uintptr_t>(dst));
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(voff), "s"(rs), "s"(soff),
               "s"(m0)
               : "memory", "m0");
}

template <int BM_, int BN_, int ST_, int NW_, int WM_>
struct Fp8Geometry {
  static constexpr int BM = BM_, BN = BN_, ST = ST_, NW = NW_, MF = 16, BK = 128;
  static constexpr int THREADS = NW * 64, WM = WM_, WN = NW / WM;
  static constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 16, TN = WTN / 16;
  static constexpr int CA = BK / 16;  // 16-byte chunks of a row
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
  static constexpr int S_LOADS = (BM + BN + 64 * NW - 1) / (64 * NW);  // 256-byte wave loads of scales
  static constexpr int S_BYTES = S_LOADS * NW * 256;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + S_BYTES;
  static constexpr int A_LOADS = A_BYTES / 1024 / NW, B_LOADS = B_BYTES / 1024 / NW;
  static constexpr int LPW = A_LOADS + B_LOADS + S_LOADS;
  static constexpr int LDS_BYTES = ST * STAGE_BYTES;
  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0,
                "whole wave loads");
  static_assert(TM % 4 == 0 && TM >= 4 && WTN % 16 == 0 && 128 % WTN == 0, "a wave's columns lie in one block of 128");
  static_assert(8 * NW % 16 == 0, "the swizzle is the same for every load of a lane");
  static_assert(LDS_BYTES <= 163840 && (ST - 2) * LPW < 64, "LDS, vmcnt");
  // chunk c of row r lives at c ^ swz(r): 16 consecutive rows read at one
  // logical chunk land in 16 distinct 16-byte bank groups
  static __device__ __forceinline__ int swz(int r) { return (r / 2) % CA; }
};

// The tile of a workgroup.
struct Fp8Tile {
  int group, row0, row_end, n0, split;
  bool any;
};

// Tile `id` of the product, bm x bn.
template <int BM, int BN, bool GROUPED>
__device__ __forceinline__ Fp8Tile fp8_tile_at(const Fp8Args &p, int id, int lane) {
  if constexpr (GROUPED) {
    const int tm = id / p.tiles_n, tn = id - tm * p.tiles_n;
    const GroupTile g = find_group_tile<BM>(p.sizes, p.groups, p.M, tm, lane);
    return {g.group, g.row0, g.row_end, tn * BN, 0, true};
  } else {
    const int mn = p.tiles_m * p.tiles_n, split = id / mn, in = id - split * mn;
    constexpr int GM = 4;  // tile rows that share an XCD's run of tiles (as in the fp16 kernel)
    const int span = GM * p.tiles_n, first = in / span * GM, gm = min(p.tiles_m - first, GM), r = in % span;
    const int row0 = (first + r % gm) * BM;
    return {0, row0, min(row0 + BM, p.M), r / gm * BN, split, true};
  }
}

// Every workgroup one tile; in XCD order only the tiles that there are take
// part (grouped: the launch's spare workgroups end here).
template <int BM, int BN, bool GROUPED>
__device__ __forceinline__ Fp8Tile fp8_tile(const Fp8Args &p, int lane) {
  int n = gridDim.x;
  if constexpr (GROUPED) {
    n = int(count_group_tiles<BM>(p.sizes, p.groups, p.M, lane)) * p.tiles_n;
    if (int(blockIdx.x) >= n) return {0, 0, 0, 0, 0, false};
  }
  return fp8_tile_at<BM, BN, GROUPED>(p, xcd_run(blockIdx.x, n), lane);
}

// Rows of C that do not start on 16-byte borders (N not a multiple of 8; C itself does):
// staged through LDS as in store_tile, but each row at its place within 16
// bytes of memory, so that whole 16-byte pieces of memory are written from
// aligned pieces of LDS; the elements of the pieces at a row's ends are
// written one by one (their other elements are another wave's).  Measured at
// 8192 x 8191 x 512, bf16: 4-byte words 118 us, this 80 to 90 (N 8192: 66).
template <typename G, typename O, typename Acc>
__device__ __forceinline__ void store_tile_unaligned(const Acc (&acc)[G::TM][G::TN], O *C, char *smem, int m0, int n0,
                                                     int wave, int wr, int wc, int lane, int M, int N) {
  using E = LdsEpilogue<G, O>;
  static_assert(E::fits, "the staging area holds a row of MFMA tiles of every wave");
  typedef __attribute__((address_space(3))) O lds_o;
  constexpr int SIZE = int(sizeof(O)), PER = 16 / SIZE, CPR = G::WTN / PER;
  char *area = smem + wave * E::WAVE_BYTES;
  const int col0 = n0 + wc * G::WTN, row0 = m0 + wr * G::WTM;
  const int cols = min(G::WTN, N - col0);
  // bytes that the wave's part of a row starts past a 16-byte border
  auto shift = [&](int row) __attribute__((always_inline)) {
    return int(((uint32_t(row) * uint32_t(N) + uint32_t(col0)) * uint32_t(SIZE)) & 15u);
  };
  block_barrier();  // every wave is done with the last stage's fragments
  if (cols <= 0) return;
#pragma unroll
  for (int i = 0; i < G::TM; ++i) {
    {
      const int r = lane % 16;
      char *to = area + r * E::PITCH + shift(row0 + i * 16 + r) + lane / 16 * 4 * SIZE;
#pragma unroll
      for (int j = 0; j < G::TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) *(lds_o *)(to + (j * 16 + e) * SIZE) = convert_out<O>(acc[i][j][e]);
    }
#pragma unroll
    for (int c = 0; c < 16 * CPR / 64; ++c) {
      const int r = (c * 64 + lane) / CPR, row = row0 + i * 16 + r, a = shift(row);
      const int q = (c * 64 + lane) % CPR + (a ? 1 : 0);  // the piece of memory, from the one that the row starts in
      if (row < M && (q + 1) * 16 <= a + cols * SIZE)
        *(i16x8 *)((char *)(C + int64_t(row) * N + col0) - a + q * 16) = *(const lds_i16x8 *)(area + r * E::PITCH + q * 16);
    }
#pragma unroll
    for (int c = 0; c < 16 * PER / 64; ++c) {
      const int r = (c * 64 + lane) / PER, x = (c * 64 + lane) % PER, row = row0 + i * 16 + r, a = shift(row);
      const int end = a + cols * SIZE, last = end & ~15;  // the piece that the row ends in
      O *to = C + int64_t(row) * N + col0;
      const char *from = area + r * E::PITCH;
      const int head = a + x * SIZE, tail = last + x * SIZE;
      if (row < M && (a || end < 16) && head < 16 && head < end) to[x] = *(const lds_o *)(from + head);
      if (row < M && last > 0 && tail < end) to[(tail - a) / SIZE] = *(const lds_o *)(from + tail);
    }
  }
}

// One tile's product.  A step of K (128) of a wave's TM x TN MFMA tiles runs
// in two halves, so that neither the step's first fragments nor its barrier
// leave the matrix cores idle:
//   1. rows 0 .. TM/2-1, one after the other; as a row ends, its A fragment is
//      replaced by that of the row TM/2 below;
//   -- the next step's tile has landed, and this one's slot is read --
//   2. rows TM/2 .., column by column; as a column ends, its B fragment is
//      replaced by the next step's, and after the last column the A fragments
//      are; the slot is refilled meanwhile.
// The sums of one group of MFMAs are scaled while the next group's run.
// Measured at 8192^3 (e4m3, 128 x 128 scales of B, bf16 out) on one box: all of
// a step's fragments read and copies spread over it behind the barrier 482 us,
// copies in its first half 449-459, this 439; 440 to 475 (2.3 to 2.5 PFLOP/s)
// over boxes and inputs.  Of 459 us,
// leaving out the copies took 62, the scaling 47, the fragment reads 118; the
// MFMAs alone took 271.
//
// KG > 1: as many sets of G::NW waves share the tile, each taking a range of K
// with a ring of its own; their sums are added at the end, in order.  It fills
// a CU where there are too few tiles for two workgroups each.
template <typename G, int KG, bool A_E5M2, bool B_ROWS, bool GROUPED, bool EXACT>
__device__ __forceinline__ void fp8_tile_product(const Fp8Args &p, const Fp8Tile &t, char *smem0) {
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int set = KG > 1 ? wave_all / G::NW : 0, wave = KG > 1 ? wave_all % G::NW : wave_all;
  const int wr = wave / G::WN, wc = wave % G::WN;
  char *smem = smem0 + set * G::LDS_BYTES;
  const int rows = t.row_end - t.row0, cols = min(G::BN, p.N - t.n0);
  int kbeg = t.split * p.k_split;
  // rows of no group: no product, zeros are written
  int K = GROUPED && t.group == p.groups ? 0 : max(0, min(p.k_split, p.K - kbeg));
  const int steps = (K + KG * 128 - 1) / (KG * 128);  // of every set; past a set's end they add zeros
  if constexpr (KG > 1) {
    kbeg += set * steps * 128;
    K = max(0, min(K - set * steps * 128, steps * 128));
  }
  const int nk = (K + 127) / 128;
  const int kb0 = kbeg / 128, kblocks = (p.K + 127) / 128;
  const int group = GROUPED && t.group < p.groups ? t.group : 0;

  const i32x4 rsA = buffer_rsrc(p.A + int64_t(t.row0) * p.K + kbeg, K ? uint32_t(rows - 1) * uint32_t(p.K) + uint32_t(K) : 0u);
  const i32x4 rsB = buffer_rsrc(p.B + (int64_t(group) * p.N + t.n0) * p.K + kbeg,
                                K ? uint32_t(cols - 1) * uint32_t(p.K) + uint32_t(K) : 0u);
  const i32x4 rsSA = buffer_rsrc(p.sa + int64_t(kb0) * p.M + t.row0, nk ? (uint32_t(nk - 1) * uint32_t(p.M) + uint32_t(rows)) * 4u : 0u);
  const i32x4 rsSB = buffer_rsrc(p.sb + (int64_t(group) * kblocks + kb0) * p.sb_cols, uint32_t(nk) * uint32_t(p.sb_cols) * 4u);

  // Copy plan: wave load j of an operand covers LDS chunks (j*NW + wave)*64 +
  // lane, so a lane's loads are 8*NW rows apart and at one place in their
  // rows (the swizzle repeats every 16 rows).  Rows past the operand's last
  // lie past its range, and read as zero; so does K past its end (kOOB).
  const int cr = (wave * 64 + lane) / G::CA, cc = ((lane % G::CA) ^ G::swz(cr)) * 16;
  const uint32_t off0 = uint32_t(cr) * uint32_t(p.K) + uint32_t(cc);
  const uint32_t jstep = uint32_t(8 * G::NW) * uint32_t(p.K);
  // scales: LDS words 0 .. BM-1 hold sa, ordered so that a lane's TM rows
  // (16 apart) are neighbours; BM .. BM+BN-1 hold sb per column
  // (words past them fill up the last wave's load)
  uint32_t soff[G::S_LOADS];
#pragma unroll
  for (int j = 0; j < G::S_LOADS; ++j) {
    const int w0 = (j * G::NW + wave) * 64;
    if (w0 < G::BM) {
      const int w = w0 + lane, in = w % G::WTM;
      const int r = w - in + (in % G::TM) * 16 + in / G::TM;
      soff[j] = r < rows ? uint32_t(r) * 4u : kOOB;
    } else {
      const int c = w0 - G::BM + lane;
      soff[j] = c < cols ? uint32_t(B_ROWS ? t.n0 + c : (t.n0 + c) / 128) * 4u : kOOB;
    }
  }
  // copy j of K tile kt (past the last one: zeros) into `slot`
  auto issue = [&](int kt, int slot, int j) __attribute__((always_inline)) {
    char *st = smem + slot * G::STAGE_BYTES;
    if (j < G::A_LOADS + G::B_LOADS) {
      const bool a = j < G::A_LOADS;
      const int jj = a ? j : j - G::A_LOADS, k0 = kt * 128;
      const lds_void *dst = (lds_void *)(st + (a ? 0 : G::A_BYTES) + (jj * G::NW + wave) * 1024);
      copy_to_lds16(a ? rsA : rsB, (k0 + cc < K ? off0 : kOOB) + uint32_t(jj) * jstep, uint32_t(k0), dst);
    } else {
      const int js = j - G::A_LOADS - G::B_LOADS, w0 = (js * G::NW + wave) * 64;
      const lds_void *dst = (lds_void *)(st + G::A_BYTES + G::B_BYTES + w0 * 4);
      const bool sa = w0 < G::BM;
      const uint32_t row = uint32_t(sa ? p.M : p.sb_cols) * 4u;
      copy_to_lds4(sa ? rsSA : rsSB, kt < nk ? soff[js] : kOOB, kt < nk ? uint32_t(kt) * row : 0u, dst);
    }
  };

  // fragments: lane's row lane % 16, chunks lane / 16 and 4 + lane / 16 (any
  // order of K serves, being the same for both operands)
  const int fr = lane % 16;
  uint32_t f0 = uint32_t(fr * 128 + ((lane / 16) ^ G::swz(fr)) * 16);
  uint32_t f1 = uint32_t(fr * 128 + ((4 + lane / 16) ^ G::swz(fr)) * 16);
  auto frag = [&](const char *base) __attribute__((always_inline)) -> i32x8 {
    const i32x4 lo = *(const __attribute__((address_space(3))) i32x4 *)(base + f0);
    const i32x4 hi = *(const __attribute__((address_space(3))) i32x4 *)(base + f1);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  f32x4 acc[G::TM][G::TN];
#pragma unroll
  for (int i = 0; i < G::TM; ++i)
#pragma unroll
    for (int j = 0; j < G::TN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  asm volatile("s_nop 4" ::: "memory");  // descriptors written by v_readfirstlane, before the first copy

  constexpr int TM = G::TM, TN = G::TN, R = TM / 2, ST = G::ST;
  float sav[TM], sbv[TN][4];
  Fragment<EXACT> fa[R], fb[TN];
  auto read_scales = [&](const char *st) __attribute__((always_inline)) {
    const float *ss = reinterpret_cast<const float *>(st + G::A_BYTES + G::B_BYTES);
#pragma unroll
    for (int i = 0; i < TM; i += 4) {
      const f32x4 v = *(const __attribute__((address_space(3))) f32x4 *)(ss + wr * G::WTM + fr * TM + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) sav[i + e] = v[e];
    }
    if constexpr (B_ROWS) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const f32x4 v = *(const __attribute__((address_space(3))) f32x4 *)(ss + G::BM + wc * G::WTN + j * 16 + lane / 16 * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) sbv[j][e] = v[e];
      }
    } else {
      const float v = *(const __attribute__((address_space(3))) float *)(ss + G::BM + wc * G::WTN);
#pragma unroll
      for (int i = 0; i < TM; ++i) sav[i] *= v;
    }
  };
  constexpr int NP = TN > R ? TN : R;
  f32x4 part[2][NP];
  auto scale_tile = [&](f32x4 v, int i, int j) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[i][j][e] = __builtin_fmaf(B_ROWS ? v[e] * sbv[j][e] : v[e], sav[i], acc[i][j][e]);
  };
#pragma unroll
  for (int s = 0; s < ST; ++s)
#pragma unroll
    for (int j = 0; j < G::LPW; ++j) issue(s, s, j);
  wait_vmcnt_lgkm0<(ST - 1) * G::LPW>();
  block_barrier();
  int slot = 0;
  {
    const char *sta = smem + wr * G::WTM * 128, *stb = smem + G::A_BYTES + wc * G::WTN * 128;
#pragma unroll
    for (int i = 0; i < R; ++i) fa[i].template set<A_E5M2>(frag(sta + i * 16 * 128));
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[j].template set<false>(frag(stb + j * 16 * 128));
    read_scales(smem);
  }
  // A wave whose rows are all past the tile's end (the last tile of a group,
  // say) only copies: its SIMD's other wave then has the matrix core alone.
  // (A loop of its own: with the test inside the loop below the registers
  // spill.)
  if (wr * G::WTM >= rows) {
    for (int kt = 0; kt < steps; ++kt) {
      wait_vmcnt_lgkm0<(ST - 2) * G::LPW>();
      block_barrier();
#pragma unroll
      for (int c = 0; c < G::LPW; ++c) issue(kt + ST, slot, c);
      slot = slot + 1 == ST ? 0 : slot + 1;
    }
  } else {
    for (int kt = 0; kt < steps; ++kt) {
      const int next = slot + 1 == ST ? 0 : slot + 1;
      const char *sta = smem + slot * G::STAGE_BYTES + wr * G::WTM * 128;
      const char *stn = smem + next * G::STAGE_BYTES;
      const char *stna = stn + wr * G::WTM * 128, *stnb = stn + G::A_BYTES + wc * G::WTN * 128;
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j) part[i % 2][j] = mfma_block<A_E5M2>(fb[j], fa[i]);
        fa[i].template set<A_E5M2>(frag(sta + (R + i) * 16 * 128));
        if (i > 0) {
#pragma unroll
          for (int j = 0; j < TN; ++j) scale_tile(part[(i - 1) % 2][j], i - 1, j);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // tile kt + 1 has landed, and tile kt's slot is read
      wait_vmcnt_lgkm0<(ST - 2) * G::LPW>();
      block_barrier();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int g = R + j;  // the group's number in the step
#pragma unroll
        for (int i = 0; i < R; ++i) part[g % 2][i] = mfma_block<A_E5M2>(fb[j], fa[i]);
        fb[j].template set<false>(frag(stnb + j * 16 * 128));
        if (j == TN - 1) {
#pragma unroll
          for (int i = 0; i < R; ++i) fa[i].template set<A_E5M2>(frag(stna + i * 16 * 128));
        }
        if (j == 0) {
#pragma unroll
          for (int jj = 0; jj < TN; ++jj) scale_tile(part[(R - 1) % 2][jj], R - 1, jj);
        } else {
#pragma unroll
          for (int i = 0; i < R; ++i) scale_tile(part[(g - 1) % 2][i], R + i, j - 1);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = j * G::LPW / TN; c < (j + 1) * G::LPW / TN; ++c) issue(kt + ST, slot, c);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) scale_tile(part[(R + TN - 1) % 2][i], R + i, TN - 1);
      read_scales(stn);
      slot = next;
    }
  }
  wait_vmcnt_lgkm0<0>();  // copies past the end still land in the LDS that the epilogue reuses
  if constexpr (KG > 1) {
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    lds_f32x4 *sums = (lds_f32x4 *)smem0;  // [set - 1][MFMA tile][wave][lane]
    static_assert((KG - 1) * G::TM * G::TN * G::NW * 1024 <= KG * G::LDS_BYTES, "the sets' sums fit");
    block_barrier();
    if (set > 0) {
#pragma unroll
      for (int i = 0; i < G::TM; ++i)
#pragma unroll
        for (int j = 0; j < G::TN; ++j)
          sums[(((set - 1) * G::TM * G::TN + i * G::TN + j) * G::NW + wave) * 64 + lane] = acc[i][j];
      wait_vmcnt_lgkm0<0>();
    }
    block_barrier();
    if (set > 0) {
      block_barrier();  // the one that the store begins with
      return;
    }
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int i = 0; i < G::TM; ++i)
#pragma unroll
        for (int j = 0; j < G::TN; ++j) {
          const f32x4 v = sums[((g * G::TM * G::TN + i * G::TN + j) * G::NW + wave) * 64 + lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += v[e];
        }
    wait_vmcnt_lgkm0<0>();
  }

  auto store = [&](auto o) __attribute__((always_inline)) {
    using O = decltype(o);
    O *C = static_cast<O *>(p.C) + t.split * slice_elements(p.M, p.N);
    if (GROUPED || p.N % 8 == 0)
      store_tile<G, O>(acc, C, smem, t.row0, t.n0, wave, wr, wc, lane, t.row_end, p.N);
    else
      store_tile_unaligned<G, O>(acc, C, smem, t.row0, t.n0, wave, wr, wc, lane, t.row_end, p.N);
  };
  if (p.out_dtype == TSS_F32) store(float{});  // also the partial sums of a split K
  else if (p.out_dtype == TSS_F16) store(_Float16{});
  else store(__bf16{});
}

template <typename G, int KG, bool A_E5M2, bool B_ROWS, bool GROUPED, bool EXACT>
__global__ __launch_bounds__(G::THREADS *KG) void gemm_fp8_tile_kernel(Fp8Args p) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const Fp8Tile t = fp8_tile<G::BM, G::BN, GROUPED>(p, threadIdx.x & 63);
  if (t.any) fp8_tile_product<G, KG, A_E5M2, B_ROWS, GROUPED, EXACT>(p, t, smem);
}

// Large products: one workgroup fills a CU, and the last round's tiles are cut
// into pieces as in grouped_gemm_kernel.
template <typename G, typename Half, typename Quarter, bool A_E5M2, bool B_ROWS, bool GROUPED>
__global__ __launch_bounds__(G::THREADS) void gemm_fp8_rounds_kernel(Fp8Args p) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  static_assert(G::THREADS == Half::THREADS && G::THREADS == Quarter::THREADS && Half::BM * 2 == G::BM &&
                    Quarter::BM * 2 == G::BM && Half::BN == G::BN && Quarter::BN * 2 == G::BN, "pieces of a tile");
  const int lane = threadIdx.x & 63, bid = blockIdx.x;
  const int n = (GROUPED ? int(count_group_tiles<G::BM>(p.sizes, p.groups, p.M, lane)) : p.tiles_m) * p.tiles_n;
  const int whole = n / kCUs * kCUs, rest = n - whole, pieces = tile_pieces(rest, GROUPED);
  if (bid < whole || pieces == 1) {
    if (bid >= n) return;
    const int id = bid < whole ? xcd_run(bid, whole) : whole + xcd_run(bid - whole, rest);
    const Fp8Tile t = fp8_tile_at<G::BM, G::BN, GROUPED>(p, id, lane);
    // the last tile of a group, when half empty: one piece holds it
    if (GROUPED && t.row_end - t.row0 <= Half::BM)
      fp8_tile_product<Half, 1, A_E5M2, B_ROWS, GROUPED, false>(p, t, smem);
    else
      fp8_tile_product<G, 1, A_E5M2, B_ROWS, GROUPED, false>(p, t, smem);
    return;
  }
  if (bid >= whole + rest * pieces) return;
  const int piece = xcd_run(bid - whole, rest * pieces), id = whole + piece / pieces, part = piece % pieces;
  Fp8Tile t = fp8_tile_at<G::BM, G::BN, GROUPED>(p, id, lane);
  t.row0 += (pieces == 2 ? part : part / 2) * Half::BM;
  t.row_end = min(t.row_end, t.row0 + Half::BM);
  if (pieces == 4) t.n0 += part % 2 * Quarter::BN;
  if (t.row0 >= t.row_end || t.n0 >= p.N) return;
  if (pieces == 2) fp8_tile_product<Half, 1, A_E5M2, B_ROWS, GROUPED, false>(p, t, smem);
  else fp8_tile_product<Quarter, 1, A_E5M2, B_ROWS, GROUPED, false>(p, t, smem);
}

// Few rows: B's bytes are the cost, and each is used by one wave only, so it
// goes from memory straight into MFMA fragments.  A workgroup takes 16 rows
// and 16 columns; its waves share K, block by block of 128, and their sums
// are joined through LDS in the order of the waves: one launch, where the
// tiles above need a second for a split K.  A (read by every workgroup) comes
// from L2.  4 x 8192 x 8192: 15.0 us, 4.5 TB/s of B; 64 x 2048 x 2048: 7.2 us.
constexpr int kRowsUnroll = 4;  // blocks of K whose loads a wave has in flight

template <bool A_E5M2, bool B_ROWS, bool GROUPED, bool EXACT>
__global__ __launch_bounds__(1024) void gemm_fp8_rows_kernel(Fp8Args p) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Fp8Tile t = fp8_tile<16, 16, GROUPED>(p, lane);
  if (!t.any) return;
  const int rows = t.row_end - t.row0, cols = min(16, p.N - t.n0);
  const bool none = GROUPED && t.group == p.groups;  // rows of no group: zeros
  const int K = p.K, kblocks = (K + 127) / 128, nk = none ? 0 : kblocks, group = none ? 0 : t.group;
  auto rsrc = [](const void *base, uint32_t range) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, int(range), 0x00020000);
  };
  const auto rsA = rsrc(p.A + int64_t(t.row0) * K, uint32_t(rows) * uint32_t(K));
  const auto rsB = rsrc(p.B + (int64_t(group) * p.N + t.n0) * K, uint32_t(cols) * uint32_t(K));
  const auto rsSA = rsrc(p.sa + t.row0, (uint32_t(kblocks - 1) * uint32_t(p.M) + uint32_t(rows)) * 4u);
  const auto rsSB = rsrc(p.sb + int64_t(group) * kblocks * p.sb_cols, uint32_t(kblocks) * uint32_t(p.sb_cols) * 4u);
  const int fr = lane % 16, ch = lane / 16 * 16;
  const uint32_t a_off = fr < rows ? uint32_t(fr) * uint32_t(K) + uint32_t(ch) : kOOB;
  const uint32_t b_off = fr < cols ? uint32_t(fr) * uint32_t(K) + uint32_t(ch) : kOOB;
  // a lane's 16 bytes at k (zeros from K on); `ch` is its place within 64
  auto load = [&](auto rs, uint32_t off, int k) __attribute__((always_inline)) -> i32x4 {
    const uint32_t o = k + ch < K && off != kOOB ? off + uint32_t(k) : kOOB;
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0));
  };
  auto loadf = [&](auto rs, uint32_t off) __attribute__((always_inline)) -> float {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0));
  };
  f32x4 acc = {0, 0, 0, 0};
  for (int kb = wave; kb < nk; kb += nw * kRowsUnroll) {
    i32x4 b[kRowsUnroll][2], a[kRowsUnroll][2];
    float sa[kRowsUnroll], sb[kRowsUnroll][4];
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
      const int kk = kb + u * nw, k = kk * 128;
      const bool in = kk < nk;
#pragma unroll
      for (int h = 0; h < 2; ++h) b[u][h] = load(rsB, b_off, k + 64 * h);
#pragma unroll
      for (int h = 0; h < 2; ++h) a[u][h] = load(rsA, a_off, k + 64 * h);
      sa[u] = loadf(rsSA, in && fr < rows ? (uint32_t(kk) * uint32_t(p.M) + uint32_t(fr)) * 4u : kOOB);
      if constexpr (B_ROWS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = lane / 16 * 4 + e;
          sb[u][e] = loadf(rsSB, in && c < cols ? (uint32_t(kk) * uint32_t(p.sb_cols) + uint32_t(t.n0 + c)) * 4u : kOOB);
        }
      } else {
        sb[u][0] = loadf(rsSB, in ? (uint32_t(kk) * uint32_t(p.sb_cols) + uint32_t(t.n0 / 128)) * 4u : kOOB);
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
      Fragment<EXACT> fa, fb;
      fb.template set<false>(__builtin_shufflevector(b[u][0], b[u][1], 0, 1, 2, 3, 4, 5, 6, 7));
      fa.template set<A_E5M2>(__builtin_shufflevector(a[u][0], a[u][1], 0, 1, 2, 3, 4, 5, 6, 7));
      const f32x4 part = mfma_block<A_E5M2>(fb, fa);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(part[e] * sb[u][B_ROWS ? e : 0], sa[u], acc[e]);
    }
  }
  f32x4 *red = reinterpret_cast<f32x4 *>(smem);
  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  f32x4 s = red[lane];
  for (int w = 1; w < nw; ++w) {
    const f32x4 v = red[w * 64 + lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += v[e];
  }
  const int row = t.row0 + fr, col = t.n0 + lane / 16 * 4;
  if (row >= t.row_end || col >= p.N) return;
  auto put = [&](auto o) __attribute__((always_inline)) {
    using O = decltype(o);
    typename Vec4<O>::type v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = convert_out<O>(s[e]);
    O *to = static_cast<O *>(p.C) + int64_t(row) * p.N + col;
    if (p.N % 4 == 0) {
      *reinterpret_cast<typename Vec4<O>::type *>(to) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.N) to[e] = v[e];
    }
  };
  if (EXACT && p.out_dtype == TSS_F32) put(float{});
  else if (p.out_dtype == TSS_F16) put(_Float16{});
  else put(__bf16{});
}

}  // namespace tss

// Products grouped by expert in fp16 / bf16, on the GEMM's geometry, copies,
// fragments and K loop (gemm_kernel.h says why each is as it is): rows sorted
// by group, the groups' sizes in device memory (groups.h).
//   kGroupForward: C[rows of e] = A[rows of e] B[e]; as the GEMM, the rows of
//     a tile ending with their group;
//   kGroupGradA:   dA[rows of e] = dC[rows of e] B[e]^T; the B operand's rows
//     are contiguous along the reduction, so it is copied and read like A;
//   kGroupGradB:   dB[e] = A[rows of e]^T dC[rows of e]; the reduction runs
//     over the group's rows, so the A operand is copied and read like the
//     GEMM's B, with the transpose read.
// Bound by the matrix cores where groups are large: 16384 rows, 8 groups, K =
// 4096, N = 2048, bf16: forward 239 us (1.15 PFLOP/s; the GEMM's 8192^3: 1.50,
// the library's 1.39), dA 248, dB 244 (fp32, 268 MB written).
// A body of its own: with these modes in the GEMM's, the convolution's kernel
// came out 7% slower.
#pragma once
#include "gemm_kernel.h"
#include "groups.h"
#include "plans.h"

namespace tss {

enum GroupMode { kGroupForward, kGroupGradA, kGroupGradB };

struct GroupedArgs {
  const void *A, *B;  // the operands of the mode's product, above
  void *C;
  const int32_t *sizes;  // rows of each group, device memory
  int32_t M, N, K;  // forward T x N x K; GradA T x K x N; GradB K x N with T rows to reduce over
  int32_t tiles_m, tiles_n;
  int32_t groups, rows_total;  // rows_total: T
  int32_t lda, ldb;            // elements between A's rows; GradA: between B's
  int32_t out_dtype;
  int64_t b_stride, c_stride;  // elements from group to group: B (forward, GradA), C (GradB)
};

// Geometry::swz_b and frag_n_rows for rows of CHUNKS 16-byte chunks, or WIDTH
// elements: the transposed A operand's are BM wide.
template <int CHUNKS>
__device__ __forceinline__ int swz_rows(int k) {
  const int q = CHUNKS >= 16 ? 4 * (k % 4) : 4 * ((k / 2) % 2);
  return q ^ (2 * ((k / 8) % 2));
}
template <typename G, int WIDTH>
__device__ __forceinline__ uint32_t frag_rows(int col0, int lane) {
  const int g = lane / 16, s = lane % 16;
  const int krow = G::MF == 32 ? (g / 2) * 8 + s / 4 : g * 8 + s / 4;
  const int n = col0 + (G::MF == 32 ? (g % 2) * 16 + 4 * (s % 4) : 4 * (s % 4));
  return uint32_t(krow * WIDTH * 2 + ((n / 8) ^ swz_rows<WIDTH / 8>(krow)) * 16 + (n % 8) * 2);
}

// The product of one tile: rows m0 .. M - 1 (at most BM) and columns from n0,
// over K elements (K == 0 for rows of no group: zeros); GradB: the K rows from
// kbeg of group `group`.
template <typename G, typename T, int GRP>
__device__ __forceinline__ void grouped_tile_product(const GroupedArgs &p, char *smem, int m0, int n0, int M, int K,
                                                     int group, int kbeg) {
  constexpr bool AT = GRP == kGroupGradB;       // A operand K-outer, read with the transpose read
  constexpr bool BK_ROWS = GRP == kGroupGradA;  // B operand K-contiguous, copied and read like A
  using Acc = typename AccType<G::MF>::type;
  constexpr int MF = G::MF;
  constexpr int S = G::ST;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / G::WN, wc = wave % G::WN;
  const int lda = p.lda;

  const int N = p.N;
  // the operands' rows and columns of this tile, over K; rows past the last one read as zero
  const T *Ab = static_cast<const T *>(p.A) + (AT ? int64_t(kbeg) * lda + m0 : int64_t(m0) * lda);
  const int a_rows = min(G::BM, M - m0);
  const i32x4 rsA4 = buffer_rsrc(Ab, a_rows <= 0 || K <= 0 ? 0u
                                     : AT ? (uint32_t(K) * uint32_t(lda) - uint32_t(m0)) * 2u
                                          : (uint32_t(a_rows - 1) * uint32_t(lda) + uint32_t(K)) * 2u);
  i32x4 rsB4;
  if constexpr (BK_ROWS) {
    // B's rows are the result's columns
    const T *Bb = static_cast<const T *>(p.B) + int64_t(group) * p.b_stride + int64_t(n0) * p.ldb;
    const int b_rows = min(G::BN, N - n0);
    rsB4 = buffer_rsrc(Bb, K > 0 ? (uint32_t(b_rows - 1) * uint32_t(p.ldb) + uint32_t(K)) * 2u : 0u);
  } else {
    const T *Bb = static_cast<const T *>(p.B) + (AT ? int64_t(kbeg) * N : int64_t(group) * p.b_stride) + n0;
    // elements [n0, K*N); with K == 0 the range is empty (otherwise n0 < N <= K*N)
    rsB4 = buffer_rsrc(Bb, K > 0 ? (uint32_t(K) * uint32_t(N) - uint32_t(n0)) * 2u : 0u);
  }

  // -- A copy plan: wave load j of a stage covers LDS chunks (j*NW+wave)*64 + lane
  uint32_t a_off[G::A_LOADS];
  int a_kc[G::A_LOADS];  // first K element of the lane's chunk within the stage
#pragma unroll
  for (int j = 0; j < G::A_LOADS; ++j) {
    int pchunk = (j * G::NW + wave) * 64 + lane;
    if constexpr (AT) {
      // chunk (k, lc): elements m0 + 8lc .. +7 of row k
      constexpr int CM = G::BM / 8;
      const int k = pchunk / CM, lc = pchunk % CM ^ swz_rows<CM>(k);
      const bool ok = m0 + lc * 8 < M;
      a_off[j] = ok ? uint32_t(k) * uint32_t(lda) * 2u + uint32_t(lc) * 16u : kOOB;
      a_kc[j] = ok ? k : (1 << 30);
    } else {
      int r = pchunk / G::CA, pc = pchunk % G::CA;
      int lc = pc ^ G::swz_a(r);
      a_off[j] = uint32_t(r) * uint32_t(lda) * 2u + uint32_t(lc) * 16u;
      a_kc[j] = lc * 8;
    }
  }
  // -- B copy plan: chunk (k, lc) of the stage holds columns 8lc .. 8lc+7 of
  // row k, or (GradA) chunk lc of row r, as A's
  uint32_t b_off[G::B_LOADS];
  int b_k[G::B_LOADS];
#pragma unroll
  for (int j = 0; j < G::B_LOADS; ++j) {
    const int pchunk = (j * G::NW + wave) * 64 + lane;
    if constexpr (BK_ROWS) {
      const int r = pchunk / G::CA, lc = pchunk % G::CA ^ G::swz_a(r);
      const bool ok = n0 + r < N;
      b_off[j] = ok ? uint32_t(r) * uint32_t(p.ldb) * 2u + uint32_t(lc) * 16u : kOOB;
      b_k[j] = ok ? lc * 8 : (1 << 30);
    } else {
      const int k = pchunk / G::CB, lc = pchunk % G::CB ^ G::swz_b(k);
      const bool ok = n0 + lc * 8 < N;
      b_off[j] = ok ? uint32_t(k) * uint32_t(N) * 2u + uint32_t(lc) * 16u : kOOB;
      b_k[j] = ok ? k : (1 << 30);
    }
  }

  // bytes that A and B advance by for each step of K
  const uint32_t a_step = AT ? uint32_t(lda) * 2u : 2u;
  const uint32_t b_step = BK_ROWS ? 2u : uint32_t(N) * 2u;
  const int nk = (K + G::BK - 1) / G::BK;
  const int nfull = K / G::BK;  // K tiles that lie inside K

  // LDS slots.  The plain ring: stage s holds A at s*STAGE_BYTES and B right
  // after it.  The A3 ring (GEMM, 2 stages): three A slots, then two B slots.
  constexpr bool A3 = G::A3;
  auto a_slot = [&](int s) __attribute__((always_inline)) -> char * {
    return smem + (A3 ? s * G::A_BYTES : s * G::STAGE_BYTES);
  };
  auto b_slot = [&](int s) __attribute__((always_inline)) -> char * {
    return smem + (A3 ? 3 * G::A_BYTES + s * G::B_BYTES : s * G::STAGE_BYTES + G::A_BYTES);
  };
  // Copy j (0 .. LPW-1) of full K tile kt, A copies (j < A_LOADS) into A slot
  // sa, B copies into B slot sb.  A (and the GEMM's B) advance through the
  // scalar offset: the per-lane offsets stay fixed over the K loop.
  auto issue_one = [&](int kt, int sa, int sb, int j) __attribute__((always_inline)) {
    const int k0 = kt * G::BK;
    if (j < G::A_LOADS) {
      lds_void *dst = (lds_void *)(a_slot(sa) + (j * G::NW + wave) * 1024);
      copy_to_lds16(rsA4, a_off[j], uint32_t(k0) * a_step, dst);
    } else {
      const int jb = j - G::A_LOADS;
      lds_void *dst = (lds_void *)(b_slot(sb) + (jb * G::NW + wave) * 1024);
      copy_to_lds16(rsB4, b_off[jb], uint32_t(k0) * b_step, dst);
    }
  };
  // Copy j of any K tile ckt: a full tile as above; the ragged last tile
  // masks the chunks at or past K per lane; a tile past the end reads zeros.
  auto copy = [&](int ckt, int sa, int sb, int j) __attribute__((always_inline)) {
    if (ckt < nfull) {
      issue_one(ckt, sa, sb, j);
    } else {
      const int k0 = ckt * G::BK;
      if (j < G::A_LOADS) {
        lds_void *dst = (lds_void *)(a_slot(sa) + (j * G::NW + wave) * 1024);
        copy_to_lds16(rsA4, k0 + a_kc[j] < K ? a_off[j] + uint32_t(k0) * a_step : kOOB, 0u, dst);
      } else {
        const int jb = j - G::A_LOADS;
        lds_void *dst = (lds_void *)(b_slot(sb) + (jb * G::NW + wave) * 1024);
        copy_to_lds16(rsB4, k0 + b_k[jb] < K ? b_off[jb] + uint32_t(k0) * b_step : kOOB, 0u, dst);
      }
    }
  };

  // -- per-lane fragment addresses (bytes within an A or B slot)
  // A: one address per MFMA K step (MFMA tile i adds i*MF rows).
  // B, else: one address per MFMA tile (K step q adds q*FK rows).
  // B, GradA (K-contiguous rows): read like A, one address per K step.
  constexpr int NFA = AT ? G::TM : G::KSUB;
  uint32_t fa[NFA];
#pragma unroll
  for (int q = 0; q < NFA; ++q)
    fa[q] = AT ? frag_rows<G, G::BM>(wr * G::WTM + q * MF, lane) : G::frag_k_rows(wr * G::WTM, lane, q);
  constexpr int NFB = BK_ROWS ? G::KSUB : G::TN;
  uint32_t fb[NFB];
  if constexpr (BK_ROWS) {
#pragma unroll
    for (int q = 0; q < G::KSUB; ++q) fb[q] = G::frag_k_rows(wc * G::WTN, lane, q);
  } else {
#pragma unroll
    for (int nt = 0; nt < G::TN; ++nt) fb[nt] = G::frag_n_rows(wc * G::WTN + nt * MF, lane);
  }

  Acc acc[G::TM][G::TN];
#pragma unroll
  for (int i = 0; i < G::TM; ++i)
#pragma unroll
    for (int j = 0; j < G::TN; ++j) acc[i][j] = Acc{};

  int kt = 0;
  int ca = 0, cb = 0;  // A and B slots of the tile being computed

  // The copies read buffer descriptors that may have just been written by a
  // vector instruction (v_readfirstlane); five wait states cover that hazard
  // once, before the first copy.
  asm volatile("s_nop 4" ::: "memory");
  {
    // The K loop.  Changes to a plain ring (barrier, burst of copies, fragment
    // reads, MFMAs), all against stalls of the matrix pipe:
    //  * fragment reads cross the barrier: the last MFMA step of tile kt runs
    //    on fragments already in registers while the first step's fragments
    //    of tile kt+1 are read, and the barrier sits inside that last step,
    //    after its first MFMA rows, so the pipe has work while the waves meet;
    //  * the refill copies are spread over MFMA rows (a copy occupies the
    //    CU's load path for about as long as four MFMAs; issued as a burst,
    //    they block the in-order issue of every wave in front of its MFMAs).
    //    The plain ring refills the stage freed at the barrier during the
    //    last step.  The A3 ring (a 2-stage GEMM ring with a third A buffer)
    //    refills A during the first step, into the A slot freed a tile
    //    earlier, and B during the last step, so the copies of a tile are
    //    spread over all of it;
    //  * every tile refills: refills past the last K tile copy zeros into
    //    slots nobody reads again, so the waits are the same for every tile
    //    and one loop body serves the whole K loop.
    // A fragments are single-buffered (slot i is refilled right after the
    // last MFMA that reads it); B fragments are double-buffered, every MFMA
    // row of a step reads all of them.  The steps alternate B buffers and
    // every tile starts on buffer 0.
    i16x8 fa_[G::TM], fb_[2][G::TN];
    // 8 consecutive k of one column of rows of `width` elements: two transpose reads, 4 rows apart
    auto read_tr = [](const char *p, int width) __attribute__((always_inline)) -> i16x8 {
      i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p));
      i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p + 4 * width * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto read_a = [&](const char *sta, int q, int i) __attribute__((always_inline)) {
      if constexpr (AT) fa_[i] = read_tr(sta + fa[i] + q * G::FK * G::BM * 2, G::BM);
      else fa_[i] = *(const lds_i16x8 *)(sta + fa[q] + i * MF * G::BK * 2);
    };
    auto read_b = [&](const char *stb, int q, int pb, int j) __attribute__((always_inline)) {
      if constexpr (BK_ROWS) fb_[pb][j] = *(const lds_i16x8 *)(stb + fb[q] + j * MF * G::BK * 2);
      else fb_[pb][j] = read_tr(stb + fb[j] + q * G::FK * G::BN * 2, G::BN);
    };
    constexpr int AREADS = AT ? 2 : 1, BREADS = BK_ROWS ? 1 : 2;  // LDS reads per fragment
    // outstanding copies at the barrier once the next tile has landed: the
    // plain ring's S-2 younger tiles; the A3 ring's A refill of this tile
    constexpr int WAIT_VM = A3 ? G::A_LOADS : (S - 2) * G::LPW;
    // copy selections: which copies of a tile a step issues, and whether the
    // tile is a full K tile (copied without a per-copy test)
    enum { kNone = 0, kAll = 1, kA = 2, kB = 3 };
    // One MFMA step on (fa_, fb_[PB]).  NEXT: the fragments of step nq of the
    // slots at (nsa, nsb) are read into (fa_, fb_[1-PB]) meanwhile, each A
    // fragment right after its last MFMA row, the B fragments spread over the
    // rows.  CP = 2*part + full: the selected copies of K tile ckt into A slot
    // csa / B slot csb are spread over the rows.  BAR >= 0: the step starts
    // with BAR MFMA rows, then the wait and barrier that make the next tile
    // readable and free the slots computed; the reads and copies fill the
    // rows from there on, while the MFMAs already issued keep the matrix
    // pipe busy through the barrier.
    auto step = [&](auto pb_c, auto next_c, auto cp_c, auto bar_c, const char *nsa, const char *nsb, int nq, int ckt,
                    int csa, int csb) __attribute__((always_inline)) {
      constexpr int PB = decltype(pb_c)::value;
      constexpr bool NEXT = decltype(next_c)::value;
      constexpr int PART = decltype(cp_c)::value / 2;
      constexpr bool FULL = decltype(cp_c)::value % 2 == 1;
      constexpr int NC = PART == kAll ? G::LPW : PART == kA ? G::A_LOADS : PART == kB ? G::B_LOADS : 0;
      constexpr int J0 = PART == kB ? G::A_LOADS : 0;
      constexpr int BAR = decltype(bar_c)::value;
      constexpr int R0 = BAR > 0 ? BAR : 0;     // first row that may read or copy
      constexpr int NR = G::TM - R0;            // rows that read and copy
      auto row = [&](auto i_c) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value;
        if constexpr (i == BAR) {
          __builtin_amdgcn_sched_barrier(0);
          wait_vmcnt_lgkm0<WAIT_VM>();  // the next tile has landed (this wave's copies)
          block_barrier();              // ... every wave's; the slots computed are free
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < G::TN; ++j) {
          if constexpr (MF == 32) acc[i][j] = Mfma<T>::m32(fb_[PB][j], fa_[i], acc[i][j]);
          else acc[i][j] = Mfma<T>::m16(fb_[PB][j], fa_[i], acc[i][j]);
        }
        if constexpr (i >= R0) {
          constexpr int r = i - R0;
          constexpr int a0 = r == 0 ? 0 : i, a1 = i + 1;                     // A fragments refilled here
          constexpr int b0 = r * G::TN / NR, b1 = (r + 1) * G::TN / NR;     // B fragments read here
          if constexpr (NEXT) {
#pragma unroll
            for (int j = b0; j < b1; ++j) read_b(nsb, nq, 1 - PB, j);
#pragma unroll
            for (int a = a0; a < a1; ++a) read_a(nsa, nq, a);
            // the row's MFMAs with its LDS reads in between, one read after each MFMA
            constexpr int NRD = BREADS * (b1 - b0) + AREADS * (a1 - a0);
            [&]<int... U>(std::integer_sequence<int, U...>) __attribute__((always_inline)) {
              ((__builtin_amdgcn_sched_group_barrier(0x008, 1, 0),
                (U < NRD ? __builtin_amdgcn_sched_group_barrier(0x100, 1, 0) : (void)0)),
               ...);
            }(std::make_integer_sequence<int, G::TN>{});
            if constexpr (NRD > G::TN) __builtin_amdgcn_sched_group_barrier(0x100, NRD - G::TN, 0);
          }
          if constexpr (NC > 0) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = r * NC / NR; c < (r + 1) * NC / NR; ++c) {
              if constexpr (FULL) issue_one(ckt, csa, csb, J0 + c);
              else copy(ckt, csa, csb, J0 + c);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
          __builtin_amdgcn_sched_group_barrier(0x008, G::TN, 0);
        }
      };
      [&]<int... I>(std::integer_sequence<int, I...>) __attribute__((always_inline)) {
        (row(std::integral_constant<int, I>{}), ...);
      }(std::make_integer_sequence<int, G::TM>{});
    };
    using F = std::false_type;
    using Tr = std::true_type;
    using NoBar = std::integral_constant<int, -1>;
    using BarRow = std::integral_constant<int, (kBarrierRows < G::TM ? kBarrierRows : G::TM - 1)>;
    using NoCopy = std::integral_constant<int, 0>;
    // One tile.  MODE 2: its refill is a full K tile; 1: any tile (ragged or
    // past the end); 0: the last tile, no refill and no read-ahead.
    auto tile = [&](auto mode_c) __attribute__((always_inline)) {
      constexpr int MODE = decltype(mode_c)::value;
      constexpr int FULL = MODE == 2 ? 1 : 0;
      const char *sta = a_slot(ca), *stb = b_slot(cb);
      // the A3 ring's A refill (tile kt+2, into the A slot computed a tile ago)
      // rides the first step; the plain ring refills everything in the last
      const int ra = ca == 0 ? 2 : ca - 1;
      using FirstCopy = std::integral_constant<int, (A3 && MODE != 0) ? 2 * kA + FULL : 0>;
      // steps 0 .. KSUB-2, each reading the next step's fragments from this tile's slots
      [&]<int... Q>(std::integer_sequence<int, Q...>) __attribute__((always_inline)) {
        (step(std::integral_constant<int, Q & 1>{}, Tr{},
              std::integral_constant<int, Q == 0 ? FirstCopy::value : 0>{}, NoBar{}, sta, stb, Q + 1, kt + 2, ra,
              0),
         ...);
      }(std::make_integer_sequence<int, G::KSUB - 1>{});
      using PLast = std::integral_constant<int, (G::KSUB - 1) & 1>;
      if constexpr (MODE != 0) {
        const int na = A3 ? (ca == 2 ? 0 : ca + 1) : (ca + 1 == S ? 0 : ca + 1);
        const int nb = A3 ? 1 - cb : na;
        using LastCopy = std::integral_constant<int, 2 * (A3 ? kB : kAll) + FULL>;
        step(PLast{}, Tr{}, LastCopy{}, BarRow{}, a_slot(na), b_slot(nb), 0, A3 ? kt + 2 : kt + S, ca, cb);
        if constexpr (PLast::value == 0) {
          // odd number of steps: the next tile's first B fragments were read
          // into buffer 1; move them so that every tile starts on buffer 0
#pragma unroll
          for (int j = 0; j < G::TN; ++j) fb_[0][j] = fb_[1][j];
        }
        ca = na;
        cb = nb;
        ++kt;
      } else {
        step(PLast{}, F{}, NoCopy{}, NoBar{}, sta, stb, 0, 0, 0, 0);
      }
    };

    // prologue: tiles 0 .. S-1 in flight (the A3 ring: tiles 0 and 1), tile
    // 0's first fragments read
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < G::LPW; ++j) copy(s, s, s, j);
    }
    wait_vmcnt_lgkm0<(S - 1) * G::LPW>();
    block_barrier();
    if (nk > 0) {
#pragma unroll
      for (int i = 0; i < G::TM; ++i) read_a(a_slot(0), 0, i);
#pragma unroll
      for (int j = 0; j < G::TN; ++j) read_b(b_slot(0), 0, 0, j);
    }
    // steady state: the refill is a full K tile; then the tiles whose refill
    // is the ragged tile or past the end; then the last tile
    constexpr int AHEAD = A3 ? 2 : S;  // the refill of tile kt is tile kt + AHEAD
    while (kt + AHEAD < nfull) tile(std::integral_constant<int, 2>{});
    while (kt + 1 < nk) tile(std::integral_constant<int, 1>{});
    if (kt < nk) tile(std::integral_constant<int, 0>{});
    // the refills past the end are still landing in LDS, which the epilogue reuses
    wait_vmcnt_lgkm0<0>();
  }

  const int64_t cbase = GRP == kGroupGradB ? int64_t(group) * p.c_stride : 0;
  auto store = [&](auto o) __attribute__((always_inline)) {
    using O = decltype(o);
    store_tile<G, O>(acc, static_cast<O *>(p.C) + cbase, smem, m0, n0, wave, wr, wc, lane, M, N);
  };
  if (p.out_dtype == TSS_F32) store(float{});
  else if (p.out_dtype == TSS_F16) store(_Float16{});
  else store(__bf16{});
}

// Grouped products.  The tiles are those of G, 512 threads and one workgroup
// a CU; where the last round of kCUs tiles has few of them they are cut into
// pieces, two of 128 x 256 or four of 128 x 128 (an element's sums are the
// same in any of them).  Half == G: small tiles, all alike.
template <typename G, typename Half, typename Quarter, typename T, int GRP>
__global__ __launch_bounds__(G::THREADS) void grouped_gemm_kernel(GroupedArgs p) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  constexpr bool PIECES = !__is_same(G, Half);
  constexpr bool RAGGED = GRP != kGroupGradB;
  static_assert(G::THREADS == Half::THREADS && G::THREADS == Quarter::THREADS, "one launch");
  static_assert(!PIECES || (Half::BM * 2 == G::BM && Quarter::BM * 2 == G::BM && Half::BN == G::BN &&
                            Quarter::BN * 2 == G::BN), "pieces of a tile");
  const int lane = threadIdx.x & 63, bid = blockIdx.x;
  // only the tiles there are take part; the launch's spare workgroups end here
  const int n = (RAGGED ? int(count_group_tiles<G::BM>(p.sizes, p.groups, p.M, lane)) : p.groups * p.tiles_m) * p.tiles_n;
  const int whole = PIECES ? n / kCUs * kCUs : n, rest = n - whole;
  const int pieces = PIECES ? tile_pieces(rest, RAGGED) : 1;
  if (bid >= whole + rest * pieces) return;
  // RAGGED: the XCDs get runs of equal length.  GradB's tiles cost as much as
  // their group has rows, so there each group is dealt over the XCDs (given
  // whole groups, the XCD of the largest one held up the others: 365 -> 244 us
  // on 16384 rows in 8 uneven groups, K 4096, N 2048).
  int id = bid, part = 0;
  if (bid >= whole) {
    const int x = RAGGED ? xcd_run(bid - whole, rest * pieces) : bid - whole;
    id = whole + x / pieces;
    part = x % pieces;
  } else if constexpr (RAGGED) {
    id = xcd_run(bid, whole);
  }
  int m0, n0, M = p.M, K, group, kbeg = 0;
  if constexpr (RAGGED) {
    // one tile row after the other: the column tiles of a group's rows are
    // neighbours in an XCD's run
    const int tm = id / p.tiles_n;
    const GroupTile g = find_group_tile<G::BM>(p.sizes, p.groups, p.M, tm, lane);
    m0 = g.row0;
    n0 = (id - tm * p.tiles_n) * G::BN;
    M = g.row_end;
    const bool none = g.group == p.groups;  // rows of no group
    K = none ? 0 : p.K;
    group = none ? 0 : g.group;
  } else {
    const int mn = p.tiles_m * p.tiles_n;
    group = id / mn;
    constexpr int GM = 4;  // tile rows that share an XCD's run of tiles
    const int in = xcd_run(id - group * mn, mn), span = GM * p.tiles_n, first = in / span * GM;
    const int gm = min(p.tiles_m - first, GM), r = in % span;
    m0 = (first + r % gm) * G::BM;
    n0 = r / gm * G::BN;
    const GroupTile g = group_rows(p.sizes, p.groups, p.rows_total, group, lane);
    kbeg = g.row0;
    K = g.row_end - g.row0;
  }
  if (!PIECES || bid < whole || pieces == 1) {
    if constexpr (PIECES && RAGGED) {
      // the last tile of a group, when half empty: one piece holds it
      if (M - m0 <= Half::BM) {
        grouped_tile_product<Half, T, GRP>(p, smem, m0, n0, M, K, group, kbeg);
        return;
      }
    }
    grouped_tile_product<G, T, GRP>(p, smem, m0, n0, M, K, group, kbeg);
  } else if constexpr (PIECES) {
    m0 += (pieces == 2 ? part : part / 2) * Half::BM;
    if (pieces == 4) n0 += part % 2 * Quarter::BN;
    if (m0 >= M || n0 >= p.N) return;
    if (pieces == 2) grouped_tile_product<Half, T, GRP>(p, smem, m0, n0, M, K, group, kbeg);
    else grouped_tile_product<Quarter, T, GRP>(p, smem, m0, n0, M, K, group, kbeg);
  }
}

}  // namespace tss

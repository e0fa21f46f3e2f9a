// How the 8-bit and grouped products are cut up: rules on the sizes alone,
// host code without HIP, so that a test can ask them which way a size runs.
#pragma once
#include <stdint.h>

namespace tss {

constexpr int kCUs = 256;

// Pieces that a tile of the last round is cut into.  Of ragged rows a group's
// last tile is often less than half full and its empty pieces end at once, so
// a third more than a round may be launched.
constexpr int tile_pieces(int rest, bool ragged) {
  const int most = ragged ? kCUs * 4 / 3 : kCUs;
  return rest * 4 <= most ? 4 : rest * 2 <= most ? 2 : 1;
}

// An 8-bit product: by tiles of bm x bn, K in `splits` ranges of their own
// workgroups and each of them in `sets` of a workgroup's waves; or (bn == 16)
// by the kernel for few rows.
struct ProductPlan {
  int bm, bn, splits, sets = 1;
};

// exact: the blocks of K are summed in fp32 (on fp16 fragments).
inline ProductPlan plan_product(int64_t M, int64_t N, int64_t K, bool exact) {
  const int64_t kb = (K + 127) / 128;
  // The kernel for few rows takes about 3.6 us and, every 16 x 16 tile reading
  // its own rows of both operands from L2, MNK / 8 bytes at 8 TB/s; tiles take
  // about 5 us and 0.37 a step, or about 10 with K split.  76 x 480 x 3200:
  // 6.2 against 10.4 us; 64 x 2048 x 2048: 7.2 and 10; 64 x 8192 x 4096: 33 and 13.
  const int64_t steps100 = 160 + 37 * kb;
  if (M <= 16 || M * N * K <= 640000 * (steps100 < 700 ? steps100 : 700)) return {16, 16, 1};
  auto blocks = [&](int64_t bm, int64_t bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); };
  // One round of 128 x 128 tiles where they fit it (3249 x 1098 x 2384: 20.6 us,
  // and 27.7 in halves of 256 x 256).
  const int64_t b128 = blocks(128, 128);
  if (!exact && b128 >= 160) return b128 <= kCUs ? ProductPlan{128, 128, 1} : ProductPlan{256, 256, 1};
  if (exact && b128 >= kCUs) return {128, 128, 1};
  const int64_t b = blocks(64, 128);
  int64_t s = b >= kCUs ? 1 : kCUs / b;
  if (s > kb / 8) s = kb / 8;  // at least eight steps of K a range
  s = s > 8 ? 8 : s < 1 ? 1 : s;
  // Two sets of waves in a workgroup, where a CU has but one: they shorten the
  // steps' chains of waits (1620 x 776 x 3584: 17.0 -> 15.2 us; fp32 output,
  // 1236 x 1382 x 5008: 37.8 -> 29.2) but cost 1 to 2 us at the ends (968 x
  // 2052 x 864: 12.1 -> 18.5).
  const bool sets = b * s <= kCUs && kb / s >= (exact ? 8 : 16);
  return {64, 128, int(s), sets ? 2 : 1};
}

// Elements between the partial sums of two ranges: whole 16-byte pieces.  (As
// an argument of the kernel instead: 8192^3 452 us, this 442.)
constexpr int64_t slice_elements(int64_t M, int64_t N) { return (M * N + 3) / 4 * 4; }

// K of a range: a multiple of 128; the ranges that hold any.
inline void split_ranges(int64_t K, int splits, int32_t *n, int32_t *k_split) {
  const int64_t kb = (K + 127) / 128, per = (kb + splits - 1) / splits;
  *k_split = int32_t(per * 128);
  *n = int32_t((kb + per - 1) / per);
}

// Products of 8-bit integers.  Groups of 16 columns of a workgroup of the
// kernel for few rows: two where workgroups of one would be more than the CUs,
// which then take a second round (us with one group and with two, weights in no
// cache; 16 rows, K = 4096: N = 4000 7.6 and 9.1, 4096 7.8 and 9.4, 4112 9.9 and
// 9.1, 5120 11.0 and 9.3; K = 8192: 4096 12.7 and 16.9, 5120 21.7 and 17.8; 64
// rows, K = 4096: 1024 7.3 and 9.0, 1040 10.1 and 9.0; K <= 1024 within 0.2).
inline int int8_row_groups(int64_t M, int64_t N) { return (M + 15) / 16 * ((N + 15) / 16) > kCUs ? 2 : 1; }

// The launch of the kernel for few rows: groups of 16 columns of a workgroup,
// workgroups, and waves of each (as many as join a group each, at least).
struct Int8RowsLaunch {
  int groups;
  int64_t workgroups;
  int waves;
};
inline Int8RowsLaunch int8_rows_launch(int64_t M, int64_t N, int64_t K) {
  const int groups = int8_row_groups(M, N), blocks = groups == 2 ? 1 : 4;  // blocks of 128 of K that a wave takes at a time
  const int64_t nk = (K + 127) / 128, nw = (nk + blocks - 1) / blocks, most = nw > 16 ? 16 : nw;
  return {groups, (M + 15) / 16 * ((N + 16 * groups - 1) / (16 * groups)), int(most > groups ? most : groups)};
}

// By the time that each way takes, in ns.  The kernel for few rows: 3200, and
// the longer of a workgroup's own reads and all of them, from L2 at 8.5 TB/s
// (64 x 4096 x 4096: 14.8 us, 64 x 1024 x 8192 11.1, 64 x 8192 x 1024 9.0).
// Tiles of 64 x 128: 5300 and 320 a step of K; ranges of K cost a second launch
// and 4 bytes of partial sums an element each (128 x 4096 x 4096: 16.2, 13.6 and
// 15.1 us in 1, 2 and 4 ranges; 1024 x 1024 x 4096: 16.4, 17.8 and 20.4; 256 x 512
// x 8192: 25.7, 18.2, 14.4 and in 8 ranges 13.9).  More of them than CUs: one
// round of 128 x 128 (634 x 3778 x 5088: 30.2 us, in 300 of 64 x 128 39.7), else
// 256 x 256 (5139 x 2722 x 7440: 115, 164 and 200 us; 836 x 5581 x 240: 13.6, 16.4
// and 15.5).
inline ProductPlan plan_int8(int64_t M, int64_t N, int64_t K) {
  if (M <= 16) return {16, 16, 1};
  auto blocks = [&](int64_t bm, int64_t bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); };
  const int64_t kb = (K + 127) / 128, b = blocks(64, 128), b128 = blocks(128, 128), b256 = blocks(256, 256);
  if (b > kCUs) {
    // two rounds of 128 x 128 where 256 x 256 would be one that is not cut (135 of these: 43.4 us, 493 of those 37.5)
    const bool two = b128 <= 2 * kCUs && b256 > kCUs / 2 && b256 < kCUs;
    return b128 <= kCUs || two ? ProductPlan{128, 128, 1} : ProductPlan{256, 256, 1};
  }
  auto tiles = [&](int64_t s) { return 5300 + 320 * ((kb + s - 1) / s) + (s > 1 ? 1200 + s * (300 + M * N / 430) : 0); };
  ProductPlan p{64, 128, 1};
  for (int s = 2; s <= 8 && b * s <= kCUs; ++s)
    if (tiles(s) < tiles(p.splits)) p.splits = s;
  const int64_t columns = 16 * int8_row_groups(M, N);
  const int64_t own = 830 * K / 1024, all = blocks(16, columns) * (16 + columns) * K / 8500;
  if (3200 + (own > all ? own : all) < tiles(p.splits)) return {16, 16, 1};
  return p;
}

// 8-bit products grouped by expert.
// Small tiles where they leave CUs free anyway (581 rows in 3 groups, K 2240, N
// 792: 13.9 us against 16.0 and 15.5 with 128 x 128 and 256 x 256) and for few
// rows a group; large ones from 192 (128 rows a group, E = 32, K = 4096, N =
// 2048: 95, 85 and 92 us with the three tiles; 256 rows: 155, 141 and 111).
inline ProductPlan plan_grouped_fp8(int64_t T, int64_t N, int64_t K, int64_t E, bool exact) {
  const int64_t rows = T / E;  // of an average group
  const int64_t tiles64 = (T / 64 + E < T ? T / 64 + E : T) * ((N + 127) / 128), a_reads = (N + 15) / 16 * T * K;
  if (K > 0 && tiles64 < kCUs && a_reads <= int64_t(40) << 20) return {16, 16, 1};
  if (rows <= 64 || tiles64 <= kCUs) return {64, 128, 1, tiles64 <= kCUs && K >= (exact ? 1024 : 4096) ? 2 : 1};
  if (rows <= 192 || exact) return {128, 128, 1};
  return {256, 256, 1};
}

// The 16-bit products grouped by expert, forward and gradient of A: 256 x 256
// tiles (256), 64 x 64 tiles (64) or the kernel for few rows (16).
// Few rows in an average group: the groups' weights are the cost, and small
// tiles put more of their loads in flight.  Forward, E = 32, K = N = 2048,
// 64 x 64 against 256 x 256 tiles: 16 rows a group 57 and 61 us, 64 rows 73
// and 63, 256 rows 181 and 99; where the small ones fit the chip at once, 78
// rows in 25 groups, K = 2208, N = 640: 22 and 38; 300 rows in 2, K = 4096, N =
// 1024: 19 and 29; 323 rows in 3, K = 2016, N = 1952, 558 small tiles: 27 and 21.
inline int plan_grouped_rows(int64_t T, int64_t N, int64_t E) {
  // The kernel for few rows reads 3/16 of a byte for each of T K N from L2, at
  // 5.5 TB/s, against 0.2 us for each 64 of K where the small tiles leave CUs
  // free: T N up to about 1e5.  162 rows in 2 groups, K = 2560, N = 344: 10.1
  // and 13.1 us; 64 rows in 32 groups, K = 4096, N = 2048: 89 and 83.
  const int64_t rows64 = T / 64 + E, tiles64 = (rows64 < T ? rows64 : T) * ((N + 63) / 64);
  if (tiles64 <= 2 * kCUs && T * N <= int64_t(1) << 17) return 16;
  const int64_t rows = T / E;  // of an average group
  return rows <= 32 || tiles64 <= (rows <= 128 ? 3 * kCUs : 7 * kCUs / 4) ? 64 : 256;
}

// The gradient of B: 256 x 256 or 128 x 128 tiles.  With few rows to reduce
// over the writes are the cost.  E = 32, K = 4096, N = 2048, 2 rows a group:
// 128 x 128 tiles 165 us, 256 x 256 178; K = N = 2048, 64 rows a group 99 and
// 100, 256 rows 143 and 136.
inline int plan_grad_b(int64_t T, int64_t E) { return T / E <= 64 ? 128 : 256; }

}  // namespace tss

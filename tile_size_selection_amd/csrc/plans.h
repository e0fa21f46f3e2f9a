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

// Ragged groups of rows, resolved on the device: rows 0 .. T-1 are cut into
// groups of sizes[0], sizes[1], ... (a negative size counts as 0, groups end
// at row T), each group into tiles of BM rows, and the rows past the last
// group into tiles of their own.  The launch has one workgroup for every
// tile there can be (max_group_tiles); every wave finds its tile from the
// sizes, so nothing is read back to the host and a replayed graph follows
// the sizes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tss {

constexpr int kMaxGroups = 4096;

// Workgroups are dealt to the 8 XCDs round-robin: this gives each XCD a
// contiguous run of 0 .. n-1, so that lines shared by neighbours are shared
// in one L2.
__device__ __forceinline__ int xcd_run(int bid, int n) {
  const int xcd = bid & 7, local = bid >> 3, per = n >> 3, extra = n & 7;
  return xcd < extra ? xcd * (per + 1) + local : extra * (per + 1) + (xcd - extra) * per + local;
}

// Tiles of BM rows that T rows in E groups (and a rest) can need: each group
// and the rest end at most one tile short, and no tile is empty.
inline int64_t max_group_tiles(int64_t T, int64_t E, int64_t BM) {
  const int64_t most = T / BM + E + 1;
  return most < T ? most : T;
}

// Inclusive sum over the lanes of a wave, each step cut off at `limit` (< 2^31: no step overflows).
__device__ __forceinline__ uint32_t scan64(uint32_t v, uint32_t limit, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(v, d);
    if (lane >= d) v = min(v + o, limit);
  }
  return v;
}

struct GroupTile {
  int group;  // E: rows of no group
  int row0, row_end;  // the tile's rows; row0 == row_end: past the last tile
};

// One chunk of 64 groups: each lane's rows and tiles, from the rows and tiles before the chunk.
template <int BM>
struct GroupChunk {
  uint32_t end, start;   // rows of the lane's group
  uint32_t tiles;        // tiles up to and with it
  __device__ __forceinline__ void scan(const int32_t *sizes, int E, uint32_t T, int base, uint32_t rows, uint32_t before,
                                       int lane) {
    const int g = base + lane;
    const uint32_t n = g < E ? min(uint32_t(max(sizes[g], 0)), T) : 0u;
    end = min(scan64(n, T, lane) + rows, T);
    start = __shfl_up(end, 1);
    if (lane == 0) start = rows;
    tiles = scan64((end - start + BM - 1) / BM, 0x7fffffffu, lane) + before;
  }
};

// The number of tiles of all groups and the rest.
template <int BM>
__device__ __forceinline__ uint32_t count_group_tiles(const int32_t *sizes, int E, uint32_t T, int lane) {
  uint32_t rows = 0, before = 0;
  for (int base = 0; base < E; base += 64) {
    GroupChunk<BM> c;
    c.scan(sizes, E, T, base, rows, before, lane);
    rows = __builtin_amdgcn_readlane(c.end, 63);
    before = __builtin_amdgcn_readlane(c.tiles, 63);
  }
  return before + (T - rows + BM - 1) / BM;
}

template <int BM>
__device__ __forceinline__ GroupTile find_group_tile(const int32_t *sizes, int E, uint32_t T, uint32_t want, int lane) {
  uint32_t rows = 0, before = 0;
  for (int base = 0; base < E; base += 64) {
    GroupChunk<BM> c;
    c.scan(sizes, E, T, base, rows, before, lane);
    const uint64_t past = __ballot(c.tiles > want);
    if (past) {
      const int l = __builtin_ctzll(past);
      const uint32_t first = l ? uint32_t(__builtin_amdgcn_readlane(c.tiles, l - 1)) : before;
      const uint32_t s = __builtin_amdgcn_readlane(c.start, l), e = __builtin_amdgcn_readlane(c.end, l);
      const uint32_t r0 = s + (want - first) * BM;
      return {base + l, int(r0), int(min(r0 + uint32_t(BM), e))};
    }
    rows = __builtin_amdgcn_readlane(c.end, 63);
    before = __builtin_amdgcn_readlane(c.tiles, 63);
  }
  const uint32_t r0 = min(rows + (want - before) * BM, T);
  return {E, int(r0), int(min(r0 + uint32_t(BM), T))};
}

// The rows of one group.
__device__ __forceinline__ GroupTile group_rows(const int32_t *sizes, int E, uint32_t T, int group, int lane) {
  uint32_t rows = 0;
  for (int base = 0;; base += 64) {
    GroupChunk<1> c;
    c.scan(sizes, E, T, base, rows, 0, lane);
    if (group < base + 64)
      return {group, int(__builtin_amdgcn_readlane(c.start, group - base)),
              int(__builtin_amdgcn_readlane(c.end, group - base))};
    rows = __builtin_amdgcn_readlane(c.end, 63);
  }
}

}  // namespace tss

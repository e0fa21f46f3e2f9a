// Rows sorted by expert and joined again.
//
// The router gives each of `tokens` tokens `top` choices of an expert; choice
// i = t * top + j.  A stable counting sort by expert gives each choice its
// row: row[i], and choice[row] = i; sizes[e] rows belong to expert e.  A
// choice outside 0 .. E-1 is dropped: its place is behind the routed rows (in
// order), and both entries hold the complement (~place, ~i: negative), so
// that whoever reads them knows without the sizes.
//
//   gather:             rows[row[t][j]] = x[t]                (dropped: zeros)
//   combine:            y[t] = sum_j w[t][j] rows[row[t][j]]  (dropped: not read)
//   combine's backward: drows[row[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], rows[row[t][j]]>
//
// All are bound by memory and go token by token: a token's row is read (or
// written) once, its choices' rows are the bulk.  Sums run over j in order in
// fp32: no atomics on values, the same bits on every run.  Indices that lie
// outside the rows are taken as dropped ones without a place.
//
// Measured: 131072 choices of 128 experts sorted in 12.2 us (two launches of
// dependent steps; 8 choices: 3.6), 16384 x 8 x 4096 bytes with scales gathered
// in 107 us (5.8 TB/s; a large copy: 5.1), 5001 x 6 x 5120 bf16 combined in 70
// (4.9), the gradients of 8200 x 4 x 2048 fp16 in 57 (5.3).  131072 choices of
// 1000 experts: 17.5 us, of 4096 28.6 (places by fewer waves, and the counts
// added up by a launch of their own).  Gradients of rows of 32768 columns: fp32
// 2000 x 4 673 us, 3.5 TB/s (4 choices of 4 chunks are 128 registers: 304 bytes a
// lane are spilled), bf16 234 (5.0).
#include "ranges.h"
#include "row_launch.h"

using namespace tss;

namespace {

// ---- the sort ----

constexpr int kSortThreads = 1024;
constexpr int kSortCounters = 9600;        // LDS counters
constexpr int64_t kOneGroup = 4096;        // choices that one workgroup sorts by itself
constexpr int kHeld = 8192;                // choices whose bins a workgroup keeps
constexpr int64_t kScannedCounts = 8192;   // more counts than these are added up by a launch of their own

struct SortArgs {
  const void *expert;
  int n, E;
  int per_group;      // choices of a workgroup, a multiple of 64
  int placing;        // waves that share them
  bool scanned;
  int32_t *sizes, *row, *choice;
  uint32_t *counts;   // [workgroups + 1][E + 1]
};

// Waves that place choices: as many as have counters of their own.
__host__ __device__ constexpr int sort_waves(int E) {
  const int w = kSortCounters / (E + 1);
  return w >= 16 ? 16 : w >= 8 ? 8 : w >= 4 ? 4 : w >= 2 ? 2 : 1;
}

// The bin of choice i: its expert, or E.
template <typename I>
__device__ __forceinline__ int bin_of(const SortArgs &p, int i) {
  const I e = static_cast<const I *>(p.expert)[i];
  return e >= 0 && e < I(p.E) ? int(e) : p.E;
}

template <typename I>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs p) {
  extern __shared__ uint32_t count[];  // [E + 1]: all waves share them, a sum of integers has no order
  const int bins = p.E + 1;
  for (int b = threadIdx.x; b < bins; b += blockDim.x) count[b] = 0;
  __syncthreads();
  const int from = blockIdx.x * p.per_group, end = min(p.n, from + p.per_group);
  for (int i = from + threadIdx.x; i < end; i += blockDim.x) atomicAdd(&count[bin_of<I>(p, i)], 1u);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += blockDim.x) p.counts[int64_t(blockIdx.x) * bins + b] = count[b];
}

// Each bin's counts become its choices in the workgroups before; the row
// behind the last holds the totals.  For many bins or workgroups: else every
// placing workgroup adds them up by itself, which saves a launch.
__global__ __launch_bounds__(256) void sort_scan_kernel(int groups, int bins, uint32_t *counts) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= bins) return;
  uint32_t sum = 0;
  for (int g0 = 0; g0 < groups; g0 += 16) {
    uint32_t c[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) c[u] = g0 + u < groups ? counts[int64_t(g0 + u) * bins + b] : 0;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      if (g0 + u < groups) counts[int64_t(g0 + u) * bins + b] = sum;
      sum += c[u];
    }
  }
  counts[int64_t(groups) * bins + b] = sum;
}

// Places: a bin begins behind all smaller bins, a workgroup's part of it
// behind those of the workgroups before it, a wave's behind those of its
// workgroup's earlier waves; within a wave 64 choices at a time, each behind
// the lanes before it that have the same bin.
template <typename I, bool MANY>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs p) {
  extern __shared__ uint32_t count[];  // [placing waves][bins]
  __shared__ uint32_t wave_sum[kSortThreads / 64], share[2][MANY ? kSortThreads : 1];
  __shared__ uint16_t held_bins[kHeld];
  const int bins = p.E + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int groups = MANY ? gridDim.x : 1, group = MANY ? blockIdx.x : 0;  // not MANY: one workgroup sorts all
  const int placing = p.placing;
  const int per_wave = p.per_group / placing;  // a multiple of 64
  const int group_end = min(int64_t(p.n), (int64_t(group) + 1) * p.per_group);
  const int from = wave < placing ? min(group_end, group * p.per_group + wave * per_wave) : group_end;
  const int end = min(group_end, from + per_wave);
  uint32_t *mine = count + wave * bins;
  // Bins b0 .. b0 + width - 1 of the workgroups (few bins: the threads share the
  // workgroups among them): in all, and of those before this one.
  int width = kSortThreads;
  while (width / 2 >= bins) width /= 2;
  const int parts = kSortThreads / width, at = threadIdx.x & (width - 1), part = threadIdx.x / width;
  uint32_t total = 0, before = 0;
  auto add_groups = [&](int b) __attribute__((always_inline)) {
    total = before = 0;
    if (b >= bins) return;
    if (p.scanned) {
      total = p.counts[int64_t(groups) * bins + b];
      before = p.counts[int64_t(group) * bins + b];
    } else {
#pragma unroll 8
      for (int g = part; g < groups; g += parts) {
        const uint32_t c = p.counts[int64_t(g) * bins + b];
        total += c;
        before += g < group ? c : 0;
      }
    }
  };
  const bool shared = MANY && !p.scanned && parts > 1;
  if constexpr (MANY) add_groups(p.scanned ? threadIdx.x : at);
  for (int b = threadIdx.x; b < placing * bins; b += kSortThreads) count[b] = 0;
  if (shared) {
    share[0][threadIdx.x] = total;
    share[1][threadIdx.x] = before;
  }
  __syncthreads();
  // the bins are kept for the second time, if the workgroup's fit
  const bool held = !MANY || p.per_group <= kHeld;
  const int group_from = group * p.per_group;
#pragma unroll 4
  for (int i = from + lane; i < end; i += 64) {
    const int b = bin_of<I>(p, i);
    if (held) held_bins[i - group_from] = uint16_t(b);
    atomicAdd(&mine[b], 1u);
  }
  if (shared) {
    total = before = 0;
    if (part == 0)
      for (int i = 0; i < parts; ++i) {
        total += share[0][i * width + at];
        before += share[1][i * width + at];
      }
  }
  __syncthreads();
  // the waves' counters become the waves' first places, bin by bin
  uint32_t before_bins = 0;
  for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
    const int b = b0 + threadIdx.x;
    if constexpr (!MANY) {
      total = 0;
      if (b < bins)
#pragma unroll 4
        for (int w = 0; w < placing; ++w) total += count[w * bins + b];
    } else if (b0 > 0) {
      add_groups(b);  // as many bins as threads: none is shared
    }
    uint32_t upto = scan64(total, 0x7fffffffu, lane);
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
    uint32_t all = 0;
#pragma unroll 4
    for (int w = 0; w < kSortThreads / 64; ++w) {
      const uint32_t s = wave_sum[w];
      upto += w < wave ? s : 0;
      all += s;
    }
    if (b < bins) {
      uint32_t first = before_bins + upto - total + before;
#pragma unroll 1
      for (int w0 = 0; w0 < placing; w0 += 4) {
        uint32_t c[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) c[u] = w0 + u < placing ? count[(w0 + u) * bins + b] : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (w0 + u < placing) count[(w0 + u) * bins + b] = first;
          first += c[u];
        }
      }
      if (group == 0 && b < p.E) p.sizes[b] = int32_t(total);
    }
    before_bins += all;
    __syncthreads();
  }
#pragma unroll 1
  for (int i0 = from; i0 < end; i0 += 64) {
    const int i = i0 + lane;
    const bool in = i < end;
    const int b = !in ? bins : held ? held_bins[i - group_from] : bin_of<I>(p, i);
    uint64_t same = __ballot(in);  // the lanes with this lane's bin
#pragma unroll 1
    for (int bit = 1; bit < bins; bit *= 2) {
      const uint64_t set = __ballot(b & bit);
      same &= b & bit ? set : ~set;
    }
    if (in) {
      const int first = __builtin_ctzll(same);
      uint32_t to = 0;
      if (lane == first) to = atomicAdd(&mine[b], uint32_t(__builtin_popcountll(same)));
      to = __shfl(to, first) + __builtin_popcountll(same & ((uint64_t(1) << lane) - 1));
      const bool kept = b < p.E;
      p.row[i] = kept ? int32_t(to) : ~int32_t(to);
      p.choice[to] = kept ? i : ~i;
    }
  }
}

// How choices are dealt to workgroups.  One up to 4096 (us, captured, E = 128 to
// 256: 4096 choices 7.0 by one workgroup, 7.9 by two launches; 8192 9.7 and
// 8.2), then 2048 each, 4096 from 2^16 on (32768: 10.5 and 11.3; 131072: 12.9
// and 12.2; 2^20: 43 and 27).  The counts of the workgroups before are added up
// by every workgroup, or from 8192 of them on by a launch of their own (4112
// counts: 10.5 and 10.4; 8256: 12.9 and 12.4; 2064: 8.6 and 9.5).
struct SortShape {
  int64_t groups, per_group;
  bool scanned;
};
SortShape sort_shape(int64_t n, int64_t E) {
  const int64_t nw = sort_waves(int(E)), unit = nw * 64;
  if (n <= kOneGroup && (nw == 16 || n <= nw * 512)) return {1, (n + unit - 1) / unit * unit, false};
  const int64_t each = nw < 16 ? nw * 512 : n < 1 << 16 ? 2048 : 4096;
  int64_t groups = (n + each - 1) / each;
  groups = groups > 512 ? 512 : groups < 1 ? 1 : groups;
  const int64_t per = ((n + groups - 1) / groups + unit - 1) / unit * unit;
  return {groups, per, groups * (E + 1) > kScannedCounts};
}

// ---- rows ----

constexpr int kRowThreads = 256;

// Bytes of gathered rows from which on they pass the caches by (131072 x 4096
// bytes: 102 us, through them 113; x 4160 109 and 122); fewer are read from there
// by the product that follows.  Rows that share 64 bytes with their neighbours
// go through the caches, which join the parts (x 4112 143 us, past them 155;
// 64000 x 8200 144 and 168).
constexpr int64_t kStreamed = int64_t(1) << 28;

// What 16 (or 8) bytes of a row are to the copies below.
template <int BYTES>
struct Piece {
  typedef u32x4 type;
};
template <>
struct Piece<8> {
  typedef u32x2 type;
};

struct GatherArgs {
  const void *x;
  void *rows;
  const int32_t *row, *choice;
  const float *scale;
  float *scale_out;
  int tokens, top, pieces;  // pieces of a row
  int blocks_scale;         // column blocks of the scales
  uint32_t scale_groups;    // workgroups of the scales; those of the rows follow
};

constexpr int kScalesTogether = 16;  // 5186 x 6 x 6832 bytes, 54 blocks: 60 us, a thread for all blocks of a row 77
constexpr int kPlacesTogether = 8;  // places read before the first is written (one by one: 129 us, 126 with 8 a token)

// STREAMED: a template argument, because stores of both kinds behind a test are made one of the plain kind.
template <int BYTES, bool STREAMED>
__global__ __launch_bounds__(kRowThreads) void gather_rows_kernel(GatherArgs p) {
  using P = typename Piece<BYTES>::type;
  const int n = p.tokens * p.top;
  if (blockIdx.x >= p.scale_groups) {
    const uint32_t id = (blockIdx.x - p.scale_groups) * kRowThreads + threadIdx.x;
    const int t = int(id / uint32_t(p.pieces)), c = int(id - uint32_t(t) * uint32_t(p.pieces));
    if (t >= p.tokens) return;
    const P v = static_cast<const P *>(p.x)[int64_t(t) * p.pieces + c];
    P *rows = static_cast<P *>(p.rows);
    for (int j0 = 0; j0 < p.top; j0 += kPlacesTogether) {
      int r[kPlacesTogether];
#pragma unroll
      for (int u = 0; u < kPlacesTogether; ++u) r[u] = j0 + u < p.top ? p.row[int64_t(t) * p.top + j0 + u] : n;
#pragma unroll
      for (int u = 0; u < kPlacesTogether; ++u) {
        const int at = r[u] < 0 ? ~r[u] : r[u];
        if (at >= n) continue;
        P *to = rows + int64_t(at) * p.pieces + c;
        if constexpr (STREAMED) __builtin_nontemporal_store(r[u] < 0 ? P{} : v, to);
        else *to = r[u] < 0 ? P{} : v;
      }
    }
  } else {
    // the scales: a thread takes a row of the output and kScalesTogether of its column blocks
    const uint32_t across = uint32_t(p.blocks_scale + kScalesTogether - 1) / kScalesTogether;
    const int r = int(blockIdx.x / across * kRowThreads + threadIdx.x), b0 = int(blockIdx.x % across) * kScalesTogether;
    if (r >= n) return;
    const int i = p.choice[r];
    const bool in = i >= 0 && i < n;
    const int t = in ? i / p.top : 0;
    float v[kScalesTogether];
#pragma unroll
    for (int u = 0; u < kScalesTogether; ++u)
      v[u] = in && b0 + u < p.blocks_scale ? p.scale[int64_t(b0 + u) * p.tokens + t] : 0.0f;
#pragma unroll
    for (int u = 0; u < kScalesTogether; ++u)
      if (b0 + u < p.blocks_scale) p.scale_out[int64_t(b0 + u) * n + r] = v[u];
  }
}

struct CombineArgs {
  const void *rows;
  const int32_t *row;
  const float *weight;
  void *y;
  int tokens, top, chunks;  // chunks of 8 elements of a row
};

constexpr int kTogether = 4;  // choices whose rows a thread has in flight

// One thread, 8 columns of one token.
template <typename R, typename O>
__global__ __launch_bounds__(kRowThreads) void combine_rows_kernel(CombineArgs p) {
  const uint32_t id = blockIdx.x * kRowThreads + threadIdx.x;
  const int t = int(id / uint32_t(p.chunks)), c = int(id - uint32_t(t) * uint32_t(p.chunks));
  if (t >= p.tokens) return;
  const int n = p.tokens * p.top;
  const int32_t *row = p.row + int64_t(t) * p.top;
  const float *weight = p.weight ? p.weight + int64_t(t) * p.top : nullptr;
  const int64_t d = int64_t(p.chunks) * 8;
  const R *rows = static_cast<const R *>(p.rows) + c * 8;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int j0 = 0; j0 < p.top; j0 += kTogether) {
    Raw8<R> v[kTogether];
    float w[kTogether];
    bool in[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const int r = j0 + u < p.top ? row[j0 + u] : -1;
      in[u] = r >= 0 && r < n;
      w[u] = in[u] && weight ? weight[j0 + u] : 1.0f;
      if (in[u]) v[u] = load8(rows + r * d);
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      if (!in[u]) continue;
      float f[8];
      widen8(v[u], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[u], f[i], sum[i]);
    }
  }
  store8(static_cast<O *>(p.y) + t * d + c * 8, sum);
}

struct CombineBackArgs {
  const void *dy, *rows;
  const int32_t *row;
  const float *weight;
  void *drows;
  float *dweight;
  int tokens, top, d;
};

// A token is held by L neighbouring lanes, or (L == 64) by the workgroup's
// waves; kTogether choices at a time.
template <typename R, typename D, int CH, int L>
__global__ __launch_bounds__(kMaxThreads) void combine_backward_kernel(CombineBackArgs p) {
  __shared__ float red[2][kTogether][kMaxThreads / 64];
  constexpr bool kNarrow = L < 64;
  const int lanes = kNarrow ? L : int(blockDim.x), nw = blockDim.x >> 6, wave = threadIdx.x >> 6;
  const int l = threadIdx.x % lanes;
  const int t = blockIdx.x * (blockDim.x / lanes) + threadIdx.x / lanes;
  if (t >= p.tokens) return;  // L == 64: one token, the whole workgroup
  const int n = p.tokens * p.top, d = p.d;
  auto col_of = [&](int c) __attribute__((always_inline)) { return (c * lanes + l) * 8; };
  float dy[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
    widen8(col_of(c) < d ? load8(static_cast<const D *>(p.dy) + int64_t(t) * d + col_of(c)) : zero8<D>(), dy[c]);
  int slot = 0;
  for (int j0 = 0; j0 < p.top; j0 += kTogether) {
    int at[kTogether];
    bool in[kTogether];
    float w[kTogether], dot[kTogether];
    Raw8<R> v[kTogether][CH];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const bool has = j0 + u < p.top;
      const int r = has ? p.row[int64_t(t) * p.top + j0 + u] : n;
      at[u] = r < 0 ? ~r : r;
      in[u] = r >= 0 && r < n;
      w[u] = in[u] ? p.weight[int64_t(t) * p.top + j0 + u] : 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        v[u][c] = in[u] && col_of(c) < d ? load8(static_cast<const R *>(p.rows) + int64_t(at[u]) * d + col_of(c)) : zero8<R>();
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      dot[u] = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float f[8], o[8];
        widen8(v[u][c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[u] += dy[c][i] * f[i];
          o[i] = in[u] ? w[u] * dy[c][i] : 0.0f;
        }
        if (at[u] < n && col_of(c) < d) store8(static_cast<D *>(p.drows) + int64_t(at[u]) * d + col_of(c), o);
      }
      dot[u] = sum_lanes<L>(dot[u]);
    }
    if (!kNarrow && nw > 1) {
      // two sets of slots: a wave writes the next choices' while others may still read these
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int u = 0; u < kTogether; ++u) red[slot][u][wave] = dot[u];
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        dot[u] = 0;
        for (int i = 0; i < nw; ++i) dot[u] += red[slot][u][i];
      }
      slot ^= 1;
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      if (l == 0 && j0 + u < p.top) p.dweight[int64_t(t) * p.top + j0 + u] = in[u] ? dot[u] : 0.0f;
  }
}

// ---- host ----

constexpr int64_t kMaxThreadsOfLaunch = UINT32_MAX;

// tokens x top choices, and rows of d elements of a type.
int32_t check_tokens(int64_t tokens, int64_t top, int64_t d) {
  if (tokens < 0 || top < 1 || d < 1 || tokens > INT32_MAX || top > INT32_MAX || d > INT32_MAX / 8) return TSS_E_ARG;
  if (tokens * top > int64_t(1) << 30) return TSS_E_ARG;
  return d % 8 ? TSS_E_ALIGN : TSS_OK;
}

int size_of(int32_t dtype) {
  switch (dtype) {
    case TSS_F32: return 4;
    case TSS_F16: case TSS_BF16: return 2;
    case TSS_E4M3: case TSS_E5M2: case TSS_I8: return 1;
    default: return 0;
  }
}

bool is_float(int32_t dtype) { return dtype == TSS_F16 || dtype == TSS_BF16 || dtype == TSS_F32; }

// f with values of the two types; b is a's type or fp32, or a is fp32.
template <typename F>
int32_t with_types(int32_t a, int32_t b, F f) {
  if (!is_float(a) || !is_float(b) || (a != b && a != TSS_F32 && b != TSS_F32)) return TSS_E_DTYPE;
  if (a == TSS_F32 && b == TSS_F32) return f(float{}, float{});
  if (a == TSS_F32) return b == TSS_F16 ? f(float{}, _Float16{}) : f(float{}, __bf16{});
  if (b == TSS_F32) return a == TSS_F16 ? f(_Float16{}, float{}) : f(__bf16{}, float{});
  return a == TSS_F16 ? f(_Float16{}, _Float16{}) : f(__bf16{}, __bf16{});
}

int32_t launched() { return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP; }

}  // namespace

extern "C" {

int64_t tss_sort_by_expert_workspace_size(int64_t tokens, int64_t top, int64_t E) {
  const int32_t st = check_tokens(tokens, top, 8);
  if (st != TSS_OK) return st;
  if (E < 1 || E > kMaxGroups) return TSS_E_ARG;
  const int64_t g = sort_shape(tokens * top, E).groups;
  return g > 1 ? (g + 1) * (E + 1) * 4 : 0;
}

int32_t tss_sort_by_expert(int64_t tokens, int64_t top, int64_t E, const void *expert, int32_t expert_bits,
                           int32_t *sizes, int32_t *row, int32_t *choice, void *workspace, int64_t workspace_bytes,
                           void *stream) {
  const int64_t need = tss_sort_by_expert_workspace_size(tokens, top, E);
  if (need < 0) return int32_t(need);
  if (expert_bits != 32 && expert_bits != 64) return TSS_E_DTYPE;
  const int64_t n = tokens * top;
  if (!sizes || (n > 0 && (!expert || !row || !choice)) || (need && (!workspace || workspace_bytes < need))) return TSS_E_ARG;
  for (const void *q : {(const void *)sizes, (const void *)row, (const void *)choice, (const void *)workspace})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return TSS_E_ALIGN;
  if (reinterpret_cast<uintptr_t>(expert) & (expert_bits / 8 - 1)) return TSS_E_ALIGN;
  Ranges at;
  const uint32_t choices = at.reads(expert, n * expert_bits / 8);
  at.writes(sizes, E * 4);
  at.writes(row, n * 4, expert_bits == 32 ? choices : 0);  // a choice's own place, written when its bin is known
  at.writes(choice, n * 4);
  at.writes(workspace, need);
  if (at.clash()) return TSS_E_ARG;
  const SortShape f = sort_shape(n, E);
  const int nw = sort_waves(int(E));
  const SortArgs a{expert, int(n), int(E), int(f.per_group), nw, f.scanned, sizes, row, choice, static_cast<uint32_t *>(workspace)};
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto i) {
    using I = decltype(i);
    if (f.groups > 1)
      hipLaunchKernelGGL(sort_count_kernel<I>, dim3(uint32_t(f.groups)), dim3(kSortThreads), (E + 1) * 4, s, a);
    if (f.scanned)
      hipLaunchKernelGGL(sort_scan_kernel, dim3(uint32_t((E + 256) / 256)), dim3(256), 0, s, int(f.groups), int(E + 1),
                         a.counts);
    if (f.groups > 1)
      hipLaunchKernelGGL((sort_place_kernel<I, true>), dim3(uint32_t(f.groups)), dim3(kSortThreads), nw * (E + 1) * 4, s, a);
    else
      hipLaunchKernelGGL((sort_place_kernel<I, false>), dim3(1), dim3(kSortThreads), nw * (E + 1) * 4, s, a);
  };
  if (expert_bits == 32) go(int32_t{});
  else go(int64_t{});
  return launched();
}

int32_t tss_gather_rows(int64_t tokens, int64_t top, int64_t d, int32_t dtype, const void *x, const int32_t *row,
                        const int32_t *choice, void *rows, const float *scale, int64_t scale_blocks, float *scale_out,
                        void *stream) {
  const int32_t st = check_tokens(tokens, top, d);
  if (st != TSS_OK) return st;
  const int size = size_of(dtype);
  if (!size) return TSS_E_DTYPE;
  if (scale_blocks < 0 || scale_blocks > INT32_MAX) return TSS_E_ARG;
  if (tokens == 0) return TSS_OK;
  if (!x || !row || !rows || (scale_blocks && (!scale || !scale_out || !choice))) return TSS_E_ARG;
  if (misaligned(x) || misaligned(rows)) return TSS_E_ALIGN;
  const bool wide = d * size % 16 == 0;
  const int64_t pieces = d * size / (wide ? 16 : 8), n = tokens * top;
  const int64_t scale_groups = (n + kRowThreads - 1) / kRowThreads * ((scale_blocks + kScalesTogether - 1) / kScalesTogether);
  const int64_t all = scale_groups + (tokens * pieces + kRowThreads - 1) / kRowThreads;
  if (all > (kMaxThreadsOfLaunch - kRowThreads) / kRowThreads) return TSS_E_ARG;
  Ranges at;
  at.reads(x, tokens * d * size);
  at.reads(row, n * 4);
  at.writes(rows, n * d * size);
  if (scale_blocks) {
    at.reads(choice, n * 4);
    at.reads(scale, scale_blocks * tokens * 4);
    at.writes(scale_out, scale_blocks * n * 4);
  }
  if (at.clash()) return TSS_E_ARG;
  const GatherArgs a{x, rows, row, choice, scale, scale_out, int(tokens), int(top), int(pieces), int(scale_blocks),
                     uint32_t(scale_groups)};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool streamed = n * d * size >= kStreamed && d * size % 64 == 0;
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(uint32_t(all)), dim3(kRowThreads), 0, s, a); };
  if (wide) streamed ? go(gather_rows_kernel<16, true>) : go(gather_rows_kernel<16, false>);
  else go(gather_rows_kernel<8, false>);
  return launched();
}

int32_t tss_combine_rows(int64_t tokens, int64_t top, int64_t d, int32_t dtype, const void *rows, const int32_t *row,
                         const float *weight, int32_t out_dtype, void *y, void *stream) {
  const int32_t st = check_tokens(tokens, top, d);
  if (st != TSS_OK) return st;
  return with_types(dtype, out_dtype, [&](auto r, auto o) -> int32_t {
    if (tokens == 0) return TSS_OK;
    if (!rows || !row || !y) return TSS_E_ARG;
    if (misaligned(rows) || misaligned(y)) return TSS_E_ALIGN;
    const int64_t chunks = d / 8;
    if (tokens * chunks > kMaxThreadsOfLaunch - kRowThreads) return TSS_E_ARG;
    Ranges at;
    at.reads(rows, tokens * top * d * size_of(dtype));
    at.reads(row, tokens * top * 4);
    at.reads(weight, tokens * top * 4);
    at.writes(y, tokens * d * size_of(out_dtype));
    if (at.clash()) return TSS_E_ARG;
    const CombineArgs a{rows, row, weight, y, int(tokens), int(top), int(chunks)};
    hipLaunchKernelGGL((combine_rows_kernel<decltype(r), decltype(o)>),
                       dim3(uint32_t((tokens * chunks + kRowThreads - 1) / kRowThreads)), dim3(kRowThreads), 0,
                       static_cast<hipStream_t>(stream), a);
    return launched();
  });
}

int32_t tss_combine_rows_backward(int64_t tokens, int64_t top, int64_t d, int32_t dtype, const void *dy,
                                  int32_t rows_dtype, const void *rows, const int32_t *row, const float *weight,
                                  void *drows, float *dweight, void *stream) {
  const int32_t st = check_tokens(tokens, top, d);
  if (st != TSS_OK) return st;
  if (d > kMaxD) return TSS_E_UNSUPPORTED;
  if (is_float(dtype) && rows_dtype != dtype && rows_dtype != TSS_F32) return TSS_E_DTYPE;
  return with_types(rows_dtype, dtype, [&](auto r, auto g) -> int32_t {
    using R = decltype(r);
    using D = decltype(g);
    if constexpr (__is_same(D, float) && !__is_same(R, float)) {
      return TSS_E_DTYPE;
    } else {
      if (tokens == 0) return TSS_OK;
      if (!dy || !rows || !row || !weight || !drows || !dweight) return TSS_E_ARG;
      if (misaligned(dy) || misaligned(rows) || misaligned(drows)) return TSS_E_ALIGN;
      const RowShape f = row_shape(d, 1);
      const int lanes = d <= 128 ? 16 : d <= 256 ? 32 : 64;
      const int block = lanes < 64 ? kRowThreads : f.waves * 64, per = lanes < 64 ? kRowThreads / lanes : 1;
      const int64_t groups = (tokens + per - 1) / per;
      if (groups * block > kMaxThreadsOfLaunch) return TSS_E_ARG;
      const int64_t n = tokens * top;
      Ranges at;
      at.reads(dy, tokens * d * sizeof(D));
      at.reads(row, n * 4);
      const uint32_t values = at.reads(rows, n * d * sizeof(R)), weights = at.reads(weight, n * 4);
      at.writes(drows, n * d * sizeof(D), __is_same(D, R) ? values : 0);
      at.writes(dweight, n * 4, weights);
      if (at.clash()) return TSS_E_ARG;
      const CombineBackArgs a{dy, rows, row, weight, drows, dweight, int(tokens), int(top), int(d)};
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(uint32_t(groups)), dim3(block), 0, static_cast<hipStream_t>(stream), a);
      };
      if (lanes == 16) go(combine_backward_kernel<R, D, 1, 16>);
      else if (lanes == 32) go(combine_backward_kernel<R, D, 1, 32>);
      else if (f.chunks == 1) go(combine_backward_kernel<R, D, 1, 64>);
      else if (f.chunks == 2) go(combine_backward_kernel<R, D, 2, 64>);
      else go(combine_backward_kernel<R, D, 4, 64>);
      return launched();
    }
  });
}

}  // extern "C"

// Layer norm of x + residual and its gradients.
//
//   h = x + residual                        (fp32; written rounded to x's type)
//   m = mean(h),  r = 1 / sqrt(mean((h - m)^2) + eps)
//   y = (h - m) r w + b                     (from the fp32 h; x's type, or int8 with a scale for the row)
//
// With xhat = (h - m) r and g = dy w:
//   dx = dh + r (g - mean(g) - xhat mean(g xhat))   (= the residual's gradient)
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// Both are bound by memory: every element is read and written once and stays
// in registers between the row's reductions and its output.  The squares are
// summed about a first mean; the mean's own error, which that second sum
// shows, is taken out again, so that a mean far from zero costs no digits.
// 16384 x 4096, bf16: 50 us (5.3 TB/s; a large copy: 5.1), with residual 99 to 105,
// to int8 60 and 91; backward with dh 107, of which 5 add up dw and db, without 84;
// 300000 x 128, fp16: 29.5 us (5.2 TB/s), to int8 38; one row of 4096: 2.5 us,
// its backward 4.2 (in a graph of such calls on the same operands 3.5).
// 2000 x 32768, bf16: 69 us, to int8 66 (fp16 91: four chunks of a row in 128
// registers, 16 of them spilled; fp32 to int8 115, 20 spilled), backward 364.
#include "ranges.h"
#include "row_launch.h"

using namespace tss;

namespace {

// The sum of n <= 16 slots, to every lane: a lane reads one (in turn, each read would wait for the one before).
__device__ __forceinline__ float sum_slots(const float *slots, int n) {
  const int i = threadIdx.x & 15;
  return sum_lanes<16>(i < n ? slots[i] : 0.0f);
}

// The same for rows of CH chunks a thread.  The widest in turn: their registers
// are full, and what the lanes' sums keep in some more is spilled (2000 x
// 32768, bf16, the gradients: 356 us, by lanes and with several teams' indices 528).
template <int CH>
__device__ __forceinline__ float wave_sums(const float *slots, int n) {
  if constexpr (CH <= 2) {
    return sum_slots(slots, n);
  } else {
    float s = 0;
    for (int i = 0; i < n; ++i) s += slots[i];
    return s;
  }
}

// ---- forward ----

struct NormArgs {
  int rows, d, wpr;
  const void *x, *residual, *weight, *bias;
  float eps;
  void *y;
  float *scale;
  void *h;
  float *mean, *rstd;
};

// A row is held by L neighbouring lanes, or (L == 64) by wpr waves, one row
// per workgroup where wpr > 1; lane t of it holds columns (c * lanes + t) * 8
// .. + 7 for c < CH.  Rows are taken a launch's teams apart: weight and bias
// stay in registers, and the next row's loads are in flight while a row is
// reduced and written.
template <typename T, bool INT8, int CH, int L>
__global__ __launch_bounds__(kMaxThreads) void layer_norm_kernel(NormArgs p) {
  __shared__ float red[2][4][kMaxThreads / 64];
  const int wave = threadIdx.x >> 6, wpr = L == 64 ? p.wpr : 1;
  const int lanes = L * wpr;
  const int t = L < 64 ? threadIdx.x % L : wpr == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int teams = blockDim.x / lanes;
  const int64_t stride = int64_t(gridDim.x) * teams;
  const int d = p.d;
  const T *x = static_cast<const T *>(p.x), *residual = static_cast<const T *>(p.residual);
  const T *weight = static_cast<const T *>(p.weight), *bias = static_cast<const T *>(p.bias);
  auto col_of = [&](int c) __attribute__((always_inline)) { return (c * lanes + t) * 8; };
  int set = 0;
  // two sums over the row; each use its own slots, `slot` and the next, and each row the other set of
  // them: a wave writes the next row's while others may still read this row's
  auto row_sums = [&](float &u, float &v, int slot) __attribute__((always_inline)) {
    u = sum_lanes<L>(u);
    v = sum_lanes<L>(v);
    if (L < 64 || wpr == 1) return;
    if ((threadIdx.x & 63) == 0) {
      red[set][slot][wave] = u;
      red[set][slot + 1][wave] = v;
    }
    __syncthreads();
    u = wave_sums<CH>(red[set][slot], wpr);
    v = wave_sums<CH>(red[set][slot + 1], wpr);
  };

  Raw8<T> xr[CH], rr[CH], wr[CH], br[CH];
  auto load_row = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col_of(c);
      const bool in = col < d && row < p.rows;
      xr[c] = in ? load8(x + row * d + col) : zero8<T>();
      rr[c] = in && residual ? load8(residual + row * d + col) : zero8<T>();
    }
  };
  // The widest rows: there are not enough registers to hold weight and bias, nor the next row.
  constexpr bool kHeld = CH < 4;
  int64_t row = int64_t(blockIdx.x) * teams + threadIdx.x / lanes;
  if constexpr (kHeld) load_row(row);
  auto load_weight = [&](int c) __attribute__((always_inline)) {
    const bool in = col_of(c) < d;
    wr[c] = in ? load8(weight + col_of(c)) : zero8<T>();
    br[c] = in && bias ? load8(bias + col_of(c)) : zero8<T>();
  };
  if constexpr (kHeld)
#pragma unroll
    for (int c = 0; c < CH; ++c) load_weight(c);
  const float inv_d = 1.0f / float(d);
  for (; row < p.rows; row += stride, set ^= 1) {
    const int64_t base = row * d;
    float h[CH][8], sum = 0, none = 0;
    if constexpr (!kHeld) load_row(row);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      widen8(xr[c], h[c]);
      if (residual) {
        float r[8];
        widen8(rr[c], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += h[c][i];
    }
    if constexpr (kHeld) load_row(row + stride);
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (p.h && col_of(c) < d) store8(static_cast<T *>(p.h) + base + col_of(c), h[c]);
    row_sums(sum, none, 0);
    const float mean0 = sum * inv_d;
    float rest = 0, sq = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const bool in = col_of(c) < d;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[c][i] = in ? h[c][i] - mean0 : 0.0f;
        rest += h[c][i];
        sq += h[c][i] * h[c][i];
      }
    }
    row_sums(rest, sq, 2);
    const float off = rest * inv_d;  // the mean of h - mean0: what mean0 lacks
    const float var = fmaxf(sq * inv_d - off * off, 0.0f);
    // a NaN in the row has to come through the max above
    const float r = var == var && off == off ? 1.0f / __builtin_sqrtf(var + p.eps) : off;
    if (t == 0) {
      if (p.mean) p.mean[row] = mean0 + off;
      if (p.rstd) p.rstd[row] = r;
    }
    float amax = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8], b[8];
      if constexpr (!kHeld) load_weight(c);
      widen8(wr[c], w);
      widen8(br[c], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[c][i] = (h[c][i] - off) * r * w[i] + b[i];
        if constexpr (INT8) amax = max_abs(amax, h[c][i]);  // columns past the row: w = b = 0
      }
      if constexpr (!INT8)
        if (col_of(c) < d) store8(static_cast<T *>(p.y) + base + col_of(c), h[c]);
    }
    if constexpr (INT8) {
      amax = max_lanes<L>(amax);
      if (L == 64 && wpr > 1) {
        if ((threadIdx.x & 63) == 0) red[set][0][wave] = amax;  // read before the second sums' barrier
        __syncthreads();
        for (int i = 0; i < wpr; ++i) amax = __builtin_elementwise_maximum(amax, red[set][0][i]);
      }
      const BlockScale<I8> s(amax);
      if (t == 0) p.scale[row] = s.scale;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (col_of(c) < d)
          *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(p.y) + base + col_of(c)) = pack8(h[c], s);
    }
  }
}

template <typename T, bool INT8>
int32_t launch_norm(const NormArgs &a, hipStream_t s) {
  // Few rows: one chunk a thread, a row's latency is all that counts.  Else two.
  const Team f = team_of(a.d, a.rows < 1024 || a.d <= 512 ? 1 : 2);
  const int block = f.waves == 1 ? 256 : f.waves * 64, rpb = f.waves == 1 ? 256 / f.lanes : 1;
  int64_t blocks = (int64_t(a.rows) + rpb - 1) / rpb;
  // Rows of two chunks a thread: as many workgroups as the CUs hold at once, four waves a SIMD of which a
  // workgroup may put one more on the first, and each takes rows in turn (16384 x 4096, bf16: 50.7 us, one
  // row a workgroup 62; 60000 x 520 31 and 44; where some of them wait, 5 waves three times a CU, 7031 x
  // 5120: 43, twice 34).  One chunk: 200000 x 256, bf16 with residual, takes 72 us with a row a team, 76 in turn.
  if (f.chunks > 1) {
    const int waves = block / 64, per_cu = waves < 4 ? 16 / waves : 4 / ((waves + 3) / 4);
    const int64_t most = 256 * (per_cu < 1 ? 1 : per_cu);
    blocks = blocks < most ? blocks : most;
  }
  if (blocks * block > int64_t(UINT32_MAX)) return TSS_E_ARG;  // the launch's thread count is 32 bits
  NormArgs p = a;
  p.wpr = f.waves;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(uint32_t(blocks)), dim3(block), 0, s, p);
  };
  if (f.lanes == 8) go(layer_norm_kernel<T, INT8, 1, 8>);
  else if (f.lanes == 16) go(layer_norm_kernel<T, INT8, 1, 16>);
  else if (f.lanes == 32) go(layer_norm_kernel<T, INT8, 1, 32>);
  else if (f.chunks == 1) go(layer_norm_kernel<T, INT8, 1, 64>);
  else if (f.chunks == 2) go(layer_norm_kernel<T, INT8, 2, 64>);
  else go(layer_norm_kernel<T, INT8, 4, 64>);
  return TSS_OK;
}

// ---- backward ----

struct BackArgs {
  int rows, d, wpr;  // waves of a row
  const void *dy, *h, *weight;
  const float *mean, *rstd;
  const void *dh;
  void *dx;
  float *partial;  // [2][workgroups][d]: shares of dw and of db
};

// dh + r (g w - sg - (x - m) r sx), its fused steps written out, and none with a conversion to fp16 (the
// empty statement): the kernels below give the same bits.
__device__ __forceinline__ float dx_of(float g, float w, float x, float m, float r, float sg, float sx, float dh) {
  float v = __builtin_fmaf(r, __builtin_fmaf(-((x - m) * r), sx, __builtin_fmaf(g, w, -sg)), dh);
  asm("" : "+v"(v));
  return v;
}

constexpr int kNarrowThreads = 256;
constexpr int kTeamWaves = 8;  // of a workgroup of several teams

// Teams of L lanes, or (L == 64) of wpr waves, take a row each, a
// launch's teams apart; a lane keeps its columns' shares of dw and db in
// registers over its rows, a workgroup joins its teams' and writes them to its
// own slice of the workspace (added up in a fixed order afterwards: no
// atomics, the same bits on every run).  D rows' loads are in flight while a
// row is reduced and written; D == 0 (wide rows, whose registers are full with dw and db):
// none are, and the row is read again, from the caches, for its output (8000 x 8200, fp16: 139 us, with
// one row ahead, which spills, 190; with dh).
template <typename T, int CH, int D, int L>
__global__ __launch_bounds__(L == 64 ? kMaxThreads : kNarrowThreads) void layer_norm_backward_kernel(BackArgs p) {
  constexpr bool kNarrow = L < 64;
  __shared__ float red[2][2][kMaxThreads / 64];
  const int wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  constexpr bool kOne = CH > 1;  // one team: known here, because the widest rows have no register to spare
  const int wpr = kNarrow ? 1 : p.wpr, lanes = kNarrow ? L : wpr * 64, t = kOne ? threadIdx.x : threadIdx.x % lanes;
  const int teams = kNarrow ? kNarrowThreads / L : kOne ? 1 : nw / wpr, team = kOne ? 0 : threadIdx.x / lanes;
  const int stride = gridDim.x * teams;
  const int rows = p.rows, d = p.d;
  const T *dy = static_cast<const T *>(p.dy), *hh = static_cast<const T *>(p.h), *dh = static_cast<const T *>(p.dh);
  T *dx = static_cast<T *>(p.dx);
  auto col_of = [&](int c) __attribute__((always_inline)) { return (c * lanes + t) * 8; };
  Raw8<T> weight[CH];
  float dw[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    weight[c] = col_of(c) < d ? load8(static_cast<const T *>(p.weight) + col_of(c)) : zero8<T>();
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0;
  }
  constexpr int S = D ? D : 1;
  Raw8<T> a[S][CH], b[S][CH], e[S][CH];
  // keeps the compiler from holding several chunks' values in fp32 over the loop
  auto opaque = [](Raw8<T> &v) __attribute__((always_inline)) {
    if constexpr (CH > 1)
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i) asm("" : "+v"(v.v[i]));
  };
  float mean[S], rstd[S];
  auto load_row = [&](int s, int64_t row) __attribute__((always_inline)) {
    const int64_t base = row * d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col_of(c);
      const bool in = col < d && row < rows;
      a[s][c] = in ? load8(dy + base + col) : zero8<T>();
      b[s][c] = in ? load8(hh + base + col) : zero8<T>();
      e[s][c] = in && dh ? load8(dh + base + col) : zero8<T>();
    }
    mean[s] = row < rows ? p.mean[row] : 0.0f;
    rstd[s] = row < rows ? p.rstd[row] : 0.0f;
  };
#pragma unroll
  for (int s = 0; s < D; ++s) load_row(s, int64_t(blockIdx.x) * teams + team + int64_t(s) * stride);
  const float inv_d = 1.0f / float(d);
  int slot = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * teams; row0 < rows; row0 += int64_t(S) * stride) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int64_t row = row0 + team + int64_t(s) * stride;
      if ((kNarrow ? row : row - team) >= rows) break;  // teams that meet at the barrier go on together
      Raw8<T> ca[CH], cb[CH], ce[CH];
      if constexpr (D > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          ca[c] = a[s][c];
          cb[c] = b[s][c];
          ce[c] = e[s][c];
        }
      } else {
        mean[0] = p.mean[row];
        rstd[0] = p.rstd[row];
      }
      const float m = mean[s], r = rstd[s];
      if constexpr (D > 0) load_row(s, row + int64_t(D) * stride);
      float sg = 0, sx = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float g[8], x[8], w[8];
        if constexpr (D > 0) {
          widen8(ca[c], g);
          widen8(cb[c], x);
        } else {
          if constexpr (CH > 2) asm volatile("" ::: "memory");  // one chunk's registers at a time
          const bool in = col_of(c) < d;
          widen8(in ? load8(dy + row * d + col_of(c)) : zero8<T>(), g);
          widen8(in ? load8(hh + row * d + col_of(c)) : zero8<T>(), x);
        }
        opaque(weight[c]);
        widen8(weight[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // columns past the row: g = w = 0
          const float gx = (x[i] - m) * r * g[i];
          dw[c][i] += gx;
          db[c][i] += g[i];
          sg = __builtin_fmaf(g[i], w[i], sg);
          sx = __builtin_fmaf(gx, w[i], sx);
        }
      }
      sg = sum_lanes<L>(sg);
      sx = sum_lanes<L>(sx);
      if (!kNarrow && wpr > 1) {
        // two sets of slots: a wave writes the next row's while others may still read this row's
        if ((threadIdx.x & 63) == 0) {
          red[slot][0][wave] = sg;
          red[slot][1][wave] = sx;
        }
        __syncthreads();
        sg = wave_sums<CH>(&red[slot][0][team * wpr], wpr);
        sx = wave_sums<CH>(&red[slot][1][team * wpr], wpr);
        slot ^= 1;
      }
      sg *= inv_d;
      sx *= inv_d;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = col_of(c);
        if (col >= d || (!kOne && row >= rows)) continue;
        float g[8], x[8], o[8], w[8];
        if constexpr (D > 0) {
          opaque(ca[c]);
          opaque(cb[c]);
          widen8(ca[c], g);
          widen8(cb[c], x);
          widen8(ce[c], o);
        } else {
          widen8(load8(dy + row * d + col), g);
          widen8(load8(hh + row * d + col), x);
          widen8(dh ? load8(dh + row * d + col) : zero8<T>(), o);
        }
        opaque(weight[c]);
        widen8(weight[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = dx_of(g[i], w[i], x[i], m, r, sg, sx, o[i]);
        store8(dx + row * d + col, o);
        if constexpr (CH > 2) asm volatile("" ::: "memory");
      }
    }
  }
  float *pw = p.partial + int64_t(blockIdx.x) * d, *pb = pw + int64_t(gridDim.x) * d;
  if constexpr (kNarrow) {
    // the lanes of a wave that hold the same columns, then the waves in order
    __shared__ float join[2][kNarrowThreads / 64][L * 8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int k = L; k < 64; k *= 2) {
        dw[0][i] += __shfl_xor(dw[0][i], k);
        db[0][i] += __shfl_xor(db[0][i], k);
      }
      if ((threadIdx.x & 63) < L) {
        join[0][wave][t * 8 + i] = dw[0][i];
        join[1][wave][t * 8 + i] = db[0][i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += kNarrowThreads) {
      float vw = 0, vb = 0;
#pragma unroll
      for (int i = 0; i < kNarrowThreads / 64; ++i) {
        vw += join[0][i][c];
        vb += join[1][i][c];
      }
      pw[c] = vw;
      pb[c] = vb;
    }
  } else if (CH == 1 && teams > 1) {
    extern __shared__ float join_teams[];  // [team][8 columns of each lane]
#pragma unroll
    for (int of = 0; of < 2; ++of) {
      store8(join_teams + threadIdx.x * 8, of ? db[0] : dw[0]);
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += blockDim.x) {
        float v = 0;
        for (int i = 0; i < teams; ++i) v += join_teams[i * lanes * 8 + c];
        (of ? pb : pw)[c] = v;
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (col_of(c) < d) {
        store8(pw + col_of(c), dw[c]);
        store8(pb + col_of(c), db[c]);
      }
  }
}

// Few elements: one launch, whose first workgroups take 8 L columns each over all rows, for
// dw and db, and the others the rows, W waves each (CH > 1: a workgroup each), for dx.  They share
// nothing, so dy and h are read twice, the second time from the caches.
constexpr int kFewThreads = 1024;
template <typename T>
constexpr int kRowsTogether = 8 / sizeof(T);  // rows whose loads a thread has in flight
template <typename T, int W, int CH, int L>
__global__ __launch_bounds__(kFewThreads) void layer_norm_backward_few_kernel(BackArgs p, int column_groups, float *dweight,
                                                                              float *dbias) {
  constexpr int kWaves = kFewThreads / 64, kTogether = kRowsTogether<T>;
  const int wave = threadIdx.x >> 6, nw = CH > 1 ? blockDim.x >> 6 : kWaves, rows = p.rows, d = p.d;
  const T *dy = static_cast<const T *>(p.dy), *hh = static_cast<const T *>(p.h), *dh = static_cast<const T *>(p.dh);
  if (int(blockIdx.x) < column_groups) {
    __shared__ float join[2][kWaves][L * 8];
    const int l = threadIdx.x % L, col = (blockIdx.x * L + l) * 8;
    float dw[8] = {0, 0, 0, 0, 0, 0, 0, 0}, db[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int row0 = threadIdx.x / L; row0 < rows; row0 += kTogether * (nw * 64 / L)) {
      Raw8<T> a[kTogether], b[kTogether];
      float m[kTogether], r[kTogether];
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        const int row = row0 + u * (nw * 64 / L);
        const bool in = row < rows && col < d;
        a[u] = in ? load8(dy + int64_t(row) * d + col) : zero8<T>();
        b[u] = in ? load8(hh + int64_t(row) * d + col) : zero8<T>();
        m[u] = in ? p.mean[row] : 0.0f;
        r[u] = in ? p.rstd[row] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        float g[8], x[8];
        widen8(a[u], g);
        widen8(b[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[i] += (x[i] - m[u]) * r[u] * g[i];
          db[i] += g[i];
        }
      }
    }
    // the lanes of a wave that hold the same columns, then the waves in order
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int k = L; k < 64; k *= 2) {
        dw[i] += __shfl_xor(dw[i], k);
        db[i] += __shfl_xor(db[i], k);
      }
      if ((threadIdx.x & 63) < L) {
        join[0][wave][l * 8 + i] = dw[i];
        join[1][wave][l * 8 + i] = db[i];
      }
    }
    __syncthreads();
    constexpr int columns = L * 8;
    const int c = threadIdx.x % columns, of = threadIdx.x / columns, at = blockIdx.x * columns + c;
    float *out = of == 0 ? dweight : dbias;
    if (of > 1 || !out || at >= d) return;
    float v = 0;
    for (int i = 0; i < nw; ++i) v += join[of][i][c];
    out[at] = v;
    return;
  }
  __shared__ float red[2][kWaves];
  const int wpr = CH > 1 ? nw : W, team = wave / wpr, t = threadIdx.x - team * wpr * 64;
  const int row = (int(blockIdx.x) - column_groups) * (nw / wpr) + team;
  auto col_of = [&](int c) __attribute__((always_inline)) { return (c * wpr * 64 + t) * 8; };
  const int64_t base = int64_t(row) * d;
  Raw8<T> a[CH], b[CH], e[CH], weight[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = col_of(c);
    const bool in = row < rows && col < d;
    a[c] = in ? load8(dy + base + col) : zero8<T>();
    b[c] = in ? load8(hh + base + col) : zero8<T>();
    e[c] = in && dh ? load8(dh + base + col) : zero8<T>();
    weight[c] = in ? load8(static_cast<const T *>(p.weight) + col) : zero8<T>();
  }
  const float m = row < rows ? p.mean[row] : 0.0f, r = row < rows ? p.rstd[row] : 0.0f, inv_d = 1.0f / float(d);
  float sg = 0, sx = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float g[8], x[8], w[8];
    widen8(a[c], g);
    widen8(b[c], x);
    widen8(weight[c], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // columns past the row: g = w = 0
      const float gx = (x[i] - m) * r * g[i];
      sg = __builtin_fmaf(g[i], w[i], sg);
      sx = __builtin_fmaf(gx, w[i], sx);
    }
  }
  sg = sum_lanes<64>(sg);
  sx = sum_lanes<64>(sx);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) {
      red[0][wave] = sg;
      red[1][wave] = sx;
    }
    __syncthreads();
    sg = sum_slots(&red[0][team * wpr], wpr);
    sx = sum_slots(&red[1][team * wpr], wpr);
  }
  sg *= inv_d;
  sx *= inv_d;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (row >= rows || col_of(c) >= d) continue;
    float g[8], x[8], o[8], w[8];
    widen8(a[c], g);
    widen8(b[c], x);
    widen8(e[c], o);
    widen8(weight[c], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = dx_of(g[i], w[i], x[i], m, r, sg, sx, o[i]);
    store8(static_cast<T *>(p.dx) + base + col_of(c), o);
  }
}

// Rows that a workgroup takes at a time.
int64_t backward_teams(const Team &f) {
  return f.lanes < 64 ? kNarrowThreads / f.lanes : f.waves < kTeamWaves ? kTeamWaves / f.waves : 1;
}

// Workgroups of the backward pass: two a CU (narrow rows: four; fp32 rows in
// teams: one, whose loads are twice the bytes), but each adds 16 bytes a column
// (its shares of dw and db, written and read) to the 8 a column that a row of
// 16-bit elements moves, so no more than one for every 8 turns where that still
// gives every CU one.  With dh: 100000 x 512, bf16: 83 us, 60000 x 1024 100, by one
// workgroup a CU 80 and 104, by four 84 and 106, and by more of one row each,
// without teams, 87 and 107; 200000 x 264 86 (128 without); fp32 100000 x 512
// 152, by two workgroups 164.  Without dh: 64, 77, 80 and 115.
int64_t backward_blocks(int64_t rows, int64_t d, int64_t size) {
  constexpr int64_t cus = 256;
  const Team f = team_of(d, 1);
  const int64_t teams = backward_teams(f), fill = cus * (f.lanes < 64 ? 4 : teams > 1 && size == 4 ? 1 : 2);
  const int64_t turns = (rows + teams - 1) / teams;
  const int64_t n = turns / 8 < cus ? cus : turns / 8 > fill ? fill : turns / 8;
  return turns < n ? turns : n;
}

// The columns' workgroups take 4 us and 2 more for 1000 rows; rows of more bytes in all keep the CUs busy in
// two launches too (us in a graph of such calls on the same operands, with dh, one launch and two; bf16 256 x 4096: 5.3 and 10.9; 1000 x 1024 6.4 and 9.5, 8192 17.9
// and 21.0; 2000 x 128 8.6 and 8.1; fp32 1000 x 4096: 17.9 and 18.5, 8192 34 and 30; 500 x 16384 42.0 and 41.5).
bool few(int64_t rows, int64_t d, int64_t size) {
  return rows <= 1024 && d <= kFewThreads * 16 && rows * d * size <= int64_t(1) << 24;
}

template <typename T, int L>
void launch_few(const BackArgs &a, float *dweight, float *dbias, hipStream_t s) {
  const Team f = team_of(a.d, 1);
  const int columns = (a.d / 8 + L - 1) / L;
  auto go = [&](auto kernel, int rows, int threads) {  // rows of a workgroup
    hipLaunchKernelGGL(kernel, dim3(uint32_t(columns + (a.rows + rows - 1) / rows)), dim3(threads), 0, s, a, columns,
                       dweight, dbias);
  };
  if (a.d <= 512) go(layer_norm_backward_few_kernel<T, 1, 1, L>, 16, kFewThreads);
  else if (a.d <= 2048) go(layer_norm_backward_few_kernel<T, 4, 1, L>, 4, kFewThreads);
  else if (f.chunks == 1) go(layer_norm_backward_few_kernel<T, 16, 1, L>, 1, kFewThreads);
  else go(layer_norm_backward_few_kernel<T, 16, 2, L>, 1, f.waves * 64);
}

// Columns of a workgroup: 128 bytes, which makes the most of the CUs; up to 64
// rows 256 columns, fewer workgroups (in a graph, as above: 64 x 16384, bf16: 4.7
// us, fp32 1 x 16384 4.7 and by 32 columns 11.5).
template <typename T>
void launch_few(const BackArgs &a, float *dweight, float *dbias, hipStream_t s) {
  if (a.rows <= 64) launch_few<T, 32>(a, dweight, dbias, s);
  else launch_few<T, 16 / sizeof(T)>(a, dweight, dbias, s);
}

template <typename T>
void launch_backward(const BackArgs &a, hipStream_t s) {
  const Team f = team_of(a.d, 1);
  // One row ahead: two rows' registers leave room for fewer waves (300000 x 128,
  // bf16, with dh: 65 us, two ahead 68; 16384 x 4096, fp32: 199 and 249; bf16 107 and 110).
  const dim3 grid(uint32_t(backward_blocks(a.rows, a.d, sizeof(T)))), block(f.lanes < 64 ? kNarrowThreads : backward_teams(f) * f.waves * 64);
  const int lds = f.lanes == 64 && backward_teams(f) > 1 ? int(block.x) * 32 : 0;  // to join the teams' sums
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, lds, s, a); };
  if (f.lanes == 8) go(layer_norm_backward_kernel<T, 1, 1, 8>);
  else if (f.lanes == 16) go(layer_norm_backward_kernel<T, 1, 1, 16>);
  else if (f.lanes == 32) go(layer_norm_backward_kernel<T, 1, 1, 32>);
  else if (f.chunks == 1) go(layer_norm_backward_kernel<T, 1, 1, 64>);
  else if (f.chunks == 2) go(layer_norm_backward_kernel<T, 2, 0, 64>);
  else go(layer_norm_backward_kernel<T, 4, 0, 64>);
}

}  // namespace

extern "C" {

int32_t tss_layer_norm(int64_t rows, int64_t d, int32_t dtype, const void *x, const void *residual, const void *weight,
                       const void *bias, float eps, int32_t out_dtype, void *y, float *scale, void *residual_out,
                       float *mean, float *rstd, void *stream) {
  int32_t st = check_rows(rows, d, dtype, INT32_MAX);
  if (st != TSS_OK) return st;
  if (out_dtype != dtype && out_dtype != TSS_I8) return TSS_E_DTYPE;
  if (!(eps >= 0)) return TSS_E_ARG;
  if (rows == 0) return TSS_OK;
  if (!x || !weight || !y || (out_dtype == TSS_I8 && !scale)) return TSS_E_ARG;
  if (misaligned(x) || misaligned(residual) || misaligned(weight) || misaligned(bias) || misaligned(y) ||
      misaligned(residual_out))
    return TSS_E_ALIGN;
  const int64_t size = dtype == TSS_F32 ? 4 : 2, bytes = rows * d * size;
  Ranges at;
  const uint32_t inputs = at.reads(x, bytes) | at.reads(residual, bytes);
  at.reads(weight, d * size);
  at.reads(bias, d * size);
  if (out_dtype == TSS_I8) {
    at.writes(y, rows * d);
    at.writes(scale, rows * 4);
  } else {
    at.writes(y, bytes, inputs);
  }
  at.writes(residual_out, bytes, inputs);
  at.writes(mean, rows * 4);
  at.writes(rstd, rows * 4);
  if (at.clash()) return TSS_E_ARG;
  const NormArgs a{int(rows), int(d), 1, x, residual, weight, bias, eps, y, scale, residual_out, mean, rstd};
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto t) {
    using T = decltype(t);
    st = out_dtype == TSS_I8 ? launch_norm<T, true>(a, s) : launch_norm<T, false>(a, s);
  };
  if (dtype == TSS_F16) go(_Float16{});
  else if (dtype == TSS_BF16) go(__bf16{});
  else go(float{});
  if (st != TSS_OK) return st;
  return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
}

int64_t tss_layer_norm_backward_workspace_size(int64_t rows, int64_t d) {
  const int32_t st = check_rows(rows, d, TSS_F32, INT32_MAX);
  return st != TSS_OK ? st : backward_blocks(rows, d, 2) * d * 8;  // fp32 takes no more
}

int32_t tss_layer_norm_backward(int64_t rows, int64_t d, int32_t dtype, const void *dy, const void *h,
                                const void *weight, const float *mean, const float *rstd, const void *dh, void *dx,
                                float *dweight, float *dbias, void *workspace, int64_t workspace_bytes, void *stream) {
  const int32_t st = check_rows(rows, d, dtype, INT32_MAX);
  if (st != TSS_OK) return st;
  if (!dweight) return TSS_E_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) {
    for (float *out : {dweight, dbias})
      if (out) launch_zero_f32(d, out, s);
    return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
  }
  if (!dy || !h || !weight || !mean || !rstd || !dx) return TSS_E_ARG;
  if (!workspace || workspace_bytes < tss_layer_norm_backward_workspace_size(rows, d)) return TSS_E_ARG;
  if (misaligned(dy) || misaligned(h) || misaligned(weight) || misaligned(dh) || misaligned(dx) ||
      misaligned(workspace))
    return TSS_E_ALIGN;
  const int64_t size = dtype == TSS_F32 ? 4 : 2, bytes = rows * d * size;
  Ranges at;
  const uint32_t inputs = at.reads(dy, bytes) | at.reads(h, bytes) | at.reads(dh, bytes);
  at.reads(weight, d * size);
  at.reads(mean, rows * 4);
  at.reads(rstd, rows * 4);
  at.writes(dx, bytes, inputs);
  at.writes(dweight, d * 4);
  at.writes(dbias, d * 4);
  at.writes(workspace, tss_layer_norm_backward_workspace_size(rows, d));
  if (at.clash()) return TSS_E_ARG;
  float *partial = static_cast<float *>(workspace);
  const BackArgs a{int(rows), int(d), team_of(d, 1).waves, dy, h, weight, mean, rstd, dh, dx, partial};
  if (few(rows, d, size) && dx != dy && dx != h) {  // over dy or h: what one workgroup writes another may still have to read
    if (dtype == TSS_F16) launch_few<_Float16>(a, dweight, dbias, s);
    else if (dtype == TSS_BF16) launch_few<__bf16>(a, dweight, dbias, s);
    else launch_few<float>(a, dweight, dbias, s);
    return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
  }
  if (dtype == TSS_F16) launch_backward<_Float16>(a, s);
  else if (dtype == TSS_BF16) launch_backward<__bf16>(a, s);
  else launch_backward<float>(a, s);
  launch_column_sums(backward_blocks(rows, d, size), d, partial, dweight, dbias, s);
  return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
}

}  // extern "C"

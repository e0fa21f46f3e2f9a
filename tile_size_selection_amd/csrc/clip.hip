// The norm over many tensors, and the tensors scaled to at most a given norm:
//
//   norm = sqrt(sum of all elements' squares),  out = g * min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: every element is read for the norm, and read again and
// written to be scaled.  Squares are added in 64 bits: their sum neither
// overflows nor loses what many elements add to few, and the rate of 64-bit
// FMAs is far above memory's.  The elements are dealt evenly to the workgroups,
// wherever tensors begin and end; the workgroups' sums are added in a fixed
// order by every workgroup that scales (the same bits on every run, and one
// launch fewer than with a pass of its own).
// 226505854 elements in 60 tensors, fp32 and bf16: 352 us, 110 of it the norm's
// pass (5.6 TB/s); the outputs pass the caches by (through them 379).
// The tensors' addresses travel in the kernel's arguments, kTable at a time:
// no copy from host memory, so a captured graph holds all that it needs.  Every
// workgroup that scales reads the sums of all tables, which costs more than the
// elements where there are many tables: n tensors of 100000 bf16 elements, in
// place, kernels only: n = 128 24 us, 256 50, 512 122, 1000 323, 2000 907, 4000
// 2755 (their bytes at a large copy's rate: 15, 30, 60, 117, 234, 468).
// Tensors off 16-byte borders are taken element by element: 2^26 bf16 elements
// 140 us, on a border 84; fp32 166 and 135.
#include <algorithm>
#include <new>
#include <vector>

#include "row_launch.h"

using namespace tss;

namespace {

constexpr int kTable = 128, kSmallTable = 16;
constexpr int kClipThreads = 256;
constexpr int kUnit = kClipThreads * 8;     // elements; a tensor's last unit may be short
constexpr uint32_t kClipGroups = 2048;      // eight workgroups a CU
constexpr int kTogether = 2;                // loads a thread has in flight
constexpr int64_t kStreamed = int64_t(1) << 28;  // bytes of output from which on it passes the caches by
constexpr float kNormEps = 1e-6f;

// N: kTable, or kSmallTable where that holds all tensors: its launches cost the
// host 0.5 us less each (12 tensors of 24000 elements: 6.7 us a call, 7.2).
template <int N>
struct ClipTable {
  const void *in[N];
  void *out[N];
  int64_t n[N];
  uint32_t first[N + 1];  // a tensor's first unit, in this table
  uint8_t type[N];
  int32_t count;
  uint32_t base;               // the table's first sum among all
};
static_assert(sizeof(ClipTable<kTable>) <= 3840, "kernel arguments are 4 KiB");

// The tensor that unit `at` of the table belongs to (uniform over the workgroup).
template <int K>
__device__ __forceinline__ int tensor_of(const ClipTable<K> &t, uint32_t at) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= at) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double sum64d(double v) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// Sum over the workgroup of N threads, to every thread; red: one slot a wave.
template <int N>
__device__ __forceinline__ double group_sum(double v, double *red) {
  v = sum64d(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int i = 0; i < N / 64; ++i) s += red[i];
  return s;
}

template <int N, typename T>
__device__ __forceinline__ double piece_squares(const T *g, int thread, int64_t from, int64_t end, bool wide) {
  double s = 0;
  if (wide) {
    const int64_t whole = from + (end - from) / 8 * 8;
    int64_t i = from + thread * 8;
    for (; i + (kTogether - 1) * N * 8 < whole; i += kTogether * N * 8) {
      Raw8<T> r[kTogether];
#pragma unroll
      for (int u = 0; u < kTogether; ++u) r[u] = load8(g + i + u * N * 8);
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        float f[8];
        widen8(r[u], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = __builtin_fma(double(f[k]), double(f[k]), s);
      }
    }
    for (; i < whole; i += N * 8) {
      float f[8];
      widen8(load8(g + i), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) s = __builtin_fma(double(f[k]), double(f[k]), s);
    }
    from = whole;
  }
  for (int64_t i = from + thread; i < end; i += N) {
    const double f = double(float(g[i]));
    s = __builtin_fma(f, f, s);
  }
  return s;
}

// STREAMED: the output passes the caches by (a template argument: stores of
// both kinds behind a test are made one of the plain kind).
template <int N, bool STREAMED, typename T>
__device__ __forceinline__ void piece_scale(const T *g, T *out, int thread, int64_t from, int64_t end, bool wide, float factor) {
  if (wide) {
    const int64_t whole = from + (end - from) / 8 * 8;
    int64_t i = from + thread * 8;
    for (; i + (kTogether - 1) * N * 8 < whole; i += kTogether * N * 8) {
      Raw8<T> r[kTogether];
#pragma unroll
      for (int u = 0; u < kTogether; ++u) r[u] = load8(g + i + u * N * 8);
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        float f[8];
        widen8(r[u], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= factor;
        if constexpr (STREAMED) store8_streamed(out + i + u * N * 8, f);
        else store8(out + i + u * N * 8, f);
      }
    }
    for (; i < whole; i += N * 8) {
      float f[8];
      widen8(load8(g + i), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= factor;
      store8(out + i, f);
    }
    from = whole;
  }
  for (int64_t i = from + thread; i < end; i += N) out[i] = (T)(float(g[i]) * factor);
}

// f(element type, tensor's index, first element, end) of each tensor in the
// range of group `group` of `groups` (a workgroup, or a wave).
template <int K, typename F>
__device__ __forceinline__ void with_range(const ClipTable<K> &t, uint32_t group, uint32_t groups, F f) {
  const uint64_t units = t.first[t.count];
  uint32_t at = uint32_t(units * group / groups);
  const uint32_t end = uint32_t(units * (group + 1) / groups);
  for (int k = tensor_of(t, at); at < end; ++k) {
    const uint32_t upto = min(end, t.first[k + 1]);
    const int64_t from = int64_t(at - t.first[k]) * kUnit, to = min(t.n[k], int64_t(upto - t.first[k]) * kUnit);
    if (t.type[k] == TSS_F32) f(float{}, k, from, to);
    else if (t.type[k] == TSS_F16) f(_Float16{}, k, from, to);
    else f(__bf16{}, k, from, to);
    at = upto;
  }
}

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int K>
__global__ __launch_bounds__(kClipThreads) void clip_squares_kernel(ClipTable<K> t, double *partial) {
  __shared__ double red[kClipThreads / 64];
  double s = 0;
  with_range(t, blockIdx.x, gridDim.x, [&](auto v, int k, int64_t from, int64_t end) {
    using T = decltype(v);
    s += piece_squares<kClipThreads>(static_cast<const T *>(t.in[k]), threadIdx.x, from, end, aligned16(t.in[k]));
  });
  s = group_sum<kClipThreads>(s, red);
  if (threadIdx.x == 0) partial[t.base + blockIdx.x] = s;
}

// All workgroups' sums, in a fixed order.
__device__ __forceinline__ double total_squares(const double *partial, uint32_t sums, double *red) {
  double s = 0;
  for (uint32_t i = threadIdx.x; i < sums; i += kClipThreads) s += partial[i];
  return group_sum<kClipThreads>(s, red);
}

__global__ __launch_bounds__(kClipThreads) void clip_norm_kernel(const double *partial, uint32_t sums, float *norm) {
  __shared__ double red[kClipThreads / 64];
  const double s = total_squares(partial, sums, red);
  if (threadIdx.x == 0) *norm = float(sqrt(s));
}

__device__ __forceinline__ float clip_factor(double norm, float max_norm) {
  const double q = double(max_norm) / (norm + double(kNormEps));
  return q > 1 ? 1.0f : float(q);  // a NaN comes through
}

template <int K, bool STREAMED>
__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipTable<K> t, const double *partial, uint32_t sums,
                                                                  float max_norm, float *norm) {
  __shared__ double red[kClipThreads / 64];
  const double n = sqrt(total_squares(partial, sums, red));
  if (t.base == 0 && blockIdx.x == 0 && threadIdx.x == 0) *norm = float(n);
  const float factor = clip_factor(n, max_norm);
  // The table's last elements first: of a single table, the norm's pass has left them in the caches.
  with_range(t, gridDim.x - 1 - blockIdx.x, gridDim.x, [&](auto v, int k, int64_t from, int64_t end) {
    using T = decltype(v);
    if (factor == 1.0f && t.out[k] == t.in[k]) return;
    piece_scale<kClipThreads, STREAMED>(static_cast<const T *>(t.in[k]), static_cast<T *>(t.out[k]), threadIdx.x, from, end,
                aligned16(t.in[k]) && aligned16(t.out[k]), factor);
  });
}

// Few elements: one workgroup adds and scales all of them, dealt evenly to its
// waves (12 tensors of 30000 elements in all: 6.8 us a call, by two launches 10.5;
// 60000: 10.8 and 9.3).
constexpr int kOneThreads = 1024;
constexpr uint32_t kOneUnits = 20;

template <int K>
__global__ __launch_bounds__(kOneThreads) void clip_one_kernel(ClipTable<K> t, bool scale, float max_norm, float *norm) {
  __shared__ double red[kOneThreads / 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double s = 0;
  with_range(t, wave, kOneThreads / 64, [&](auto v, int k, int64_t from, int64_t end) {
    using T = decltype(v);
    s += piece_squares<64>(static_cast<const T *>(t.in[k]), lane, from, end, aligned16(t.in[k]));
  });
  const double n = sqrt(group_sum<kOneThreads>(s, red));
  if (threadIdx.x == 0) *norm = float(n);
  if (!scale) return;
  const float factor = clip_factor(n, max_norm);
  with_range(t, wave, kOneThreads / 64, [&](auto v, int k, int64_t from, int64_t end) {
    using T = decltype(v);
    if (factor == 1.0f && t.out[k] == t.in[k]) return;
    piece_scale<64, false>(static_cast<const T *>(t.in[k]), static_cast<T *>(t.out[k]), lane, from, end,
                           aligned16(t.in[k]) && aligned16(t.out[k]), factor);
  });
}

int bytes_of(int32_t dtype) { return dtype == TSS_F32 ? 4 : dtype == TSS_F16 || dtype == TSS_BF16 ? 2 : 0; }

constexpr int64_t kMostElements = int64_t(1) << 40;

uint32_t groups_of(uint32_t units) { return units < kClipGroups ? units : kClipGroups; }

// Workgroups' sums over all tables, and the tables.
struct Sums {
  int64_t sums = 0, tables = 0, units = 0;
  bool one() const { return tables == 1 && units <= kOneUnits; }  // a single workgroup, which needs no workspace
};

// Calls f(first tensor, one past the last, units) for the tables: kTable tensors that are not empty, or the last of them.
template <typename F>
int32_t each_table(int64_t n, const int64_t *sizes, F f) {
  if (n < 0 || n > INT32_MAX || (n > 0 && !sizes)) return TSS_E_ARG;
  int64_t total = 0, begin = 0, units = 0;
  int count = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (sizes[i] < 0 || sizes[i] > kMostElements || (total += sizes[i]) > kMostElements) return TSS_E_ARG;
    if (sizes[i] > 0) {
      ++count;
      units += (sizes[i] + kUnit - 1) / kUnit;
    }
    if (count == kTable || (i == n - 1 && count)) {
      f(begin, i + 1, uint32_t(units));
      begin = i + 1;
      units = count = 0;
    }
  }
  return TSS_OK;
}

int32_t count_sums(int64_t n, const int64_t *sizes, Sums *out) {
  Sums c;
  const int32_t st = each_table(n, sizes, [&](int64_t, int64_t, uint32_t units) {
    c.sums += groups_of(units);
    c.units += units;
    ++c.tables;
  });
  *out = c;
  return st;
}

// Whether `bytes` at p overlap a tensor that is read or written.
bool touches(const void *p, int64_t bytes, int64_t n, const void *const *in, void *const *out, const int64_t *sizes,
             const int32_t *types) {
  const uintptr_t begin = reinterpret_cast<uintptr_t>(p), end = begin + uintptr_t(bytes);
  for (int64_t i = 0; i < n; ++i) {
    const uintptr_t length = uintptr_t(sizes[i]) * bytes_of(types[i]);
    for (const void *q : {in[i], out ? static_cast<const void *>(out[i]) : in[i]}) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(q);
      if (begin < end && length && begin < at + length && at < end) return true;
    }
  }
  return false;
}

// An output may be its own input; apart from that no output overlaps another
// output or an input, nor does the norm's place.
bool overlapping(int64_t n, const void *const *in, void *const *out, const int64_t *sizes, const int32_t *types,
                 const float *norm) {
  struct Span {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Span> spans;
  spans.reserve(size_t(2 * n + 1));
  spans.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm + 1), true});
  for (int64_t i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    const uintptr_t bytes = uintptr_t(sizes[i]) * bytes_of(types[i]);
    const uintptr_t a = reinterpret_cast<uintptr_t>(in[i]), b = reinterpret_cast<uintptr_t>(out[i]);
    spans.push_back({b, b + bytes, true});
    if (a != b) spans.push_back({a, a + bytes, false});
  }
  std::sort(spans.begin(), spans.end(), [](const Span &a, const Span &b) { return a.begin < b.begin; });
  uintptr_t written = 0, read = 0;  // the furthest ends so far
  for (const Span &s : spans) {
    if (s.begin < written || (s.written && s.begin < read)) return true;
    (s.written ? written : read) = std::max(s.written ? written : read, s.end);
  }
  return false;
}

// The launches of checked arguments.
template <int K>
int32_t launch_clip(int64_t n, const void *const *grads, const int64_t *sizes, const int32_t *dtypes, float max_norm,
                    void *const *out, float *norm, double *partial, const Sums &c, int64_t bytes, hipStream_t s) {
  const int64_t sums = c.sums;
  // launch(table, its workgroups) for each table
  auto tables = [&](auto launch) {
    ClipTable<K> t{};
    each_table(n, sizes, [&](int64_t begin, int64_t end, uint32_t units) {
      t.count = 0;
      for (int64_t i = begin; i < end; ++i) {
        if (sizes[i] == 0) continue;
        const int k = t.count++;
        t.in[k] = grads[i];
        t.out[k] = out ? out[i] : nullptr;
        t.n[k] = sizes[i];
        t.type[k] = uint8_t(dtypes[i]);
        t.first[k + 1] = t.first[k] + uint32_t((sizes[i] + kUnit - 1) / kUnit);
      }
      launch(t, groups_of(units));
      t.base += groups_of(units);
    });
  };
  if (c.one()) {
    tables([&](const ClipTable<K> &t, uint32_t) {
      hipLaunchKernelGGL(clip_one_kernel<K>, dim3(1), dim3(kOneThreads), 0, s, t, out != nullptr, max_norm, norm);
    });
    return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
  }
  tables([&](const ClipTable<K> &t, uint32_t groups) {
    hipLaunchKernelGGL(clip_squares_kernel<K>, dim3(groups), dim3(kClipThreads), 0, s, t, partial);
  });
  if (!out || sums == 0) {
    hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(kClipThreads), 0, s, partial, uint32_t(sums), norm);
  } else {
    tables([&](const ClipTable<K> &t, uint32_t groups) {
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(groups), dim3(kClipThreads), 0, s, t, partial, uint32_t(sums), max_norm, norm);
      };
      bytes >= kStreamed ? go(clip_scale_kernel<K, true>) : go(clip_scale_kernel<K, false>);
    });
  }
  return hipGetLastError() == hipSuccess ? TSS_OK : TSS_E_HIP;
}

int32_t clip(int64_t n, const void *const *grads, const int64_t *sizes, const int32_t *dtypes, float max_norm,
             void *const *out, float *norm, void *workspace, int64_t workspace_bytes, hipStream_t s) {
  Sums c;
  const int32_t st = count_sums(n, sizes, &c);
  if (st != TSS_OK) return st;
  if (!norm || (n > 0 && (!grads || !dtypes))) return TSS_E_ARG;
  if (out && !(max_norm >= 0)) return TSS_E_ARG;
  int64_t bytes = 0, tensors = 0;  // that are not empty
  for (int64_t i = 0; i < n; ++i) {
    const int size = bytes_of(dtypes[i]);
    if (!size) return TSS_E_DTYPE;
    tensors += sizes[i] > 0;
    bytes += sizes[i] * size;
    if (sizes[i] > 0 && (!grads[i] || (out && !out[i]))) return TSS_E_ARG;
    if (reinterpret_cast<uintptr_t>(grads[i]) % size || (out && reinterpret_cast<uintptr_t>(out[i]) % size)) return TSS_E_ALIGN;
  }
  if (reinterpret_cast<uintptr_t>(norm) % 4 || reinterpret_cast<uintptr_t>(workspace) % 8) return TSS_E_ALIGN;
  const int64_t sums = c.sums;
  if (sums && !c.one() && (!workspace || workspace_bytes < sums * 8)) return TSS_E_ARG;
  if (out ? overlapping(n, grads, out, sizes, dtypes, norm) : touches(norm, sizeof(float), n, grads, out, sizes, dtypes))
    return TSS_E_ARG;
  if (sums && !c.one()) {
    const uintptr_t begin = reinterpret_cast<uintptr_t>(workspace), at = reinterpret_cast<uintptr_t>(norm);
    if (at < begin + uintptr_t(sums) * 8 && begin < at + sizeof(float)) return TSS_E_ARG;
    if (touches(workspace, sums * 8, n, grads, out, sizes, dtypes)) return TSS_E_ARG;
  }
  double *partial = static_cast<double *>(workspace);
  auto go = [&](auto launch) { return launch(n, grads, sizes, dtypes, max_norm, out, norm, partial, c, bytes, s); };
  return tensors <= kSmallTable ? go(launch_clip<kSmallTable>) : go(launch_clip<kTable>);
}

}  // namespace

extern "C" {

int64_t tss_clip_grad_norm_workspace_size(int64_t n, const int64_t *sizes) {
  Sums c;
  const int32_t st = count_sums(n, sizes, &c);
  return st != TSS_OK ? st : c.one() ? 0 : c.sums * 8;
}

int32_t tss_clip_grad_norm(int64_t n, const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                           float max_norm, void *const *out, float *norm, void *workspace, int64_t workspace_bytes,
                           void *stream) {
  try {
    return clip(n, grads, sizes, dtypes, max_norm, out, norm, workspace, workspace_bytes, static_cast<hipStream_t>(stream));
  } catch (const std::bad_alloc &) {
    return TSS_E_ARG;
  }
}

}  // extern "C"

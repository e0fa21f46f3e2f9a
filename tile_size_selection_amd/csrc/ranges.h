// Which bytes a call reads and writes: host code without HIP, for the entry
// points whose workgroups run in no order, so that an output over anything
// else that the call touches would be a race.
#pragma once
#include <stdint.h>

namespace tss {

class Ranges {
 public:
  // Bytes that are read (none without an address); the mark names them to `writes`.
  uint32_t reads(const void *p, int64_t bytes) {
    add(p, bytes, false, 0);
    return p && bytes > 0 ? uint32_t(1) << (n_ - 1) : 0;
  }
  // Bytes that are written.  They may begin where the marked ones do: a
  // thread reads its elements there before it writes them.
  void writes(const void *p, int64_t bytes, uint32_t over = 0) { add(p, bytes, true, over); }

  // Whether any written bytes are read, or written twice, in another way than that.
  bool clash() const {
    for (int i = 0; i < n_; ++i) {
      const Range &a = of_[i];
      if (!a.written) continue;
      for (int j = 0; j < n_; ++j) {
        const Range &b = of_[j];
        if (i == j || a.begin >= b.end || b.begin >= a.end) continue;
        if (b.written || a.begin != b.begin || !(a.over >> j & 1)) return true;
      }
    }
    return false;
  }

 private:
  struct Range {
    uintptr_t begin, end;
    bool written;
    uint32_t over;
  };
  static constexpr int kMost = 12;
  Range of_[kMost];
  int n_ = 0;

  void add(const void *p, int64_t bytes, bool written, uint32_t over) {
    if (!p || bytes <= 0) return;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    of_[n_++] = {at, at + uintptr_t(bytes), written, over};
  }
};

}  // namespace tss

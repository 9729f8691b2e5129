// resident.h -- how many clusters of a kernel a device holds at once, for each cluster size:
// asked of the runtime once a device and size.  Plain C++.
#pragma once

#include <atomic>

namespace gbs {

template <int DEVICES, int SIZES> class ResidentTable {
 public:
  // The number for clusters of `size` (1 .. SIZES) on `device`.  ask(size) answers where it is
  // not known: a number, or less than 0 where the query failed.  That counts as none this
  // time and is asked again the next.
  template <class F> int get(int device, unsigned size, F&& ask) {
    std::atomic<int>& known = known_[device][size - 1];
    const int k = known.load(std::memory_order_relaxed);
    if (k > 0) return k - 1;
    const int n = ask(size);
    if (n < 0) return 0;
    known.store(n + 1, std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<int> known_[DEVICES][SIZES] = {};  // the number + 1; 0: not known
};

}  // namespace gbs

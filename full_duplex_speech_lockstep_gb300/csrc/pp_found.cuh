// pp_found.cuh - a value that is looked up when it is first needed and kept once it was found (host
// code only; the calls may come from several threads).
#pragma once
#include <atomic>

namespace pp {

// A lookup that fails (null) is tried again by the next call: the driver may not have been ready.
// Threads that look at once find the same.
template <typename P>
class Found {
 public:
  template <typename Lookup>
  P get(Lookup lookup) {
    P p = found_.load(std::memory_order_acquire);
    if (!p && (p = lookup())) found_.store(p, std::memory_order_release);
    return p;
  }

 private:
  std::atomic<P> found_{nullptr};
};

}  // namespace pp

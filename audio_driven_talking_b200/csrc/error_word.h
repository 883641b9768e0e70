// error_word.h - host side of a device's error word: host memory that kernels latch bits into, which any
// thread may report.
#pragma once

#include <atomic>

namespace fh {

struct ErrorWord {
  std::atomic<unsigned*> host{nullptr};  // null until it is allocated
  unsigned* dev = nullptr;               // the kernels' address of it

  // What the word holds, and clears it: one exchange, so that of several threads one is told. What a
  // kernel latches meanwhile is told to this caller or to the next: its write leaves the bit set,
  // whether it comes before the exchange or after, or read the word before and writes it after.
  unsigned take() {
    unsigned* w = host.load(std::memory_order_acquire);
    if (!w || !__atomic_load_n(w, __ATOMIC_RELAXED)) return 0;
    return __atomic_exchange_n(w, 0u, __ATOMIC_ACQ_REL);
  }
};

}  // namespace fh

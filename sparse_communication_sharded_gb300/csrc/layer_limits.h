// layer_limits.h -- what the host keeps about kernels between calls: what CUDA has
// been told they may use, and how long their waits may last.  Host code without
// CUDA's headers, so that a test can interleave its callers.
#pragma once

#include <atomic>
#include <cstdint>
#include <mutex>

namespace scapek {
namespace layer {

// Each kernel's limit on each device, which only rises.  CUDA's call sets a limit
// and does not raise it, so the comparison, the call and the record are one step
// under a lock: with two callers between them, the smaller limit could be the one
// that stays while the larger is on record, and the larger launch fails from then on.
// A limit on record is read without the lock.
class RaisedLimits {
 public:
  static constexpr int kDevices = 64, kKernels = 64;

  // Calls set(bytes), which returns 0 or an error, unless the kernel has that much
  // already.  Returns set's error, or `full` where there is no place left.
  template <typename E, typename Set>
  E raise(int device, const void* kernel, int bytes, E full, Set&& set) {
    Place* const places = places_[device];
    for (int i = 0; i < kKernels; ++i) {
      const void* k = places[i].kernel.load(std::memory_order_acquire);
      if (!k) break;
      if (k == kernel && places[i].bytes.load(std::memory_order_acquire) >= bytes) return E(0);
    }
    std::lock_guard<std::mutex> hold(lock_);
    for (int i = 0; i < kKernels; ++i) {
      Place& p = places[i];
      const void* k = p.kernel.load(std::memory_order_relaxed);
      if (k && k != kernel) continue;
      if (k && p.bytes.load(std::memory_order_relaxed) >= bytes) return E(0);
      const E e = set(bytes);
      if (e != E(0)) return e;
      p.bytes.store(bytes, std::memory_order_release);
      p.kernel.store(kernel, std::memory_order_release);
      return E(0);
    }
    return full;
  }

 private:
  struct Place {
    std::atomic<const void*> kernel{nullptr};
    std::atomic<int> bytes{0};
  };
  Place places_[kDevices][kKernels];
  std::mutex lock_;
};

// Every wait of the product kernels ends: one for a copy, a stage or an accumulator
// to be read after two seconds.  An accumulator is not ready before its whole
// contraction is done, so the wait for it has 5 us a stage of that more (a stage
// takes 0.3 us): 2^31 rows make a weight gradient of 4 million stages a block, which
// can last longer than two seconds.
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t product_wait_ns(int64_t stages) { return kWaitLimitNs + (uint64_t)stages * 5000u; }

// A device's count of waits given up only grows; who asks for news is told what was
// added since anyone last asked.  Nothing is cleared on the device, so no report falls
// between a read and a clear.
class LastSeen {
 public:
  // How many were added since the last call, for a count read as v.  Of two callers
  // the later read may arrive first; the other then has nothing new.
  int news(unsigned v) {
    unsigned seen = seen_.load(std::memory_order_relaxed);
    for (;;) {
      const int more = (int)(v - seen);
      if (more <= 0) return 0;
      if (seen_.compare_exchange_weak(seen, v, std::memory_order_relaxed)) return more;
    }
  }

 private:
  std::atomic<unsigned> seen_{0};
};

}  // namespace layer
}  // namespace scapek

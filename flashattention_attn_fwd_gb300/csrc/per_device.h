// Set-up that has to be done on every device of the process (internal header;
// no CUDA, so that it can be tested without a GPU).
#pragma once

#include <atomic>
#include <mutex>

namespace fl {

constexpr int kMaxDevices = 64;

// A step that has to succeed once on each device.  run(dev, step) is the result
// of step() until one on `dev` is a success (0); after that the step is not
// called again and what it wrote is visible.  A failure is returned, not kept:
// the next call tries again.
class OncePerDevice {
  std::atomic<bool> done_[kMaxDevices] = {};
  std::mutex mutex_;

 public:
  template <class Step>
  auto run(int dev, Step&& step) -> decltype(step()) {
    using Result = decltype(step());
    if (done_[dev].load(std::memory_order_acquire)) return Result{};
    std::lock_guard<std::mutex> lock(mutex_);
    if (done_[dev].load(std::memory_order_relaxed)) return Result{};
    const Result r = step();
    if (r == Result{}) done_[dev].store(true, std::memory_order_release);
    return r;
  }
};

}  // namespace fl

// Work that is done once for each device.
#pragma once

#include <atomic>
#include <mutex>

namespace tcg {

// Runs a device's setup on the first call, and again on the next one as long as
// it fails: what failed for want of memory may have it then.
template <class Error>
class OncePerDevice {
 public:
  static constexpr int MAX_DEVICES = 64;
  template <class F>
  Error operator()(int dev, F&& setup) {
    std::atomic<bool>& done = done_[dev];
    if (done.load(std::memory_order_acquire)) return Error{};
    std::lock_guard<std::mutex> lk(mu_);
    if (done.load(std::memory_order_relaxed)) return Error{};
    const Error e = setup();
    if (e == Error{}) done.store(true, std::memory_order_release);
    return e;
  }

 private:
  std::mutex mu_;
  std::atomic<bool> done_[MAX_DEVICES] = {};
};

}  // namespace tcg

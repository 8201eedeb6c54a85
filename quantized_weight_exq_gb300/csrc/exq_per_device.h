// What a launch sets up once on each device: a kernel's attributes belong to
// the device that is current when they are set, not to the process.
#pragma once

#include <mutex>

namespace exq {

class PerDevice {
 public:
  // Calls set_up() (true: it worked) unless it has worked for `device` before;
  // a failure is not kept, the next call tries again. Thread-safe. False for
  // a device outside the range.
  template <typename F>
  bool once(int device, F&& set_up) {
    if (device < 0 || device >= kMaxDevices) return false;
    std::lock_guard<std::mutex> lock(mutex_);
    if (!done_[device]) done_[device] = set_up();
    return done_[device];
  }

 private:
  static constexpr int kMaxDevices = 64;
  std::mutex mutex_;
  bool done_[kMaxDevices] = {};
};

}  // namespace exq

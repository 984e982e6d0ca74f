// Which devices a process has prepared for a kernel, shared by the host threads that launch it.
//
// The preparation (attributes of a function) may be done twice: threads that come first
// together both do it.  Only the reads and writes of the note must not race.
#pragma once

#include <atomic>

namespace pkv {

class DeviceSet {
 public:
  bool has(int device) const {
    return device >= 0 && device < 32 && (bits_.load(std::memory_order_acquire) >> device & 1u) != 0;
  }
  // (devices past the 32nd are prepared on every launch)
  void add(int device) {
    if (device >= 0 && device < 32) bits_.fetch_or(1u << device, std::memory_order_release);
  }

 private:
  std::atomic<unsigned> bits_{0};
};

}  // namespace pkv

// What a launcher sets or asks once: function attributes and occupancy belong
// to the device that is current at the call, so each device has its own.
#pragma once

#include <atomic>
#include <mutex>

#include <cuda_runtime.h>

namespace dg {

constexpr int kMaxDevices = 64;

// A value for each index, made by the first call that succeeds for it (any
// thread); a failure is returned and tried again by the next call.
template <class T>
class PerIndex {
 public:
  template <class F>   // cudaError_t make(T *)
  cudaError_t get(int i, T *out, F &&make) {
    if (i < 0 || i >= kMaxDevices) return make(out);   // not kept
    Slot &s = slots_[i];
    if (!s.made.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mu_);
      if (!s.made.load(std::memory_order_relaxed)) {
        const cudaError_t e = make(&s.value);
        if (e != cudaSuccess) return e;
        s.made.store(true, std::memory_order_release);
      }
    }
    *out = s.value;
    return cudaSuccess;
  }

 private:
  struct Slot {
    std::atomic<bool> made{false};
    T value{};
  };
  std::mutex mu_;
  Slot slots_[kMaxDevices];
};

// The current device's value.
template <class T>
class PerDevice {
 public:
  template <class F>
  cudaError_t get(T *out, F &&make) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : slots_.get(dev, out, make);
  }

 private:
  PerIndex<T> slots_;
};

// Nothing but the setting itself, once on each device.
class OnceOnDevice {
 public:
  template <class F>   // cudaError_t set()
  cudaError_t run(F &&set) {
    char none;
    return slots_.get(&none, [&](char *) { return set(); });
  }

 private:
  PerDevice<char> slots_;
};

}  // namespace dg

// What is done once in a process, by whichever call comes first.
#pragma once

#include <atomic>

namespace moe {

// Runs f until it has succeeded once (0, cudaSuccess). A failure is returned and not kept: what failed for a passing
// reason (no memory to load a kernel's module) is tried again by the next call. Calls on several host threads may run
// f at the same time.
class Once {
 public:
  template <typename F>
  auto operator()(F f) -> decltype(f()) {
    using Result = decltype(f());
    if (done_.load(std::memory_order_acquire)) return Result{};
    const Result r = f();
    if (r == Result{}) done_.store(true, std::memory_order_release);
    return r;
  }

 private:
  std::atomic<bool> done_{false};
};

}  // namespace moe

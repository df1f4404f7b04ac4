// Answers that belong to a device, kept by its number.
#pragma once
#include <atomic>

namespace nf {

constexpr int MAX_DEVICES = 64;  // devices of a process that something is kept for

// One number of 0 or more for each device and each of N questions, asked for when it is
// first wanted.  A process may plan for several devices, whose SMs are grouped otherwise.
// What could not be had is not kept: the next call asks again.
template <int N>
class ByDevice {
 public:
  // *answer by ask(answer), which returns an error code (0: none), or as kept; the code.
  template <typename F>
  auto get(int device, int which, int* answer, F ask) -> decltype(ask(answer)) {
    using Code = decltype(ask(answer));
    const bool counted = device >= 0 && device < MAX_DEVICES;
    if (counted) {
      const int kept = kept_[device][which].load(std::memory_order_relaxed);
      if (kept) {
        *answer = kept - 1;
        return Code{};
      }
    }
    const Code code = ask(answer);
    if (code == Code{} && counted) kept_[device][which].store(*answer + 1, std::memory_order_relaxed);
    return code;
  }

 private:
  std::atomic<int> kept_[MAX_DEVICES][N] = {};  // answer + 1, 0: not asked yet
};

}  // namespace nf

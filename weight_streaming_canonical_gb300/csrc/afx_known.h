// Numbers of the device or the driver that are asked for once (host code).
#pragma once

#include <atomic>
#include <cstdint>

namespace afx {
namespace serve {

// A number that does not change: asked for until an answer comes, kept from then on.  ask(uint64_t* value) returns whether
// there was one; a call that failed (no memory, an error of earlier work) says nothing about the next.
class Known {
public:
    template <typename Ask>
    bool get(uint64_t* value, Ask&& ask) {
        if (there_.load(std::memory_order_acquire)) {
            *value = value_.load(std::memory_order_relaxed);
            return true;
        }
        if (!ask(value)) {
            *value = 0;
            return false;
        }
        value_.store(*value, std::memory_order_relaxed);  // by several threads at once: the same number
        there_.store(true, std::memory_order_release);
        return true;
    }

private:
    std::atomic<uint64_t> value_{0};
    std::atomic<bool> there_{false};
};

}  // namespace serve
}  // namespace afx

// How much dynamic shared memory a kernel may use, raised as launches need it.
// Host code without CUDA types, so that its order of events can be tested without a GPU.
#pragma once

#include <cstddef>
#include <mutex>

namespace rb {

// One per kernel. The limit is an attribute of the kernel on a device, which a
// call may also lower: launches of one kernel with different sizes, from
// several threads, must neither lower what another has raised nor believe in
// more than was set. So check, call and note are one step under a lock, and the
// call is only made to raise.
class SmemLimit {
public:
    // `set(bytes)` sets the limit on device `dev` and returns 0 if it did so.
    template <class Set>
    auto raise(int dev, size_t bytes, Set set) -> decltype(set(bytes)) {
        std::lock_guard<std::mutex> lk(mu_);
        if (dev < 0 || dev >= DEVICES) return set(bytes);       // no machine has as many
        if (at_[dev] >= bytes) return {};
        const auto e = set(bytes);
        if (e == decltype(set(bytes)){}) at_[dev] = bytes;
        return e;
    }

private:
    static constexpr int DEVICES = 256;
    std::mutex mu_;
    size_t at_[DEVICES] = {};
};

}  // namespace rb

// smem_grant.h -- what each kernel has been allowed of dynamic shared memory (host only).
#pragma once

#include <map>
#include <mutex>
#include <utility>

namespace wsw {

// The largest limit granted to each (kernel, device).  A request up to it makes no call; a larger
// one sets it.  Two host threads may ask for the same kernel at once.
class SmemGrants {
public:
    // set(bytes) changes the limit and returns 0 or an error code, which is passed on
    template <typename Set>
    int ensure(const void *kernel, int device, int bytes, Set set) {
        std::lock_guard<std::mutex> lk(mu_);  // over the call, too: a smaller limit must not be set after a larger one
        int &g = granted_[{kernel, device}];
        if (g >= bytes) return 0;
        const int e = set(bytes);
        if (e == 0) g = bytes;
        return e;
    }

private:
    std::mutex mu_;
    std::map<std::pair<const void *, int>, int> granted_;
};

}  // namespace wsw

// cluster_choice.h -- clusters of more CTAs than every device can hold (host only).
#pragma once

#include <map>
#include <mutex>

namespace wsw {

// The CTAs of a kernel's cluster on each device: 16, an option beyond the portable 8, where one such
// cluster fits.  It does not on a partition of the device whose SMs are too few in each GPC.
class ClusterChoice {
public:
    // fits() says whether a cluster of 16 can be resident; asked once per device
    template <typename Fits>
    unsigned of(int device, Fits fits) {
        std::lock_guard<std::mutex> lk(mu_);
        auto it = ctas_.find(device);
        if (it == ctas_.end()) it = ctas_.emplace(device, fits() ? 16u : 8u).first;
        return it->second;
    }

private:
    std::mutex mu_;
    std::map<int, unsigned> ctas_;
};

}  // namespace wsw

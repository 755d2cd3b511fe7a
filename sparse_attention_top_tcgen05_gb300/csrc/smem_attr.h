// smem_attr.h -- how much dynamic shared memory each kernel has been allowed on each device.
#pragma once
#include <mutex>

namespace lidx {

// A kernel's limit only ever grows, and it is recorded under the lock it is set under.  (Two threads whose calls need
// different sizes of one kernel: were the lock given up in between, the smaller could be set last and the larger recorded.)
template <int KERNELS, int DEVICES>
class SmemLimits {
public:
    // allow(bytes) sets the limit of kernel fn on device dev; 0: done.
    template <class Allow>
    int ensure(int dev, const void* fn, int bytes, Allow allow) {
        std::lock_guard<std::mutex> lock(mu_);
        int i = 0;
        while (i < n_ && fn_[i] != fn) ++i;
        if (i < n_ && bytes_[i][dev] >= bytes) return 0;
        if (i == KERNELS) return -1;  // more kernels than the table was made for
        const int e = allow(bytes);
        if (e) return e;
        if (i == n_) fn_[n_++] = fn;
        bytes_[i][dev] = bytes;
        return 0;
    }

private:
    const void* fn_[KERNELS] = {};
    int bytes_[KERNELS][DEVICES] = {};
    int n_ = 0;
    std::mutex mu_;
};

}  // namespace lidx

// What the host keeps of a kernel on a device (plain C++, no CUDA).
#pragma once

namespace pkv {

// A value for each (kernel, device): a kernel's attributes and occupancy are the
// device's they were set or asked on.  Fixed room, no allocation, no lock.
template <class T, int N>
class KernelTable {
    struct Entry {
        const void *fn;
        int device;
        T value;
    };
    Entry entries_[N] = {};
    int n_ = 0;

public:
    // The value kept for fn on device, or null.
    T *find(const void *fn, int device) {
        for (int i = 0; i < n_; ++i)
            if (entries_[i].fn == fn && entries_[i].device == device) return &entries_[i].value;
        return nullptr;
    }
    // Keeps a value; null where there is no device (< 0) or no room: it is worked out again then.
    T *add(const void *fn, int device, const T &value) {
        if (device < 0 || n_ == N) return nullptr;
        entries_[n_] = Entry{fn, device, value};
        return &entries_[n_++].value;
    }
};

}  // namespace pkv

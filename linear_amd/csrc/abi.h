// abi.h -- host-side checks shared by the C ABI's files.
#pragma once

#include <stdint.h>

namespace lin {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLdIn = (int64_t(1) << 22) - 1;
constexpr int64_t kMaxLdOut = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxGridX = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxGridY = 65535;
// Columns of one launch.  The one-row kernels take 64 threads a column and a launch holds
// fewer than 2^32 (see launch_kernel); wider outputs are taken in parts, each a layer of its own.
constexpr int64_t kColumnPart = int64_t(1) << 25;

// The compute units and XCDs of the device a call runs on, read from the device
// (a partitioned part has fewer).  Plans made without a usable device (the
// pure-host linear_f16_plan) assume a whole MI355X: 256 CUs in 8 XCDs.
struct DevInfo {
    int cus;
    int xcd_shift;   // log2 of the XCD count; 0 (no XCD-aware remap) when not a power of two
};
constexpr DevInfo kWholeMI355X{256, 3};

struct Extent {
    uintptr_t lo, hi;  // [lo, hi) in bytes; hi == lo when empty
};

inline Extent extent(const void* p, int64_t rows, int64_t ld, int64_t cols, int64_t elem_bytes = 2) {
    Extent e{(uintptr_t)p, (uintptr_t)p};
    if (p && rows > 0 && cols > 0) e.hi = e.lo + (uintptr_t)(((rows - 1) * ld + cols) * elem_bytes);
    return e;
}

inline bool overlaps(Extent a, Extent b) { return a.lo < b.hi && b.lo < a.hi; }

// A gfx950 must be current: its index and figures (linear_abi.hip).
int32_t check_device(int* dev_out, DevInfo* info = nullptr);
// What linear_last_hip_error returns on this thread.
void set_last_hip_error(int32_t e);

}  // namespace lin

// What the library's host files share: the device's topology and small helpers.
#pragma once

#include <stdint.h>

namespace libgemm_host {

// Compute units and XCDs of the current device, read once per device from
// its attributes (MI355X: 256 CUs in 8 XCDs, which is also the answer when no
// device can be queried, e.g. for gemm_select_config on a host without GPU).
struct Topology {
    int cus, xcds;
};
constexpr int kMaxDevices = 64;
Topology topology();

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace libgemm_host

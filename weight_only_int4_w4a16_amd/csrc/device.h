// The once-per-device record of properties that the entry points check and plan with.
#pragma once

#include <stdint.h>

namespace w4a16 {

struct DeviceInfo {
    bool ok;
    int cus;
    int64_t lds_limit;
};

// Current device's cached properties, or null when it is missing or not gfx950.
const DeviceInfo *current_device();

}  // namespace w4a16

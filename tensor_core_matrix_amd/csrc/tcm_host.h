// Host-only definitions shared by the C ABI's translation units.
#pragma once

#include "../../include/tcm.h"

#include <hip/hip_runtime.h>

namespace tcm {

struct DeviceInfo {
    int cus = 0;
    bool gfx950 = false;
    hipError_t err = hipSuccess;
};

// The current device's properties (read once per device); TCM_ERR_NO_DEVICE
// where there is none or it is not gfx950.
tcm_status device_info(DeviceInfo* out);

}  // namespace tcm

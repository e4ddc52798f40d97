// api_common.h -- what the translation units of the C ABI share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "gmm.h"

namespace scem {

// Status after enqueuing n kernels (counted for gmm_launch_count).
gmm_status api_launched(int n);
// SM count of the current device.
gmm_status api_device_sms(int* sms);
// Nanoseconds after which a device-side wait gives up (gmm_set_wait_budget).
uint64_t api_wait_budget();

}  // namespace scem

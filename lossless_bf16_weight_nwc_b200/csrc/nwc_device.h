// nwc_device.h — what the C ABI's sources share about the current device.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cstddef>
#include <cstdint>

#include "../../include/nwc.h"

namespace nwc {

// SM count and per-block opt-in shared memory of the current device (cached).
nwc_status current_device(int* dev, int* sms, size_t* smem);

// cuTensorMapEncodeTiled from the driver, looked up once; null when it is missing.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Polls before a bounded wait in a kernel gives up; 0 = the kernels' default
// (nwc_test_set_wait_limit).
uint32_t wait_limit();

}  // namespace nwc

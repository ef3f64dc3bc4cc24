// dc_host.h -- what the host units of the C ABI share (defined in dc_api.cu):
// the error text of the calling thread, the launch bookkeeping, the options
// every launch looks at and the properties of the current device.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dc.h"

namespace dc {

// Sets the calling thread's dc_last_error() text and returns `s`.
dc_status_t fail(dc_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it and returns DC_OK.
dc_status_t ok();
// The status of a launch; counts it and records its grid.
dc_status_t check_launch(cudaError_t e, const char* what, int grid);
dc_status_t current_device(int* dev);
dc_status_t sm_count(int dev, int* sms);

void read_options();               // the environment's initial values, once
bool pdl_option();                 // "pdl"
bool launch_failure_injected();    // "test_fail_launch"

}  // namespace dc

// What the entry points of the C ABI share across translation units.
#pragma once

#include "specv.h"

namespace specv {

// The calling thread's error message (as by printf) and the status returned.
specv_status api_fail(specv_status s, const char* fmt, ...);
// Success: clears the message, sets the launch count of the call.
specv_status api_done(int32_t launches);
// SMs of the current device (read once per process).
int api_sm_count();

}  // namespace specv

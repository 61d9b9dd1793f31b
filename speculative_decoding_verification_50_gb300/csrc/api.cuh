// What the entry points of the C ABI share across translation units.
#pragma once

#include "specv.h"

namespace specv {

// The calling thread's error message (as by printf) and the status returned.
specv_status api_fail(specv_status s, const char* fmt, ...);
// Success: clears the message, sets the launch count of the call.
specv_status api_done(int32_t launches);
// The test hook SPECV_TEST_STALL: 1 + the index given for kernel `which`, else 0.
int api_test_stall(char which);
// SMs of the current device (read once per process).
int api_sm_count();

}  // namespace specv

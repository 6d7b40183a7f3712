// api.hpp - what the files of the C ABI share: the error record and the device set-up.
#pragma once

#include <stdint.h>

namespace nvfp4 {

// records a per-thread message for nvfp4_last_error() and returns `status`
int api_fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// clears the record; returns NVFP4_OK
int api_ok();
// one-time set-up of the current device; its silu table
int api_device(const uint16_t** silu_table);

}  // namespace nvfp4

// Host helpers shared by the files of the C ABI: the calling thread's last
// error and the device check (defined in fg_api.cpp).
#pragma once

#include <stdint.h>

#include "../../include/fp32gemm.h"

namespace fg {

// Records the failure (1-based argument position or 0, and a message) for
// fg_last_bad_arg / fg_last_error and returns s.
fg_status fail(fg_status s, int32_t bad_arg, const char* fmt, ...)
    __attribute__((format(printf, 3, 4)));
void clear_error();
// FG_OK when the current device is a gfx950.
fg_status check_device();

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace fg

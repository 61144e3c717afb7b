// Status reporting and argument checks shared by the C ABI's translation units.
#pragma once

#include <stdint.h>

#include "../../include/qmm.h"

namespace qmm {

// Sets this thread's qmm_last_error() message and returns the status.
qmm_status fail(qmm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message.
qmm_status ok();
qmm_status from_hip(hipError_t e, const char* what);

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
inline bool bits_ok(int bits) { return bits == 1 || bits == 2 || bits == 3 || bits == 4 || bits == 8; }

}  // namespace qmm

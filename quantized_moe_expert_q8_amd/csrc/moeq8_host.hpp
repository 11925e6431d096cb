// Host-side helpers shared by the libmoeq8 entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/moeq8.h"

namespace moeq8 {

// Status of the launch just enqueued: MOEQ8_EHIP (and the error cleared) when
// the runtime reports a failure.
inline int check_launch() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOEQ8_OK : MOEQ8_EHIP;
}

// Bytes of one element of an enum moeq8_dtype.
inline int dtype_bytes(int32_t dtype) { return dtype == MOEQ8_F32 ? 4 : 2; }

inline bool ranges_overlap(const void* p, int64_t p_bytes, const void* q, int64_t q_bytes) {
    const uint8_t* a = (const uint8_t*)p;
    const uint8_t* b = (const uint8_t*)q;
    return a < b + q_bytes && b < a + p_bytes;
}

}  // namespace moeq8

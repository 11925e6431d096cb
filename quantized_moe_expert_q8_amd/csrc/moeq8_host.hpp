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

// Most blocks of a launch: HIP counts a grid's threads in 32 bits.
inline int64_t most_blocks(int64_t threads) { return 0xffffffffll / threads; }

// Bytes of one element of an enum moeq8_dtype.
inline int dtype_bytes(int32_t dtype) { return dtype == MOEQ8_F32 ? 4 : 2; }

inline bool ranges_overlap(const void* p, int64_t p_bytes, const void* q, int64_t q_bytes) {
    const uint8_t* a = (const uint8_t*)p;
    const uint8_t* b = (const uint8_t*)q;
    return a < b + q_bytes && b < a + p_bytes;
}

// Whether rows of `bytes` bytes at p and at o overlap otherwise than by being the
// same rows, where each element is read before it is written.  Rows of one
// stride may take turns in a buffer.
inline bool rows_clash(const void* p, int64_t p_stride, const void* o, int64_t o_stride, int64_t rows, int64_t bytes) {
    if (p == o && (p_stride == o_stride || rows == 1)) return false;
    if (!ranges_overlap(p, (rows - 1) * p_stride + bytes, o, (rows - 1) * o_stride + bytes)) return false;
    if (p_stride != o_stride) return true;
    const int64_t apart = ((const uint8_t*)o - (const uint8_t*)p) % p_stride, behind = apart < 0 ? apart + p_stride : apart;
    return behind < bytes || p_stride - behind < bytes;
}

}  // namespace moeq8

// Host-side helpers shared by the libmoeq8 entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <numeric>

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

// Pieces of `bytes` bytes at p + i stride[0] + j stride[1] + l stride[2], each index below its count.
struct Pieces {
    const void* p;
    int64_t bytes, count[3], stride[3];
};

// Bytes from the first to the last of them, along the dimensions that `without` has no bit for.
inline int64_t extent(const Pieces& x, int without = 0) {
    int64_t n = x.bytes;
    for (int i = 0; i < 3; ++i)
        if (!(without >> i & 1) && x.count[i] > 1) n += (x.count[i] - 1) * x.stride[i];
    return n;
}

// Whether pieces of two arrays overlap.  Arrays that take turns in one buffer do not:
// steps along some of the dimensions leave a place's remainder by the greatest
// common divisor of their strides as it is, and where the remainders that the other
// dimensions reach lie apart, so do the arrays.
inline bool pieces_overlap(const Pieces& a, const Pieces& b) {
    if (!ranges_overlap(a.p, extent(a), b.p, extent(b))) return false;
    for (int outer = 1; outer < 8; ++outer) {
        int64_t g = 0;
        for (int i = 0; i < 3; ++i)
            if (outer >> i & 1) g = std::gcd(g, std::gcd(a.count[i] > 1 ? a.stride[i] : 0, b.count[i] > 1 ? b.stride[i] : 0));
        if (g == 0) continue;
        const int64_t apart = ((const uint8_t*)b.p - (const uint8_t*)a.p) % g, behind = apart < 0 ? apart + g : apart;
        if (behind >= extent(a, outer) && g - behind >= extent(b, outer)) return false;
    }
    return true;
}

}  // namespace moeq8

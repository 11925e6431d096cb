// RMS norm with the residual's addition and 8-bit outputs, and the same 8-bit
// rows without the norm.
//
//   s = f32(x) + f32(residual)          residual_out = T(s)
//   y = (s * inv) * w                   inv = f32(1 / sqrt(mean(s^2) + eps)), the mean in 64 bits;
//                                       at most the largest finite value, NaN where s is not finite
//   i8 rows:   d = max|y| / 127 over the row, codes roundf(y / d) on the fp32 quotient
//   q8_1 rows: the block rule of q8_1_quantize_rows on y
//
// The sum of squares is held in 64 bits: a code is decided by one rounding of
// y / d, and with a sum in 32 bits its order would move codes that lie next to
// a half.  One pass over the data: a thread keeps its 8-value vectors of s in
// registers between the two row reductions, so x and the residual are read
// once, and the weights are loaded with them.  What bounds it is the memory
// traffic: 8192 x 8192 in bf16 with a residual takes 84 to 86 us, 5.5 TB/s, the
// rate of a large copy.  Without a residual the arithmetic of the q8_1 codes is
// more than that (16000 x 4096 to q8_1 rows 59 us, 3.5 TB/s, to both formats 73,
// 3.7 TB/s; with a residual 86 and 102 us, 5.4 and 5.3 TB/s).  For few rows it is
// the launch: 3.1 us for one of 4096.
#include "moeq8_lds.hpp"
#include "moeq8_types.hpp"
#include "moeq8_host.hpp"

namespace moeq8 {
namespace {

struct NormArgs {
    const void* x; int64_t x_stride;
    const void* res; int64_t res_stride;          // null: no residual
    void* res_out; int64_t res_out_stride;
    const void* w;
    int64_t rows, k;
    double eps;
    int8_t* q; int64_t q_stride;                  // null: no i8 rows
    float* scale;
    uint8_t* xq;                                  // null: no q8_1 rows
};

constexpr int VEC = 8;                            // values a thread takes at a time: a quarter of a block

// Bits of |v|: as unsigned numbers they are in the order of the magnitudes, a
// NaN above all, so a maximum of them keeps a NaN.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL, typename V>
__device__ __forceinline__ V moved(V v) {          // v of the lane that the DPP control names, an active one
    if constexpr (sizeof(V) == 8) {
        const uint2 u = __builtin_bit_cast(uint2, v);
        return __builtin_bit_cast(V, uint2{(uint32_t)__builtin_amdgcn_mov_dpp((int)u.x, CTRL, 0xf, 0xf, false),
                                           (uint32_t)__builtin_amdgcn_mov_dpp((int)u.y, CTRL, 0xf, 0xf, false)});
    } else {
        return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
    }
}
constexpr int XOR1 = 0xB1, XOR2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140;

// Largest over the TPR threads of a row; every thread gets it.  Over a full wave
// in registers: the 16 lanes of a row by DPP, then the four rows.  (Through LDS,
// as __shfl_xor goes, the reductions of one row of 4096 took a seventh of its
// time.)
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* lds) {
    v = larger(v, moved<XOR1>(v));
    v = larger(v, moved<XOR2>(v));
    v = larger(v, moved<HALF_MIRROR>(v));
    v = larger(v, moved<MIRROR>(v));
    auto of_row = [&](int r) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * r); };
    v = larger(larger(of_row(0), of_row(1)), larger(of_row(2), of_row(3)));
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        lds_barrier();
        v = lds[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) v = larger(v, lds[i]);
    }
    return v;
}

// Lower halves of a wave's a and b beside the upper ones: {a.lo, b.lo} + {a.hi,
// b.hi}; or rows of 16 lanes: {a0, b0, a2, b2} + {a1, b1, a3, b3}.
template <bool HALVES>
__device__ __forceinline__ double added_crosswise(double a, double b) {
    auto swap = [](uint32_t x, uint32_t y) {
        if constexpr (HALVES) return __builtin_amdgcn_permlane32_swap(x, y, false, false);
        else return __builtin_amdgcn_permlane16_swap(x, y, false, false);
    };
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    const auto lo = swap(x.x, y.x), hi = swap(x.y, y.y);
    return __builtin_bit_cast(double, uint2{lo[0], hi[0]}) + __builtin_bit_cast(double, uint2{lo[1], hi[1]});
}

// Sum over LANES lanes (a power of two), in every group of as many.
template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
    if constexpr (LANES >= 2) v += moved<XOR1>(v);
    if constexpr (LANES >= 4) v += moved<XOR2>(v);
    if constexpr (LANES >= 8) v += moved<HALF_MIRROR>(v);
    if constexpr (LANES >= 16) v += moved<MIRROR>(v);
    if constexpr (LANES >= 32) v = added_crosswise<false>(v, v);
    if constexpr (LANES >= 64) v = added_crosswise<true>(v, v);
    return v;
}

// Sum over a row, of which thread t of TPR has the sums of its vectors i * TPR +
// t; every thread gets it.  The order is that of spans of 64 vectors, each
// summed over its lanes, and of a tree over the spans: the same for every TPR,
// since the form goes by the number of rows too and a row's outputs are not to
// depend on it.  (With a thread's NV sums added first, a row among 2049 could
// differ from the same row alone.)  The NV spans of a wave go through one tree,
// in its halves or rows of lanes: with a tree each, 3000 x 16384 in fp16 took
// 77 us and not 58, 16000 x 4096 in bf16 to q8_1 rows 61 and not 58.5.
template <int TPR, int NV>
__device__ __forceinline__ double row_sum(const double (&v)[NV], double* lds) {
    static_assert(NV <= 4 && (TPR > 64 || NV == 1), "a row of lanes a span");
    double u = added_crosswise<true>(v[0], v[NV > 1 ? 1 : 0]);
    if constexpr (NV > 2) u = added_crosswise<false>(u, added_crosswise<true>(v[2], NV > 3 ? v[NV - 1] : 0.0));
    else u = added_crosswise<false>(u, u);
    u = lanes_sum<16>(u);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64, SPANS = NV * W, SLOTS = SPANS <= 2 ? 2 : SPANS <= 4 ? 4 : SPANS <= 8 ? 8 : SPANS <= 16 ? 16
                                                               : SPANS <= 32 ? 32 : 64;
        const int lane = threadIdx.x & 63, i = (lane >> 4 & 1) << 1 | lane >> 5;       // the span that this row of lanes has
        if ((lane & 15) == 0 && i < NV) lds[i * W + (threadIdx.x >> 6)] = u;
        lds_barrier();
        const int slot = lane & (SLOTS - 1);
        u = lanes_sum<SLOTS>(SLOTS == SPANS || slot < SPANS ? lds[slot] : 0.0);
    }
    return u;
}

// Codes of 8 values of scale d, packed; their sum.  d = 0 and a d that is not
// finite give zeros (the scale says which).
//
// The code of y is roundf of the correctly rounded quotient y / d.  y * rcp(d)
// differs from it by less than 2.3e-5 (v_rcp_f32 within an ulp, the quotient
// rounded by half of one, both times 127), so where it lies more than 2^-14
// from every half both round to the same integer; a vector with another value,
// about one wave's in 16, takes the division.  Adding 1.5 * 2^23 rounds to an
// integer whose low byte is the code.
__device__ __forceinline__ uint2 codes8(const float (&y)[VEC], float d, int& sum) {
    uint2 o = {0u, 0u};
    sum = 0;
    if (!(d > 0.0f && d < __builtin_inff())) return o;
    constexpr float ROUND = 12582912.0f;
    const float rd = __builtin_amdgcn_rcpf(d);
    uint32_t u[VEC];
    float off = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float r = __builtin_fmaf(y[i], rd, ROUND);
        off = fmaxf(off, fabsf(__builtin_fmaf(y[i], rd, ROUND - r)));
        u[i] = __float_as_uint(r);
    }
    // below the normal range the reciprocal is not what the above takes it for
    if (__builtin_expect(off >= 0.5f - 0x1p-14f || d < 0x1p-126f, 0)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            // d is so coarse there that a quotient may round past 127
            const int c = (int)roundf(y[i] / d);
            u[i] = (uint32_t)(c > 127 ? 127 : (c < -127 ? -127 : c));
        }
    }
    o.x = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u) | __builtin_amdgcn_perm(u[3], u[2], 0x04000c0cu);
    o.y = __builtin_amdgcn_perm(u[5], u[4], 0x0c0c0400u) | __builtin_amdgcn_perm(u[7], u[6], 0x04000c0cu);
    sum = __builtin_amdgcn_sdot4((int)o.x, 0x01010101, __builtin_amdgcn_sdot4((int)o.y, 0x01010101, 0, false), false);
    return o;
}

// Vector of n valid values at p, the others zero.
template <typename T>
__device__ __forceinline__ void load_raw(T (&v)[VEC], const T* p, int n) {
    if (n >= VEC) {
        load_vec(v, p);
    } else {
        T zero;
        from_f32(zero, 0.0f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = zero;
        if (n <= 0) return;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = p[i < n ? i : 0];       // no load waits for another
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = i < n ? v[i] : zero;
    }
}

template <typename T>
__device__ __forceinline__ void load8(float (&v)[VEC], const T* p, int n) {
    T t[VEC];
    load_raw(t, p, n);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = to_f32(t[i]);
}

// The residual, which the next block reads: nontemporal (8192 x 8192 in bf16
// 96 and 100 us, 1024 x 4096 10.3 and 12.3).
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[VEC], int n) {
    T t[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) from_f32(t[i], v[i]);
    if (n >= VEC) {
        store_vec<true>(p, t);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < n) p[i] = t[i];
    }
}

// s of vector i (n valid values) of row r.
template <typename T>
__device__ __forceinline__ void load_sum(float (&v)[VEC], const NormArgs& a, int64_t r, int64_t i, int n) {
    load8(v, (const T*)a.x + r * a.x_stride + i * VEC, n);
    if (a.res) {
        float u[VEC];
        load8(u, (const T*)a.res + r * a.res_stride + i * VEC, n);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += u[j];
    }
}

// At most the largest finite value: with no eps to speak of, a row of zeros would
// else be 0 * inf, and the padding of every row below the normal range too.  NaN
// where the row holds an infinity (fp32 squares cannot pass 64 bits otherwise):
// its reciprocal root is 0, which would make the row's other blocks valid zeros.
__device__ __forceinline__ float inv_rms(double sum, int64_t k, double eps) {
    const float inv = (float)(1.0 / sqrt(sum / (double)k + eps));
    return fminf(inv, __FLT_MAX__) + (float)(sum - sum);        // 0, or NaN
}

// Outputs of one vector: y, with d the row's scale when i8 rows are wanted.
__device__ __forceinline__ void store_codes(const NormArgs& a, const float (&y)[VEC], int64_t r, int64_t i, int n,
                                            float d) {
    int sum;
    if (a.q) {
        const uint2 c = codes8(y, d, sum);
        int8_t* o = a.q + r * a.q_stride + i * VEC;
        if (n >= VEC) {
            *reinterpret_cast<u32x2b*>(o) = u32x2b{c.x, c.y};
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (j < n) o[j] = (int8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
        }
    }
    if (a.xq) {                                    // k % 32 == 0: the 4 lanes of a block are all here
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < VEC; ++j) m = larger(m, magnitude(y[j]));
        m = larger(m, moved<XOR1>(m));
        m = larger(m, moved<XOR2>(m));
        const float db = __uint_as_float(m) / 127.0f;
        const uint2 c = codes8(y, db, sum);
        sum += moved<XOR1>(sum);
        sum += moved<XOR2>(sum);
        uint32_t* o = reinterpret_cast<uint32_t*>(a.xq + (r * (a.k / QK) + i / 4) * Q81_BYTES);
        if ((i & 3) == 0)
            o[0] = float_to_half_bits(db) | (float_to_half_bits(materialize_f32(db * (float)sum)) << 16);
        *reinterpret_cast<u32x2b*>(o + 1 + 2 * (i & 3)) = u32x2b{c.x, c.y};
    }
}

// TPR threads hold a row, NV vectors each (vector i of a thread is vector
// i * TPR + thread of the row, so a wave's loads are contiguous).
template <typename T, bool NORM, int TPR, int NV>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void k_norm_q8(NormArgs a) {
    __shared__ double lds_sum[NV * TPR / 64];
    __shared__ uint32_t lds_max[TPR / 64];
    constexpr int RPB = TPR == 64 ? 4 : 1;
    const int t = threadIdx.x & (TPR - 1);
    const int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (r >= a.rows) return;                       // whole waves; with barriers a block is one row
    float v[NV][VEC];
    T wt[NORM ? NV : 1][VEC];
    double sq[NV] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t at = (int64_t)i * TPR + t;
        const int64_t left = a.k - at * VEC;
        const int n = left < VEC ? (left < 0 ? 0 : (int)left) : VEC;
        load_sum<T>(v[i], a, r, n > 0 ? at : 0, n);
        if constexpr (NORM) load_raw(wt[i], (const T*)a.w + (n > 0 ? at * VEC : 0), n);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t at = (int64_t)i * TPR + t;
        const int64_t left = a.k - at * VEC;
        const int n = left < VEC ? (left < 0 ? 0 : (int)left) : VEC;
        if (a.res) store8((T*)a.res_out + r * a.res_out_stride + at * VEC, v[i], n);
        if constexpr (NORM) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sq[i] += (double)v[i][j] * (double)v[i][j];
        }
    }
    if constexpr (NORM) {
        const float inv = inv_rms(row_sum<TPR>(sq, lds_sum), a.k, a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i][j] = (v[i][j] * inv) * to_f32(wt[i][j]);
        }
    }
    float d = 0.0f;
    if (a.q) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) m = larger(m, magnitude(v[i][j]));
        }
        m = row_max<TPR>(m, lds_max);
        d = __uint_as_float(m) / 127.0f;
        if (t == 0) a.scale[r] = d;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t at = (int64_t)i * TPR + t;
        const int64_t left = a.k - at * VEC;
        const int n = left < VEC ? (left < 0 ? 0 : (int)left) : VEC;
        if (n > 0) store_codes(a, v[i], r, at, n, d);
    }
}

// Rows longer than the registers of one block hold: three passes over the row
// (53248 values in bf16 with a residual: one row 18 us, 1000 rows 115, 3.2 TB/s;
// without the norm, in two passes, 6.5 and 43 us, 3.7 TB/s).  Each thread comes back to its own vectors, and residual_out is written
// in the last pass, so it may be the residual or x itself.
template <typename T, bool NORM>
__global__ __launch_bounds__(1024) void k_norm_q8_long(NormArgs a) {
    __shared__ double lds_sum[16];
    __shared__ uint32_t lds_max[16];
    const int64_t r = blockIdx.x;
    const int64_t nvec = (a.k + VEC - 1) / VEC;
    float inv = 1.0f;
    if constexpr (NORM) {
        double sq[1] = {};
        for (int64_t at = threadIdx.x; at < nvec; at += 1024) {
            float v[VEC];
            const int n = (int)(a.k - at * VEC < VEC ? a.k - at * VEC : VEC);
            load_sum<T>(v, a, r, at, n);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sq[0] += (double)v[j] * (double)v[j];
        }
        inv = inv_rms(row_sum<1024>(sq, lds_sum), a.k, a.eps);
    }
    auto row_y = [&](float (&v)[VEC], int64_t at, int n) {
        load_sum<T>(v, a, r, at, n);
        if constexpr (NORM) {
            float w[VEC];
            load8(w, (const T*)a.w + at * VEC, n);
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = (v[j] * inv) * w[j];
        }
    };
    float d = 0.0f;
    if (a.q) {
        uint32_t m = 0u;
        for (int64_t at = threadIdx.x; at < nvec; at += 1024) {
            float v[VEC];
            const int n = (int)(a.k - at * VEC < VEC ? a.k - at * VEC : VEC);
            row_y(v, at, n);
#pragma unroll
            for (int j = 0; j < VEC; ++j) m = larger(m, magnitude(v[j]));
        }
        m = row_max<1024>(m, lds_max);
        d = __uint_as_float(m) / 127.0f;
        if (threadIdx.x == 0) a.scale[r] = d;
    }
    for (int64_t at = threadIdx.x; at < nvec; at += 1024) {
        float v[VEC], s[VEC];
        const int n = (int)(a.k - at * VEC < VEC ? a.k - at * VEC : VEC);
        row_y(v, at, n);
        if (a.res) {
            load_sum<T>(s, a, r, at, n);
            store8((T*)a.res_out + r * a.res_out_stride + at * VEC, s, n);
        }
        store_codes(a, v, r, at, n, d);
    }
}

template <typename T, bool NORM, int TPR, int NV>
int launch(const NormArgs& a, hipStream_t stream) {
    constexpr int RPB = TPR == 64 ? 4 : 1;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    if (blocks > most_blocks(RPB * TPR)) return MOEQ8_EUNSUPPORTED;
    hipLaunchKernelGGL((k_norm_q8<T, NORM, TPR, NV>), dim3((uint32_t)blocks), dim3(RPB * TPR), 0, stream, a);
    return check_launch();
}

template <typename T, bool NORM>
int launch_rows(const NormArgs& a, hipStream_t stream) {
    // Few rows: the time is that of one row, so a thread takes as few vectors as
    // 1024 threads allow (64 x 8192 bf16 in 512 x 2 and 1024 x 1: 4.9 and 4.5 us).
    // Many: what counts is the work of a CU, in which vectors past a row's end
    // cost as much as others, and smaller blocks wait less at their barriers
    // (4000 x 8192 in the same two: 47.4 and 49.3 us; 600 x 10304 in 512 x 3 and
    // 1024 x 2: 13.1 and 15.1; 16000 x 1504 in 128 x 2 and 256 x 1: 33.8 and 36.8,
    // but 600 rows of them 5.5 and 4.8).
    const bool many = a.rows > 512;
    if (a.k <= 512) return launch<T, NORM, 64, 1>(a, stream);
    if (a.k <= 1024) return launch<T, NORM, 128, 1>(a, stream);
    if (a.k <= 2048) return a.rows > 2048 ? launch<T, NORM, 128, 2>(a, stream) : launch<T, NORM, 256, 1>(a, stream);
    if (a.k <= 4096) return many ? launch<T, NORM, 256, 2>(a, stream) : launch<T, NORM, 512, 1>(a, stream);
    if (a.k <= 6144 && many) return launch<T, NORM, 256, 3>(a, stream);
    if (a.k <= 8192) return many ? launch<T, NORM, 512, 2>(a, stream) : launch<T, NORM, 1024, 1>(a, stream);
    if (a.k <= 12288 && many) return launch<T, NORM, 512, 3>(a, stream);
    if (a.k <= 16384) return launch<T, NORM, 1024, 2>(a, stream);
    if (a.k <= 32768) return launch<T, NORM, 1024, 4>(a, stream);
    if (a.rows > most_blocks(1024)) return MOEQ8_EUNSUPPORTED;
    hipLaunchKernelGGL((k_norm_q8_long<T, NORM>), dim3((uint32_t)a.rows), dim3(1024), 0, stream, a);
    return check_launch();
}

template <bool NORM>
int launch_dtype(int32_t dtype, const NormArgs& a, void* stream) {
    switch (dtype) {
        case MOEQ8_F32: return launch_rows<float, NORM>(a, (hipStream_t)stream);
        case MOEQ8_F16: return launch_rows<f16_t, NORM>(a, (hipStream_t)stream);
        default: return launch_rows<bf16_t, NORM>(a, (hipStream_t)stream);
    }
}

}  // namespace
}  // namespace moeq8

extern "C" int rms_norm_q8(const void* x, int64_t x_row_stride, const void* residual, int64_t residual_row_stride,
                           void* residual_out, int64_t residual_out_row_stride, const void* w, int32_t dtype,
                           int64_t n_rows, int64_t k, double eps, int8_t* q, int64_t q_row_stride, float* scale,
                           void* xq, void* stream) {
    using namespace moeq8;
    if (dtype < MOEQ8_F32 || dtype > MOEQ8_BF16 || n_rows < 0 || k <= 0 || !(eps >= 0.0)) return MOEQ8_EINVAL;
    if (!x || !w || (!q && !xq) || !q != !scale || !residual != !residual_out) return MOEQ8_EINVAL;
    if (x_row_stride < k || (residual && (residual_row_stride < k || residual_out_row_stride < k)) ||
        (q && q_row_stride < k) || (xq && k % QK != 0))
        return MOEQ8_EINVAL;
    const int es = dtype_bytes(dtype);
    if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)residual | (uintptr_t)residual_out) & (uintptr_t)(es - 1))
        return MOEQ8_EALIGN;
    if (((uintptr_t)scale | (uintptr_t)xq) & 3u) return MOEQ8_EALIGN;
    if (n_rows == 0) return MOEQ8_OK;
    if (residual && (rows_clash(x, x_row_stride * es, residual_out, residual_out_row_stride * es, n_rows, k * es) ||
                     rows_clash(residual, residual_row_stride * es, residual_out, residual_out_row_stride * es, n_rows, k * es)))
        return MOEQ8_EINVAL;
    NormArgs a{x, x_row_stride, residual, residual_row_stride, residual_out, residual_out_row_stride, w,
               n_rows, k, eps, q, q_row_stride, scale, (uint8_t*)xq};
    return launch_dtype<true>(dtype, a, stream);
}

extern "C" int i8_quantize_rows(const void* x, int32_t dtype, int64_t n_rows, int64_t k, int64_t x_row_stride,
                                int8_t* q, int64_t q_row_stride, float* scale, void* stream) {
    using namespace moeq8;
    if (dtype < MOEQ8_F32 || dtype > MOEQ8_BF16 || n_rows < 0 || k <= 0 || !x || !q || !scale ||
        x_row_stride < k || q_row_stride < k)
        return MOEQ8_EINVAL;
    if ((uintptr_t)x & (uintptr_t)(dtype_bytes(dtype) - 1)) return MOEQ8_EALIGN;
    if ((uintptr_t)scale & 3u) return MOEQ8_EALIGN;
    if (n_rows == 0) return MOEQ8_OK;
    NormArgs a{x, x_row_stride, nullptr, 0, nullptr, 0, nullptr, n_rows, k, 0.0, q, q_row_stride, scale, nullptr};
    return launch_dtype<false>(dtype, a, stream);
}

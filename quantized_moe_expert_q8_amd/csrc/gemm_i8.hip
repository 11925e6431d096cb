// Product of int8 rows with a scale for each token (row of a) and each output
// channel (row of b):
//
//   out[i, j] = T(fp32(sum_k a[i, k] * b[j, k]) * sa[i] * sb[j] + bias[j])
//
// The sum is exact in int32 for k < 131072 (|code| <= 128), so no order of it
// changes a result; it is rounded once to fp32, and the two scales, the bias
// and the output type round once each.
#include "moeq8_types.hpp"
#include "moeq8_host.hpp"

namespace moeq8 {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

struct GemmArgs {
    const int8_t* a; int64_t a_stride;
    const int8_t* b; int64_t b_stride;
    const float* sa;
    const float* sb;
    const float* bias;                            // null: none
    void* out; int64_t out_stride;
    int64_t m, n, k;
};

// 16 bytes from byte k0 of a row of k bytes, zeros past its end.
__device__ __forceinline__ i32x4 load_piece(const int8_t* row, int64_t k0, int64_t k) {
    union { i32x4 v; u32x4b u; int8_t c[16]; } t;
    t.v = i32x4{0, 0, 0, 0};
    if (k0 + 16 <= k) {
        t.u = *reinterpret_cast<const u32x4b*>(row + k0);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (k0 + i < k) t.c[i] = row[k0 + i];
    }
    return t.v;
}

// Four consecutive channels j .. j + 3 of token i.
template <typename T>
__device__ __forceinline__ void store_quad(const GemmArgs& g, int64_t i, int64_t j, i32x4 acc) {
    if (i >= g.m) return;
    const float sa = g.sa[i];
    T* o = (T*)g.out + i * g.out_stride + j;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (j + e >= g.n) break;
        float v = ((float)acc[e] * sa) * g.sb[j + e];
        if (g.bias) v += g.bias[j + e];
        from_f32(o[e], v);
    }
}

// A tile of 64 tokens x 64 channels, 64 values of k at a time through LDS.
// The weights are the matrix instruction's first operand: a lane then holds
// four consecutive channels of one token, which lie together in out.
template <typename T>
__global__ __launch_bounds__(256) void k_gemm_i8(GemmArgs g) {
    constexpr int ROW = 80;                        // 64 bytes of k and 16 of padding
    __shared__ __attribute__((aligned(16))) int8_t la[64 * ROW];
    __shared__ __attribute__((aligned(16))) int8_t lb[64 * ROW];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t n_tiles = (g.n + 63) / 64;
    const int64_t i0 = blockIdx.x / n_tiles * 64, j0 = blockIdx.x % n_tiles * 64;
    const int64_t ar = i0 + t / 4 < g.m ? i0 + t / 4 : g.m - 1;
    const int64_t br = j0 + t / 4 < g.n ? j0 + t / 4 : g.n - 1;
    const int wi = (wave & 1) * 32, wj = (wave >> 1) * 32;
    i32x4 acc[2][2] = {};
    for (int64_t k0 = 0; k0 < g.k; k0 += 64) {
        const i32x4 pa = load_piece(g.a + ar * g.a_stride, k0 + t % 4 * 16, g.k);
        const i32x4 pb = load_piece(g.b + br * g.b_stride, k0 + t % 4 * 16, g.k);
        __syncthreads();
        *reinterpret_cast<i32x4*>(la + t / 4 * ROW + t % 4 * 16) = pa;
        *reinterpret_cast<i32x4*>(lb + t / 4 * ROW + t % 4 * 16) = pb;
        __syncthreads();
        i32x4 fa[2], fb[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int off = (16 * s + lane % 16) * ROW + lane / 16 * 16;
            fa[s] = *reinterpret_cast<const i32x4*>(la + wi * ROW + off);
            fb[s] = *reinterpret_cast<const i32x4*>(lb + wj * ROW + off);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                acc[s][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u], fa[s], acc[s][u], 0, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u)
            store_quad<T>(g, i0 + wi + 16 * s + lane % 16, j0 + wj + 16 * u + lane / 16 * 4, acc[s][u]);
}

template <typename T>
int launch_gemm(const GemmArgs& g, hipStream_t stream) {
    const int64_t blocks = ((g.m + 63) / 64) * ((g.n + 63) / 64);
    if (blocks > 0x7fffffff) return MOEQ8_EUNSUPPORTED;
    hipLaunchKernelGGL(k_gemm_i8<T>, dim3((uint32_t)blocks), dim3(256), 0, stream, g);
    return check_launch();
}

}  // namespace
}  // namespace moeq8

extern "C" int gemm_i8(const int8_t* a, int64_t a_row_stride, const float* sa, const int8_t* b, int64_t b_row_stride,
                       const float* sb, const float* bias, int64_t m, int64_t n, int64_t k, int32_t out_dtype,
                       void* out, int64_t out_row_stride, void* stream) {
    using namespace moeq8;
    if (!a || !sa || !b || !sb || !out || m < 0 || n < 0 || k <= 0) return MOEQ8_EINVAL;
    if (out_dtype < MOEQ8_F32 || out_dtype > MOEQ8_BF16) return MOEQ8_EINVAL;
    if (a_row_stride < k || b_row_stride < k || out_row_stride < n) return MOEQ8_EINVAL;
    if (k > MOEQ8_MAX_I8_K) return MOEQ8_EUNSUPPORTED;
    if (((uintptr_t)sa | (uintptr_t)sb | (uintptr_t)bias) & 3u) return MOEQ8_EALIGN;
    if ((uintptr_t)out & (uintptr_t)(dtype_bytes(out_dtype) - 1)) return MOEQ8_EALIGN;
    if (m == 0 || n == 0) return MOEQ8_OK;
    const GemmArgs g{a, a_row_stride, b, b_row_stride, sa, sb, bias, out, out_row_stride, m, n, k};
    switch (out_dtype) {
        case MOEQ8_F32: return launch_gemm<float>(g, (hipStream_t)stream);
        case MOEQ8_F16: return launch_gemm<f16_t>(g, (hipStream_t)stream);
        default: return launch_gemm<bf16_t>(g, (hipStream_t)stream);
    }
}

// Product of int8 rows with a scale for each token (row of a) and each output
// channel (row of b):
//
//   out[i, j] = T(fp32(sum_k a[i, k] * b[j, k]) * sa[i] * sb[j] + bias[j])
//
// The sum is exact in int32 for k < 131072 (|code| <= 128), so no order of it
// changes a result; it is rounded once to fp32, and the two scales, the bias
// and the output type round once each.
#include "moeq8_lds.hpp"
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

// Bytes of the 16-byte piece p of a row of k >= 16 bytes: loaded from byte
// piece_at(p, k), which for the row's last, cut piece is its last 16 bytes and
// never past its end; drop_head then clears the bytes in front of the piece
// (all of them where the piece lies past the row).  One operand cleared is
// enough, so the weights' pieces are left as loaded.
__device__ __forceinline__ int64_t piece_at(int64_t p, int64_t k) { return 16 * p <= k - 16 ? 16 * p : k - 16; }

__device__ __forceinline__ i32x4 drop_head(i32x4 v, int64_t p, int64_t k) {
    const int64_t over = 16 * p - (k - 16);        // bytes to clear
    if (over <= 0) return v;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int c = (int)(over < 16 ? over : 16) - 4 * d;
        if (c >= 4) v[d] = 0;
        else if (c > 0) v[d] = (int)((uint32_t)v[d] & (0xffffffffu << (8 * c)));
    }
    return v;
}

// Few tokens (MT tiles of 16): the weights are read once from memory and are
// what the time goes to.  A block of 8 waves takes tiles of 16 channels; the
// waves split k, each keeping its part of the tokens' rows in registers over
// all tiles of the block, so that nothing but weights is loaded in the loop
// (16 rows x 64 bytes an instruction, straight into the matrix instruction's
// layout).  The next tile's weights are in flight while the waves' sums are
// added through LDS.  A wave takes `steps` steps of 64 values (NS at most) a
// chunk; rows longer than 8 waves x NS steps are taken in chunks, with the
// tokens' part loaded for each.
//
// 5 x 131072 x 4096: 95 us, 5.7 TB/s (the 64 x 64 tiles below: 132 us);
// 1 x 4096 x 4096: 5.8 us in a graph (29 us), where the launch and one trip to
// memory are most of it.
template <typename T, int MT, int NS>
__global__ __launch_bounds__(512) void k_gemm_i8_few(GemmArgs g, int steps, int chunks) {
    constexpr int ROW = 20;                        // 16 sums and padding against bank conflicts
    __shared__ __attribute__((aligned(16))) int32_t part[2][8][MT][16 * ROW];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, quarter = lane >> 4;
    const int64_t tiles = (g.n + 15) / 16, all_steps = (g.k + 63) / 64;
    i32x4 act[MT][NS], w[NS];
    auto first_step = [&](int c) { return ((int64_t)c * 8 + wave) * steps; };
    auto own_steps = [&](int c) {                  // steps of the wave that lie inside the row
        const int64_t left = all_steps - first_step(c);
        return (int)(left < steps ? (left < 0 ? 0 : left) : steps);
    };
    auto load_act = [&](int c) {
        const int own = own_steps(c);
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const int64_t row = 16 * u + r < g.m ? 16 * u + r : g.m - 1;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                act[u][i] = i32x4{0, 0, 0, 0};
                if (i < own) {
                    const int64_t p = (first_step(c) + i) * 4 + quarter;
                    const u32x4b v = *reinterpret_cast<const u32x4b*>(g.a + row * g.a_stride + piece_at(p, g.k));
                    act[u][i] = drop_head((i32x4)v, p, g.k);
                }
            }
        }
    };
    auto load_w = [&](int64_t tile, int c) {
        const int own = own_steps(c);
        const int64_t row = tile * 16 + r < g.n ? tile * 16 + r : g.n - 1;
        const int8_t* base = g.b + row * g.b_stride;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (i < own)
                w[i] = (i32x4) * reinterpret_cast<const u32x4b*>(base + piece_at((first_step(c) + i) * 4 + quarter, g.k));
    };
    int64_t tile = blockIdx.x;
    int c = 0, buf = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) w[i] = i32x4{0, 0, 0, 0};
    load_w(tile, 0);
    load_act(0);
    i32x4 acc[MT] = {};
    constexpr int PER = (MT * 256 + 511) / 512;    // outputs of a thread
    while (true) {
        // scales of this thread's outputs: token e / 16, channel e % 16 of the tile
        float sa[PER], sb[PER], bias[PER];
        const bool last = c == chunks - 1;
        if (last) {
#pragma unroll
            for (int o = 0; o < PER; ++o) {
                const int e = threadIdx.x + 512 * o;
                const int64_t i = e >> 4, j = tile * 16 + (e & 15);
                const bool in = e < MT * 256 && i < g.m && j < g.n;
                sa[o] = in ? g.sa[i] : 0.0f;
                sb[o] = in ? g.sb[j] : 0.0f;
                bias[o] = in && g.bias ? g.bias[j] : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int u = 0; u < MT; ++u) acc[u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], act[u][i], acc[u], 0, 0, 0);
        const int64_t this_tile = tile;
        if (last) { tile += gridDim.x; c = 0; } else { ++c; }
        if (tile < tiles) {
            load_w(tile, c);
            if (chunks > 1) load_act(c);
        }
        if (last) {
#pragma unroll
            for (int u = 0; u < MT; ++u) {
                *reinterpret_cast<i32x4*>(&part[buf][wave][u][r * ROW + quarter * 4]) = acc[u];
                acc[u] = i32x4{0, 0, 0, 0};
            }
            lds_barrier();
#pragma unroll
            for (int o = 0; o < PER; ++o) {
                const int e = threadIdx.x + 512 * o;
                const int64_t i = e >> 4, j = this_tile * 16 + (e & 15);
                if (e < MT * 256 && i < g.m && j < g.n) {
                    int32_t sum = 0;
#pragma unroll
                    for (int v = 0; v < 8; ++v) sum += part[buf][v][e >> 8][((e >> 4) & 15) * ROW + (e & 15)];
                    float f = ((float)sum * sa[o]) * sb[o];
                    if (g.bias) f += bias[o];
                    from_f32(((T*)g.out)[i * g.out_stride + j], f);
                }
            }
            buf ^= 1;                              // the other buffer is free: all waves are past its reads
            if (tile >= tiles) break;
        }
    }
}

template <typename T, int MT, int NS>
int launch_few_steps(const GemmArgs& g, int steps, int chunks, hipStream_t stream) {
    // two blocks of 8 waves a CU, all with the same number of tiles (or one less)
    const int64_t tiles = (g.n + 15) / 16, rounds = (tiles + 511) / 512;
    const int64_t blocks = (tiles + rounds - 1) / rounds;
    hipLaunchKernelGGL((k_gemm_i8_few<T, MT, NS>), dim3((uint32_t)blocks), dim3(512), 0, stream, g, steps, chunks);
    return check_launch();
}

template <typename T, int MT>
int launch_few(const GemmArgs& g, hipStream_t stream) {
    constexpr int MAX_NS = MT == 1 ? 16 : 8;       // the tokens' part and the weights within 256 registers
    const int64_t all = (g.k + 63) / 64, chunks = (all + 8 * MAX_NS - 1) / (8 * MAX_NS);
    const int steps = (int)(((all + chunks - 1) / chunks + 7) / 8);
    if (steps <= 1) return launch_few_steps<T, MT, 1>(g, steps, (int)chunks, stream);
    if (steps <= 2) return launch_few_steps<T, MT, 2>(g, steps, (int)chunks, stream);
    if (steps <= 4) return launch_few_steps<T, MT, 4>(g, steps, (int)chunks, stream);
    if (steps <= 8) return launch_few_steps<T, MT, 8>(g, steps, (int)chunks, stream);
    return launch_few_steps<T, MT, MAX_NS>(g, steps, (int)chunks, stream);
}

template <typename T>
int launch_gemm(const GemmArgs& g, hipStream_t stream) {
    if (g.k >= 16 && g.m <= 16) return launch_few<T, 1>(g, stream);
    if (g.k >= 16 && g.m <= 32) return launch_few<T, 2>(g, stream);
    if (g.k >= 16 && g.m <= 64) return launch_few<T, 4>(g, stream);
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

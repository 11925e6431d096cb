// Product of int8 rows with a scale for each token (row of a) and each output
// channel (row of b):
//
//   out[i, j] = T(fp32(sum_k a[i, k] * b[j, k]) * sa[i] * sb[j] + bias[j])
//
// The sum is exact in int32 for k < 131072 (|code| <= 128), so no order of it
// changes a result; it is rounded once to fp32, and the two scales, the bias
// and the output type round once each.
#include <type_traits>
#include "moeq8_lds.hpp"
#include "moeq8_types.hpp"
#include "moeq8_host.hpp"

namespace moeq8 {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_by4 __attribute__((ext_vector_type(4), aligned(4), may_alias));

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

// Scales and biases of four consecutive channels j .. j + 3, loaded ahead of
// their use: a load at the end of a kernel is a trip to memory that nothing
// hides (333 x 2047 x 4096 with a bias: 12.5 us, loaded ahead 10.5).
struct Channels {
    float sb[4], bias[4];
    __device__ __forceinline__ void load(const GemmArgs& g, int64_t j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t c = j + e < g.n ? j + e : g.n - 1;
            sb[e] = g.sb[c];
            bias[e] = g.bias ? g.bias[c] : 0.0f;
        }
    }
};

// Four consecutive channels j .. j + 3 of token i.
template <typename T>
__device__ __forceinline__ void store_quad(const GemmArgs& g, int64_t i, int64_t j, i32x4 acc, float sa, const Channels& c) {
    if (i >= g.m) return;
    T* o = (T*)g.out + i * g.out_stride + j;
    union { T e[4]; u32x4b q; u32x2b d; } t;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float v = ((float)acc[e] * sa) * c.sb[e];
        if (g.bias) v += c.bias[e];
        from_f32(t.e[e], v);
    }
    if (j + 4 <= g.n) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<u32x4b*>(o) = t.q;
        else *reinterpret_cast<u32x2b*>(o) = t.d;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < g.n) o[e] = t.e[e];
    }
}

__device__ __forceinline__ float token_scale(const GemmArgs& g, int64_t i) { return g.sa[i < g.m ? i : g.m - 1]; }

// Rows of fewer than 16 values, and rows too far apart for the kernels below:
// a tile of 64 tokens x 64 channels, 64 values of k at a time through LDS.
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
        for (int u = 0; u < 2; ++u) {
            const int64_t i = i0 + wi + 16 * s + lane % 16, j = j0 + wj + 16 * u + lane / 16 * 4;
            Channels c;
            c.load(g, j);
            store_quad<T>(g, i, j, acc[s][u], token_scale(g, i), c);
        }
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

// 16 bytes at an address that is no multiple of 4, as the 4 dwords it begins in
// and the one it ends in, each of which holds one of its bytes and so lies in
// the row's allocation.  Loaded as they lie, from lanes whose neighbours read
// other rows, such vectors cost many times an aligned one: 14 x 71 x 3305 8.8
// and 6.1 us, 1 x 19623 x 3710 38 and 26.  (Where the lanes of a row lie
// together, as in the tiles below, they cost less than these two loads.)
struct OddPiece {
    i32x4 v;
    int32_t last;
    __device__ __forceinline__ void load(const int8_t* p) {
        const uintptr_t at = (uintptr_t)p;
        v = *reinterpret_cast<const i32x4_by4*>(at & ~(uintptr_t)3);
        last = *reinterpret_cast<const int32_t*>((at + 15) & ~(uintptr_t)3);
    }
    __device__ __forceinline__ i32x4 piece(uint32_t shift) const {     // shift: the address modulo 4 in its low two bits
        return i32x4{(int)__builtin_amdgcn_alignbyte((uint32_t)v[1], (uint32_t)v[0], shift),
                     (int)__builtin_amdgcn_alignbyte((uint32_t)v[2], (uint32_t)v[1], shift),
                     (int)__builtin_amdgcn_alignbyte((uint32_t)v[3], (uint32_t)v[2], shift),
                     (int)__builtin_amdgcn_alignbyte((uint32_t)last, (uint32_t)v[3], shift)};
    }
};

// At most 16 tokens: the weights are read once from memory and are what the
// time goes to.  The W waves of a block form groups of KW; a group takes TP
// tiles of 16 channels at a time and its waves split k, each keeping its part
// of the tokens' rows in registers over all tiles of the block, so that
// nothing but weights is loaded in the loop (16 rows x 64 bytes an
// instruction, straight into the matrix instruction's layout).  The next
// tiles' weights are in flight while the waves' sums are added through LDS.  A
// wave takes `steps` steps of 64 values (NS at most) a chunk; rows longer than
// KW waves x NS steps are taken in chunks, with the tokens' part loaded for each.
//
// 5 x 131072 x 4096: 90 us, 6.0 TB/s (64 x 64 tiles: 132 us); 1 x 4096 x 4096:
// 5.2 us in a graph (29 us), where the launch and one trip to memory are most
// of it.
template <typename T, int W, int KW, int NS, int TP, bool ODD>
__global__ __launch_bounds__(W * 64) void k_gemm_i8_few(GemmArgs g, int steps, int chunks) {
    constexpr int ROW = 20;                        // 16 sums and padding against bank conflicts
    constexpr int G = W / KW, PER = (TP * 256 + KW * 64 - 1) / (KW * 64);      // groups, outputs of a thread
    __shared__ __attribute__((aligned(16))) int32_t part[KW > 1 ? 2 : 1][KW > 1 ? W : 1][KW > 1 ? TP : 1][16 * ROW];
    const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) % KW, group = (threadIdx.x >> 6) / KW;
    const int r = lane & 15, quarter = lane >> 4;
    const int64_t rounds = (g.n + 16 * G * TP - 1) / (16 * G * TP), all_steps = (g.k + 63) / 64;
    static_assert(TP * NS <= 16, "two bits of shift a piece");
    i32x4 act[NS], w[TP][NS];
    int32_t w_last[ODD ? TP : 1][NS];              // with ODD: the rest of OddPiece, and all pieces' shifts
    uint32_t w_shift = 0;
    auto first_step = [&](int c) { return ((int64_t)c * KW + wave) * steps; };
    auto own_steps = [&](int c) {                  // steps of the wave that lie inside the row
        const int64_t left = all_steps - first_step(c);
        return (int)(left < steps ? (left < 0 ? 0 : left) : steps);
    };
    auto load_act = [&](int c) {
        const int own = own_steps(c);
        const int8_t* base = g.a + (r < g.m ? r : g.m - 1) * g.a_stride;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            act[i] = i32x4{0, 0, 0, 0};
            if (i < own) {
                const int64_t p = (first_step(c) + i) * 4 + quarter;
                const int8_t* at = base + piece_at(p, g.k);
                if constexpr (ODD) {
                    OddPiece o;
                    o.load(at);
                    act[i] = o.piece((uint32_t)(uintptr_t)at);
                } else {
                    act[i] = *reinterpret_cast<const i32x4_by4*>(at);
                }
                act[i] = drop_head(act[i], p, g.k);
            }
        }
    };
    // Of each 256 rounds, blocks of one XCD (every 8th) take 32 that follow each
    // other, so that the parts of a line of out meet in one L2 (where a round is
    // less than a line: 5 x 131072 x 4096 f32 90 and 95.5 us, 8 tokens bf16 94 and
    // 103; with 8 of each 64 1% slower).
    const int64_t whole = G * TP < 4 ? rounds / 256 * 256 : 0;
    auto channel = [&](int64_t round, int u) {
        if (round < whole) round = (round & ~(int64_t)255) + (round & 7) * 32 + (round >> 3 & 31);
        return ((round * G + group) * TP + u) * 16;
    };
    auto load_w = [&](int64_t round, int c) {
        const int own = own_steps(c);
        w_shift = 0;
#pragma unroll
        for (int u = 0; u < TP; ++u) {
            const int64_t j = channel(round, u) + r;
            const int8_t* base = g.b + (j < g.n ? j : g.n - 1) * g.b_stride;
#pragma unroll
            for (int i = 0; i < NS; ++i)
                if (i < own) {
                    const int8_t* at = base + piece_at((first_step(c) + i) * 4 + quarter, g.k);
                    if constexpr (ODD) {
                        OddPiece o;
                        o.load(at);
                        w[u][i] = o.v;
                        w_last[u][i] = o.last;
                        w_shift |= ((uint32_t)(uintptr_t)at & 3) << (2 * (u * NS + i));
                    } else {
                        w[u][i] = *reinterpret_cast<const i32x4_by4*>(at);
                    }
                }
        }
    };
    int64_t round = blockIdx.x;
    int c = 0, buf = 0;
#pragma unroll
    for (int u = 0; u < TP; ++u)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            w[u][i] = i32x4{0, 0, 0, 0};
            if constexpr (ODD) w_last[u][i] = 0;
        }
    load_w(round, 0);
    load_act(0);
    i32x4 acc[TP] = {};
    // output e of the group: token e / 16 % 16 of channel e % 16 of tile e / 256
    const int first_out = threadIdx.x % (KW * 64);
    while (true) {
        const bool last = c == chunks - 1;
        const int64_t this_round = round;
        float sa[PER], sb[PER], bias[PER];
        Channels own[KW == 1 ? TP : 1];
        if constexpr (KW == 1) {
            sa[0] = token_scale(g, r);
#pragma unroll
            for (int u = 0; u < TP; ++u) own[u].load(g, channel(round, u) + quarter * 4);
        } else if (last) {
#pragma unroll
            for (int o = 0; o < PER; ++o) {
                const int e = first_out + o * KW * 64;
                const int64_t i = (e >> 4) & 15, j = channel(round, e >> 8) + (e & 15);
                const bool in = e < TP * 256 && i < g.m && j < g.n;
                sa[o] = in ? g.sa[i] : 0.0f;
                sb[o] = in ? g.sb[j] : 0.0f;
                bias[o] = in && g.bias ? g.bias[j] : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int u = 0; u < TP; ++u) {
                i32x4 x = w[u][i];
                if constexpr (ODD) x = OddPiece{x, w_last[u][i]}.piece(w_shift >> (2 * (u * NS + i)));
                acc[u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x, act[i], acc[u], 0, 0, 0);
            }
        if (last) { round += gridDim.x; c = 0; } else { ++c; }
        if (round < rounds) {
            load_w(round, c);
            if (chunks > 1) load_act(c);
        }
        if (last) {
            if constexpr (KW == 1) {
#pragma unroll
                for (int u = 0; u < TP; ++u) store_quad<T>(g, r, channel(this_round, u) + quarter * 4, acc[u], sa[0], own[u]);
            } else {
#pragma unroll
                for (int u = 0; u < TP; ++u)
                    *reinterpret_cast<i32x4*>(&part[buf][group * KW + wave][u][r * ROW + quarter * 4]) = acc[u];
                lds_barrier();
#pragma unroll
                for (int o = 0; o < PER; ++o) {
                    const int e = first_out + o * KW * 64;
                    const int64_t i = (e >> 4) & 15, j = channel(this_round, e >> 8) + (e & 15);
                    if (e < TP * 256 && i < g.m && j < g.n) {
                        int32_t sum = 0;
#pragma unroll
                        for (int v = 0; v < KW; ++v) sum += part[buf][group * KW + v][e >> 8][i * ROW + (e & 15)];
                        float f = ((float)sum * sa[o]) * sb[o];
                        if (g.bias) f += bias[o];
                        from_f32(((T*)g.out)[i * g.out_stride + j], f);
                    }
                }
                buf ^= 1;                          // the other buffer is free: all waves are past its reads
            }
#pragma unroll
            for (int u = 0; u < TP; ++u) acc[u] = i32x4{0, 0, 0, 0};
            if (round >= rounds) break;
        }
    }
}

// Whether every piece of every row begins at a multiple of 16 or of 4 bytes.
uint64_t row_bits(const GemmArgs& g) {
    return (uintptr_t)g.a | (uintptr_t)g.b | (uint64_t)g.a_stride | (uint64_t)g.b_stride | (uint64_t)g.k;
}
bool by_vectors(const GemmArgs& g) { return (row_bits(g) & 15) == 0; }
bool by_dwords(const GemmArgs& g) { return (row_bits(g) & 3) == 0; }

template <typename T, int W, int KW, int NS, int TP>
int launch_few_form(const GemmArgs& g, int chunks, hipStream_t stream) {
    // 16 waves a CU, the blocks with the same number of rounds (or one less)
    constexpr int64_t CHANNELS = 16 * (W / KW) * TP, MOST = 256 * (16 / W);
    const int64_t rounds = (g.n + CHANNELS - 1) / CHANNELS, each = (rounds + MOST - 1) / MOST;
    const int64_t blocks = (rounds + each - 1) / each, all = (g.k + 63) / 64;
    const int steps = (int)((all + (int64_t)chunks * KW - 1) / ((int64_t)chunks * KW));
    if (by_dwords(g))
        hipLaunchKernelGGL((k_gemm_i8_few<T, W, KW, NS, TP, false>), dim3((uint32_t)blocks), dim3(W * 64), 0, stream, g, steps, chunks);
    else
        hipLaunchKernelGGL((k_gemm_i8_few<T, W, KW, NS, TP, true>), dim3((uint32_t)blocks), dim3(W * 64), 0, stream, g, steps, chunks);
    return check_launch();
}

template <typename T>
int launch_few(const GemmArgs& g, hipStream_t stream) {
    const int64_t all = (g.k + 63) / 64;           // steps of 64 values
    // Each wave takes as few steps in a row as 8 waves allow; past 8 steps a wave
    // the registers of 16 waves a CU are full, so such rows get 16 waves.
    if (all > 64) return launch_few_form<T, 16, 16, 8, 1>(g, (int)((all + 127) / 128), stream);
    // More tiles than CUs: 16 waves too, which split a tile's rows finer (5 x 9000 x
    // 4096 13.6 and 11.5 us, 14 x 20000 x 2048 11.6 and 10.0; 1 x 4096 x 4096 5.35 and
    // 5.6; 5 x 100000 x 1088, whose 17 steps leave waves idle, 23 and 28).
    if (all > 32) {
        if (g.n > 4096) return launch_few_form<T, 16, 16, 4, 1>(g, 1, stream);
        return launch_few_form<T, 8, 8, 8, 1>(g, 1, stream);
    }
    if (all > 24 && g.n > 4096) return launch_few_form<T, 16, 16, 2, 1>(g, 1, stream);
    if (all > 16) return launch_few_form<T, 8, 8, 4, 1>(g, 1, stream);
    if (all > 8) return launch_few_form<T, 8, 8, 2, 1>(g, 1, stream);
    // Short rows leave a wave a load or two a tile, too few to keep memory busy
    // over many tiles: then it takes several (5 x 131072 x 512: 15.2 and 19.4 us,
    // but 8 x 6000 x 448 3.4 and 3.1), the shortest rows without splitting k (5 x
    // 131072 x 256: 10.3 and 17.0 us; 1 x 20000 x 256 5.6 and 4.7).
    if (all <= 4 && g.n > 32768) return launch_few_form<T, 8, 1, 4, 2>(g, 1, stream);
    if (g.n > 16384) return launch_few_form<T, 8, 8, 1, 4>(g, 1, stream);
    return launch_few_form<T, 8, 8, 1, 1>(g, 1, stream);
}

// Tile of block b.  Blocks are dealt to the 8 XCDs in turn; each XCD takes a
// contiguous range of the tiles, in groups of 8 token tiles by all channel
// tiles with the token tile fastest, so the tiles it works on at a time share
// rows of a and of b in its L2.
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t tiles_m, uint32_t tiles_n, int64_t& ti, int64_t& tj) {
    const uint32_t total = tiles_m * tiles_n, per = total / 8, extra = total % 8;
    const uint32_t x = b % 8, i = x * per + (x < extra ? x : extra) + b / 8;
    const uint32_t group = i / (8 * tiles_n), in = i - group * 8 * tiles_n;
    const uint32_t high = tiles_m - group * 8 < 8 ? tiles_m - group * 8 : 8;
    ti = __builtin_amdgcn_readfirstlane(group * 8 + in % high);
    tj = __builtin_amdgcn_readfirstlane(in / high);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

// Tiles of BM tokens x BN channels, WM x WN waves of FU x FV tiles of 32 x 32,
// 128 values of k a stage, ST stages in LDS.
//
// The 32x32x32 matrix instruction takes 32 cycles, so everything else is
// issued between two of them: at each of a stage's four steps the FU x FV
// products of the held fragments, with them the reads of the next step's
// fragments from LDS, and at the last step the loads of a stage into the
// buffer just read.  The barrier lies in front of that step: by then every
// wave has read all of the stage, and has waited for its own loads of the next
// one, which were issued ST - 1 stages earlier.
//
// A buffer holds BM rows of a, then BN rows of b, 128 bytes each; slot t of row
// r holds the row's 16-byte piece t ^ ((r >> 1) & 7), so that the lanes whose
// fragments LDS delivers together (0-3 with 12-15 and 20-27, 4-11 with 16-19
// and 28-31, and the same in the upper half) take 16 different bank groups.
// With DMA the loads go straight into LDS, which needs 16-byte aligned rows;
// otherwise they pass through registers, at any alignment, and ST is 2.
//
// 8192 x 8192 x 4096 in tiles of 256: 240 to 256 us by the card, 2150 to 2290
// TOP/s, the rate it holds in int8 products of this size (its clock falls under
// this load; right after a pause 290 us); the same with rows of 4097 bytes 315 us.
// The ends of the tiles, about 7 us each, are what keeps short rows below that:
// 8192 x 8192 x 1024 83 to 87 us, x 256 43 to 47 (its bytes take 27).
template <typename T, int WM, int WN, int FU, int FV, int ST, bool DMA>
__global__ __launch_bounds__(WM * WN * 64) void k_gemm_i8_tile(GemmArgs g) {
    constexpr int BM = WM * FU * 32, BN = WN * FV * 32, WAVES = WM * WN, STAGE = (BM + BN) * 128;
    constexpr int LA = BM / 8 / WAVES, LB = BN / 8 / WAVES, L = LA + LB;      // loads of 1 KB (8 rows) a wave and stage
    constexpr int N = FU * FV, R = FU + FV;        // products, fragment reads a step
    static_assert(LA * WAVES * 8 == BM && LB * WAVES * 8 == BN && (DMA || ST == 2), "whole loads");
    __shared__ __attribute__((aligned(1024))) int8_t ring[ST * STAGE];
    __shared__ __attribute__((aligned(16))) float lds_sa[BM], lds_sb[BN], lds_bias[BN];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t ti, tj;
    tile_of(blockIdx.x, (uint32_t)((g.m + BM - 1) / BM), (uint32_t)((g.n + BN - 1) / BN), ti, tj);
    const int64_t i0 = ti * BM, j0 = tj * BN;
    const int k = (int)g.k, steps = (k + 127) / 128;

    // this lane's rows and its piece of them; rows past the end are the last one
    auto piece_of = [&](int first) { return (lane & 7) ^ (((first + (lane >> 3)) >> 1) & 7); };
    auto first_row = [&](int u) { return u < LA ? (wave * LA + u) * 8 : (wave * LB + u - LA) * 8; };
    int32_t off[L];
#pragma unroll
    for (int u = 0; u < L; ++u) {
        const int64_t r = first_row(u) + (lane >> 3);
        const int64_t end = u < LA ? g.m - 1 - i0 : g.n - 1 - j0;
        off[u] = (int32_t)((r < end ? r : end) * (u < LA ? g.a_stride : g.b_stride) + piece_of(first_row(u)) * 16);
    }
    const int8_t* base_a = g.a + i0 * g.a_stride;
    const int8_t* base_b = g.b + j0 * g.b_stride;
    const uint32_t lds0 = (uint32_t)(uintptr_t)ring;
    auto slot_of = [&](int u) { return first_row(u) * 128 + (u < LA ? 0 : BM * 128); };
    // the last stage's pieces past the row are taken from its last 16 bytes
    // (which begin in front of that stage if fewer than 16 of its bytes are
    // left: an offset may be negative then, and with DMA never is)
    auto clamp_offsets = [&]() {
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int at = (steps - 1) * 128 + piece_of(first_row(u)) * 16;
            off[u] -= at > k - 16 ? at - (k - 16) : 0;
        }
    };
    i32x4 held[DMA ? 1 : L];
    auto load_one = [&](int u, int s, int buf) {   // load u of stage s
        const int8_t* base = (u < LA ? base_a : base_b) + (int64_t)s * 128;
        if constexpr (DMA) load_lds16_at(base, (uint32_t)off[u], lds0 + (uint32_t)buf * STAGE + slot_of(u));
        else held[u] = (i32x4) * reinterpret_cast<const u32x4b*>(base + off[u]);
    };
    auto put_one = [&](int u, int buf) {
        if constexpr (!DMA) *reinterpret_cast<i32x4*>(ring + buf * STAGE + slot_of(u) + lane * 16) = held[u];
    };

    const int fr = lane & 31, half = lane >> 5;
    const int wm = wave % WM * (FU * 32), wn = wave / WM * (FV * 32);
    auto read = [&](int buf, int row, int t) {     // this lane's fragment of step t: piece 2 t + half
        return *reinterpret_cast<const i32x4*>(ring + buf * STAGE + (row + fr) * 128 + ((2 * t + half) ^ ((fr >> 1) & 7)) * 16);
    };
    i32x16 acc[FU][FV] = {};
    i32x4 fa[2][FU], fb[2][FV];
    auto read_one = [&](int x, int at, int buf, int t) {
        if (x < FV) fb[at][x] = read(buf, BM + wn + 32 * x, t);
        else fa[at][x - FV] = read(buf, wm + 32 * (x - FV), t);
    };
    // step t of the stage in buffer buf; READ: with the reads of the next step's
    // fragments, at t = 3 from the buffer next; LOAD: with the loads of stage ahead
    auto step = [&](auto tc, auto readc, auto loadc, int buf, int next, int ahead) {
        constexpr int t = decltype(tc)::value;
        constexpr bool READ = decltype(readc)::value, LOAD = decltype(loadc)::value;
        constexpr int cur = t & 1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            acc[i / FV][i % FV] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[cur][i % FV], fa[cur][i / FV], acc[i / FV][i % FV], 0, 0, 0);
            if constexpr (READ) {
#pragma unroll
                for (int x = i * R / N; x < (i + 1) * R / N; ++x) read_one(x, cur ^ 1, t == 3 ? next : buf, (t + 1) & 3);
            }
            if constexpr (LOAD) {
#pragma unroll
                for (int x = i * L / N; x < (i + 1) * L / N; ++x) {
                    put_one(x, buf);
                    load_one(x, ahead, buf);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using std::integral_constant;
    using yes = integral_constant<bool, true>;
    using no = integral_constant<bool, false>;
    auto drop_tail = [&](int t) {                  // clear the tokens' values past the row's end
        if ((steps - 1) * 128 + 32 * t + 32 <= k) return;
#pragma unroll
        for (int u = 0; u < FU; ++u) fa[t & 1][u] = drop_head(fa[t & 1][u], (int64_t)(steps - 1) * 8 + 2 * t + half, k);
    };

    // the scales, on their way to LDS for the end, are not waited for here
    static_assert(BM <= WAVES * 64 && BN <= WAVES * 64, "one scale a thread");
    const int x = threadIdx.x;
    const int64_t scale_j = j0 + x < g.n ? j0 + x : g.n - 1;
    const float own_sa = token_scale(g, i0 + x), own_sb = g.sb[scale_j], own_bias = g.bias ? g.bias[scale_j] : 0.0f;
    // Stages past the last are the last one again, into buffers that no one
    // reads any more: a form of the step without loads would make the compiler
    // move the accumulators through memory.
    auto load_stage = [&](int s, int buf) {
        if (s == steps - 1) clamp_offsets();
#pragma unroll
        for (int u = 0; u < L; ++u) load_one(u, s < steps ? s : steps - 1, buf);
    };
    if constexpr (DMA) {
#pragma unroll
        for (int s = 0; s < ST; ++s) load_stage(s, s);
        wait_vm<(ST - 1) * L>();
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            load_stage(s, s);
#pragma unroll
            for (int u = 0; u < L; ++u) put_one(u, s);
        }
        load_stage(2, 0);
    }
    lds_barrier();
#pragma unroll
    for (int x = 0; x < R; ++x) read_one(x, 0, 0, 0);
    int buf = 0;
    constexpr int AHEAD = DMA ? ST : 3;
    for (int s = 0; s + 1 < steps; ++s) {
        const int next = buf + 1 < ST ? buf + 1 : 0;
        step(integral_constant<int, 0>{}, yes{}, no{}, buf, next, 0);
        step(integral_constant<int, 1>{}, yes{}, no{}, buf, next, 0);
        step(integral_constant<int, 2>{}, yes{}, no{}, buf, next, 0);
        if constexpr (DMA) wait_vm<(ST - 2) * L>();
        lds_barrier();
        if (s + AHEAD == steps - 1) clamp_offsets();
        step(integral_constant<int, 3>{}, yes{}, yes{}, buf, next, s + AHEAD < steps ? s + AHEAD : steps - 1);
        buf = next;
    }
    drop_tail(0);
    step(integral_constant<int, 0>{}, yes{}, no{}, buf, 0, 0);
    drop_tail(1);
    step(integral_constant<int, 1>{}, yes{}, no{}, buf, 0, 0);
    drop_tail(2);
    step(integral_constant<int, 2>{}, yes{}, no{}, buf, 0, 0);
    drop_tail(3);
    step(integral_constant<int, 3>{}, no{}, no{}, buf, 0, 0);
    wait_vm<0>();                                  // no load may reach LDS after the block has left it
    if (x < BM) lds_sa[x] = own_sa;
    if (x < BN) lds_sb[x] = own_sb, lds_bias[x] = own_bias;

    // A lane holds token fr of each 32 x 32 tile and channels 8 q + 4 half .. +
    // 3.  The wave turns 32 tokens at a time round through its own LDS, so that
    // it stores whole lines: its channels of a token lie together.  The barrier
    // is the last reads of the ring.
    lds_barrier();
    constexpr int ROW = FV * 32 * sizeof(T) + 16;  // padding against bank conflicts
    static_assert(WAVES * 32 * ROW <= ST * STAGE, "the ring's LDS");
    int8_t* own = ring + wave * (32 * ROW);
    constexpr int LANES = FV * 32 * sizeof(T) / 16;     // lanes of 16 bytes a row
    constexpr int PER = 16 / sizeof(T);            // channels of a lane
    const int64_t j = j0 + wn + lane % LANES * PER;
#pragma unroll
    for (int u = 0; u < FU; ++u) {
        const float sa = lds_sa[wm + 32 * u + fr];
#pragma unroll
        for (int v = 0; v < FV; ++v)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = 32 * v + 8 * q + 4 * half;
                const float4 sb = *reinterpret_cast<const float4*>(lds_sb + wn + c);
                float f[4] = {((float)acc[u][v][4 * q] * sa) * sb.x, ((float)acc[u][v][4 * q + 1] * sa) * sb.y,
                              ((float)acc[u][v][4 * q + 2] * sa) * sb.z, ((float)acc[u][v][4 * q + 3] * sa) * sb.w};
                if (g.bias) {
                    const float4 bi = *reinterpret_cast<const float4*>(lds_bias + wn + c);
                    f[0] += bi.x, f[1] += bi.y, f[2] += bi.z, f[3] += bi.w;
                }
                union { T e[4]; float4 q4; float2 d2; } t;
#pragma unroll
                for (int e = 0; e < 4; ++e) from_f32(t.e[e], f[e]);
                int8_t* to = own + fr * ROW + c * sizeof(T);
                if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(to) = t.q4;
                else *reinterpret_cast<float2*>(to) = t.d2;
            }
#pragma unroll
        for (int r = 0; r < 32; r += 64 / LANES) {
            const int row = r + lane / LANES;
            T e[PER];
            load_vec(e, (const T*)(own + row * ROW + lane % LANES * 16));
            const int64_t i = i0 + wm + 32 * u + row;
            if (i < g.m) {
                T* o = (T*)g.out + i * g.out_stride + j;
                if (j + PER <= g.n) {
                    store_vec(o, e);
                } else {
#pragma unroll
                    for (int x = 0; x < PER; ++x)
                        if (j + x < g.n) o[x] = e[x];
                }
            }
        }
    }
}

template <typename T, int WM, int WN, int FU, int FV, int ST>
int launch_tile(const GemmArgs& g, bool dma, hipStream_t stream) {
    constexpr int BM = WM * FU * 32, BN = WN * FV * 32;
    const int64_t blocks = ((g.m + BM - 1) / BM) * ((g.n + BN - 1) / BN);
    if (blocks > most_blocks(WM * WN * 64)) return MOEQ8_EUNSUPPORTED;
    if (dma)
        hipLaunchKernelGGL((k_gemm_i8_tile<T, WM, WN, FU, FV, ST, true>), dim3((uint32_t)blocks), dim3(WM * WN * 64), 0,
                           stream, g);
    else
        hipLaunchKernelGGL((k_gemm_i8_tile<T, WM, WN, FU, FV, 2, false>), dim3((uint32_t)blocks), dim3(WM * WN * 64), 0,
                           stream, g);
    return check_launch();
}

// Small tiles, of FU x FV tiles of 32 x 32: the 8 waves of a block split k, not
// the tile.  A stage is 32 values of k for each wave; every wave multiplies its
// part of it for the whole tile, so its products are FU x FV independent sums
// and a fragment is read from LDS once, where waves that split the tile would
// each wait for a short chain of products on the same few fragments.  The
// waves' sums are added through LDS at the end.  Stages go round ST buffers as
// above, with the reads of a whole stage one stage ahead of its products.
//
// 333 x 2047 x 4096 in tiles of 64: 10.5 us (waves that split the tile: 14 us).
// What bounds it is the fetch of a tile's rows by its CU: 64 bytes a clock
// (147 GB/s) from L2, about 80 GB/s where they come from memory.
//
// The swizzle: slot t of row r (256 bytes) holds piece t ^ (r & 15), which
// spreads the lanes that LDS serves together over all banks.
template <typename T, int FU, int FV, int ST, bool DMA>
__global__ __launch_bounds__(512) void k_gemm_i8_split(GemmArgs g) {
    constexpr int W = 8, BM = FU * 32, BN = FV * 32, KB = W * 32, STAGE = (BM + BN) * KB, SUMS = W * BM * BN * 4;
    constexpr int LDS = ST * STAGE > SUMS ? ST * STAGE : SUMS;
    constexpr int L = FU + FV;                     // loads of 1 KB a wave and stage, and fragments
    constexpr int LR = 1024 / KB, SLOTS = KB / 16; // rows a load, 16-byte slots a row
    static_assert(DMA || ST == 2, "");
    __shared__ __attribute__((aligned(1024))) int8_t ring[LDS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t ti, tj;
    tile_of(blockIdx.x, (uint32_t)((g.m + BM - 1) / BM), (uint32_t)((g.n + BN - 1) / BN), ti, tj);
    const int64_t i0 = ti * BM, j0 = tj * BN;
    const int k = (int)g.k, steps = (k + KB - 1) / KB;
    auto mix = [&](int r) { return r & 15; };

    // load u of the wave: rows of a for u < FU, of b for the others
    auto first_row = [&](int u) { return u < FU ? (wave * FU + u) * LR : (wave * FV + u - FU) * LR; };
    auto piece_of = [&](int u) { return (lane % SLOTS) ^ mix(first_row(u) + lane / SLOTS); };
    int32_t off[L];
#pragma unroll
    for (int u = 0; u < L; ++u) {
        const int64_t r = first_row(u) + lane / SLOTS;
        const int64_t end = u < FU ? g.m - 1 - i0 : g.n - 1 - j0;
        off[u] = (int32_t)((r < end ? r : end) * (u < FU ? g.a_stride : g.b_stride) + piece_of(u) * 16);
    }
    const int8_t* base_a = g.a + i0 * g.a_stride;
    const int8_t* base_b = g.b + j0 * g.b_stride;
    const uint32_t lds0 = (uint32_t)(uintptr_t)ring;
    auto slot_of = [&](int u) { return (first_row(u) + (u < FU ? 0 : BM)) * KB; };
    auto clamp_offsets = [&]() {                   // as in the kernel above
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int at = (steps - 1) * KB + piece_of(u) * 16;
            off[u] -= at > k - 16 ? at - (k - 16) : 0;
        }
    };
    // The blocks of an XCD begin at different stages of k (where none is cut), so
    // that they do not all ask the same memory channels at a time: 20 x 16384 x
    // 4096 15.4 and 17.6 us, 128 x 4096 x 4096 9.6 and 9.1.
    const int turn = DMA && k % KB == 0 ? (int)(blockIdx.x / 8) % steps : 0;
    i32x4 held[DMA ? 1 : L];
    auto load_stage = [&](int s, int buf) {
        if (s == steps - 1) clamp_offsets();
        int q = (s < steps ? s : steps - 1) + turn;
        if (q >= steps) q -= steps;
        const int64_t at = (int64_t)q * KB;
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int8_t* base = (u < FU ? base_a : base_b) + at;
            if constexpr (DMA) load_lds16_at(base, (uint32_t)off[u], lds0 + (uint32_t)buf * STAGE + slot_of(u));
            else held[u] = (i32x4) * reinterpret_cast<const u32x4b*>(base + off[u]);
        }
    };
    auto put_stage = [&](int buf) {
#pragma unroll
        for (int u = 0; u < (DMA ? 0 : L); ++u)
            *reinterpret_cast<i32x4*>(ring + buf * STAGE + slot_of(u) + lane * 16) = held[u];
    };

    const int fr = lane & 31, half = lane >> 5;
    i32x16 acc[FU][FV] = {};
    i32x4 fa[2][FU], fb[2][FV];
    const int own = fr * KB + ((2 * wave + half) ^ mix(fr)) * 16;   // this lane's piece of row fr
    auto read_stage = [&](int at, int buf) {
        const int8_t* st = ring + buf * STAGE + own;
#pragma unroll
        for (int v = 0; v < FV; ++v) fb[at][v] = *reinterpret_cast<const i32x4*>(st + (BM + 32 * v) * KB);
#pragma unroll
        for (int u = 0; u < FU; ++u) fa[at][u] = *reinterpret_cast<const i32x4*>(st + 32 * u * KB);
    };
    auto multiply = [&](int at) {
#pragma unroll
        for (int u = 0; u < FU; ++u)
#pragma unroll
            for (int v = 0; v < FV; ++v)
                acc[u][v] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[at][v], fa[at][u], acc[u][v], 0, 0, 0);
    };

    // a thread's outputs: quads of the same four channels, of every TOKENS-th token
    constexpr int QUADS = BN / 4, TOKENS = W * 64 / QUADS, OUTS = BM > TOKENS ? BM / TOKENS : 1;
    const int out_i = threadIdx.x / QUADS, out_q = threadIdx.x % QUADS;
    Channels channels;
    channels.load(g, j0 + out_q * 4);
    float sa[OUTS];
#pragma unroll
    for (int o = 0; o < OUTS; ++o) sa[o] = token_scale(g, i0 + out_i + o * TOKENS);

    constexpr int AHEAD = DMA ? ST : 3;
    if constexpr (DMA) {
#pragma unroll
        for (int s = 0; s < ST; ++s) load_stage(s, s);
        wait_vm<(ST - 1) * L>();
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            load_stage(s, s);
            put_stage(s);
        }
        load_stage(2, 0);
    }
    lds_barrier();
    read_stage(0, 0);
    int buf = 0;
    auto stage = [&](int at, int s) {              // stage s, held in set at, with the reads of the next one
        const int next = buf + 1 < ST ? buf + 1 : 0;
        if constexpr (DMA) wait_vm<(ST - 2) * L>();
        lds_barrier();
        read_stage(at ^ 1, next);
        put_stage(buf);
        load_stage(s + AHEAD, buf);
        multiply(at);
        buf = next;
    };
    int s = 0;
    for (; s + 2 < steps; s += 2) {
        stage(0, s);
        stage(1, s + 1);
    }
    if (s + 1 < steps) {                           // the last set is held in 0
        stage(0, s);
#pragma unroll
        for (int u = 0; u < FU; ++u) fa[0][u] = fa[1][u];
#pragma unroll
        for (int v = 0; v < FV; ++v) fb[0][v] = fb[1][v];
    }
    if (steps * KB > k) {
#pragma unroll
        for (int u = 0; u < FU; ++u) fa[0][u] = drop_head(fa[0][u], (int64_t)(steps - 1) * SLOTS + 2 * wave + half, k);
    }
    multiply(0);
    wait_vm<0>();                                  // no load may reach LDS after the ring's use
    lds_barrier();

    // [wave][token][channel]: quad of channels x of token i at x ^ (i & (BN / 4 - 1))
    int32_t* sums = reinterpret_cast<int32_t*>(ring);
    auto quad_at = [&](int w, int i, int x) { return ((w * BM + i) * QUADS + (x ^ (i & (QUADS - 1)))) * 4; };
#pragma unroll
    for (int u = 0; u < FU; ++u)
#pragma unroll
        for (int v = 0; v < FV; ++v)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<i32x4*>(sums + quad_at(wave, 32 * u + fr, 8 * v + 2 * q + half)) =
                    i32x4{acc[u][v][4 * q], acc[u][v][4 * q + 1], acc[u][v][4 * q + 2], acc[u][v][4 * q + 3]};
    lds_barrier();
#pragma unroll
    for (int o = 0; o < OUTS; ++o) {
        const int i = out_i + o * TOKENS;
        if (i >= BM) break;
        i32x4 sum = *reinterpret_cast<const i32x4*>(sums + quad_at(0, i, out_q));
#pragma unroll
        for (int w = 1; w < W; ++w) sum += *reinterpret_cast<const i32x4*>(sums + quad_at(w, i, out_q));
        store_quad<T>(g, i0 + i, j0 + out_q * 4, sum, sa[o], channels);
    }
}

template <typename T, int FU, int FV, int ST>
int launch_split(const GemmArgs& g, bool dma, hipStream_t stream) {
    const int64_t blocks = ((g.m + FU * 32 - 1) / (FU * 32)) * ((g.n + FV * 32 - 1) / (FV * 32));
    if (blocks > most_blocks(512)) return MOEQ8_EUNSUPPORTED;
    if (dma)
        hipLaunchKernelGGL((k_gemm_i8_split<T, FU, FV, ST, true>), dim3((uint32_t)blocks), dim3(512), 0, stream, g);
    else
        hipLaunchKernelGGL((k_gemm_i8_split<T, FU, FV, 2, false>), dim3((uint32_t)blocks), dim3(512), 0, stream, g);
    return check_launch();
}

// Time of a product in tiles of bm x bn, in us: the start of a block and, for
// each tile of a CU, its end; between them the largest of what a CU takes in
// (rate, in GB/s), what all of them can (18 TB/s, most of it from L2) and what
// the matrix cores do at the clock they hold (two thirds of peak).  The
// constants are fitted to the times of the six tiles on 66 products of 17 to
// 8192 tokens, 64 to 16384 channels and k = 128 to 8192, where the tile chosen
// was the best one in each (within 1% on average for rows off 16 bytes).  More
// channels were not among them, and nothing here stands for the memory that a
// head of many channels comes from: 17, 32, 64 and 256 x 131072 x 4096 take 120,
// 120, 124 and 167 us, where the rate of a large copy would allow 104 to 116 (the
// last 133 by its operations).
double tile_cost(const GemmArgs& g, int bm, int bn, double rate, double start, double end) {
    const double tiles = (double)((g.m + bm - 1) / bm) * (double)((g.n + bn - 1) / bn), k = (double)g.k;
    const double rounds = (double)((int64_t)((tiles + 255) / 256));
    const double fetch = (bm + bn) * k, one = rounds * fetch / (rate * 1e3), all = tiles * fetch / 17.8e6;
    const double mul = rounds * bm * bn * k / 6.77e6;
    return start + std::max(std::max(one, all), mul) + rounds * end;
}

// Tiles of 128 x 128 in WM x 8 / WM waves.  Up to one tile a CU three stages,
// above it two blocks a CU of two stages: 1024 x 4096 x 4096 22 and 25 us, 2048 x
// 4096 x 4096 44 and 40.  (Four stages were no faster: 800 x 3873 x 3488 20.6 and
// 20.1.)  With outputs of 16 bits a wave's part is 32 x 64, whose rows in out are
// whole lines: the same product 20.6 us, in parts of 64 x 32 21.4.  (In tiles of
// 256 the higher parts are better: 8192 x 8192 x 4096 without a pause 248 us, in
// parts of 64 x 128 253.)
template <typename T, int WM>
int launch_middle(const GemmArgs& g, bool dma, hipStream_t stream) {
    if (((g.m + 127) / 128) * ((g.n + 127) / 128) <= 256) return launch_tile<T, WM, 8 / WM, 4 / WM, WM / 2, 3>(g, dma, stream);
    return launch_tile<T, WM, 8 / WM, 4 / WM, WM / 2, 2>(g, dma, stream);
}

template <typename T>
int launch_gemm(const GemmArgs& g, hipStream_t stream) {
    constexpr int64_t MAX_STRIDE = 1 << 23;        // a tile's rows within 31-bit offsets
    if (g.k >= 16 && g.m <= 16) return launch_few<T>(g, stream);
    if (g.k >= 16 && g.a_stride < MAX_STRIDE && g.b_stride < MAX_STRIDE) {
        const bool dma = by_vectors(g);
        // The tile with the least time.  A CU takes in its rows at a rate that hardly
        // depends on the tile, so small ones cost most a product; large ones leave
        // CUs idle.  Measured (us, the tiles in this order): 333 x 2047 x 4096 13.6
        // 15.0 10.4 13.7 17.9 44; 1007 x 1217 x 7168 33 31 29 22 29 71; 1024 x 4096 x
        // 4096 56 52 37 26 23 42; 481 x 2434 x 960 11.6 12.6 11.4 7.0 8.3 19.2.
        const double cost[6] = {tile_cost(g, 32, 32, 87, 2.3, 0.88), tile_cost(g, 32, 64, 87, 1.4, 2.6),
                                tile_cost(g, 64, 64, 87, 1.9, 2.5), tile_cost(g, 64, 128, 87, 1.8, 1.9),
                                tile_cost(g, 128, 128, 61, 2.25, 1.8), tile_cost(g, 256, 256, 87, 1.7, 7.7)};
        switch (std::min_element(cost, cost + 6) - cost) {
            case 0: return launch_split<T, 1, 1, 4>(g, dma, stream);
            case 1: return launch_split<T, 1, 2, 4>(g, dma, stream);
            case 2: return launch_split<T, 2, 2, 4>(g, dma, stream);
            case 3: return launch_tile<T, 2, 4, 1, 1, 3>(g, dma, stream);
            case 4: return launch_middle<T, sizeof(T) == 2 ? 4 : 2>(g, dma, stream);
            default:
                // 16 waves end a tile sooner, 8 read fewer fragments a product: 1029 x
                // 12114 x 2240 40.3 and 41.2 us, 5626 x 5808 x 3840 131 and 128.  (The end
                // of 16 with outputs of 32 bits has no room in the ring.)  On rows off 16
                // bytes 16 waves have 4 registers too few and keep them in memory, which
                // costs what they gain: 4090 x 4080 x 2001 49.1 and 47.3 us, x 1297 38.7 and
                // 38.5, 1029 x 12114 x 2233 50.1 and 50.8.
                if constexpr (sizeof(T) == 2) {
                    if (g.k <= 2560) return launch_tile<T, 4, 4, 2, 2, 2>(g, dma, stream);
                }
                return launch_tile<T, 2, 4, 4, 2, 2>(g, dma, stream);
        }
    }
    const int64_t blocks = ((g.m + 63) / 64) * ((g.n + 63) / 64);
    if (blocks > most_blocks(256)) return MOEQ8_EUNSUPPORTED;
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

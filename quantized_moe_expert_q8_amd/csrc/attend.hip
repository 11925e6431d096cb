// Attention of a step's columns over the paged int8 cache.
//
//   t_i = scale * (q . kc_i) * kd_i                 codes kc, vc; scales kd, vd
//   out = (sum_i e^(t_i - m) vd_i vc_i) / (sum_i e^(t_i - m)),  m = max t_i
//
// over the positions i that a column sees, in one pass: a running maximum m and
// sum, and the outputs' sums rescaled where m grows.
//
// What it reads is the cache, once: a block takes a span of one sequence's
// positions for one key head, with all rows (columns times query heads of the key
// head) that read it; its waves take turns at tiles of 32 positions.  Both
// products go through v_mfma_f32_16x16x32_f16 with the rows as the 16 columns of
// the result:
//
//   S^T [positions x rows] = K [positions x d] Q^T     lane: one row, 2 x 4 positions
//   O^T [d x rows]         = V^T [d x positions] P^T   lane: one row, 4 x 4 NC values
//
// A lane's scores of the first product are, as they are, its operand of the
// second: which position a place of the product's inner index stands for is free as
// long as both operands agree, so the lane's V rows are loaded by that order.
// Everything of a row (maximum, sum, factors) lies in the lane that has it, and
// nothing of a tile goes through LDS.  int8 codes are exact in fp16: a code's byte
// under 0x64 is the fp16 number 1024 + byte.
//
// fp16 operands: a row of q is scaled by a power of two to a largest value in
// [2^13, 2^14), so what its smallest values lose is below 2^-38 of the largest; fp32
// rows go as two parts (22 bits), and bf16 and fp16 rows are exact in one.  The
// weights e^(t - m) vd of a row are scaled by the power of two that brings the
// largest of them so far to [2^12, 2^15), so what each loses is below 2^-37 of the
// largest.  (The largest vd would not do: that of a position of next to no weight
// pushed the others below fp16.  It is a number for each row and not for all, which
// costs 1.1 of 22.2 us where a wave has few tiles and two row tiles, 37 x 5 x 1500,
// and 0.3 or less elsewhere.)  They go as two parts whatever the outputs' type.
// (One part for bf16 outputs, 11 bits, gave 1 to 4 of 100 values as the neighbours of
// the right ones; the second costs 0.1 of 9.1 us for 777 positions, 1.5 of 21.0 for 5
// columns of 32768 and nothing for a batch at the rate of memory.)
//
// Spans: one sequence and key head rarely fill the card, so positions are split
// over blocks; each writes its rows' sums, maximum and total, and k_join adds them.
//
// What bounds it: for large batches memory (64 sequences of 2048 to 8192 positions, 8
// key heads of 128, bf16: 143 us and 5 for the join, 4.8 TB/s; a wave keeps one tile
// of 8.4 KB on its way while it works on another).  For one sequence in a long context a
// block's start and end, about 5 of 20 us, around the reading (5 columns, 32768
// positions: 20 + 5 us).  For short ones the chain of loads and of the join (777
// positions 9.2 us in a graph).  With more than 16 rows or fp32 the arithmetic: a tile
// of 32 positions takes 340 vector instructions for d = 128 and one row tile (and 56
// where a row's maximum grows), half of them the conversion of its codes, which the
// rows of a wave share (16 x 8 x 4096, d = 256, 64 rows in 4 parts, f32: 36 us).  Row
// tiles of 16 for d > 128: two of them left
// registers for one wave a SIMD (51 us).  What the rules of the split leave: from 129 to
// 255 pairs of sequence and key head get a span each, one block a CU (37 x 5 x 1500, 148
// pairs: 23 us, 108 CUs without work and up to six rounds a wave), and four row tiles
// go as three and one.
#include "moeq8_cache.hpp"
#include "moeq8_lds.hpp"

#include <type_traits>
#include <utility>

namespace moeq8 {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int TILE = 32, SEGMENT = 1024;          // positions a tile; positions whose pages a wave holds at a time
constexpr float STEEP = 0x1p20f;                  // maxima whose last place is not small
constexpr int WEIGHT_BITS = 12;                   // the largest weight of a row comes to [2^12, 2^13), and may grow to 2^15

struct AttendArgs {
    const void* q; int64_t q_seq, q_col, q_head;
    void* out; int64_t o_seq, o_col, o_head;
    Cache c;
    const int32_t* pages; int64_t pages_row;
    const int32_t* visible;
    float* sums;                                  // [seqs][heads][rows][spans][d], then {m, l} [...][spans]
    float2* stats;
    uint32_t cols, group, rows, limit;            // rows: cols * group; limit: what visible is taken within
    uint32_t span, spans, seqs, parts;            // parts: of the rows, 16 * NT each
    double factor;                                // |scale| * log2(e): fp32 holds it with a row's power of two
    uint32_t flip;                                // the scale's sign bit, which the queries take
};

__device__ __forceinline__ uint32_t seen_by(const AttendArgs& a, uint32_t seq, uint32_t col) {
    const int32_t n = a.visible[(int64_t)seq * a.cols + col];
    return n < 0 ? 0u : ((uint32_t)n < a.limit ? (uint32_t)n : a.limit);
}

// Over the four lanes that have a row (or a position of the other product): l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float quad_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The power of two that weights are scaled by, for their largest so far.  For one below
// 2^-115 it stays: the last place in fp16 is then below that of fp32.
__device__ __forceinline__ int up_for(float peak) {
    const int up = 127 + WEIGHT_BITS - (int)(__float_as_uint(peak) >> 23);
    return up < 127 ? up : 127;
}

// Largest of lanes 0 to 7, in every lane.
__device__ __forceinline__ uint32_t eight_max(uint32_t v) {
    v = larger(v, moved<XOR1>(v));
    v = larger(v, moved<XOR2>(v));
    v = larger(v, moved<HALF_MIRROR>(v));
    return __builtin_amdgcn_readfirstlane(v);
}

// The four codes of a dword, their sign bits flipped, as fp16 numbers: two a dword.
__device__ __forceinline__ half2v halves(uint32_t bytes, uint32_t select) {
    const uint32_t u = __builtin_amdgcn_perm(0x64646464u, bytes, select);      // 1024 + 128 + code
    return __builtin_bit_cast(half2v, u) - half2v{(_Float16)1152.0f, (_Float16)1152.0f};
}
__device__ __forceinline__ half8 as_half8(half2v a, half2v b, half2v c, half2v d) {
    return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
constexpr uint32_t FLIP = 0x80808080u, LOW = 0x04010400u, HIGH = 0x04030402u;

template <typename T>
constexpr int query_parts() { return std::is_same_v<T, float> ? 2 : 1; }     // fp16 parts of a query value

template <typename T, int NC, int NT>
constexpr int query_bytes() { return query_parts<T>() * NT * NC * 2 * 64 * 16; }

// LDS of a block: the queries' operands; their rows' factors; then, over both, the
// waves' statistics and one row tile's sums of each wave.
template <typename T, int NC, int NT>
constexpr int lds_bytes(int waves) {
    const int queries = query_bytes<T, NC, NT>() + NT * 16 * 4, join = waves * (NT * 16 * 8 + 64 * 16 * NC * 4);
    return queries > join ? queries : join;
}

// Waves a SIMD that the registers have to leave room for: what keeps loads in flight.
template <int NC, int NT>
constexpr int min_waves() { return NC * NT <= 1 ? 4 : NC * NT <= 2 ? 3 : NC * NT <= 4 ? 2 : 1; }

template <typename T, int NC, int NT, int W>
__global__ __launch_bounds__(W * 64, (W == 8 ? 2 : min_waves<NC, NT>())) void k_attend(AttendArgs a) {
    constexpr int DV = 4 * NC;                    // values of a V row a lane loads
    constexpr int QP = query_parts<T>(), PP = 2;  // fp16 parts of a query value and of a weight
    __shared__ __attribute__((aligned(16))) uint8_t lds[lds_bytes<T, NC, NT>(W)];
    constexpr uint32_t waves = W;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;

    // Units of work, a span of a sequence for a key head: heads fastest, then the
    // sequence, the span slowest.  Blocks go to the 8 XCDs in turn: with the spans
    // fastest, the XCDs that got short sequences' last spans had nothing to do (64 x 1 x
    // 8192: 171 and 149 us).  The blocks of a unit that have different rows are 8 apart,
    // and find its keys and values in their XCD's L2.
    const uint32_t eight = blockIdx.x / 8, part = eight % a.parts;
    uint32_t id = eight / a.parts * 8 + blockIdx.x % 8;
    const uint32_t head = id % a.c.n_heads, row0 = part * (16 * NT);
    id /= a.c.n_heads;
    const uint32_t seq = id % a.seqs, split = id / a.seqs;
    if (split >= a.spans) return;
    const uint32_t begin = split * a.span;

    // what depends on nothing is loaded first: what the columns see (a lane each), the
    // pages of the first positions (a lane for every 16), the queries
    const int32_t sees = a.visible[(int64_t)seq * a.cols + (lane < (int)a.cols ? lane : 0)];
    auto page_of = [&](uint32_t from) {
        const uint32_t i = from + 16 * lane;
        return i < a.limit ? (uint32_t)a.pages[seq * a.pages_row + (i >> a.c.page_shift)] : ~0u;
    };
    uint32_t page = page_of(begin);

    half8* const query = reinterpret_cast<half8*>(lds);          // [part][tile][chunk][step][lane]
    float* const factors = reinterpret_cast<float*>(lds + query_bytes<T, NC, NT>());
    for (uint32_t t = wave; t < NT; t += waves) {
        const uint32_t row = row0 + 16 * t + n;
        const bool real = row < a.rows;
        const uint32_t col = real ? row / a.group : 0u, sub = real ? row - col * a.group : 0u;
        const T* q = (const T*)a.q + seq * a.q_seq + col * a.q_col + ((int64_t)head * a.group + sub) * a.q_head;
        float v[NC][16];
        float m = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint32_t at = 64 * c + 16 * g;
            T raw[16];
            load_vec(raw, q + (at < a.c.d ? at : 0u));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[c][i] = real && at < a.c.d ? to_f32(raw[i]) : 0.0f;
                m = fmaxf(m, fabsf(v[c][i]));
            }
        }
        m = quad_max(m);
        const int up = m > 0.0f && m < __builtin_inff() ? 14 - __builtin_amdgcn_frexp_expf(m) : 0;
        if (g == 0) factors[16 * t + n] = (float)fmin(__builtin_ldexp(a.factor, -up), (double)__FLT_MAX__);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                half8 hi, lo;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = __uint_as_float(__float_as_uint(ldexpf(v[c][8 * s + i], up)) ^ a.flip);
                    hi[i] = (_Float16)x;
                    lo[i] = (_Float16)(x - (float)hi[i]);
                }
                half8* o = query + ((t * NC + c) * 2 + s) * 64 + lane;
                *o = hi;
                if constexpr (QP == 2) o[NT * NC * 2 * 64] = lo;
            }
    }

    // positions that any column sees; the fewest that one does
    const uint32_t mine = sees < 0 ? 0u : ((uint32_t)sees < a.limit ? (uint32_t)sees : a.limit);
    const uint32_t length = eight_max(mine), least = ~eight_max(~mine);
    if (begin >= length && a.spans > 1) return;   // k_join reads spans with a position only
    const uint32_t end = length - begin < a.span ? length : begin + a.span;      // 0 for a sequence of no position

    // a lane's part of a row: 16 values of each 64 of K, DV values of V; a row
    // shorter than that reads its first values again, against queries of 0 and
    // into outputs that no one stores
    const uint32_t in_page = (1u << a.c.page_shift) - 1u, stride = (uint32_t)a.c.token_stride;
    uint32_t k_at[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) k_at[c] = n * stride + (64u * c + 16u * g < a.c.d ? 64u * c + 16u * g : 0u);
    const uint32_t v_at = 4 * g * stride + ((uint32_t)(DV * n) < a.c.d ? DV * n : 0u);

    // a tile: where its two rows of 16 positions lie, and, of K and V, the operands and scales
    struct Place {
        int64_t row[2], scale[2];
        bool ok[2];
    };
    const int64_t head_row = head * a.c.head_stride, head_scale = head * a.c.scale_head_stride;
    auto place_of = [&](uint32_t at, uint32_t from) {
        Place p;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t n = (uint32_t)__builtin_amdgcn_readlane((int)page, (int)((at - from) / 16 + h));
            p.ok[h] = n < a.c.n_pages;
            n = p.ok[h] ? n : 0u;
            const uint32_t place = (at + 16 * h) & in_page;
            p.row[h] = n * a.c.page_stride + head_row + (int64_t)place * stride;
            p.scale[h] = n * a.c.scale_page_stride + head_scale + place;
        }
        return p;
    };
    u32x4 kq[2][NC];
    uint32_t vq[8][NC];
    f32x4 kd[2], vd[2];
    auto load_k = [&](const Place& p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int8_t* k = a.c.k + p.row[h];
#pragma unroll
            for (int c = 0; c < NC; ++c) kq[h][c] = *reinterpret_cast<const u32x4*>(k + k_at[c]);
            kd[h] = *reinterpret_cast<const f32x4*>(a.c.k_scale + p.scale[h] + 4u * g);
        }
    };
    auto load_v = [&](const Place& p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int8_t* v = a.c.v + p.row[h];
            vd[h] = *reinterpret_cast<const f32x4*>(a.c.v_scale + p.scale[h] + 4u * g);
#pragma unroll
            for (int j = 0; j < 4; ++j, v += stride) {
                if constexpr (NC == 1) {
                    vq[4 * h + j][0] = *reinterpret_cast<const uint32_t*>(v + v_at);
                } else if constexpr (NC == 2) {
                    const u32x2 u = *reinterpret_cast<const u32x2*>(v + v_at);
                    vq[4 * h + j][0] = u[0];
                    vq[4 * h + j][1] = u[1];
                } else {
                    const u32x4 u = *reinterpret_cast<const u32x4*>(v + v_at);
#pragma unroll
                    for (int i = 0; i < 4; ++i) vq[4 * h + j][i] = u[i];
                }
            }
        }
    };

    f32x4 o[NT][DV];
    float m[NT], l[NT], peak[NT];                 // of a row: maximum, sum, the weight that up was set for
    int up[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t] = -__builtin_inff();
        l[t] = peak[t] = 0.0f;
        up[t] = up_for(0.0f);
#pragma unroll
        for (int i = 0; i < DV; ++i) o[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // the first tile is on its way while the queries are written
    Place here = place_of(begin + TILE * wave, begin);
    if (begin + TILE * wave < end) {
        load_k(here);
        load_v(here);
    }
    lds_barrier();
    float factor[NT];
    uint32_t seen[NT];                            // positions that this lane's rows see
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint32_t row = row0 + 16 * t + n;
        factor[t] = factors[16 * t + n];
        seen[t] = (uint32_t)__shfl((int)mine, (int)(row < a.rows ? row / a.group : 0u));
        if (row >= a.rows) seen[t] = ~0u;
    }

    for (uint32_t from = begin; from < end; from += SEGMENT) {
        const uint32_t to = end - from < SEGMENT ? end : from + SEGMENT;
        if (from != begin) {
            page = page_of(from);
            here = place_of(from + TILE * wave, from);
            if (from + TILE * wave < to) {
                load_k(here);
                load_v(here);
            }
        }
        for (uint32_t at = from + TILE * wave; at < to; at += TILE * waves) {
            // the next tile's loads are issued whether there is one or not (then this one's
            // again): under a branch, what is waited for before would be unknown, and
            // every wait would be for all of them (64 x 1 x 8192: 187 us and not 171)
            const uint32_t next = at + TILE * waves < to ? at + TILE * waves : at;
            const Place then = place_of(next, from);

            // scores
            f32x4 s[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    half8 k[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x = kq[h][c][2 * st] ^ FLIP, y = kq[h][c][2 * st + 1] ^ FLIP;
                        k[h] = as_half8(halves(x, LOW), halves(x, HIGH), halves(y, LOW), halves(y, HIGH));
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int p = 0; p < QP; ++p) {
                            const half8 b = query[(((p * NT + t) * NC + c) * 2 + st) * 64 + lane];
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                s[t][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[h], b, s[t][h], 0, 0, 0);
                        }
                }
            const bool whole = at + TILE <= least && here.ok[0] && here.ok[1];
            float x[NT][8];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[t][i] = s[t][i / 4][i % 4] * kd[i / 4][i % 4];
            load_k(then);                         // K's registers are free again

            float ve[8];                          // the value scales, past the length 0, whatever is there
#pragma unroll
            for (int i = 0; i < 8; ++i) ve[i] = vd[i / 4][i % 4];
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t pos = at + 16 * (i / 4) + 4 * g + i % 4;
                    ve[i] = here.ok[i / 4] && pos < length ? ve[i] : 0.0f;
#pragma unroll
                    for (int t = 0; t < NT; ++t) x[t][i] = here.ok[i / 4] && pos < seen[t] ? x[t][i] : -__builtin_inff();
                }
            }
            // maxima are of the scores before the factor, which is not negative
            float now[NT], base[NT];
            bool plain = whole;                   // nothing of what the tile's rows see needs another look
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float top_t = x[t][0];
#pragma unroll
                for (int i = 1; i < 8; ++i) top_t = fmaxf(top_t, x[t][i]);
                now[t] = fmaxf(m[t], quad_max(top_t));
                base[t] = now[t] == -__builtin_inff() ? 0.0f : now[t] * factor[t];
                plain = plain && !__any(fabsf(base[t]) >= STEEP);
            }
            half8 w[PP][NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float e[8], v[8], sum = 0.0f, most = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    e[i] = __builtin_fmaf(x[t][i], factor[t], -base[t]);
                    v[i] = ve[i];
                }
                if (!plain) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // the product as the maximum's was rounded, whose own rounding would count
                        e[i] = fabsf(base[t]) >= STEEP ? x[t][i] * factor[t] - base[t] : e[i];
                        // the factor may be 0; a position that others see may have a scale that is not finite
                        e[i] = x[t][i] == -__builtin_inff() ? x[t][i] : e[i];
                        v[i] = x[t][i] == -__builtin_inff() ? 0.0f : v[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    e[i] = __builtin_amdgcn_exp2f(e[i]);
                    sum += e[i];
                    v[i] *= e[i];
                    most = fmaxf(most, fabsf(v[i]));
                }
                // a maximum that grows, or weights past their power of two
                if (__any(now[t] > m[t] || most >= ldexpf(1.0f, WEIGHT_BITS + 3 - up[t]))) {
                    if (__any(most == __builtin_inff())) {       // infinite ones do not count
                        most = 0.0f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]) < __builtin_inff() ? fabsf(v[i]) : 0.0f);
                    }
                    const float was = m[t] == -__builtin_inff() ? m[t] : m[t] * factor[t];
                    const float fall = now[t] > m[t] ? was - base[t] : 0.0f, keep = __builtin_amdgcn_exp2f(fall);
                    l[t] *= keep;
                    peak[t] = fmaxf(peak[t] * keep, quad_max(most));
                    const int next = up_for(peak[t]);
                    const float by = __builtin_amdgcn_exp2f(fall + (float)(next - up[t]));
#pragma unroll
                    for (int i = 0; i < DV; ++i) o[t][i] *= by;
                    m[t] = now[t];
                    up[t] = next;
                }
                l[t] += sum;
                const float unit = __uint_as_float((uint32_t)(127 + up[t]) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = v[i] * unit;
                    const _Float16 hi = (_Float16)u;
                    w[0][t][i] = hi;
                    w[1][t][i] = (_Float16)(u - (float)hi);
                }
            }

            // outputs
#pragma unroll
            for (int d4 = 0; d4 < NC; ++d4) {
                uint32_t b01[4], b23[4];          // codes 0 and 1, 2 and 3 of two positions each
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t y0 = vq[2 * j][d4] ^ FLIP, y1 = vq[2 * j + 1][d4] ^ FLIP;
                    b01[j] = __builtin_amdgcn_perm(y1, y0, 0x05010400u);
                    b23[j] = __builtin_amdgcn_perm(y1, y0, 0x07030602u);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t(&b)[4] = i < 2 ? b01 : b23;
                    const uint32_t sel = i & 1 ? HIGH : LOW;
                    const half8 v = as_half8(halves(b[0], sel), halves(b[1], sel), halves(b[2], sel), halves(b[3], sel));
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int p = 0; p < PP; ++p)
                            o[t][4 * d4 + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[p][t], o[t][4 * d4 + i], 0, 0, 0);
                }
            }
            load_v(then);
            here = then;
        }
    }

    // ---- the waves' sums together ------------------------------------------------
    __syncthreads();                              // the queries are done with
    float2* const stats = reinterpret_cast<float2*>(lds);        // [wave][row]
    f32x4* const sums = reinterpret_cast<f32x4*>(stats + waves * NT * 16);     // [wave][DV][lane]
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float total = quad_sum(l[t]);
        m[t] = m[t] == -__builtin_inff() ? m[t] : m[t] * factor[t];      // from here on with the factor
        if (g == 0) stats[(wave * NT + t) * 16 + n] = float2{m[t], total};
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float most = -__builtin_inff(), total = 0.0f;
        for (uint32_t w = 0; w < waves; ++w) most = fmaxf(most, stats[(w * NT + t) * 16 + n].x);
        const float base = most == -__builtin_inff() ? 0.0f : most;
        for (uint32_t w = 0; w < waves; ++w) {
            const float2 s = stats[(w * NT + t) * 16 + n];
            total += s.y * __builtin_amdgcn_exp2f(s.x - base);
        }
        const float keep = __builtin_amdgcn_exp2f(m[t] - base);
        // i counts the values of a lane's row in order: DV of each r
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < DV; i += 4) {
                f32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = ldexpf(o[t][i + j][r] * keep, -up[t]);
                sums[(wave * DV + (r * DV + i) / 4) * 64 + lane] = v;
            }
        __syncthreads();
        const uint32_t row = row0 + 16 * t + n;
        if (row < a.rows) {                       // this thread's lane number names the row in every wave
            const uint32_t col = row / a.group, sub = row - col * a.group;
            const int64_t place = (((int64_t)seq * a.c.n_heads + head) * a.rows + row) * a.spans + split;
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
            for (uint32_t i = wave; i < DV; i += waves) {
                const uint32_t d = 4 * DV * g + 4 * i;
                if (d >= a.c.d) break;
                f32x4 v = sums[i * 64 + lane];
                for (uint32_t w = 1; w < waves; ++w) v += sums[(w * DV + i) * 64 + lane];
                if (a.spans == 1) {
                    T* out = (T*)a.out + seq * a.o_seq + col * a.o_col + ((int64_t)head * a.group + sub) * a.o_head + d;
#pragma unroll
                    for (int j = 0; j < 4; ++j) from_f32(out[j], v[j] * inv);
                } else {
                    *reinterpret_cast<f32x4*>(a.sums + place * a.c.d + d) = v;
                }
            }
            if (a.spans > 1 && wave == 0 && g == 0) a.stats[place] = float2{most, total};
        }
        __syncthreads();
    }
}

// A row's spans together.  LANES threads have the same 4 values of a row, of every
// LANES-th span each; a block has as many rows as fit.
template <typename T, int LANES>
__global__ __launch_bounds__(256) void k_join(AttendArgs a, uint32_t row_count) {
    __shared__ f32x4 part[LANES > 1 ? 256 : 1];
    const uint32_t vecs = a.c.d / 4, tid = threadIdx.x, slot = tid / (vecs * LANES), in = tid - slot * (vecs * LANES), k = in / vecs,
                   at = in - k * vecs, per_block = 256 / (vecs * LANES);
    const uint32_t row_id = blockIdx.x * per_block + slot;
    const bool real = slot < per_block && row_id < row_count;
    const uint32_t id = real ? row_id : 0u, row = id % a.rows, pair = id / a.rows, head = pair % a.c.n_heads, seq = pair / a.c.n_heads;
    uint32_t length = 0;
#pragma unroll
    for (uint32_t c = 0; c < MOEQ8_MAX_COLS; ++c) {              // no load waits for another
        const uint32_t n = seen_by(a, seq, c < a.cols ? c : 0u);
        length = n > length ? n : length;
    }
    const uint32_t spans = (length + a.span - 1) / a.span;
    const float2* stats = a.stats + (int64_t)id * a.spans;
    const f32x4* sums = reinterpret_cast<const f32x4*>(a.sums) + (int64_t)id * a.spans * vecs;
    // each span's statistics and values with the running maximum of those before
    constexpr uint32_t AHEAD = 8;
    float m = -__builtin_inff(), l = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t from = k; from < spans; from += LANES * AHEAD) {
        float2 st[AHEAD];
        f32x4 u[AHEAD];
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) {
            const uint32_t s = from + i * LANES < spans ? from + i * LANES : from;
            st[i] = stats[s];
            u[i] = sums[(int64_t)s * vecs + at];
            if (from + i * LANES >= spans) st[i] = float2{-__builtin_inff(), 0.0f};
        }
        float now = m;
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) now = fmaxf(now, st[i].x);
        const float base = now == -__builtin_inff() ? 0.0f : now, keep = __builtin_amdgcn_exp2f(m - base);
        l *= keep;
        v *= keep;
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) {
            const float w = __builtin_amdgcn_exp2f(st[i].x - base);
            l += st[i].y * w;
            v += u[i] * w;
        }
        m = now;
    }
    if constexpr (LANES > 1) {                    // the lanes' together, in their order
        __shared__ float2 mine[256];
        part[tid] = v;
        mine[tid] = float2{m, l};
        __syncthreads();
        if (k == 0 && real) {
            float now = m;
            for (uint32_t i = 1; i < LANES; ++i) now = fmaxf(now, mine[tid + i * vecs].x);
            const float base = now == -__builtin_inff() ? 0.0f : now, keep = __builtin_amdgcn_exp2f(m - base);
            l *= keep;
            v *= keep;
            for (uint32_t i = 1; i < LANES; ++i) {
                const float2 st = mine[tid + i * vecs];
                const float w = __builtin_amdgcn_exp2f(st.x - base);
                l += st.y * w;
                v += part[tid + i * vecs] * w;
            }
        }
    }
    if (k == 0 && real) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const uint32_t col = row / a.group, sub = row - col * a.group;
        T* out = (T*)a.out + seq * a.o_seq + col * a.o_col + ((int64_t)head * a.group + sub) * a.o_head + 4 * at;
#pragma unroll
        for (int j = 0; j < 4; ++j) from_f32(out[j], v[j] * inv);
    }
}

// How a call's work is split.
struct Plan {
    int64_t rows, parts, span, spans, blocks;
    int chunks, tiles, waves;                     // 64 values of a row, 16 rows; waves a block
    size_t sums_bytes, bytes;
};

Plan plan_for(int64_t seqs, int64_t cols, int64_t q_heads, int64_t heads, int64_t d, int64_t limit) {
    Plan p;
    p.rows = cols * (q_heads / heads);
    p.chunks = d <= 64 ? 1 : d <= 128 ? 2 : 4;
    const int64_t tiles = (p.rows + 15) / 16, most = p.chunks == 4 ? 1 : 3;
    p.tiles = (int)std::min(tiles, most);
    p.parts = (tiles + p.tiles - 1) / p.tiles;
    const int64_t pairs = seqs * heads * p.parts;
    // Blocks of 8 waves where one a CU is all there is, and of 4 where several fit and
    // the loads of one go on under the ends of another: from two pairs a CU (64 x 1 x 500
    // bf16, 8 key heads of 128: 15 us, with 8 waves 19) or 768 spans of 1024 positions on
    // (64 x 1 x 8192: 142 us; but 32 x 1 x 2000 25 with 8 and 29 with 4), and for row
    // tiles whose registers leave room for one wave a SIMD.
    p.waves = p.chunks * p.tiles > 4 || pairs >= 512 || pairs * ((limit + 1023) / 1024) >= 768 ? 4 : 8;
    if (p.waves == 8) {
        // a block for each of 256 CUs, of at least one round of its waves' tiles (1 x 1 x
        // 1500: 9.1 us, with spans of 512 10.7); two rounds are no longer than the join
        // (1 x 1 x 300: 7.0 us, split 9.0)
        const int64_t want = std::max<int64_t>(1, 256 / pairs);
        p.span = limit <= 512 ? 512 : std::max<int64_t>(256, ((limit + want - 1) / want + 255) / 256 * 256);
    } else {
        // 8 blocks a CU, so that short and long sequences even out (64 x 1 x 8192, from a
        // quarter of that on: spans of 512 154 us, 1024 and 2048 142, 4096 149)
        const int64_t want = std::max<int64_t>(1, 2048 / pairs);
        p.span = std::max<int64_t>(512, ((limit + want - 1) / want + 127) / 128 * 128);
    }
    p.spans = std::max<int64_t>(1, (limit + p.span - 1) / p.span);
    p.blocks = (seqs * heads * p.spans + 7) / 8 * 8 * p.parts;
    p.sums_bytes = p.spans > 1 ? (size_t)(seqs * heads * p.rows * p.spans * d * 4) : 0;
    p.bytes = p.spans > 1 ? p.sums_bytes + (size_t)(seqs * heads * p.rows * p.spans * 8) : 0;
    return p;
}

template <typename T, int NC, int NT>
int launch_attend(const AttendArgs& a, const Plan& p, hipStream_t stream) {
    if constexpr (NC * NT <= 4) {
        if (p.waves == 8) {
            hipLaunchKernelGGL((k_attend<T, NC, NT, 8>), dim3((uint32_t)p.blocks), dim3(512), 0, stream, a);
            return check_launch();
        }
    }
    hipLaunchKernelGGL((k_attend<T, NC, NT, 4>), dim3((uint32_t)p.blocks), dim3(256), 0, stream, a);
    return check_launch();
}

template <typename T>
int attend(const AttendArgs& a, const Plan& p, hipStream_t stream) {
    int s;
    switch (p.chunks * 4 + p.tiles) {
        case 5: s = launch_attend<T, 1, 1>(a, p, stream); break;
        case 6: s = launch_attend<T, 1, 2>(a, p, stream); break;
        case 7: s = launch_attend<T, 1, 3>(a, p, stream); break;
        case 9: s = launch_attend<T, 2, 1>(a, p, stream); break;
        case 10: s = launch_attend<T, 2, 2>(a, p, stream); break;
        case 11: s = launch_attend<T, 2, 3>(a, p, stream); break;
        default: s = launch_attend<T, 4, 1>(a, p, stream); break;
    }
    if (s != MOEQ8_OK || p.spans == 1) return s;
    const uint32_t rows = (uint32_t)((int64_t)a.seqs * a.c.n_heads * a.rows), vecs = a.c.d / 4;
    auto join = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        const uint32_t per_block = 256 / (vecs * L);
        hipLaunchKernelGGL((k_join<T, L>), dim3((rows + per_block - 1) / per_block), dim3(256), 0, stream, a, rows);
        return check_launch();
    };
    // a row of 256 values takes 64 threads a lane
    return p.spans <= 8 ? join(std::integral_constant<int, 1>{}) : join(std::integral_constant<int, 4>{});
}

// What both entry points refuse of the sizes.
int check_sizes(int64_t seqs, int64_t cols, int64_t q_heads, int64_t heads, int64_t d, int64_t limit) {
    if (seqs < 0 || cols < 1 || cols > MOEQ8_MAX_COLS || heads < 1 || q_heads < heads || q_heads % heads || d < 1 || limit < 0)
        return MOEQ8_EINVAL;
    if (d % 16 || d > MOEQ8_MAX_HEAD_DIM || limit >= (1 << 30) || q_heads >= (1 << 20) || seqs >= (1 << 24))
        return MOEQ8_EUNSUPPORTED;
    if (seqs && heads > (1 << 26) / seqs) return MOEQ8_EUNSUPPORTED;
    return MOEQ8_OK;
}

}  // namespace
}  // namespace moeq8

extern "C" size_t paged_attention_workspace_bytes(int64_t n_seqs, int64_t n_cols, int64_t n_q_heads, int64_t n_heads, int64_t d,
                                                  int64_t max_visible) {
    using namespace moeq8;
    if (check_sizes(n_seqs, n_cols, n_q_heads, n_heads, d, max_visible) != MOEQ8_OK || n_seqs == 0) return 0;
    return plan_for(n_seqs, n_cols, n_q_heads, n_heads, d, max_visible).bytes;
}

extern "C" int paged_attention_i8(const void* q, int64_t q_seq_stride, int64_t q_col_stride, int64_t q_head_stride,
                                  int32_t dtype, int64_t n_seqs, int64_t n_cols, int64_t n_q_heads,
                                  const moeq8_kv_cache* cache, const int32_t* pages, int64_t pages_row_stride, int64_t n_table,
                                  const int32_t* visible, int64_t max_visible, double scale, void* out,
                                  int64_t out_seq_stride, int64_t out_col_stride, int64_t out_head_stride, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    using namespace moeq8;
    AttendArgs a;
    if (dtype < MOEQ8_F32 || dtype > MOEQ8_BF16) return MOEQ8_EINVAL;
    if (const int s = check_cache(cache, a.c)) return s;
    const int64_t heads = a.c.n_heads, d = a.c.d;
    if (const int s = check_sizes(n_seqs, n_cols, n_q_heads, heads, d, max_visible)) return s;
    if (n_table < 0 || !(scale - scale == 0.0)) return MOEQ8_EINVAL;
    if (n_seqs == 0) return MOEQ8_OK;
    if (!q || !out || !visible || (n_table && !pages)) return MOEQ8_EINVAL;
    if ((n_seqs > 1 && pages_row_stride < n_table)) return MOEQ8_EINVAL;
    const int64_t strides[2][3] = {{q_seq_stride, q_col_stride, q_head_stride}, {out_seq_stride, out_col_stride, out_head_stride}};
    const int64_t counts[3] = {n_seqs, n_cols, n_q_heads};
    int64_t bytes[2];
    const int64_t es = dtype_bytes(dtype);
    for (int i = 0; i < 2; ++i) {
        bytes[i] = d;
        for (int j = 0; j < 3; ++j) {
            if (counts[j] > 1 && strides[i][j] < d) return MOEQ8_EINVAL;
            if (counts[j] > 1) bytes[i] += (counts[j] - 1) * strides[i][j];
        }
        bytes[i] *= es;
    }
    if (((uintptr_t)q | (uintptr_t)out) & (uintptr_t)(es - 1) || ((uintptr_t)pages | (uintptr_t)visible) & 3u) return MOEQ8_EALIGN;
    if (a.c.token_stride > (1ll << 26) || n_table >= (1ll << 31)) return MOEQ8_EUNSUPPORTED;     // a lane's offsets have 32 bits
    const Plan p = plan_for(n_seqs, n_cols, n_q_heads, heads, d, max_visible);
    if (p.blocks > most_blocks(p.waves * 64) || n_seqs * n_q_heads * n_cols > most_blocks(256)) return MOEQ8_EUNSUPPORTED;
    if (p.bytes && (!workspace || workspace_bytes < p.bytes)) return MOEQ8_EINVAL;
    if (p.bytes && (uintptr_t)workspace & 15u) return MOEQ8_EALIGN;
    // what is written lies apart from itself and from what other blocks and the join still read
    const int64_t ws_bytes = (int64_t)p.bytes;
    const int64_t page_bytes = 4 * ((n_seqs > 1 ? (n_seqs - 1) * pages_row_stride : 0) + n_table), seen_bytes = 4 * n_seqs * n_cols;
    for (const auto& [at, n] : {std::pair<const void*, int64_t>{out, bytes[1]}, {workspace, ws_bytes}}) {
        if (n == 0) continue;
        if (ranges_overlap(at, n, q, bytes[0]) || ranges_overlap(at, n, visible, seen_bytes) ||
            (n_table && ranges_overlap(at, n, pages, page_bytes)) || clashes_with_cache(a.c, at, n))
            return MOEQ8_EINVAL;
    }
    if (p.bytes && ranges_overlap(workspace, ws_bytes, out, bytes[1])) return MOEQ8_EINVAL;
    a.q = q; a.q_seq = q_seq_stride; a.q_col = q_col_stride; a.q_head = q_head_stride;
    a.out = out; a.o_seq = out_seq_stride; a.o_col = out_col_stride; a.o_head = out_head_stride;
    a.pages = pages; a.pages_row = pages_row_stride;
    a.visible = visible;
    a.sums = (float*)workspace;
    a.stats = (float2*)((uint8_t*)workspace + p.sums_bytes);
    a.cols = (uint32_t)n_cols; a.group = (uint32_t)(n_q_heads / heads); a.rows = (uint32_t)p.rows;
    const int64_t positions = n_table << a.c.page_shift;
    a.limit = (uint32_t)std::min(max_visible, positions);
    a.span = (uint32_t)p.span; a.spans = (uint32_t)p.spans; a.seqs = (uint32_t)n_seqs; a.parts = (uint32_t)p.parts;
    a.factor = std::abs(scale) * 1.4426950408889634;
    a.flip = scale < 0.0 ? 0x80000000u : 0u;
    switch (dtype) {
        case MOEQ8_F32: return attend<float>(a, p, (hipStream_t)stream);
        case MOEQ8_F16: return attend<f16_t>(a, p, (hipStream_t)stream);
        default: return attend<bf16_t>(a, p, (hipStream_t)stream);
    }
}

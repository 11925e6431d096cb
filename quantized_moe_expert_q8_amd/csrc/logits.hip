// Sampling rules on logits: penalties for repeated tokens, biases and a
// grammar mask, in one pass.  For a row with logits z, its tokens
// tokens[begin .. end) (those from prompt_end on written by the model):
//
//   seen tokens:     z = z > 0 ? z / repetition : z * repetition
//   written tokens:  z = z - (count * frequency + presence)
//   biased tokens:   z = z + bias
//   masked tokens:   z = -inf
//
// in that order, in fp32 with each operation rounded, the output rounded once.
//
// A block takes one tile of one row's vocabulary.  Its logits, mask words, the
// first tokens and biases of the row are all loaded before anything waits.  It
// then marks the row's tokens that fall into the tile in LDS, a bit and a count
// each (integer atomics, whose order does not matter and whose results no one
// waits for).  The seen and the biased tokens, few of a tile, get their values
// one by one in the tile's copy in LDS; the tile is written with the mask
// applied on the way.  Nothing of vocabulary size is kept in memory: the row's
// list is read again by each of its tiles, from L2.
#include "moeq8_lds.hpp"
#include "moeq8_types.hpp"
#include "moeq8_host.hpp"

namespace moeq8 {
namespace {

struct LogitsArgs {
    const void* z; int64_t z_stride;
    void* out; int64_t out_stride;
    int64_t vocab;
    const int32_t* tokens; int64_t n_tokens;      // null: no penalties
    const int64_t* begin;
    const int64_t* end;
    const int64_t* prompt_end;                    // null: begin
    const float* repetition;                      // null: 1
    const float* frequency;                       // null: 0
    const float* presence;                        // null: 0
    const int32_t* bias_ids;                      // null: no biases
    const float* bias_values;
    int64_t n_bias;
    const int64_t* bias_offsets;
    const int32_t* mask; int64_t mask_stride;     // null: no mask
};

constexpr int AHEAD = 4;                           // loads of 4 tokens a thread has in flight
typedef uint16_t half_t __attribute__((may_alias));

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) {
    return v < lo ? lo : (v > hi ? hi : v);
}

// VEC elements from 16 bytes at p, of which [from, to) exist.
template <typename T, int VEC>
__device__ __forceinline__ void load_part(T (&v)[VEC], const T* p, int from, int to) {
    if (from <= 0 && to >= VEC) {
        load_vec(v, p);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (j >= from && j < to) v[j] = p[j];
    }
}

// Element j stays where bit j is set and becomes -inf elsewhere.
template <int VEC>
__device__ __forceinline__ void keep_bits(float (&v)[VEC], uint32_t bits) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = bits >> j & 1 ? v[j] : -__builtin_inff();
}
template <typename H, int VEC>
__device__ __forceinline__ void keep_bits(H (&v)[VEC], uint32_t bits) {
    H inf;
    from_f32(inf, -__builtin_inff());
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {             // two elements a dword
        const uint32_t x = (uint32_t)v[j].bits | (uint32_t)v[j + 1].bits << 16;
        const uint32_t keep = ((uint32_t)__builtin_amdgcn_sbfe((int)bits, j, 1) & 0xffffu) |
                              ((uint32_t)__builtin_amdgcn_sbfe((int)bits, j + 1, 1) & 0xffff0000u);
        const uint32_t y = (x & keep) | (((uint32_t)inf.bits | (uint32_t)inf.bits << 16) & ~keep);
        v[j].bits = (uint16_t)y;
        v[j + 1].bits = (uint16_t)(y >> 16);
    }
}

template <typename T, int THREADS, int TILE>
__global__ __launch_bounds__(THREADS) void k_logits(LogitsArgs a, uint32_t rows, uint32_t tiles) {
    constexpr int VEC = 16 / sizeof(T), NV = TILE / VEC / THREADS;
    static_assert(NV * VEC * THREADS == TILE, "whole vectors");
    __shared__ __attribute__((aligned(16))) T tile[TILE];
    __shared__ __attribute__((aligned(16))) uint32_t count[TILE / 2];   // written tokens: 16 bits each, or 32 of half a tile
    __shared__ uint32_t seen[TILE / 32], biased[TILE / 32], again[TILE / 32];   // a bit each token; again: more than one bias
    __shared__ int repeated;                       // any bit of again
    // All rows' first tiles come first: where frequent tokens have low ids, those
    // take longest, and the last rows' would be the last to end.
    uint32_t r = blockIdx.x, tile_no = 0;
    if (r >= rows) {
        const uint32_t rest = r - rows;
        r = rest / (tiles - 1);
        tile_no = 1 + rest - r * (tiles - 1);
    }
    const T* z = (const T*)a.z + r * a.z_stride;
    // the tile begins where the row's 16-byte units do: v0 < 0 in the first one
    // of a row that starts inside a unit
    const int v0 = (int)(tile_no * TILE) - (int)(((uintptr_t)z & 15) / sizeof(T)), vocab = (int)a.vocab;
    if (v0 >= vocab) return;
    const uint32_t low = v0 < 0 ? (uint32_t)-v0 : 0u, high = (uint32_t)(vocab - v0 < TILE ? vocab - v0 : TILE);
    const int tid = threadIdx.x;

    T held[NV][VEC];
    uint32_t bits[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int at = (n * THREADS + tid) * VEC;
        load_part(held[n], z + v0 + at, (int)low - at, (int)high - at);
    }
    const bool any = a.tokens || a.bias_ids;
    int64_t b = 0, lo = 0;
    uint32_t length = 0, written = 0, biases = 0;  // written: the first position that counts
    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    if (a.tokens) {
        b = clamp64(a.begin[r], 0, a.n_tokens);
        length = (uint32_t)(clamp64(a.end[r], b, a.n_tokens) - b);
        if (a.prompt_end) written = (uint32_t)(clamp64(a.prompt_end[r], b, b + length) - b);
        if (a.repetition) rep = a.repetition[r];
        if (a.frequency) freq = a.frequency[r];
        if (a.presence) pres = a.presence[r];
    }
    if (a.bias_ids) {
        lo = clamp64(a.bias_offsets[r], 0, a.n_bias);
        biases = (uint32_t)(clamp64(a.bias_offsets[r + 1], lo, a.n_bias) - lo);
    }
    if (a.mask) {
        const int32_t* mask = a.mask + r * a.mask_stride;
#pragma unroll
        for (int n = 0; n < NV; ++n) {             // the vector's words: two, or one twice
            const int v = v0 + (n * THREADS + tid) * VEC;
            const int first = v < 0 ? 0 : (v < vocab ? v : vocab - 1), last = v + VEC <= vocab ? v + VEC - 1 : vocab - 1;
            const uint32_t b0 = (uint32_t)mask[first >> 5], b1 = (uint32_t)mask[last >> 5];
            bits[n] = __builtin_amdgcn_alignbit(b1, b0, (uint32_t)first & 31) << (v < 0 ? -v : 0);
        }
    }
    const int32_t* tokens = a.tokens + b;
    const int32_t* bias_ids = a.bias_ids + lo;
    const float* bias_values = a.bias_values + lo;

    if (any) {
        // the first tokens and the first bias of this thread
        u32x4 token[AHEAD];
        auto load_tokens = [&](uint32_t i) {
#pragma unroll
            for (int n = 0; n < AHEAD; ++n)
                if (i + n * THREADS * 4 + 4 <= length) token[n] = *reinterpret_cast<const u32x4*>(tokens + i + n * THREADS * 4);
        };
        load_tokens(tid * 4);
        int32_t bias_id = -1;
        float bias_value = 0.0f;
        if (tid < biases) {
            bias_id = bias_ids[tid];
            bias_value = bias_values[tid];
        }
        // its own part of the tile, from registers
#pragma unroll
        for (int n = 0; n < NV; ++n) store_vec(tile + (n * THREADS + tid) * VEC, held[n]);
        // A count of 16 bits holds a list of 65535; a longer one is taken in two
        // halves of the tile, with counts of 32 bits.
        const bool wide = length - written > 65535u;
        // The tokens with more than one bias.  A token's are added in the list's
        // order, so one wave has all of a token's (those of every WAVES-th word of
        // the bits) and goes through the list.  That is read once, however many
        // repeat: 50000 biases on 131072 fp32 logits take 53 us where all differ, 157
        // where one or all come twice (with a search of the list for each such
        // token 270000).  Between two additions the value is kept in fp32: for 16-bit
        // elements its low half is where the token's count was.
        auto add_repeated = [&](auto place, auto penalised) {
            constexpr int WAVES = THREADS / 64, WORDS = TILE / 32 / WAVES, LOADS = 2;
            static_assert(WORDS <= 64, "a word a lane");
            uint32_t id = tid;
            asm volatile("" : "+v"(id));           // or what is made of it takes registers from the start, and waves from the CU
            const uint32_t wave = __builtin_amdgcn_readfirstlane(id >> 6), lane = id & 63;
            auto low_half = [&](uint32_t at) -> half_t& {
                return reinterpret_cast<half_t*>(count)[wide ? 2 * (at & (TILE / 2 - 1)) : at];
            };
            auto value = [&](uint32_t at) {
                if constexpr (sizeof(T) == 4) return tile[at];
                else return __uint_as_float((uint32_t)tile[at].bits << 16 | low_half(at));
            };
            auto hold = [&](uint32_t at, float v) {
                if constexpr (sizeof(T) == 4) {
                    tile[at] = v;
                } else {
                    tile[at].bits = (uint16_t)(__float_as_uint(v) >> 16);
                    low_half(at) = (uint16_t)__float_as_uint(v);
                }
            };
            auto each = [&](auto f) {              // this lane's tokens
                const uint32_t word = wave + lane * WAVES;
                for (uint32_t left = lane < WORDS ? again[word] : 0u; left; left &= left - 1) f(word * 32 + __builtin_ctz(left));
            };
            each([&](uint32_t at) { hold(at, seen[at >> 5] >> (at & 31) & 1 ? penalised(at) : to_f32(tile[at])); });
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // for the wave's other lanes
            for (uint32_t first = 0; first < biases; first += 64 * LOADS) {
                uint32_t at[LOADS];
                float add[LOADS];
#pragma unroll
                for (int n = 0; n < LOADS; ++n) {
                    const uint32_t i = first + n * 64 + lane < biases ? first + n * 64 + lane : biases - 1;
                    at[n] = (uint32_t)bias_ids[i];
                    add[n] = bias_values[i];
                }
#pragma unroll
                for (int n = 0; n < LOADS; ++n) {
                    at[n] = place((int32_t)at[n]);
                    const bool own = first + n * 64 + lane < biases && at[n] != TILE && (at[n] >> 5) % WAVES == wave &&
                                     (again[at[n] >> 5] >> (at[n] & 31) & 1);
                    for (uint64_t left = __ballot(own); left; left &= left - 1) {
                        const int l = __builtin_ctzll(left);       // all lanes write the same
                        const uint32_t to = __builtin_amdgcn_readlane((int)at[n], l);
                        hold(to, value(to) + __uint_as_float(__builtin_amdgcn_readlane(__float_as_int(add[n]), l)));
                    }
                }
            }
            if constexpr (sizeof(T) == 2) each([&](uint32_t at) { from_f32(tile[at], value(at)); });
        };
        for (uint32_t from = low, to; from < high; from = to) {
            to = wide && from < TILE / 2 && high > TILE / 2 ? TILE / 2 : high;
#pragma unroll
            for (int n = tid; n < TILE / 8; n += THREADS) reinterpret_cast<uint4*>(count)[n] = uint4{0u, 0u, 0u, 0u};
            for (int n = tid; n < TILE / 32; n += THREADS) seen[n] = biased[n] = again[n] = 0u;
            if (tid == 0) repeated = 0;
            lds_barrier();
            // position of a token in this part of the tile, or one past it
            // (vocab < 2^30: no wrap reaches back into the tile)
            auto place = [&](int32_t token) {
                const uint32_t at = (uint32_t)token - (uint32_t)v0;
                return at >= from && at < to ? at : (uint32_t)TILE;
            };
            auto count_of = [&](uint32_t at) {
                return wide ? count[at & (TILE / 2 - 1)] : count[at >> 1] >> (16 * (at & 1)) & 0xffffu;
            };
            auto meet = [&](uint32_t i, int32_t token) {
                const uint32_t at = place(token), bit = 1u << (at & 31);
                if (at == TILE) return;
                atomicOr(&seen[at >> 5], bit);
                if (i >= written) {
                    if (wide) atomicAdd(&count[at & (TILE / 2 - 1)], 1u);
                    else atomicAdd(&count[at >> 1], 1u << (16 * (at & 1)));
                }
            };
            for (uint32_t i = tid * 4; i < length; i += THREADS * 4 * AHEAD) {
                if (i != tid * 4 || from != low) load_tokens(i);
#pragma unroll
                for (int n = 0; n < AHEAD; ++n) {
                    const uint32_t at = i + n * THREADS * 4;
                    if (at + 4 <= length) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) meet(at + j, (int32_t)token[n][j]);
                    } else {
                        for (uint32_t j = at; j < length; ++j) meet(j, tokens[j]);
                    }
                }
            }
            for (uint32_t i = tid; i < biases; i += THREADS) {
                const uint32_t at = place(i == tid ? bias_id : bias_ids[i]), bit = 1u << (at & 31);
                if (at < TILE && (atomicOr(&biased[at >> 5], bit) & bit)) {
                    atomicOr(&again[at >> 5], bit);
                    repeated = 1;
                }
            }
            lds_barrier();
            auto penalised = [&](uint32_t at) {
                const uint32_t n = count_of(at);
                float v = to_f32(tile[at]);
                v = v > 0.0f ? v / rep : v * rep;
                return n ? v - ((float)n * freq + pres) : v;
            };
            // the seen tokens without a bias, then the biased ones: no token twice
            constexpr int FIELD = TILE / THREADS;  // bits of a thread; most threads have none or one set
            const uint32_t first = tid * FIELD;
            uint32_t left = (seen[first >> 5] & ~biased[first >> 5]) >> (first & 31) & ((2u << (FIELD - 1)) - 1);
            while (left) {
                const uint32_t at = first + __builtin_ctz(left);
                left &= left - 1;
                from_f32(tile[at], penalised(at));
            }
            if (biases) {
                for (uint32_t i = tid; i < biases; i += THREADS) {
                    const uint32_t at = place(i == tid ? bias_id : bias_ids[i]);
                    if (at == TILE || again[at >> 5] >> (at & 31) & 1) continue;
                    const float v = seen[at >> 5] >> (at & 31) & 1 ? penalised(at) : to_f32(tile[at]);
                    from_f32(tile[at], v + (i == tid ? bias_value : bias_values[i]));
                }
                if (__builtin_expect(repeated, 0)) add_repeated(place, penalised);
            }
            lds_barrier();
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) load_vec(held[n], tile + (n * THREADS + tid) * VEC);
    }

    T* out = (T*)a.out + r * a.out_stride + v0;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int at = (n * THREADS + tid) * VEC;
        if (a.mask) keep_bits(held[n], bits[n]);
        if (at >= (int)low && at + VEC <= (int)high) {
            store_vec(out + at, held[n]);
        } else {                                   // the row's ends
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (at + j >= (int)low && at + j < (int)high) out[at + j] = held[n][j];
        }
    }
}

template <typename T, int THREADS, int TILE>
int launch_form(const LogitsArgs& a, int64_t rows, hipStream_t stream) {
    const int64_t tiles = (a.vocab + 16 / (int64_t)sizeof(T) - 1 + TILE - 1) / TILE;     // with a shifted first tile
    if (rows > most_blocks(THREADS) / tiles) return MOEQ8_EUNSUPPORTED;
    hipLaunchKernelGGL((k_logits<T, THREADS, TILE>), dim3((uint32_t)(rows * tiles)), dim3(THREADS), 0, stream, a, (uint32_t)rows,
                       (uint32_t)tiles);
    return check_launch();
}

template <typename T>
int launch_logits(const LogitsArgs& a, int64_t rows, hipStream_t stream) {
    // More blocks of 512 threads than run at a time, 4 a CU: a thread takes two
    // vectors (us, with two and with one: 17 x 131072 f32, 1088 blocks, 8.2 and 9.5;
    // 220 x 19809 bf16 9.8 and 10.9; 256 x 131072 bf16 with 2048 tokens a row 39 and
    // 55; but 91 x 21061 f32, 1001 blocks, 8.0 and 7.7; 1024 blocks to the block,
    // 16 x 131072 f32, would still be better with two, 7.8 and 8.5).  Fewer: what
    // counts is how soon one block is done, so a thread takes one vector, and blocks
    // of long lists are larger (5 x 131072 f32 with 8192 tokens a row: 512 threads
    // 7.0, 1024 6.3 us; 32 x 32000 bf16 with 1000: 5.8 and 6.1).  The lists' own
    // lengths are on the device: rows that share a list count as having a part of it
    // each (8 x 100000 f32 on one list of 8000 tokens 7.2 us, in larger blocks 6.6).
    constexpr int VEC = 16 / sizeof(T);
    const int64_t tiles = (a.vocab + 512 * VEC - 1) / (512 * VEC);
    if (rows > 1024 / tiles) return launch_form<T, 512, 1024 * VEC>(a, rows, stream);
    if (a.n_tokens / rows < 1024) return launch_form<T, 512, 512 * VEC>(a, rows, stream);
    return launch_form<T, 1024, 1024 * VEC>(a, rows, stream);
}

}  // namespace
}  // namespace moeq8

extern "C" int logits_process(const void* logits, int64_t logits_row_stride, int32_t dtype, int64_t n_rows,
                              int64_t vocab, const int32_t* tokens, int64_t n_tokens, const int64_t* begin,
                              const int64_t* end, const int64_t* prompt_end, const float* repetition,
                              const float* frequency, const float* presence, const int32_t* bias_ids,
                              const float* bias_values, int64_t n_bias, const int64_t* bias_offsets,
                              const int32_t* mask, int64_t mask_row_stride, void* out, int64_t out_row_stride,
                              void* stream) {
    using namespace moeq8;
    if (!logits || !out || dtype < MOEQ8_F32 || dtype > MOEQ8_BF16 || n_rows < 0 || vocab < 0) return MOEQ8_EINVAL;
    if (logits_row_stride < vocab || out_row_stride < vocab) return MOEQ8_EINVAL;
    if (n_tokens < 0 || n_bias < 0) return MOEQ8_EINVAL;
    if (tokens ? (!begin || !end) : (begin || end || prompt_end || repetition || frequency || presence))
        return MOEQ8_EINVAL;
    if (!bias_ids != !bias_values || !bias_ids != !bias_offsets) return MOEQ8_EINVAL;
    if (mask && mask_row_stride < (vocab + 31) / 32) return MOEQ8_EINVAL;
    if (vocab >= (1 << 30) || n_tokens >= (1 << 30) || n_bias >= (1 << 30)) return MOEQ8_EUNSUPPORTED;
    const int es = dtype_bytes(dtype);
    if (((uintptr_t)logits | (uintptr_t)out) & (uintptr_t)(es - 1)) return MOEQ8_EALIGN;
    if (((uintptr_t)tokens | (uintptr_t)repetition | (uintptr_t)frequency | (uintptr_t)presence | (uintptr_t)bias_ids |
         (uintptr_t)bias_values | (uintptr_t)mask) & 3u)
        return MOEQ8_EALIGN;
    if (((uintptr_t)begin | (uintptr_t)end | (uintptr_t)prompt_end | (uintptr_t)bias_offsets) & 7u) return MOEQ8_EALIGN;
    if (n_rows == 0 || vocab == 0) return MOEQ8_OK;
    if (rows_clash(logits, logits_row_stride * es, out, out_row_stride * es, n_rows, vocab * es)) return MOEQ8_EINVAL;
    const LogitsArgs a{logits, logits_row_stride, out, out_row_stride, vocab, tokens, n_tokens, begin, end, prompt_end,
                       repetition, frequency, presence, bias_ids, bias_values, n_bias, bias_offsets,
                       mask, mask_row_stride};
    switch (dtype) {
        case MOEQ8_F32: return launch_logits<float>(a, n_rows, (hipStream_t)stream);
        case MOEQ8_F16: return launch_logits<f16_t>(a, n_rows, (hipStream_t)stream);
        default: return launch_logits<bf16_t>(a, n_rows, (hipStream_t)stream);
    }
}


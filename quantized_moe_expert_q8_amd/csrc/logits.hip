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
// A block takes one tile of one row's vocabulary.  It counts the row's tokens
// that fall into its tile in LDS (integer atomics, whose order does not
// matter), so nothing of vocabulary size is kept in memory: the list is read
// again by each tile of the row, from L2, which costs far less than the
// logits as long as it is not much longer than a tile.
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

constexpr int THREADS = 256;
constexpr int TILE = 4096;
// A tile's word: how often the token was written, and whether it was seen at
// all or has a bias.
constexpr uint32_t SEEN = 1u << 31, BIASED = 1u << 30, COUNT = BIASED - 1;

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) {
    return v < lo ? lo : (v > hi ? hi : v);
}

template <typename T>
__global__ __launch_bounds__(THREADS) void k_logits(LogitsArgs a) {
    __shared__ uint32_t word[TILE];
    __shared__ float bias[TILE];
    __shared__ int repeated;                       // a token has more than one bias
    const int64_t tiles = (a.vocab + TILE - 1) / TILE;
    const int64_t r = blockIdx.x / tiles, v0 = blockIdx.x % tiles * TILE;
    const int size = (int)(a.vocab - v0 < TILE ? a.vocab - v0 : TILE);
    for (int i = threadIdx.x; i < TILE; i += THREADS) word[i] = 0u;
    if (threadIdx.x == 0) repeated = 0;
    __syncthreads();
    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    if (a.tokens) {
        const int64_t b = clamp64(a.begin[r], 0, a.n_tokens), e = clamp64(a.end[r], b, a.n_tokens);
        const int64_t p = a.prompt_end ? clamp64(a.prompt_end[r], b, e) : b;
        if (a.repetition) rep = a.repetition[r];
        if (a.frequency) freq = a.frequency[r];
        if (a.presence) pres = a.presence[r];
        for (int64_t i = b + threadIdx.x; i < e; i += THREADS) {
            const int64_t at = (int64_t)a.tokens[i] - v0;
            if (at >= 0 && at < size) {
                atomicOr(&word[at], SEEN);
                if (i >= p) atomicAdd(&word[at], 1u);
            }
        }
    }
    int64_t lo = 0, hi = 0;
    if (a.bias_ids) {
        lo = clamp64(a.bias_offsets[r], 0, a.n_bias);
        hi = clamp64(a.bias_offsets[r + 1], lo, a.n_bias);
        for (int64_t i = lo + threadIdx.x; i < hi; i += THREADS) {
            const int64_t at = (int64_t)a.bias_ids[i] - v0;
            if (at >= 0 && at < size) {
                if (atomicOr(&word[at], BIASED) & BIASED) repeated = 1;
                bias[at] = a.bias_values[i];
            }
        }
    }
    __syncthreads();
    const T* z = (const T*)a.z + r * a.z_stride + v0;
    T* out = (T*)a.out + r * a.out_stride + v0;
    for (int i = threadIdx.x; i < size; i += THREADS) {
        float v = to_f32(z[i]);
        const uint32_t w = word[i];
        if (w & SEEN) v = v > 0.0f ? v / rep : v * rep;
        if (w & COUNT) v = v - ((float)(w & COUNT) * freq + pres);
        if (w & BIASED) {
            if (!repeated) {
                v += bias[i];
            } else {                               // every bias of the token, in the list's order
                for (int64_t j = lo; j < hi; ++j)
                    if (a.bias_ids[j] == v0 + i) v += a.bias_values[j];
            }
        }
        if (a.mask && !((a.mask[r * a.mask_stride + ((v0 + i) >> 5)] >> ((v0 + i) & 31)) & 1)) v = -__builtin_inff();
        from_f32(out[i], v);
    }
}

template <typename T>
int launch_logits(const LogitsArgs& a, int64_t rows, hipStream_t stream) {
    const int64_t tiles = (a.vocab + TILE - 1) / TILE;
    if (rows > 0x7fffffff / tiles) return MOEQ8_EUNSUPPORTED;
    hipLaunchKernelGGL(k_logits<T>, dim3((uint32_t)(rows * tiles)), dim3(THREADS), 0, stream, a);
    return check_launch();
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
    if (vocab > 0x7fffffff || n_tokens >= (1 << 30)) return MOEQ8_EUNSUPPORTED;
    const int es = dtype_bytes(dtype);
    if (((uintptr_t)logits | (uintptr_t)out) & (uintptr_t)(es - 1)) return MOEQ8_EALIGN;
    if (((uintptr_t)tokens | (uintptr_t)repetition | (uintptr_t)frequency | (uintptr_t)presence | (uintptr_t)bias_ids |
         (uintptr_t)bias_values | (uintptr_t)mask) & 3u)
        return MOEQ8_EALIGN;
    if (((uintptr_t)begin | (uintptr_t)end | (uintptr_t)prompt_end | (uintptr_t)bias_offsets) & 7u) return MOEQ8_EALIGN;
    if (n_rows == 0 || vocab == 0) return MOEQ8_OK;
    if (!(logits == out && logits_row_stride == out_row_stride) &&
        ranges_overlap(logits, ((n_rows - 1) * logits_row_stride + vocab) * es, out,
                       ((n_rows - 1) * out_row_stride + vocab) * es))
        return MOEQ8_EINVAL;
    const LogitsArgs a{logits, logits_row_stride, out, out_row_stride, vocab, tokens, n_tokens, begin, end, prompt_end,
                       repetition, frequency, presence, bias_ids, bias_values, n_bias, bias_offsets,
                       mask, mask_row_stride};
    switch (dtype) {
        case MOEQ8_F32: return launch_logits<float>(a, n_rows, (hipStream_t)stream);
        case MOEQ8_F16: return launch_logits<f16_t>(a, n_rows, (hipStream_t)stream);
        default: return launch_logits<bf16_t>(a, n_rows, (hipStream_t)stream);
    }
}

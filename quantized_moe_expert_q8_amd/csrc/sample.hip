// A token for each row of logits, from a given random number: temperature, top-k,
// top-p, min-p, and a draw in the order of the indexes.
//
// Weights e^((z - max) / T) are taken in 64 bits and summed as integers of 2^-S of
// the largest, S so that a row's sum stays below 2^63 (131072 tokens: 2^-46 each):
// sums are exact, whatever their order, so a token does not depend on how a row was
// split, and next to a border (u times the kept mass, p times the mass) the choice is
// that of the definition but for the weights' own roundings.
//
// The kept tokens are those above a threshold of the order-preserving keys, and of
// those equal to it the first few by index.
#include "moeq8_host.hpp"
#include "moeq8_types.hpp"

namespace moeq8 {
namespace {

struct SampleArgs {
    const void* z; int64_t z_stride;
    int64_t vocab;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    int32_t* token;
    float* logprob;
    int bits;                                     // S
};

constexpr int THREADS = 1024;

// Keys of the logits in their order, equal for equal logits; 0 for what is never drawn.
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return z > -__builtin_inff() ? k : 0u;        // false for NaN too
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t KEY_INF = 0xff800000u;

struct Weigh {                                    // weights of a row's logits
    double top, inv;                              // the largest logit; 1 / T
    bool infinite;
    __device__ double real(uint32_t key) const {
        if (infinite) return key == KEY_INF ? 1.0 : 0.0;
        return key ? exp(log_of(key)) : 0.0;
    }
    __device__ double log_of(uint32_t key) const { return infinite ? 0.0 : ((double)logit_of(key) - top) * inv; }
};

// Sum over the block; every thread gets it.
template <typename V>
__device__ V block_sum(V v, V* lds) {
    for (int i = 32; i; i >>= 1) v += (V)__shfl_xor((unsigned long long)v, i);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    V t = 0;
    for (int i = 0; i < THREADS / 64; ++i) t += lds[i];
    return t;
}
// Sum over the threads before this one, and over all.
__device__ uint64_t block_scan(uint64_t v, uint64_t* lds, uint64_t& all) {
    uint64_t s = v;
    for (int i = 1; i < 64; i <<= 1) {
        const uint64_t t = (uint64_t)__shfl_up((unsigned long long)s, i);
        if ((int)(threadIdx.x & 63) >= i) s += t;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    uint64_t before = 0;
    all = 0;
    for (int i = 0; i < THREADS / 64; ++i) {
        if (i < (int)(threadIdx.x >> 6)) before += lds[i];
        all += lds[i];
    }
    return before + s - v;
}

template <typename T>
__global__ __launch_bounds__(THREADS) void k_sample(SampleArgs a) {
    __shared__ uint64_t lds[THREADS / 64];
    __shared__ unsigned long long mass[256];
    __shared__ uint32_t count[256];
    __shared__ uint32_t pick;
    __shared__ uint64_t above_mass, above_count;
    const int64_t row = blockIdx.x, vocab = a.vocab;
    const T* z = (const T*)a.z + row * a.z_stride;
    const int tid = threadIdx.x;

    auto each = [&](auto f) {
        for (int64_t i = tid; i < vocab; i += THREADS) f(i, key_of(to_f32(z[i])));
    };

    uint32_t top = 0;
    uint64_t valid = 0;
    each([&](int64_t, uint32_t k) { top = k > top ? k : top; valid += k != 0; });
    for (int i = 32; i; i >>= 1) { const uint32_t t = __shfl_xor(top, i); top = t > top ? t : top; }
    __syncthreads();
    if ((tid & 63) == 0) count[tid >> 6] = top;
    __syncthreads();
    for (int i = 0; i < THREADS / 64; ++i) top = count[i] > top ? count[i] : top;
    valid = block_sum(valid, lds);
    if (top == 0) {
        if (tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = -__builtin_inff();
        }
        return;
    }

    float t = a.temperature ? a.temperature[row] : 1.0f;
    if (t != t && !a.temperature) t = 1.0f;
    const bool greedy = !(t > 0.0f);
    Weigh weigh;
    weigh.infinite = top == KEY_INF;
    weigh.top = (double)logit_of(top);
    weigh.inv = 1.0 / (double)t;
    const double unit = ldexp(1.0, a.bits);
    auto weight = [&](uint32_t k) { return (uint64_t)rint(weigh.real(k) * unit); };

    int64_t k = a.top_k ? a.top_k[row] : 0;
    if (greedy) k = 1;
    float p = a.top_p ? a.top_p[row] : 1.0f, least = a.min_p ? a.min_p[row] : 0.0f;
    if (!(p < 1.0f) || greedy) p = 1.0f;
    if (!(least > 0.0f) || greedy) least = 0.0f;
    if (least > 1.0f) least = 1.0f;

    // kept: keys above `floor`, and `ties` of those equal to it
    uint32_t floor = 0;
    uint64_t ties = 0;

    // The key at which a running sum of what is at or above it reaches `want`;
    // by_mass: of weights, counting of the keys at `floor` the ties only.
    auto select = [&](bool by_mass, uint64_t want, uint64_t& before) {
        uint32_t prefix = 0;
        before = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            for (int i = tid; i < 256; i += THREADS) mass[i] = 0;
            __syncthreads();
            each([&](int64_t, uint32_t key) {
                if (key == 0 || key < floor || (shift < 24 && (key >> (shift + 8)) != (prefix >> (shift + 8)))) return;
                if (key == floor) return;
                atomicAdd(&mass[key >> shift & 255], by_mass ? (unsigned long long)weight(key) : 1ull);
            });
            __syncthreads();
            if (tid == 0) {
                if (by_mass && floor && (shift == 24 || (floor >> (shift + 8)) == (prefix >> (shift + 8))))
                    mass[floor >> shift & 255] += ties * weight(floor);
                int b = 255;
                uint64_t s = before;
                while (b > 0 && s + mass[b] < want) s += mass[b--];
                pick = prefix | (uint32_t)b << shift;
                above_mass = s;
            }
            __syncthreads();
            prefix = pick;
            before = above_mass;
        }
        return prefix;
    };

    if (k > 0 && (uint64_t)k < valid) {
        uint64_t before;
        const uint32_t key = select(false, (uint64_t)k, before);
        floor = key;
        ties = (uint64_t)k - before;
    }
    if (p < 1.0f) {
        uint64_t s = 0;
        each([&](int64_t, uint32_t key) { if (key > floor) s += weight(key); });
        s = block_sum(s, lds) + (floor ? ties * weight(floor) : 0);
        uint64_t want = (uint64_t)ceil(fmax(p, 0.0f) * (double)s), before;
        if (want < 1) want = 1;
        const uint32_t key = select(true, want, before);
        const uint64_t w = weight(key);
        uint64_t n = w ? (want - before + w - 1) / w : ~0ull;
        if (key == floor) { if (n < ties) ties = n; }
        else { floor = key; ties = n; }
    }
    // the last of the ties, and the kept mass
    int64_t last = vocab;
    if (floor) {
        uint64_t seen = 0;
        last = -1;
        for (int64_t from = 0; from < vocab && seen < ties; from += THREADS) {
            const int64_t i = from + tid;
            const bool is = i < vocab && key_of(to_f32(z[i])) == floor;
            uint64_t all;
            const uint64_t at = seen + block_scan(is, lds, all);
            __syncthreads();
            if (is && at + 1 == ties) above_count = (uint64_t)i;
            __syncthreads();
            if (seen + all >= ties) last = (int64_t)above_count;
            else last = from + THREADS;
            seen += all;
        }
    }
    auto kept = [&](int64_t i, uint32_t key) -> uint64_t {
        if (key == 0 || key < floor || (key == floor && i > last)) return 0;
        const double e = weigh.real(key);
        if (greedy) return 1;
        return e >= (double)least ? (uint64_t)rint(e * unit) : 0;
    };
    uint64_t total = 0;
    each([&](int64_t i, uint32_t key) { total += kept(i, key); });
    total = block_sum(total, lds);
    float uf = a.u[row];
    if (!(uf > 0.0f)) uf = 0.0f;
    uint64_t target = (uint64_t)((double)uf * (double)total);
    if (target >= total) target = total - 1;
    uint64_t done = 0;
    for (int64_t from = 0; from < vocab; from += THREADS) {
        const int64_t i = from + tid;
        const uint32_t key = i < vocab ? key_of(to_f32(z[i])) : 0u;
        const uint64_t w = i < vocab ? kept(i, key) : 0;
        uint64_t all;
        const uint64_t before = done + block_scan(w, lds, all);
        if (w && before <= target && target < before + w) {
            a.token[row] = (int32_t)i;
            if (a.logprob) a.logprob[row] = greedy ? 0.0f : (float)(weigh.log_of(key) - log((double)total / unit));
        }
        done += all;
        if (done > target) break;
    }
}

}  // namespace
}  // namespace moeq8

extern "C" size_t logits_sample_workspace_bytes(int64_t n_rows, int64_t vocab) {
    (void)n_rows;
    (void)vocab;
    return 0;
}

extern "C" int logits_sample(const void* logits, int64_t logits_row_stride, int32_t dtype, int64_t n_rows, int64_t vocab,
                             const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                             const float* min_p, int32_t* token, float* logprob, void* workspace, size_t workspace_bytes,
                             void* stream) {
    using namespace moeq8;
    (void)workspace;
    if (dtype < MOEQ8_F32 || dtype > MOEQ8_BF16 || n_rows < 0 || vocab < 0) return MOEQ8_EINVAL;
    if (n_rows > 1 && logits_row_stride < vocab) return MOEQ8_EINVAL;
    if (n_rows && ((vocab && !logits) || !u || !token)) return MOEQ8_EINVAL;
    if (vocab >= (1 << 30)) return MOEQ8_EUNSUPPORTED;
    const int es = dtype_bytes(dtype);
    if ((uintptr_t)logits & (uintptr_t)(es - 1)) return MOEQ8_EALIGN;
    if (((uintptr_t)u | (uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)token |
         (uintptr_t)logprob) & 3u)
        return MOEQ8_EALIGN;
    if (n_rows == 0) return MOEQ8_OK;
    if (n_rows > most_blocks(THREADS)) return MOEQ8_EUNSUPPORTED;
    int bits = 63;
    while (vocab > (1ll << (63 - bits))) --bits;
    if (bits > 62) bits = 62;
    const SampleArgs a{logits, logits_row_stride, vocab, u, temperature, top_p, min_p, top_k, token, logprob, bits};
    const dim3 grid((uint32_t)n_rows);
    switch (dtype) {
        case MOEQ8_F32: hipLaunchKernelGGL((k_sample<float>), grid, dim3(THREADS), 0, (hipStream_t)stream, a); break;
        case MOEQ8_F16: hipLaunchKernelGGL((k_sample<f16_t>), grid, dim3(THREADS), 0, (hipStream_t)stream, a); break;
        default: hipLaunchKernelGGL((k_sample<bf16_t>), grid, dim3(THREADS), 0, (hipStream_t)stream, a); break;
    }
    return check_launch();
}

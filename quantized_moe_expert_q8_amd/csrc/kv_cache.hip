// Keys and values into a paged int8 cache, and back.
//
//   write:  d = max|x| / 127, code = roundf(x / d)      (the rule of the int8 rows)
//   read:   x = T(fp32(code * d))
//
// A row, one token's key or value of one head, belongs to the 2 to 32 lanes that
// its vectors of 8 values take (a power of two, so that the maximum goes through
// lanes in registers); a wave has as many rows as fit.  Both calls do nothing but
// move bytes, so what bounds them is memory (65536 x 8 x 128 back to bf16 83 us, 4.9
// TB/s, the rate of a large copy; writing 8192 x 8 x 128 bf16 12.8 us, 4.0 TB/s, with
// the arithmetic of the codes beside it), and for a step's few tokens the launch (5 x
// 8 x 128 f32 2.2 us in a graph).
#include "moeq8_cache.hpp"

namespace moeq8 {
namespace {

struct RowsArgs {
    Cache c;
    void* k; int64_t k_token, k_head;             // the rows outside the cache, strides in elements
    void* v; int64_t v_token, v_head;
    const int64_t* slots;
    uint32_t tokens;
    uint32_t rows;                                // 2 * tokens * heads
};

constexpr int THREADS = 256;

// Largest over LANES neighbouring lanes.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LANES >= 2) v = larger(v, moved<XOR1>(v));
    if constexpr (LANES >= 4) v = larger(v, moved<XOR2>(v));
    if constexpr (LANES >= 8) v = larger(v, moved<HALF_MIRROR>(v));
    if constexpr (LANES >= 16) v = larger(v, moved<MIRROR>(v));
    if constexpr (LANES >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = larger(s[0], s[1]);
    }
    return v;
}

// A row by its number: tokens in order, the heads of a token side by side, all
// keys before all values.
struct Row {
    bool value;
    uint32_t token, head;
};
__device__ __forceinline__ Row row_of(const RowsArgs& a, uint32_t r) {
    const uint32_t half = a.rows / 2;
    Row o;
    o.value = r >= half;
    r = o.value ? r - half : r;
    o.token = r / a.c.n_heads;
    o.head = r - o.token * a.c.n_heads;
    return o;
}

template <typename T, int LANES>
__global__ __launch_bounds__(THREADS) void k_cache_write(RowsArgs a) {
    const uint32_t r = (blockIdx.x * THREADS + threadIdx.x) / LANES, at = (threadIdx.x & (LANES - 1)) * VEC;
    const Row row = row_of(a, r < a.rows ? r : a.rows - 1);      // every lane goes through the maximum
    const int64_t slot = a.slots[row.token];
    const T* x = row.value ? (const T*)a.v + row.token * a.v_token + row.head * a.v_head
                           : (const T*)a.k + row.token * a.k_token + row.head * a.k_head;
    T raw[VEC];
    load_vec(raw, x + (at < a.c.d ? at : 0));     // the lanes past the row have its first vector again
    float y[VEC];
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        y[j] = to_f32(raw[j]);
        m = larger(m, magnitude(y[j]));
    }
    m = lanes_max<LANES>(m);
    if (r >= a.rows || at >= a.c.d || (uint64_t)slot >= (uint64_t)a.c.n_pages << a.c.page_shift) return;
    const float d = __uint_as_float(m) / 127.0f;
    int sum;
    const uint2 codes = codes8(y, d, sum);
    const int64_t page = slot >> a.c.page_shift, place = slot & ((1ll << a.c.page_shift) - 1);
    int8_t* o = (row.value ? a.c.v : a.c.k) + page * a.c.page_stride + row.head * a.c.head_stride + place * a.c.token_stride;
    *reinterpret_cast<uint2*>(o + at) = codes;
    if (at == 0)
        (row.value ? a.c.v_scale : a.c.k_scale)[page * a.c.scale_page_stride + row.head * a.c.scale_head_stride + place] = d;
}

// A thread has PER rows, a grid apart, whose chains of loads and a store run side by
// side.  The rows are written nontemporally: what reads them next does so from memory.
template <typename T, int LANES, int PER>
__global__ __launch_bounds__(THREADS) void k_cache_read(RowsArgs a) {
    const uint32_t first = (blockIdx.x * THREADS + threadIdx.x) / LANES, step = gridDim.x * (THREADS / LANES),
                   at = (threadIdx.x & (LANES - 1)) * VEC;
    if (at >= a.c.d) return;
    Row row[PER];
    int64_t slot[PER];
    bool ok[PER];
    uint2 u[PER];
    float d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t r = first + i * step;
        row[i] = row_of(a, r < a.rows ? r : a.rows - 1);
        slot[i] = a.slots[row[i].token];
        ok[i] = (uint64_t)slot[i] < (uint64_t)a.c.n_pages << a.c.page_shift;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {               // a slot outside the cache reads the first one
        const int64_t in = ok[i] ? slot[i] : 0, page = in >> a.c.page_shift, place = in & ((1ll << a.c.page_shift) - 1);
        const int8_t* p =
            (row[i].value ? a.c.v : a.c.k) + page * a.c.page_stride + row[i].head * a.c.head_stride + place * a.c.token_stride;
        u[i] = *reinterpret_cast<const uint2*>(p + at);
        d[i] = (row[i].value ? a.c.v_scale : a.c.k_scale)[page * a.c.scale_page_stride + row[i].head * a.c.scale_head_stride + place];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (first + i * step >= a.rows) break;
        T y[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float x = (float)(int8_t)((j < 4 ? u[i].x : u[i].y) >> (8 * (j & 3))) * d[i];
            from_f32(y[j], ok[i] ? x : 0.0f);
        }
        T* o = row[i].value ? (T*)a.v + row[i].token * a.v_token + row[i].head * a.v_head
                            : (T*)a.k + row[i].token * a.k_token + row[i].head * a.k_head;
        store_vec<true>(o + at, y);
    }
}

template <typename T, bool WRITE>
int launch_rows(const RowsArgs& a, hipStream_t stream) {
    auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        constexpr int64_t PER_BLOCK = THREADS / L;
        // Reading more rows than threads run at a time: four rows a thread (65536 x 8 x
        // 128 to bf16 83 us, 4.9 TB/s, and 91 with one; with ordinary stores 88).
        // Writing gained nothing from it (8192 x 8 x 128 bf16: 13.3 us and 12.8).
        const bool many = !WRITE && a.rows >= 4 * 2048 * PER_BLOCK;
        const int64_t blocks = (a.rows + (many ? 4 : 1) * PER_BLOCK - 1) / ((many ? 4 : 1) * PER_BLOCK);
        if (blocks > most_blocks(THREADS)) return (int)MOEQ8_EUNSUPPORTED;
        void (*kernel)(RowsArgs);
        if constexpr (WRITE) kernel = k_cache_write<T, L>;
        else kernel = many ? k_cache_read<T, L, 4> : k_cache_read<T, L, 1>;
        hipLaunchKernelGGL(kernel, dim3((uint32_t)blocks), dim3(THREADS), 0, stream, a);
        return check_launch();
    };
    const uint32_t vectors = a.c.d / VEC;
    if (vectors <= 2) return go(std::integral_constant<int, 2>{});
    if (vectors <= 4) return go(std::integral_constant<int, 4>{});
    if (vectors <= 8) return go(std::integral_constant<int, 8>{});
    if (vectors <= 16) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
}

template <bool WRITE>
int cache_rows(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head, int32_t dtype,
               int64_t n_tokens, const int64_t* slots, const moeq8_kv_cache* cache, hipStream_t stream) {
    RowsArgs a;
    if (dtype < MOEQ8_F32 || dtype > MOEQ8_BF16 || n_tokens < 0) return MOEQ8_EINVAL;
    if (const int s = check_cache(cache, a.c)) return s;
    if (n_tokens == 0) return MOEQ8_OK;
    if (!k || !v || !slots) return MOEQ8_EINVAL;
    const int64_t heads = a.c.n_heads, d = a.c.d, es = dtype_bytes(dtype);
    for (const int64_t s : {k_head, v_head})
        if (heads > 1 && s < d) return MOEQ8_EINVAL;
    for (const int64_t s : {k_token, v_token})
        if (n_tokens > 1 && s < d) return MOEQ8_EINVAL;
    if (((uintptr_t)k | (uintptr_t)v) & (uintptr_t)(es - 1) || (uintptr_t)slots & 7u) return MOEQ8_EALIGN;
    if (n_tokens > (1ll << 31) / (2 * heads)) return MOEQ8_EUNSUPPORTED;
    const int64_t k_bytes = ((n_tokens - 1) * k_token + (heads > 1 ? (heads - 1) * k_head : 0) + d) * es;
    const int64_t v_bytes = ((n_tokens - 1) * v_token + (heads > 1 ? (heads - 1) * v_head : 0) + d) * es;
    if (clashes_with_cache(a.c, k, k_bytes) || clashes_with_cache(a.c, v, v_bytes)) return MOEQ8_EINVAL;
    // what is written lies apart from itself and from the slots, which other rows still read
    const int64_t slot_bytes = 8 * n_tokens;
    if (WRITE) {
        if (overlaps_itself(a.c) || clashes_with_cache(a.c, slots, slot_bytes)) return MOEQ8_EINVAL;
    } else {
        const Pieces ko{k, d * es, {n_tokens, heads, 1}, {k_token * es, k_head * es, 0}};
        const Pieces vo{v, d * es, {n_tokens, heads, 1}, {v_token * es, v_head * es, 0}};
        if (pieces_overlap(ko, vo) || ranges_overlap(slots, slot_bytes, k, k_bytes) || ranges_overlap(slots, slot_bytes, v, v_bytes))
            return MOEQ8_EINVAL;
    }
    a.k = const_cast<void*>(k); a.k_token = k_token; a.k_head = k_head;
    a.v = const_cast<void*>(v); a.v_token = v_token; a.v_head = v_head;
    a.slots = slots;
    a.tokens = (uint32_t)n_tokens;
    a.rows = (uint32_t)(2 * n_tokens * heads);
    switch (dtype) {
        case MOEQ8_F32: return launch_rows<float, WRITE>(a, stream);
        case MOEQ8_F16: return launch_rows<f16_t, WRITE>(a, stream);
        default: return launch_rows<bf16_t, WRITE>(a, stream);
    }
}

}  // namespace
}  // namespace moeq8

extern "C" int kv_cache_write_i8(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                 int64_t v_token_stride, int64_t v_head_stride, int32_t dtype, int64_t n_tokens,
                                 const int64_t* slots, const moeq8_kv_cache* cache, void* stream) {
    return moeq8::cache_rows<true>(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, dtype, n_tokens, slots,
                                   cache, (hipStream_t)stream);
}

extern "C" int kv_cache_read_i8(const moeq8_kv_cache* cache, const int64_t* slots, int64_t n_tokens, int32_t dtype,
                                void* k_out, int64_t k_token_stride, int64_t k_head_stride, void* v_out,
                                int64_t v_token_stride, int64_t v_head_stride, void* stream) {
    return moeq8::cache_rows<false>(k_out, k_token_stride, k_head_stride, v_out, v_token_stride, v_head_stride, dtype, n_tokens,
                                    slots, cache, (hipStream_t)stream);
}

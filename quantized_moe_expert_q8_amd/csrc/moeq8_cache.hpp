// The paged key/value cache as the kernels see it, and the host's checks of it.
#pragma once

#include "moeq8_codes.hpp"
#include "moeq8_host.hpp"

namespace moeq8 {

struct Cache {
    int8_t* k; float* k_scale;
    int8_t* v; float* v_scale;
    int64_t page_stride, head_stride, token_stride;
    int64_t scale_page_stride, scale_head_stride;
    uint32_t n_pages, n_heads, page_shift, d;
};

// Status of a cache's description; `out` is filled where it is MOEQ8_OK.
inline int check_cache(const moeq8_kv_cache* c, Cache& out) {
    if (!c || !c->k || !c->k_scale || !c->v || !c->v_scale) return MOEQ8_EINVAL;
    if (c->n_pages < 1 || c->n_heads < 1 || c->page_size < 1 || c->d < 1) return MOEQ8_EINVAL;
    if (c->page_size < 16 || (c->page_size & (c->page_size - 1)) || c->d % 16 || c->d > MOEQ8_MAX_HEAD_DIM)
        return MOEQ8_EUNSUPPORTED;
    if (c->n_pages >= (1ll << 31) || c->n_heads >= (1 << 20) || c->page_size >= (1 << 24)) return MOEQ8_EUNSUPPORTED;
    if (c->token_stride < c->d || (c->n_heads > 1 && c->head_stride < c->d) || (c->n_pages > 1 && c->page_stride < c->d))
        return MOEQ8_EINVAL;
    if ((c->n_heads > 1 && c->scale_head_stride < c->page_size) || (c->n_pages > 1 && c->scale_page_stride < c->page_size))
        return MOEQ8_EINVAL;
    const int64_t hs = c->n_heads > 1 ? c->head_stride : 0, ps = c->n_pages > 1 ? c->page_stride : 0;
    const int64_t sh = c->n_heads > 1 ? c->scale_head_stride : 0, sp = c->n_pages > 1 ? c->scale_page_stride : 0;
    if (((uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 15u) return MOEQ8_EALIGN;
    if (((uint64_t)c->token_stride | (uint64_t)hs | (uint64_t)ps) & 15u || ((uint64_t)sh | (uint64_t)sp) & 3u)
        return MOEQ8_EALIGN;
    out = Cache{c->k, c->k_scale, c->v, c->v_scale, ps, hs, c->token_stride, sp, sh, (uint32_t)c->n_pages,
                (uint32_t)c->n_heads, (uint32_t)__builtin_ctzll((uint64_t)c->page_size), (uint32_t)c->d};
    return MOEQ8_OK;
}

// Whether `bytes` bytes at p overlap any of the cache's four arrays.
inline bool clashes_with_cache(const Cache& c, const void* p, int64_t bytes) {
    const int64_t places = 1ll << c.page_shift;
    const int64_t codes = (c.n_pages - 1ll) * c.page_stride + (c.n_heads - 1ll) * c.head_stride +
                          (places - 1) * c.token_stride + c.d;
    const int64_t scales = 4 * ((c.n_pages - 1ll) * c.scale_page_stride + (c.n_heads - 1ll) * c.scale_head_stride + places);
    return ranges_overlap(p, bytes, c.k, codes) || ranges_overlap(p, bytes, c.v, codes) ||
           ranges_overlap(p, bytes, c.k_scale, scales) || ranges_overlap(p, bytes, c.v_scale, scales);
}

// Whether any two of the cache's four arrays overlap.
inline bool overlaps_itself(const Cache& c) {
    const int64_t pages = c.n_pages, heads = c.n_heads, places = 1ll << c.page_shift;
    auto codes = [&](const void* p) { return Pieces{p, c.d, {pages, heads, places}, {c.page_stride, c.head_stride, c.token_stride}}; };
    auto scales = [&](const void* p) { return Pieces{p, 4 * places, {pages, heads, 1}, {4 * c.scale_page_stride, 4 * c.scale_head_stride, 0}}; };
    const Pieces all[] = {codes(c.k), codes(c.v), scales(c.k_scale), scales(c.v_scale)};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (pieces_overlap(all[i], all[j])) return true;
    return false;
}

}  // namespace moeq8

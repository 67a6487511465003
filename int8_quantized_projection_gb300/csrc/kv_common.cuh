// kv_common.cuh -- what the paged key/value cache's kernels share: the checks
// of a cache descriptor, the error bits, and division by a product.
#pragma once

#include "q8_common.cuh"

namespace q8 {

inline int kv_element_bytes(const q8_kv_cache &c) { return c.dtype == Q8_KV_F16 ? 2 : 1; }

// Rows of one layer (a row: one token's values of one head).
inline int64_t kv_layer_rows(const q8_kv_cache &c)
{
    return c.n_pages * c.kv_heads * static_cast<int64_t>(c.page_size);
}

inline bool kv_pages_ok(int64_t page_size, int64_t n_pages)
{
    return page_size >= 16 && page_size % 16 == 0 && page_size < (int64_t(1) << 31) && n_pages >= 1 &&
           n_pages < (int64_t(1) << 31) && n_pages * page_size < (int64_t(1) << 31);
}

// Q8_OK, or what a call returns for this descriptor.
inline int kv_cache_status(const q8_kv_cache *c)
{
    if (!c || !c->k || !c->v || c->layers < 1 || c->kv_heads < 1 || c->kv_heads > 1024) return Q8_ERR_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return Q8_ERR_ARG;
    if (c->dtype != Q8_KV_F16 && c->dtype != Q8_KV_INT8) return Q8_ERR_ARG;
    if ((c->dtype == Q8_KV_INT8) != (c->k_scale != nullptr) || (c->dtype == Q8_KV_INT8) != (c->v_scale != nullptr))
        return Q8_ERR_ARG;
    if (!kv_pages_ok(c->page_size, c->n_pages)) return Q8_ERR_ARG;
    if (kv_layer_rows(*c) >= (int64_t(1) << 31)) return Q8_ERR_ARG;
    if (c->layers > (int64_t(1) << 31) / 2) return Q8_ERR_ARG;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale)) return Q8_ERR_ALIGN;
    return Q8_OK;
}

// An array of a call; {nullptr, any} where it has none.
struct Span {
    const void *p;
    int64_t bytes;
};

// Whether one of the first `outs` arrays shares a byte with any other of the n.  A CTA writes its part of an output while
// others still read the inputs, so an output in an input's place would change what they compute.
inline bool outputs_overlap(const Span *a, int outs, int n)
{
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j) {
            const uintptr_t x = reinterpret_cast<uintptr_t>(a[i].p), y = reinterpret_cast<uintptr_t>(a[j].p);
            if (x && y && x < y + a[j].bytes && y < x + a[i].bytes) return true;
        }
    return false;
}

// max(a, b), NaN when either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// n / d by a product, for 0 <= n < 2^31 (a division takes some 40 instructions).  inv = kv_inverse(d) is 2^32 / d
// rounded up, or 2^32 - 1 for d = 1: n * inv / 2^32 is off by at most one either way.  n < 0 gives some value.
inline unsigned kv_inverse(int64_t d) { return d == 1 ? ~0u : ~0u / static_cast<unsigned>(d) + 1; }

__device__ __forceinline__ int kv_divide(int n, int d, unsigned inv)
{
    const int q = __umulhi(n, inv), r = n - q * d;
    return q + (r >= d) - (r < 0);
}

} // namespace q8

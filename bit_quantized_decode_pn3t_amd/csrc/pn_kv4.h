// pn_kv4.h - the paged pn4t cache as its kernels and entry points see it
// (layout and rules: include/pn.h).  Internal to libpn.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pn_host.h"

namespace pn {

// A cache, by value into kernels.
struct Kv4 {
    uint8_t *pages;
    int32_t num_pages;
    int32_t shift;  // log2(page_size)
    int32_t heads;
    int32_t chunk;  // bytes of one head in one page
};

// Byte offsets inside one head of a page of P tokens.
template <int D> struct Kv4Layout {
    static constexpr int R = D / 64;       // blocks of a head
    static constexpr int W = D / 8;        // code words of a row
    static constexpr int kRow = D / 2;     // bytes of a row's codes
    static constexpr int chunk(int P) { return P * (2 * kRow + 4 * R); }
    __host__ __device__ static constexpr int v_codes(int P) { return P * kRow; }
    __host__ __device__ static constexpr int k_scales(int P) { return 2 * P * kRow; }
    __host__ __device__ static constexpr int v_scales(int P) { return 2 * P * kRow + 2 * P * R; }
    // natural word w of token o
    __host__ __device__ static constexpr int k_word(int o, int w)
    {
        return o * kRow + 4 * ((w & 3) * 2 * R + 2 * (w >> 3) + ((w >> 2) & 1));
    }
    __host__ __device__ static constexpr int v_word(int o, int w) { return 4 * (((o >> 2) * W + w) * 4 + (o & 3)); }
};

namespace host {

inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline int page_shift(int page_size)
{
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

inline bool dim_ok(int dim) { return dim == 64 || dim == 128 || dim == 256; }

// Checks shared by the entry points that take a cache; fills `out`.
inline pn_status check_cache(const pn_kv4_cache *c, Kv4 *out)
{
    if (!c || !c->pages) return PN_EINVAL;
    const int shift = page_shift(c->page_size);
    if (shift < 0 || !dim_ok(c->dim) || c->heads < 1 || c->num_pages < 1) return PN_ESHAPE;
    if (!aligned(c->pages, 16)) return PN_EALIGN;
    const int chunk = c->page_size * (c->dim + c->dim / 16);
    if (c->heads > 65535 || (int64_t)c->heads * chunk > INT32_MAX) return PN_EUNSUPPORTED;  // a page's bytes are an int
    out->pages = (uint8_t *)c->pages;
    out->num_pages = c->num_pages;
    out->shift = shift;
    out->heads = c->heads;
    out->chunk = chunk;
    return PN_OK;
}

}  // namespace host
}  // namespace pn

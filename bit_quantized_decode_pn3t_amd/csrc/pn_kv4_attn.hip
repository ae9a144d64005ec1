// pn_kv4_attn.hip - the entry points of attention over the paged pn4t cache
// (pn_kv4_attn), for AMD Instinct MI355X (gfx950).  The kernels: pn_kv4_attn.h.
#include "pn_kv4_attn.h"

extern "C" size_t pn_kv4_attn_workspace(const pn_kv4_cache *cache, int q_heads, int B, int64_t total_q, int64_t max_q,
                                        int64_t max_kv, int window, int sinks)
{
    Kv4 c;
    if (check_cache(cache, &c) || !sizes_ok(cache, q_heads, B, total_q, max_q, max_kv, sinks) || total_q == 0) return 0;
    if (max_q > total_q) max_q = total_q;
    if (!sizes_fit(cache, q_heads, B, total_q, max_q, max_kv)) return 0;
    const Cut t = cut(cache, q_heads, B, max_q, max_kv, window, sinks);
    return t.whole ? 0 : t.workers * t.part;
}

extern "C" pn_status pn_kv4_attn(const pn_kv4_cache *cache, const uint16_t *q, int64_t ldq, int q_heads,
                                 const int32_t *q_start, const int32_t *kv_len, const int32_t *table, int64_t ld_table,
                                 int B, int64_t total_q, int64_t max_q, int64_t max_kv, float scale, int window,
                                 int sinks, uint16_t *out, int64_t ldo, void *ws, size_t ws_bytes, void *stream)
{
    AttnArgs a = {};
    if (const pn_status st = check_cache(cache, &a.c)) return st;
    if (!q || !q_start || !kv_len || !table || !out || (!ws && ws_bytes)) return PN_EINVAL;
    if (!sizes_ok(cache, q_heads, B, total_q, max_q, max_kv, sinks)) return PN_ESHAPE;
    if (!scale_ok(scale)) return PN_ESHAPE;
    const int64_t cols = (int64_t)q_heads * cache->dim;
    if (ldq < cols || ldo < cols) return PN_ESHAPE;
    const int64_t pages = (max_kv + cache->page_size - 1) / cache->page_size;
    if (ld_table < pages) return PN_ESHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || ldq % 8 || ldo % 8 || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
        !aligned(table, 4) || !aligned(ws, 16))
        return PN_EALIGN;
    if (max_q > total_q) max_q = total_q;  // no request has more
    if (!sizes_fit(cache, q_heads, B, total_q, max_q, max_kv)) return PN_EUNSUPPORTED;
    if (total_q == 0) return PN_OK;
    Cut t = cut(cache, q_heads, B, max_q, max_kv, window, sinks);
    a.q = q;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = table;
    a.out = out;
    a.ldq = ldq;
    a.ldo = ldo;
    a.ld_table = ld_table;
    a.total_q = total_q;
    a.max_q = max_q;
    a.max_kv = max_kv;
    a.q_heads = q_heads;
    a.group = q_heads / cache->heads;
    a.B = B;
    a.max_pages = (int)pages;
    a.window = window;
    a.sinks = sinks;
    set_scale(a, scale);
    set_cut(a, cache, t, ws, ws_bytes);
    if (!once_per_device(kAttrKv4, raise_pass<kWhole>)) return PN_ELAUNCH;
    const pn_status st = launch_pass<kWhole>(a, t, cache->dim, (hipStream_t)stream);
    if (st == PN_OK) g_last_variant = t.rg == kWaves ? kVarKv4Prompt : kVarKv4Attn;
    return st;
}

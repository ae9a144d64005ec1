// pn_kv4_shared.hip - attention for requests that share a long prefix
// (pn_kv4_attn_shared), for AMD Instinct MI355X (gfx950).
//
//   out = (sum_front w v + sum_own w v) / (sum_front w + sum_own w)
//
// The first launch (kFront) takes the queries of a whole group as the rows of
// one attention over the shared keys, which every one of them sees whole: a key
// is unpacked and multiplied for all rows of a tile at once.  The rows' sums
// stay in fp32, relative to their own maxima, and in as many parts as
// workgroups shared a tile's keys.  The second launch gives each request's
// queries its own keys and joins them with those parts: a workgroup an item
// (kOwn), or dealt as pn_kv4_attn deals them, with its join (kTail).
//
// A tile is up to four 16-row groups, two where heads are 256 wide: what the
// registers hold.  Its eight waves take every eighth step of 32 tokens and do
// not wait for one another.  A form whose waves unpacked the keys together into
// LDS had a barrier a step: 64 requests behind 16384 tokens 71 us and 32 behind
// 65536 161, this form's first version 61 and 115.
//
// What bounds it: issue of vector instructions and products, and what is run
// once.  64 requests behind 16384 tokens, 128 wide (25.8 GFLOP): kFront 56.5 us,
// vector instructions active 56 % of a SIMD's time, products 24 %, which barely
// overlap (two waves a SIMD of 32 products and 128 fma each, ns: 463 and 483
// alone, 778 one after the other).  kOwn 17.6: about 5 until its first step, 5
// for that and the waves' join, 5 for further steps, 3.6 for the front's parts.
// 32 behind 65536, 256 wide (51.5 GFLOP): 112 us, vector instructions 62 %,
// then 24.4 and 11.3.  Each request by pn_kv4_attn instead, passes of one run:
// 64 requests 230 us (here 75), 32 393 (137); 16 of 8 drafts behind 5024 71.0
// (71.7) and 4 behind 1024 16.8 (19.4): there sharing does not pay.
#include "pn_kv4_attn.h"

namespace {

// The launches of a call.
struct Plan {
    Cut front, own;
    bool line;        // the requests' own keys are dealt as a line (kTail), not a workgroup an item (kOwn)
    int tiles;        // kOwn: of a request
    int64_t tile;     // rows of kFront's tiles
    int64_t grid;     // kFront's workgroups
    size_t members, items, front_ml, front_parts, own_parts;  // bytes
    size_t bytes() const { return members + items + front_ml + front_parts + own_parts; }
};

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

// n spread over as few tiles of up to `most` as hold it: tiles, and the largest.
void spread(int64_t n, int most, int64_t &tiles, int64_t &each)
{
    tiles = (n + most - 1) / most;
    each = (n + tiles - 1) / tiles;
}

Plan plan(const pn_kv4_cache *c, int q_heads, int B, int G, int64_t total_q, int64_t max_q, int64_t max_kv, int64_t max_shared)
{
    Plan p;
    const int group = q_heads / c->heads, most = c->dim == 256 ? 2 : 4;  // row groups of a wave that the registers hold
    int64_t tiles, each;
    // No group has more rows than there are; a tile takes no more than it needs.
    spread((total_q * group + 15) / 16, most, tiles, each);
    if (G > 1 && tiles > 1) each = most;
    p.front.nt = (int)each;
    p.front.rg = 1;
    p.front.two = c->dim < 256 && each == 1;
    p.front.workers = device_cus() * (p.front.two ? 2 : 1);
    p.front.whole = false;
    p.front.parts = 0;
    p.tile = 16 * each;
    const int64_t items = (total_q * group / p.tile + G) * c->heads;  // at most
    p.grid = 1 + (G > 64 ? p.front.workers + items : items > p.front.workers - 1 ? items : p.front.workers - 1);
    p.own = cut(c, q_heads, B, max_q, max_kv, 0, 0);
    spread((max_q * group + 15) / 16, most, tiles, each);
    p.tiles = (int)tiles;
    // What requests behind the longest prefix have of their own; others may have more, which only costs time
    // (one of 64 outside of the group with 16616 keys of its own: 73 -> 166 us).
    const int64_t tails = max_kv - max_shared * c->page_size;
    // A line where tails are long and items few (32 requests of up to 4000 own
    // tokens, 256 wide: a workgroup an item 61.6 us, a line 31.7 and 17.0 for its
    // join when this was taken); else an item a workgroup (64 requests of up to
    // 1000, 128 wide: 22.1 us, a line 30.3 before its join).
    p.line = p.own.rg > 1 || (tails > 2 * kShare * kStep && B * c->heads * tiles < 2 * device_cus());
    if (!p.line) {
        p.own.nt = (int)each;
        p.own.whole = true;
    }
    p.members = (size_t)B * sizeof(Member);
    p.items = round16((size_t)(total_q * group / p.tile + G + 1) * c->heads * sizeof(int2));
    p.front_ml = (size_t)p.grid * p.tile * sizeof(float2);
    p.front_parts = (size_t)p.grid * p.tile * c->dim * sizeof(float);
    p.own_parts = p.own.whole ? 0 : round16(p.own.workers * p.own.part);
    return p;
}

// At least the plan's bytes, and growing with every size: a plan for less may
// need more (fewer rows spread over other tiles, a line where there were items),
// and what is kept for the largest call has to serve it.  The front's rows are
// counted with the largest tile that the rows allow, the own keys' parts as if
// every call dealt them as a line.
size_t room(const pn_kv4_cache *c, int q_heads, int B, int G, int64_t total_q, int64_t max_q, int64_t max_kv)
{
    const int64_t rows = total_q * (q_heads / c->heads), groups = (rows + 15) / 16;
    const int64_t most = c->dim == 256 ? 2 : 4, least = c->dim == 256 ? 1 : 2;  // least: two workgroups share a compute unit
    const int64_t tile = 16 * (groups < least ? least : groups < most ? groups : most);
    const int64_t units = device_cus() * tile, items = (rows + G * 16 * most) * c->heads;
    const int64_t front = tile + (G > 64 ? units + items : units > items ? units : items);
    size_t n = B * sizeof(Member) + round16((size_t)(rows / 16 + G + 1) * c->heads * sizeof(int2));
    n += (size_t)front * (sizeof(float2) + c->dim * sizeof(float));
    if (max_kv > 2 * kShare * kStep) {  // else no item is cut
        const Cut t = cut(c, q_heads, B, max_q, max_kv, 0, 0);
        Cut all = t;
        if (t.rg == 1 && t.nt < least) all.nt = (int)least;
        n += round16(device_cus() * (part_bytes(c, all) + sizeof(Cutoff)));
    }
    return n;
}

bool shared_fit(const pn_kv4_cache *c, int q_heads, int B, int G, int64_t total_q, int64_t max_q, int64_t max_kv,
                int64_t max_shared)
{
    const int64_t rows = total_q * (q_heads / c->heads);
    return sizes_fit(c, q_heads, B, total_q, max_q, max_kv) && G <= 65535 && max_shared <= INT32_MAX / 2 / c->page_size &&
           rows <= INT32_MAX / 4 && (rows / 16 + G) * c->heads <= INT32_MAX / 2 && (max_q * (q_heads / c->heads) / 16 + 1) * B * c->heads <= INT32_MAX;
}

// A launch holds less than 2^32 threads.
bool launches_fit(const Plan &p, const pn_kv4_cache *c, int B)
{
    constexpr int64_t most = (int64_t)UINT32_MAX / kThreads;
    return p.grid <= most && (p.line || (int64_t)B * c->heads * p.tiles <= most);
}

bool raise_shared()
{
    return raise_pass<kFront>() && raise_pass<kTail>() && raise_pass<kOwn>();
}

}  // namespace

extern "C" size_t pn_kv4_attn_shared_workspace(const pn_kv4_cache *cache, int q_heads, int B, int G, int64_t total_q,
                                               int64_t max_q, int64_t max_kv, int64_t max_shared)
{
    Kv4 c;
    if (check_cache(cache, &c) || !sizes_ok(cache, q_heads, B, total_q, max_q, max_kv, 0) || G < 1 || max_shared < 1 ||
        total_q == 0)
        return 0;
    if (max_q > total_q) max_q = total_q;
    const int64_t pages = (max_kv + cache->page_size - 1) / cache->page_size;
    if (max_shared > pages) max_shared = pages;
    if (!shared_fit(cache, q_heads, B, G, total_q, max_q, max_kv, max_shared)) return 0;
    const Plan p = plan(cache, q_heads, B, G, total_q, max_q, max_kv, max_shared);
    return launches_fit(p, cache, B) ? room(cache, q_heads, B, G, total_q, max_q, max_kv) : 0;
}

extern "C" pn_status pn_kv4_attn_shared(const pn_kv4_cache *cache, const uint16_t *q, int64_t ldq, int q_heads,
                                        const int32_t *q_start, const int32_t *kv_len, const int32_t *table,
                                        int64_t ld_table, int B, const int32_t *g_start, const int32_t *prefix,
                                        int64_t ld_prefix, const int32_t *shared, int G, int64_t total_q, int64_t max_q,
                                        int64_t max_kv, int64_t max_shared, float scale, uint16_t *out, int64_t ldo,
                                        void *ws, size_t ws_bytes, void *stream)
{
    AttnArgs a = {};
    if (const pn_status st = check_cache(cache, &a.c)) return st;
    if (!q || !q_start || !kv_len || !table || !g_start || !prefix || !shared || !out || (!ws && total_q > 0)) return PN_EINVAL;
    if (!sizes_ok(cache, q_heads, B, total_q, max_q, max_kv, 0) || G < 1 || max_shared < 1) return PN_ESHAPE;
    if (!scale_ok(scale)) return PN_ESHAPE;
    const int64_t cols = (int64_t)q_heads * cache->dim;
    if (ldq < cols || ldo < cols) return PN_ESHAPE;
    const int64_t pages = (max_kv + cache->page_size - 1) / cache->page_size;
    if (ld_table < pages || ld_prefix < max_shared) return PN_ESHAPE;
    const void *words[] = {q_start, kv_len, table, g_start, prefix, shared};
    for (const void *p : words)
        if (!aligned(p, 4)) return PN_EALIGN;
    if (!aligned(q, 16) || !aligned(out, 16) || ldq % 8 || ldo % 8 || !aligned(ws, 16)) return PN_EALIGN;
    if (max_q > total_q) max_q = total_q;  // no request has more
    if (max_shared > pages) max_shared = pages;
    if (!shared_fit(cache, q_heads, B, G, total_q, max_q, max_kv, max_shared)) return PN_EUNSUPPORTED;
    if (total_q == 0) return PN_OK;
    Plan p = plan(cache, q_heads, B, G, total_q, max_q, max_kv, max_shared);
    if (!launches_fit(p, cache, B)) return PN_EUNSUPPORTED;
    if (ws_bytes < p.bytes()) return PN_ESHAPE;
    if (!once_per_device(kAttrKv4Shared, raise_shared)) return PN_ELAUNCH;

    uint8_t *at = (uint8_t *)ws;
    auto take = [&](size_t n) { uint8_t *x = at; at += n; return x; };
    a.members = (Member *)take(p.members);
    a.items = (int2 *)take(p.items);
    a.part_ml = (float2 *)take(p.front_ml);
    a.part = (float *)take(p.front_parts);
    uint8_t *own_parts = take(p.own_parts);
    a.g_start = g_start;
    a.g_pages = shared;
    a.requests = B;
    a.groups = G;
    a.max_shared = (int)max_shared;
    a.q = q;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.out = out;
    a.ldq = ldq;
    a.ldo = ldo;
    a.total_q = total_q;
    a.max_kv = max_kv;
    a.q_heads = q_heads;
    a.group = q_heads / cache->heads;
    set_scale(a, scale);
    const hipStream_t s = (hipStream_t)stream;

    a.table = prefix;
    a.ld_table = ld_prefix;
    a.max_pages = (int)max_shared;
    a.max_q = total_q;  // of a group
    a.B = G;
    a.f_tile = (int)p.tile;
    a.f_part = a.part;
    a.f_part_ml = a.part_ml;
    a.workers = p.front.workers;
    a.grid = (int)p.grid;
    a.least = kWaves;
    pn_status st = launch_pass<kFront>(a, p.front, cache->dim, s);
    if (st != PN_OK) return st;

    a.table = table;
    a.ld_table = ld_table;
    a.max_pages = (int)pages;
    a.max_q = max_q;
    a.B = B;
    a.tiles = p.tiles;
    set_cut(a, cache, p.own, own_parts, p.own_parts);
    st = p.line ? launch_pass<kTail>(a, p.own, cache->dim, s) : launch_pass<kOwn>(a, p.own, cache->dim, s);
    if (st == PN_OK) g_last_variant = kVarKv4AttnShared;
    return st;
}

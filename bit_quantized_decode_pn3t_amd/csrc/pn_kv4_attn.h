// pn_kv4_attn.h - the kernels of attention over the paged pn4t cache
// (pn_kv4_attn, pn_kv4_attn_shared), for AMD Instinct MI355X (gfx950).
// Internal to libpn.so.
//
//   out = sum_t w_t v_t / sum_t w_t,   w_t = exp2(c (s_t - m)),  c = scale log2(e)
//   s_t = sum_b dk[t][b] * (sum over block b of q . (n_k - 8))
//
// One pass over the keys with a running maximum and sum for each row (rows:
// the queries of a request times the query heads that share a key-value
// head).  A wave takes 16 NT rows and steps through 32 tokens at a time:
//   S^T = K Q^T   v_mfma_f32_16x16x32_f16, A = 16 tokens, B = 16 rows.  A code
//                 word is one lane's 8 elements of A: the cache keeps a row's
//                 words in the order that gives each lane its words of all
//                 blocks side by side, and every product lies in one block, so
//                 the codes enter as exact small integers and the block's
//                 scale multiplies the fp32 sum.
//   O^T += V^T P  A = 16 elements x 32 tokens, B = P^T.  A score's place after
//                 the first product is already a lane's place of B: tokens
//                 4 g .. 4 g + 3 of both 16-token tiles.  Weights and values
//                 (scale times code) are rounded once each to fp16, half a
//                 step, 2^-11 relative: with the scale in the weights instead
//                 the codes would be exact, but each block of the head then
//                 needs weights of its own (48 query heads, a prompt of 4096,
//                 128 wide: 0.60 ms that way and 0.51 this way, in kv4_attn).
//                 Neither factor leaves fp16's full precision: the running
//                 maximum m follows only scores that pass it by 4 (in log2),
//                 so that O is rarely scaled, and weights carry 2^10: they
//                 stay below 2^14, normal down to 2^-24 of the largest.
//                 Scales may have any fp16 size, so each wave keeps a power of
//                 two 2^u that puts the scales it has met below 2^7 at first
//                 and 2^11 at most, values below 2^14.  It is a factor in
//                 fp16, so u is at most 15: the smallest subnormal scale then is
//                 2^-9, and products with codes stay normal.
// A row of A is element 2 i + (r >> 3) of word r & 7 of a block (r = lane &
// 15, product i < 4), so that one product stays in one block; two v_perm-ed
// words give the token pairs.
//
// Packed bytes go from the pages into LDS by DMA, a few steps ahead, each
// wave into a ring of its own (no barrier in the loop); a key row's 16-byte
// pieces are permuted on the way so that the reads spread over the banks.
//
// Work is dealt in equal shares, whatever the lengths: the items (request,
// key-value head, row tile), each about as long as the steps it sees and what
// its start and end cost, form one line that the workgroups cut into equal
// parts.  Every workgroup sums the requests for itself and finds its items;
// an item cut between workgroups leaves parts in the workspace, which
// kv4_join adds.  With few rows (RG = 1) a workgroup's eight waves take every
// eighth step of the same rows; with more (RG = 4) four groups of two waves
// take rows of their own and share the staged steps, one of two each.  The
// waves of the same rows are joined through LDS.  All sums have a fixed order.
//
// What bounds it: latency; no pipe is full.  One 256-wide token over 65536 keys
// (4 key-value heads, 71 MB): 26.5 us and 7.8 for the join, 2.1 TB/s in all,
// vector instructions 33 % of the time: four steps a wave between code that is
// run once.  64 128-wide requests of up to 16384 (135 MB): 54 and 5.3, 2.3
// TB/s, vector instructions (half of one a code) 45 % of the time and products
// 7; with 64 full requests of 16384 the loop alone runs at 4.4 to 4.8 TB/s, so
// the rest is where items start and end.  16 requests of 8 drafts over up to
// 5003 keys, 256 wide: 36.7 and 5.5 us.  One token over one key, 64 wide: 9.6
// us, 1.7 of them until a workgroup has its part of the line, 1.4 until it has
// an item, 2.4 until its queries and loads are under way, 2.2 for a step and
// 1.1 to join the waves: code that is run once.  1000 requests of up to 2000,
// 128 wide (313 MB): 212 us.  A 256-wide prompt of 4096 with 24 heads (206
// GFLOP): 536 us and 17.7.
#pragma once

#include <type_traits>

#include "pn_kv4.h"
#include "pn_device.h"

using namespace pn;
using namespace pn::host;

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kThreads = 512;
constexpr int kWaves = 8;
constexpr int kStep = 32;          // tokens of a step
// A maximum before any score: below all of them (65504^2 * 8 * 256 = 9e12), and
// no further, so that its product with a large scale stays finite.
constexpr float kLowest = -1e15f;
constexpr float kBias = 10.0f;     // weights carry 2^kBias
// Steps of a workgroup at least.  One 256-wide token over 8000 keys of two
// heads: 22 us, with 32 27 us; 256 tokens over up to 1024 keys: 81 us, with 4
// 86 us.
constexpr int kShare = 16;
// And of each of two on a compute unit, else one takes the steps of both.
// 64 wide, 4 key-value heads: one token over 65536 keys (16 steps each) 29 us
// with two, 22 with one; 24 requests of up to 16384 (48) 31 and 32; 64 of them
// (128) 54 and 61.
constexpr int kTwo = 48;
constexpr int kNothing = (int)0x80000000;  // an offset past every buffer: reads zero

struct AttnArgs {
    Kv4 c;
    const uint16_t *q;
    const int32_t *q_start, *kv_len, *table;
    uint16_t *out;
    float *part;      // fragments of a workgroup's first and last cut item
    float2 *part_ml;  // their rows' maxima and sums
    struct Cutoff *cuts;  // [workgroup]: the item that it leaves unfinished
    int64_t ldq, ldo, ld_table, total_q;
    int64_t max_q, max_kv;
    int32_t q_heads, group, B, max_pages, window, sinks;
    int32_t workers, whole;  // workgroups; whole: items are not cut
    int32_t two;             // of the workgroups share a compute unit
    int32_t parts;           // that an item is cut into, about
    int32_t queries, grow;   // of a row tile; what a tile's length is more than the last one's (Cost)
    int32_t over;            // what an item's start and end cost, in steps
    int32_t negate;          // scale < 0: the queries are negated
    // Of the passes of requests that share keys:
    const int32_t *g_start, *g_pages;  // the groups' first requests, the pages they share
    struct Member *members;  // [request]
    int2 *items;             // [tile of a group][head]: first part, parts
    const float *f_part;     // the parts that kFront left, as `part` and `part_ml` are
    const float2 *f_part_ml;
    int32_t f_tile;          // rows of a tile of kFront at most
    int32_t requests, groups, max_shared;
    int32_t least;           // kFront: steps of a part at least
    int32_t grid;            // kFront: workgroups; `workers` of them, unless there are more items
    int32_t tiles;           // kOwn: of a request
    float c2;                // |scale| log2(e), above 0
    float slack;             // 4 / c2
};

// What a launch computes.  kWhole: attention.  For requests that share their
// first keys (pn_kv4_attn_shared): kFront, the queries of a whole group against
// the keys that it shares, left in parts as sums with their maxima; kTail and
// kOwn, each request's queries against its own keys, joined with those parts.
// kFront and kOwn give a workgroup one item (a part of one), kWhole and kTail a
// part of the line.
enum Pass { kWhole = 0, kFront = 1, kTail = 2, kOwn = 3 };
constexpr bool joins(int pass) { return pass == kTail || pass == kOwn; }

// What a request takes from its group.
struct Member {
    int32_t skip;  // pages
    int32_t q0;    // the group's first query
    int32_t tile;  // and first place in `items`
    int32_t rows;  // and rows of its tiles
};

// An item whose steps go on in the workgroups behind this one.
struct Cutoff {
    int64_t q0;          // the request's first query
    int32_t row0, rows;  // of the tile, of the request
    int32_t head;        // kTail: and 2^16 times the request
    int32_t parts;       // workgroups that work on it; 0: none is unfinished
};

// The part of a request that a row tile works on.
struct Request {
    int64_t q0;       // first query row of the request
    int32_t qn;       // queries of the request that are computed
    int32_t first;    // position of query 0
    int32_t len;      // keys
    int32_t skip;     // kTail, kOwn: pages ahead of them, whose sums exist
};
struct Work : Request {
    int32_t sink_steps, lo, steps;  // steps [0, sink_steps), then from lo; steps in all
};

// Request b; of kFront, group b as one request that sees all of its keys.
template <int PASS> __device__ __forceinline__ Request request(const AttnArgs &a, int b)
{
    Request w;
    w.skip = 0;
    if constexpr (PASS == kFront) {
        int32_t b0 = a.g_start[b], b1 = a.g_start[b + 1], n = a.g_pages[b];
        b0 = b0 < 0 ? 0 : b0 > a.requests ? a.requests : b0;
        b1 = b1 < b0 ? b0 : b1 > a.requests ? a.requests : b1;
        n = n < 0 ? 0 : n > a.max_shared ? a.max_shared : n;
        int64_t q0 = a.q_start[b0], q1 = a.q_start[b1];
        q0 = q0 < 0 ? 0 : q0 > a.total_q ? a.total_q : q0;
        q1 = q1 < q0 ? q0 : q1 > a.total_q ? a.total_q : q1;
        w.q0 = q0;
        w.qn = n > 0 ? (int32_t)(q1 - q0) : 0;
        w.len = (int64_t)n << a.c.shift < a.max_kv ? n << a.c.shift : (int32_t)a.max_kv;
        w.first = w.len;
        return w;
    }
    int64_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
    q0 = q0 < 0 ? 0 : q0 > a.total_q ? a.total_q : q0;
    q1 = q1 < q0 ? q0 : q1 > a.total_q ? a.total_q : q1;
    const int32_t kv = a.kv_len[b] < 0 ? 0 : a.kv_len[b];
    w.q0 = q0;
    w.first = (int32_t)(kv - (q1 - q0));
    w.qn = (int32_t)(q1 - q0 < a.max_q ? q1 - q0 : a.max_q);
    w.len = kv < a.max_kv ? kv : (int32_t)a.max_kv;
    if constexpr (joins(PASS)) {
        w.skip = a.members[b].skip;
        const int32_t ahead = w.skip << a.c.shift;
        w.first -= ahead;  // not below 0: group_members
        w.len = w.len > ahead ? w.len - ahead : 0;
    }
    return w;
}

// The steps of STEP tokens that queries i0 .. i1 of the request can see.
template <int STEP>
__device__ __forceinline__ void span(const AttnArgs &a, Work &w, int i0, int i1)
{
    int32_t hi = w.first + i1 + 1;
    hi = hi < 0 ? 0 : hi < w.len ? hi : w.len;
    const int32_t end = (hi + STEP - 1) / STEP;
    w.sink_steps = 0;
    w.lo = 0;
    if (a.window > 0) {
        const int64_t from = (int64_t)w.first + i0 - a.window + 1;
        const int32_t lo = from < 0 ? 0 : from < hi ? (int32_t)(from / STEP) : end;
        const int32_t s = a.sinks < hi ? a.sinks : hi;
        const int32_t ss = (s + STEP - 1) / STEP;
        w.sink_steps = ss < lo ? ss : 0;  // sinks that meet the window are one stretch
        w.lo = ss < lo ? lo : 0;
    }
    w.steps = w.sink_steps + (end > w.lo ? end - w.lo : 0);
}

// The last position that the window of a query at `pos` leaves out, -1 or less
// if there is none.  (A query ahead of all keys has a negative position, from
// which a wide window must not be taken off.)
__device__ __forceinline__ int32_t before_window(const AttnArgs &a, int32_t pos)
{
    return a.window > 0 && pos >= 0 ? pos - a.window : -1;
}

// a / b for non-negative a: a 64-bit quotient takes some hundred instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((uint64_t)a | (uint64_t)b) >> 32 == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// The rows of a group's tiles: its 16-row groups spread evenly over as few
// tiles as hold them.
__device__ __forceinline__ int32_t front_rows(const AttnArgs &a, const Request &w)
{
    const int32_t rows = w.qn * a.group, tiles = (rows + a.f_tile - 1) / a.f_tile;
    return tiles > 0 ? ((rows + 15) / 16 + tiles - 1) / tiles * 16 : a.f_tile;
}

// The first place in `items` of group g, whose queries start at q0.
__device__ __forceinline__ int32_t front_tile(const AttnArgs &a, int64_t q0, int g)
{
    return (int32_t)quotient(q0 * a.group, a.f_tile) + g;
}

// kFront: what the requests take from their groups.  A request takes its
// group's part if all of its queries stand behind the shared pages.
__device__ __forceinline__ void group_members(const AttnArgs &a)
{
    for (int b = threadIdx.x; b < a.requests; b += blockDim.x) {
        int lo = 0, hi = a.groups;  // the last group that starts at b or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.g_start[mid] <= b) lo = mid;
            else hi = mid;
        }
        const int32_t b0 = a.g_start[lo], b1 = a.g_start[lo + 1];
        const Request w = request<kWhole>(a, b), group = request<kFront>(a, lo);
        int32_t n = a.g_pages[lo];
        n = n < 0 ? 0 : n > a.max_shared ? a.max_shared : n;
        const bool in = b0 <= b && b < b1 && w.qn > 0 && w.q0 >= group.q0 && w.q0 + w.qn <= group.q0 + group.qn &&
                        w.first >= 0 && (int64_t)n << a.c.shift <= w.first;
        a.members[b] = {in ? n : 0, (int32_t)group.q0, front_tile(a, group.q0, lo), front_rows(a, group)};
    }
}

// What the line counts for request b: its row tiles, and for tile t a length
// of min(base + t grow, top) sixteenths of a step: what its start and end
// cost, and about the steps it sees (a later tile of a prompt more, up to the
// window).  Only the balance depends on these lengths.
constexpr int kUnit = 16;
struct Cost {
    Request w;
    int32_t tiles, base, grow, top;
};

template <int STEP, int PASS>
__device__ __forceinline__ Cost cost(const AttnArgs &a, int b, int tile_rows)
{
    Cost c;
    c.w = request<PASS>(a, b);
    c.tiles = c.base = c.top = c.grow = 0;
    if (c.w.qn < 1) return c;
    c.tiles = (c.w.qn * a.group + tile_rows - 1) / tile_rows;
    int32_t see = c.w.first + (c.w.qn < a.queries ? c.w.qn : a.queries);
    see = see < 0 ? 0 : see < c.w.len ? see : c.w.len;
    int32_t most = c.w.len;
    if (a.window > 0 && (int64_t)a.window + a.sinks + a.queries < most) most = a.window + a.sinks + a.queries;
    const int32_t fixed = (a.over + 1) * kUnit;
    c.top = fixed + (int32_t)((int64_t)most * kUnit / STEP);
    c.base = fixed + (int32_t)((int64_t)see * kUnit / STEP);
    if (c.base > c.top) c.base = c.top;
    c.grow = a.grow;
    return c;
}

// Tiles whose length still grows, and the length of the first t tiles.
__device__ __forceinline__ int32_t growing(const Cost &c)
{
    if (c.base >= c.top) return 0;
    if (c.grow == 0) return c.tiles;
    const int32_t n = (c.top - c.base + c.grow - 1) / c.grow;
    return n < c.tiles ? n : c.tiles;
}
__device__ __forceinline__ int64_t before_tile(const Cost &c, int32_t n, int64_t t)
{
    const int64_t g = t < n ? t : n;
    return g * c.base + g * (g - 1) / 2 * c.grow + (t - g) * c.top;
}
__device__ __forceinline__ int64_t length(const AttnArgs &a, const Cost &c)
{
    if (c.tiles == 1) return (int64_t)c.base * a.c.heads;
    return before_tile(c, growing(c), c.tiles) * a.c.heads;
}

// The same in every lane: into scalar registers.
__device__ __forceinline__ int64_t uniform64(int64_t v)
{
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v));
}
template <int PASS> __device__ __forceinline__ Cost scalar(const Cost &m)
{
    Cost c;
    c.w.q0 = uniform64(m.w.q0);
    c.w.qn = uniform(m.w.qn);
    c.w.first = uniform(m.w.first);
    c.w.len = uniform(m.w.len);
    c.w.skip = joins(PASS) ? uniform(m.w.skip) : 0;
    c.tiles = uniform(m.tiles);
    c.base = uniform(m.base);
    c.grow = uniform(m.grow);
    c.top = uniform(m.top);
    return c;
}

// ---------------------------------------------------------------------------
// A workgroup's part of the line.
// ---------------------------------------------------------------------------
struct LineLds {
    int64_t scan[kWaves];
    int64_t at[2];
    Cost known[64];
};
static_assert(sizeof(LineLds) <= 2944, "two workgroups' LDS (narrow heads, few rows)");

struct Line {
    int64_t lo, hi, share;
    int64_t start;  // of request b on the line
    int32_t b;
    bool few;
};

// Up to 64 requests are summed by every wave for itself and kept in LDS; more
// are summed by the workgroup and read again as they come.  False: nothing is
// left for this workgroup.
template <int STEP, int PASS>
__device__ __forceinline__ bool line_part(const AttnArgs &a, LineLds &s, Line &t, int tile_rows)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    t.few = a.B <= 64;
    const int per = (a.B + kThreads - 1) / kThreads;
    int64_t mine = 0, total = 0, before = 0;
    if (t.few) {
        const Cost c = cost<STEP, PASS>(a, lane < a.B ? lane : 0, tile_rows);
        mine = lane < a.B ? length(a, c) : 0;
        if (wave == 0) s.known[lane] = c;
    } else {
        for (int b = tid * per; b < (tid + 1) * per && b < a.B; ++b) mine += length(a, cost<STEP, PASS>(a, b, tile_rows));
    }
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t x = __shfl_up(sum, d, 64);
        if (lane >= d) sum += x;
    }
    before = sum - mine;
    if (t.few) {
        total = __shfl(sum, 63, 64);
    } else {
        if (lane == 63) s.scan[wave] = sum;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) before += s.scan[w];
            total += s.scan[w];
        }
    }
    total = uniform64(total);
    // A few workgroups fewer than there are: with four items or more no item
    // then has over 64 parts, which is what the join takes at a time.
    // Two workgroups a compute unit only share it: with short parts one does more.
    const int32_t used = a.two && total < (int64_t)a.workers * (kTwo * kUnit) ? a.workers / 2 : a.workers;
    const int32_t dealt = used - used / 64;
    t.share = quotient(total + dealt - 1, dealt);
    if (t.share < kShare * kUnit && !a.whole) t.share = kShare * kUnit;
    t.lo = blockIdx.x * t.share;
    t.hi = t.lo + t.share < total ? t.lo + t.share : total;
    if (tid == 0 && !a.whole) a.cuts[blockIdx.x].parts = 0;
    if (t.lo >= total) return false;  // the whole workgroup
    const bool here = t.lo >= before && t.lo < before + mine;  // one lane of each wave, or one thread
    if (t.few) {
        __syncthreads();
        t.b = __builtin_ctzll(__ballot(here));
        t.start = uniform64(__shfl(before, t.b, 64));
    } else {
        if (here) {
            int x = tid * per;
            for (;; ++x) {
                const int64_t n = length(a, cost<STEP, PASS>(a, x, tile_rows));
                if (t.lo < before + n) break;
                before += n;
            }
            s.at[0] = x;
            s.at[1] = before;
        }
        __syncthreads();
        t.b = uniform((int)s.at[0]);
        t.start = uniform64(s.at[1]);
    }
    return true;
}

// The next item of the part.
struct Item {
    Cost c;
    int32_t s0, s1, all;        // its part [s0, s1) of `all` (lengths on the line)
    int32_t head, tile0, rows;  // the tile's first row, the request's rows
    bool cut;
};

// Steps that a part of an item stands for: the same part of the `steps` it has.
__device__ __forceinline__ int share_of(int32_t s, int32_t all, int steps)
{
    return s == 0 ? 0 : s == all ? steps : uniform((int)quotient((int64_t)s * steps, all));
}

// Go on along the line from x; false: a stretch without an item's steps.
template <int STEP, int PASS>
__device__ __forceinline__ bool next_item(const AttnArgs &a, const LineLds &s, Line &t, int64_t &x, Item &m, int tile_rows)
{
    m.c = scalar<PASS>(t.few ? s.known[t.b] : cost<STEP, PASS>(a, t.b, tile_rows));
    const bool single = m.c.tiles == 1;  // most requests: few instructions, which is what an item's start costs
    const int32_t n = single ? 0 : growing(m.c);
    const int64_t head_len = single ? m.c.base : before_tile(m.c, n, m.c.tiles);
    if (x >= t.start + head_len * a.c.heads) {
        t.start += head_len * a.c.heads;
        ++t.b;
        return false;
    }
    m.head = uniform((int)quotient(x - t.start, head_len));
    int64_t first = t.start + m.head * head_len;  // of the item on the line
    int one = (int)head_len;
    int32_t tile = 0;
    if (!single) {
        // the tile: largest with before_tile <= off
        const int64_t off = x - first, flat = before_tile(m.c, n, n);
        if (off >= flat) {
            tile = n + (int32_t)quotient(off - flat, m.c.top);
        } else if (m.c.grow == 0) {
            tile = (int32_t)quotient(off, m.c.base);
        } else {
            const double h = m.c.base - 0.5 * m.c.grow;
            tile = (int32_t)((__builtin_sqrt(h * h + 2.0 * m.c.grow * (double)off) - h) / m.c.grow);
            if (tile >= n) tile = n - 1;
            if (tile < 0) tile = 0;
            while (tile > 0 && before_tile(m.c, n, tile) > off) --tile;
            while (tile + 1 < n && before_tile(m.c, n, tile + 1) <= off) ++tile;
        }
        tile = uniform(tile);
        const int64_t at = before_tile(m.c, n, tile);
        first += at;
        one = (int)(before_tile(m.c, n, tile + 1) - at);
    }
    int s0 = (int)(x - first), s1 = (int)(t.hi - first < one ? t.hi - first : one);
    x = first + s1;
    if (a.whole) {  // items are taken whole, by the workgroup they start in
        if (s0 > 0) return false;
        s1 = one;
    }
    const int over = a.over * kUnit;  // the first stretch of an item: nobody's steps
    s0 = s0 > over ? s0 - over : 0;
    s1 -= over;
    if (s1 <= s0) return false;
    m.s0 = uniform(s0), m.s1 = uniform(s1), m.all = uniform(one - over);
    m.cut = s0 > 0 || s1 < m.all;
    m.tile0 = tile * tile_rows;
    m.rows = m.c.w.qn * a.group;
    if (m.s0 == 0 && m.cut && threadIdx.x == 0)
        a.cuts[blockIdx.x] = {m.c.w.q0, m.tile0, m.rows, PASS == kTail ? (int32_t)((uint32_t)t.b << 16 | m.head) : m.head,
                              (int)quotient(first + one - 1, t.share) - (int)blockIdx.x + 1};
    return true;
}

// kOwn: the workgroup's one item, a row tile and head of a request.  False: the
// request has no such tile.
__device__ __forceinline__ bool own_item(const AttnArgs &a, Line &t, Item &m, int tile_rows)
{
    const uint32_t item = blockIdx.x / (uint32_t)a.c.heads;
    m.head = (int32_t)(blockIdx.x % (uint32_t)a.c.heads);
    m.tile0 = (int32_t)(item % (uint32_t)a.tiles) * tile_rows;
    t.b = (int32_t)(item / (uint32_t)a.tiles);
    m.c.w = request<kOwn>(a, t.b);
    m.rows = m.c.w.qn * a.group;
    m.s0 = 0;
    m.s1 = m.all = 1;
    m.cut = false;
    return m.tile0 < m.rows;
}

// kFront: workgroup 0 notes the members; the others' parts, in order: group,
// row tile, head, place along the keys.  All items are cut into parts of up to
// T steps, T the least with which the parts are no more than the workgroups:
// equal parts, one a workgroup, so that none starts and ends two items.  Against
// parts of an even line, when this was taken, whole calls: 64 requests behind
// 16384 tokens 72.4 -> 69.8 us, 32 behind 65536 138.2 -> 135.6, 4 behind 1024
// 22.6 -> 21.4, but 16 of 8 drafts behind 5024 68.9 -> 72.0 and three groups of
// 15 83.4 -> 86.3.  More than 64 groups are not searched for T: it is their
// mean.  False: no such part.
struct FrontLds {
    int64_t scan[kWaves];
    int64_t before, steps;  // (not in scan, which slower waves may still read)
    int32_t b, found;
};

template <int STEP>
__device__ __forceinline__ bool front_item(const AttnArgs &a, FrontLds &s, Line &t, Item &m)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t me = (int64_t)blockIdx.x - 1, most = a.workers - 1;
    // items and steps of group b
    auto size = [&](int b, int64_t &items, int64_t &steps) {
        const Request w = request<kFront>(a, b);
        items = (int64_t)((w.qn * a.group + a.f_tile - 1) / a.f_tile) * a.c.heads;
        steps = (w.len + STEP - 1) / STEP;
    };
    auto wave_total = [&](int64_t v) {  // a sum over lanes, by moves within rows and between them
        auto add = [](int64_t x, auto move) {
            return x + (int64_t)((uint64_t)move((uint32_t)(x >> 32)) << 32 | move((uint32_t)x));
        };
        v = add(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xb1, 0xf, 0xf, false); });
        v = add(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4e, 0xf, 0xf, false); });
        v = add(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, false); });
        v = add(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xf, 0xf, false); });
        int64_t total = 0;
#pragma unroll
        for (int row = 0; row < 64; row += 16)
            total += (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), row) << 32 |
                               (uint32_t)__builtin_amdgcn_readlane((int)v, row));
        return total;
    };
    int64_t items = 0, steps = 0, T, before = 0;
    if (a.groups == 1) {
        size(0, items, steps);
        if (items == 0) return false;
        const int64_t parts = items < most ? quotient(most, items) : 1;
        T = quotient(steps + parts - 1, parts);
        if (T < a.least) T = a.least;
        if (me < 0 || me >= items * quotient(steps + T - 1, T)) return false;
        t.b = 0;
    } else if (a.groups <= 64) {  // every wave for itself
        if (lane < a.groups) size(lane, items, steps);
        // the mean, and what leaves each item room for one part more
        const int64_t work = wave_total(items * steps), all = wave_total(items);
        T = quotient(work + most - 1, most);
        int64_t high = all < most ? quotient(work, most - all) + 1 : 0;
        if (all >= most) {  // one part each
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t o = __shfl_xor(steps > high ? steps : high, d, 64);
                high = o > high ? o : high;
            }
            T = high > steps ? high : steps;
            T = uniform64(T);
            high = T;
        }
        if (T < a.least) T = a.least;
        while (T < high) {
            const int64_t mid = (T + high) >> 1;
            if (wave_total(items * quotient(steps + mid - 1, mid)) <= most) high = mid;
            else T = mid + 1;
        }
        const int64_t mine = items * quotient(steps + T - 1, T);
        int64_t sum = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = __shfl_up(sum, d, 64);
            if (lane >= d) sum += o;
        }
        const uint64_t here = __ballot(me >= sum - mine && me < sum);
        if (!here) return false;
        t.b = __builtin_ctzll(here);
        before = __shfl(sum - mine, t.b, 64);
        steps = __shfl(steps, t.b, 64);
    } else {
        const int per = (a.groups + kThreads - 1) / kThreads, first = tid * per;
        const int last = first + per < a.groups ? first + per : a.groups;
        int64_t sum = 0;
        for (int b = first; b < last; ++b) size(b, items, steps), sum += items * steps;
        sum = wave_total(sum);
        if (lane == 0) s.scan[wave] = sum;
        if (tid == 0) s.found = 0;
        __syncthreads();
        T = 0;
        for (int w = 0; w < kWaves; ++w) T += s.scan[w];
        T = quotient(T + most - 1, most);
        if (T < a.least) T = a.least;
        sum = 0;
        for (int b = first; b < last; ++b) size(b, items, steps), sum += items * quotient(steps + T - 1, T);
        int64_t upto = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = __shfl_up(upto, d, 64);
            if (lane >= d) upto += o;
        }
        __syncthreads();
        if (lane == 63) s.scan[wave] = upto;
        __syncthreads();
        for (int w = 0; w < wave; ++w) upto += s.scan[w];
        if (me >= upto - sum && me < upto) {  // one thread at most
            before = upto - sum;
            for (int b = first; b < last; ++b) {
                size(b, items, steps);
                const int64_t n = items * quotient(steps + T - 1, T);
                if (me < before + n) {
                    s.before = before;
                    s.steps = steps;
                    s.b = b;
                    s.found = 1;
                    break;
                }
                before += n;
            }
        }
        __syncthreads();
        if (!s.found) return false;
        t.b = s.b;
        before = s.before;
        steps = s.steps;
    }
    t.b = uniform(t.b);
    const int parts = uniform((int)quotient(steps + T - 1, T)), at = uniform((int)(me - before));
    const int item = at / parts, part = at - item * parts;
    m.head = item % a.c.heads;
    const int tile = item / a.c.heads;
    m.c.w = request<kFront>(a, t.b);
    const int tile_rows = front_rows(a, m.c.w), end = (tile + 1) * tile_rows;
    m.tile0 = tile * tile_rows;
    m.rows = m.c.w.qn * a.group < end ? m.c.w.qn * a.group : end;  // up to the tile's end
    m.all = uniform((int)steps);
    m.s0 = uniform((int)(part * T));
    m.s1 = uniform((int)((part + 1) * T < steps ? (part + 1) * T : steps));
    m.cut = true;
    if (part == 0 && tid == 0)
        a.items[(int64_t)(front_tile(a, m.c.w.q0, t.b) + tile) * a.c.heads + m.head] = make_int2((int)me, parts);
    return true;
}

// ---------------------------------------------------------------------------
// A wave's ring of staged steps.
// ---------------------------------------------------------------------------
template <int D> struct Ring {
    using L = Kv4Layout<D>;
    static constexpr int R = L::R;
    static constexpr int kTile = 16 * L::kRow;         // codes of 16 tokens
    static constexpr int kV = 2 * kTile;               // K of both tiles, then V, then the scales
    static constexpr int kScales = 4 * kTile;          // of a tile: K's, V's (32 R bytes each), 256 bytes kept
    static constexpr int kStage = kScales + 512;
    static constexpr int kWide = D == 64 ? 4 : 16;     // bytes of a lane's DMA
    static constexpr int kEach = kTile / (64 * kWide); // DMA instructions of a tile's codes

    // 16-byte piece u (of a key row's D / 32) of row r
    __device__ static constexpr int piece(int r, int u)
    {
        return D == 128 ? 4 * r + (u ^ (r >> 2)) : 8 * r + (u ^ (r >> 1 & 7));
    }
};

// A lane's offsets within a head's part of a page (k[1] less the 1024 that
// its instruction adds).
template <int D> struct Offsets {
    int k[D == 256 ? 2 : 1], v, s;
    __device__ __forceinline__ void set(int lane, int P)
    {
        using G = Ring<D>;
        using L = Kv4Layout<D>;
#pragma unroll
        for (int j = 0; j < (D == 256 ? 2 : 1); ++j) {
            const int x = 64 * j + lane;
            if (D == 64) k[j] = 4 * x;
            else if (D == 128) k[j] = 64 * (x >> 2) + 16 * ((x & 3) ^ (x >> 4));
            else k[j] = 128 * (x >> 3) + 16 * ((x & 7) ^ (x >> 4 & 7)) - 1024 * j;
        }
        v = L::v_codes(P) + G::kWide * lane;
        s = lane < 8 * G::R ? L::k_scales(P) + 4 * lane
            : lane < 16 * G::R ? L::v_scales(P) + 4 * (lane - 8 * G::R) : kNothing;
    }
};

// The pages of a step's two 16-token tiles (-1: not of the cache).  Scalar
// loads: a vector load here would be the youngest behind the ring's, and
// waiting for it would wait for all of those.
#define PN_CONST __attribute__((address_space(4)))
struct Pages {
    int32_t p[2];
};

__device__ __forceinline__ Pages pages_of(const AttnArgs &a, const int32_t *row, int32_t max_pages, int step, bool there)
{
    Pages t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // (no branch around a load: all of a call's are on their way at once)
        const int at = (step * kStep + 16 * i) >> a.c.shift;
        const bool in = there && at < max_pages;
        const int32_t p = ((const PN_CONST int32_t *)row)[uniform(in ? at : 0)];
        t.p[i] = in ? p : -1;
    }
    return t;
}

__device__ __forceinline__ int32_t valid(const AttnArgs &a, int32_t p)
{
    return uniform((uint32_t)p < (uint32_t)a.c.num_pages ? p : -1);
}

// One tile's loads into LDS: K codes to m on; V codes to m on and the scales
// to m_s, from page offsets o, o_s and the lane's own.  The compiler does not
// see these loads, so that it does not wait for all of them before any LDS
// read (it cannot tell the stages of a ring apart); they have no register
// results, and wait_loads counts them.  An offset in the instruction moves
// both addresses.  s_nop 4: a scalar register that a vector instruction wrote
// must not be read by a load for five states; s_nop 0: nor M0 for one.  (M0 is
// the compiler's to use, but nothing else here uses it.)
template <int D>
__device__ __forceinline__ void load_k(u32x4_t rs, const Offsets<D> &off, uint32_t m, int o)
{
    if constexpr (D == 64)
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\t"
                     "buffer_load_dword %0, %1, %3 offen lds\n\t"
                     "buffer_load_dword %0, %1, %3 offen offset:256 lds"
                     :: "v"(off.k[0]), "s"(rs), "s"(m), "s"(o) : "memory");
    else if constexpr (D == 128)
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %0, %1, %3 offen lds"
                     :: "v"(off.k[0]), "s"(rs), "s"(m), "s"(o) : "memory");
    else
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %0, %2, %4 offen lds\n\t"
                     "buffer_load_dwordx4 %1, %2, %4 offen offset:1024 lds"
                     :: "v"(off.k[0]), "v"(off.k[1]), "s"(rs), "s"(m), "s"(o) : "memory");
}

template <int D>
__device__ __forceinline__ void load_v(u32x4_t rs, const Offsets<D> &off, uint32_t m, int o, uint32_t m_s, int o_s)
{
    if constexpr (D == 64)
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
                     "buffer_load_dword %0, %2, %4 offen lds\n\t"
                     "buffer_load_dword %0, %2, %4 offen offset:256 lds\n\t"
                     "s_mov_b32 m0, %5\n\ts_nop 0\n\t"
                     "buffer_load_dword %1, %2, %6 offen lds"
                     :: "v"(off.v), "v"(off.s), "s"(rs), "s"(m), "s"(o), "s"(m_s), "s"(o_s) : "memory");
    else if constexpr (D == 128)
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %0, %2, %4 offen lds\n\t"
                     "s_mov_b32 m0, %5\n\ts_nop 0\n\t"
                     "buffer_load_dword %1, %2, %6 offen lds"
                     :: "v"(off.v), "v"(off.s), "s"(rs), "s"(m), "s"(o), "s"(m_s), "s"(o_s) : "memory");
    else
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
                     "buffer_load_dwordx4 %0, %2, %4 offen lds\n\t"
                     "buffer_load_dwordx4 %0, %2, %4 offen offset:1024 lds\n\t"
                     "s_mov_b32 m0, %5\n\ts_nop 0\n\t"
                     "buffer_load_dword %1, %2, %6 offen lds"
                     :: "v"(off.v), "v"(off.s), "s"(rs), "s"(m), "s"(o), "s"(m_s), "s"(o_s) : "memory");
}

// Start the loads of a step (pages of -1 load nothing; the count stays the
// same).  head_base: the head's part of page 0.  RG = 1: a wave loads its
// step whole; RG = 4: row group rg loads K or V of one of the tiles.
template <int D, int RG>
__device__ __forceinline__ void stage(const AttnArgs &a, uint8_t *to, const Offsets<D> &off, const Pages &t, int step,
                                      uint64_t head_base, int32_t page_bytes, int rg)
{
    using G = Ring<D>;
    using L = Kv4Layout<D>;
    const uint32_t m = uniform((int)(uint32_t)(size_t)(lds_void *)to);
#pragma unroll
    for (int i0 = 0; i0 < (RG == 1 ? 2 : 1); ++i0) {
        const int i = RG == 1 ? i0 : rg >> 1;
        const int32_t page = valid(a, i ? t.p[1] : t.p[0]);
        const int o = (step * kStep + 16 * i) & ((1 << a.c.shift) - 1);
        const uint64_t base = head_base + (uint64_t)(uint32_t)(page < 0 ? 0 : page) * (uint32_t)page_bytes;
        // raw buffer: 48-bit base, no stride, the head's part of the page (or nothing) in range
        const u32x4_t rs = {(uint32_t)uniform((int)base), (uint32_t)uniform((int)(base >> 32) & 0xffff),
                            page < 0 ? 0u : (uint32_t)a.c.chunk, 0x00020000u};
        if (RG == 1 || !(rg & 1)) load_k<D>(rs, off, m + i * G::kTile, o * L::kRow);
        if (RG == 1 || (rg & 1))
            load_v<D>(rs, off, m + G::kV + i * G::kTile, o * L::kRow, m + G::kScales + 256 * i, o * 2 * G::R);
    }
}

template <int N> __device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4) << 14);  // vmcnt(N)
    asm volatile("" ::: "memory");
}

// The compiler schedules nothing across this: left alone it unpacks a whole
// step ahead of its products and runs out of registers.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// The power of two on the value scales for a largest scale of the bits `big`,
// and the largest scale (fp16 bits) that it leaves below 2^11.  The scales are
// below 2^(e - 14); e from 6 on keeps the factor, 2^15 at most, inside fp16.
__device__ __forceinline__ void fit_scales(uint32_t big, float &up, uint32_t &cap)
{
    int e = (int)(big >> 10);
    e = e < 6 ? 6 : e < 30 ? e : 30;
    up = __builtin_ldexpf(1.0f, 21 - e);
    cap = e + 5 > 30 ? 0xffffu : (uint32_t)((e + 5) << 10) - 1;
}

__device__ __forceinline__ half8_t codes8(uint32_t word)
{
    half2_t t[4];
    Unpack<1>::run(word, t);
    half8_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[2 * i] = t[i][0], r[2 * i + 1] = t[i][1];
    return r;
}

// A barrier for what is in LDS: loads in flight stay so.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// N dwords from LDS, 8 or 16 bytes at a time.
template <int N> __device__ __forceinline__ void read_words(uint32_t (&w)[N], const uint8_t *from)
{
    if constexpr (N == 2) {
        const uint2 x = *(const uint2 *)from;
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int j = 0; j < N / 4; ++j) {
            const uint4 x = *(const uint4 *)(from + 16 * j);
            w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
        }
    }
}

// Half h of packed fp16 values, as fp32 (folded into v_fma_mix).
template <int N> __device__ __forceinline__ float half_at(const uint32_t (&w)[N], int h)
{
    return (float)as_half2(w[h >> 1])[h & 1];
}

// The larger of two, of three.  (fmaxf first quiets NaNs, one instruction an
// operand; there are none here, and one would come through.)
__device__ __forceinline__ float max2(float a, float b)
{
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// Largest over, or sum of, the four 16-lane groups, in all of them.
__device__ __forceinline__ float group_max(float v)
{
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = max2(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return max2(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_sum(float v)
{
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A wave's running state for 16 NT rows; lane (r, g): row r of each 16, and
// of O^T the elements of rows 4 g .. 4 g + 3 of A.
template <int D, int NT> struct State {
    static constexpr int R = D / 64;
    float4_t o[NT][R][4];
    float m[NT];   // the score (before c2) that weights are relative to, kLowest if none
    float l[NT];   // this lane's share of the sum of the weights exp2(c2 (s - m) + kBias)
    float up;      // 2^u, the power of two on the value scales
    uint32_t cap;  // largest scale (fp16 bits) that 2^u leaves below 2^11
};

// What a step that is not visible as a whole needs to know.
struct Mask {
    bool some;         // anything masked
    bool page[2];      // the tiles' pages are of the cache
    int32_t token0;    // of the step
    int32_t end;       // keys of the request
    int32_t low, high; // positions of the wave's first and last query
    int32_t row0, rows, first;  // the wave's first row, the request's rows, the position of query 0
};

template <int D, int NT>
__device__ __forceinline__ void advance(State<D, NT> &st, const uint8_t *from, const half8_t *q, const AttnArgs &a,
                                        const Mask &mask, int lane)
{
    using G = Ring<D>;
    constexpr int R = G::R;
    const int r = lane & 15, g = lane >> 4;

    // scores
    float4_t sc[NT][2];
    uint32_t ks[2][2 * R];
#pragma unroll
    for (int i = 0; i < 2; ++i) read_words(ks[i], from + G::kScales + 256 * i + 8 * R * g);
#pragma unroll
    for (int b = 0; b < R; ++b) {
        half8_t k[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t *row = from + i * G::kTile;
            // words (b, 0) and (b, 1) of the lane's share of its token's row
            const uint2 x = *(const uint2 *)(R == 1 ? row + 32 * r + 8 * g
                                                    : row + 16 * G::piece(r, (R / 2) * g + b / 2) + 8 * (b & 1));
            k[i][0] = codes8(x.x);
            k[i][1] = codes8(x.y);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const half8_t q0 = q[(n * 2 * R + 2 * b) * 64 + lane], q1 = q[(n * 2 * R + 2 * b + 1) * 64 + lane];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float4_t c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[i][0], q0, (float4_t){0, 0, 0, 0}, 0, 0, 0);
                c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[i][1], q1, c, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sc[n][i][j] = __builtin_fmaf(c[j], half_at(ks[i], R * j + b), b == 0 ? 0.0f : sc[n][i][j]);
            }
        }
        keep_order();
    }

    // Value scales of the lane's tokens.  One that no row sees may be
    // anything, infinite or NaN: it becomes 0.
    uint32_t d[2][2 * R];
#pragma unroll
    for (int i = 0; i < 2; ++i) read_words(d[i], from + G::kScales + 256 * i + 32 * R + 8 * R * g);
    if (mask.some) {
        const int32_t under = before_window(a, mask.low);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int key = mask.token0 + 16 * (j >> 2) + 4 * g + (j & 3);
            const bool ok = mask.page[j >> 2] && key < mask.end && key <= mask.high && (key > under || key < a.sinks);
#pragma unroll
            for (int b = 0; b < R; ++b) {
                const int h = R * (j & 3) + b;
                if (!ok) d[j >> 2][h >> 1] &= h & 1 ? 0x0000ffffu : 0xffff0000u;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int at = mask.row0 + 16 * n + r;
            const int32_t pos = at < mask.rows ? mask.first + at / a.group : -1;
            const int32_t below = before_window(a, pos);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = mask.token0 + 16 * (j >> 2) + 4 * g + (j & 3);
                const bool ok = mask.page[j >> 2] && key < mask.end && key <= pos && (key > below || key < a.sinks);
                sc[n][j >> 2][j & 3] = ok ? sc[n][j >> 2][j & 3] : -__builtin_inff();
            }
        }
    }

#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2 * R; ++j) asm("" : "+v"(d[i][j]));  // words, not halves

    // The scales against the cap: lane r looks at one word of its group's 4 R.
    uint32_t big;
    {
        const int x = r & (4 * R - 1), i = x / (2 * R), h = x % (2 * R);
        uint32_t w = *(const uint32_t *)(from + G::kScales + 256 * i + 32 * R + 8 * R * g + 4 * h) & 0x7fff7fffu;
        if (mask.some) {  // as above
            const int32_t under = before_window(a, mask.low);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int key = mask.token0 + 16 * i + 4 * g + (2 * h + y) / R;
                const bool ok = (i ? mask.page[1] : mask.page[0]) && key < mask.end && key <= mask.high &&
                                (key > under || key < a.sinks);
                if (!ok) w &= y ? 0x0000ffffu : 0xffff0000u;
            }
        }
        big = (w >> 16) > (w & 0xffffu) ? w >> 16 : w & 0xffffu;
    }
    if (__ballot(big > st.cap)) {
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) {
            const uint32_t y = __shfl_xor(big, x, 64);
            big = y > big ? y : big;
        }
        float up;
        fit_scales(big, up, st.cap);
        const float f = up / st.up;  // the first time O is 0
        st.up = up;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < R; ++b)
#pragma unroll
                for (int i2 = 0; i2 < 4; ++i2) st.o[n][b][i2] *= f;
    }

    keep_order();
    // weights
    half8_t p[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float mx = max3(sc[n][0][0], sc[n][0][1], sc[n][0][2]);
        mx = max3(mx, sc[n][0][3], sc[n][1][0]);
        mx = max3(mx, sc[n][1][1], sc[n][1][2]);
        mx = group_max(max2(mx, sc[n][1][3]));
        if (__ballot(mx > st.m[n] + a.slack)) {
            const float f = mx > st.m[n] ? __builtin_amdgcn_exp2f((st.m[n] - mx) * a.c2) : 1.0f;
            st.m[n] = max2(st.m[n], mx);
            st.l[n] *= f;
#pragma unroll
            for (int b = 0; b < R; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) st.o[n][b][i] *= f;
        }
        const float mm = kBias - st.m[n] * a.c2;
        float w[8], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][j >> 2][j & 3], a.c2, mm));
            sum += w[j];
            p[n][j] = (_Float16)w[j];
        }
        st.l[n] += sum;
    }

    keep_order();
    // values
    const uint32_t sel = r < 8 ? 0x05040100u : 0x07060302u;  // even (low) or odd (high) elements of a token pair
    const half2_t up2 = {(_Float16)st.up, (_Float16)st.up};
#pragma unroll
    for (int b = 0; b < R; ++b) {
        uint32_t v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            read_words(v[i], from + G::kV + i * G::kTile + 16 * (g * (D / 8) + 8 * b + (r & 7)));
        half8_t va[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // the scales of the token pair for this block
            const int i2 = u >> 1, t = 2 * (u & 1), word = R * t / 2 + b / 2, next = R / 2;
            const half2_t sc2 = up2 * as_half2(R == 1 ? d[i2][u & 1]
                                                      : __builtin_amdgcn_perm(d[i2][word + next], d[i2][word],
                                                                              b & 1 ? 0x07060302u : 0x05040100u));
            half2_t e[4];
            Unpack<1>::run(__builtin_amdgcn_perm(v[i2][t + 1], v[i2][t], sel), e);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[i] *= sc2;
                va[i][2 * u] = e[i][0], va[i][2 * u + 1] = e[i][1];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                st.o[n][b][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(va[i], p[n], st.o[n][b][i], 0, 0, 0);
        keep_order();
    }
}

// The same for rows that see every key that is there (kFront).  seen: tokens of
// each tile that are; `some` are not.  Fewer instructions where the arithmetic
// is what counts: maxima are looked at lane by lane and joined across lanes only
// when one passes the running maximum by the slack, and the weights' sums are a
// product with ones (of the rounded weights, and over all lanes: l is the row's).
struct Seen {
    bool some;
    int32_t n[2];
};

template <int D, int NT>
__device__ __forceinline__ void advance_front(State<D, NT> &st, const uint8_t *from, const half8_t *q, const AttnArgs &a,
                                              const Seen &seen, int lane)
{
    using G = Ring<D>;
    constexpr int R = G::R;
    const int r = lane & 15, g = lane >> 4;

    // scores
    float4_t sc[NT][2];
    uint32_t ks[2][2 * R];
#pragma unroll
    for (int i = 0; i < 2; ++i) read_words(ks[i], from + G::kScales + 256 * i + 8 * R * g);
#pragma unroll
    for (int b = 0; b < R; ++b) {
        half8_t k[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t *row = from + i * G::kTile;
            const uint2 x = *(const uint2 *)(R == 1 ? row + 32 * r + 8 * g
                                                    : row + 16 * G::piece(r, (R / 2) * g + b / 2) + 8 * (b & 1));
            k[i][0] = codes8(x.x);
            k[i][1] = codes8(x.y);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const half8_t q0 = q[(n * 2 * R + 2 * b) * 64 + lane], q1 = q[(n * 2 * R + 2 * b + 1) * 64 + lane];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float4_t c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[i][0], q0, (float4_t){0, 0, 0, 0}, 0, 0, 0);
                c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[i][1], q1, c, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sc[n][i][j] = __builtin_fmaf(c[j], half_at(ks[i], R * j + b), b == 0 ? 0.0f : sc[n][i][j]);
            }
        }
        keep_order();
    }

    // Value scales of the lane's tokens; 0 for those that are not there.
    uint32_t d[2][2 * R];
#pragma unroll
    for (int i = 0; i < 2; ++i) read_words(d[i], from + G::kScales + 256 * i + 32 * R + 8 * R * g);
    // The scales against the cap: lane r looks at one word of its group's 4 R.
    const int x = r & (4 * R - 1), xi = x / (2 * R), xh = x % (2 * R);
    uint32_t word = *(const uint32_t *)(from + G::kScales + 256 * xi + 32 * R + 8 * R * g + 4 * xh) & 0x7fff7fffu;
    if (seen.some) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool ok = 4 * g + (j & 3) < seen.n[j >> 2];
#pragma unroll
            for (int b = 0; b < R; ++b) {
                const int h = R * (j & 3) + b;
                if (!ok) d[j >> 2][h >> 1] &= h & 1 ? 0x0000ffffu : 0xffff0000u;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[n][j >> 2][j & 3] = ok ? sc[n][j >> 2][j & 3] : -__builtin_inff();
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
            if (4 * g + (2 * xh + y) / R >= (xi ? seen.n[1] : seen.n[0])) word &= y ? 0x0000ffffu : 0xffff0000u;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2 * R; ++j) asm("" : "+v"(d[i][j]));  // words, not halves
    uint32_t big = (word >> 16) > (word & 0xffffu) ? word >> 16 : word & 0xffffu;
    if (__ballot(big > st.cap)) {
#pragma unroll
        for (int x2 = 1; x2 < 64; x2 <<= 1) {
            const uint32_t y = __shfl_xor(big, x2, 64);
            big = y > big ? y : big;
        }
        float up;
        fit_scales(big, up, st.cap);
        const float f = up / st.up;  // the first time O is 0
        st.up = up;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < R; ++b)
#pragma unroll
                for (int i2 = 0; i2 < 4; ++i2) st.o[n][b][i2] *= f;
    }

    keep_order();
    // weights
    float mx[NT], more = kLowest;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        mx[n] = max3(sc[n][0][0], sc[n][0][1], sc[n][0][2]);
        mx[n] = max3(mx[n], sc[n][0][3], sc[n][1][0]);
        mx[n] = max3(mx[n], sc[n][1][1], sc[n][1][2]);
        mx[n] = max2(mx[n], sc[n][1][3]);
        more = max2(more, mx[n] - st.m[n]);
    }
    if (__ballot(more > a.slack)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float top = group_max(mx[n]);
            const float f = top > st.m[n] ? __builtin_amdgcn_exp2f((st.m[n] - top) * a.c2) : 1.0f;
            st.m[n] = max2(st.m[n], top);
            st.l[n] *= f;
#pragma unroll
            for (int b = 0; b < R; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) st.o[n][b][i] *= f;
        }
    }
    half8_t p[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float mm = kBias - st.m[n] * a.c2;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2_t w = {__builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][j >> 2][j & 3], a.c2, mm)),
                                __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][j >> 2][(j & 3) + 1], a.c2, mm))};
            const half2_t w2 = __builtin_convertvector(w, half2_t);
            p[n][j] = w2[0], p[n][j + 1] = w2[1];
        }
    }

    // values
    const half8_t ones = {1, 1, 1, 1, 1, 1, 1, 1};
    const uint32_t sel = r < 8 ? 0x05040100u : 0x07060302u;  // even (low) or odd (high) elements of a token pair
    const half2_t up2 = {(_Float16)st.up, (_Float16)st.up};
    float4_t sum[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p[n], (float4_t){0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
    for (int b = 0; b < R; ++b) {
        uint32_t v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            read_words(v[i], from + G::kV + i * G::kTile + 16 * (g * (D / 8) + 8 * b + (r & 7)));
        half8_t va[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // the scales of the token pair for this block
            const int i2 = u >> 1, t = 2 * (u & 1), word2 = R * t / 2 + b / 2, next = R / 2;
            const half2_t sc2 = up2 * as_half2(R == 1 ? d[i2][u & 1]
                                                      : __builtin_amdgcn_perm(d[i2][word2 + next], d[i2][word2],
                                                                              b & 1 ? 0x07060302u : 0x05040100u));
            half2_t e[4];
            Unpack<1>::run(__builtin_amdgcn_perm(v[i2][t + 1], v[i2][t], sel), e);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[i] *= sc2;
                va[i][2 * u] = e[i][0], va[i][2 * u + 1] = e[i][1];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                st.o[n][b][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(va[i], p[n], st.o[n][b][i], 0, 0, 0);
        if (b == 0) {
            // The other three results stay in use until the product has ended: left to themselves their
            // registers would be free at once, for inline assembly that no one keeps apart from the product.
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                st.l[n] += sum[n][0];
                asm volatile("" : "+v"(st.l[n]) : "v"(sum[n]));
            }
        }
        keep_order();
    }
}

// Lane (r, g) holds x[j] = element 64 b + 8 (4 (g & 1) + j) + 2 i + (g >> 1)
// of row r.  As fp16 pairs: elements 2 i and 2 i + 1 of word 4 (g & 1) + j +
// (g & 2) of the block, j < 2 (lanes below 32 take x[j], those above x[j + 2]).
__device__ __forceinline__ uint32_t row_pair(const float4_t &x, int j)
{
    auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[j]), __float_as_uint(x[j + 2]), false, false);
    const uint32_t lo = __builtin_bit_cast(uint16_t, (_Float16)__uint_as_float(s[0]));
    const uint32_t hi = __builtin_bit_cast(uint16_t, (_Float16)__uint_as_float(s[1]));
    return lo | hi << 16;
}
__device__ __forceinline__ void store_row(uint16_t *out, const float4_t &x, int b, int i, int g)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t pair = row_pair(x, j);
        if (out) *(uint32_t *)(out + 64 * b + 8 * (4 * (g & 1) + j + (g & 2)) + 2 * i) = pair;
    }
}

// How a workgroup's waves are used.
template <int D, int NT, int RG> struct Shape {
    using G = Ring<D>;
    static constexpr int KW = kWaves / RG;             // waves along the keys
    static constexpr int kRows = 16 * NT * RG;         // of a workgroup
    static constexpr int kStages = RG > 1 ? 3 : D == 64 ? 3 : 2;
    static constexpr int kRing = (RG == 1 ? kWaves : KW) * kStages * G::kStage;
    static constexpr int kLds = kRing + RG * NT * 2 * G::R * 1024;  // and the queries
    // Steps staged ahead of the one at work.  A wave with a ring of its own
    // refills a stage when it has read it; a shared stage is refilled one
    // step later, when a barrier has shown that all have.
    static constexpr int kAhead = RG == 1 ? kStages : kStages - 1;
    // Fragments of the join: RG = 1: all waves'; else those of all but the first along the keys.
    static_assert((RG == 1 ? kWaves : RG * (KW - 1)) * 4 * G::R * 1024 <= kLds, "room for the join");
    // Floats of a part, [row group][n][4 b + i][lane][4]; (m, l) of its rows
    // are apart, [part][row][2], so that the join reads them together.
    static constexpr int kPart = RG * NT * 4 * G::R * 256;
};

// Two workgroups share a compute unit where registers and LDS allow it (64
// requests of up to 16384 tokens, 64 wide: 54 us, one a unit 61 us; 128 wide
// 73 and 80 us).
template <int D, int NT, int RG> constexpr int waves_per_simd() { return D < 256 && NT == 1 && RG == 1 ? 4 : 2; }

// Where the parts of the shared keys' sums for a row are.
struct FrontPlace {
    int32_t first, parts;  // in f_part; parts 0: none
    int32_t local;         // the row in its tile
};
// Without a row (not live) nothing is read.
__device__ __forceinline__ FrontPlace front_place(const AttnArgs &a, const Member &in, int64_t query, int q_head, bool live)
{
    FrontPlace p = {0, 0, 0};
    if (live) {
        const int head = q_head / a.group, row = (int32_t)(query - in.q0) * a.group + q_head - head * a.group;
        const int tile = row / in.rows;
        const int2 item = a.items[(int64_t)(in.tile + tile) * a.c.heads + head];
        p.first = item.x;
        p.parts = item.y;
        p.local = row - tile * in.rows;
    }
    return p;
}

// As lane (r, g) sees them.
struct FrontRow {
    const float4_t *at;   // of the first part
    const float2 *ml;
    int64_t step;         // from one part to the next; f_tile in ml
    int32_t parts;
    float top;            // their largest maximum
    float own, front;     // factors of the row's own sum and of the parts relative to top
};
template <int D> __device__ __forceinline__ void front_at(const AttnArgs &a, const FrontPlace &p, int g, FrontRow &f)
{
    // (groups that overlap may leave an entry unwritten)
    const bool ok = p.first >= 0 && p.parts > 0 && p.parts < a.grid - p.first;
    const int64_t first = ok ? p.first : 0;
    f.parts = ok ? p.parts : 0;
    f.step = (int64_t)a.f_tile * (D / 4);
    f.at = (const float4_t *)a.f_part + first * f.step + (p.local >> 4) * (D * 4) + (p.local & 15) + 16 * g;
    f.ml = a.f_part_ml + first * a.f_tile + p.local;
}
// The factors for a row's own (m, l) and parts of `sum` relative to f.top.  All are 0 where nothing is visible.
__device__ __forceinline__ void front_factors(const AttnArgs &a, float m, float l, float sum, FrontRow &f)
{
    const float all = max2(m, f.top);
    const float f0 = __builtin_amdgcn_exp2f((m - all) * a.c2), f1 = __builtin_amdgcn_exp2f((f.top - all) * a.c2);
    const float total = l * f0 + sum * f1, by = total > 0.0f ? 1.0f / total : 0.0f;
    f.own = f0 * by;
    f.front = f1 * by;
}

// Joined with the row's own (m, l), for all lanes of a wave together.
template <int D>
__device__ __forceinline__ FrontRow front_row(const AttnArgs &a, const FrontPlace &p, float m, float l, int g)
{
    FrontRow f;
    front_at<D>(a, p, g, f);
    float top = kLowest, sum = 0.0f;
    for (int j = g; j < f.parts; j += 4) top = max2(top, f.ml[(int64_t)j * a.f_tile].x);
    f.top = top = group_max(top);
    for (int j = g; j < f.parts; j += 4) {
        const float2 x = f.ml[(int64_t)j * a.f_tile];
        sum += x.y * __builtin_amdgcn_exp2f((x.x - top) * a.c2);
    }
    front_factors(a, m, l, group_sum(sum), f);
    return f;
}

// Product y's share of the output from the shared keys.
__device__ __forceinline__ float4_t front_sum(const AttnArgs &a, const FrontRow &f, int y)
{
    constexpr int kDeep = 8;  // parts on their way at a time
    float4_t v = {0, 0, 0, 0};
    for (int j0 = 0; j0 < f.parts; j0 += kDeep) {
        float4_t x[kDeep];
        float w[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int64_t at = j0 + j < f.parts ? j0 + j : 0;
            x[j] = f.at[at * f.step + 64 * y];
            w[j] = f.ml[at * a.f_tile].x;
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
            if (j0 + j < f.parts) v += x[j] * __builtin_amdgcn_exp2f((w[j] - f.top) * a.c2);
    }
    return v * f.front;
}

// Product y of a row, v relative to its own (m, l), joined with its parts: of
// few of them all that is needed is on its way at once.
template <int D>
__device__ __forceinline__ float4_t front_join(const AttnArgs &a, const FrontPlace &p, float m, float l, float4_t v, int y, int g)
{
    constexpr int kFew = 8;
    FrontRow f;
    front_at<D>(a, p, g, f);
    float4_t x[kFew];
    float2 ml[kFew];
    const int few = f.parts < kFew ? f.parts : kFew;
    if (few > 0) {  // (not a place of the row's)
#pragma unroll
        for (int j = 0; j < kFew; ++j) {
            const int64_t at = j < few ? j : 0;
            x[j] = f.at[at * f.step + 64 * y];
            ml[j] = f.ml[at * a.f_tile];
        }
    }
    f.top = kLowest;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kFew; ++j)
        if (j < few) f.top = max2(f.top, ml[j].x);
    for (int j = kFew; j < f.parts; ++j) f.top = max2(f.top, f.ml[(int64_t)j * a.f_tile].x);
    float4_t all = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kFew; ++j)
        if (j < few) {
            const float w = __builtin_amdgcn_exp2f((ml[j].x - f.top) * a.c2);
            sum += ml[j].y * w;
            all += x[j] * w;
        }
    for (int j = kFew; j < f.parts; ++j) {
        const float2 z = f.ml[(int64_t)j * a.f_tile];
        const float w = __builtin_amdgcn_exp2f((z.x - f.top) * a.c2);
        sum += z.y * w;
        all += f.at[j * f.step + 64 * y] * w;
    }
    front_factors(a, m, l, sum, f);
    return v * f.own + all * f.front;
}

// One item (or part of one) of request b, by the whole workgroup.  ml: a wave's
// rows' maxima and sums.
template <int D, int NT, int RG, int PASS>
__device__ __forceinline__ void attend(const AttnArgs &a, const Item &item, int b, const Offsets<D> &off, uint8_t *lds, float *ml)
{
    using G = Ring<D>;
    using S = Shape<D, NT, RG>;
    constexpr int R = G::R, kRows = S::kRows, KW = S::KW;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int rg = wave / KW, kg = wave % KW;
    uint8_t *ring = lds + (RG == 1 ? wave : kg) * (S::kStages * G::kStage);
    // operands as the products take them: [16-row group][32 elements][lane]
    half8_t *queries = (half8_t *)(lds + S::kRing), *q = queries + rg * NT * 2 * R * 64;
    auto ml_at = [&](int w, int row) { return ml + 2 * (w * 16 * NT + row); };

    const int s0 = item.s0, head = item.head, tile0 = item.tile0, rows = item.rows;
    const bool cut = item.cut;

    Work w{item.c.w};
    span<kStep>(a, w, tile0 / a.group, ((tile0 + kRows < rows ? tile0 + kRows : rows) - 1) / a.group);
    // the wave's own rows (none: nothing is visible)
    const int row0 = tile0 + rg * 16 * NT;
    const int last = (row0 + 16 * NT < rows ? row0 + 16 * NT : rows) - 1;
    const int32_t p0 = row0 < rows ? w.first + row0 / a.group : -1, p1 = row0 < rows ? w.first + last / a.group : -1;

    // The same part of the steps that this tile has.
    auto place = [&](int e) { return e < w.sink_steps ? e : e - w.sink_steps + w.lo; };
    const int e1 = PASS == kFront ? item.s1 : share_of(item.s1, item.all, w.steps);
    int e = PASS == kFront ? s0 : share_of(s0, item.all, w.steps);
    const int turns = (e1 - e + KW - 1) / KW;  // the same for all waves
    e += kg;
    const int32_t max_pages = a.max_pages - w.skip;  // 0: no keys of its own, and no entry behind the row's end is read
    const int32_t *row = uniform_ptr(a.table + (int64_t)b * a.ld_table + (max_pages > 0 ? w.skip : 0));
    const uint64_t head_base = (uint64_t)a.c.pages + (uint64_t)head * a.c.chunk;
    const int32_t page_bytes = a.c.heads * a.c.chunk;
    // pages of the steps in the ring, and of the next to be staged
    Pages held[S::kAhead + 1];
#pragma unroll
    for (int i = 0; i <= S::kAhead; ++i) held[i] = pages_of(a, row, max_pages, place(e + KW * i), e + KW * i < e1);
    // where the shared keys' parts are, for the end
    FrontPlace fronts[joins(PASS) ? NT : 1];
    const bool joined = joins(PASS) && !cut && w.skip > 0;  // the same for the item
    if (joined) {
        const Member in = a.members[b];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int at = row0 + 16 * n + r, i = at / a.group;
            fronts[n] = front_place(a, in, w.q0 + i, head * a.group + at - i * a.group, at < rows);
        }
    }
    // the queries into LDS
    for (int y = tid; y < RG * NT * 2 * R * 64; y += kThreads) {
        const int at = tile0 + 16 * (y / (2 * R * 64)) + (y & 15), i = at / a.group;
        const int e = 32 * (y / 64 % (2 * R)) + 8 * (y >> 4 & 3);
        half8_t v = (half8_t)(_Float16)0.0f;
        if (at < rows) v = *(const half8_t *)(a.q + (w.q0 + i) * a.ldq + (head * a.group + at - i * a.group) * D + e);
        queries[y] = a.negate ? -v : v;
    }
    State<D, NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int y = 0; y < R; ++y)
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) st.o[n][y][i2] = (float4_t){0, 0, 0, 0};
        st.m[n] = kLowest;
        st.l[n] = 0.0f;
    }
    st.up = 1.0f;
    st.cap = 0;

#pragma unroll
    for (int i = 0; i < S::kAhead; ++i)
        stage<D, RG>(a, ring + i * G::kStage, off, held[i], place(e + KW * i), head_base, page_bytes, rg);
    // the queries are there; a bare barrier, so that the loads fly on
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    int at = 0;  // stage of the step at work
    for (int turn2 = 0; turn2 < turns && (RG > 1 || e < e1); ++turn2, e += KW) {
        if constexpr (RG == 1) {
            wait_loads<(S::kStages - 1) * 2 * (2 * G::kEach + 1)>();
        } else {
            // this wave's loads of the step have landed; after the
            // barrier all have, and no wave reads the stage before it
            if (rg & 1) wait_loads<(S::kStages - 2) * (G::kEach + 1)>();
            else wait_loads<(S::kStages - 2) * G::kEach>();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            const int to = at > 0 ? at - 1 : S::kStages - 1;
            stage<D, RG>(a, ring + to * G::kStage, off, held[S::kAhead], place(e + KW * S::kAhead), head_base, page_bytes,
                         rg);
        }
        const int token0 = place(e) * kStep;
        uint8_t *from = ring + at * G::kStage;
        at = at + 1 < S::kStages ? at + 1 : 0;
        Mask mask;
        mask.page[0] = valid(a, held[0].p[0]) >= 0;
        mask.page[1] = valid(a, held[0].p[1]) >= 0;
        mask.token0 = token0;
        mask.end = w.len;
        mask.low = p0;
        mask.high = p1;
        mask.row0 = row0;
        mask.rows = rows;
        mask.first = w.first;
        mask.some = !(mask.page[0] && mask.page[1] && token0 + kStep <= w.len && token0 + kStep - 1 <= p0 &&
                      (a.window <= 0 || (int64_t)token0 + a.window > p1 || token0 + kStep <= a.sinks));
        // A row group sees less than its workgroup's tile.
        const bool none = RG > 1 && (e >= e1 || token0 > p1 ||
                                     (a.window > 0 && (int64_t)token0 + kStep - 1 + a.window <= p0 && token0 >= a.sinks));
        if constexpr (PASS == kFront) {
            const int left = w.len - token0;  // 1 and up
            const Seen seen = {!(mask.page[0] && mask.page[1] && left >= kStep),
                               {mask.page[0] ? left : 0, mask.page[1] ? left - 16 : 0}};
            advance_front<D, NT>(st, from, q, a, seen, lane);
        } else {
            if (!none) advance<D, NT>(st, from, q, a, mask, lane);
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the stage has been read
        asm volatile("" ::: "memory");
        if constexpr (RG == 1)
            stage<D, RG>(a, from, off, held[S::kAhead], place(e + KW * S::kAhead), head_base, page_bytes, rg);
#pragma unroll
        for (int y = 0; y < S::kAhead; ++y) held[y] = held[y + 1];
        const int s = e + KW * (S::kAhead + 1);
        held[S::kAhead] = pages_of(a, row, max_pages, place(s), s < e1);
    }
    wait_loads<0>();  // nothing is written into the ring any more

    // Join the waves of the same rows: the rows' maxima and sums, then
    // the fragments.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float l = PASS == kFront ? st.l[n] : group_sum(st.l[n]);
        if (g == 0) ml_at(wave, 16 * n + r)[0] = st.m[n], ml_at(wave, 16 * n + r)[1] = l;
    }
    float4_t *frag = (float4_t *)lds;  // [wave][4 b + i][lane]
    const float down = 1.0f / st.up;
    // A share goes on with at most one item, its first (part 0), and
    // leaves at most one unfinished, its last (part 1).
    const int part_at = PASS == kFront ? (int)blockIdx.x - 1 : 2 * (int)blockIdx.x + (s0 == 0 ? 1 : 0);
    float4_t *part = (float4_t *)(a.part + (int64_t)part_at * (PASS == kFront ? a.f_tile * D : S::kPart));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        lds_barrier();  // (not for the last rows' stores)
        float m = kLowest, all_l = 0.0f;
        for (int y = 0; y < KW; ++y) m = max2(m, ml_at(rg * KW + y, 16 * n + r)[0]);
        for (int y = 0; y < KW; ++y)
            all_l += ml_at(rg * KW + y, 16 * n + r)[1] * __builtin_amdgcn_exp2f((ml_at(rg * KW + y, 16 * n + r)[0] - m) * a.c2);
        float f = __builtin_amdgcn_exp2f((st.m[n] - m) * a.c2) * down;
        const int row_at = row0 + 16 * n + r, i = row_at / a.group;
        const bool live = row_at < rows;
        const int q_head = head * a.group + row_at - i * a.group;
        uint16_t *out = a.out + (w.q0 + i) * a.ldo + (int64_t)q_head * D;
        if (!cut && !joined) {
            f = all_l > 0.0f ? f / all_l : 0.0f;
        }
        auto join = [&](float4_t v, int y) {  // product y of all
            if constexpr (joins(PASS)) {
                if (live) v = front_join<D>(a, fronts[n], m, all_l, v, y, g);
            }
            return v;
        };
        auto give = [&](float4_t v, int y, int i4) {  // block y, product i4
            if (cut) {
                if (live) part[((rg * NT + n) * 4 * R + 4 * y + i4) * 64 + lane] = v;
            } else {
                store_row(live ? out : nullptr, v, y, i4, g);
            }
        };
        if constexpr (RG == 1) {  // each wave adds its share of all waves' fragments
#pragma unroll
            for (int y = 0; y < 4 * R; ++y) frag[(wave * 4 * R + y) * 64 + lane] = st.o[n][y >> 2][y & 3] * f;
            lds_barrier();
#pragma unroll
            for (int y = wave >> 2; y < R; y += kWaves / 4) {
                const int f4 = 4 * y + (wave & 3);
                float4_t v = frag[f4 * 64 + lane];
#pragma unroll
                for (int z = 1; z < kWaves; ++z) v += frag[(z * 4 * R + f4) * 64 + lane];
                give(joined ? join(v, f4) : v, y, wave & 3);
            }
        } else {  // the first along the keys adds the others'
            if (kg > 0) {
#pragma unroll
                for (int y = 0; y < 4 * R; ++y)
                    frag[((rg * (KW - 1) + kg - 1) * 4 * R + y) * 64 + lane] = st.o[n][y >> 2][y & 3] * f;
            }
            lds_barrier();
            if (kg == 0) {
#pragma unroll
                for (int y = 0; y < 4 * R; ++y) {
                    float4_t v = st.o[n][y >> 2][y & 3] * f;
#pragma unroll
                    for (int z = 0; z < KW - 1; ++z) v += frag[((rg * (KW - 1) + z) * 4 * R + y) * 64 + lane];
                    if (joined) frag[(rg * (KW - 1) * 4 * R + y) * 64 + lane] = v;  // where the lane alone has read
                    else give(v, y >> 2, y & 3);
                }
                if (joined) {
#pragma unroll 1
                    for (int y = 0; y < 4 * R; ++y) give(join(frag[(rg * (KW - 1) * 4 * R + y) * 64 + lane], y), y >> 2, y & 3);
                }
            }
        }
        if (cut && kg == 0 && g == 0) a.part_ml[(int64_t)part_at * (PASS == kFront ? a.f_tile : kRows) + (rg * NT + n) * 16 + r] = make_float2(m, all_l);
    }
    lds_barrier();
}

template <int D, int NT, int RG, int PASS>
__global__ __launch_bounds__(kThreads, (waves_per_simd<D, NT, RG>())) void kv4_attn(AttnArgs a)
{
    constexpr int kRows = Shape<D, NT, RG>::kRows;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // the ring, then the queries
    __shared__ float ml[kWaves * 16 * NT * 2];
    __shared__ typename std::conditional<PASS == kFront, FrontLds, LineLds>::type line_lds;
    Line line;
    Item item;
    Offsets<D> off;
    off.set(threadIdx.x & 63, 1 << a.c.shift);
    if constexpr (PASS == kOwn) {
        if (own_item(a, line, item, kRows)) attend<D, NT, RG, PASS>(a, item, line.b, off, lds, ml);
    } else if constexpr (PASS == kFront) {
        if (blockIdx.x == 0) {
            group_members(a);
            return;
        }
        if (!front_item<kStep>(a, line_lds, line, item)) return;
        // as many 16-row groups as the tile has
        const int rows = item.rows - item.tile0;
        if (NT > 1 && rows <= 16) attend<D, 1, RG, PASS>(a, item, line.b, off, lds, ml);
        else if (NT > 2 && rows <= 32) attend<D, NT < 2 ? NT : 2, RG, PASS>(a, item, line.b, off, lds, ml);
        else if (NT > 3 && rows <= 48) attend<D, NT < 3 ? NT : 3, RG, PASS>(a, item, line.b, off, lds, ml);
        else attend<D, NT, RG, PASS>(a, item, line.b, off, lds, ml);
    } else {
        if (!line_part<kStep, PASS>(a, line_lds, line, kRows)) return;
        for (int64_t x = line.lo; x < line.hi;)
            if (next_item<kStep, PASS>(a, line_lds, line, x, item, kRows)) attend<D, NT, RG, PASS>(a, item, line.b, off, lds, ml);
    }
}

// ---------------------------------------------------------------------------
// Prompts: eight waves with 16 NT rows each share every step's keys and
// values, which they unpack together.  Half of the waves turn a step's key
// words into A operands of the first product, half its value words, scaled,
// into those of the second, both as fp16 fragments in LDS that all waves then
// read; the words come straight into registers two steps ahead.  64 tokens a
// step, one barrier: while it is worked on, the next one is unpacked.
// Unpacking costs a wave an eighth of what it would alone.  What bounds the
// kernel is that a part's scores, softmax and values wait for each other, with
// two waves a SIMD to fill the gaps: exp2 and the arithmetic around it take
// twice as long as the products they go with and overlap with them in part, and
// neither pipe is full.  A prompt of 4096 with 48 heads, 128 wide (206 GFLOP):
// 357 to 383 us and 23 for the join, vector instructions 47 % of the time and
// the matrix units 23; kv4_attn with four row groups took 510.  Three chunks of
// 1000 queries under a window of 2048, 64 wide (151 GFLOP): 305 to 329 us and
// 19; 54 % and 19.
// ---------------------------------------------------------------------------
constexpr int kPromptStep = 64;  // tokens of a prompt's step

template <int D, int NT> struct Prompt {
    static constexpr int R = D / 64;
    static constexpr int kRows = kWaves * 16 * NT;
    static constexpr int kFrags = kPromptStep / 16 * 2 * R;       // of K: [tile][block][h]; of V: [32 tokens][block][product], as many
    static constexpr int kBuf = 2 * kFrags * 1024;          // one step's K and V
    static constexpr int kScale = kPromptStep * R * 2;            // K's scales of a step: [token][block] fp16
    static constexpr int kOut = kRows * 2 * D;              // the rows on their way out, where the fragments were
    static constexpr int kSteps = 2 * kBuf + 3 * kScale;
    static constexpr int kLds = kSteps > kOut ? kSteps : kOut;
    static constexpr int kPart = kWaves * NT * 4 * R * 256; // floats of a part
    static constexpr int kUnits = 2 * D;                    // 16-byte units of a step's key codes, and of its value codes
};

// What a thread has of a step to come: one unit of codes, and the scales of
// the four tokens that its own belongs to.
template <int D> struct Raw {
    uint4 w;
    uint32_t s[2 * (D / 64)];
};

template <int D, int NT, int PASS>
__global__ __launch_bounds__(kThreads) void kv4_prompt(AttnArgs a)
{
    using P = Prompt<D, NT>;
    using L = Kv4Layout<D>;
    constexpr int R = P::R, kRows = P::kRows;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // two steps' fragments, three steps' key scales
    __shared__ LineLds line_lds;
    // A step's largest value scale past the cap, read one step ahead of it;
    // whether it misses a page, read with it.  Cleared in the step after.
    __shared__ uint32_t most[3], bad[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const bool keys = wave >= 4;       // unpacks keys; else values
    const int T = 1 << a.c.shift;      // tokens of a page
    // A thread's unit (narrow heads leave every second thread a copy of
    // another's, which it does not write).  Of keys: D / 32 units a row, four
    // words.  Of values: word `part` of four tokens.
    const int unit = tid & (P::kUnits - 1);
    const bool on = (tid & 255) < P::kUnits;
    const int part = keys ? unit % (D / 32) : unit % (D / 8);
    const int token = keys ? unit / (D / 32) : unit / (D / 8) * 4;  // of the step
    Line line;
    if (!line_part<kPromptStep, PASS>(a, line_lds, line, kRows)) return;
    for (int64_t x = line.lo; x < line.hi;) {
        Item item;
        if (!next_item<kPromptStep, PASS>(a, line_lds, line, x, item, kRows)) continue;
        const int head = item.head, tile0 = item.tile0, rows = item.rows, b = line.b;
        Work w{item.c.w};
        const int tile_last = (tile0 + kRows < rows ? tile0 + kRows : rows) - 1;
        span<kPromptStep>(a, w, tile0 / a.group, tile_last / a.group);
        const int32_t t_low = w.first + tile0 / a.group, t_high = w.first + tile_last / a.group;  // the tile's positions
        const int row0 = tile0 + wave * 16 * NT;
        const int last = (row0 + 16 * NT < rows ? row0 + 16 * NT : rows) - 1;
        const int32_t p0 = row0 < rows ? w.first + row0 / a.group : -1, p1 = row0 < rows ? w.first + last / a.group : -1;

        half8_t q[NT][2 * R];
        float4_t o[NT][R][4];
        float m[NT], l[NT];
        int32_t pos[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int at = row0 + 16 * n + r, i = at / a.group;
            const bool live = at < rows;
            pos[n] = live ? w.first + i : -1;
            const uint16_t *from = a.q + (w.q0 + (live ? i : 0)) * a.ldq + (head * a.group + (live ? at - i * a.group : 0)) * D;
#pragma unroll
            for (int y = 0; y < 2 * R; ++y) {
                q[n][y] = *(const half8_t *)(from + 32 * y + 8 * g);
                if (!live) q[n][y] = (half8_t)(_Float16)0.0f;
                if (a.negate) q[n][y] = -q[n][y];
            }
#pragma unroll
            for (int y = 0; y < R; ++y)
#pragma unroll
                for (int i2 = 0; i2 < 4; ++i2) o[n][y][i2] = (float4_t){0, 0, 0, 0};
            m[n] = kLowest;
            l[n] = 0.0f;
        }
        float up = 1.0f;   // 2^u on the values being added
        uint32_t cap = 0;  // largest scale (fp16 bits) that the next step's u leaves below 2^11

        const int e0 = share_of(item.s0, item.all, w.steps);
        const int count = share_of(item.s1, item.all, w.steps) - e0;
        auto token_of = [&](int i) {
            const int e = e0 + i;
            return (e < w.sink_steps ? e : e - w.sink_steps + w.lo) * kPromptStep;
        };
        const int32_t max_pages = a.max_pages - w.skip;  // 0: no keys of its own, and no entry behind the row's end is read
        const int32_t *row = uniform_ptr(a.table + (int64_t)b * a.ld_table + (max_pages > 0 ? w.skip : 0));
        // Page of the thread's token in step i.  Steps past the end repeat the last.
        auto page_of = [&](int i) {
            const int at = (token_of(i < count ? i : count - 1) + token) >> a.c.shift;
            return ((const PN_GLOBAL int32_t *)row)[at < max_pages ? at : max_pages - 1];
        };
        auto ok_page = [&](int32_t page, int i) {
            return (uint32_t)page < (uint32_t)a.c.num_pages && (token_of(i) + token) >> a.c.shift < max_pages;
        };
        // Start the loads of step i; without a branch, or a join of branches
        // would wait for them.  A page that is none of the cache reads page 0.
        auto fetch = [&](Raw<D> &raw, int32_t page, int i) {
            const int o = (token_of(i < count ? i : count - 1) + token) & (T - 1);
            const int64_t at = (uint32_t)page < (uint32_t)a.c.num_pages ? page : 0;
            const uint8_t *from = a.c.pages + (at * a.c.heads + head) * a.c.chunk;
            raw.w = *(const uint4 *)(from + (uint32_t)(keys ? o * L::kRow + 16 * part
                                                            : L::v_codes(T) + ((o >> 2) * (D / 8) + part) * 16));
            const uint8_t *sc = from + (uint32_t)((keys ? L::k_scales(T) : L::v_scales(T)) + 2 * R * (o & ~3));
            if constexpr (R == 1) {
                const uint2 y = *(const uint2 *)sc;
                raw.s[0] = y.x, raw.s[1] = y.y;
            } else {
                const uint4 y = *(const uint4 *)sc;
                raw.s[0] = y.x, raw.s[1] = y.y, raw.s[2] = y.z, raw.s[3] = y.w;
            }
        };
        // The step's words have come: value scales that no row sees become 0
        // (they may be anything), the others are held against the cap; key
        // scales go to LDS, NaN for a token without a page.
        auto look = [&](Raw<D> &raw, int32_t page, int i) {
            if (i >= count) return;
            const bool gone = !ok_page(page, i);
            if (keys) {
                if (part == 0 && on) {
                    uint8_t *to = lds + 2 * P::kBuf + i % 3 * P::kScale + 2 * R * token;
                    if constexpr (R == 1) {
                        const uint32_t w2 = token & 2 ? raw.s[1] : raw.s[0];
                        *(uint16_t *)to = gone ? 0x7e00 : (uint16_t)(token & 1 ? w2 >> 16 : w2);
                    } else {
                        const uint32_t lo = token & 1 ? raw.s[1] : raw.s[0], hi = token & 1 ? raw.s[3] : raw.s[2];
                        *(uint32_t *)to = gone ? 0x7e007e00u : token & 2 ? hi : lo;
                    }
                    if (gone) bad[i % 4] = 1;
                }
            } else {
                const int t0 = token_of(i);
                const int32_t under = before_window(a, t_low);
                const int t1 = t0 + kPromptStep;
                const bool whole = t1 <= w.len && t1 - 1 <= t_high && (t0 > under || t1 <= a.sinks);
                if (!whole || gone) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = t0 + token + j;
                        const bool seen = !gone && t < w.len && t <= t_high && (t > under || t < a.sinks);
#pragma unroll
                        for (int z = 0; z < R; ++z) {
                            const int h = R * j + z;
                            if (!seen) raw.s[h >> 1] &= h & 1 ? 0x0000ffffu : 0xffff0000u;
                        }
                    }
                }
                ushort2_t any = {0, 0};
#pragma unroll
                for (int y = 0; y < 2 * R; ++y)
                    any = __builtin_elementwise_max(any, __builtin_bit_cast(ushort2_t, raw.s[y] & 0x7fff7fffu));
                const uint32_t big = any[0] > any[1] ? any[0] : any[1];
                if (big > cap) atomicMax(&most[i % 3], big);
            }
        };
        // Words into fragments.
        auto unpack = [&](const Raw<D> &raw, int i, float factor) {
            if (i >= count || !on) return;
            half8_t *buf = (half8_t *)(lds + (i & 1) * P::kBuf);
            const uint32_t words[4] = {raw.w.x, raw.w.y, raw.w.z, raw.w.w};
            if (keys) {
                // words (b, h) of one group g of the row, or with one block (h) of two groups
                half8_t *to = buf + (token >> 4) * 2 * R * 64 + (R == 1 ? 32 : 16) * part + (token & 15);
#pragma unroll
                for (int y = 0; y < 4; ++y) to[R == 1 ? (y & 1) * 64 + (y >> 1) * 16 : y * 64] = codes8(words[y]);
            } else {
                const int vb = part >> 3, group = token >> 5, second = token >> 4 & 1, vg = token >> 2 & 3;
                const half2_t f2 = {(_Float16)factor, (_Float16)factor};
                half2_t e[2][2][4];  // [token pair][odd element][product]
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    half2_t sc;
                    if constexpr (R == 1) sc = as_half2(raw.s[u]);
                    else sc = as_half2(__builtin_amdgcn_perm(raw.s[2 * u + 1], raw.s[2 * u], vb ? 0x07060302u : 0x05040100u));
                    sc *= f2;
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        Unpack<1>::run(__builtin_amdgcn_perm(words[2 * u + 1], words[2 * u], odd ? 0x07060302u : 0x05040100u), e[u][odd]);
#pragma unroll
                        for (int i4 = 0; i4 < 4; ++i4) e[u][odd][i4] *= sc;
                    }
                }
                // a lane's 16 bytes: tokens 4 g .. of the first tile, then of the second
                uint8_t *to = (uint8_t *)(buf + (P::kFrags + (group * R + vb) * 4) * 64 + 16 * vg + (part & 7)) + 8 * second;
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd)
                        *(uint2 *)(to + 1024 * i4 + 128 * odd) =
                            make_uint2(__builtin_bit_cast(uint32_t, e[0][odd][i4]), __builtin_bit_cast(uint32_t, e[1][odd][i4]));
            }
        };

        __syncthreads();  // the last item's LDS has been read
        if (tid < 3) most[tid] = 0;
        if (tid < 4) bad[tid] = 0;
        __syncthreads();
        Raw<D> raw;
        int32_t d0 = 0, d1 = 0;  // pages of steps it + 1 and it + 2
        if (count > 0) {
            d0 = page_of(0), d1 = page_of(1);
            fetch(raw, d0, 0);
            if (!keys) look(raw, d0, 0);
        }
        for (int it = -1; it < count && count > 0; ++it) {
            // Step it's fragments are written, step it + 1's words are looked
            // at, and no wave reads step it - 1 any more.  __syncthreads()
            // would wait for the global loads in flight too.
            lds_barrier();
            float next_up = up, f = 1.0f;
            if (it + 1 < count) {
                const uint32_t big = uniform((int)most[(it + 1) % 3]);
                if (big > cap) {  // the same in every wave
                    fit_scales(big, next_up, cap);
                    f = next_up / up;
                }
            }
            if (it >= 0 && tid == 0) {
                most[it % 3] = 0;        // for step it + 3, looked at after the next barrier
                bad[(it + 3) % 4] = 0;   // step it - 1's, for step it + 3
            }
            // Waves that share a SIMD unpack before and after their products,
            // so that one's products meet the other's arithmetic.
            const int32_t d2 = page_of(it + 3);
            if (!keys) {
                unpack(raw, it + 1, next_up);
                fetch(raw, d1, it + 2);
            }
            if (it >= 0) {
                const half8_t *buf = (const half8_t *)(lds + (it & 1) * P::kBuf);
                const uint8_t *scales = lds + 2 * P::kBuf + it % 3 * P::kScale;
                const bool gone = uniform((int)bad[it % 4]) != 0;
#pragma unroll 1
                for (int sub = 0; sub < kPromptStep / 32; ++sub) {
                    const int token0 = token_of(it) + 32 * sub;
                    // nothing of it is visible to the wave's rows
                    if (token0 > p1 || (a.window > 0 && (int64_t)token0 + 31 + a.window <= p0 && token0 >= a.sinks)) continue;
                    const bool some = gone || token0 + 32 > w.len || token0 + 31 > p0 ||
                                      !(a.window <= 0 || (int64_t)token0 + a.window > p1 || token0 + 32 <= a.sinks);
                    // scores: all products, then the scales
                    float4_t sc[NT][2], c[NT][2][R];
                    uint32_t ks[2][2 * R];
#pragma unroll
                    for (int i = 0; i < 2; ++i) read_words(ks[i], scales + 2 * R * (32 * sub + 16 * i + 4 * g));
                    const half8_t *k = buf + sub * 4 * R * 64 + lane;  // [tile][block][h]
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int y = 0; y < R; ++y) {
                                const half8_t kk = k[(i * 2 * R + 2 * y + h) * 64];
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    c[n][i][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                        kk, q[n][2 * y + h], h ? c[n][i][y] : (float4_t){0, 0, 0, 0}, 0, 0, 0);
                            }
                    // the first half of the values on their way meanwhile
                    const half8_t *v = buf + (P::kFrags + sub * R * 4) * 64 + lane;
                    half8_t vv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) vv[i] = v[i * 64];
                    keep_order();
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int y = 0; y < R; ++y)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    sc[n][i][j] = __builtin_fmaf(c[n][i][y][j], half_at(ks[i], R * j + y), y == 0 ? 0.0f : sc[n][i][j]);
                    if (some) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int32_t below = before_window(a, pos[n]);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int key = token0 + 16 * (j >> 2) + 4 * g + (j & 3), h = R * (j & 3);
                                const uint32_t bits = ks[j >> 2][h >> 1] >> (16 * (h & 1)) & 0x7fffu;
                                const bool ok = bits <= 0x7c00u && key < w.len && key <= pos[n] && (key > below || key < a.sinks);
                                sc[n][j >> 2][j & 3] = ok ? sc[n][j >> 2][j & 3] : -__builtin_inff();
                            }
                        }
                    }
                    // weights
                    float mx[NT], more = kLowest;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mx[n] = max3(sc[n][0][0], sc[n][0][1], sc[n][0][2]);
                        mx[n] = max3(mx[n], sc[n][0][3], sc[n][1][0]);
                        mx[n] = max3(mx[n], sc[n][1][1], sc[n][1][2]);
                        mx[n] = max2(mx[n], sc[n][1][3]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) mx[n] = group_max(mx[n]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) more = max2(more, mx[n] - m[n]);
                    if (__ballot(more > a.slack)) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float s = mx[n] > m[n] ? __builtin_amdgcn_exp2f((m[n] - mx[n]) * a.c2) : 1.0f;
                            m[n] = max2(m[n], mx[n]);
                            l[n] *= s;
#pragma unroll
                            for (int y = 0; y < R; ++y)
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[n][y][i] *= s;
                        }
                    }
                    half8_t p[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float mm = kBias - m[n] * a.c2;
                        float sum = 0.0f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float x2 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][j >> 2][j & 3], a.c2, mm));
                            sum += x2;
                            p[n][j] = (_Float16)x2;
                        }
                        l[n] += sum;
                    }
                    // values
#pragma unroll
                    for (int y = 0; y < R; ++y) {
                        half8_t next[4];
                        if (y + 1 < R) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) next[i] = v[(4 * y + 4 + i) * 64];
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                o[n][y][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv[i], p[n], o[n][y][i], 0, 0, 0);
                        if (y + 1 < R) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) vv[i] = next[i];
                        }
                    }
                }
            }
            if (f != 1.0f) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int y = 0; y < R; ++y)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[n][y][i] *= f;
            }
            up = next_up;
            if (!keys) {
                look(raw, d1, it + 2);
            } else {
                look(raw, d0, it + 1);
                unpack(raw, it + 1, 0.0f);
                fetch(raw, d1, it + 2);
            }
            d0 = d1;
            d1 = d2;
        }

        const float down = 1.0f / up;
        const int part_at = 2 * (int)blockIdx.x + (item.s0 == 0 ? 1 : 0);
        if (item.cut) {
            float4_t *part = (float4_t *)(a.part + (int64_t)part_at * P::kPart);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float all_l = group_sum(l[n]);
                if (row0 + 16 * n + r < rows) {
#pragma unroll
                    for (int y = 0; y < 4 * R; ++y) part[((wave * NT + n) * 4 * R + y) * 64 + lane] = o[n][y >> 2][y & 3] * down;
                    if (g == 0) a.part_ml[(int64_t)part_at * kRows + (wave * NT + n) * 16 + r] = make_float2(m[n], all_l);
                }
            }
            continue;
        }
        // By way of LDS into whole rows: a wave's rows lie where the
        // fragments were, a row's 16-byte pieces permuted by its number.
        lds_barrier();
        uint8_t *mine = lds + wave * (16 * NT * 2 * D);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float all_l = group_sum(l[n]);
            float f = all_l > 0.0f ? down / all_l : 0.0f;
            if constexpr (PASS == kTail) {
                const int row_at = row0 + 16 * n + r, i = row_at / a.group, q_head = head * a.group + row_at - i * a.group;
                if (w.skip > 0) {
                    const FrontPlace place = front_place(a, a.members[b], w.q0 + i, q_head, row_at < rows);
                    const FrontRow front = front_row<D>(a, place, m[n], all_l, g);
                    f = 1.0f;
#pragma unroll
                    for (int y = 0; y < 4 * R; ++y) {
                        o[n][y >> 2][y & 3] *= front.own * down;
                        if (row_at < rows) o[n][y >> 2][y & 3] += front_sum(a, front, y);
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < 4 * R; ++y)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int word = 8 * (y >> 2) + 4 * (g & 1) + j + (g & 2);  // piece of the row
                    *(uint32_t *)(mine + (16 * n + r) * 2 * D + 16 * (word ^ (r & (D / 8 - 1))) + 4 * (y & 3)) =
                        row_pair(o[n][y >> 2][y & 3] * f, j);
                }
        }
        asm volatile("" ::: "memory");  // a wave reads what it wrote itself
#pragma unroll
        for (int y = 0; y < 16 * NT * D / 8; y += 64) {
            const int at = (y + lane) / (D / 8), c = (y + lane) % (D / 8), row_at = row0 + at, i = row_at / a.group;
            const uint4 v = *(const uint4 *)(mine + at * 2 * D + 16 * (c ^ (at & 15 & (D / 8 - 1))));
            if (row_at < rows)
                *(uint4 *)(a.out + (w.q0 + i) * a.ldo + (int64_t)(head * a.group + row_at - i * a.group) * D + 8 * c) = v;
        }
    }
}

// Add the parts of an item that a workgroup left unfinished.  Grid: x =
// workgroup, y = block, z = 16-row group.  Product i = wave & 3; of W = 4, 8 or
// 16 waves those of a product share its parts, 16 of them each at a time: many
// parts take more waves, but those cost where there are many items (256 wide,
// 4 heads, 16 requests of 8 queries and up to 5000 tokens, 64 items of about
// 4 parts: 36 us in all with 4 waves, 40 with 8, 49 with 16; one token over
// 65536 keys, 4 items of 63 parts: this launch 15, 9.5 and 7.9 us).
template <int D, int W, int PASS>
__global__ __launch_bounds__(64 * W) void kv4_join(AttnArgs a, int groups)
{
    constexpr int R = D / 64, F = W / 4;  // F: waves that share a product's parts
    constexpr int kDeep = 16, kAt = F * kDeep;  // parts of a wave, and in all, at a time
    __shared__ float4_t frag[W][64];
    __shared__ float2 ml[kAt][16];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int y = blockIdx.y, n = blockIdx.z, i = wave & 3;
    const Cutoff c = a.cuts[blockIdx.x];
    const int parts = c.parts;
    if (parts < 2 || c.row0 + 16 * n >= c.rows) return;  // the whole workgroup
    // The first workgroup has the item's start (its part 1), the others go on with it (their part 0).
    auto part = [&](int j) { return 2 * ((int64_t)blockIdx.x + j) + (j == 0 ? 1 : 0); };
    float m = kLowest, l = 0.0f;
    float4_t o = {0, 0, 0, 0};
    // each wave takes its share of the parts for its product, and the rows'
    // (m, l) come one a thread
    for (int j0 = 0; j0 < parts; j0 += kAt) {
        float4_t v[kDeep];
#pragma unroll
        for (int x = 0; x < kDeep; ++x) {
            const int j = j0 + (wave >> 2) + F * x;
            v[x] = (float4_t){0, 0, 0, 0};
            if (j < parts) v[x] = ((const float4_t *)a.part)[(part(j) * groups + n) * 4 * R * 64 + (4 * y + i) * 64 + lane];
        }
        const int j = j0 + ((int)threadIdx.x >> 4);
        const float2 x = j < parts ? a.part_ml[(part(j) * groups + n) * 16 + (threadIdx.x & 15)] : make_float2(kLowest, 0.0f);
        __syncthreads();
        ml[threadIdx.x >> 4][threadIdx.x & 15] = x;
        __syncthreads();
        float top = m;
        for (int j2 = g; j2 < kAt; j2 += 4) top = max2(top, ml[j2][r].x);
        top = group_max(top);
        const float f = __builtin_amdgcn_exp2f((m - top) * a.c2);
        l *= f;
        o *= f;
        for (int j2 = g; j2 < kAt; j2 += 4) l += ml[j2][r].y * __builtin_amdgcn_exp2f((ml[j2][r].x - top) * a.c2);
#pragma unroll
        for (int x2 = 0; x2 < kDeep; ++x2)
            if (j0 + (wave >> 2) + F * x2 < parts)
                o += v[x2] * __builtin_amdgcn_exp2f((ml[(wave >> 2) + F * x2][r].x - top) * a.c2);
        m = top;
    }
    l = group_sum(l);
    frag[wave][lane] = o;
    __syncthreads();
    if (wave < 4) {
        const int at = c.row0 + 16 * n + r, q = at / a.group;
        o = frag[wave][lane];
#pragma unroll
        for (int x = 1; x < F; ++x) o += frag[4 * x + wave][lane];
        const bool live = at < c.rows;
        const int q_head = (PASS == kTail ? c.head & 0xffff : c.head) * a.group + at - q * a.group;
        float f = l > 0.0f ? 1.0f / l : 0.0f;
        if constexpr (PASS == kTail) {
            const int b = (int)((uint32_t)c.head >> 16);
            if (uniform(a.members[b].skip) > 0) {
                const FrontRow front = front_row<D>(a, front_place(a, a.members[b], c.q0 + q, q_head, live), m, l, g);
                f = front.own;
                if (live) o = o * f + front_sum(a, front, 4 * y + wave);
                f = 1.0f;
            }
        }
        uint16_t *out = a.out + (c.q0 + q) * a.ldo + (int64_t)q_head * D;
        store_row(live ? out : nullptr, o * f, y, wave, g);
    }
}

// 16-row groups of a prompt's waves.  64 wide: two would do for the registers'
// sake but give each unpacked step half the work (16 heads, a prompt of 4096:
// 104 us with four, 118 with two); 128 wide has registers for two.
template <int D> constexpr int kPromptRows = D == 64 ? 4 : 2;

// How a call is cut.
struct Cut {
    int nt, rg;   // 16-row groups of a wave, row groups of a workgroup
    int workers;
    bool two;     // of them a compute unit
    bool whole;
    int parts;    // of an item, about, with one workgroup a compute unit
    size_t part;  // bytes that one workgroup's parts and record need
};

size_t part_bytes(const pn_kv4_cache *c, const Cut &t)
{
    return 2 * (size_t)t.rg * t.nt * (c->dim * 16 * sizeof(float) + 16 * sizeof(float2)) + sizeof(Cutoff);
}

Cut cut(const pn_kv4_cache *c, int q_heads, int B, int64_t max_q, int64_t max_kv, int window, int sinks)
{
    Cut t;
    const int64_t rows = max_q * (q_heads / c->heads);
    const int most = c->dim == 256 ? 2 : 4;  // that the registers hold
    t.nt = rows >= 16 * most ? most : (int)((rows + 15) / 16);
    // A prompt's workgroup pays for its whole row tile; up to one tile's rows
    // the kernel of few rows is faster, each 16 nt rows a tile of its own and
    // the keys read again for each.  8 requests over 4096 keys: 64 wide, 512
    // rows 78 us either way, 192 rows 43 (prompt kernel 58), 768 rows 98
    // (86); 128 wide, 256 rows 67 (68), 192 rows 57 (65), 384 rows 88 (75);
    // 256 wide, 96 rows 63 (66), 256 rows 115 (106).
    const int tile = c->dim == 256 ? 128 : 16 * kWaves * (c->dim == 128 ? kPromptRows<128> : kPromptRows<64>);
    t.rg = rows > tile ? c->dim == 256 ? 4 : kWaves : 1;
    if (t.rg == kWaves) t.nt = c->dim == 128 ? kPromptRows<128> : kPromptRows<64>;
    int64_t keys = max_kv;
    if (window > 0) {
        const int64_t reach = (int64_t)window + max_q + sinks + 2 * kStep;
        if (reach < keys) keys = reach;
    }
    t.two = c->dim < 256 && t.nt == 1;
    t.workers = device_cus() * (t.two ? 2 : 1);
    t.whole = keys <= 2 * kShare * kStep;
    const int64_t tile_rows = 16 * t.nt * t.rg, items = (int64_t)B * c->heads * ((rows + tile_rows - 1) / tile_rows);
    const int64_t longest = keys / (kShare * kStep) + 1;
    t.parts = (int)(items * longest < device_cus() ? longest : device_cus() / items);
    t.part = part_bytes(c, t);
    return t;
}

template <int D, int NT, int RG, int PASS> bool raise_one()
{
    return hipFuncSetAttribute((const void *)kv4_attn<D, NT, RG, PASS>, hipFuncAttributeMaxDynamicSharedMemorySize,
                               Shape<D, NT, RG>::kLds) == hipSuccess;
}

template <int D, int PASS> bool raise_prompt()
{
    return hipFuncSetAttribute((const void *)kv4_prompt<D, kPromptRows<D>, PASS>, hipFuncAttributeMaxDynamicSharedMemorySize,
                               Prompt<D, kPromptRows<D>>::kLds) == hipSuccess;
}

// Raise the LDS limits of a pass's kernels.
template <int PASS> bool raise_pass()
{
    if constexpr (PASS == kWhole || PASS == kTail) {
        if (!raise_one<256, 2, 4, PASS>() || !raise_prompt<64, PASS>() || !raise_prompt<128, PASS>()) return false;
    }
    return raise_one<64, 1, 1, PASS>() && raise_one<64, 2, 1, PASS>() && raise_one<64, 3, 1, PASS>() &&
           raise_one<64, 4, 1, PASS>() && raise_one<128, 1, 1, PASS>() && raise_one<128, 2, 1, PASS>() &&
           raise_one<128, 3, 1, PASS>() && raise_one<128, 4, 1, PASS>() && raise_one<256, 1, 1, PASS>() &&
           raise_one<256, 2, 1, PASS>();
}

template <int D, int NT, int RG, int PASS>
pn_status launch(const AttnArgs &a, hipStream_t s)
{
    const unsigned workers = PASS == kOwn ? (unsigned)((int64_t)a.B * a.c.heads * a.tiles) : (unsigned)(PASS == kFront ? a.grid : a.workers);
    hipLaunchKernelGGL((kv4_attn<D, NT, RG, PASS>), dim3(workers), dim3(kThreads), (Shape<D, NT, RG>::kLds), s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    if constexpr (PASS == kWhole || PASS == kTail) {
        if (a.whole) return PN_OK;
        const dim3 grid((unsigned)a.workers, D / 64, NT * RG);
        if (RG > 1 || a.parts <= 4) hipLaunchKernelGGL((kv4_join<D, 4, PASS>), grid, dim3(256), 0, s, a, NT * RG);
        else if (a.parts <= 32) hipLaunchKernelGGL((kv4_join<D, 8, PASS>), grid, dim3(512), 0, s, a, NT * RG);
        else hipLaunchKernelGGL((kv4_join<D, 16, PASS>), grid, dim3(1024), 0, s, a, NT * RG);
        if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    }
    return PN_OK;
}

template <int D, int NT, int PASS>
pn_status launch_prompt(const AttnArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((kv4_prompt<D, NT, PASS>), dim3((unsigned)a.workers), dim3(kThreads), (Prompt<D, NT>::kLds), s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    if (!a.whole) {
        hipLaunchKernelGGL((kv4_join<D, 4, PASS>), dim3((unsigned)a.workers, D / 64, NT * kWaves), dim3(256), 0, s, a, NT * kWaves);
        if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    }
    return PN_OK;
}

template <int D, int PASS>
pn_status launch_rows(const AttnArgs &a, const Cut &t, hipStream_t s)
{
    constexpr int most = D == 256 ? 2 : 4;
    if constexpr (PASS == kOwn || PASS == kFront) {
        if (t.rg > 1) return PN_EUNSUPPORTED;
    } else if constexpr (D == 256) {
        if (t.rg > 1) return launch<D, most, 4, PASS>(a, s);
    } else {
        if (t.rg > 1) return launch_prompt<D, kPromptRows<D>, PASS>(a, s);
    }
    if (t.nt == 1) return launch<D, 1, 1, PASS>(a, s);
    if (t.nt == 2) return launch<D, 2, 1, PASS>(a, s);
    if constexpr (D <= 128) {
        if (t.nt == 3) return launch<D, 3, 1, PASS>(a, s);
        if (t.nt == 4) return launch<D, 4, 1, PASS>(a, s);
    }
    return PN_EUNSUPPORTED;
}

template <int PASS> pn_status launch_pass(const AttnArgs &a, const Cut &t, int dim, hipStream_t s)
{
    return dim == 64 ? launch_rows<64, PASS>(a, t, s) : dim == 128 ? launch_rows<128, PASS>(a, t, s)
                                                                   : launch_rows<256, PASS>(a, t, s);
}

bool sizes_ok(const pn_kv4_cache *c, int q_heads, int B, int64_t total_q, int64_t max_q, int64_t max_kv, int sinks)
{
    return q_heads >= c->heads && q_heads % c->heads == 0 && B >= 1 && total_q >= 0 && max_q >= 1 && max_kv >= 1 &&
           sinks >= 0;
}

bool sizes_fit(const pn_kv4_cache *c, int q_heads, int B, int64_t total_q, int64_t max_q, int64_t max_kv)
{
    return B <= 65535 && q_heads <= 65535 && total_q <= INT32_MAX / 2 && max_kv <= INT32_MAX / 2 &&
           max_q * (q_heads / c->heads) <= INT32_MAX / 4;
}

bool scale_ok(float scale) { return __builtin_fabsf(scale) <= 0x1.fffffep127f; }  // not infinite or NaN

void set_scale(AttnArgs &a, float scale)
{
    a.negate = scale < 0.0f;
    // Not 0: a masked score is -inf, whose product with c2 has to stay so.
    a.c2 = __builtin_fmaxf(__builtin_fabsf(scale) * 1.4426950408889634f, 0x1p-100f);
    a.slack = 4.0f / a.c2;
}

// The parts' memory of a launch cut by t, and fewer workgroups (or items that
// are not cut) where there is not room for all.
void set_cut(AttnArgs &a, const pn_kv4_cache *cache, Cut &t, void *ws, size_t ws_bytes)
{
    if (!t.whole && ws_bytes < t.workers * t.part) {
        // As many workgroups as there is room for, while that leaves most of
        // the device at work; else every item is one workgroup's.
        const int fit = (int)(ws_bytes / t.part);
        if (fit >= t.workers / 4) t.workers = fit;
        else t.whole = true;
    }
    a.part = (float *)ws;
    const size_t groups = 2 * (size_t)t.workers * t.nt * t.rg;
    a.part_ml = (float2 *)(a.part + groups * cache->dim * 16);
    a.cuts = (Cutoff *)(a.part_ml + groups * 16);
    a.workers = t.workers;
    a.two = t.two;
    a.parts = t.parts;
    const int tile_rows = 16 * t.nt * t.rg;
    a.queries = (tile_rows + a.group - 1) / a.group;
    a.grow = tile_rows * kUnit / (a.group * (t.rg == kWaves ? kPromptStep : kStep));
    a.whole = t.whole;
    // What an item's start and end cost in steps.  64 wide, 64 requests of up
    // to 16384: 54 us, counted as nothing 80, twice as much 57; 128 wide, a
    // prompt of 4096 with 16 heads: 149 us, nothing 185, twice 162.
    a.over = t.rg == kWaves ? 6 : 32;
}

}  // namespace

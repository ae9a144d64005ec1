// pn_kv4_plan.hip - block tables, slots and positions of one decoding step,
// built on the device from request lengths (pn_kv4_plan), for AMD Instinct
// MI355X (gfx950).
//
// Two prefix sums over the requests (new tokens, fresh pages) order
// everything else: token t belongs to the last request that starts at or
// before t, and the i-th fresh page to the last request whose pages start at
// or before i.  Every workgroup computes both sums for itself into LDS (at
// most 8192 requests of 12 bytes, which the L2s hold) and then takes its
// share of the tokens and of the fresh pages by binary search, so the whole
// step is one launch with no workgroup waiting for another, no atomics, and
// the same result every time.  One more workgroup counts the lost tokens,
// which takes table entries and free pages that the others need not read
// alike: 4000 requests 12.4 us so, 11.7 where it counted by lengths alone (and
// missed entries of -1).  Sums saturate at INT32_MAX: saturating addition of
// non-negative numbers is associative, so the scan may group as it likes.
//
// Latency bounds it: the bytes are a few MB at most.  16 requests of 8 new
// tokens: 5.4 us, 4000 requests of 8 tokens or a prompt: 12.4 us, where a
// launch alone takes 3.6: the rest is three dependent rounds of loads, the
// scan and the searches in LDS.  (All loads of a thread's requests first
// changes neither.)
#include "pn_kv4.h"

using namespace pn::host;

namespace {

constexpr int kThreads = 1024;
constexpr int kPer = PN_KV4_MAX_BATCH / kThreads;  // requests a thread scans at most
constexpr int kOwn = 2;  // columns of a request that a thread looks at alone

struct PlanArgs {
    const int32_t *ctx, *fresh, *held, *free_pages;
    int32_t *table, *held_out, *q_start, *kv_len, *positions, *info;
    int64_t *slots;
    int64_t ld_table, max_tokens;
    int32_t B, num_free, shift, max_pages;
};

__device__ __forceinline__ int32_t sat(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int32_t)v; }
__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b) { return sat((int64_t)a + b); }
__device__ __forceinline__ int32_t pos0(int32_t v) { return v < 0 ? 0 : v; }

// Last index i in [0, n) with a[i] <= v; a ascending, a[0] <= v.
__device__ __forceinline__ int last_at_most(const int32_t *a, int n, int32_t v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int32_t pages_for(int64_t tokens, int shift)
{
    return (int32_t)((tokens + ((int64_t)1 << shift) - 1) >> shift);
}

// The tokens without a place, by one workgroup: a request loses a tail (from
// its first column without an entry, or from max_tokens on) and what lies in
// columns before it whose entry is -1.
__device__ void count_lost(const PlanArgs &a, const int32_t *start, const int32_t *page0)
{
    __shared__ int32_t lost[kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t pages = page0[a.B];
    int32_t mine = 0;
    // New tokens of request i before its tail.
    auto keep_of = [&](int i) {
        const int64_t n = pos0(a.fresh[i]), held = pos0(a.held[i]), took = page0[i + 1] - page0[i];
        int64_t got = (int64_t)a.num_free - page0[i];
        got = got < 0 ? 0 : got < took ? got : took;
        const int64_t cols = held + got < a.max_pages ? held + got : a.max_pages;
        int64_t keep = (cols << a.shift) - pos0(a.ctx[i]);
        if (n < keep) keep = n;
        if (a.max_tokens - start[i] < keep) keep = a.max_tokens - start[i];
        return keep < 0 ? 0 : keep;
    };
    // Of the first `keep` new tokens of a request with ctx before, those in column c.
    auto in_column = [&](int64_t ctx, int64_t keep, int64_t c) {
        const int64_t lo = c << a.shift, hi = lo + ((int64_t)1 << a.shift);
        const int64_t n = (hi < ctx + keep ? hi : ctx + keep) - (lo > ctx ? lo : ctx);
        return (int32_t)(n < 0 ? 0 : n);
    };
    for (int i0 = 0; i0 < a.B; i0 += kThreads) {
        const int i = i0 + tid;
        int64_t ctx = 0, keep = 0;
        int32_t c0 = 0, c1 = 0;  // held columns that its new tokens lie in
        if (i < a.B) {
            ctx = pos0(a.ctx[i]);
            keep = keep_of(i);
            mine = sat_add(mine, (int32_t)(pos0(a.fresh[i]) - keep));
            const int32_t held = pos0(a.held[i]), end = pages_for(ctx + keep, a.shift);
            c0 = (int32_t)(ctx >> a.shift);
            c1 = keep > 0 ? end < held ? end : held : 0;
        }
        // Entries of -1 among them.  A few are this thread's, many (pages held
        // far ahead of a prompt) the whole wave's.
        const bool many = c1 - c0 > kOwn;
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (!many && c0 + j < c1 && a.table[i * a.ld_table + c0 + j] < 0)
                mine = sat_add(mine, in_column(ctx, keep, c0 + j));
        for (uint64_t left = __ballot(many); left; left &= left - 1) {
            const int l = __builtin_ctzll(left), from = __shfl(c0, l, 64), to = __shfl(c1, l, 64);
            const int64_t row = (int64_t)(i0 + (tid & ~63) + l) * a.ld_table;
            const int64_t its_ctx = __shfl(ctx, l, 64), its_keep = __shfl(keep, l, 64);
            for (int c = from + lane; c < to; c += 64)
                if (a.table[row + c] < 0) mine = sat_add(mine, in_column(its_ctx, its_keep, c));
        }
    }
    // Entries of -1 among the fresh ones.
    for (int64_t p = tid; p < pages && p < a.num_free; p += kThreads) {
        if (a.free_pages[p] >= 0) continue;
        const int i = last_at_most(page0, a.B, (int32_t)p);
        mine = sat_add(mine, in_column(pos0(a.ctx[i]), keep_of(i), (int64_t)pos0(a.held[i]) + (p - page0[i])));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) mine = sat_add(mine, __shfl_xor(mine, d, 64));
    if (lane == 0) lost[wave] = mine;
    __syncthreads();
    if (tid == 0) {
        int32_t all = 0;
        for (int w = 0; w < kThreads / 64; ++w) all = sat_add(all, lost[w]);
        a.info[0] = pages < a.num_free ? pages : a.num_free;
        a.info[1] = all;
    }
}

__global__ __launch_bounds__(kThreads) void kv4_plan(PlanArgs a)
{
    __shared__ int32_t start[PN_KV4_MAX_BATCH + 1];  // first token of each request
    __shared__ int32_t page0[PN_KV4_MAX_BATCH + 1];  // first fresh page of each request
    __shared__ int32_t part[2][kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.B + kThreads - 1) / kThreads;

    // thread-local sums, then a wave scan, then the waves' totals
    int32_t tok[kPer], pg[kPer], ts = 0, ps = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid * per + j;
        tok[j] = ts;
        pg[j] = ps;
        if (j < per && i < a.B) {
            const int32_t n = pos0(a.fresh[i]);
            const int32_t need = pages_for((int64_t)pos0(a.ctx[i]) + n, a.shift);
            ts = sat_add(ts, n);
            ps = sat_add(ps, pos0(need - pos0(a.held[i])));
        }
    }
    int32_t ti = ts, pi = ps;  // inclusive over the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t t = __shfl_up(ti, d, 64), p = __shfl_up(pi, d, 64);
        if (lane >= d) {
            ti = sat_add(ti, t);
            pi = sat_add(pi, p);
        }
    }
    if (lane == 63) {
        part[0][wave] = ti;
        part[1][wave] = pi;
    }
    // exclusive over the wave
    int32_t te = __shfl_up(ti, 1, 64), pe = __shfl_up(pi, 1, 64);
    if (lane == 0) te = pe = 0;
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        te = sat_add(te, part[0][w]);
        pe = sat_add(pe, part[1][w]);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid * per + j;
        if (j < per && i < a.B) {
            start[i] = sat_add(te, tok[j]);
            page0[i] = sat_add(pe, pg[j]);
        }
    }
    if (tid == kThreads - 1) {
        start[a.B] = sat_add(te, ts);
        page0[a.B] = sat_add(pe, ps);
    }
    __syncthreads();

    if (blockIdx.x == gridDim.x - 1) {  // the last workgroup has this alone to do
        count_lost(a, start, page0);
        return;
    }
    const int64_t step = (int64_t)(gridDim.x - 1) * kThreads, first = (int64_t)blockIdx.x * kThreads + tid;
    const int32_t total = start[a.B], pages = page0[a.B];

    // what each request gets
    for (int64_t i = first; i <= a.B; i += step) {
        a.q_start[i] = start[i];
        if (i == a.B) break;
        const int64_t len = (int64_t)pos0(a.ctx[i]) + pos0(a.fresh[i]);
        const int32_t need = pages_for(len, a.shift), held = pos0(a.held[i]);
        a.kv_len[i] = sat(len);
        a.held_out[i] = need > held ? need : held;
    }
    // fresh pages into the table
    for (int64_t p = first; p < pages; p += step) {
        const int i = last_at_most(page0, a.B, (int32_t)p);
        const int64_t col = (int64_t)pos0(a.held[i]) + (p - page0[i]);
        if (col < a.max_pages) a.table[i * a.ld_table + col] = p < a.num_free ? a.free_pages[p] : -1;
    }
    // the step's tokens
    for (int64_t t = first; t < a.max_tokens; t += step) {
        int32_t pos = -1;
        int64_t slot = -1;
        if (t < total) {
            const int i = last_at_most(start, a.B, (int32_t)t);
            const int64_t at = (int64_t)pos0(a.ctx[i]) + (t - start[i]);
            const int32_t col = (int32_t)(at >> a.shift), held = pos0(a.held[i]);
            int32_t page = -1;
            if (col < a.max_pages) {
                if (col < held) {
                    page = a.table[i * a.ld_table + col];
                } else {
                    const int64_t p = (int64_t)page0[i] + (col - held);
                    if (p < a.num_free) page = a.free_pages[p];
                }
            }
            pos = sat(at);
            if (page >= 0) slot = ((int64_t)page << a.shift) + (at & ((1 << a.shift) - 1));
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
}

}  // namespace

extern "C" pn_status pn_kv4_plan(const int32_t *ctx_len, const int32_t *new_len, const int32_t *held, int B,
                                 const int32_t *free_pages, int num_free, int page_size, int32_t *table,
                                 int64_t ld_table, int max_pages, int32_t *held_out, int32_t *q_start,
                                 int32_t *kv_len, int32_t *positions, int64_t *slots, int64_t max_tokens,
                                 int32_t *info, void *stream)
{
    if (!ctx_len || !new_len || !held || !table || !held_out || !q_start || !kv_len || !positions || !slots || !info ||
        (!free_pages && num_free != 0))
        return PN_EINVAL;
    const int shift = page_shift(page_size);
    if (B < 1 || num_free < 0 || shift < 0 || max_pages < 1 || ld_table < max_pages || max_tokens < 1) return PN_ESHAPE;
    const void *words[] = {ctx_len, new_len, held, free_pages, table, held_out, q_start, kv_len, positions, info};
    for (const void *p : words)
        if (!aligned(p, 4)) return PN_EALIGN;
    if (!aligned(slots, 8)) return PN_EALIGN;
    if (B > PN_KV4_MAX_BATCH || max_tokens > INT32_MAX) return PN_EUNSUPPORTED;
    // Workgroups read the first five while others write the last seven (of the table different entries).
    const struct { const void *p; int64_t bytes; } arrays[] = {
        {ctx_len, 4 * (int64_t)B}, {new_len, 4 * (int64_t)B}, {held, 4 * (int64_t)B}, {free_pages, 4 * (int64_t)num_free},
        {table, 4 * ((int64_t)(B - 1) * ld_table + max_pages)}, {held_out, 4 * (int64_t)B}, {q_start, 4 * ((int64_t)B + 1)},
        {kv_len, 4 * (int64_t)B}, {positions, 4 * max_tokens}, {slots, 8 * max_tokens}, {info, 8}};
    for (int i = 4; i < 11; ++i)
        for (int j = 0; j < i; ++j) {
            const uintptr_t x = (uintptr_t)arrays[i].p, y = (uintptr_t)arrays[j].p;
            if (x < y + (uintptr_t)arrays[j].bytes && y < x + (uintptr_t)arrays[i].bytes) return PN_EINVAL;
        }
    const PlanArgs a = {ctx_len, new_len, held, free_pages, table, held_out, q_start, kv_len, positions, info,
                        slots, ld_table, max_tokens, B, num_free, shift, max_pages};
    int64_t grid = (max_tokens + kThreads - 1) / kThreads;
    if (grid > device_cus()) grid = device_cus();
    hipLaunchKernelGGL(kv4_plan, dim3((unsigned)grid + 1), dim3(kThreads), 0, (hipStream_t)stream, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    g_last_variant = kVarKv4Plan;
    return PN_OK;
}

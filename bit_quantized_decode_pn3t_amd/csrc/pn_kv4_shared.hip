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
// queries its own keys and joins them with those parts.
#include "pn_kv4_attn.h"

namespace {

// ---------------------------------------------------------------------------
// Many rows (16 row groups and more a tile): eight waves of up to NT 16-row
// groups share every step's keys and values, which they unpack together into
// fp16 fragments in LDS, one step ahead.  Group j of a tile is wave j % 8's: a
// tile's groups are spread evenly, and the two waves of a SIMD (w and w + 4)
// between them.  Every key is visible to every row, so a step is products,
// exp2 and products; steps with tokens that are not there (behind the prefix's
// end, pages that are none) are masked by key scales of NaN.  A step's maximum
// is looked at lane by lane, and across lanes only where one passes the running
// maximum by more than the slack; sums of weights are a product with ones.
// ---------------------------------------------------------------------------
template <int D> struct Front {
    static constexpr int R = D / 64;
    static constexpr int NT = D == 64 ? 4 : D == 128 ? 2 : 1;  // that the registers hold
    static constexpr int kTokens = D == 256 ? 32 : 64;         // of a step
    static constexpr int kRows = kWaves * 16 * NT;
    static constexpr int kFrags = kTokens / 16 * 2 * R;        // of K: [tile][block][h]; of V: [32 tokens][block][product], as many
    static constexpr int kBuf = 2 * kFrags * 1024;             // one step's K and V
    static constexpr int kScale = kTokens * R * 2;             // K's scales of a step: [token][block] fp16
    static constexpr int kLds = 2 * kBuf + 3 * kScale;
    static constexpr int kUnits = kTokens * D / 32;            // 16-byte units of a step's key codes, and of its value codes
};

// What a wave holds of its row groups.
template <int D> struct Rows {
    static constexpr int R = D / 64, NT = Front<D>::NT;
    half8_t q[NT][2 * R];
    float4_t o[NT][R][4], l[NT];  // l: in all lanes, the sum of the weights exp2(c2 (s - m) + kBias)
    float m[NT];
};

// SUBS times 32 tokens for NA row groups.  k, v: the lane's place in their fragments.
template <int D, int NA, int SUBS>
__device__ __forceinline__ void front_steps(Rows<D> &w, const half8_t *k, const half8_t *v, const uint8_t *scales, bool bad,
                                            float c2, float slack, int g)
{
    constexpr int R = D / 64;
    float4_t sc[NA][2 * SUBS];
#pragma unroll
    for (int i = 0; i < 2 * SUBS; ++i) {
        uint32_t ks[2 * R];
        read_words(ks, scales + 2 * R * (16 * i + 4 * g));
        float4_t c[NA][R];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int y = 0; y < R; ++y) {
                const half8_t kk = k[(i * 2 * R + 2 * y + h) * 64];
#pragma unroll
                for (int n = 0; n < NA; ++n)
                    c[n][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk, w.q[n][2 * y + h], h ? c[n][y] : (float4_t){0, 0, 0, 0}, 0, 0, 0);
            }
#pragma unroll
        for (int n = 0; n < NA; ++n)
#pragma unroll
            for (int y = 0; y < R; ++y)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sc[n][i][j] = __builtin_fmaf(c[n][y][j], half_at(ks, R * j + y), y == 0 ? 0.0f : sc[n][i][j]);
    }
    if (bad) {
#pragma unroll
        for (int n = 0; n < NA; ++n)
#pragma unroll
            for (int i = 0; i < 2 * SUBS; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[n][i][j] = sc[n][i][j] == sc[n][i][j] ? sc[n][i][j] : -__builtin_inff();
    }
    float mx[NA], more = kLowest;
#pragma unroll
    for (int n = 0; n < NA; ++n) {
        mx[n] = max3(sc[n][0][0], sc[n][0][1], sc[n][0][2]);
        mx[n] = max2(mx[n], sc[n][0][3]);
#pragma unroll
        for (int i = 1; i < 2 * SUBS; ++i) {
            mx[n] = max3(mx[n], sc[n][i][0], sc[n][i][1]);
            mx[n] = max3(mx[n], sc[n][i][2], sc[n][i][3]);
        }
        more = max2(more, mx[n] - w.m[n]);
    }
    if (__ballot(more > slack)) {
#pragma unroll
        for (int n = 0; n < NA; ++n) {
            const float top = group_max(mx[n]);
            const float s = top > w.m[n] ? __builtin_amdgcn_exp2f((w.m[n] - top) * c2) : 1.0f;
            w.m[n] = max2(w.m[n], top);
            w.l[n] *= s;
#pragma unroll
            for (int y = 0; y < R; ++y)
#pragma unroll
                for (int i = 0; i < 4; ++i) w.o[n][y][i] *= s;
        }
    }
    const half8_t ones = {1, 1, 1, 1, 1, 1, 1, 1};
    half8_t p[NA][SUBS];
#pragma unroll
    for (int sub = 0; sub < SUBS; ++sub) {
#pragma unroll
        for (int n = 0; n < NA; ++n) {
            const float mm = kBias - w.m[n] * c2;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                p[n][sub][j] = (_Float16)__builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][2 * sub + (j >> 2)][j & 3], c2, mm));
        }
#pragma unroll
        for (int n = 0; n < NA; ++n) w.l[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p[n][sub], w.l[n], 0, 0, 0);
#pragma unroll
        for (int y = 0; y < R; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const half8_t vv = v[((sub * R + y) * 4 + i) * 64];
#pragma unroll
                for (int n = 0; n < NA; ++n)
                    w.o[n][y][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, p[n][sub], w.o[n][y][i], 0, 0, 0);
            }
    }
}

template <int D, int NA>
__device__ __forceinline__ void front_step(Rows<D> &w, const half8_t *k, const half8_t *v, const uint8_t *scales, bool bad,
                                           float c2, float slack, int g)
{
    using P = Front<D>;
    constexpr int SUBS = P::kTokens == 64 && NA <= 2 ? 2 : 1;
#pragma unroll 1
    for (int sub = 0; sub < P::kTokens / 32; sub += SUBS)
        front_steps<D, NA, SUBS>(w, k + sub * 4 * P::R * 64, v + sub * 4 * P::R * 64, scales + 64 * P::R * sub, bad, c2, slack, g);
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv4_front(AttnArgs a)
{
    using P = Front<D>;
    using L = Kv4Layout<D>;
    constexpr int R = P::R, NT = P::NT;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // two steps' fragments, three steps' key scales
    __shared__ LineLds line_lds;
    // A step's largest value scale past the cap, read one step ahead of it;
    // whether it misses tokens, read with it.  Cleared in the step after.
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
    if (blockIdx.x == 0) group_members(a);
    if (!line_part<P::kTokens, kFront>(a, line_lds, line, a.f_tile)) return;
    for (int64_t x = line.lo; x < line.hi;) {
        Item item;
        if (!next_item<P::kTokens, kFront>(a, line_lds, line, x, item, a.f_tile)) continue;
        const int head = item.head, tile0 = item.tile0, b = line.b;
        const Request req = item.c.w;
        const int rows = item.rows - tile0 < a.f_tile ? item.rows - tile0 : a.f_tile;  // of the tile
        const int active = uniform(((rows + 15) / 16 - wave + kWaves - 1) / kWaves);   // the wave's groups; 0 or less: none

        Rows<D> w;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int at = 16 * (wave + kWaves * n) + r, row = tile0 + at, i = row / a.group;
            const bool live = at < rows;
            const uint16_t *from = a.q + (req.q0 + (live ? i : 0)) * a.ldq + (head * a.group + (live ? row - i * a.group : 0)) * D;
#pragma unroll
            for (int y = 0; y < 2 * R; ++y) {
                w.q[n][y] = *(const half8_t *)(from + 32 * y + 8 * g);
                if (!live) w.q[n][y] = (half8_t)(_Float16)0.0f;
                if (a.negate) w.q[n][y] = -w.q[n][y];
            }
#pragma unroll
            for (int y = 0; y < R; ++y)
#pragma unroll
                for (int i2 = 0; i2 < 4; ++i2) w.o[n][y][i2] = (float4_t){0, 0, 0, 0};
            w.m[n] = kLowest;
            w.l[n] = (float4_t){0, 0, 0, 0};
        }
        float up = 1.0f;   // 2^u on the values being added
        uint32_t cap = 0;  // largest scale (fp16 bits) that the next step's u leaves below 2^11

        const int steps = (req.len + P::kTokens - 1) / P::kTokens;
        const int e0 = share_of(item.s0, item.all, steps);
        const int count = share_of(item.s1, item.all, steps) - e0;
        const int32_t *row = uniform_ptr(a.table + (int64_t)b * a.ld_table);
        // The thread's token in step i of the part.  Steps past the end repeat the last.
        auto token_at = [&](int i) { return (e0 + (i < count ? i : count - 1)) * P::kTokens + token; };
        auto page_of = [&](int i) {
            const int at = token_at(i) >> a.c.shift;
            return ((const PN_GLOBAL int32_t *)row)[at < a.max_pages ? at : a.max_pages - 1];
        };
        // Start the loads of step i; without a branch, or a join of branches
        // would wait for them.  A page that is none of the cache reads page 0.
        struct Raw {
            uint4 w;
            uint32_t s[2 * R];  // scales of the four tokens that its own belongs to
        };
        auto fetch = [&](Raw &raw, int32_t page, int i) {
            const int o = token_at(i) & (T - 1);
            const int64_t at = (uint32_t)page < (uint32_t)a.c.num_pages ? page : 0;
            const uint8_t *from = a.c.pages + (at * a.c.heads + head) * a.c.chunk;
            raw.w = *(const uint4 *)(from + (uint32_t)(keys ? o * L::kRow + 16 * part
                                                            : L::v_codes(T) + ((o >> 2) * (D / 8) + part) * 16));
            const uint8_t *sc = from + (uint32_t)((keys ? L::k_scales(T) : L::v_scales(T)) + 2 * R * (o & ~3));
            if constexpr (R == 1) {
                const uint2 y = *(const uint2 *)sc;
                raw.s[0] = y.x, raw.s[1] = y.y;
            } else {
#pragma unroll
                for (int z = 0; z < R / 2; ++z) {
                    const uint4 y = *(const uint4 *)(sc + 16 * z);
                    raw.s[4 * z] = y.x, raw.s[4 * z + 1] = y.y, raw.s[4 * z + 2] = y.z, raw.s[4 * z + 3] = y.w;
                }
            }
        };
        // The step's words have come: value scales of tokens that are not there
        // become 0, the others are held against the cap; key scales go to LDS,
        // NaN for those tokens.
        auto look = [&](Raw &raw, int32_t page, int i) {
            if (i >= count) return;
            const int at = token_at(i);
            const bool gone = (uint32_t)page >= (uint32_t)a.c.num_pages || at >= req.len || at >> a.c.shift >= a.max_pages;
            if (keys) {
                if (part == 0 && on) {
                    uint8_t *to = lds + 2 * P::kBuf + i % 3 * P::kScale + 2 * R * token;
                    // its R halves of the four tokens'
                    const uint32_t z = token & 3;
                    if constexpr (R == 1) {
                        const uint32_t w2 = z & 2 ? raw.s[1] : raw.s[0];
                        *(uint16_t *)to = gone ? 0x7e00 : (uint16_t)(z & 1 ? w2 >> 16 : w2);
                    } else {
                        uint32_t s[R / 2];
#pragma unroll
                        for (int y = 0; y < R / 2; ++y) {
                            const uint32_t lo = z & 1 ? raw.s[R / 2 + y] : raw.s[y], hi = z & 1 ? raw.s[3 * R / 2 + y] : raw.s[R + y];
                            s[y] = gone ? 0x7e007e00u : z & 2 ? hi : lo;
                        }
                        if constexpr (R == 2) *(uint32_t *)to = s[0];
                        else *(uint2 *)to = make_uint2(s[0], s[1]);
                    }
                    if (gone) bad[i % 4] = 1;
                }
            } else {
                ushort2_t any = {0, 0};
#pragma unroll
                for (int y = 0; y < 2 * R; ++y) {
                    if (gone) raw.s[y] = 0;
                    else if (at + 3 >= req.len) {  // max_kv may end the keys anywhere
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            if (at + (2 * y + half) / R >= req.len) raw.s[y] &= half ? 0x0000ffffu : 0xffff0000u;
                    }
                    any = __builtin_elementwise_max(any, __builtin_bit_cast(ushort2_t, raw.s[y] & 0x7fff7fffu));
                }
                const uint32_t big = any[0] > any[1] ? any[0] : any[1];
                if (big > cap) atomicMax(&most[i % 3], big);
            }
        };
        // Words into fragments.
        auto unpack = [&](const Raw &raw, int i, float factor) {
            if (i >= count || !on) return;
            half8_t *buf = (half8_t *)(lds + (i & 1) * P::kBuf);
            const uint32_t words[4] = {raw.w.x, raw.w.y, raw.w.z, raw.w.w};
            if (keys) {
                // Words (b, h) in order of a group g of the row; a unit holds two groups' of one block, one group's
                // of two blocks, or two of a group's four blocks.
                half8_t *to = buf + (token >> 4) * 2 * R * 64 + (token & 15) +
                              (R == 1 ? 32 * part : R == 2 ? 16 * part : 16 * (part >> 1) + 4 * 64 * (part & 1));
#pragma unroll
                for (int y = 0; y < 4; ++y) to[R == 1 ? (y & 1) * 64 + (y >> 1) * 16 : y * 64] = codes8(words[y]);
            } else {
                const int vb = part >> 3, group = token >> 5, second = token >> 4 & 1, vg = token >> 2 & 3;
                const half2_t f2 = {(_Float16)factor, (_Float16)factor};
                half2_t e[2][2][4];  // [token pair][odd element][product]
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    half2_t sc;
                    if constexpr (R == 1) {
                        sc = as_half2(raw.s[u]);
                    } else {
                        uint32_t lo = raw.s[R * u], hi = raw.s[R * u + R / 2];
                        if (R == 4 && (vb & 2)) lo = raw.s[R * u + 1], hi = raw.s[R * u + R / 2 + 1];
                        sc = as_half2(__builtin_amdgcn_perm(hi, lo, vb & 1 ? 0x07060302u : 0x05040100u));
                    }
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
        Raw raw;
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
                const half8_t *k = (const half8_t *)(lds + (it & 1) * P::kBuf) + lane, *v = k + P::kFrags * 64;
                const uint8_t *scales = lds + 2 * P::kBuf + it % 3 * P::kScale;
                const bool gone = uniform((int)bad[it % 4]) != 0;
                if constexpr (NT >= 3) {
                    if (active == 3) front_step<D, 3>(w, k, v, scales, gone, a.c2, a.slack, g);
                    else if (active >= 4) front_step<D, 4>(w, k, v, scales, gone, a.c2, a.slack, g);
                }
                if constexpr (NT >= 2) {
                    if (active == 2) front_step<D, 2>(w, k, v, scales, gone, a.c2, a.slack, g);
                }
                if (active == 1) front_step<D, 1>(w, k, v, scales, gone, a.c2, a.slack, g);
            }
            if (f != 1.0f) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int y = 0; y < R; ++y)
#pragma unroll
                        for (int i = 0; i < 4; ++i) w.o[n][y][i] *= f;
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

        // The rows' sums: a part, or the whole.
        const float down = 1.0f / up;
        const int64_t part_at = 2 * (int64_t)blockIdx.x + (item.s0 == 0 ? 1 : 0);
        float4_t *to = (float4_t *)(a.part + part_at * a.f_floats);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int j = wave + kWaves * n, at = 16 * j + r, at_row = tile0 + at, i = at_row / a.group;
            if (at >= rows) continue;
            const int q_head = head * a.group + at_row - i * a.group;
#pragma unroll
            for (int y = 0; y < 4 * R; ++y) {
                const float4_t sum = w.o[n][y >> 2][y & 3] * down;
                if (item.cut) to[(j * 4 * R + y) * 64 + lane] = sum;
                else *front_of<D>(a, req.q0 + i, q_head, y >> 2, y & 3, g) = sum;
            }
            if (g == 0) {
                const float2 ml = make_float2(w.m[n], w.l[n][0]);
                if (item.cut) a.part_ml[part_at * a.f_rows + at] = ml;
                else a.front_ml[(req.q0 + i) * a.q_heads + q_head] = ml;
            }
        }
    }
}

// The launches of a call.
struct Plan {
    Cut front, own;
    bool many;        // kFront's rows are kv4_front's
    bool line;        // the requests' own keys are dealt as a line (kTail), not a workgroup an item (kOwn)
    int tiles;        // kOwn: of a request
    int least;        // kFront: steps of a workgroup at least
    int64_t tile;     // rows of kFront's tiles
    size_t sums, ml, members, items, front_parts, own_parts;  // bytes
    size_t bytes() const { return sums + ml + members + items + front_parts + own_parts; }
};

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

// n spread over as few tiles of up to `most` as hold it: tiles, and the largest.
void spread(int64_t n, int most, int64_t &tiles, int64_t &each)
{
    tiles = (n + most - 1) / most;
    each = (n + tiles - 1) / tiles;
}

#ifndef MANY
#define MANY 9999
#endif
#ifndef LEAST
#define LEAST 4
#endif
Plan plan(const pn_kv4_cache *c, int q_heads, int B, int G, int64_t total_q, int64_t max_q, int64_t max_kv, int64_t max_shared)
{
    Plan p;
    const int group = q_heads / c->heads, most = c->dim == 256 ? 2 : 4;  // row groups of a wave that the registers hold
    int64_t tiles, each;
    // As one request a group, of about as many queries as a group has.
    const int64_t keys = max_shared * c->page_size;
    p.front = cut(c, q_heads, G, (total_q + G - 1) / G, keys, 0, 0);
    const int64_t row_groups = ((total_q + G - 1) / G * group + 15) / 16;
    p.many = row_groups >= MANY;
    if (p.many) {
        p.front.nt = c->dim == 64 ? Front<64>::NT : c->dim == 128 ? Front<128>::NT : Front<256>::NT;
        p.front.rg = kWaves;
        p.front.two = false;
        p.front.workers = device_cus();
        spread(row_groups, p.front.nt * kWaves, tiles, each);
        p.tile = 16 * each;
    } else {
        spread(row_groups, most, tiles, each);
        p.front.nt = (int)each;
        p.front.rg = 1;
        p.front.two = c->dim < 256 && each == 1;
        p.front.workers = device_cus() * (p.front.two ? 2 : 1);
        p.tile = 16 * each;
    }
    p.least = LEAST;
    p.front.whole = false;
    p.front.part = part_bytes(c, p.front);
    p.own = cut(c, q_heads, B, max_q, max_kv, 0, 0);
    spread((max_q * group + 15) / 16, most, tiles, each);
    p.tiles = (int)tiles;
    const int64_t tails = max_kv - keys;
    p.line = p.own.rg > 1 || (tails > 2 * kShare * kStep && B * c->heads * tiles < 2 * device_cus());
    if (!p.line) {
        p.own.nt = (int)each;
        p.own.whole = true;
    }
    p.sums = (size_t)total_q * q_heads * c->dim * sizeof(float);
    p.ml = round16((size_t)total_q * q_heads * sizeof(float2));
    p.members = (size_t)B * sizeof(Member);
    p.items = round16((size_t)(total_q * group / p.tile + G + 1) * c->heads * sizeof(int2));
    p.front_parts = p.front.whole ? 0 : round16(p.front.workers * p.front.part);
    p.own_parts = p.own.whole ? 0 : round16(p.own.workers * p.own.part);
    return p;
}

template <int D> pn_status launch_front(const AttnArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((kv4_front<D>), dim3((unsigned)a.workers), dim3(kThreads), Front<D>::kLds, s, a);
    return hipGetLastError() == hipSuccess ? PN_OK : PN_ELAUNCH;
}

template <int D> bool raise_front()
{
    return hipFuncSetAttribute((const void *)kv4_front<D>, hipFuncAttributeMaxDynamicSharedMemorySize, Front<D>::kLds) == hipSuccess;
}

bool shared_fit(const pn_kv4_cache *c, int q_heads, int B, int G, int64_t total_q, int64_t max_q, int64_t max_kv,
                int64_t max_shared)
{
    const int64_t rows = total_q * (q_heads / c->heads);
    return sizes_fit(c, q_heads, B, total_q, max_q, max_kv) && G <= 65535 && max_shared <= INT32_MAX / 2 / c->page_size &&
           rows <= INT32_MAX / 4 && (max_q * (q_heads / c->heads) / 16 + 1) * B * c->heads <= INT32_MAX;
}

bool raise_shared()
{
    return raise_front<64>() && raise_front<128>() && raise_front<256>() && raise_pass<kFront>() && raise_pass<kTail>() &&
           raise_pass<kOwn>();
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
    return plan(cache, q_heads, B, G, total_q, max_q, max_kv, max_shared).bytes();
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
    if (ws_bytes < p.bytes()) return PN_ESHAPE;
    if (!once_per_device(kAttrKv4Shared, raise_shared)) return PN_ELAUNCH;

    uint8_t *at = (uint8_t *)ws;
    auto take = [&](size_t n) { uint8_t *x = at; at += n; return x; };
    a.front = (float *)take(p.sums);
    a.front_ml = (float2 *)take(p.ml);
    a.members = (Member *)take(p.members);
    a.items = (int2 *)take(p.items);
    uint8_t *front_parts = take(p.front_parts), *own_parts = take(p.own_parts);
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
    a.f_tile = a.f_rows = (int)p.tile;
    a.f_floats = (int)p.tile * cache->dim;
    set_cut(a, cache, p.front, front_parts, p.front_parts);
    a.f_part = a.part;
    a.f_part_ml = a.part_ml;
    a.least = p.least;
    pn_status st;
    if (p.many)
        st = cache->dim == 64 ? launch_front<64>(a, s) : cache->dim == 128 ? launch_front<128>(a, s) : launch_front<256>(a, s);
    else
        st = launch_pass<kFront>(a, p.front, cache->dim, s);
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

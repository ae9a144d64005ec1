// pn_kv4_attn.hip - attention over the paged pn4t cache (pn_kv4_attn), for
// AMD Instinct MI355X (gfx950).
//
//   out = sum_t w_t v_t / sum_t w_t,   w_t = exp2(s_t - m),
//   s_t = scale log2(e) * sum_b dk[t][b] * (sum over block b of q . (n_k - 8))
//
// One pass over the keys with a running maximum m and sum per query row
// (rows: the queries of a request times the query heads that share a
// key-value head).  A wave takes 16 NT rows and steps through 32 tokens at a
// time:
//   S^T = K Q^T   v_mfma_f32_16x16x32_f16, A = 16 tokens, B = 16 rows.  A code
//                 word is one lane's 8 elements of A: the cache keeps a row's
//                 words in the order that gives each lane its words of all
//                 blocks in one load, and every product lies in one block, so
//                 the codes enter as exact small integers and the block's
//                 scale multiplies the fp32 sum.
//   O^T += V^T P  A = 16 elements x 32 tokens, B = P^T.  A score's place after
//                 the first product is already a lane's place of B: tokens
//                 4 g .. 4 g + 3 of both 16-token tiles.  V's codes enter
//                 exactly too; the scale of a token's block multiplies the
//                 weight, and that product is the one rounding to fp16 (half a
//                 step, 2^-11 relative).  Weights are <= 1 and scales may have
//                 any fp16 size, so each wave keeps a power of two that puts
//                 the scales it has met below 2^11: with fp32 sums nothing
//                 overflows, and products down to 2^-25 of the largest keep
//                 full precision.
// A row of A is element 2 i + (r >> 3) of word r & 7 of a block (r = lane &
// 15, product i < 4), so that one product stays in one block; two v_perm-ed
// words give the token pairs.
//
// Keys are cut into chunks over workgroups when the rows alone do not fill
// the device (kv4_merge joins the parts), and inside a workgroup over its
// four waves (KW = 4); with enough rows each wave takes rows of its own
// (KW = 1).  All sums have a fixed order.
#include "pn_kv4.h"
#include "pn_device.h"

using namespace pn;
using namespace pn::host;

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kStep = 32;         // tokens of a step
constexpr float kLowest = -1e30f; // a maximum before any score

struct AttnArgs {
    Kv4 c;
    const uint16_t *q;
    const int32_t *q_start, *kv_len, *table;
    uint16_t *out;
    float *lse;   // [splits][rows of the call], with more than one split
    float *part;  // [splits][rows of the call][dim]
    int64_t ldq, ldo, ld_table, total_q;
    int64_t max_q, max_kv;
    int32_t q_heads, group, B, max_pages, window, sinks, splits, chunk;  // chunk: steps of a split
    float scale2;  // scale * log2(e)
};

// The part of a request that a row tile works on.
struct Work {
    int64_t q0;       // first query row of the request
    int32_t qn;       // queries of the request that are computed
    int32_t first;    // position of query 0
    int32_t len;      // keys
    int32_t sink_steps, lo, steps;  // steps [0, sink_steps), then from lo; steps in all
};

__device__ __forceinline__ Work request(const AttnArgs &a, int b)
{
    Work w;
    int64_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
    q0 = q0 < 0 ? 0 : q0 > a.total_q ? a.total_q : q0;
    q1 = q1 < q0 ? q0 : q1 > a.total_q ? a.total_q : q1;
    const int32_t kv = a.kv_len[b] < 0 ? 0 : a.kv_len[b];
    w.q0 = q0;
    w.first = (int32_t)(kv - (q1 - q0));
    w.qn = (int32_t)(q1 - q0 < a.max_q ? q1 - q0 : a.max_q);
    w.len = kv < a.max_kv ? kv : (int32_t)a.max_kv;
    w.sink_steps = w.lo = w.steps = 0;
    return w;
}

// The steps that queries i0 .. i1 of the request can see.
__device__ __forceinline__ void span(const AttnArgs &a, Work &w, int i0, int i1)
{
    int32_t hi = w.first + i1 + 1;
    hi = hi < 0 ? 0 : hi < w.len ? hi : w.len;
    const int32_t end = (hi + kStep - 1) / kStep;
    w.sink_steps = 0;
    w.lo = 0;
    if (a.window > 0) {
        const int64_t from = (int64_t)w.first + i0 - a.window + 1;
        const int32_t lo = from < 0 ? 0 : from < hi ? (int32_t)(from / kStep) : end;
        const int32_t s = a.sinks < hi ? a.sinks : hi;
        const int32_t ss = (s + kStep - 1) / kStep;
        w.sink_steps = ss < lo ? ss : 0;  // sinks that meet the window are one stretch
        w.lo = ss < lo ? lo : 0;
    }
    w.steps = w.sink_steps + (end > w.lo ? end - w.lo : 0);
}

// The pages of a step's two 16-token tiles (-1: not visible).
struct Tiles {
    int32_t page[2];
};

__device__ __forceinline__ Tiles tiles(const AttnArgs &a, const int32_t *row, int step)
{
    Tiles t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = (step * kStep + 16 * i) >> a.c.shift;
        int32_t p = -1;
        if (at < a.max_pages) p = row[at];
        t.page[i] = uniform((uint32_t)p < (uint32_t)a.c.num_pages ? p : -1);
    }
    return t;
}

// What a lane holds of one step: two tiles' key words, value words and scales.
template <int D> struct Step {
    static constexpr int R = D / 64;
    uint32_t k[2][2 * R];   // [tile][2 b + h]
    uint32_t v[2][R][4];    // [tile][block][token]
    uint32_t ks[2][2 * R];  // fp16 [token 4 g ..][block]
    uint32_t vs[2][2 * R];
};

template <int D>
__device__ __forceinline__ void fetch(Step<D> &s, const AttnArgs &a, const Tiles &t, int step, int head, int lane)
{
    using L = Kv4Layout<D>;
    constexpr int R = L::R;
    const int P = 1 << a.c.shift, r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t page = t.page[i] < 0 ? 0 : t.page[i];
        const uint8_t *base = a.c.pages + ((int64_t)page * a.c.heads + head) * a.c.chunk;
        const int o = (step * kStep + 16 * i) & (P - 1);
        const uint8_t *k = base + (o + r) * L::kRow + g * (8 * R);
        if constexpr (R == 1) {
            const uint2 x = *(const uint2 *)k;
            s.k[i][0] = x.x, s.k[i][1] = x.y;
        } else {
#pragma unroll
            for (int j = 0; j < R / 2; ++j) {
                const uint4 x = *(const uint4 *)(k + 16 * j);
                s.k[i][4 * j] = x.x, s.k[i][4 * j + 1] = x.y, s.k[i][4 * j + 2] = x.z, s.k[i][4 * j + 3] = x.w;
            }
        }
        const uint8_t *v = base + L::v_codes(P) + ((o >> 2) + g) * (16 * L::W) + (r & 7) * 16;
#pragma unroll
        for (int b = 0; b < R; ++b) {
            const uint4 x = *(const uint4 *)(v + 128 * b);
            s.v[i][b][0] = x.x, s.v[i][b][1] = x.y, s.v[i][b][2] = x.z, s.v[i][b][3] = x.w;
        }
        const uint8_t *d = base + L::k_scales(P) + (o + 4 * g) * (2 * R);
        const uint8_t *e = base + L::v_scales(P) + (o + 4 * g) * (2 * R);
        if constexpr (R == 1) {
            const uint2 x = *(const uint2 *)d, y = *(const uint2 *)e;
            s.ks[i][0] = x.x, s.ks[i][1] = x.y;
            s.vs[i][0] = y.x, s.vs[i][1] = y.y;
        } else {
#pragma unroll
            for (int j = 0; j < R / 2; ++j) {
                const uint4 x = *(const uint4 *)(d + 16 * j), y = *(const uint4 *)(e + 16 * j);
                s.ks[i][4 * j] = x.x, s.ks[i][4 * j + 1] = x.y, s.ks[i][4 * j + 2] = x.z, s.ks[i][4 * j + 3] = x.w;
                s.vs[i][4 * j] = y.x, s.vs[i][4 * j + 1] = y.y, s.vs[i][4 * j + 2] = y.z, s.vs[i][4 * j + 3] = y.w;
            }
        }
    }
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

// Half h of token-major scales: token i, block b.
template <int R> __device__ __forceinline__ float scale_of(const uint32_t *s, int i, int b)
{
    const int h = i * R + b;
    return half_bits_to_float((s[h >> 1] >> (16 * (h & 1))) & 0xffffu);
}

// Largest over the four 16-lane groups, in all of them.
__device__ __forceinline__ float group_max(float v)
{
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
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
    half8_t q[NT][2 * R];
    float4_t o[NT][R][4];
    float m[NT], l[NT];
    float up;      // the power of two on the value scales
    uint32_t cap;  // largest scale (fp16 bits) that `up` leaves below 2^15
};

template <int D, int NT, bool MASKED>
__device__ __forceinline__ void advance(State<D, NT> &st, Step<D> &s, const AttnArgs &a, const Tiles &t, int token0,
                                        const int32_t (&pos)[NT], int end, int lane)
{
    constexpr int R = D / 64;
    const int r = lane & 15, g = lane >> 4;

    if (MASKED) {  // scales of unwritten places may be anything
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = t.page[i] < 0 ? 0 : end - (token0 + 16 * i + 4 * g);  // written tokens of the lane's four
#pragma unroll
            for (int h = 0; h < 4 * R; ++h)
                if (h / R >= n) s.vs[i][h >> 1] &= (h & 1) ? 0x0000ffffu : 0xffff0000u;
        }
    }

    // the value scales against the cap
    ushort2_t top = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2 * R; ++h)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2_t, s.vs[i][h] & 0x7fff7fffu));
    uint32_t big = top[0] > top[1] ? top[0] : top[1];
    if (__ballot(big > st.cap)) {
#pragma unroll
        for (int d = 16; d < 64; d <<= 1) {
            const uint32_t o = __shfl_xor(big, d, 64);
            big = o > big ? o : big;
        }
        const int e = (int)(big >> 10) < 30 ? (int)(big >> 10) : 30;  // scales < 2^(e - 14)
        const float up = __builtin_ldexpf(1.0f, 25 - e);
        const float f = up / st.up;  // the first time O is 0
        st.up = up;
        st.cap = e + 5 > 30 ? 0xffffu : (uint32_t)((e + 5) << 10) - 1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < R; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) st.o[n][b][i] *= f;
    }

    // scores
    float4_t sc[NT][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int b = 0; b < R; ++b) {
            const half8_t k0 = codes8(s.k[i][2 * b]), k1 = codes8(s.k[i][2 * b + 1]);
            float d[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = scale_of<R>(s.ks[i], j, b) * a.scale2;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float4_t c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, st.q[n][2 * b], (float4_t){0, 0, 0, 0}, 0, 0, 0);
                c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, st.q[n][2 * b + 1], c, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[n][i][j] = b == 0 ? c[j] * d[j] : __builtin_fmaf(c[j], d[j], sc[n][i][j]);
            }
        }
    }

    uint32_t seen[NT];
    if (MASKED) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            seen[n] = 0;
            const int32_t under = a.window > 0 ? pos[n] - a.window : -1;  // >= INT32_MIN: pos >= -1
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = token0 + 16 * (j >> 2) + 4 * g + (j & 3);
                const bool ok = t.page[j >> 2] >= 0 && key < end && key <= pos[n] && (key > under || key < a.sinks);
                seen[n] |= (uint32_t)ok << j;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (!(seen[n] >> j & 1)) sc[n][j >> 2][j & 3] = -__builtin_inff();
        }
    }

    // weights
    half8_t p[NT][R];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float mx = sc[n][0][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) mx = fmaxf(mx, sc[n][j >> 2][j & 3]);
        mx = group_max(mx);
        if (__ballot(mx > st.m[n])) {
            const float m = fmaxf(st.m[n], mx), f = __builtin_amdgcn_exp2f(st.m[n] - m);
            st.m[n] = m;
            st.l[n] *= f;
#pragma unroll
            for (int b = 0; b < R; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) st.o[n][b][i] *= f;
        }
        float w[8], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = __builtin_amdgcn_exp2f(sc[n][j >> 2][j & 3] - st.m[n]);
            sum += w[j];
        }
        st.l[n] += sum;
#pragma unroll
        for (int b = 0; b < R; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float x = w[j] * (scale_of<R>(s.vs[j >> 2], j & 3, b) * st.up);
                if (MASKED && !(seen[n] >> j & 1)) x = 0.0f;  // the scale may be infinite or NaN
                p[n][b][j] = (_Float16)x;
            }
    }

    // values
    const uint32_t sel = r < 8 ? 0x05040100u : 0x07060302u;  // even (low) or odd (high) elements of a token pair
#pragma unroll
    for (int b = 0; b < R; ++b) {
        half8_t va[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t *w = &s.v[u >> 1][b][2 * (u & 1)];
            half2_t e[4];
            Unpack<1>::run(__builtin_amdgcn_perm(w[1], w[0], sel), e);
#pragma unroll
            for (int i = 0; i < 4; ++i) va[i][2 * u] = e[i][0], va[i][2 * u + 1] = e[i][1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                st.o[n][b][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(va[i], p[n][b], st.o[n][b][i], 0, 0, 0);
    }
}

// Element of the head that row `row` of product i of block b computes.
__device__ __forceinline__ int element(int b, int i, int row) { return 64 * b + 8 * (row & 7) + 2 * i + (row >> 3); }

// Grid: x = split + splits * row tile, y = key-value head, z = request.
template <int D, int NT, int KW>
__global__ __launch_bounds__(kThreads) void kv4_attn(AttnArgs a)
{
    constexpr int R = D / 64;
    constexpr int kRows = 16 * NT;                            // of a wave
    constexpr int kTileRows = kRows * (kWaves / KW);          // of the workgroup
    constexpr int kPad = D + 4;
    __shared__ float buf[KW == 1 ? 1 : kRows * kPad];
    __shared__ float ml[KW == 1 ? 1 : kWaves][KW == 1 ? 1 : kRows][2];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits, head = blockIdx.y, b = blockIdx.z;

    Work w = request(a, b);
    const int row0 = tile * kTileRows + (KW == 1 ? wave * kRows : 0);  // of qn * group
    const int rows = w.qn * a.group;
    if (KW == 1 ? row0 >= rows : tile * kTileRows >= rows) return;  // KW > 1: the whole workgroup
    const int last = (row0 + kRows < rows ? row0 + kRows : rows) - 1;
    const int i0 = row0 / a.group, i1 = last / a.group;
    span(a, w, i0, i1);
    const int e0 = split * a.chunk, e1 = a.splits == 1 ? w.steps : e0 + a.chunk < w.steps ? e0 + a.chunk : w.steps;
    if (split > 0 && e0 >= w.steps) return;  // the merge knows

    State<D, NT> st;
    int32_t pos[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = row0 + 16 * n + r, i = row / a.group;
        const bool live = row < rows;
        pos[n] = live ? w.first + i : -1;
        const uint16_t *q = a.q + (w.q0 + (live ? i : 0)) * a.ldq + (head * a.group + (live ? row - i * a.group : 0)) * D;
#pragma unroll
        for (int x = 0; x < 2 * R; ++x) {
            st.q[n][x] = *(const half8_t *)(q + 32 * x + 8 * g);
            if (!live) st.q[n][x] = (half8_t)(_Float16)0.0f;
        }
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) st.o[n][x][i2] = (float4_t){0, 0, 0, 0};
        st.m[n] = kLowest;
        st.l[n] = 0.0f;
    }
    st.up = 1.0f;
    st.cap = 0;

    const int32_t *row = a.table + b * a.ld_table;
    const int32_t p0 = w.first + i0, p1 = w.first + i1;
    auto place = [&](int e) { return e < w.sink_steps ? e : e - w.sink_steps + w.lo; };
    auto work = [&](Step<D> &s, const Tiles &t, int step) {
        const int token0 = step * kStep;
        const bool whole = t.page[0] >= 0 && t.page[1] >= 0 && token0 + kStep <= w.len && token0 + kStep - 1 <= p0 &&
                           (a.window <= 0 || (int64_t)token0 + a.window > p1 || token0 + kStep <= a.sinks);
        if (whole) advance<D, NT, false>(st, s, a, t, token0, pos, w.len, lane);
        else advance<D, NT, true>(st, s, a, t, token0, pos, w.len, lane);
    };
    int e = e0 + (KW == 1 ? 0 : wave);
    if (e < e1) {
        Tiles t = tiles(a, row, place(e));
        Step<D> s;
        fetch<D>(s, a, t, place(e), head, lane);
        for (;;) {
            const int next = e + KW;
            Tiles tn = t;
            Step<D> sn;
            if (next < e1) {
                tn = tiles(a, row, place(next));
                fetch<D>(sn, a, tn, place(next), head, lane);
            }
            work(s, t, place(e));
            if (next >= e1) break;
            s = sn;
            t = tn;
            e = next;
        }
    }

    const float down = 1.0f / st.up;
    const int64_t call_rows = a.total_q * a.q_heads;
    if constexpr (KW == 1) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float l = group_sum(st.l[n]);
            const int at = row0 + 16 * n + r;
            if (at >= rows) continue;  // no exchange below
            const int i = at / a.group;
            const int64_t q = w.q0 + i;
            const int h = head * a.group + at - i * a.group;
            const float f = l > 0.0f ? down / l : 0.0f;
            if (a.splits > 1) {
                const int64_t to = split * call_rows + q * a.q_heads + h;
                if (g == 0) a.lse[to] = l > 0.0f ? st.m[n] + __builtin_amdgcn_logf(l) : -__builtin_inff();
#pragma unroll
                for (int x = 0; x < R; ++x)
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2)
#pragma unroll
                        for (int j = 0; j < 4; ++j) a.part[to * D + element(x, i2, 4 * g + j)] = st.o[n][x][i2][j] * f;
            } else {
                uint16_t *o = a.out + q * a.ldo + h * D;
#pragma unroll
                for (int x = 0; x < R; ++x)
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            o[element(x, i2, 4 * g + j)] =
                                __builtin_bit_cast(uint16_t, (_Float16)(st.o[n][x][i2][j] * f));
            }
        }
    } else {
        // join the waves: common maximum, then one wave after another adds
        float f[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float l = group_sum(st.l[n]);
            if (g == 0) ml[wave][16 * n + r][0] = st.m[n], ml[wave][16 * n + r][1] = l;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float m = kLowest, l = 0.0f;
            for (int x = 0; x < kWaves; ++x) m = fmaxf(m, ml[x][16 * n + r][0]);
            for (int x = 0; x < kWaves; ++x)
                l += ml[x][16 * n + r][1] * __builtin_amdgcn_exp2f(ml[x][16 * n + r][0] - m);
            f[n] = l > 0.0f ? __builtin_amdgcn_exp2f(st.m[n] - m) * down / l : 0.0f;
            const int at = row0 + 16 * n + r;
            if (wave == 0 && g == 0 && a.splits > 1 && at < rows) {
                const int i = at / a.group;
                const int64_t to = split * call_rows + (w.q0 + i) * a.q_heads + head * a.group + at - i * a.group;
                a.lse[to] = l > 0.0f ? m + __builtin_amdgcn_logf(l) : -__builtin_inff();
            }
        }
        for (int x = 0; x < kWaves; ++x) {
            if (wave == x) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int y = 0; y < R; ++y)
#pragma unroll
                        for (int i2 = 0; i2 < 4; ++i2)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float *to = buf + (16 * n + r) * kPad + element(y, i2, 4 * g + j);
                                const float v = st.o[n][y][i2][j] * f[n];
                                *to = x == 0 ? v : *to + v;
                            }
            }
            __syncthreads();
        }
        const int n = last - row0 + 1;  // live rows
        for (int x = threadIdx.x; x < n * (D / 4); x += kThreads) {
            const int at = row0 + x / (D / 4), c = x % (D / 4) * 4, i = at / a.group;
            const float4_t v = *(const float4_t *)(buf + (at - row0) * kPad + c);
            const int64_t q = w.q0 + i;
            const int h = head * a.group + at - i * a.group;
            if (a.splits > 1) {
                *(float4_t *)(a.part + (split * call_rows + q * a.q_heads + h) * D + c) = v;
            } else {
                uint32_t u[2];
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    u[y] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * y]) |
                           (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * y + 1]) << 16;
                *(uint2 *)(a.out + q * a.ldo + h * D + c) = make_uint2(u[0], u[1]);
            }
        }
    }
}

// Join the splits of each row: one wave a row (query, head).  tile_rows: rows
// of a wave of kv4_attn, whose span says how many splits there are.
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_merge(AttnArgs a, int tile_rows)
{
    const int lane = threadIdx.x & 63, b = blockIdx.z, h = blockIdx.y;
    Work w = request(a, b);
    const int head = h / a.group;
    const int i = blockIdx.x * kWaves + (int)(threadIdx.x >> 6);
    if (i >= w.qn) return;
    const int row = i * a.group + h - head * a.group, rows = w.qn * a.group;
    const int row0 = row / tile_rows * tile_rows, last = (row0 + tile_rows < rows ? row0 + tile_rows : rows) - 1;
    span(a, w, row0 / a.group, last / a.group);
    const int n = (w.steps + a.chunk - 1) / a.chunk;
    const int64_t call_rows = a.total_q * a.q_heads, at = (w.q0 + i) * a.q_heads + h;

    float m = -__builtin_inff();
    for (int s = lane; s < n; s += 64) m = fmaxf(m, a.lse[s * call_rows + at]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    constexpr int kEach = D / 64;
    float o[kEach] = {}, l = 0.0f;
    if (m > -__builtin_inff()) {
        for (int s = 0; s < n; ++s) {
            const float x = __builtin_amdgcn_exp2f(a.lse[s * call_rows + at] - m);
            l += x;
            const float *p = a.part + (s * call_rows + at) * D + lane * kEach;
#pragma unroll
            for (int j = 0; j < kEach; ++j) o[j] = __builtin_fmaf(x, p[j], o[j]);
        }
    }
    const float f = l > 0.0f ? 1.0f / l : 0.0f;
    uint16_t *out = a.out + (w.q0 + i) * a.ldo + (int64_t)h * D + lane * kEach;
#pragma unroll
    for (int j = 0; j < kEach; ++j) out[j] = __builtin_bit_cast(uint16_t, (_Float16)(o[j] * f));
}

// How a call is cut.
struct Cut {
    int nt, kw;        // row tiles of a wave, waves along the keys
    int64_t row_tiles; // of a request
    int splits, chunk;
};

Cut cut(const pn_kv4_cache *c, int q_heads, int B, int64_t max_q, int64_t max_kv, int window, int sinks)
{
    Cut t;
    const int group = q_heads / c->heads;
    const int64_t rows = max_q * group;
    const int most = c->dim == 256 ? 1 : c->dim == 128 ? 2 : 4;  // rows of a wave that its registers hold
    const int64_t per = 16 * most;
    // Rows for four waves each: a wave takes rows of its own.
    t.kw = rows > 2 * per ? 1 : 4;
    t.nt = 1;
    while (t.nt < most && 16 * t.nt < rows) t.nt *= 2;
    const int64_t tile_rows = 16 * t.nt * (kWaves / t.kw);
    t.row_tiles = (rows + tile_rows - 1) / tile_rows;
    int64_t keys = max_kv;
    if (window > 0) {
        const int64_t reach = (int64_t)window + max_q + sinks + 2 * kStep;
        if (reach < keys) keys = reach;
    }
    const int64_t steps = (keys + kStep - 1) / kStep + 1;
    const int64_t groups = t.row_tiles * c->heads * B;
    // Enough workgroups for several on every compute unit; at least 8 steps
    // for a wave, so that its start and the merge stay small beside them.
    int64_t splits = (8 * (int64_t)device_cus() + groups - 1) / groups;
    const int64_t least = 8 * t.kw;
    if (splits > (steps + least - 1) / least) splits = (steps + least - 1) / least;
    if (splits < 1) splits = 1;
    if (splits > 1024) splits = 1024;
    t.chunk = (int)((steps + splits - 1) / splits);
    t.splits = (int)((steps + t.chunk - 1) / t.chunk);
    return t;
}

template <int D, int NT>
void attn_launch(const AttnArgs &a, const Cut &t, hipStream_t s)
{
    const dim3 grid((unsigned)(t.row_tiles * t.splits), (unsigned)a.c.heads, (unsigned)a.B);
    if (t.kw == 4)
        hipLaunchKernelGGL((kv4_attn<D, NT, 4>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((kv4_attn<D, NT, 1>), grid, dim3(kThreads), 0, s, a);
}

template <int D>
pn_status launch(const AttnArgs &a, const Cut &t, hipStream_t s)
{
    if constexpr (D == 64)
        if (t.nt == 4) attn_launch<D, 4>(a, t, s);
    if constexpr (D <= 128)
        if (t.nt == 2) attn_launch<D, 2>(a, t, s);
    if (t.nt == 1) attn_launch<D, 1>(a, t, s);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    if (t.splits > 1) {
        const dim3 grid((unsigned)((a.max_q + kWaves - 1) / kWaves), (unsigned)a.q_heads, (unsigned)a.B);
        hipLaunchKernelGGL((kv4_merge<D>), grid, dim3(kThreads), 0, s, a, 16 * t.nt);
        if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    }
    return PN_OK;
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

size_t split_bytes(const pn_kv4_cache *c, int q_heads, int64_t total_q)
{
    return (size_t)total_q * q_heads * (c->dim + 4) * sizeof(float);
}

}  // namespace

extern "C" size_t pn_kv4_attn_workspace(const pn_kv4_cache *cache, int q_heads, int B, int64_t total_q, int64_t max_q,
                                        int64_t max_kv, int window, int sinks)
{
    Kv4 c;
    if (check_cache(cache, &c) || !sizes_ok(cache, q_heads, B, total_q, max_q, max_kv, sinks) ||
        !sizes_fit(cache, q_heads, B, total_q, max_q < total_q ? max_q : total_q, max_kv))
        return 0;
    if (total_q == 0) return 0;
    const Cut t = cut(cache, q_heads, B, max_q < total_q ? max_q : total_q, max_kv, window, sinks);
    return t.splits > 1 ? t.splits * split_bytes(cache, q_heads, total_q) : 0;
}

extern "C" pn_status pn_kv4_attn(const pn_kv4_cache *cache, const uint16_t *q, int64_t ldq, int q_heads,
                                 const int32_t *q_start, const int32_t *kv_len, const int32_t *table, int64_t ld_table,
                                 int B, int64_t total_q, int64_t max_q, int64_t max_kv, float scale, int window,
                                 int sinks, uint16_t *out, int64_t ldo, void *ws, size_t ws_bytes, void *stream)
{
    AttnArgs a;
    if (const pn_status st = check_cache(cache, &a.c)) return st;
    if (!q || !q_start || !kv_len || !table || !out || (!ws && ws_bytes)) return PN_EINVAL;
    if (!sizes_ok(cache, q_heads, B, total_q, max_q, max_kv, sinks)) return PN_ESHAPE;
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
    if (t.splits > 1) {
        const size_t one = split_bytes(cache, q_heads, total_q);
        if (ws_bytes / one < (size_t)t.splits) {  // as many splits as there is room for
            const int fit = (int)(ws_bytes / one);
            const int64_t steps = (int64_t)t.chunk * t.splits;
            if (fit < 2) {
                t.chunk = (int)steps;
                t.splits = 1;
            } else {
                t.chunk = (int)((steps + fit - 1) / fit);
                t.splits = (int)((steps + t.chunk - 1) / t.chunk);
            }
        }
    }
    if (t.row_tiles * t.splits > INT32_MAX) return PN_EUNSUPPORTED;
    a.q = q;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = table;
    a.out = out;
    a.part = (float *)ws;
    a.lse = (float *)ws + (size_t)t.splits * total_q * q_heads * cache->dim;
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
    a.splits = t.splits;
    a.chunk = t.chunk;
    a.scale2 = scale * 1.4426950408889634f;
    const hipStream_t s = (hipStream_t)stream;
    const pn_status st = cache->dim == 64    ? launch<64>(a, t, s)
                         : cache->dim == 128 ? launch<128>(a, t, s)
                                             : launch<256>(a, t, s);
    if (st == PN_OK) g_last_variant = kVarKv4Attn;
    return st;
}

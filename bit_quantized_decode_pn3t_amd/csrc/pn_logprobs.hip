// pn_logprobs.hip - log probabilities of given tokens, entropy and the most
// probable alternatives of logit rows (pn_logprobs), for AMD Instinct MI355X
// (gfx950).
//
//   z_i = c (x_i - m), m = max x, c = scale log2(e);   S = sum exp2(z_i)
//   ln p_i = ln 2 z_i - ln S,   entropy = ln S - ln 2 / S * sum exp2(z_i) z_i
//
// One pass over the logits.  A wave takes a span of a row and keeps, per lane,
// the maximum so far, S (fp64, so that a row that is all but certain keeps the
// rest of its sum) and the sum of the entropy; and, per wave, the 64 best
// entries, sorted across the lanes.  An entry is tested against the K-th best;
// those that pass are gathered in LDS and sorted in 64 at a time.  Entries are
// ordered by one 64-bit key: the value, then the lower index.  Kernel
// logp_spans leaves a span's sums and K keys in the workspace, logp_join, one
// workgroup a row, joins them and looks the given tokens up.  No order of
// results depends on timing.
#include "pn_device.h"
#include "pn_kv4.h"

using namespace pn;
using namespace pn::host;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTile = 1024;       // entries of a wave's step, 16 a lane
constexpr float kLow = -__builtin_inff();
constexpr float kBig = 0x1.fffffep127f;

// What is left of a span: S and the entropy's sum relative to m.
struct Sums {
    double s;
    float m, e;
};

struct LogpArgs {
    const void *x;
    const int32_t *tokens;
    float *logp, *entropy, *top_logp;
    int32_t *top_ids;
    Sums *sums;      // [row][span]
    uint64_t *best;  // [row][span][K]
    int64_t ld, ld_tok, ld_lp, ld_top, V, rows;
    int32_t n_tok, K, spans, span;
    float scale;
};

// NaN counts as -inf, +inf as the largest finite value.
__device__ __forceinline__ float clean(float v) { return fminf(v == v ? v : kLow, kBig); }

// Larger for what comes first; 0 for nothing.  v is not NaN; -0 is +0.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t i)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (uint64_t)((int32_t)b < 0 ? ~b : b | 0x80000000u) << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float((int32_t)b < 0 ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

__device__ __forceinline__ uint64_t shuffle_xor(uint64_t v, int d)
{
    return (uint64_t)(uint32_t)__shfl_xor((int)(v >> 32), d, 64) << 32 | (uint32_t)__shfl_xor((int)v, d, 64);
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t smaller(uint64_t a, uint64_t b) { return a < b ? a : b; }

// A bitonic sequence of 64 keys into descending order, lane 0 first.
__device__ __forceinline__ uint64_t merge_down(uint64_t v, int lane)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint64_t o = shuffle_xor(v, d);
        v = lane & d ? smaller(v, o) : larger(v, o);
    }
    return v;
}
__device__ __forceinline__ uint64_t sort_down(uint64_t v, int lane)
{
#pragma unroll
    for (int k = 2; k < 64; k <<= 1)
#pragma unroll
        for (int d = k >> 1; d > 0; d >>= 1) {
            const uint64_t o = shuffle_xor(v, d);
            v = ((lane & d) != 0) == ((lane & k) != 0) ? larger(v, o) : smaller(v, o);
        }
    return merge_down(v, lane);
}

// The best 64 keys of a wave, and a buffer of those that may join them.
struct Best {
    uint64_t list;   // this lane's of the sorted list
    uint64_t least;  // the K-th best
    float value;     // its value
    int count;       // in the buffer
    uint64_t *buf;   // 128 keys of LDS, the wave's own

    __device__ __forceinline__ void init(uint64_t *b)
    {
        list = least = 0;
        value = kLow;
        count = 0;
        buf = b;
    }
    // The first `many` of the buffer, 64 at most, into the list.
    __device__ __forceinline__ void take(int many, int K, int lane)
    {
        const uint64_t v = sort_down(lane < many ? buf[lane] : 0, lane);
        const uint64_t back = (uint64_t)(uint32_t)__shfl((int)(v >> 32), 63 - lane, 64) << 32 | (uint32_t)__shfl((int)v, 63 - lane, 64);
        list = merge_down(larger(list, back), lane);
        least = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(list >> 32), K - 1) << 32 |
                (uint32_t)__builtin_amdgcn_readlane((int)list, K - 1);
        value = least ? value_of(least) : kLow;
        const int rest = count - many;
        const uint64_t v2 = lane < rest ? buf[64 + lane] : 0;
        if (lane < rest) buf[lane] = v2;
        count = rest;
    }
    __device__ __forceinline__ void push(uint64_t key, bool ok, int K, int lane)
    {
        const bool in = ok && key > least;
        const uint64_t mask = __ballot(in);
        if (!mask) return;
        const int at = count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
        if (in) buf[at] = key;
        count += __builtin_popcountll(mask);
        if (count >= 64) take(64, K, lane);
    }
    __device__ __forceinline__ void finish(int K, int lane)
    {
        if (count > 0) take(count, K, lane);
    }
};

// A lane's running sums.
struct Running {
    double s;
    float m, e;
    __device__ __forceinline__ void raise(float to, float c2)
    {
        if (to > m) {
            const float f = __builtin_amdgcn_exp2f((m - to) * c2);
            if (f > 0.0f) {  // (nothing so far, or all of it too small: as nothing)
                e = f * (e - (to - m) * c2 * (float)s);
                s *= (double)f;
            } else {
                e = 0.0f;
                s = 0.0;
            }
            m = to;
        }
    }
    // v <= m
    __device__ __forceinline__ void add(float v, float c2)
    {
        const float z = fmaxf((v - m) * c2, -kBig);
        const float w = __builtin_amdgcn_exp2f(z);
        s += (double)w;
        e = __builtin_fmaf(w, z, e);
    }
};

typedef float float4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 half8_a2 __attribute__((ext_vector_type(8), aligned(2)));

// A lane's 16 entries of a tile: vector j (of 4 or 8 entries) starts at
// place(j); entries past `end` are -inf.
template <bool HALF> struct Tile {
    static constexpr int kVec = HALF ? 8 : 4;
    __device__ static constexpr int place(int lane, int e) { return (lane + 64 * (e / kVec)) * kVec + e % kVec; }
    __device__ static __forceinline__ void load(float (&v)[16], const void *row, int64_t at, int64_t end, int lane)
    {
        if (at + kTile <= end) {
            if constexpr (HALF) {
                half8_a2 w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) w[j] = *(const half8_a2 *)((const _Float16 *)row + at + place(lane, 8 * j));
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = (float)w[e / 8][e % 8];
            } else {
                float4_a4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = *(const float4_a4 *)((const float *)row + at + place(lane, 4 * j));
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = w[e / 4][e % 4];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int64_t i = at + place(lane, e);
                v[e] = kLow;
                if (i < end) v[e] = HALF ? (float)((const _Float16 *)row)[i] : ((const float *)row)[i];
            }
        }
    }
};

// The wave's lanes as one, in every lane.
__device__ __forceinline__ Running join_lanes(Running r, float c2)
{
    float m = r.m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    r.raise(m, c2);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        r.s += __shfl_xor(r.s, d, 64);
        r.e += __shfl_xor(r.e, d, 64);
    }
    return r;
}

template <bool HALF>
__global__ __launch_bounds__(kThreads) void logp_spans(LogpArgs a)
{
    __shared__ uint64_t buf[kWaves][128];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t unit = (int64_t)blockIdx.x * kWaves + wave;
    const int64_t row = unit / a.spans;
    const int span = (int)(unit - row * a.spans);
    if (row >= a.rows) return;  // no barrier in this kernel
    const void *x = (const uint8_t *)a.x + row * a.ld * (HALF ? 2 : 4);
    const int64_t lo = (int64_t)span * a.span, hi = lo + a.span < a.V ? lo + a.span : a.V;
    const float c2 = a.scale * 1.4426950408889634f;
    Running r = {0.0, kLow, 0.0f};
    Best best;
    best.init(buf[wave]);
    for (int64_t at = lo; at < hi; at += kTile) {
        float v[16];
        Tile<HALF>::load(v, x, at, hi, lane);
        float top = kLow;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            v[e] = clean(v[e]);
            top = fmaxf(top, v[e]);
        }
        if (top > kLow) {
            r.raise(top, c2);
#pragma unroll
            for (int e = 0; e < 16; ++e) r.add(v[e], c2);
        }
        if (a.K > 0 && __ballot(top > kLow && top >= best.value)) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (__ballot(v[e] > kLow && v[e] >= best.value))
                    best.push(key_of(v[e], (uint32_t)(at + Tile<HALF>::place(lane, e))), v[e] > kLow, a.K, lane);
        }
    }
    r = join_lanes(r, c2);
    if (lane == 0) a.sums[unit] = {r.s, r.m, r.e};
    if (a.K > 0) {
        best.finish(a.K, lane);
        if (lane < a.K) a.best[unit * a.K + lane] = best.list;
    }
}

template <bool HALF>
__global__ __launch_bounds__(kThreads) void logp_join(LogpArgs a)
{
    __shared__ uint64_t buf[kWaves][128];
    __shared__ Sums part[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t row = blockIdx.x;
    const float c2 = a.scale * 1.4426950408889634f;
    Running r = {0.0, kLow, 0.0f};
    for (int i = tid; i < a.spans; i += kThreads) {
        const Sums o = a.sums[row * a.spans + i];
        if (o.m > kLow) {
            Running other = {o.s, o.m, o.e};
            const float m = fmaxf(r.m, o.m);
            r.raise(m, c2);
            other.raise(m, c2);
            r.s += other.s;
            r.e += other.e;
        }
    }
    Best best;
    best.init(buf[wave]);
    if (a.K > 0) {
        const uint64_t *keys = a.best + row * a.spans * a.K;
        const int64_t many = (int64_t)a.spans * a.K;
        for (int64_t i = 64 * wave; i < many; i += kThreads) {
            const uint64_t key = i + lane < many ? keys[i + lane] : 0;
            best.push(key, key != 0, a.K, lane);
        }
        best.finish(a.K, lane);
    }
    r = join_lanes(r, c2);
    if (lane == 0) part[wave] = {r.s, r.m, r.e};
    __syncthreads();
    buf[wave][lane] = best.list;
    r = {0.0, kLow, 0.0f};
    float m = kLow;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, part[w].m);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        Running o = {part[w].s, part[w].m, part[w].e};
        if (o.m > kLow) {
            o.raise(m, c2);
            r.s += o.s;
            r.e += o.e;
        }
    }
    const bool any = m > kLow;
    const double log_s = any ? log(r.s) : 0.0;
    if (tid == 0 && a.entropy) a.entropy[row] = any ? (float)(log_s - 0.6931471805599453 * (double)r.e / r.s) : 0.0f;
    auto logp = [&](float v) {
        return v > kLow ? (float)(((double)v - (double)m) * (double)a.scale - log_s) : kLow;
    };
    for (int j = tid; j < a.n_tok; j += kThreads) {
        const int32_t t = a.tokens[row * a.ld_tok + j];
        float v = kLow;
        if (t >= 0 && t < a.V) {
            const int64_t at = row * a.ld + t;
            v = clean(HALF ? (float)((const _Float16 *)a.x)[at] : ((const float *)a.x)[at]);
        }
        a.logp[row * a.ld_lp + j] = logp(v);
    }
    if (a.K < 1) return;
    __syncthreads();
    if (wave > 0) return;
    uint64_t list = best.list;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) list = merge_down(larger(list, buf[w][63 - lane]), lane);
    if (lane < a.K) {
        a.top_ids[row * a.ld_top + lane] = list ? (int32_t)index_of(list) : -1;
        a.top_logp[row * a.ld_top + lane] = list ? logp(value_of(list)) : kLow;
    }
}

// Entries of a wave's span: enough waves to fill the device where there are
// few rows, long spans (few records to join) where there are many.
int span_of(int64_t rows, int64_t V)
{
    const int64_t waves = (int64_t)device_cus() * 32;
    int64_t span = (rows * V + waves - 1) / waves;
    span = (span + kTile - 1) / kTile * kTile;
    return (int)(span < kTile ? kTile : span > 16 * kTile ? 16 * kTile : span);
}

bool sizes_fit(int64_t rows, int64_t V, int K)
{
    const int64_t spans = (V + kTile - 1) / kTile;
    return rows <= INT32_MAX && V <= INT32_MAX && K <= PN_LOGPROBS_MAX_TOP && rows * spans <= INT32_MAX;
}

}  // namespace

extern "C" size_t pn_logprobs_workspace(int64_t rows, int64_t V, int K)
{
    if (rows < 1 || V < 1 || K < 0 || !sizes_fit(rows, V, K)) return 0;
    const int span = span_of(rows, V);
    const size_t spans = (size_t)((V + span - 1) / span);
    return (size_t)rows * spans * (sizeof(Sums) + (size_t)K * sizeof(uint64_t));
}

extern "C" pn_status pn_logprobs(const void *logits, int row_type, int64_t ld, int64_t rows, int64_t V, float scale,
                                 const int32_t *tokens, int64_t ld_tok, int n_tok, float *logp, int64_t ld_lp,
                                 float *entropy, int K, int32_t *top_ids, float *top_logp, int64_t ld_top, void *ws,
                                 size_t ws_bytes, void *stream)
{
    if (!logits || (row_type != PN_ROWS_F32 && row_type != PN_ROWS_F16)) return PN_EINVAL;
    if ((n_tok > 0 && (!tokens || !logp)) || (K > 0 && (!top_ids || !top_logp)) || (!ws && rows > 0)) return PN_EINVAL;
    if (rows < 0 || V < 1 || n_tok < 0 || K < 0 || ld < V || (n_tok > 0 && (ld_tok < n_tok || ld_lp < n_tok)) ||
        (K > 0 && ld_top < K) || !(scale >= 0x1p-100f && scale <= 0x1p64f))
        return PN_ESHAPE;
    if (!aligned(logits, row_type == PN_ROWS_F16 ? 2 : 4) || !aligned(ws, 8)) return PN_EALIGN;
    const void *words[] = {tokens, logp, entropy, top_ids, top_logp};
    for (const void *p : words)
        if (!aligned(p, 4)) return PN_EALIGN;
    if (!sizes_fit(rows, V, K)) return PN_EUNSUPPORTED;
    if (rows == 0) return PN_OK;
    if (ws_bytes < pn_logprobs_workspace(rows, V, K)) return PN_ESHAPE;
    LogpArgs a;
    a.x = logits;
    a.tokens = tokens;
    a.logp = logp;
    a.entropy = entropy;
    a.top_logp = top_logp;
    a.top_ids = top_ids;
    a.span = span_of(rows, V);
    a.spans = (int)((V + a.span - 1) / a.span);
    a.sums = (Sums *)ws;
    a.best = (uint64_t *)(a.sums + rows * a.spans);
    a.ld = ld;
    a.ld_tok = ld_tok;
    a.ld_lp = ld_lp;
    a.ld_top = ld_top;
    a.V = V;
    a.rows = rows;
    a.n_tok = n_tok;
    a.K = K;
    a.scale = scale;
    const hipStream_t s = (hipStream_t)stream;
    const unsigned blocks = (unsigned)((rows * a.spans + kWaves - 1) / kWaves);
    const bool half = row_type == PN_ROWS_F16;
    if (half) hipLaunchKernelGGL((logp_spans<true>), dim3(blocks), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((logp_spans<false>), dim3(blocks), dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    if (half) hipLaunchKernelGGL((logp_join<true>), dim3((unsigned)rows), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((logp_join<false>), dim3((unsigned)rows), dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    g_last_variant = kVarLogprobs;
    return PN_OK;
}

// pn_logprobs.hip - log probabilities of given tokens, entropy and the most
// probable alternatives of logit rows (pn_logprobs), for AMD Instinct MI355X
// (gfx950).
//
//   z_i = c (x_i - m), m = max x, c = scale log2(e);   S = sum exp2(z_i)
//   ln p_i = ln 2 z_i - ln S,   entropy = ln S - ln 2 / S * sum exp2(z_i) z_i
//
// One pass over the logits.  A lane keeps m, S (fp64, so that a row that is
// all but certain keeps the rest of its sum) and the sum of the entropy.  A
// wave keeps the 64 best entries, sorted across its lanes.
// A step of 1024 entries is tested as a whole against the K-th best; entries
// that pass are gathered in LDS and sorted in, 64 at a time.  The first step
// starts from the K-th largest of the lanes' maxima, so that little more than
// K entries pass.  Entries are ordered by one 64-bit key: the value, then the
// lower index.  No order of results depends on timing.
//
// A workgroup's four waves step through a chunk of a row together (a row's
// whole length where there are rows enough); the next step's loads, past the
// caches, are in flight meanwhile.  Chunks of a row leave their sums and K
// keys in the workspace, and logp_join joins them.
//
// What bounds it: 509 rows of 248320 (505 MB) 93 us, 5.4 TB/s, with vector
// instructions (17.6 an entry) active 74 % of a SIMD's time, and 5.9 for the
// join; one row of 62080 6.3 and 4.4, two launches.
#include <type_traits>

#include "pn_device.h"
#include "pn_kv4.h"

using namespace pn;
using namespace pn::host;

namespace {

constexpr int kTile = 1024;       // entries of a wave's step, 16 a lane
constexpr float kLow = -__builtin_inff();
constexpr float kBig = 0x1.fffffep127f;
constexpr double kLn2 = 0.693147180559945309417;

// What is left of a chunk: S and the entropy's sum relative to m.
struct Sums {
    double s;
    float m, e;
};

struct LogpArgs {
    const void *x;
    const int32_t *tokens;
    float *logp, *entropy, *top_logp;
    int32_t *top_ids;
    Sums *sums;      // [row][chunk]
    uint64_t *best;  // [row][chunk][K]
    int64_t ld, ld_tok, ld_lp, ld_top, V;
    int32_t n_tok, K, chunks, chunk;
    float scale, c;  // c = scale log2(e)
};

// NaN counts as -inf, +inf as the largest finite value.
__device__ __forceinline__ float clean(float v) { return v == v ? (v < kBig ? v : kBig) : kLow; }

// Larger for what comes first; 0 for nothing.  v is not NaN; -0 is +0.
__device__ __forceinline__ uint32_t order_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_at(uint32_t order) { return __uint_as_float((int32_t)order < 0 ? order & 0x7fffffffu : ~order); }
__device__ __forceinline__ uint64_t key_of(float v, uint32_t i) { return (uint64_t)order_of(v) << 32 | (uint32_t)~i; }
__device__ __forceinline__ float value_of(uint64_t key) { return value_at((uint32_t)(key >> 32)); }
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

// The value of lane ^ X: data-parallel moves within 16 lanes, swaps of rows
// and halves beyond them (a shuffle through LDS takes ten times as long).
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int X> __device__ __forceinline__ uint32_t across(uint32_t v, int lane)
{
    if constexpr (X == 1) return dpp<0xb1>(v);        // quad_perm 1 0 3 2
    else if constexpr (X == 2) return dpp<0x4e>(v);   // quad_perm 2 3 0 1
    else if constexpr (X == 3) return dpp<0x1b>(v);   // quad_perm 3 2 1 0
    else if constexpr (X == 7) return dpp<0x141>(v);  // row_half_mirror
    else if constexpr (X == 15) return dpp<0x140>(v); // row_mirror
    else if constexpr (X == 8) return dpp<0x128>(v);  // row_ror 8
    else if constexpr (X == 4) return across<7>(across<3>(v, lane), lane);
    else if constexpr (X == 16) {
        auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return lane & 16 ? s[0] : s[1];
    } else if constexpr (X == 32) {
        auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return lane & 32 ? s[0] : s[1];
    } else if constexpr (X == 31) return across<16>(across<15>(v, lane), lane);
    else return across<32>(across<31>(v, lane), lane);  // 63
}
template <int X> __device__ __forceinline__ uint64_t across(uint64_t v, int lane)
{
    return (uint64_t)across<X>((uint32_t)(v >> 32), lane) << 32 | across<X>((uint32_t)v, lane);
}
template <typename T> __device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }

// Lanes without bit H of lanes that differ in X keep the larger.
template <int X, int H, typename T> __device__ __forceinline__ T exchange(T v, int lane)
{
    const T o = across<X>(v, lane);
    return (v > o) == ((lane & H) == 0) ? v : o;
}
// A bitonic sequence of 2 D keys in descending order.
template <int D, typename T> __device__ __forceinline__ T merge_down(T v, int lane)
{
    v = exchange<D, D>(v, lane);
    if constexpr (D > 1) v = merge_down<D / 2>(v, lane);
    return v;
}
// The wave's 64 in descending order: sorted runs of N meet mirrored.
template <int N = 2, typename T> __device__ __forceinline__ T sort_down(T v, int lane)
{
    v = exchange<N - 1, N / 2>(v, lane);
    if constexpr (N > 2) v = merge_down<N / 4>(v, lane);
    if constexpr (N < 64) v = sort_down<2 * N>(v, lane);
    return v;
}
// The best 64 of two sorted lists.
__device__ __forceinline__ uint64_t best_of(uint64_t a, uint64_t b, int lane)
{
    return merge_down<32>(larger(a, across<63>(b, lane)), lane);
}

// The best 64 keys of a wave, and a buffer of those that may join them.
struct Best {
    uint64_t list;   // this lane's of the sorted list
    uint64_t least;  // the K-th best, 0 as long as there are fewer
    float value;     // what an entry has to reach
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
        list = best_of(list, sort_down(lane < many ? buf[lane] : 0, lane), lane);
        least = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(list >> 32), K - 1) << 32 |
                (uint32_t)__builtin_amdgcn_readlane((int)list, K - 1);
        if (least) value = fmaxf(value, value_of(least));
        const int rest = count - many;
        const uint64_t v = lane < rest ? buf[64 + lane] : 0;
        if (lane < rest) buf[lane] = v;
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

// A lane's running sums; m is -inf as long as there is nothing.
struct Running {
    double s;
    float m, e;
    __device__ __forceinline__ void raise(float to, float c)
    {
        if (to > m) {
            const float d = (m - to) * c, f = __builtin_amdgcn_exp2f(d);
            if (f > 0.0f) {  // (else there is nothing, or all of it is too small)
                e = f * __builtin_fmaf(d, (float)s, e);
                s *= (double)f;
            } else {
                e = 0.0f;
                s = 0.0;
            }
            m = to;
        }
    }
};

typedef float float4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 half8_a2 __attribute__((ext_vector_type(8), aligned(2)));

// A lane's 16 entries of a step, as loaded: entry e is place(lane, e) of the
// step; those at `end` and behind it are -inf.
template <bool HALF> struct Tile {
    static constexpr int kVec = HALF ? 8 : 4;
    using Vec = typename std::conditional<HALF, half8_a2, float4_a4>::type;
    using One = typename std::conditional<HALF, _Float16, float>::type;
    Vec w[16 / kVec];
    __device__ static constexpr int place(int lane, int e) { return (lane + 64 * (e / kVec)) * kVec + e % kVec; }
    __device__ __forceinline__ float at(int e) const { return (float)w[e / kVec][e % kVec]; }
    __device__ __forceinline__ void load(const One *row, int64_t from, int64_t end, int lane)
    {
        if (from + kTile <= end) {
#pragma unroll
            for (int j = 0; j < 16 / kVec; ++j) w[j] = __builtin_nontemporal_load((const Vec *)(row + from + place(lane, kVec * j)));
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int64_t i = from + place(lane, e);
                One v = (One)kLow;
                if (i < end) v = row[i];
                w[e / kVec][e % kVec] = v;
            }
        }
    }
};

// One step into the wave's sums and best.
template <bool HALF>
__device__ __forceinline__ void step(const LogpArgs &a, const Tile<HALF> &tile, int64_t from, Running &r, Best &best, int lane)
{
    float v[16], top = kLow, low = kLow;
    asm("" : "+s"(low));  // the compiler takes the median with a constant -inf for a minimum, which drops NaNs upwards
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        v[e] = __builtin_amdgcn_fmed3f(tile.at(e), low, kBig);  // as clean(): of a NaN the least of the others
        top = fmaxf(top, v[e]);
    }
    if (top > kLow) {
        r.raise(top, a.c);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float z = fmaxf((v[e] - r.m) * a.c, -kBig);  // not -inf, which times 0 is NaN
            const float w = __builtin_amdgcn_exp2f(z);
            r.s += (double)w;
            r.e = __builtin_fmaf(w, z, r.e);
        }
    }
    if (a.K < 1) return;
    if (best.least == 0 && best.count == 0) {  // the first step, or only masked ones so far
        const uint32_t kth = (uint32_t)__builtin_amdgcn_readlane((int)sort_down(order_of(top), lane), a.K - 1);
        best.value = value_at(kth);
    }
    if (!__ballot(top > kLow && top >= best.value)) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const bool in = v[e] > kLow && v[e] >= best.value;
        if (__ballot(in)) best.push(key_of(v[e], (uint32_t)(from + Tile<HALF>::place(lane, e))), in, a.K, lane);
    }
}

// A wave's steps of a row: from `from` on, `stride` apart, the next one's loads in flight.
template <bool HALF>
__device__ __forceinline__ void scan(const LogpArgs &a, const void *x, int64_t from, int64_t stride, int64_t end, Running &r,
                                     Best &best, int lane)
{
    using One = typename Tile<HALF>::One;
    Tile<HALF> now, next;
    if (from < end) now.load((const One *)x, from, end, lane);
    for (; from < end; from += stride) {
        if (from + stride < end) next.load((const One *)x, from + stride, end, lane);
        step<HALF>(a, now, from, r, best, lane);
        now = next;
    }
}

// The wave's lanes as one, in every lane.
__device__ __forceinline__ Running join_lanes(Running r, float c, int lane)
{
    float m = r.m;
    uint64_t s;
#define PN_MAX(X) m = fmaxf(m, __uint_as_float(across<X>(__float_as_uint(m), lane)))
#define PN_ADD(X) s = __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, s) + __builtin_bit_cast(double, across<X>(s, lane)))
    PN_MAX(1); PN_MAX(2); PN_MAX(7); PN_MAX(15); PN_MAX(16); PN_MAX(32);
    r.raise(m, c);
    s = __builtin_bit_cast(uint64_t, r.s);
    PN_ADD(1); PN_ADD(2); PN_ADD(7); PN_ADD(15); PN_ADD(16); PN_ADD(32);
#undef PN_MAX
#undef PN_ADD
    r.e = wave_sum(r.e);
    r.s = __builtin_bit_cast(double, s);
    return r;
}

template <bool HALF> __device__ __forceinline__ float logit(const LogpArgs &a, int64_t row, int32_t token)
{
    if (token < 0 || token >= a.V) return kLow;
    const int64_t at = row * a.ld + token;
    return clean(HALF ? (float)((const _Float16 *)a.x)[at] : ((const float *)a.x)[at]);
}

constexpr int kWaves = 4;

// A workgroup's sums and lists as one: the sums in every thread, the list in
// the first wave.
__device__ __forceinline__ Running join_waves(const LogpArgs &a, Running r, Best &best)
{
    __shared__ uint64_t lists[kWaves / 2][64];
    __shared__ Sums part[kWaves];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    if (a.K > 0) best.finish(a.K, lane);
    r = join_lanes(r, a.c, lane);
    if (lane == 0) part[wave] = {r.s, r.m, r.e};
    if (a.K > 0 && wave >= 2) lists[wave - 2][lane] = best.list;
    __syncthreads();
    if (a.K > 0 && wave < 2) best.list = best_of(best.list, lists[wave][lane], lane);
    r = {0.0, kLow, 0.0f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) r.m = fmaxf(r.m, part[w].m);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        Running o = {part[w].s, part[w].m, part[w].e};
        o.raise(r.m, a.c);
        r.s += o.s;
        r.e += o.e;
    }
    if (a.K > 0) {
        if (wave == 1) lists[1][lane] = best.list;
        __syncthreads();
        if (wave == 0) best.list = best_of(best.list, lists[1][lane], lane);
    }
    return r;
}

// The answers of a row.
template <bool HALF>
__device__ __forceinline__ void answer(const LogpArgs &a, int64_t row, Running r, Best &best)
{
    const int tid = threadIdx.x;
    // the first given token's logit on its way meanwhile
    int32_t token = -1;
    if (tid < a.n_tok) token = a.tokens[row * a.ld_tok + tid];
    float x = logit<HALF>(a, row, token);
    r = join_waves(a, r, best);
    const bool any = r.m > kLow;
    const double log_s = any ? log(r.s) : 0.0;
    if (tid == 0 && a.entropy) a.entropy[row] = any ? (float)(log_s - kLn2 * (double)r.e / r.s) : 0.0f;
    auto logp = [&](float v) { return v > kLow ? (float)(((double)v - (double)r.m) * (double)a.scale - log_s) : kLow; };
    for (int j = tid; j < a.n_tok; j += 64 * kWaves) {
        if (j != tid) x = logit<HALF>(a, row, a.tokens[row * a.ld_tok + j]);
        a.logp[row * a.ld_lp + j] = logp(x);
    }
    if (tid < a.K) {
        a.top_ids[row * a.ld_top + tid] = best.list ? (int32_t)index_of(best.list) : -1;
        a.top_logp[row * a.ld_top + tid] = best.list ? logp(value_of(best.list)) : kLow;
    }
}

// WHOLE: a chunk is a row.
template <bool HALF, bool WHOLE>
__global__ __launch_bounds__(64 * kWaves) void logp_scan(LogpArgs a)
{
    __shared__ uint64_t buf[kWaves][128];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t row = WHOLE ? blockIdx.x : blockIdx.x / (unsigned)a.chunks;
    const int64_t lo = WHOLE ? 0 : (int64_t)(blockIdx.x % (unsigned)a.chunks) * a.chunk;
    const int64_t hi = WHOLE || lo + a.chunk > a.V ? a.V : lo + a.chunk;
    Running r = {0.0, kLow, 0.0f};
    Best best;
    best.init(buf[wave]);
    scan<HALF>(a, (const uint8_t *)a.x + row * a.ld * (HALF ? 2 : 4), lo + wave * kTile, kWaves * kTile, hi, r, best, lane);
    if constexpr (WHOLE) {
        answer<HALF>(a, row, r, best);
    } else {
        r = join_waves(a, r, best);
        if (threadIdx.x == 0) a.sums[blockIdx.x] = {r.s, r.m, r.e};
        if ((int)threadIdx.x < a.K) a.best[(int64_t)blockIdx.x * a.K + threadIdx.x] = best.list;
    }
}

template <bool HALF>
__global__ __launch_bounds__(64 * kWaves) void logp_join(LogpArgs a)
{
    __shared__ uint64_t buf[kWaves][128];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t row = blockIdx.x;
    Running r = {0.0, kLow, 0.0f};
    for (int i = tid; i < a.chunks; i += 64 * kWaves) {
        const Sums p = a.sums[row * a.chunks + i];
        Running o = {p.s, p.m, p.e};
        const float m = fmaxf(r.m, o.m);
        r.raise(m, a.c);
        o.raise(m, a.c);
        r.s += o.s;
        r.e += o.e;
    }
    Best best;
    best.init(buf[wave]);
    if (a.K > 0) {
        const uint64_t *keys = a.best + row * a.chunks * a.K;
        const int64_t many = (int64_t)a.chunks * a.K;
        for (int64_t i = 64 * wave; i < many; i += 64 * kWaves) {
            const uint64_t key = i + lane < many ? keys[i + lane] : 0;
            best.push(key, key != 0, a.K, lane);
        }
    }
    answer<HALF>(a, row, r, best);
}

// Entries of a chunk: four workgroups a compute unit, but at least a step a wave.
// (509 rows of 248320: 98 us; with two of them 117, with eight 108.)
constexpr int64_t kLeast = kWaves * kTile;
int64_t workgroups() { return (int64_t)device_cus() * 4; }
int64_t chunk_of(int64_t rows, int64_t V)
{
    const int64_t chunk = ((rows * V + workgroups() - 1) / workgroups() + kLeast - 1) / kLeast * kLeast;
    return chunk < V ? chunk : V;
}
// At least the chunks of all rows, and growing with rows and V, so that what
// is kept for the largest call serves every smaller one.
size_t most_chunks(int64_t rows, int64_t V)
{
    const int64_t split = rows * ((V + kLeast - 1) / kLeast), dealt = rows + workgroups();
    return (size_t)(split < dealt ? split : dealt);
}

bool sizes_fit(int64_t rows, int64_t V, int K)
{
    const int64_t tiles = (V + kTile - 1) / kTile;
    return rows <= INT32_MAX && V <= INT32_MAX && K <= PN_LOGPROBS_MAX_TOP && rows * tiles <= INT32_MAX;
}

template <bool HALF> pn_status launch(LogpArgs a, int64_t rows, hipStream_t s)
{
    const dim3 threads(64 * kWaves);
    if (a.chunks == 1) {  // a launch holds less than 2^32 threads; further rows go into further ones
        constexpr int64_t kMost = (int64_t)UINT32_MAX / (64 * kWaves);
        for (int64_t r = 0; r < rows; r += kMost) {
            const int64_t n = rows - r < kMost ? rows - r : kMost;
            hipLaunchKernelGGL((logp_scan<HALF, true>), dim3((unsigned)n), threads, 0, s, a);
            if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
            a.x = (const uint8_t *)a.x + kMost * a.ld * (HALF ? 2 : 4);
            if (a.tokens) a.tokens += kMost * a.ld_tok;
            if (a.logp) a.logp += kMost * a.ld_lp;
            if (a.entropy) a.entropy += kMost;
            if (a.top_ids) a.top_ids += kMost * a.ld_top;
            if (a.top_logp) a.top_logp += kMost * a.ld_top;
        }
        return PN_OK;
    }
    const dim3 blocks((unsigned)(rows * a.chunks));  // fewer rows than workgroups()
    hipLaunchKernelGGL((logp_scan<HALF, false>), blocks, threads, 0, s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    hipLaunchKernelGGL((logp_join<HALF>), dim3((unsigned)rows), threads, 0, s, a);
    return hipGetLastError() == hipSuccess ? PN_OK : PN_ELAUNCH;
}

}  // namespace

extern "C" size_t pn_logprobs_workspace(int64_t rows, int64_t V, int K)
{
    if (rows < 1 || V < 1 || K < 0 || !sizes_fit(rows, V, K)) return 0;
    return most_chunks(rows, V) * (sizeof(Sums) + (size_t)K * sizeof(uint64_t));
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
    const size_t need = pn_logprobs_workspace(rows, V, K);
    if (ws_bytes < need) return PN_ESHAPE;
    const Rows inputs[] = {{logits, ld * (row_type == PN_ROWS_F16 ? 2 : 4), V * (row_type == PN_ROWS_F16 ? 2 : 4), rows},
                           {tokens, ld_tok * 4, n_tok * (int64_t)4, rows}};
    const Rows outputs[] = {{logp, ld_lp * 4, n_tok * (int64_t)4, rows},
                            {entropy, 0, rows * 4, 1},
                            {top_ids, ld_top * 4, K * (int64_t)4, rows},
                            {top_logp, ld_top * 4, K * (int64_t)4, rows},
                            {ws, 0, (int64_t)need, 1}};
    for (const Rows &o : outputs) {
        for (const Rows &i : inputs)
            if (overlap(o, i)) return PN_EINVAL;
        for (const Rows *other = outputs; other != &o; ++other)
            if (overlap(o, *other)) return PN_EINVAL;
    }
    LogpArgs a;
    a.x = logits;
    a.tokens = tokens;
    a.logp = logp;
    a.entropy = entropy;
    a.top_logp = top_logp;
    a.top_ids = top_ids;
    a.chunk = (int32_t)chunk_of(rows, V);
    a.chunks = (int32_t)((V + a.chunk - 1) / a.chunk);
    a.sums = (Sums *)ws;
    a.best = (uint64_t *)(a.sums + rows * a.chunks);
    a.ld = ld;
    a.ld_tok = ld_tok;
    a.ld_lp = ld_lp;
    a.ld_top = ld_top;
    a.V = V;
    a.n_tok = n_tok;
    a.K = K;
    a.scale = scale;
    a.c = scale * 1.4426950408889634f;
    const pn_status st = row_type == PN_ROWS_F16 ? launch<true>(a, rows, (hipStream_t)stream) : launch<false>(a, rows, (hipStream_t)stream);
    if (st == PN_OK) g_last_variant = kVarLogprobs;
    return st;
}

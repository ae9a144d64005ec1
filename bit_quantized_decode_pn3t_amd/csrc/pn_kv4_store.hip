// pn_kv4_store.hip - norm and position rotation of query and key heads with
// the quantized store into the paged pn4t cache in the same pass
// (pn_kv4_store), and the exact read-back (pn_kv4_load), for AMD Instinct
// MI355X (gfx950).
//
//   y = x g / sqrt(mean(x^2) + eps);  (a, b) -> (a cos - b sin, a sin + b cos)
//   d = fp16_rne(-w / 8), code = 8 + clamp(rint(y / d), -8, 7) per 64 elements
//
// A lane owns 8 neighbouring elements of a head, one code word: dim / 8 lanes
// hold a head, a wave 512 elements, and a head's sum of squares, a block's
// extreme and a rotation partner are a few lanes away.  A word is packed
// without any exchange.  The angles of a token are the same for all heads:
// the workgroup computes them once (fp64, reduced in revolutions with a
// two-part 1 / 2 pi, so that far positions keep full precision) into LDS.
//
// Keys run in fp64 through the rotation and keys and values are quantized in
// fp64: a code next to a border then does not depend on how a sum was
// grouped, and the cache holds the same bytes as any correct implementation
// of the rule (gfx950 issues fp64 at the fp32 rate, and the pass is bound by
// its bytes: 8192 columns of fp32 in, 6144 of fp16 and 2048 of 4.25 bits
// out).  Queries end in fp16 and run in fp32.
//
// That shape, 128 wide, with 8191 tokens: 110 us, 3.4 TB/s, where a copy
// reaches 5.05.  Vector instructions take half of the time, at four waves a
// SIMD.  The registers are those of the fp64 path (square roots, quotients,
// selections and exchanges), which only the keys need, an eighth of the
// columns: queries, three quarters of them, and values share the kernel and so
// its registers.  Words leave four bytes at a time, 16 bytes apart for values:
// 126 MB are written where the outputs have 110.  Fewer registers spill (five
// waves 126 us, six 135), gains and angles kept in registers cost waves (133),
// and loads of four units ahead gain nothing (111).  One token: 5 us.
#include <math.h>

#include "pn_kv4.h"

using namespace pn;
using namespace pn::host;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnit = 512;  // elements a wave holds
constexpr int64_t kGrid = (int64_t)UINT32_MAX / kThreads;  // workgroups of a launch

struct StoreArgs {
    Kv4 c;
    pn_kv4_store_desc d;
    int32_t q_units, kv_units;  // wave-loads of a token's query and key rows
    int32_t split;              // workgroups a token's units are dealt to
    int32_t tokens;             // tokens of a workgroup
};

// binary64 -> fp16, rounded once (ties to even) by way of binary32 rounded
// to odd.
__device__ __forceinline__ uint16_t half_bits(double d)
{
    const float f = (float)d;
    uint32_t u = __float_as_uint(f);
    const double back = (double)f;
    if (back != d) {
        if (__builtin_fabs(back) > __builtin_fabs(d)) u -= 1u;
        u |= 1u;
    }
    return __builtin_bit_cast(uint16_t, (_Float16)__uint_as_float(u));
}

// 8 elements of a row, converted.
template <bool HALF, typename F>
__device__ __forceinline__ void load8(const void *row, int64_t at, F (&x)[8])
{
    if (HALF) {
        const uint4 w = *(const uint4 *)((const uint16_t *)row + at);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = (F)(float)__builtin_bit_cast(_Float16, (uint16_t)(u[i >> 1] >> (16 * (i & 1))));
    } else {
        const float4 a = *(const float4 *)((const float *)row + at), b = *(const float4 *)((const float *)row + at + 4);
        const float u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (F)u[i];
    }
}

__device__ __forceinline__ float root(float v) { return 1.0f / __builtin_sqrtf(v); }
__device__ __forceinline__ double root(double v) { return 1.0 / __builtin_sqrt(v); }

// Norm and rotation of one head's share of a lane; w = the lane's word.
template <int D, typename F>
__device__ __forceinline__ void norm_turn(F (&x)[8], const float *gain, float eps, const double2 *turn, int rot,
                                          bool pairs, int w)
{
    if (gain) {
        F s = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[i] * x[i];
#pragma unroll
        for (int d = 1; d < D / 8; d <<= 1) s += __shfl_xor(s, d, 64);
        const F r = root(s * (F)(1.0 / D) + (F)eps);
        const float4 a = *(const float4 *)(gain + 8 * w), b = *(const float4 *)(gain + 8 * w + 4);
        const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (F)g[i];
    }
    if (!rot) return;  // the same for every lane
    const bool in = 8 * w < rot;
    if (pairs) {
        if (in) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const double2 t = turn[4 * w + i / 2];
                const F a = x[i], b = x[i + 1], c = (F)t.x, s = (F)t.y;
                x[i] = a * c - b * s;
                x[i + 1] = a * s + b * c;
            }
        }
        return;
    }
    // The partner's word is rot / 16 words away; lanes past the rotated part
    // read their own.
    const int lane = threadIdx.x & 63, apart = rot >> 4;
    const bool first = w < apart;
    const int from = !in ? lane : first ? lane + apart : lane - apart;
    const int base = first ? 8 * w : 8 * (w - apart);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const F p = __shfl(x[i], from, 64);
        if (in) {
            const double2 t = turn[base + i];
            const F c = (F)t.x, s = (F)t.y;
            x[i] = first ? x[i] * c - p * s : p * s + x[i] * c;
        }
    }
}

// The 64-element block of 8 lanes: its scale's bits, and this lane's word.
__device__ __forceinline__ uint32_t quantize(const double (&y)[8], uint16_t &scale)
{
    const int lane = threadIdx.x & 63;
    double top = 0.0;  // the element of largest magnitude, the first of equals
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (__builtin_fabs(y[i]) > __builtin_fabs(top)) top = y[i];
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
        const double o = __shfl_xor(top, d, 64);
        const double a = __builtin_fabs(top), b = __builtin_fabs(o);
        if (b > a || (b == a && (lane & d))) top = o;
    }
    double s = top * -0.125;
    s = s > 65504.0 ? 65504.0 : s < -65504.0 ? -65504.0 : s;
    scale = half_bits(s);
    if ((scale & 0x7fff) == 0) {
        scale = 0;
        return 0x88888888u;
    }
    // y / d as the correctly rounded quotient: a rounded reciprocal and one
    // correction (Markstein), exact where y / d is, so ties go to even.
    const double step = (double)(float)__builtin_bit_cast(_Float16, scale), inv = 1.0 / step;
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        double q = y[j] * inv;
        const double fix = __builtin_fma(__builtin_fma(-q, step, y[j]), inv, q);
        q = __builtin_fabs(q) < 16.0 ? fix : q;  // infinities have no remainder
        double n = __builtin_rint(q);
        n = n > 7.0 ? 7.0 : n < -8.0 ? -8.0 : n;
        const int code = (n == n ? (int)n : 0) + 8;
        word |= (uint32_t)code << (16 * (j & 1) + 4 * (j >> 1));
    }
    return word;
}

template <int D, bool HALF>
__global__ __launch_bounds__(kThreads) void kv4_store(StoreArgs a)
{
    using L = Kv4Layout<D>;
    constexpr int kLanes = D / 8;          // lanes of a head
    constexpr int kHeads = kUnit / D;      // heads of a wave
    __shared__ double2 turn[D / 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int w = lane & (kLanes - 1), sub = lane / kLanes;
    const int part = blockIdx.x % a.split;
    const int64_t t0 = (int64_t)(blockIdx.x / a.split) * a.tokens;
    const int P = 1 << a.c.shift, half_rot = a.d.rot >> 1;
    const int units = a.q_units + 2 * a.kv_units;

    for (int64_t t = t0; t < t0 + a.tokens && t < a.d.T; ++t) {
        const int32_t pos = a.d.positions[t];
        if (pos < 0) continue;  // the same for the whole workgroup
        __syncthreads();        // the last token's angles are read
        for (int i = threadIdx.x; i < half_rot; i += kThreads) {
            // revolutions of pos * inv_freq, kept to 2^-50 of a turn
            const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
            const double x = (double)pos * (double)a.d.inv_freq[i];
            const double r = x * hi;
            const double low = __builtin_fma(x, hi, -r) + x * lo;
            double s, c;
            sincospi(2.0 * ((r - __builtin_rint(r)) + low), &s, &c);
            turn[i] = make_double2(c, s);
        }
        __syncthreads();
        const int64_t slot = a.d.slots ? a.d.slots[t] : -1;
        const bool stored = slot >= 0 && (slot >> a.c.shift) < a.c.num_pages;
        const int64_t page = slot >> a.c.shift;
        const int o = (int)(slot & (P - 1));

        for (int u = part * kWaves + wave; u < units; u += a.split * kWaves) {
            if (u < a.q_units) {
                const int head = u * kHeads + sub;
                const bool live = head < a.d.q_heads;
                float x[8] = {};
                if (live) load8<HALF>(a.d.q, t * a.d.ldq + head * D + 8 * w, x);
                norm_turn<D>(x, a.d.q_gain, a.d.eps, turn, a.d.rot, a.d.pairs != 0, w);
                if (live) {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        h[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i]) |
                               (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i + 1]) << 16;
                    *(uint4 *)(a.d.q_out + t * a.d.ldo + head * D + 8 * w) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                continue;
            }
            if (!stored) continue;
            const bool is_v = u - a.q_units >= a.kv_units;
            const int head = (u - a.q_units - (is_v ? a.kv_units : 0)) * kHeads + sub;
            const bool live = head < a.c.heads;
            double y[8] = {};
            if (live) load8<HALF>(is_v ? a.d.v : a.d.k, t * (is_v ? a.d.ldv : a.d.ldk) + head * D + 8 * w, y);
            if (!is_v) norm_turn<D>(y, a.d.k_gain, a.d.eps, turn, a.d.rot, a.d.pairs != 0, w);
            uint16_t scale;
            const uint32_t word = quantize(y, scale);
            if (live) {
                uint8_t *base = a.c.pages + (page * a.c.heads + head) * a.c.chunk;
                *(uint32_t *)(base + (is_v ? L::v_codes(P) + L::v_word(o, w) : L::k_word(o, w))) = word;
                if ((w & 7) == 0)
                    *(uint16_t *)(base + (is_v ? L::v_scales(P) : L::k_scales(P)) + 2 * (o * L::R + (w >> 3))) = scale;
            }
        }
    }
}

// One word (8 elements) a thread; bound by its stores (8191 tokens, keys and
// values of 1024 elements each: 18 us, 67 MB of fp32, 3.7 TB/s).
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_load(Kv4 c, const int64_t *slots, int64_t words, float *k, float *v)
{
    using L = Kv4Layout<D>;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= words) return;
    const int row = c.heads * L::W;  // words of a token
    const int64_t t = id / row;
    const int at = (int)(id - t * row), head = at / L::W, w = at % L::W;
    const int64_t slot = slots[t], page = slot >> c.shift;
    const int P = 1 << c.shift, o = (int)(slot & (P - 1));
    const bool there = slot >= 0 && page < c.num_pages;
    const uint8_t *base = c.pages + (there ? (page * c.heads + head) * (int64_t)c.chunk : 0);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        float *out = side ? v : k;
        if (!out) continue;
        float x[8] = {};
        if (there) {
            const uint32_t q = *(const uint32_t *)(base + (side ? L::v_codes(P) + L::v_word(o, w) : L::k_word(o, w)));
            const float d = (float)*(const _Float16 *)(base + (side ? L::v_scales(P) : L::k_scales(P)) +
                                                       2 * (o * L::R + (w >> 3)));
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = d * (float)((int)(q >> (16 * (j & 1) + 4 * (j >> 1)) & 15) - 8);
        }
        float4 *to = (float4 *)(out + id * 8);
        to[0] = make_float4(x[0], x[1], x[2], x[3]);
        to[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

template <int D>
void store_launch(const StoreArgs &a, unsigned grid, hipStream_t s)
{
    if (a.d.row_type == PN_ROWS_F16)
        hipLaunchKernelGGL((kv4_store<D, true>), dim3(grid), dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((kv4_store<D, false>), dim3(grid), dim3(kThreads), 0, s, a);
}

}  // namespace

extern "C" size_t pn_kv4_page_bytes(int page_size, int heads, int dim)
{
    if (page_shift(page_size) < 0 || heads < 1 || !dim_ok(dim)) return 0;
    return (size_t)page_size * heads * (dim + dim / 16);
}

extern "C" pn_status pn_kv4_store(const pn_kv4_cache *cache, const pn_kv4_store_desc *d, void *stream)
{
    StoreArgs a;
    if (const pn_status st = check_cache(cache, &a.c)) return st;
    if (!d || !d->positions || (!d->q && !d->k) || !d->k != !d->v || (d->k && !d->slots) || (d->q && !d->q_out) ||
        (d->rot && !d->inv_freq) || (d->row_type != PN_ROWS_F32 && d->row_type != PN_ROWS_F16))
        return PN_EINVAL;
    const int dim = cache->dim;
    const int unit = d->row_type == PN_ROWS_F16 ? 8 : 4;  // elements of 16 bytes
    if (d->T < 0 || d->rot < 0 || d->rot > dim || !(d->eps >= 0.0f)) return PN_ESHAPE;
    if (d->q && (d->q_heads < 1 || d->ldq < (int64_t)d->q_heads * dim || d->ldo < (int64_t)d->q_heads * dim))
        return PN_ESHAPE;
    const int64_t kv_cols = (int64_t)cache->heads * dim;
    if (d->k && (d->ldk < kv_cols || d->ldv < kv_cols)) return PN_ESHAPE;
    if (!aligned(d->q, 16) || !aligned(d->k, 16) || !aligned(d->v, 16) || !aligned(d->q_out, 16) ||
        !aligned(d->q_gain, 16) || !aligned(d->k_gain, 16) || !aligned(d->inv_freq, 4) || !aligned(d->positions, 4) ||
        !aligned(d->slots, 8))
        return PN_EALIGN;
    if ((d->q && (d->ldq % unit || d->ldo % 8)) || (d->k && (d->ldk % unit || d->ldv % unit))) return PN_EALIGN;
    if (d->rot % 16 || (d->q && d->q_heads > 65535)) return PN_EUNSUPPORTED;
    if (d->T == 0) return PN_OK;

    a.d = *d;
    const int heads = kUnit / dim;
    a.q_units = d->q ? (d->q_heads + heads - 1) / heads : 0;
    a.kv_units = d->k ? (cache->heads + heads - 1) / heads : 0;
    const int units = a.q_units + 2 * a.kv_units;
    // Few tokens: a token's units go to several workgroups, so that one token
    // does not wait for one workgroup's rounds.
    const int most = (units + kWaves - 1) / kWaves;
    a.split = 1;
    while (a.split < most && d->T * a.split < 2 * device_cus()) a.split *= 2;
    if (a.split > most) a.split = most;
    // A launch holds less than 2^32 threads: past 2^24 tokens a workgroup takes several.
    const int64_t tokens = d->T > kGrid ? (d->T + kGrid - 1) / kGrid : 1;
    if (tokens > INT32_MAX) return PN_EUNSUPPORTED;
    a.tokens = (int32_t)tokens;
    const unsigned grid = (unsigned)((d->T + tokens - 1) / tokens * a.split);
    const hipStream_t s = (hipStream_t)stream;
    if (dim == 64) store_launch<64>(a, grid, s);
    else if (dim == 128) store_launch<128>(a, grid, s);
    else store_launch<256>(a, grid, s);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    g_last_variant = kVarKv4Store;
    return PN_OK;
}

extern "C" pn_status pn_kv4_load(const pn_kv4_cache *cache, const int64_t *slots, int64_t T, float *k, float *v,
                                 void *stream)
{
    Kv4 c;
    if (const pn_status st = check_cache(cache, &c)) return st;
    if (!slots || (!k && !v)) return PN_EINVAL;
    if (T < 0) return PN_ESHAPE;
    if (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return PN_EALIGN;
    if (T == 0) return PN_OK;
    const int64_t per = (int64_t)cache->heads * (cache->dim / 8);
    if (T > kGrid * kThreads / per) return PN_EUNSUPPORTED;
    const int64_t words = T * per;
    const unsigned grid = (unsigned)((words + kThreads - 1) / kThreads);
    const hipStream_t s = (hipStream_t)stream;
    if (cache->dim == 64) hipLaunchKernelGGL((kv4_load<64>), dim3(grid), dim3(kThreads), 0, s, c, slots, words, k, v);
    else if (cache->dim == 128)
        hipLaunchKernelGGL((kv4_load<128>), dim3(grid), dim3(kThreads), 0, s, c, slots, words, k, v);
    else hipLaunchKernelGGL((kv4_load<256>), dim3(grid), dim3(kThreads), 0, s, c, slots, words, k, v);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    g_last_variant = kVarKv4Load;
    return PN_OK;
}
